// loss.cuh -- losses on the logits [M, V] of the output projection: the log-
// probability of each row's target, a paired preference loss and a clipped
// policy loss with a KL term, with the gradient of the logits.
//
// Row m with target y and logits l, tau = logit_scale:
//   logp_m = tau (l_y - r) - ln S,   r = max_v l_v,   S = sum_v exp(tau (l_v - r))
//   d logp_m / d l_v = tau (1[v = y] - p_v),   p_v = exp(tau (l_v - r)) / S
// evaluated in base 2, with c = tau log2 e: ex2(c l - k) with an integer k near
// c r, one fused multiply-add an element; S is then s 2^k.  A row whose s comes
// out as 0, infinite or NaN, or whose k is beyond +-2^20, is done again in the
// careful form above, l - r formed before the product: a row of equal lowest
// values is uniform, -inf entries give exactly 0, and r = 0 stands in where
// nothing is above -inf.  Sums are fp32 per
// thread, warp and block; sums over the tokens of a sequence and over rows are
// fp64 in a fixed order.
//
// Rows start at any element alignment (ld and V are arbitrary): a row is a
// head of elements up to its first 16-byte boundary, 16-byte vectors, and a
// tail.
#pragma once
#include "common.cuh"
#include "tc_gemm.cuh"

namespace qnf4 {
namespace loss {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte load without L1 allocation.  Not the read-only path: with the
// gradient written in place other CTAs write this memory later in the kernel.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Element types: uint16_t holds bf16 bits, float fp32.
template <typename T> struct El;
template <> struct El<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ uint16_t put(float x) { return (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16lo_to_f32(w[j]);
            f[2 * j + 1] = bf16hi_to_f32(w[j]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <> struct El<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// A row's elements before its first 16-byte boundary, its 16-byte vectors, and the rest.
template <typename T>
struct Row {
    int head, tail, nv;
    __device__ __forceinline__ Row(const T* x, int V) {
        constexpr int N = El<T>::N;
        const int h = (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / (int)sizeof(T);
        head = h < V ? h : V;
        nv = (V - head) / N;
        tail = V - head - nv * N;
    }
};

// Running (maximum, sum of ex2((l - maximum) c)) of a set of logits.
struct __align__(8) MS {
    float m, s;
};

__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ MS merge(const MS& a, const MS& b, float c) {
    MS o;
    o.m = fmaxf(a.m, b.m);
    const float r = ref_of(o.m);
    o.s = a.s * ex2((a.m - r) * c) + b.s * ex2((b.m - r) * c);
    return o;
}

template <int N>
__device__ __forceinline__ void add(MS& a, const float (&f)[N], float c) {
    float bm = f[0];
#pragma unroll
    for (int j = 1; j < N; ++j) bm = fmaxf(bm, f[j]);
    if (bm > a.m) {
        a.s *= ex2((a.m - bm) * c);
        a.m = bm;
    }
    const float r = ref_of(a.m);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) (j & 1 ? s1 : s0) += ex2((f[j] - r) * c);
    a.s += s0 + s1;
}

__device__ __forceinline__ void add1(MS& a, float x, float c) {
    const float f[1] = {x};
    add(a, f, c);
}

constexpr int kRowThreads = 512;                 // largest block of the row kernels
constexpr int kMaxZ = 16;                        // CTAs of a cluster that share a row, at most

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t z;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(z));
    return z;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_dsmem_f2(uint32_t addr, float a, float b) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

struct RowShared {
    MS warp[kRowThreads / 32];
    MS rank[kMaxZ];                              // written by the CTAs of the cluster
};

// (maximum, sum) of the whole row, in every thread of every CTA of the
// cluster.  A CTA's pair is pushed into the shared memory of every other
// one; the caller has arrived on the cluster barrier once at its start (so
// that every CTA is known to run) and not waited yet.
__device__ __forceinline__ MS row_total(MS v, float c, RowShared& sh, uint32_t rank, uint32_t z) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        MS o;
        o.m = __shfl_xor_sync(0xffffffffu, v.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, v.s, off);
        v = merge(v, o, c);
    }
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    v = lane < nw ? sh.warp[lane] : MS{-INFINITY, 0.f};
#pragma unroll
    for (int off = kRowThreads / 64; off >= 1; off >>= 1) {
        MS o;
        o.m = __shfl_xor_sync(0xffffffffu, v.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, v.s, off);
        v = merge(v, o, c);
    }
    v.m = __shfl_sync(0xffffffffu, v.m, 0);
    v.s = __shfl_sync(0xffffffffu, v.s, 0);
    if (z == 1) return v;
    cluster_wait();                              // every CTA of the cluster has started
    if (threadIdx.x < z) st_dsmem_f2(mapa(smem_u32(&sh.rank[rank]), threadIdx.x), v.m, v.s);
    cluster_arrive();
    cluster_wait();
    MS t = sh.rank[0];
    for (uint32_t q = 1; q < z; ++q) t = merge(t, sh.rank[q], c);
    return t;
}

// ---------------------------------------------------------------------------
// rows held in registers
// ---------------------------------------------------------------------------
// Sum of 2^(c l) over a set of logits as s 2^k with an integer k, so that
// t = c l - k is one rounding: c l - k in one fused multiply-add, to which the
// rest c_lo of c (c + c_lo is tau log2 e to 48 bits) is added.  Logits beyond
// +-2^100 leave the range that k is clamped to; a row's sum is then 0 or
// infinite, and the row is done again in the careful form above.  So is a row
// whose k is beyond +-kFar: from there on c l is no longer known to a small part
// of 1 (a step of fp32 at 2^20 is 1/8, the 48 bits of c + c_lo end at 2^-28), and
// with it neither k + log2 s nor p.
struct __align__(8) KS {
    float k, s;
};

constexpr float kTop = 0x1p100f, kFar = 0x1p20f;

__device__ __forceinline__ float round_k(float m, float c) { return ceilf(fminf(fmaxf(m * c, -kTop), kTop)); }

typedef unsigned long long f32x2;                // two fp32 in an aligned register pair

__device__ __forceinline__ f32x2 pk2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un2(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The pairs of elements of a 16-byte vector.
template <typename T> struct Pairs;
template <> struct Pairs<uint16_t> {
    static constexpr int N = 4;
    static constexpr uint32_t kNegInf = 0xff80ff80u;
    static __device__ __forceinline__ f32x2 get(const uint4& v, int j) {
        const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
        return pk2(bf16lo_to_f32(w), bf16hi_to_f32(w));
    }
    static __device__ __forceinline__ float max(const uint4& v) {
        auto b = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(b(v.x), b(v.y)), __hmax2(b(v.z), b(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
};
template <> struct Pairs<float> {
    static constexpr int N = 2;
    static constexpr uint32_t kNegInf = 0xff800000u;
    static __device__ __forceinline__ f32x2 get(const uint4& v, int j) {
        return j == 0 ? pk2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : pk2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ float max(const uint4& v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Adds up the lanes' (k, s) pairs.
__device__ __forceinline__ KS warp_total(KS v) {
    KS o;
    o.k = warp_max(v.k);
    o.s = warp_sum_f(v.s * ex2(v.k - o.k));
    return o;
}

struct BlockShared {
    KS warp[kRowThreads / 32];
    KS rank[kMaxZ];                              // written by the CTAs of the cluster
    RowShared careful;
    float4 row;                                  // what warp 0 made of the row
    float at_y;
    unsigned long long xbar;                     // what the cluster's CTAs send
    int abort;
};

// The CTAs of a cluster that share a row tell one another their sums: every
// CTA sends its (k, s) to all of them by asynchronous stores that complete on
// the receiver's barrier.  One warp sends and waits; the block learns of it at
// its next barrier.  (A cluster barrier of all threads in its place took ~1 us
// more per row.)
__device__ __forceinline__ void exchange_init(BlockShared& sh) {
    if (threadIdx.x == 0) {
        sh.abort = 0;
        tc::mbar_init(smem_u32(&sh.xbar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
}

// Warp 0 of every CTA: (k, s) of all ranks added up.
__device__ __forceinline__ KS exchange(KS v, BlockShared& sh, uint32_t rank, uint32_t z) {
    if (z == 1) return v;
    const int lane = threadIdx.x & 31;
    const uint32_t xb = smem_u32(&sh.xbar);
    if (lane == 0) tc::mbar_expect_tx(xb, z * 8);
    if (lane < (int)z) {
        const unsigned long long ks = (unsigned long long)__float_as_uint(v.s) << 32 | __float_as_uint(v.k);
        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                         mapa(smem_u32(&sh.rank[rank]), lane)),
                     "l"(ks), "r"(mapa(xb, lane))
                     : "memory");
    }
    __syncwarp();
    tc::mbar_wait(xb, 0, &sh.abort);
    return warp_total(lane < (int)z ? sh.rank[lane] : KS{-kTop, 0.f});
}

// The row's (k, s) in warp 0 of every CTA of the cluster (the other warps
// return what they have at once).
__device__ __forceinline__ KS block_total(KS v, BlockShared& sh, uint32_t rank, uint32_t z) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    v = warp_total(v);
    if (lane == 0) sh.warp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) v = exchange(warp_total(lane < nw ? sh.warp[lane] : KS{-kTop, 0.f}), sh, rank, z);
    return v;
}

// The exponentials of a vector, added up.  A thread's sum takes them in groups
// of kSumVecs vectors: one by one, terms below half an ulp of a sum that one
// large term dominates would be lost, all in one direction (131072 fp32 logits of
// standard deviation 5: log-probabilities 4e-7 too high on the mean, 2e-7 in
// groups; 1e-8 with no exponent above 0 besides).
constexpr int kSumVecs = 4;
template <typename T>
__device__ __forceinline__ f32x2 vec_sum(const uint4& v, f32x2 c2, f32x2 l2, f32x2 k2) {
    f32x2 e[Pairs<T>::N];
#pragma unroll
    for (int j = 0; j < Pairs<T>::N; ++j) {
        const f32x2 p = Pairs<T>::get(v, j);
        float t0, t1;
        un2(fma2(p, l2, fma2(p, c2, k2)), t0, t1);
        e[j] = pk2(ex2(t0), ex2(t1));
    }
    return Pairs<T>::N == 4 ? add2(add2(e[0], e[1]), add2(e[2 % Pairs<T>::N], e[3 % Pairs<T>::N])) : add2(e[0], e[1]);
}

// One CTA's part of a row: the sum of its exponentials, and its gradient.
template <typename T, int NV>
__device__ __forceinline__ KS sum_pass(const uint4 (&v)[NV], float x1, float c, float c_lo) {
    float m = x1;
#pragma unroll
    for (int u = 0; u < NV; ++u) m = fmaxf(m, Pairs<T>::max(v[u]));
    KS acc;
    acc.k = round_k(m, c);
    const f32x2 c2 = pk2(c, c), l2 = pk2(c_lo, c_lo), k2 = pk2(-acc.k, -acc.k);
    f32x2 s2 = pk2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < NV; u += kSumVecs) {
        f32x2 g2;
#pragma unroll
        for (int w = 0; w < kSumVecs; ++w)
            if (u + w < NV) {
                const f32x2 e = vec_sum<T>(v[u + w], c2, l2, k2);
                g2 = w == 0 ? e : add2(g2, e);
            }
        s2 = add2(s2, g2);
    }
    float sa, sb;
    un2(s2, sa, sb);
    acc.s = sa + sb + ex2(fmaf(x1, c_lo, fmaf(x1, c, -acc.k)));
    return acc;
}

// An element's exponent in the gradient.  In bf16 c_lo l is left out an element, and put into the
// factor before the exponential once a row for l = k / c, about the row's largest logit
// (grad_factor): what remains is c_lo (l - k / c), below 2^-23 of the exponent c l - k, which is
// lost in a bf16 result.
template <typename T>
__device__ __forceinline__ float grad_exp(float l, float c, float c_lo, float k) {
    const float t = fmaf(l, c, -k);
    return sizeof(T) == 4 ? fmaf(l, c_lo, t) : t;
}

// q of -g p = q ex2(grad_exp), from the row's sum s; c_rel = c_lo / c.
template <typename T>
__device__ __forceinline__ float grad_factor(float g, KS t, float c_rel) {
    const float q = -g / t.s;
    return sizeof(T) == 4 ? q : q * ex2(t.k * c_rel);
}

// -g p = q ex2(c l - k); the target's element is at_y, which the thread that has just written there writes:
// g (1 - p) from the log-probability, off by that one's error, some 1e-7 of g, also where p is almost 1.
template <typename T, int NT, int NV>
__device__ __forceinline__ void grad_pass(uint4 (&v)[NV], float x1, float at_y, T* o, const Row<T>& sp, int v0, int nv,
                                          int e1, int y, float c, float c_lo, float k, float q) {
    constexpr int N = El<T>::N;
    const int tid = threadIdx.x & (NT - 1);
    const f32x2 c2 = pk2(c, c), l2 = pk2(c_lo, c_lo), k2 = pk2(-k, -k), q2 = pk2(q, q);
    uint4* ov = reinterpret_cast<uint4*>(o + sp.head + v0 * N);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        // the vector is unpacked again: its elements are not kept from the first pass
        asm volatile("" : "+r"(v[u].x), "+r"(v[u].y), "+r"(v[u].z), "+r"(v[u].w));
        float f[N];
#pragma unroll
        for (int j = 0; j < Pairs<T>::N; ++j) {
            float t0, t1;
            const f32x2 p = Pairs<T>::get(v[u], j), t = fma2(p, c2, k2);
            un2(sizeof(T) == 4 ? fma2(p, l2, t) : t, t0, t1);
            un2(mul2(pk2(ex2(t0), ex2(t1)), q2), f[2 * j], f[2 * j + 1]);
        }
        if (tid + u * NT < nv) ov[tid + u * NT] = El<T>::pack(f);
    }
    if (e1 >= 0) o[e1] = El<T>::put(q * ex2(grad_exp<T>(x1, c, c_lo, k)));
    const int yv = y - sp.head - v0 * N;                  // the target among this CTA's vectors
    const bool mine = yv >= 0 && yv < nv * N ? ((yv / N) & (NT - 1)) == tid : e1 == y;
    if (mine) o[y] = El<T>::put(at_y);
}

// The careful form of one row, read again from memory (rows with k beyond kFar
// or a sum out of range: rare): this CTA's vectors [v0, v1) and, in rank 0, the head and the tail.
template <typename T>
__device__ __noinline__ MS careful_total(const T* x, int V, int v0, int v1, float c, BlockShared& sh,
                                         uint32_t rank, uint32_t z) {
    const Row<T> sp(x, V);
    MS ms{-INFINITY, 0.f};
    for (int e = sp.head + v0 * El<T>::N + threadIdx.x; e < sp.head + v1 * El<T>::N; e += blockDim.x)
        add1(ms, El<T>::get(x[e]), c);
    if (rank == 0) {
        if (threadIdx.x < sp.head) add1(ms, El<T>::get(x[threadIdx.x]), c);
        if (threadIdx.x < sp.tail) add1(ms, El<T>::get(x[V - 1 - threadIdx.x]), c);
    }
    if (z > 1) cluster_arrive();
    ms = row_total(ms, c, sh.careful, rank, z);
    __syncthreads();
    if (z > 1) {                                          // sh.careful may be written again by the next such row
        cluster_arrive();
        cluster_wait();
    }
    return ms;
}

// Zeroes this CTA's part of a gradient row: 16-byte stores where the row has
// them, which need not be the boundaries of the logits' row.
template <typename T>
__device__ __forceinline__ void zero_row(T* o, int V, int v0, int v1, uint32_t rank) {
    const Row<T> sp(o, V);
    // each rank clears its vectors [v0, v1), and rank 0 the head, the tail and what is left of the vectors
    uint4* ov = reinterpret_cast<uint4*>(o + sp.head);
    const int end = v1 < sp.nv ? v1 : sp.nv;
    for (int i = v0 + threadIdx.x; i < end; i += blockDim.x) ov[i] = make_uint4(0, 0, 0, 0);
    if (rank == 0) {
        if (threadIdx.x < sp.head) o[threadIdx.x] = El<T>::put(0.f);
        if (threadIdx.x < sp.tail) o[V - 1 - threadIdx.x] = El<T>::put(0.f);
        // the output row may have one vector more than the input row that was dealt out
        for (int e = sp.head + sp.nv * El<T>::N - El<T>::N + threadIdx.x; sp.nv > 0 && e < sp.head + sp.nv * El<T>::N;
             e += blockDim.x)
            o[e] = El<T>::put(0.f);
    }
}

// The gradient of a row element by element: in the careful form, and for a
// gradient row whose 16-byte boundaries are not the logits' (q and k as in the
// vector path, whose results these equal bit for bit).
template <typename T>
__device__ __noinline__ void scalar_grad(const T* x, T* o, int V, int y, int v0, int v1, float c, float c_lo, bool careful,
                                         MS ms, float k, float q, float g, float at_y, uint32_t rank) {
    const Row<T> sp(x, V);
    auto put = [&](int e) {
        const float l = El<T>::get(x[e]);
        if (careful) {
            const float p = ex2((l - ref_of(ms.m)) * c) / ms.s;
            o[e] = El<T>::put(e == y ? g - g * p : -g * p);
        } else {
            const float p = ex2(grad_exp<T>(l, c, c_lo, k));
            o[e] = El<T>::put(e == y ? at_y : q * p);
        }
    };
    for (int e = sp.head + v0 * El<T>::N + threadIdx.x; e < sp.head + v1 * El<T>::N; e += blockDim.x) put(e);
    if (rank == 0) {
        if (threadIdx.x < sp.head) put(threadIdx.x);
        if (threadIdx.x < sp.tail) put(V - 1 - threadIdx.x);
    }
}

// ---------------------------------------------------------------------------
// short rows: one warp or one small block each, NV vectors a thread in registers
// ---------------------------------------------------------------------------
// For few vectors a thread, the barriers of a large block and a row's latency
// took most of the time.  Rows of up to 32 x 16 vectors take a warp, without
// any barrier (65536 x 500 bf16: log-probabilities 90 us with 256 threads a row,
// 25 with a warp), rows of up to 128 x 16 a block of 128 threads; as many of
// them are in flight as the registers hold, and the hardware deals them out.
constexpr int kBlockThreads = 128;

struct ShortShared {
    KS warp[kBlockThreads / 32];
    MS careful[kBlockThreads / 32];
};

template <typename T, int NT, int NV>
struct ShortRow {
    const T* x;
    Row<T> sp;
    uint4 v[NV];
    float x1;                                    // the thread's element of the head or the tail, -inf: none
    int e1, id;

    __device__ __forceinline__ ShortRow(const T* x_, int V) : x(x_), sp(x_, V), id(threadIdx.x & (NT - 1)) {
        const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
        e1 = id < sp.head ? id : id >= 8 && id < 8 + sp.tail ? V - sp.tail + id - 8 : -1;
#pragma unroll
        for (int u = 0; u < NV; ++u)
            v[u] = id + NT * u < sp.nv ? ld_v4(xv + id + NT * u)
                                       : make_uint4(Pairs<T>::kNegInf, Pairs<T>::kNegInf, Pairs<T>::kNegInf,
                                                    Pairs<T>::kNegInf);
        x1 = e1 >= 0 ? El<T>::get(x[e1]) : -INFINITY;
    }
    __device__ __forceinline__ KS total(float c, float c_lo, ShortShared& sh) const {
        KS t = warp_total(sum_pass<T, NV>(v, x1, c, c_lo));
        if (NT == 32) return t;
        const int lane = threadIdx.x & 31;
        if (lane == 0) sh.warp[threadIdx.x >> 5] = t;
        __syncthreads();
        return warp_total(lane < NT / 32 ? sh.warp[lane] : KS{-kTop, 0.f});
    }
    // the careful form, from memory
    __device__ __noinline__ static MS careful(const T* x, int V, float c, ShortShared& sh) {
        MS a{-INFINITY, 0.f};
        for (int e = threadIdx.x & (NT - 1); e < V; e += NT) add1(a, El<T>::get(x[e]), c);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            MS o;
            o.m = __shfl_xor_sync(0xffffffffu, a.m, off);
            o.s = __shfl_xor_sync(0xffffffffu, a.s, off);
            a = merge(a, o, c);
        }
        if (NT == 32) return a;
        if ((threadIdx.x & 31) == 0) sh.careful[threadIdx.x >> 5] = a;
        __syncthreads();
        a = sh.careful[0];
        for (int w = 1; w < NT / 32; ++w) a = merge(a, sh.careful[w], c);
        return a;
    }
};

template <typename T, int NT>
__device__ __forceinline__ void zero_short_row(T* o, int V) {
    const int id = threadIdx.x & (NT - 1);
    const Row<T> sp(o, V);
    uint4* ov = reinterpret_cast<uint4*>(o + sp.head);
    for (int i = id; i < sp.nv; i += NT) ov[i] = make_uint4(0, 0, 0, 0);
    if (id < sp.head) o[id] = El<T>::put(0.f);
    if (id < sp.tail) o[V - 1 - id] = El<T>::put(0.f);
}

// ---------------------------------------------------------------------------
// log-probability of the target
// ---------------------------------------------------------------------------
struct RowArgs {
    const void* logits;
    int64_t M, ld;
    int V;
    float tau, c, c_lo;          // c + c_lo = tau log2 e
    const int64_t* targets;
    float* logp;                 // [M]
    float2* stats;               // [M] or null: (k, S), or (r, -S) for a row in the careful form
    double* lpd;                 // [M] the log-probability before its rounding to fp32; null without stats
};

// The hardware exponential is low by 5.0e-8 of its value on the mean over all
// arguments of a binade below 0, and by -3.3e-8 over [0, 1/2] (measured against
// exp2 over every fp32 argument; its largest error is 1.5e-7).  Single rows do
// not show it, but the sum of a sequence's log-probabilities would.  A row's
// exponents are not spread evenly: rows of 600 to 131072 logits of standard
// deviations 0.3 to 8 came out 2.4e-8 to 6.3e-8 too high on the mean, of which
// this, the middle, is taken off; at most 2.3e-8 remain.  (A row that is one term
// may be off by all of it, which is less than that term's own error.)
constexpr double kEx2Low = 4e-8;

// The row's log-probability from its sum, in fp64; not above 0, which the
// rounding of a sum that is one term could make it.
__device__ __forceinline__ double logp_of(float ly, KS t, float c, float c_lo) {
    const double lp = (((double)c + (double)c_lo) * (double)ly - (double)t.k - log2((double)t.s)) *
                          0.69314718055994530942 - kEx2Low;
    return lp > 0. ? 0. : lp;
}
__device__ __forceinline__ double logp_of(float ly, MS t, float tau) {
    const double lp = ((double)ly - (double)ref_of(t.m)) * (double)tau - log((double)t.s);
    return lp > 0. ? 0. : lp;
}

// Whether a row's sum stands; the row is done again in the careful form if not.
__device__ __forceinline__ bool in_range(KS t) { return t.s > 0.f && t.s < INFINITY && fabsf(t.k) <= kFar; }

__device__ __forceinline__ void put_logp(const RowArgs& a, int64_t row, double lp, float2 st) {
    a.logp[row] = (float)lp;
    if (a.stats) {
        a.stats[row] = st;
        a.lpd[row] = lp;
    }
}

template <typename T, int NT, int NV>
__global__ void __launch_bounds__(kBlockThreads) k_token_logprob_short(const RowArgs a) {
    __shared__ ShortShared sh;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = (int64_t)blockIdx.x * (kBlockThreads / NT) + threadIdx.x / NT;
    if (row >= a.M) return;
    const bool first = (threadIdx.x & (NT - 1)) == 0;
    const int64_t y = a.targets[row];
    if (y < 0 || y >= a.V) {
        if (first) put_logp(a, row, 0., make_float2(0.f, 1.f));
        return;
    }
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    const float ly = El<T>::get(x[y]);
    const KS t = ShortRow<T, NT, NV>(x, a.V).total(a.c, a.c_lo, sh);
    if (in_range(t)) {
        if (first) put_logp(a, row, logp_of(ly, t, a.c, a.c_lo), make_float2(t.k, t.s));
    } else {
        const MS ms = ShortRow<T, NT, NV>::careful(x, a.V, a.c, sh);
        if (first) put_logp(a, row, logp_of(ly, ms, a.tau), make_float2(ref_of(ms.m), -ms.s));
    }
}

constexpr int kUnroll = kSumVecs;

// One row per cluster of z CTAs (z = 1 unless there are few rows).  A thread's
// k moves when a logit comes whose exponent is above it, so that all exponents
// are at most 0, where the hardware exponential's mean error is known.  The
// bound is the one read of the logits: 1 GB in 165 us bf16 (6.5 TB/s), 156 us
// fp32 (6.9).  Other CTAs' loads cover a thread's arithmetic; loads a step
// ahead of it cover it better in fp32 (8389 x 32000: 165 -> 159 us) and cost
// bf16, with twice the arithmetic for the registers, 10 % (171 -> 187).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_token_logprob(const RowArgs a) {
    __shared__ BlockShared sh;
    const uint32_t rank = cluster_rank(), z = cluster_size();
    exchange_init(sh);
    if (z > 1) cluster_arrive();
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = blockIdx.x / z;
    const int64_t y = a.targets[row];
    if (y < 0 || y >= a.V) {
        if (rank == 0 && threadIdx.x == 0) put_logp(a, row, 0., make_float2(0.f, 1.f));
        if (z > 1) cluster_wait();
        return;
    }
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    const float ly = El<T>::get(x[y]);
    const Row<T> sp(x, a.V);
    const int per = (sp.nv + (int)z - 1) / (int)z, v0 = rank * per, v1 = v0 + per < sp.nv ? v0 + per : sp.nv;
    const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
    const int bt = blockDim.x, tid = threadIdx.x;
    KS acc{-kTop, 0.f};
    const f32x2 c2 = pk2(a.c, a.c), l2 = pk2(a.c_lo, a.c_lo);
    f32x2 s2 = pk2(0.f, 0.f), k2 = pk2(-acc.k, -acc.k);
    auto add_vec = [&](const uint4* v, int n) {
        float m = Pairs<T>::max(v[0]);
        for (int u = 1; u < n; ++u) m = fmaxf(m, Pairs<T>::max(v[u]));
        if (fmaf(m, a.c, -acc.k) > 0.f) {
            const float k = round_k(m, a.c), f = ex2(acc.k - k);
            s2 = mul2(s2, pk2(f, f));
            acc.k = k;
            k2 = pk2(-k, -k);
        }
        f32x2 g2 = vec_sum<T>(v[0], c2, l2, k2);
        for (int u = 1; u < n; ++u) g2 = add2(g2, vec_sum<T>(v[u], c2, l2, k2));
        s2 = add2(s2, g2);
    };
    int i = v0 + tid;
    auto load = [&](uint4 (&v)[kUnroll]) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = ld_v4(xv + i + u * bt);
        i += kUnroll * bt;
    };
    auto whole = [&] { return i + (kUnroll - 1) * bt < v1; };
    if (sizeof(T) == 4) {
        // fp32: the next vectors are on their way while these are added up
        if (whole()) {
            uint4 v[kUnroll];
            load(v);
            while (whole()) {
                uint4 next[kUnroll];
                load(next);
                add_vec(v, kUnroll);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) v[u] = next[u];
            }
            add_vec(v, kUnroll);
        }
    } else {
        while (whole()) {
            uint4 v[kUnroll];
            load(v);
            add_vec(v, kUnroll);
        }
    }
    for (; i < v1; i += bt) {
        const uint4 v = ld_v4(xv + i);
        add_vec(&v, 1);
    }
    if (rank == 0) {
        const int e = tid < sp.head ? tid : tid >= 8 && tid < 8 + sp.tail ? a.V - sp.tail + tid - 8 : -1;
        if (e >= 0) {
            const float x1 = El<T>::get(x[e]);
            if (fmaf(x1, a.c, -acc.k) > 0.f) {
                const float k = round_k(x1, a.c), f = ex2(acc.k - k);
                s2 = mul2(s2, pk2(f, f));
                acc.k = k;
            }
            s2 = add2(s2, pk2(ex2(fmaf(x1, a.c_lo, fmaf(x1, a.c, -acc.k))), 0.f));
        }
    }
    float sa, sb;
    un2(s2, sa, sb);
    acc.s = sa + sb;
    if (z > 1) cluster_wait();                   // every CTA of the cluster runs
    const KS t = block_total(acc, sh, rank, z);
    if (tid == 0) sh.row.x = in_range(t) ? 1.f : 0.f;
    __syncthreads();
    if (sh.row.x != 0.f) {
        if (rank == 0 && tid == 0) put_logp(a, row, logp_of(ly, t, a.c, a.c_lo), make_float2(t.k, t.s));
    } else {
        const MS ms = careful_total(x, a.V, v0, v1, a.c, sh, rank, z);
        if (rank == 0 && tid == 0) put_logp(a, row, logp_of(ly, ms, a.tau), make_float2(ref_of(ms.m), -ms.s));
    }
}

// ---------------------------------------------------------------------------
// gradient of sum_m d_m logp_m with respect to the logits
// ---------------------------------------------------------------------------
struct GradArgs {
    const void* logits;
    int64_t M, ld;
    int V;
    float tau, c, c_lo, c_rel;   // c_rel = c_lo / c
    const int64_t* targets;
    const double* lpd;           // [M] of k_token_logprob
    const float2* stats;         // [M] of k_token_logprob
    const float* dlogp;          // [M] (not used where the target is outside [0, V))
    void* out;                   // may be the logits themselves (ldo == ld)
    int64_t ldo;
    int chunks;                  // per row
};

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;                     // 16-byte vectors per thread

// One chunk of NT * VECS vectors of row `row` by NT threads: coef() is called
// once by every thread, with the chunk's loads under way, and gives
// d loss / d logp of the row (a row without a target is zeroed without it).
template <typename T, int NT, int VECS, typename Coef>
__device__ __forceinline__ void grad_chunk(const GradArgs& a, int64_t row, int ch, Coef coef) {
    constexpr int N = El<T>::N;
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    T* o = static_cast<T*>(a.out) + row * a.ldo;
    const int64_t y64 = a.targets[row];
    const float2 st = a.stats[row];
    const int y = y64 >= 0 && y64 < a.V ? (int)y64 : -1;
    const int tid = threadIdx.x & (NT - 1);
    constexpr int cv = NT * VECS;
    const bool careful = !(st.y > 0.f);          // (r, -S)
    const bool same = (((uint32_t)reinterpret_cast<uintptr_t>(x) ^ (uint32_t)reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    const Row<T> sp(x, a.V);
    const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
    uint4* ov = reinterpret_cast<uint4*>(o + sp.head);
    const int i0 = ch * cv + tid;
    uint4 v[VECS];
    if (y >= 0 && same) {
#pragma unroll
        for (int u = 0; u < VECS; ++u)
            v[u] = i0 + u * NT < sp.nv ? ld_v4(xv + i0 + u * NT) : make_uint4(0, 0, 0, 0);
    }
    const float g = y >= 0 ? coef() * a.tau : 0.f;
    const float q = grad_factor<T>(g, careful ? KS{0.f, -st.y} : KS{st.x, st.y}, a.c_rel);
    auto one = [&](float l) { return q * ex2(careful ? (l - st.x) * a.c : grad_exp<T>(l, a.c, a.c_lo, st.x)); };
    auto at_y = [&] { return -g * expm1f((float)a.lpd[row]); };
    auto put = [&](int e) {
        const float f = g == 0.f ? 0.f : one(El<T>::get(x[e]));
        o[e] = El<T>::put(g != 0.f && e == y ? at_y() : f);
    };
    if (!same) {
        // the two rows cross 16-byte boundaries at different elements
        const int e1 = (ch + 1) * cv * N < a.V ? (ch + 1) * cv * N : a.V;
        for (int e = ch * cv * N + tid; e < e1; e += NT) put(e);
        return;
    }
    if (ch == 0) {
        const int e = tid < sp.head ? tid : tid >= 8 && tid < 8 + sp.tail ? a.V - sp.tail + tid - 8 : -1;
        if (e >= 0) put(e);
    }
    if (g == 0.f) {                              // padding, or a loss that is flat here
#pragma unroll
        for (int u = 0; u < VECS; ++u)
            if (i0 + u * NT < sp.nv) ov[i0 + u * NT] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int yv = y - sp.head;                  // the target among the vectors
    const int iy = yv >= 0 && yv < sp.nv * N ? yv / N : -1;
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        const int i = i0 + u * NT;
        float f[N];
        El<T>::unpack(v[u], f);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = one(f[j]);
        if (i == iy) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j == (yv & (N - 1))) f[j] = at_y();
        }
        if (i < sp.nv) ov[i] = El<T>::pack(f);
    }
}

// One chunk per CTA, the last rows first: those are what the forward pass has
// left in L2.  HBM: 4096 x 128256 bf16 298 us, 7.0 TB/s of reads and writes.
template <typename T, int VECS>
__global__ void __launch_bounds__(kGradThreads) k_dlogits(const GradArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int row_b = blockIdx.x / (unsigned)a.chunks, ch = blockIdx.x - row_b * a.chunks;
    const int64_t row = a.M - 1 - row_b;
    const float d = a.dlogp[row];
    grad_chunk<T, kGradThreads, VECS>(a, row, ch, [&] { return d; });
}

// The same with a row per warp, for many short rows, whose CTAs' starts took
// most of the time (65536 x 500 bf16: 232 us, 50 by warps; 8192 x 4000: 38, 27).
template <typename T>
__global__ void __launch_bounds__(kGradThreads) k_dlogits_warp(const GradArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = a.M - 1 - ((int64_t)blockIdx.x * (kGradThreads / 32) + (threadIdx.x >> 5));
    if (row < 0) return;
    const float d = a.dlogp[row];
    for (int ch = 0; ch < a.chunks; ++ch) grad_chunk<T, 32, kGradVecs>(a, row, ch, [&] { return d; });
}

// ---------------------------------------------------------------------------
// preference loss over pairs of packed sequences
// ---------------------------------------------------------------------------
struct PairArgs {
    const double* lpd;           // [M]
    const float* ref;            // [M], or null (reference-free)
    const int64_t* targets;
    int64_t M, P;
    int V;
    const int32_t* cu;           // [2 P + 1]
    int kind, average;
    float beta, smooth, margin, grad_scale;
    float* loss;                 // [1]
    float* rewards;              // [2 P]
    float* dlogp;                // [M], or null
};

constexpr int kPairCtas = 8;

struct PairShared {
    double red[32][4];
    double warp_loss[32];
    double rank_loss[kPairCtas];
    float2 d;                                    // gradient of a row of either sequence
    uint32_t is_long[32];
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Rows [s0, s1) and [s1, s2) of pair p.  The boundaries are device data: they
// are clamped, so that no value of theirs leads out of the arrays.
struct PairRows {
    int64_t s0, s1, s2;
    __device__ __forceinline__ PairRows(const PairArgs& a, int64_t p) {
        auto at = [&](int64_t i, int64_t lo) {
            int64_t c = a.cu[i];
            c = c < lo ? lo : c;
            return c < a.M ? c : a.M;
        };
        s0 = at(2 * p, 0);
        s1 = at(2 * p + 1, s0);
        s2 = at(2 * p + 2, s1);
    }
};

// Thread id of n adds its rows to (chosen sum, rejected sum, chosen count, rejected count).
__device__ __forceinline__ void pair_sums(const PairArgs& a, const PairRows& r, int id, int n, double (&t)[4]) {
    t[0] = t[1] = t[2] = t[3] = 0.;
#pragma unroll 4
    for (int64_t i = r.s0 + id; i < r.s2; i += n) {
        const int64_t y = a.targets[i];
        const double lp = a.lpd[i];
        const float rf = a.ref ? a.ref[i] : 0.f;
        if (y >= 0 && y < a.V) {
            const double d = lp - (double)rf;
            if (i < r.s1) { t[0] += d; t[2] += 1.; }
            else { t[1] += d; t[3] += 1.; }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = warp_sum(t[j]);
}

// A pair's loss, its rewards over beta, and the gradient of a row of either sequence.
struct PairTerms {
    double loss, sc, sr;
    float gc, gr;
    __device__ __forceinline__ PairTerms(const PairArgs& a, const double (&t)[4]) {
        const double dc = a.average && t[2] > 0. ? 1. / t[2] : 1., dr = a.average && t[3] > 0. ? 1. / t[3] : 1.;
        sc = t[0] * dc;
        sr = t[1] * dr;
        const double delta = sc - sr, beta = (double)a.beta, eps = (double)a.smooth;
        const double zz = beta * delta - (double)a.margin;
        double g;                                // d loss / d delta
        if (a.kind == QLORA_PREF_SIGMOID) {
            const double e = exp(-fabs(zz)), sp = log1p(e);
            // a side without weight may be infinite (a target of probability 0)
            loss = (eps != 1. ? (1. - eps) * (sp + fmax(-zz, 0.)) : 0.) + (eps != 0. ? eps * (sp + fmax(zz, 0.)) : 0.);
            const double sg = zz >= 0. ? e / (1. + e) : 1. / (1. + e);      // sigmoid(-z)
            g = beta * (eps * (1. - sg) - (1. - eps) * sg);
        } else if (a.kind == QLORA_PREF_HINGE) {
            loss = zz < 1. ? 1. - zz : zz == zz ? 0. : zz;
            g = zz < 1. ? -beta : zz == zz ? 0. : zz;        // NaN stays visible
        } else {
            const double q = delta - 0.5 / beta;
            loss = q * q;
            g = 2. * q;
        }
        const double k = g * (double)a.grad_scale / (double)a.P;
        gc = (float)(k * dc);
        gr = (float)(-k * dr);
    }
    __device__ __forceinline__ void put_rewards(const PairArgs& a, int64_t p) const {
        a.rewards[2 * p] = (float)((double)a.beta * sc);
        a.rewards[2 * p + 1] = (float)((double)a.beta * sr);
    }
};

// One pair by one warp (CTA = false) or by the whole CTA; returns the pair's loss.
template <bool CTA, int NT>
__device__ __forceinline__ double do_pair(const PairArgs& a, int64_t p, PairShared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int id = CTA ? threadIdx.x : lane, n = CTA ? NT : 32;
    const PairRows r(a, p);
    double t[4], loss = 0.;
    pair_sums(a, r, id, n, t);
    if (CTA) {
        if (lane == 0)
            for (int j = 0; j < 4; ++j) sh.red[warp][j] = t[j];
        __syncthreads();
    }
    float gc = 0.f, gr = 0.f;
    if (!CTA || warp == 0) {
        if (CTA)
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = warp_sum(lane < NT / 32 ? sh.red[lane][j] : 0.);
        const PairTerms o(a, t);
        loss = o.loss;
        gc = o.gc;
        gr = o.gr;
        if (lane == 0) {
            o.put_rewards(a, p);
            if (CTA) sh.d = make_float2(gc, gr);
        }
    }
    if (CTA) {
        __syncthreads();
        gc = sh.d.x;
        gr = sh.d.y;
    }
    if (a.dlogp)
        for (int64_t i = r.s0 + id; i < r.s2; i += n) a.dlogp[i] = i < r.s1 ? gc : gr;
    return loss;
}

// One cluster.  CTA c owns the pairs c, c + 8, ...: short ones go to its
// warps, long ones are taken by the whole CTA, so that neither many short nor
// few long pairs wait on one warp; the assignment and so every sum's order is
// fixed.  Rows outside every sequence get gradient 0.  All of it is latency:
// with few pairs, blocks of 256 threads that find room beside the kernel before
// them and take all but the shortest pairs whole (16 pairs of 256 rows: 2 us less
// than blocks of 1024).
constexpr int kPairFew = 32, kPairFewRows = 16384;
template <int NT>
__global__ void __launch_bounds__(NT) k_preference(const PairArgs a) {
    constexpr int kWarpTokens = NT < 1024 ? 128 : 1024;   // longest pair that one warp takes
    __shared__ PairShared sh;
    const uint32_t rank = cluster_rank();
    cluster_arrive();
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    double acc = 0.;
    for (int64_t base = 0; base * kPairCtas + rank < a.P; base += NT) {
        const int64_t mine = (base + tid) * kPairCtas + rank;
        bool lng = false;
        if (mine < a.P) lng = (int64_t)a.cu[2 * mine + 2] - a.cu[2 * mine] > kWarpTokens;
        const uint32_t bits = __ballot_sync(0xffffffffu, lng);
        if (lane == 0) sh.is_long[warp] = bits;
        __syncthreads();
        for (int i = warp; i < NT; i += NT / 32) {
            const int64_t p = (base + i) * kPairCtas + rank;
            if (p >= a.P) break;
            if (!((sh.is_long[i >> 5] >> (i & 31)) & 1u)) acc += do_pair<false, NT>(a, p, sh);
        }
        for (int j = 0; j < NT / 32; ++j)
            for (uint32_t b = sh.is_long[j]; b; b &= b - 1) {
                const int64_t p = (base + 32 * j + __ffs(b) - 1) * kPairCtas + rank;
                acc += do_pair<true, NT>(a, p, sh);      // in warp 0
            }
        __syncthreads();
    }
    if (a.dlogp) {
        int64_t lo = a.cu[0], hi = a.cu[2 * a.P];
        lo = lo < 0 ? 0 : lo < a.M ? lo : a.M;
        hi = hi < lo ? lo : hi < a.M ? hi : a.M;
        for (int64_t i = (int64_t)rank * NT + tid; i < lo + a.M - hi; i += NT * kPairCtas)
            a.dlogp[i < lo ? i : hi + i - lo] = 0.f;
    }
    if (lane == 0) sh.warp_loss[warp] = acc;
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        const double v = warp_sum(lane < NT / 32 ? sh.warp_loss[lane] : 0.);
        if (lane == 0)
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa(smem_u32(&sh.rank_loss[rank]), 0)), "d"(v)
                         : "memory");
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && tid == 0) {
        double v = 0.;
        for (int q = 0; q < kPairCtas; ++q) v += sh.rank_loss[q];
        a.loss[0] = (float)(v / (double)a.P);
    }
}

// Pair losses and gradient of up to kFewRows rows, kFewPairs pairs and kFewBytes
// of logits in one launch.  The first CTA takes the losses and the rewards, a pair a warp; each of the others takes a chunk of a
// row, and adds up the row's pair itself while the chunk is on its way: a few
// hundred values, for which a kernel of its own before this one costs more
// (one pair of 61 x 32000: 16.5 us in three launches, 12 us in two).  With more
// chunks the sums of all of them outweigh the launch (log-probabilities included;
// in two launches and in three, us): 16 MB 256 x 32000 bf16 17.4 and 18.7, 64 x
// 128256 bf16 16.0 and 17.9, 512 x 8000 fp32 14.5 and 14.4; 33 MB 512 x 32000 bf16
// 30.3 and 27.9, 64 x 128256 fp32 23.1 and 20.0; 512 x 262144 fp32 282 and 253.
constexpr int kFewRows = 512, kFewPairs = 32;
constexpr int64_t kFewBytes = 1 << 24;

struct FewArgs {
    PairArgs p;
    GradArgs g;
};

template <typename T>
__global__ void __launch_bounds__(kGradThreads) k_preference_few(const FewArgs a) {
    __shared__ double red[kGradThreads / 32][4];
    __shared__ float s_d;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0) {
        double acc = 0.;
        for (int64_t p = warp; p < a.p.P; p += kGradThreads / 32) {
            double t[4];
            pair_sums(a.p, PairRows(a.p, p), lane, 32, t);
            const PairTerms o(a.p, t);
            if (lane == 0) o.put_rewards(a.p, p);
            acc += o.loss;
        }
        if (lane == 0) red[warp][0] = acc;
        __syncthreads();
        if (tid == 0) {
            double v = 0.;
            for (int w = 0; w < kGradThreads / 32; ++w) v += red[w][0];
            a.p.loss[0] = (float)(v / (double)a.p.P);
        }
        return;
    }
    const int b = blockIdx.x - 1, row = b / (unsigned)a.g.chunks, ch = b - row * a.g.chunks;
    grad_chunk<T, kGradThreads, kGradVecs>(a.g, row, ch, [&] {
        // sequences that begin at or before the row; the row is in the last of them
        int seq = -1;
        for (int64_t i = 0; i <= 2 * a.p.P; i += kGradThreads)
            seq += __syncthreads_count(i + tid <= 2 * a.p.P && a.p.cu[i + tid] <= row);
        if (seq < 0 || seq >= 2 * a.p.P) return 0.f;
        const PairRows r(a.p, seq >> 1);
        double t[4];
        pair_sums(a.p, r, tid, kGradThreads, t);
        if (lane == 0)
            for (int j = 0; j < 4; ++j) red[warp][j] = t[j];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = warp_sum(lane < kGradThreads / 32 ? red[lane][j] : 0.);
            const PairTerms o(a.p, t);
            if (lane == 0) s_d = seq & 1 ? o.gr : o.gc;
        }
        __syncthreads();
        return s_d;
    });
}

// ---------------------------------------------------------------------------
// clipped policy loss with a KL term
// ---------------------------------------------------------------------------
struct PolicyArgs {
    const void* logits;
    int64_t M, ld;
    int V;
    float tau, c, c_lo, c_rel;   // c + c_lo = tau log2 e, c_rel = c_lo / c
    const int64_t* targets;
    const float* old_logp;       // [M], or null: the ratio is 1 (its gradient stays)
    const float* ref_logp;       // [M], or null: no KL term
    const float* adv;            // [M]
    const float* weight;         // [M]; 0: the row takes no part
    float lo, hi, kl, grad_scale;
    float* logp;                 // [M]
    float4* part;                // [M] weighted (loss, policy, kl, clipped)
    void* out;                   // gradient, or null; may be the logits themselves (ldo == ld)
    int64_t ldo;
};

// A log-probability in base 2, unevaluated sum of two fp32.  The ratio is the
// exponential of a difference of two log-probabilities of about -10, whose
// fp32 rounding alone would be 5e-7 of the gradient of the row.
struct Lp2 {
    float hi, lo;
};

// c l_y + c_lo l_y - k - log2 S, with S = 2^e m, m in [1/2, 1)  and the integers taken off exactly
// (in_range: |k| <= 2^20, so that k + e is a whole number that fp32 holds).
__device__ __forceinline__ Lp2 lp2_of(float ly, KS t, float c, float c_lo) {
    const int b = (int)(__float_as_uint(t.s) >> 23) - 126;        // in_range: not subnormal but for S < 2^-126
    const bool normal = b > -126;
    const float m = normal ? __uint_as_float((__float_as_uint(t.s) & 0x007fffffu) | 0x3f000000u) : t.s;
    const float K = t.k + (normal ? (float)b : 0.f), p = ly * c, s = p - K, v = s - p;
    const float lo = fmaf(ly, c, -p) + ((p - (s - v)) + (-K - v)) + fmaf(ly, c_lo, -log2f(m)) -
                     (float)kEx2Low * kLog2e;
    Lp2 r{s, fabsf(s) < INFINITY ? lo : 0.f};
    if (r.hi + r.lo > 0.f) r = Lp2{0.f, 0.f};
    return r;
}
__device__ __forceinline__ Lp2 lp2_of(double lp) {
    const double d = lp * 1.4426950408889634074;
    const float hi = (float)d;
    return Lp2{hi, fabsf(hi) < INFINITY ? (float)(d - (double)hi) : 0.f};
}

constexpr float kLog2eLo = (float)(1.4426950408889634074 - (double)kLog2e);
constexpr float kLn2Lo = (float)(0.69314718055994530942 - (double)kLn2);

// lp - x in base 2, x a natural log-probability
__device__ __forceinline__ float lp2_minus(Lp2 lp, float x) {
    const float h = x * kLog2e, e = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -h));
    return (lp.hi - h) + (lp.lo - (fabsf(h) < INFINITY ? e : 0.f));
}

// 1 - p = -(e^lp - 1)
__device__ __forceinline__ float lp2_rest(Lp2 lp) { return -expm1f((lp.hi + lp.lo) * kLn2); }

// The row's loss terms (written by the thread that is told to) and d loss /
// d logit scale: what multiplies 1[v = y] - p_v.  Without a coefficient the KL
// term is left out rather than multiplied by 0: it is infinite in fp32 from a
// distance of 88.7 on.  So is the ratio, which an advantage of 0 makes 0.
__device__ __forceinline__ float policy_row(const PolicyArgs& a, int row, Lp2 lp, float A, float w, float old,
                                            float ref, bool put) {
    const float rho = a.old_logp ? exp2f(lp2_minus(lp, old)) : 1.f;
    const float free_ = A == 0.f && rho == INFINITY ? 0.f : rho * A, held = fminf(fmaxf(rho, a.lo), a.hi) * A;
    const bool clipped = held < free_;
    const float d = a.ref_logp ? -lp2_minus(lp, ref) * kLn2 : 0.f, em = expm1f(d);
    if (put) {
        const float pol = -(clipped ? held : free_), kl = em - d;
        const float r = lp.hi * kLn2;
        a.logp[row] = fabsf(r) < INFINITY ? r + (fmaf(lp.hi, kLn2, -r) + fmaf(lp.hi, kLn2Lo, lp.lo * kLn2)) : r;
        a.part[row] = make_float4(w * (a.kl != 0.f ? pol + a.kl * kl : pol), w * pol, w * kl, clipped ? w : 0.f);
    }
    const float dp = clipped ? 0.f : -free_;
    return w * (a.kl != 0.f ? dp - a.kl * em : dp) * a.grad_scale * a.tau;
}

// A row's gradient depends on that row alone, so each row is read once, held
// in registers (NV vectors per thread of a cluster of z blocks), and its
// gradient written: the 2 M V elements that cannot be done without.  Three to
// five blocks of an SM are each at another point of load, two passes and
// store, which hides the barriers and the latency of each; a persistent block
// of 256 threads with the bulk copy of its next row in flight moved less (7456
// x 72000 bf16: 652 us, this one 399; 16777 x 32000: 398 and 375).  1 GB of
// logits: bf16 5.7 TB/s of reads and writes at 32000 (its exponentials, two an
// element, share the time with the memory), fp32 6.6 TB/s, the rate of a copy.
// Left to itself the compiler takes a few registers too many for one block more
// at two widths (600 MB of fp32 logits: 6000 columns 199 us with five blocks an SM,
// 189 with six; 12280 columns 196 with three, 189 with four; bf16, where it takes
// fewer, loses 2 % by being told).
template <typename T, int NV>
constexpr int policy_ctas() {
    return sizeof(T) != 4 ? 0 : NV == 12 ? 6 : NV == 24 ? 4 : 0;      // 0: as the compiler likes
}

template <typename T, int NV>
__global__ void __launch_bounds__(kBlockThreads, policy_ctas<T, NV>()) k_policy_block(const PolicyArgs a) {
    constexpr int NT = kBlockThreads;
    __shared__ BlockShared sh;
    const uint32_t rank = cluster_rank(), z = cluster_size();
    const int tid = threadIdx.x, V = a.V;
    if (z > 1) {
        exchange_init(sh);
        cluster_arrive();
    }
    grid_dep_wait();
    grid_dep_launch();
    const int row = blockIdx.x / z;
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    T* o = static_cast<T*>(a.out) + row * a.ldo;
    const Row<T> sp(x, V);
    const int per = (sp.nv + (int)z - 1) / (int)z, v0 = (int)rank * per, v1 = v0 + per < sp.nv ? v0 + per : sp.nv;
    const int nv = v1 - v0;                               // none where negative
    // a row that takes no part is not read: that costs the others the wait for their target (8192 x 32000
    // bf16 194 -> 199 us) and pays with prompts among the rows (half of them: 166 -> 142)
    const int64_t y64 = a.targets[row];
    const float w = a.weight[row];
    const int y = y64 >= 0 && y64 < V && w != 0.f ? (int)y64 : -1;
    if (y < 0) {
        if (rank == 0 && tid == 0) {
            a.logp[row] = 0.f;
            a.part[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (a.out != nullptr) zero_row(o, V, v0, v1, rank);
        if (z > 1) cluster_wait();
        return;
    }
    const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head) + v0;
    uint4 v[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
        v[u] = tid + NT * u < nv ? ld_v4(xv + tid + NT * u)
                                 : make_uint4(Pairs<T>::kNegInf, Pairs<T>::kNegInf, Pairs<T>::kNegInf,
                                              Pairs<T>::kNegInf);
    const float A = a.adv[row], old = a.old_logp ? a.old_logp[row] : 0.f, ref = a.ref_logp ? a.ref_logp[row] : 0.f;
    const float ly0 = El<T>::get(x[y]);
    // the one element of the head or the tail that this thread holds
    const int e1 = rank != 0 ? -1 : tid < sp.head ? tid
                 : tid >= 8 && tid < 8 + sp.tail ? V - sp.tail + tid - 8 : -1;
    const float x1 = e1 >= 0 ? El<T>::get(x[e1]) : -INFINITY;
    KS t = sum_pass<T, NV>(v, x1, a.c, a.c_lo);
    // in place, another CTA of the cluster writes the target's gradient once it has this one's sum: the
    // logit has arrived when it is handed on here, before that
    const float ly = __shfl_sync(0xffffffffu, ly0, 0);
    if (z > 1) cluster_wait();                            // every CTA of the cluster runs
    t = block_total(t, sh, rank, z);
    if (tid < 32) {
        // the loss of the row and its derivative, by one warp
        const bool fine = in_range(t);
        const Lp2 lp = lp2_of(ly, t, a.c, a.c_lo);
        const float g = fine ? policy_row(a, row, lp, A, w, old, ref, rank == 0 && tid == 0) : 0.f;
        const float at_y = g * lp2_rest(lp);
        if (tid == 0) {
            sh.row = make_float4(t.k, grad_factor<T>(g, t, a.c_rel), g, fine ? 0.f : 1.f);
            sh.at_y = at_y;
        }
    }
    __syncthreads();
    const float4 rv = sh.row;
    const float k = rv.x, q = rv.y;
    float g = rv.z;
    const bool careful = rv.w != 0.f;
    MS ms{0.f, 1.f};
    if (careful) {
        // far from 0, out of k's range, NaN, or nothing above -inf
        ms = careful_total(x, V, v0, v1, a.c, sh, rank, z);
        g = policy_row(a, row, lp2_of(logp_of(ly, ms, a.tau)), A, w, old, ref, rank == 0 && tid == 0);
    }
    if (a.out == nullptr) return;
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    if (g == 0.f) {                                       // a loss that is flat here
        zero_row(o, V, v0, v1, rank);
    } else if (careful || !same) {
        scalar_grad(x, o, V, y, v0, v1, a.c, a.c_lo, careful, ms, k, q, g, sh.at_y, rank);
    } else {
        grad_pass<T, NT, NV>(v, x1, sh.at_y, o, sp, v0, nv, e1, y, a.c, a.c_lo, k, q);
    }
}

// The same for short rows, a warp each; with 16 vectors a lane five blocks an SM
// instead of four (75000 x 4000 bf16: 243 -> 225 us, 75000 x 2000 fp32 205 -> 201).
template <typename T, int NT, int NV>
__global__ void __launch_bounds__(kBlockThreads, NV == 16 ? 5 : 0) k_policy_short(const PolicyArgs a) {
    __shared__ ShortShared sh;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = (int64_t)blockIdx.x * (kBlockThreads / NT) + threadIdx.x / NT;
    if (row >= a.M) return;
    const int id = threadIdx.x & (NT - 1), V = a.V;
    const T* x = static_cast<const T*>(a.logits) + row * a.ld;
    T* o = static_cast<T*>(a.out) + row * a.ldo;
    const int64_t y64 = a.targets[row];
    const float w = a.weight[row];
    const int y = y64 >= 0 && y64 < V && w != 0.f ? (int)y64 : -1;
    if (y < 0) {
        if (id == 0) {
            a.logp[row] = 0.f;
            a.part[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (a.out != nullptr) zero_short_row<T, NT>(o, V);
        return;
    }
    const float ly = El<T>::get(x[y]), A = a.adv[row];
    const float old = a.old_logp ? a.old_logp[row] : 0.f, ref = a.ref_logp ? a.ref_logp[row] : 0.f;
    ShortRow<T, NT, NV> r(x, V);
    const KS t = r.total(a.c, a.c_lo, sh);
    const bool careful = !in_range(t);
    MS ms{0.f, 1.f};
    Lp2 lp;
    if (careful) {
        ms = ShortRow<T, NT, NV>::careful(x, V, a.c, sh);
        lp = lp2_of(logp_of(ly, ms, a.tau));
    } else {
        lp = lp2_of(ly, t, a.c, a.c_lo);
    }
    const float g = policy_row(a, (int)row, lp, A, w, old, ref, id == 0);
    if (a.out == nullptr) return;
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    const float k = t.k, q = grad_factor<T>(g, careful ? KS{0.f, ms.s} : t, a.c_rel);
    if (g == 0.f) {
        zero_short_row<T, NT>(o, V);
    } else if (careful || !same) {
        for (int e = id; e < V; e += NT) {
            const float l = El<T>::get(x[e]);
            const float p = ex2(careful ? (l - ref_of(ms.m)) * a.c : grad_exp<T>(l, a.c, a.c_lo, k));
            o[e] = El<T>::put(e == y ? g * lp2_rest(lp) : q * p);
        }
    } else {
        grad_pass<T, NT, NV>(r.v, r.x1, g * lp2_rest(lp), o, r.sp, 0, r.sp.nv, r.e1, y, a.c, a.c_lo, k, q);
    }
}

constexpr int kFinishThreads = 256, kFinishCtas = 8;

struct FinishSums {
    const float4* part;          // [M]
    int64_t M;
    float* stats;                // [4]
};

// stats[j] = sum over rows of component j, fp64 in a fixed order, by one
// cluster of blocks small enough to find room beside the kernel before it.
__global__ void __launch_bounds__(kFinishThreads) k_policy_finish(const FinishSums a) {
    __shared__ double s[kFinishThreads / 32][4], total[kFinishCtas][4];
    const uint32_t rank = cluster_rank(), z = cluster_size();
    if (z > 1) cluster_arrive();
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    double t[4] = {0., 0., 0., 0.};
#pragma unroll 4
    for (int64_t i = rank * kFinishThreads + tid; i < a.M; i += z * kFinishThreads) {
        const float4 p = a.part[i];
        t[0] += p.x; t[1] += p.y; t[2] += p.z; t[3] += p.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        t[j] = warp_sum(t[j]);
        if (lane == 0) s[warp][j] = t[j];
    }
    __syncthreads();
    if (z > 1) cluster_wait();                   // every CTA of the cluster runs
    if (tid < 4) {
        double v = 0.;
        for (int w = 0; w < kFinishThreads / 32; ++w) v += s[w][tid];
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa(smem_u32(&total[rank][tid]), 0)), "d"(v) : "memory");
    }
    if (z > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    if (rank == 0 && tid < 4) {
        double v = 0.;
        for (uint32_t q = 0; q < z; ++q) v += total[q][tid];
        a.stats[tid] = (float)v;
    }
}

}  // namespace loss
}  // namespace qnf4
