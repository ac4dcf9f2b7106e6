"""The training-step operators around the QLoRA linear layer, as cases to be measured.

Five operators of one fine-tuning step with a frozen 4-bit base:

* ``keep``    an activation stored as an 8-bit checkpoint and restored from it
              (codes of 8 bits, one power-of-two scale per 32 consecutive values of a row);
* ``bwd``     the backward of the frozen-NF4 linear layer reading its input from such a checkpoint;
* ``logprob`` the log-probability of each row's target under the row's logits (what a reference or
              behaviour policy is evaluated for);
* ``pref``    a paired preference loss over packed sequences, from the logits to their gradient;
* ``policy``  a clipped policy loss with a KL term, from the logits to their gradient.

``run`` computes them in elementary torch operations, or, where ``own`` is set, through the package's
``ops``.  ``exact`` gives the same results in 64 bits.  A target outside [0, V) takes no part.
"""
import math
import statistics

import torch

own = False

INT8, E4M3 = "int8", "e4m3"
BLOCK = 32              # values that share one scale of a checkpoint
IGNORE = -100


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the 16-token, 4096-wide layer input: a checkpoint whose cost is the launch
        {"name": "keep-int8-16x4096", "op": "keep", "M": 16, "K": 4096, "fmt": INT8},
        # input of a 7B block's down projection, an odd number of tokens
        {"name": "keep-e4m3-1999x11008", "op": "keep", "M": 1999, "K": 11008, "fmt": E4M3},
        # input of a 70B block's down projection for 4096 tokens
        {"name": "keep-int8-4096x28672", "op": "keep", "M": 4096, "K": 28672, "fmt": INT8},
        # one 4096 x 4096 layer on 16 tokens, T recomputed
        {"name": "bwd-int8-16-4096x4096", "op": "bwd", "M": 16, "N": 4096, "K": 4096, "r": 16, "fmt": INT8,
         "keep_t": False},
        # gate projection of a 7B block on 2048 tokens, T kept by the forward
        {"name": "bwd-e4m3-2048-11008x4096", "op": "bwd", "M": 2048, "N": 11008, "K": 4096, "r": 16, "fmt": E4M3,
         "keep_t": True},
        # down projection of a 70B block on 509 tokens, rank 64
        {"name": "bwd-int8-509-8192x28672", "op": "bwd", "M": 509, "N": 8192, "K": 28672, "r": 64, "fmt": INT8,
         "keep_t": True},
        # a short answer scored under a vocabulary with one added token: every row at another alignment
        {"name": "logprob-bf16-37x32001", "op": "logprob", "M": 37, "V": 32001, "dtype": "bf16", "scale": 1.0},
        # a packed batch scored by the reference, logits kept in 32 bits
        {"name": "logprob-fp32-8192x32000", "op": "logprob", "M": 8192, "V": 32000, "dtype": "fp32", "scale": 1.0},
        # one pair of short answers
        {"name": "pref-bf16-1pair-61x32000", "op": "pref", "M": 61, "V": 32000, "pairs": 1, "dtype": "bf16",
         "kind": "sigmoid", "average": False, "smooth": 0.0, "scale": 1.0},
        # a packed batch of 16 pairs under a large vocabulary
        {"name": "pref-bf16-16pairs-4096x128256", "op": "pref", "M": 4096, "V": 128256, "pairs": 16, "dtype": "bf16",
         "kind": "sigmoid", "average": False, "smooth": 0.1, "scale": 1.0},
        # one short rollout, logits in 32 bits, sampled at temperature 1 / 1.25
        {"name": "policy-fp32-53x32000", "op": "policy", "M": 53, "V": 32000, "dtype": "fp32", "scale": 1.25},
        # a packed batch of rollouts
        {"name": "policy-bf16-8192x32000", "op": "policy", "M": 8192, "V": 32000, "dtype": "bf16", "scale": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["keep", "bwd", "logprob", "pref", "policy"])
    if op == "keep":
        K = 64 * _log_int(rng, 1, 448)
        M = _log_int(rng, 1, min(16384, 4096 * 28672 // K))
        return {"op": op, "M": M, "K": K, "fmt": rng.choice([INT8, E4M3])}
    if op == "bwd":
        N, K = 8 * _log_int(rng, 8, 3584), 64 * _log_int(rng, 1, 448)
        M = _log_int(rng, 1, max(1, min(4096, 2048 * 11008 * 4096 // (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "r": rng.choice([4, 8, 16, 24, 32, 64, 100]),
                "fmt": rng.choice([INT8, E4M3]), "keep_t": rng.random() < 0.5}
    V = _log_int(rng, 500, 131072)
    dtype = rng.choice(["bf16", "fp32"])
    M = _log_int(rng, 2, min(8192, 8192 * 32000 // V * (2 if dtype == "bf16" else 1)))
    c = {"op": op, "M": M, "V": V, "dtype": dtype, "scale": rng.choice([1.0, 1.0, 0.7, 1.25])}
    if op == "pref":
        c.update(pairs=_log_int(rng, 1, max(1, min(64, M // 4))), kind=rng.choice(["sigmoid", "hinge", "ipo"]),
                 average=rng.random() < 0.3, smooth=0.0)
        if c["kind"] == "sigmoid":
            c["smooth"] = rng.choice([0.0, 0.1])
    return c


BETA = {"sigmoid": 0.1, "hinge": 0.05, "ipo": 0.2}
CLIP_LO, CLIP_HI, KL_COEF = 0.2, 0.28, 0.04


# ------------------------------------------------------------------ inputs
def _codebook(device):
    """The 16 NF4 levels (quantiles of N(0,1), largest 1), each rounded once to 32 bits."""
    z = statistics.NormalDist().inv_cdf
    d = 0.5 * ((1.0 - 1.0 / 32.0) + (1.0 - 1.0 / 30.0))
    pos = [z(d - (d - 0.5) * i / 8.0) for i in range(8)]
    neg = [-z(d - (d - 0.5) * i / 7.0) for i in range(7)]
    v = neg + [0.0] + pos[::-1]
    return torch.tensor([x / v[15] for x in v], dtype=torch.float64, device=device).float()


def _bf16(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _activation(g, M, K):
    """Layer inputs: normal values, each column with a size of its own, a few columns far larger."""
    x = torch.randn((M, K), generator=g, device="cuda")
    col = torch.exp(0.5 * torch.randn((K,), generator=g, device="cuda"))
    col = torch.where(torch.rand((K,), generator=g, device="cuda") < 0.002, col * 20, col)
    return (x * col).to(torch.bfloat16)


def _logits(g, M, V, dtype):
    """Logits with the target usually among the likelier tokens; one row in eight is prompt or padding."""
    x = torch.randn((M, V), generator=g, device="cuda") * 2.5
    y = torch.randint(0, V, (M,), generator=g, device="cuda")
    lift = 14 * torch.rand((M,), generator=g, device="cuda")
    rows = torch.arange(M, device="cuda")
    x[rows, y] += lift
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    skip = torch.rand((M,), generator=g, device="cuda") < 0.125
    return x, torch.where(skip, torch.full_like(y, IGNORE), y)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "keep":
        s["X"] = _activation(g, case["M"], case["K"])
    elif op == "bwd":
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        s["codes"], s["scales"] = _quantize(_activation(g, M, K), case["fmt"])
        s["dY"] = _bf16(g, (M, N), 1.0)
        s["A"] = ((torch.rand((r, K), generator=g, device="cuda") * 2 - 1) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = _bf16(g, (N, r), 0.05)
        s["scaling"] = 32.0 / r
        groups = -(-N * K // (64 * 256))
        s["w_packed"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["w_codes"] = torch.randint(-127, 128, (N * K // 64,), generator=g, device="cuda", dtype=torch.int8)
        s["w_mean"] = 0.04 + 0.01 * torch.rand((groups,), generator=g, device="cuda")
        s["w_scale"] = (0.01 + 0.01 * torch.rand((groups,), generator=g, device="cuda")) / 127
        s["T"] = _bf16(g, (M, r), 0.6) if case["keep_t"] else None
    else:
        M, V = case["M"], case["V"]
        s["logits"], s["targets"] = _logits(g, M, V, case["dtype"])
        if op != "logprob":
            lp = _logprob(s["logits"], s["targets"], case["scale"])[0]
            off = torch.randn((2, M), generator=g, device="cuda", dtype=torch.float64)
        if op == "pref":
            s["ref"] = (lp + 0.3 * off[0]).float()
            # 2 P sequences of unlike lengths; the last rows belong to none
            P = case["pairs"]
            share = 0.2 + torch.rand((2 * P,), generator=g, device="cuda", dtype=torch.float64)
            ends = torch.cumsum(share, 0) / share.sum() * (M - M // 32)
            s["cu"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), ends]).round().to(torch.int32)
        if op == "policy":
            # behaviour policy a few updates back; no ratio within 1e-4 of a border of the clipping
            d = 0.2 * off[0]
            rho = torch.exp(d)
            near = ((rho - (1 - CLIP_LO)).abs() < 1e-4) | ((rho - (1 + CLIP_HI)).abs() < 1e-4)
            s["old"] = (lp - torch.where(near, d + 1e-3, d)).float()
            s["ref"] = (lp + 0.3 * off[1]).float()
            s["adv"] = torch.randn((M,), generator=g, device="cuda")
            n = (s["targets"] >= 0).sum().clamp(min=1)
            s["weight"] = torch.where(s["targets"] >= 0, 1.0 / n, 0.0).float()
    return s


# ------------------------------------------------------------------ plain forms
def _quantize(X, fmt):
    """Codes and scale bytes (exponent + 127) of the 8-bit checkpoint of X."""
    M, K = X.shape
    x = X.float().view(M, K // BLOCK, BLOCK)
    amax = x.abs().amax(-1)
    m, ex = torch.frexp(amax)
    if fmt == INT8:
        e = ex - 7                              # amax / 2^e in [64, 128)
    else:
        e = ex - 9 + (m > 0.875).int()          # amax / 2^e at most 448
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    q = x * torch.ldexp(torch.ones_like(amax), -e)[..., None]
    if fmt == INT8:
        codes = q.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    else:
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(M, K), (e + 127).to(torch.uint8)


def _restore(codes, scales, fmt):
    """The 32-bit values that a checkpoint stands for."""
    M, K = codes.shape
    v = codes.view(torch.int8 if fmt == INT8 else torch.float8_e4m3fn).float()
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (v.view(M, K // BLOCK, BLOCK) * s[..., None]).view(M, K)


def _dequant_weight(s):
    """The dense bf16 weight, as 32-bit values."""
    p = s["w_packed"]
    N, half = p.shape
    q = torch.stack([p >> 4, p & 15], -1).view(-1, 64).int()
    grp = torch.arange(s["w_codes"].numel(), device=p.device) // 256
    c = (s["w_codes"].double() * s["w_scale"].double()[grp] + s["w_mean"].double()[grp]).float()
    return (_codebook(p.device)[q] * c[:, None]).to(torch.bfloat16).float().view(N, 2 * half)


def _logprob(logits, targets, scale):
    """Per row: log p(target) in 64 bits (0 where there is no target), the probabilities, and the mask."""
    x = logits.float() * scale
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    tot = e.sum(-1, keepdim=True)
    live = (targets >= 0) & (targets < logits.shape[1])
    y = torch.where(live, targets, 0)[:, None]
    lp = x.gather(1, y).double() - torch.log(tot.double())
    return torch.where(live, lp[:, 0], 0.0), e.div_(tot), live


def _dlogits(p, targets, live, d, scale, dtype):
    """Gradient of sum d log p(target) with respect to the logits."""
    d = (torch.where(live, d, 0.0) * scale).float()[:, None]
    y = torch.where(live, targets, 0)[:, None]
    gr = p.mul_(-d)
    gr.scatter_add_(1, y, d)
    return torch.where(live[:, None], gr, 0.0).to(dtype)


def _pref_plain(s):
    c = s["case"]
    beta, P, cu = BETA[c["kind"]], c["pairs"], s["cu"].long()
    lp, p, live = _logprob(s["logits"], s["targets"], c["scale"])
    seq = torch.searchsorted(cu, torch.arange(c["M"], device=cu.device), right=True) - 1
    inside = (seq >= 0) & (seq < 2 * P)
    live = live & inside
    seq = seq.clamp(0, 2 * P - 1)
    diff = torch.where(live, lp - s["ref"].double(), 0.0)
    total = torch.zeros(2 * P, dtype=torch.float64, device=cu.device).index_add_(0, seq, diff)
    count = torch.zeros(2 * P, dtype=torch.float64, device=cu.device).index_add_(0, seq, live.double())
    div = count.clamp(min=1) if c["average"] else torch.ones_like(count)
    total = total / div
    delta = total[0::2] - total[1::2]
    z = beta * delta
    if c["kind"] == "sigmoid":
        eps = c["smooth"]
        loss = (1 - eps) * torch.log1p(torch.exp(-z.abs())) + eps * torch.log1p(torch.exp(-z.abs()))
        loss = loss + (1 - eps) * (-z).clamp(min=0) + eps * z.clamp(min=0)
        sg = 1 / (1 + torch.exp(z))
        d = beta * (eps * (1 - sg) - (1 - eps) * sg)
    elif c["kind"] == "hinge":
        loss = (1 - z).clamp(min=0)
        d = torch.where(z < 1, -beta, 0.0).double()
    else:
        loss = (delta - 1 / (2 * beta)) ** 2
        d = 2 * (delta - 1 / (2 * beta))
    dseq = torch.stack([d, -d], 1).view(-1) / P / div
    dl = _dlogits(p, s["targets"], live, dseq[seq], c["scale"], s["logits"].dtype)
    own_lp = torch.where((s["targets"] >= 0) & (s["targets"] < c["V"]), lp, 0.0).float()
    return {"loss": loss.mean().float(), "rewards": (beta * total).float(), "logp": own_lp, "dlogits": dl}


def _policy_plain(s):
    c = s["case"]
    lp, p, live = _logprob(s["logits"], s["targets"], c["scale"])
    live = live & (s["weight"] != 0)
    adv, w = s["adv"].double(), torch.where(live, s["weight"].double(), 0.0)
    rho = torch.exp(torch.where(live, lp - s["old"].double(), 0.0))
    free, held = rho * adv, rho.clamp(1 - CLIP_LO, 1 + CLIP_HI) * adv
    clipped = held < free
    pol = -torch.minimum(free, held)
    d = torch.where(live, s["ref"].double() - lp, 0.0)
    kl = torch.exp(d) - d - 1
    dlp = w * (torch.where(clipped, 0.0, -free) + KL_COEF * (1 - torch.exp(d)))
    sums = torch.stack([(w * (pol + KL_COEF * kl)).sum(), (w * pol).sum(), (w * kl).sum(), (w * clipped).sum()])
    return {"stats": sums.float(), "logp": torch.where(live, lp, 0.0).float(),
            "dlogits": _dlogits(p, s["targets"], live, dlp, c["scale"], s["logits"].dtype)}


def _bwd_plain(s):
    X = _restore(s["codes"], s["scales"], s["case"]["fmt"])
    W, sc = _dequant_weight(s), s["scaling"]
    dY, A, B = s["dY"].float(), s["A"].float(), s["B"].float()
    T = X @ A.T if s["T"] is None else s["T"].float()
    U = dY @ B
    dX, dA, dB = dY @ W + sc * (U @ A), sc * (U.T @ X), sc * (dY.T @ T)
    return {"dX": dX.to(torch.bfloat16), "dA": dA.to(torch.bfloat16), "dB": dB.to(torch.bfloat16)}


def _run_own(s):
    from bit_nf4_quantized_quant_b200 import ops
    c = s["case"]
    op = c["op"]
    if op in ("keep", "bwd"):
        fmt = ops.QLORA_ACT8_INT8 if c["fmt"] == INT8 else ops.QLORA_ACT8_E4M3
    if op == "keep":
        return {"X": ops.act8_dequant(ops.act8_quantize(s["X"], fmt))}
    if op == "bwd":
        w = ops.NF4Weight(s["w_packed"], s["w_codes"], s["w_scale"], s["w_mean"], c["N"], c["K"])
        x8 = ops.Act8Tensor(s["codes"], s["scales"], c["M"], c["K"], fmt)
        dX, dA, dB = ops.qlora_linear_bwd_act8(x8, s["dY"], w, s["A"], s["B"], s["scaling"], T=s["T"])
        return {"dX": dX, "dA": dA, "dB": dB}
    if op == "logprob":
        return {"logp": ops.token_logprob(s["logits"], s["targets"], logit_scale=c["scale"])}
    if op == "pref":
        kind = {"sigmoid": ops.QLORA_PREF_SIGMOID, "hinge": ops.QLORA_PREF_HINGE, "ipo": ops.QLORA_PREF_IPO}
        o = ops.preference_loss(s["logits"], s["targets"], s["cu"], s["ref"], BETA[c["kind"]], kind=kind[c["kind"]],
                                label_smoothing=c["smooth"], average=c["average"], logit_scale=c["scale"])
        return {"loss": o.loss, "rewards": o.rewards, "logp": o.logp, "dlogits": o.dlogits}
    o = ops.policy_loss(s["logits"], s["targets"], s["adv"], s["weight"], s["old"], s["ref"], CLIP_LO, CLIP_HI,
                        KL_COEF, logit_scale=c["scale"])
    return {"stats": o.stats, "logp": o.logp, "dlogits": o.dlogits}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "keep":
        fmt = state["case"]["fmt"]
        return {"X": _restore(*_quantize(state["X"], fmt), fmt).to(torch.bfloat16)}
    if op == "bwd":
        return _bwd_plain(state)
    if op == "logprob":
        return {"logp": _logprob(state["logits"], state["targets"], state["case"]["scale"])[0].float()}
    return _pref_plain(state) if op == "pref" else _policy_plain(state)


# ------------------------------------------------------------------ work
def work(case):
    """Bytes: each input read once, each output written once.  Flops: products of the matrices, and for the
    losses about four operations per logit and direction."""
    op, M = case["op"], case["M"]
    if op == "keep":        # the bf16 values read, the checkpoint written and read, the bf16 values written
        n = M * case["K"]
        return {"bytes": 4 * n + 2 * (n + n // BLOCK), "flops": 2 * n}
    if op == "bwd":
        N, K, r = case["N"], case["K"], case["r"]
        t = 0 if case["keep_t"] else 2 * M * K * r
        nbytes = (M * K + M * K // BLOCK + N * K // 2 + N * K // 64 + 8 * -(-N * K // 16384) + 2 * M * N
                  + 2 * r * (N + K) + (2 * M * r if case["keep_t"] else 0) + 2 * M * K + 2 * r * (N + K))
        return {"bytes": nbytes, "flops": 2 * M * N * K + 4 * M * r * (N + K) + t}
    V, es = case["V"], 2 if case["dtype"] == "bf16" else 4
    if op == "logprob":
        return {"bytes": M * V * es + 12 * M, "flops": 4 * M * V}
    extra = 16 * M + 16 * case["pairs"] if op == "pref" else 28 * M
    return {"bytes": 2 * M * V * es + extra, "flops": 8 * M * V}


# ------------------------------------------------------------------ definitions in 64 bits
def _nearest_e4m3(v):
    """The E4M3 value nearest to v >= 0 (halfway: the even code), by the list of all of them."""
    grid = [m / 8 * 2.0 ** -6 for m in range(8)]
    grid += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(v, mid)
    at = mid[i.clamp(max=mid.numel() - 1)]
    return grid[torch.where((v == at) & (i % 2 == 1), i + 1, i).clamp(max=grid.numel() - 1)]


def _exact_keep(X, fmt):
    M, K = X.shape
    out = []
    for x in X.split(512):
        x = x.double().view(x.shape[0], K // BLOCK, BLOCK)
        top = x.abs().amax(-1, keepdim=True)
        # the largest power of two not above top, from the exponent field of the 64-bit value
        e = ((top.view(torch.int64) >> 52) - 1023).double()
        if fmt == INT8:
            step = torch.exp2(e - 6)
            v = torch.sign(x) * torch.clamp(torch.round(x.abs() / step), max=127) * step
        else:
            step = torch.exp2(e - 8)
            step = torch.where(top > 448 * step, 2 * step, step)
            v = torch.sign(x) * _nearest_e4m3(x.abs() / step) * step
        out.append(torch.where(top > 0, v, 0.0).view(-1, K))
    return torch.cat(out)


def _exact_bwd(s):
    c = s["case"]
    N, K, M = c["N"], c["K"], c["M"]
    e = s["scales"].double() - 127
    if c["fmt"] == INT8:
        v = s["codes"].double()
        v = torch.where(v >= 128, v - 256, v)
    else:
        b = s["codes"].int()
        ex, man = (b >> 3) & 15, (b & 7).double()
        v = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex.double() - 7))
        v = torch.where(b >= 128, -v, v)
    X = v * torch.exp2(e).repeat_interleave(BLOCK, 1)
    p = s["w_packed"]
    lev = _codebook(p.device).double()
    W = torch.empty((N, K), dtype=torch.float64, device=p.device)
    W[:, 0::2], W[:, 1::2] = lev[(p >> 4).long()], lev[(p & 15).long()]
    g = torch.arange(N * K // 64, device=p.device) // 256
    # the block constants are 32-bit values, the weights bf16 ones: both roundings belong to the format
    cb = (s["w_codes"].double() * s["w_scale"].double()[g] + s["w_mean"].double()[g]).float().double()
    W = (W * cb.view(N, K // 64).repeat_interleave(64, 1)).float().bfloat16().double()
    dY, A, B = s["dY"].double(), s["A"].double(), s["B"].double()
    T = X @ A.T if s["T"] is None else s["T"].double()
    U = dY @ B
    return {"dX": dY @ W + s["scaling"] * (U @ A), "dA": s["scaling"] * (U.T @ X), "dB": s["scaling"] * (dY.T @ T)}


def _exact_losses(s):
    """Loss by torch's 64-bit log_softmax and its gradient by autograd, rows without a target left out."""
    c = s["case"]
    M, V = c["M"], c["V"]
    rows = ((s["targets"] >= 0) & (s["targets"] < V)).nonzero()[:, 0]
    x = s["logits"].double().requires_grad_(c["op"] != "logprob")
    picked = torch.log_softmax(x[rows] * c["scale"], -1)[torch.arange(rows.numel(), device=rows.device),
                                                          s["targets"][rows]]
    logp = torch.zeros(M, dtype=torch.float64, device=rows.device)
    logp[rows] = picked.detach()
    if c["op"] == "logprob":
        return {"logp": logp}
    if c["op"] == "pref":
        beta, cu, losses, rewards = BETA[c["kind"]], s["cu"].tolist(), [], []
        for i in range(2 * c["pairs"]):
            mine = (rows >= cu[i]) & (rows < cu[i + 1])
            d = picked[mine] - s["ref"].double()[rows[mine]]
            rewards.append(d.mean() if c["average"] and d.numel() else d.sum())
        for a, b in zip(rewards[0::2], rewards[1::2]):
            z = beta * (a - b)
            if c["kind"] == "sigmoid":
                ls = torch.nn.functional.logsigmoid
                losses.append(-(1 - c["smooth"]) * ls(z) - c["smooth"] * ls(-z))
            elif c["kind"] == "hinge":
                losses.append(torch.relu(1 - z))
            else:
                losses.append((a - b - 1 / (2 * beta)) ** 2)
        loss = torch.stack(losses).mean()
        out = {"loss": loss.detach(), "rewards": beta * torch.stack(rewards).detach(), "logp": logp}
    else:
        w, adv = s["weight"].double()[rows], s["adv"].double()[rows]
        rho = torch.exp(picked - s["old"].double()[rows])
        held = torch.clamp(rho, 1 - CLIP_LO, 1 + CLIP_HI) * adv
        pol = -torch.minimum(rho * adv, held)
        d = s["ref"].double()[rows] - picked
        kl = torch.expm1(d) - d
        loss = (w * (pol + KL_COEF * kl)).sum()
        parts = [loss, (w * pol).sum(), (w * kl).sum(), (w * (held < rho * adv)).sum()]
        out = {"stats": torch.stack(parts).detach(), "logp": logp}
    if rows.numel():
        loss.backward()
    out["dlogits"] = x.grad if x.grad is not None else torch.zeros_like(x).detach()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keep":
        return {"X": _exact_keep(s["X"], case["fmt"])}
    return _exact_bwd(s) if case["op"] == "bwd" else _exact_losses(s)
