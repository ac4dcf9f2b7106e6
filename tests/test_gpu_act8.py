"""8-bit activation checkpoints on the GPU: codes, scales and restored values bit for bit the oracle's, and the
backward that reads a checkpoint bit for bit the backward of the bf16 tensor it stands for."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops
from bit_nf4_quantized_quant_b200 import inputs
from oracle import training as tr

pytestmark = pytest.mark.gpu
FMTS = [ops.QLORA_ACT8_INT8, ops.QLORA_ACT8_E4M3]


def _activation(seed, M, K):
    """Columns of unlike sizes, a few of them 20 times larger, some values exactly 0."""
    x = inputs.normal(seed, (M, K), 1.0).float()
    col = torch.exp(inputs.normal(seed + 1, (K,), 0.7).float())
    col[::41] *= 20
    x = x * col
    x[:, 5::17] = 0
    return x.to(torch.bfloat16)


def _compare(X, fmt):
    q = ops.act8_quantize(X.cuda(), fmt)
    back = ops.act8_dequant(q)
    torch.cuda.synchronize()
    codes, scales = tr.act8_quantize(inputs.to_f64(X), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    want = torch.from_numpy(tr.act8_values(codes, scales, fmt)).to(torch.bfloat16)
    assert np.array_equal(inputs.to_f64(back), want.double().numpy(), equal_nan=True)
    return q, back


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 64), (3, 192), (16, 4096), (17, 320), (257, 1088), (1999, 704)])
def test_quantize_and_dequant_bit_exact(M, K, fmt):
    _compare(_activation(M + K, M, K), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("std", [1e-40, 1e-38, 1e-36, 1e-20, 1e20, 2e37])
def test_extreme_magnitudes(fmt, std):
    X = (inputs.normal(5, (4, 256), 1.0).double() * std).to(torch.bfloat16)
    assert torch.isfinite(X).all()
    _compare(X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_special_blocks(fmt):
    """Zeros, one subnormal, the largest finite value, both sides of every rounding of the block maximum, and
    infinities and NaN, which make their block NaN and no other."""
    top = torch.arange(256, dtype=torch.int32)                 # every mantissa under two exponents
    X = torch.zeros((260, 64), dtype=torch.bfloat16)
    X[:256, 0] = (0x3F80 + top).to(torch.int16).view(torch.bfloat16)
    X[:256, 1:32] = inputs.normal(6, (256, 31), 0.4)
    X[:256, 33] = -X[:256, 0]
    X[256, 0] = 2.0 ** -133
    X[257, 0] = torch.finfo(torch.bfloat16).max
    X[257, 1] = -torch.finfo(torch.bfloat16).max
    X[258, 0], X[258, 1], X[258, 40] = float("inf"), 1.0, 2.0
    X[259, 3], X[259, 40] = float("nan"), float("-inf")
    q, back = _compare(X, fmt)
    assert torch.isnan(back[258, :32]).all() and not torch.isnan(back[258, 32:]).any()
    assert torch.isnan(back[259]).all()
    assert (back[:256, 32] == 0).all() and (q.scales[256, 1] == 0).item()


@pytest.mark.parametrize("fmt", FMTS)
def test_dequant_every_code_under_every_scale(fmt):
    """All 256 codes under all 256 scale bytes, also those that act8_quantize does not write."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 8))
    x = ops.Act8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 256, 256, fmt)
    got = inputs.to_f64(ops.act8_dequant(x))
    v = torch.from_numpy(tr.act8_values(codes, scales, fmt)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(got, v, equal_nan=True)


def test_only_the_checkpoint_is_written():
    """Codes and scales in the middle of larger buffers: their neighbours stay."""
    M, K = 5, 192
    buf = torch.full((M * K + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    sb = torch.full((M * K // 32 + 32,), 0xAB, dtype=torch.uint8, device="cuda")
    out = ops.Act8Tensor(buf[32:32 + M * K].view(M, K), sb[7:7 + M * K // 32].view(M, K // 32), M, K)
    X = _activation(3, M, K).cuda()
    ops.act8_quantize(X, out=out)
    ref = ops.act8_quantize(X)
    assert torch.equal(out.codes, ref.codes) and torch.equal(out.scales, ref.scales)
    assert (buf[:32] == 0xAB).all() and (buf[-32:] == 0xAB).all()
    assert (sb[:7] == 0xAB).all() and (sb[7 + M * K // 32:] == 0xAB).all()


def _layer(M, N, K, r, seed):
    w = ops.nf4_quantize_dq(inputs.weight(70 + seed, 0, N, K, 0.02).cuda())
    X = _activation(seed, M, K).cuda()
    A = inputs.uniform(71 + seed, (r, K), 1.0 / np.sqrt(K)).cuda()
    B = inputs.normal(72 + seed, (N, r), 0.1).cuda()
    dY = inputs.normal(73 + seed, (M, N), 1.0).cuda()
    return w, X, A, B, dY


BWD = [(1, 64, 64, 16), (3, 136, 192, 4), (16, 512, 512, 64), (17, 200, 320, 24), (32, 1024, 1024, 16),
       (33, 128, 256, 16), (100, 264, 640, 8), (128, 256, 256, 16), (200, 520, 448, 24), (257, 384, 448, 64),
       (300, 768, 1216, 100), (512, 1024, 2048, 16), (130, 256, 512, 256), (64, 256, 4160, 32), (1000, 520, 1088, 48)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r", BWD)
def test_bwd_equals_the_backward_of_the_restored_tensor(M, N, K, r, fmt):
    w, X, A, B, dY = _layer(M, N, K, r, M + r)
    s = 32.0 / r
    x8 = ops.act8_quantize(X, fmt)
    Xr = ops.act8_dequant(x8)
    T = torch.empty((M, r), dtype=torch.bfloat16, device="cuda")
    ops.qlora_linear_fwd(X, w, A, B, s, T_out=T)
    for t in (None, T):
        got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, s, T=t)
        want = ops.qlora_linear_bwd(Xr, dY, w, A, B, s, T=t)
        for a, b, name in zip(got, want, ("dX", "dA", "dB")):
            assert torch.equal(a, b), (name, t is None)
    got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, s, T=T, dropout_p=0.1, seed=5, offset=9)
    want = ops.qlora_linear_bwd_dropout(Xr, dY, w, A, B, s, 0.1, 5, 9, T=T)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert ops.qlora_device_status() == 0


@pytest.mark.parametrize("M", [17, 70, 200])
def test_bwd_dropout_without_T_and_fp4(M):
    """T recomputed from the dropped checkpoint, and an FP4 weight."""
    _, X, A, B, dY = _layer(M, 200, 320, 24, M)
    w = ops.quant4_quantize_dq(inputs.weight(9, 0, 200, 320, 0.02).cuda(), ops.QLORA_QUANT_FP4)
    for fmt in FMTS:
        x8 = ops.act8_quantize(X, fmt)
        Xr = ops.act8_dequant(x8)
        got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, 1.5, dropout_p=0.3, seed=11, offset=2)
        want = ops.qlora_linear_bwd_dropout(Xr, dY, w, A, B, 1.5, 0.3, 11, 2)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, 1.5)
        assert all(torch.equal(a, b) for a, b in zip(got, ops.qlora_linear_bwd(Xr, dY, w, A, B, 1.5)))


@pytest.mark.parametrize("M", [24, 160])
def test_bwd_against_the_formula(oracle_mod, M):
    """dA and dB against fp64 products of the checkpoint's values (the tolerance of the layer's own parity tests:
    1e-2 max(1, |ref|))."""
    N, K, r, s = 512, 1024, 16, 2.0
    w, X, A, B, dY = _layer(M, N, K, r, 11)
    Wd = inputs.to_f64(ops.nf4_dequant(w))
    for fmt in FMTS:
        x8 = ops.act8_quantize(X, fmt)
        Xv = tr.act8_values(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), fmt)
        ref = oracle_mod.linear_bwd(Xv, inputs.to_f64(dY), Wd, inputs.to_f64(A), inputs.to_f64(B), s)
        for g, r64 in zip(ops.qlora_linear_bwd_act8(x8, dY, w, A, B, s), ref):
            assert (np.abs(inputs.to_f64(g) - r64) <= 1e-2 * np.maximum(1, np.abs(r64))).all()


@pytest.mark.parametrize("M", [8, 96, 300])
def test_captured_and_two_streams(M):
    """A captured quantize + backward replays to the eager result with new inputs; two backwards on two streams,
    each with its own workspace, do not disturb one another."""
    N, K, r, s = 256, 512, 16, 2.0
    w, X, A, B, dY = _layer(M, N, K, r, 21)
    ws = ops.act8_workspace(M, N, K, r)
    x8 = ops.Act8Tensor.empty(M, K)
    outs = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in ((M, K), (r, K), (N, r))]

    def step():
        ops.act8_quantize(X, out=x8)
        ops.qlora_linear_bwd_act8(x8, dY, w, A, B, s, dX=outs[0], dA=outs[1], dB=outs[2], ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    X.copy_(_activation(99, M, K))
    want = ops.qlora_linear_bwd(ops.act8_dequant(ops.act8_quantize(X)), dY, w, A, B, s)
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    del g
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [ops.act8_quantize(X, f) for f in FMTS]
    refs = [ops.qlora_linear_bwd_act8(x, dY, w, A, B, s) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [ops.qlora_linear_bwd_act8(x, dY, w, A, B, s, stream=st) for x, st in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals_on_the_gpu():
    x8 = ops.act8_quantize(_activation(1, 4, 64).cuda())
    w, _, A, B, dY = _layer(4, 64, 64, 16, 1)
    with pytest.raises(ValueError, match="dY"):
        ops.qlora_linear_bwd_act8(x8, dY[:3], w, A, B, 2.0)
    with pytest.raises(ValueError, match="B"):
        ops.qlora_linear_bwd_act8(x8, dY, w, A, B[:, :8].contiguous(), 2.0)
    with pytest.raises(ops.QLoRAError) as e:
        ops.qlora_linear_bwd_act8(x8, dY, w, A, B, 2.0, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -5
    with pytest.raises(ValueError, match="out"):
        ops.act8_dequant(x8, out=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r", [(3092, 72, 28480, 8), (3092, 1000, 28480, 16), (509, 64, 28672, 16),
                                     (2000, 128, 12800, 24), (4096, 64, 8192, 64), (2048, 4096, 4096, 16)])
def test_bwd_repeats_bit_identically(M, N, K, r, fmt):
    """Hundreds of calls, in long reductions by several CTAs an SM among others: the gradients of the restored tensor
    bit for bit, every time (a stage of the ring refilled under loads still in flight shows as a rare difference)."""
    w, X, A, B, dY = _layer(M, N, K, r, M + r)
    x8 = ops.act8_quantize(X, fmt)
    T = torch.empty((M, r), dtype=torch.bfloat16, device="cuda")
    ops.qlora_linear_fwd(X, w, A, B, 2.0, T_out=T)
    want = ops.qlora_linear_bwd(ops.act8_dequant(x8), dY, w, A, B, 2.0, T=T)
    ws = ops.act8_workspace(M, N, K, r)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    for _ in range(300):
        got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, 2.0, T=T, ws=ws)
        for i in range(3):
            off[i] += (got[i].view(torch.int16) != want[i].view(torch.int16)).any()
    assert off.tolist() == [0, 0, 0]
    assert ops.qlora_device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_bwd_with_t_recomputed_repeats_bit_identically(fmt):
    """The same for the T product, whose ring is the longest here (56 stages on 392 CTAs, three an SM)."""
    M, N, K, r = 3092, 72, 28480, 8
    w, X, A, B, dY = _layer(M, N, K, r, 5)
    x8 = ops.act8_quantize(X, fmt)
    ws = ops.act8_workspace(M, N, K, r)
    want = ops.qlora_linear_bwd(ops.act8_dequant(x8), dY, w, A, B, 2.0)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(3000):
        got = ops.qlora_linear_bwd_act8(x8, dY, w, A, B, 2.0, ws=ws)
        off += sum((g.view(torch.int16) != t.view(torch.int16)).any() for g, t in zip(got, want))
    assert off.item() == 0 and ops.qlora_device_status() == 0
