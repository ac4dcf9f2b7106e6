"""Refusals of the 8-bit checkpoints and the losses (CPU, nothing is launched): the documented error
codes of the C entry points, and the shape, type and device checks of the binding."""
import ctypes

import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops

NAN, INF = float("nan"), float("inf")
P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1001)                # never dereferenced: every call is rejected first


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_quant_b200 import build
    build.build()
    return ops.lib()


def test_act8_sizes(lib):
    assert ops.act8_sizes(2048, 4096) == (2048 * 4096, 2048 * 128)
    for M, K in [(0, 64), (4, 0), (4, 96), (-1, 64), (1 << 40, 64)]:
        with pytest.raises(ops.QLoRAError) as e:
            ops.act8_sizes(M, K)
        assert e.value.code == -2
    assert lib.act8_sizes(1, 64, None, None) == 0


def test_act8_quantize_and_dequant_refusals(lib):
    q = lib.act8_quantize
    assert q(None, 1, 64, 0, FAKE, FAKE, None) == -1
    assert q(FAKE, 1, 64, 0, None, FAKE, None) == -1
    assert q(FAKE, 1, 64, 0, FAKE, None, None) == -1
    assert q(FAKE, 1, 96, 0, FAKE, FAKE, None) == -2
    assert q(FAKE, 0, 64, 0, FAKE, FAKE, None) == -2
    assert q(FAKE, 1, 64, 2, FAKE, FAKE, None) == -9
    assert q(P(0x1008), 1, 64, 0, FAKE, FAKE, None) == -4
    assert q(FAKE, 1, 64, 0, P(0x1008), FAKE, None) == -4
    x = ops._Act8(0x1000, 0x1000, 1, 64, 0)
    assert lib.act8_dequant(None, FAKE, None) == -1
    assert lib.act8_dequant(ctypes.byref(x), None, None) == -1
    assert lib.act8_dequant(ctypes.byref(x), P(0x1008), None) == -4
    bad = ops._Act8(0x1000, 0x1000, 1, 64, 7)
    assert lib.act8_dequant(ctypes.byref(bad), FAKE, None) == -9


def _bwd(lib, x, w, p=0.0, r=16, dY=FAKE, ws=FAKE, n=1 << 40):
    return lib.qlora_linear_bwd_act8(ctypes.byref(x), dY, ctypes.byref(w), FAKE, FAKE, r, 2.0, p, 0, 0, None, FAKE,
                                     FAKE, FAKE, ws, n, None)


def test_bwd_act8_refusals(lib):
    x, w = ops._Act8(0x1000, 0x1000, 4, 128, 0), ops._Weight(0x1000, 0x1000, 0x1000, 0x1000, 64, 128)
    assert _bwd(lib, x, ops._Weight(0x1000, 0x1000, 0x1000, 0x1000, 64, 64)) == -2      # K of X and W differ
    assert _bwd(lib, ops._Act8(0, 0x1000, 4, 128, 0), w) == -1
    assert _bwd(lib, ops._Act8(0x1000, 0, 4, 128, 0), w) == -1
    assert _bwd(lib, ops._Act8(0x1000, 0x1000, 4, 128, 5), w) == -9
    assert _bwd(lib, x, w, dY=None) == -1
    assert _bwd(lib, x, w, r=0) == -3
    for p in (1.0, -0.1, NAN):
        assert _bwd(lib, x, w, p=p) == -9
    assert _bwd(lib, x, w, ws=None) == -5
    assert lib.qlora_linear_bwd_act8(None, FAKE, ctypes.byref(w), FAKE, FAKE, 16, 2.0, 0.0, 0, 0, None, FAKE, FAKE,
                                     FAKE, FAKE, 1 << 30, None) == -1


def test_act8_workspace(lib):
    for M in (1, 16, 300):
        plain, drop = (ops.qlora_act8_workspace_bytes(M, 256, 512, 16, d) for d in (False, True))
        assert plain >= ops.qlora_workspace_bytes(M, 256, 512, 16)
        assert drop >= ops.qlora_dropout_workspace_bytes(M, 256, 512, 16)
    assert ops.qlora_act8_workspace_bytes(4, 256, 500, 16) == 0
    assert ops.qlora_act8_workspace_bytes(4, 256, 512, 0, True) == 0
    with pytest.raises(ops.QLoRAError):
        ops.act8_workspace(0, 256, 512, 16, device="cpu")


def _logits_refusals(call):
    """call(logits=, dtype=, M=, V=, ld=, tau=, targets=) of one entry point."""
    assert call(logits=None) == -1
    assert call(targets=None) == -1
    assert call(dtype=2) == -9
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(V=0), dict(V=(1 << 18) + 1, ld=1 << 20), dict(ld=31)):
        assert call(**kw) == -2, kw
    for tau in (0.0, -1.0, NAN, INF, 3e38):
        assert call(tau=tau) == -9, tau
    assert call(logits=ODD) == -4
    assert call(logits=P(0x1002), dtype=1) == -4
    assert call(targets=P(0x1004)) == -4


def test_token_logprob_refusals(lib):
    def call(logits=FAKE, dtype=0, M=4, V=32, ld=32, tau=1.0, targets=FAKE, out=FAKE):
        return lib.token_logprob(logits, dtype, M, V, ld, tau, targets, out, None)
    _logits_refusals(call)
    assert call(out=None) == -1
    assert call(out=ODD) == -4


def test_preference_refusals(lib):
    def call(logits=FAKE, dtype=0, M=4, V=32, ld=32, tau=1.0, targets=FAKE, cu=FAKE, pairs=2, ref=FAKE, kind=0,
             beta=0.1, eps=0.0, margin=0.0, gs=1.0, loss=FAKE, rewards=FAKE, logp=FAKE, dl=FAKE, ldd=32, ws=FAKE,
             n=1 << 20):
        return lib.preference_loss(logits, dtype, M, V, ld, tau, targets, cu, pairs, ref, kind, beta, eps, margin, 0,
                                   gs, loss, rewards, logp, dl, ldd, ws, n, None)
    _logits_refusals(call)
    for k in ("cu", "loss", "rewards", "logp"):
        assert call(**{k: None}) == -1
        assert call(**{k: ODD}) == -4
    assert call(ref=ODD) == -4 and call(dl=ODD) == -4
    assert call(pairs=0) == -2 and call(ldd=31) == -2
    for kw in (dict(kind=3), dict(beta=0.0), dict(beta=NAN), dict(beta=INF), dict(eps=-0.1), dict(eps=1.5),
               dict(eps=NAN), dict(kind=1, eps=0.1), dict(kind=2, eps=0.1), dict(kind=2, margin=0.5),
               dict(margin=INF), dict(gs=NAN)):
        assert call(**kw) == -9, kw
    assert call(ws=None) == -5 and call(n=16) == -5 and call(ws=P(0x1010)) == -4


def test_policy_refusals(lib):
    def call(logits=FAKE, dtype=0, M=4, V=32, ld=32, tau=1.0, targets=FAKE, adv=FAKE, w=FAKE, old=FAKE, ref=FAKE,
             lo=0.2, hi=0.2, kl=0.1, gs=1.0, stats=FAKE, logp=FAKE, dl=FAKE, ldd=32, ws=FAKE, n=1 << 20):
        return lib.policy_loss(logits, dtype, M, V, ld, tau, targets, adv, w, old, ref, lo, hi, kl, gs, stats, logp,
                               dl, ldd, ws, n, None)
    _logits_refusals(call)
    for k in ("adv", "w", "stats", "logp"):
        assert call(**{k: None}) == -1
        assert call(**{k: ODD}) == -4
    assert call(old=ODD) == -4 and call(ref=ODD) == -4 and call(dl=ODD) == -4
    assert call(ldd=31) == -2
    for kw in (dict(lo=-0.1), dict(lo=1.1), dict(lo=NAN), dict(hi=-0.1), dict(hi=INF), dict(kl=NAN), dict(gs=INF)):
        assert call(**kw) == -9, kw
    assert call(ws=None) == -5 and call(n=16) == -5 and call(ws=P(0x1010)) == -4


@pytest.mark.parametrize("es", [2, 4])
def test_gradient_rows_that_overlap_other_rows_are_refused(lib, es):
    """At the logits' own place the gradient is in place; beside their rows, in the same buffer, it
    is apart; everywhere else in their range two rows would be written and read at once.  The
    workspace is missing in every call, so that what is not refused ends there."""
    base, M, V = 1 << 20, 4, 32
    dtype = 0 if es == 2 else 1

    def want(off, ld, ldd):
        if off == 0 and ld == ldd:
            return -5
        rows = {i * ld + v for i in range(M) for v in range(V)}
        grads = {off + i * ldd + v for i in range(M) for v in range(V)}
        if ld == ldd:
            return -2 if rows & grads else -5
        lo, hi = (0, (M - 1) * ld + V), (off, off + (M - 1) * ldd + V)
        return -2 if lo[0] < hi[1] and hi[0] < lo[1] else -5

    for ld, ldd in [(32, 32), (40, 40), (64, 64), (80, 80), (64, 32), (32, 64)]:
        for off in range(-330, 331):
            g, l = P(base + off * es), P(base)
            assert lib.policy_loss(l, dtype, M, V, ld, 1.0, FAKE, FAKE, FAKE, None, None, 0.2, 0.2, 0.0, 1.0, FAKE,
                                   FAKE, g, ldd, None, 0, None) == want(off, ld, ldd), (ld, ldd, off)
            assert lib.preference_loss(l, dtype, M, V, ld, 1.0, FAKE, FAKE, 1, None, 0, 0.1, 0.0, 0.0, 0, 1.0, FAKE,
                                       FAKE, FAKE, g, ldd, None, 0, None) == want(off, ld, ldd), (ld, ldd, off)
    # one row has no pitch
    assert lib.policy_loss(P(base), dtype, 1, V, 32, 1.0, FAKE, FAKE, FAKE, None, None, 0.2, 0.2, 0.0, 1.0, FAKE, FAKE,
                           P(base), 64, None, 0, None) == -5


def test_loss_workspace(lib):
    assert ops.loss_workspace_bytes(1) >= 16 and ops.loss_workspace_bytes(1000) >= 16000
    assert ops.loss_workspace_bytes(0) == 0 and ops.loss_workspace_bytes((1 << 24) + 1) == 0


def test_binding_refuses_what_the_pointers_cannot_say(lib):
    """Types, shapes, strides and devices are checked before a pointer is taken."""
    bf = torch.bfloat16
    l, y, f = torch.zeros((4, 32), dtype=bf), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        ops._need(f, "f", torch.float32, (4,))
    for bad in (l.half(), l.view(-1), l.t()):
        with pytest.raises(ValueError, match="logits"):
            ops.token_logprob(bad, y)
    with pytest.raises(ValueError, match="logits"):
        ops.preference_loss(l, y, cu, f, 0.1)
    with pytest.raises(ValueError, match="logits"):
        ops.policy_loss(l, y, f, f, None, None)
    with pytest.raises(ValueError, match="X"):
        ops.act8_quantize(l.float())
    with pytest.raises(ValueError, match="codes"):
        ops.Act8Tensor(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=torch.uint8), 4, 64).c_struct()
    with pytest.raises(ValueError, match="contiguous"):
        ops._need(torch.zeros((4, 4)).t(), "t", torch.float32, (4, 4))
    with pytest.raises(ValueError, match="got NoneType"):
        ops._need(None, "t", torch.float32, (4,))
