"""The losses on logits where their arithmetic is at its limits: rows far from 0, exponentials and sums out of range.

Tolerances, from the kernels' fp32 arithmetic (u = 2^-24):
  logp:    1e-5 for the exponentials and the merging of partial sums, n u for the n terms that a thread adds one
           after another in the careful form (V / 32 where a warp has the row, V / 128 where a block has it), and
           4 u (|logp| + |scale (l_y - r)|) for the subtraction, the product with the scale and the roundings.
  dlogits = g (1[v = y] - p): p is off by the same (1e-5 + n u) of itself and by 3 u |t| for its exponent (|t| < 200
           where p counts: 4e-5); g by 8 u (seven products and an exponential of one unit in the last place) and by
           what the derivative of the loss makes of the error of logp; then half a step of the output type, and what
           flushes to zero (2^-126 of g).
"""
import math

import numpy as np
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops
from oracle import training as tr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": U}
# a warp a row, a block a row, clusters of CTAs, rows beyond the registers of a block
SHAPES = [(9, 300), (700, 5003), (9, 40000), (330, 20001), (3, 131072)]


def _rows_at(M, V, dtype, at):
    """Rows of equal logits near `at` (even ones) and of logits up to three steps of the type towards 0 from there
    (odd ones), with a target each."""
    g = np.random.default_rng(V)
    l = torch.full((M, V), at, dtype=torch.float64)
    step = 2.0 ** (math.floor(math.log2(abs(at))) - (7 if dtype == "bf16" else 23))
    l[1::2] -= torch.from_numpy(g.integers(0, 4, l[1::2].shape)) * math.copysign(step, at)
    return l.to(DT[dtype]).cuda(), g.integers(0, V, M)


def _check_rows(l, yn, tau, dtype):
    """Log-probabilities of the three entry points and gradients of both losses (a policy loss of ratio 1 and
    advantage -1: g = 1; an IPO loss of one row against none a pair: g = 2 (logp - 1))."""
    M, V = l.shape
    y = torch.from_numpy(yn).cuda()
    l64 = l.double().cpu().numpy()
    ref, ls, _ = tr.token_logprob(l64, yn, tau)
    n = V / (32 if V * l.element_size() <= 8192 + 16 else 128)
    e_lp = 1e-5 + n * U + 4 * U * (np.abs(ref) + np.abs(tau * (l64[np.arange(M), yn] - l64.max(-1))))
    ones = torch.ones(M, device="cuda")
    pol = ops.policy_loss(l, y, -ones, ones, None, None, logit_scale=tau)
    cu = torch.arange(M + 1, device="cuda", dtype=torch.int32).repeat_interleave(2)[1:].contiguous()
    pre = ops.preference_loss(l, y, cu, None, 0.5, kind=ops.QLORA_PREF_IPO, grad_scale=M, logit_scale=tau)
    for name, lp in (("token", ops.token_logprob(l, y, tau)), ("policy", pol.logp), ("preference", pre.logp)):
        err = np.abs(lp.double().cpu().numpy() - ref)
        assert (err <= e_lp).all(), (name, err.max())
    p = np.exp(ls)
    want = np.where(np.arange(V)[None] == yn[:, None], 1.0, 0.0) - p
    e_lp = e_lp[:, None]
    for name, got, g, e_g in (("policy", pol.dlogits, np.ones((M, 1)), 0.0),
                              ("preference", pre.dlogits, 2 * (ref - 1.0)[:, None], 2 * e_lp)):
        got, g = got.double().cpu().numpy(), g * tau
        e = (e_g * tau + 8 * U * np.abs(g)) * np.where(want != 0, 1.0, 0.0)
        lim = np.abs(g) * p * (e_lp + 5e-5) + e + HALF[dtype] * np.abs(want * g) + (np.abs(g) + tau) * 2.0 ** -126
        bad = ~(np.abs(got - want * g) <= lim * 1.0001)
        assert not bad.any(), (name, bad.sum(), np.abs(got - want * g)[bad].max(), np.argwhere(bad)[:3])


# (about) the logits, the scale: |scale * logits| from 1e6 on, up to 2^45
FAR = [(1e6, 1.0), (-1e7, 1.0), (2e7, 1.25), (-2e7, 1.0), (1e8, 1.0), (-1e8, 1.25), (1e9, 1.0), (-1e9, 1.0),
       (-1e9, 1e-3), (3e3, 1e4), (30.0, 2.0 ** 40)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
@pytest.mark.parametrize("at,tau", FAR)
def test_rows_far_from_zero(at, tau, M, V, dtype):
    """What the log-probability keeps of logits that are large and alike: their differences, whole."""
    _check_rows(*_rows_at(M, V, dtype, at), tau, dtype)


# offsets at which the rest of the scale times log2 e, 2^-24 to 2^-23 of it, times the logits is more than bf16 keeps
NEAR = [(1e4, 1.25), (-1e5, 1.25), (1e5, 1.0), (-1e5, 0.6), (3e5, 1.0), (-5e5, 1.25), (1e6, 0.6), (-1e6, 0.6)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
@pytest.mark.parametrize("at,tau", NEAR)
def test_rows_with_a_large_offset(at, tau, M, V, dtype):
    _check_rows(*_rows_at(M, V, dtype, at), tau, dtype)


def test_gradient_rows_with_a_large_offset_at_another_alignment():
    """A gradient row whose 16-byte boundaries are not the logits' equals the one whose boundaries are."""
    for M, V in ((9, 300), (9, 40001)):
        l, yn = _rows_at(M, V, "bf16", -1e5)
        y, w = torch.from_numpy(yn).cuda(), torch.ones(M, device="cuda")
        cu = torch.tensor([0, 4, M], dtype=torch.int32, device="cuda")
        out = torch.empty((M * (V + 7) + 1,), dtype=torch.bfloat16, device="cuda")
        dl = out.as_strided((M, V), (V + 7, 1), 1)
        for f in (lambda **k: ops.policy_loss(l, y, -w, w, None, None, logit_scale=1.25, **k),
                  lambda **k: ops.preference_loss(l, y, cu, None, 0.1, logit_scale=1.25, **k)):
            want = f().dlogits
            f(dlogits=dl)
            assert torch.equal(dl, want)


@pytest.mark.parametrize("V", [200, 9000, 70000])
def test_policy_reference_without_a_coefficient(V):
    """kl_coef = 0 with a reference whose distance is beyond the exponential's range: the loss and the gradient are
    those without a reference, and the KL sum alone is infinite."""
    M = 8
    l = torch.randn((M, V), device="cuda")
    y = torch.arange(M, device="cuda")
    w = torch.ones(M, device="cuda")
    old = ops.token_logprob(l, y) - 0.1
    for far in (old + 100, old + 1000, old.new_full((M,), 1e30)):
        a = ops.policy_loss(l, y, w, w, old, None)
        b = ops.policy_loss(l, y, w, w, old, far, kl_coef=0.0)
        assert torch.isfinite(a.dlogits).all() and torch.equal(a.dlogits, b.dlogits) and torch.equal(a.logp, b.logp)
        assert torch.equal(a.stats[[0, 1, 3]], b.stats[[0, 1, 3]]) and b.stats[2] == float("inf")


@pytest.mark.parametrize("V", [200, 9000, 70000])
def test_policy_ratio_beyond_the_range(V):
    """A ratio above the largest fp32 number: nothing at advantage 0, the clipped term where it is the smaller one,
    infinite where it is not; and a NaN among the logits stays one at advantage 0."""
    M = 8
    l = torch.randn((M, V), device="cuda")
    y = torch.arange(M, device="cuda")
    w = torch.ones(M, device="cuda")
    old = ops.token_logprob(l, y) - 100
    o = ops.policy_loss(l, y, 0 * w, w, old, None)
    assert (o.stats == 0).all() and (o.dlogits == 0).all()
    o = ops.policy_loss(l, y, w, w, old, None, clip_high=0.25)
    assert o.stats.tolist() == [-10.0, -10.0, 0.0, 8.0] and (o.dlogits == 0).all()
    o = ops.policy_loss(l, y, -w, w, old, None)
    assert (o.stats[:2] == float("inf")).all() and o.stats[3] == 0
    l[3, V - 1] = float("nan")
    o = ops.policy_loss(l, y, 0 * w, w, old, None)
    assert torch.isnan(o.stats[:2]).all() and torch.isnan(o.dlogits[3]).all() and (o.dlogits[[0, 1, 2, 4, 5, 6, 7]] == 0).all()


@pytest.mark.parametrize("M,P", [(8, 2), (600, 3)])
@pytest.mark.parametrize("kind", [ops.QLORA_PREF_SIGMOID, ops.QLORA_PREF_HINGE, ops.QLORA_PREF_IPO])
def test_a_nan_shows_in_its_pair_alone(kind, M, P):
    """A NaN logit in a row that counts: its pair's gradient and rewards and the loss are NaN, the other pairs' not."""
    l = torch.randn((M, 200), device="cuda")
    l[0, 3] = float("nan")
    y = torch.arange(M, device="cuda") % 200
    cu = torch.linspace(0, M, 2 * P + 1, device="cuda").int()
    o = ops.preference_loss(l, y, cu, None, 0.1, kind=kind)
    a, b = int(cu[1]), int(cu[2])
    assert torch.isnan(o.loss) and torch.isnan(o.rewards[0]) and torch.isfinite(o.rewards[1:]).all()
    assert torch.isnan(o.dlogits[:b]).all() and torch.isfinite(o.dlogits[b:]).all()
    assert torch.isnan(o.logp[0]) and torch.isfinite(o.logp[1:]).all() and a < b


@pytest.mark.parametrize("M", [4, 600])
@pytest.mark.parametrize("eps", [0.0, 1.0])
def test_preference_target_of_probability_zero(eps, M):
    """A target at -inf makes its sequence's reward -inf.  The side of the smoothed loss that has no weight may then be
    infinite without a trace: with all weight on the other label the loss is that of -z."""
    l = torch.randn((M, 200), device="cuda")
    y = torch.arange(M, device="cuda") % 200
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    worse = 0 if eps else 1                                    # the sequence whose loss of probability is no loss
    base = ops.preference_loss(l[2:4], y[2:4], cu[:3], None, 0.1, label_smoothing=eps)
    l[worse, worse] = -float("inf")
    o = ops.preference_loss(l, y, cu, None, 0.1, label_smoothing=eps)
    assert o.rewards[worse] == -float("inf") and torch.isfinite(o.rewards[1 - worse])
    assert abs(2 * o.loss.item() - base.loss.item()) <= 1e-6
    assert (o.dlogits[:2] == 0).all() and torch.isfinite(o.dlogits).all()


@pytest.mark.parametrize("M,P", [(700, 20), (700, 32), (700, 33), (520, 300), (4000, 2100)])
def test_every_pair_is_taken(M, P):
    """Short pairs of every number that the blocks of either width share out: each one's rewards and gradient."""
    g = np.random.default_rng(P)
    l = torch.from_numpy(g.standard_normal((M, 40)).astype(np.float32)).cuda()
    yn = g.integers(0, 40, M)
    cu = np.sort(g.integers(0, M + 1, 2 * P + 1)).astype(np.int32)
    o = ops.preference_loss(l, torch.from_numpy(yn).cuda(), torch.from_numpy(cu).cuda(), None, 0.1)
    loss, rewards, lp, dl, d = tr.preference_loss(l.double().cpu().numpy(), yn, cu, None, 0.1, 0)
    n = np.diff(cu)
    # beta = 0.1 times a log-probability's 1e-5 a row; the derivative moves by beta times as much
    assert (np.abs(o.rewards.cpu().numpy() - rewards) <= 1e-6 * n + 2 * U * np.abs(rewards)).all()
    e = 0.1 * 1e-6 * (n[0::2] + n[1::2]).max() / P
    assert (np.abs(o.dlogits.cpu().numpy() - dl) <= 5e-5 * np.abs(d)[:, None] + e).all()


@pytest.mark.parametrize("dtype,M,V,P", [("bf16", 255, 32768, 4), ("bf16", 256, 32768, 4), ("bf16", 257, 32768, 4),
                                         ("fp32", 32, 131072, 1), ("fp32", 33, 131072, 1)])
def test_preference_on_both_sides_of_the_few_rows(dtype, M, V, P):
    """Around the bytes of logits up to which the pair terms are taken by the gradient's CTAs: one call against one
    call a pair, each of them within that bound."""
    l = (torch.randn((M, V), device="cuda") * 2).to(DT[dtype])
    y = torch.arange(M, device="cuda") * 37 % V
    y[::6] = -100
    cu = torch.linspace(0, M - 1, 2 * P + 1, device="cuda").int()
    o = ops.preference_loss(l, y, cu, None, 0.05)
    losses = []
    for p in range(P):
        a, b = int(cu[2 * p]), int(cu[2 * p + 2])
        s = ops.preference_loss(l[a:b], y[a:b], cu[2 * p:2 * p + 3] - a, None, 0.05)
        losses.append(s.loss.item())
        # log-probabilities are off by 1e-5 on either side (sums in another order), a sequence's by that times its rows
        e = 2e-5 * (b - a)
        assert torch.allclose(o.rewards[2 * p:2 * p + 2], s.rewards, rtol=1e-6, atol=0.05 * e)
        d = (o.dlogits[a:b].float() * P - s.dlogits.float()).abs()
        # g moves by beta^2 / 4 of it; p by 2e-5 of itself; two roundings of the type, one of them of the P-th part
        assert (d <= (2.5 * HALF[dtype] + 4e-5) * s.dlogits.float().abs() + 0.05 ** 2 / 4 * e).all()
    assert abs(o.loss.item() - np.mean(losses)) <= 0.05 * 2e-5 * M
    assert (o.dlogits[M - 1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_far_rows_in_place(M, V, dtype):
    """Rows far from 0 among ordinary ones, the gradient over the logits and captured: bit for bit the one elsewhere."""
    l = torch.randn((M, V), device="cuda")
    l[::3] = l[::3].mul(1e7).sub(1e9)
    l[1::3] = -1e9
    l = l.to(DT[dtype])
    y = torch.arange(M, device="cuda") * 31 % V
    w = torch.rand(M, device="cuda") + 0.5
    cu = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    ws = ops.loss_workspace(M)
    for f in (lambda t, **k: ops.policy_loss(t, y, -w, w, None, None, ws=ws, **k),
              lambda t, **k: ops.preference_loss(t, y, cu, None, 0.1, average=True, ws=ws, **k)):
        want = f(l)
        t = l.clone()
        got = f(t, dlogits=t)
        assert torch.equal(want.dlogits, got.dlogits) and torch.equal(want.logp, got.logp)
        assert torch.isfinite(want.dlogits).all() and torch.isfinite(want.logp).all()
        t.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = f(t, dlogits=t)
        for _ in range(2):
            t.copy_(l)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(want.dlogits, t) and torch.equal(want.logp, got.logp)
    assert ops.qlora_device_status() == 0
