"""What the losses' fp32 arithmetic keeps: errors on the mean over many rows, and of ratios and gradients, below what any
one of its parts (the second half of the scale, sums in groups, the correction of the hardware exponential, the
log-probability in two fp32) would cost if it were missing.

Bounds, with u = 2^-24:
  mean error of logp: the hardware exponential is low by 2.4e-8 to 6.3e-8 on the mean over a row, 4e-8 are taken off:
         at most 2.3e-8, and 3 standard deviations of what a row's roundings leave of the mean (a sum rounded at 20
         levels by u / sqrt(3) each is off by 1.6e-7: 1.6e-7 / sqrt(rows)).
  g of the policy loss: the sum as above and eight roundings of the row's terms, u / sqrt(3) each: 1.9e-7 together.
  target's gradient: 1.5e-7 for the exponential, 20 additions of at most u / 2 each, 4e-8: 8e-7 of g at most.
"""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _exact(l, y, tau):
    lp = torch.empty(len(l), dtype=torch.float64, device="cuda")
    for i in range(0, len(l), 512):
        d = l[i:i + 512].double() * tau
        lp[i:i + 512] = d.gather(1, y[i:i + 512, None])[:, 0] - torch.logsumexp(d, 1)
    return lp


def _mean_errors(l, y, tau):
    """Of the log-probabilities before their rounding, from the sum that a preference loss makes of them (the reference
    is the exact one, rounded, so that the sum is small), and of the policy loss's."""
    M = len(l)
    lp = _exact(l, y, tau)
    ref = lp.float()
    cu = torch.tensor([0, M, M], dtype=torch.int32, device="cuda")
    s = ops.preference_loss(l, y, cu, ref, 1.0, logit_scale=tau, want_grad=False).rewards[0].item()
    ones = torch.ones(M, device="cuda")
    pol = ops.policy_loss(l, y, ones, ones, None, None, logit_scale=tau, want_grad=False).logp.double()
    return (s - (lp - ref.double()).sum().item()) / M, (pol - lp).mean().item(), lp


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [600, 4000, 32000, 131072])
@pytest.mark.parametrize("std,tau,at", [(0.3, 1.0, 0.0), (1.0, 1.0, 0.0), (2.0, 1.25, 0.0), (5.0, 1.25, 0.0),
                                        (1.0, 1.25, 4096.0)])
def test_mean_error_of_logp(std, tau, at, V, dtype):
    if at and dtype == "bf16":
        at = 64.0                                              # steps of a quarter: a spread is left
    M = min(20000, (1 << 28) // V)
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    l = (torch.randn((M, V), generator=g, device="cuda") * std + at).to(DT[dtype])
    y = torch.randint(0, V, (M,), generator=g, device="cuda")
    pre, pol, lp = _mean_errors(l, y, tau)
    noise = 3 * 1.6e-7 / M ** 0.5
    e = 2.3e-8
    if at and dtype == "bf16":
        # every row holds the same few numbers, at + j / 4 and at + j / 2 for some ten j each, so that its sum's error is
        # the weighted mean of the exponential's errors at some twenty arguments, which need not be that of a binade:
        # each is 1.5e-7 at most, and so is their mean, of which 4e-8 are taken off
        e = 1.5e-7 + 4e-8
    # the policy loss's log-probabilities are rounded to fp32, evenly in both directions
    step = 3 * 2 * U * 2.0 ** np.floor(np.log2(lp.abs().max().item())) / 12 ** 0.5 / M ** 0.5
    assert abs(pre) <= e + noise, (pre, noise)
    assert abs(pol) <= e + noise + step, (pol, noise, step)


@pytest.mark.parametrize("V", [1000, 4000, 32000])
@pytest.mark.parametrize("tau", [1.0, 1.25])
def test_ratio_of_the_policy_loss(tau, V):
    """The ratio exp(logp - old_logp) in the gradient: by the target's entry, whose own probability is small."""
    M = 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    l = torch.randn((M, V), generator=g, device="cuda") * 1.5
    y = torch.randint(0, V, (M,), generator=g, device="cuda")
    lp = _exact(l, y, tau)
    old = (lp + 0.1 * torch.randn(M, generator=g, device="cuda", dtype=torch.float64)).float()
    ones = torch.ones(M, device="cuda")
    got = ops.policy_loss(l, y, -ones, ones, old, None, clip_low=1.0, clip_high=9.0, logit_scale=tau).dlogits
    rho = torch.exp(lp - old.double())
    want = rho * tau * -torch.expm1(lp)
    rel = (got.gather(1, y[:, None])[:, 0].double() - want) / want
    use = lp < -7                                              # p below 1e-3, logp with steps of 4.8e-7 and more
    assert use.sum() > M // 4
    assert rel[use].square().mean().sqrt() <= 1.9e-7
    # the rest of the row: -g p, p off by its own exponential besides (1.5e-7 at most, 0.8e-7 rms)
    off = (y + 1) % V
    p = torch.stack([torch.softmax(l[i:i + 512].double() * tau, 1).gather(1, off[i:i + 512, None])[:, 0]
                     for i in range(0, M, 512)]).flatten()
    rel = (got.gather(1, off[:, None])[:, 0].double() + rho * tau * p) / (rho * tau * p)
    assert rel.square().mean().sqrt() <= (1.9e-7 ** 2 + 0.8e-7 ** 2) ** 0.5 + 3 * U


@pytest.mark.parametrize("V", [1000, 9000, 70000])
@pytest.mark.parametrize("above", [2.0, 12.0, 16.0, 30.0])
def test_target_that_has_almost_all(above, V):
    """A target far above the others: the gradient there, g (1 - p), is right to 8e-7 of g, and 0 or more."""
    M = 512
    l = torch.randn((M, V), device="cuda")
    y = torch.arange(M, device="cuda") * 7 % V
    l[torch.arange(M, device="cuda"), y] = above
    ones = torch.ones(M, device="cuda")
    lp = _exact(l, y, 1.0)
    o = ops.policy_loss(l, y, -ones, ones, None, None)
    cu = torch.arange(M + 1, device="cuda", dtype=torch.int32).repeat_interleave(2)[1:].contiguous()
    q = ops.preference_loss(l, y, cu, None, 0.5, kind=ops.QLORA_PREF_IPO, grad_scale=M)
    for got, g in ((o.dlogits, torch.ones_like(lp)), (q.dlogits, 2 * (lp - 1))):
        e = (got.gather(1, y[:, None])[:, 0].double() - g * -torch.expm1(lp)) / g
        assert e.abs().max() <= 8e-7, e.abs().max()
        assert (got.gather(1, y[:, None])[:, 0].double() * g >= 0).all()
    assert (o.logp <= 0).all() and (q.logp <= 0).all()
    assert (o.logp.double() - lp).abs().max() <= 8e-7 + U * 16
