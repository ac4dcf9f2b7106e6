"""Pins of the oracle of the 8-bit checkpoints and the losses (CPU)."""
import numpy as np
import pytest
import torch

from oracle import training as tr


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def test_e4m3_table_is_torch_float8():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, tr.e4m3_values(), equal_nan=True)


@pytest.mark.parametrize("fmt", [tr.INT8, tr.E4M3])
def test_act8_every_code_round_trips(fmt):
    """A block whose largest code uses the top of the range comes back code for code."""
    top = 127 if fmt == tr.INT8 else 126                        # 127, 448
    codes = np.concatenate([np.arange(top + 1), np.arange(129 if fmt == tr.INT8 else 128, 255)]).astype(np.uint8)
    codes = codes[:len(codes) // 31 * 31].reshape(-1, 31)
    codes = np.concatenate([np.full((len(codes), 1), top, np.uint8), codes], 1)
    codes = np.concatenate([codes, codes], 1)
    for sb in (7, 127, 200):
        s = np.full((len(codes), 2), sb, np.uint8)
        x = tr.act8_values(codes, s, fmt)
        c2, s2 = tr.act8_quantize(x, fmt)
        assert np.array_equal(s2, s) and np.array_equal(tr.act8_values(c2, s2, fmt), x)


@pytest.mark.parametrize("fmt", [tr.INT8, tr.E4M3])
@pytest.mark.parametrize("std", [1e-39, 1e-30, 1.0, 1e30])
def test_act8_error_bound_and_bf16_values(fmt, std):
    x = _bf16(np.random.default_rng(1).standard_normal((16, 256)) * std).double().numpy()
    c, s = tr.act8_quantize(x, fmt)
    v = tr.act8_values(c, s, fmt)
    assert np.array_equal(_bf16(v).double().numpy(), v)         # exact in bf16
    amax = np.abs(x).reshape(16, 8, 32).max(-1).repeat(32, 1)
    step = 2.0 ** (s.astype(np.float64) - 127).repeat(32, 1)
    if fmt == tr.INT8:
        # half a step; s = 0 blocks have steps of 2^-127, above amax / 64
        assert (np.abs(v - x) <= np.maximum(amax / 128, step / 2)).all()
    else:
        assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10)).all()
        q = torch.from_numpy(x / step).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(q, c)


def test_act8_special_blocks():
    x = np.zeros((1, 128))
    x[0, 32] = np.inf
    x[0, 64] = np.nan
    x[0, 96] = 127.5
    for fmt in (tr.INT8, tr.E4M3):
        c, s = tr.act8_quantize(x, fmt)
        assert list(s[0, :3]) == [0, 255, 255] and (c[0, :96] == 0).all()
        v = tr.act8_values(c, s, fmt)
        assert (v[0, :32] == 0).all() and np.isnan(v[0, 32:96]).all()
    assert tr.act8_values(*tr.act8_quantize(x, tr.INT8), tr.INT8)[0, 96] == 127


def _case(seed=0, M=24, V=37):
    g = np.random.default_rng(seed)
    l = g.standard_normal((M, V)) * 2
    y = g.integers(0, V, M)
    y[::7] = -100
    y[5] = V
    return g, l, y


def test_logprob_is_torch_log_softmax():
    _, l, y = _case()
    lp, ls, live = tr.token_logprob(l, y, 0.7)
    ref = torch.log_softmax(torch.from_numpy(l) * 0.7, -1).numpy()
    assert np.allclose(ls[live], ref[live], rtol=0, atol=1e-13) and (lp[~live] == 0).all()


def _differences(f, l, h=1e-6):
    out = np.zeros_like(l)
    for i in np.ndindex(*l.shape):
        a, b = l.copy(), l.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


@pytest.mark.parametrize("kind,eps,margin,average", [(0, 0.0, 0.0, False), (0, 0.1, 0.3, True), (1, 0.0, 0.2, False),
                                                     (2, 0.0, 0.0, True), (2, 0.0, 0.0, False)])
def test_preference_gradient_by_differences(kind, eps, margin, average):
    g, l, y = _case(kind + 1, 16, 9)
    ref = g.standard_normal(16) - 2
    cu = np.array([0, 4, 7, 7, 14])                              # an empty sequence; rows 14, 15 in none
    kw = dict(eps=eps, margin=margin, average=average, tau=1.25)
    _, _, _, dl, _ = tr.preference_loss(l, y, cu, ref, 0.4, kind, **kw)
    num = _differences(lambda x: tr.preference_loss(x, y, cu, ref, 0.4, kind, **kw)[0], l)
    assert np.abs(dl - num).max() < 1e-7
    assert (dl[14:] == 0).all()


def test_policy_gradient_by_differences():
    g, l, y = _case(9, 16, 9)
    lp = tr.token_logprob(l, y, 0.8)[0]
    old, ref = lp + g.choice([-0.6, -0.1, 0.1, 0.6], 16), lp + 0.3 * g.standard_normal(16)
    adv, w = g.standard_normal(16), g.random(16) / 16
    w[3] = 0
    args = (adv, w, old, ref, 0.2, 0.28, 0.3, 0.8)
    stats, _, dl, _ = tr.policy_loss(l, y, *args)
    num = _differences(lambda x: tr.policy_loss(x, y, *args)[0][0], l)
    assert np.abs(dl - num).max() < 1e-7
    assert (dl[3] == 0).all()


@pytest.mark.parametrize("shift,adv,clipped", [(0.5, 1.0, 1), (0.5, -1.0, 0), (-0.5, 1.0, 0), (-0.5, -1.0, 1),
                                               (0.1, 1.0, 0), (-0.1, -1.0, 0)])
def test_policy_clipping_cases(shift, adv, clipped):
    """One row on each side of each border: which term is taken, and whether it has a gradient."""
    l = np.random.default_rng(3).standard_normal((2, 5))
    y = np.array([1, 2])
    lp = tr.token_logprob(l, y)[0]
    stats, _, dl, d = tr.policy_loss(l, y, np.full(2, adv), np.full(2, 0.5), lp - shift, None)
    rho = np.exp(shift)
    taken = np.clip(rho, 0.8, 1.2) if clipped else rho
    assert np.allclose(stats, [-taken * adv, -taken * adv, 0, clipped], atol=1e-12)
    assert np.allclose(d, 0.0 if clipped else -rho * adv / 2, atol=1e-12)
