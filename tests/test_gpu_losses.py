"""Log-probabilities, preference loss and policy loss on the GPU against their fp64 definitions.

Tolerances, from the kernels' fp32 arithmetic (u = 2^-24):
  logp:  a thread adds at most about 40 terms one after another, 14 levels of merging follow, every term is off
         by the exponent's rounding (at most 3 u |t| for exponent t, and |t| 2^t <= 1) and the 2^-22 of the
         hardware exponential; together below 1e-5.  The subtraction, the product with the scale and the last
         rounding add 4 u (|logp| + |scale (l_y - r)|).
  dlogits = g (1[v = y] - p): p is off by the same 1e-5 and by 3 u |t| of itself (|t| < 200 here: 4e-5 more),
         so |g| p 6e-5, plus the relative error of g, plus half a step of the output type (2^-8, 2^-24) and what
         flushes to zero (2^-126 |g|).
  g:     the loss's derivative moves with the error of the log-probabilities it sees (bound given per test).
"""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops
from oracle import training as tr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": U}
E_LP = 1e-5


def _make(seed, M, V, dtype, ld=None, off=0, std=3.0):
    """Logits [M, V] at an element offset in rows of ld, and targets with some rows out of play."""
    g = np.random.default_rng(seed)
    ld = ld or V
    buf = torch.full((off + M * ld,), 777.0, dtype=DT[dtype], device="cuda")
    l = buf.as_strided((M, V), (ld, 1), off)
    l.copy_(torch.from_numpy((g.standard_normal((M, V)) * std).astype(np.float32)).to(DT[dtype]))
    y = g.integers(0, V, M)
    for i in range(M):
        if g.random() < 0.7:
            l[i, y[i]] += 6.0
    y[2::5] = -100
    if M > 8:
        y[7] = V
        y[8] = -1
    return g, buf, l, torch.from_numpy(y).cuda(), l.double().cpu().numpy(), y


def _check_logp(lp, l64, y, tau):
    ref, ls, live = tr.token_logprob(l64, y, tau)
    safe = np.where(live, y, 0)
    d = tau * (l64[np.arange(len(y)), safe] - l64.max(-1))
    lim = np.where(live, E_LP + 4 * U * (np.abs(ref) + np.abs(d)), 0.0)
    got = lp.double().cpu().numpy()
    assert (np.abs(got - ref) <= lim).all(), np.abs(got - ref).max()
    return ref, ls, live


def _check_grad(dl, want, ls, d, tau, dtype, e_g):
    """want: exact gradient; d: exact d loss / d logp [M]; e_g: absolute error allowed to d."""
    got = dl.double().cpu().numpy()
    p = np.exp(np.nan_to_num(ls, nan=-np.inf, neginf=-np.inf))
    g = np.abs(d)[:, None] * tau
    e = np.broadcast_to(np.asarray(e_g), d.shape)[:, None] * tau
    lim = g * p * 6e-5 + e * np.where(want != 0, 1.0, 0.0) + HALF[dtype] * np.abs(want) + (g + e) * 2.0 ** -126
    bad = ~(np.abs(got - want) <= lim * 1.0001)
    assert not bad.any(), (bad.sum(), np.abs(got - want)[bad].max(), np.argwhere(bad)[:3])


SHAPES = [(1, 1), (3, 2), (5, 7), (9, 8), (12, 9), (6, 15), (4, 63), (40, 500), (33, 1000), (11, 4097), (7, 8192),
          (37, 32001), (150, 20000), (600, 2050), (2, 131072), (1, 262144)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_logprob(M, V, dtype):
    for tau in (1.0, 0.6):
        _, _, l, y, l64, yn = _make(M + V, M, V, dtype)
        _check_logp(ops.token_logprob(l, y, tau), l64, yn, tau)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ld,off", [(1003, 0), (1003, 1), (1024, 3), (1007, 7), (1001, 8)])
def test_logprob_rows_at_any_alignment(ld, off, dtype):
    _, _, l, y, l64, yn = _make(ld + off, 21, 1001, dtype, ld, off)
    _check_logp(ops.token_logprob(l, y), l64, yn, 1.0)


def _masked_rows(dtype, V):
    """Rows with -inf entries, of the type's lowest value, of one finite entry, without any; a target at -inf; NaN
    and +inf rows; rows out of play that hold NaN; values beyond 2^100 on both sides."""
    low, big = torch.finfo(DT[dtype]).min, 2.0 ** 110
    inf = float("inf")
    l = torch.from_numpy(np.random.default_rng(4).standard_normal((12, V)).astype(np.float32)).to(DT[dtype])
    y = np.array([5, 5, 5, 5, 5, 5, 5, -100, V + 3, 5, 5, 5])
    l[0, 6:] = -inf
    l[1] = low
    l[2] = -inf
    l[2, 5] = -3.0
    l[3] = -inf
    l[4, 5] = -inf
    l[5, 8] = float("nan")
    l[6, 9] = inf
    l[7] = float("nan")
    l[8] = inf
    l[9, 10:200] = low
    l[10] = -big
    l[10, ::2] = -2 * big                                       # only entries beyond the range: half of them lead
    l[11] = 1.0
    l[11, 5] = big
    return l.cuda(), torch.from_numpy(y).cuda(), y


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [300, 5000, 40000])
def test_masked_rows(V, dtype):
    l, y, yn = _masked_rows(dtype, V)
    M = len(yn)
    lp = ops.token_logprob(l, y).cpu().numpy().astype(np.float64)
    l64 = l.double().cpu().numpy()
    ref, ls, live = tr.token_logprob(l64, yn)
    assert np.isnan(lp[[3, 5, 6]]).all() and np.isnan(ref[[3, 5, 6]]).all()
    # (row 2, one finite entry: 0 within E_LP like any other, by the check below, and never above 0)
    assert lp[4] == -np.inf and lp[2] <= 0 and lp[7] == 0 and lp[8] == 0
    assert abs(lp[10] + np.log(V // 2)) <= E_LP and abs(lp[11]) <= E_LP     # 5 is one of row 10's V / 2 leaders
    assert abs(lp[1] + np.log(V)) <= E_LP
    ok = [0, 1, 2, 9, 10, 11]
    assert (np.abs(lp[ok] - ref[ok]) <= E_LP + 4 * U * np.abs(ref[ok])).all()
    # the gradient of a sum of log-probabilities, by a policy loss with ratio 1 and advantage -1
    ones = torch.ones(M, device="cuda")
    out = ops.policy_loss(l, y, -ones, ones, None, None)
    # and by the chosen sequences of an IPO loss: d loss / d delta = 2 (delta - 1 / (2 beta)), one pair a row
    for r in (0, 1, 2, 4, 9, 10, 11):
        want = np.exp(ls[r])
        want = np.where(np.arange(V) == yn[r], 1.0, 0.0) - want
        grads = [out.dlogits[r]]
        if r != 4:
            cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
            pair = torch.stack([l[r], l[0]])
            o = ops.preference_loss(pair, y[[r, 7]], cu, None, 0.5, kind=ops.QLORA_PREF_IPO)
            grads.append(o.dlogits[0].float() / (2 * (ref[r] - 1.0)))
        for g in grads:
            # the second gradient was divided by a factor that is off by 2 E_LP of 2 or more, and rounded before that
            lim = np.exp(ls[r]) * 6e-5 + (HALF[dtype] + 2 * E_LP) * np.abs(want) + 2.0 ** -126
            assert (np.abs(g.double().cpu().numpy() - want) <= lim).all(), r
    g = out.dlogits.double().cpu().numpy()
    assert np.isnan(g[[3, 5, 6]]).all() and (g[[7, 8]] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", [(1500, 700), (1400, 5003), (1300, 20001), (700, 40003)])
def test_in_place_equals_out_of_place(M, V, dtype):
    """Many rows of every kernel's width: the gradient over the logits, bit for bit the one written elsewhere."""
    l = (torch.randn((M, V), device="cuda") * 3).to(DT[dtype])
    y = torch.randint(0, V, (M,), device="cuda")
    y[::5] = -100
    w = torch.rand(M, device="cuda")
    w[1::7] = 0
    cu = torch.linspace(0, M - 3, 21, device="cuda").int()
    for f in (lambda t, **k: ops.policy_loss(t, y, w - 0.5, w, None, None, **k),
              lambda t, **k: ops.preference_loss(t, y, cu, None, 0.01, **k)):
        a = f(l)
        t = l.clone()
        b = f(t, dlogits=t)
        assert torch.equal(a.dlogits, b.dlogits) and torch.equal(a.logp, b.logp)
        assert torch.isfinite(a.dlogits).all() and (a.dlogits[::5] == 0).all()


# ------------------------------------------------------------------ preference
def _pairs(g, M, P, tail):
    cuts = np.sort(g.integers(0, M - tail + 1, 2 * P - 1))
    return np.concatenate([[0], cuts, [M - tail]]).astype(np.int32)


KINDS = [(ops.QLORA_PREF_SIGMOID, 0.0, 0.0, False), (ops.QLORA_PREF_SIGMOID, 0.15, 0.4, True),
         (ops.QLORA_PREF_HINGE, 0.0, 0.3, False), (ops.QLORA_PREF_IPO, 0.0, 0.0, False),
         (ops.QLORA_PREF_IPO, 0.0, 0.0, True)]


def _run_preference(seed, M, V, P, dtype, kind, eps, margin, average, ld=None, off=0, tau=1.0, beta=0.1, ref_free=False,
                    inplace=False):
    g, buf, l, y, l64, yn = _make(seed, M, V, dtype, ld, off)
    cu = _pairs(g, M, P, M // 10)
    lp0 = tr.token_logprob(l64, yn, tau)[0]
    ref = None if ref_free else (lp0 + 0.3 * g.standard_normal(M)).astype(np.float32)
    if ref is not None:
        ref[~((yn >= 0) & (yn < V))] = np.nan                  # never read there
    before = buf.clone()
    o = ops.preference_loss(l, y, torch.from_numpy(cu).cuda(), None if ref is None else torch.from_numpy(ref).cuda(),
                            beta, kind=kind, label_smoothing=eps, margin=margin, average=average, logit_scale=tau,
                            grad_scale=0.5, dlogits=l if inplace else None)
    torch.cuda.synchronize()
    r64 = None if ref is None else np.nan_to_num(ref.astype(np.float64))
    loss, rewards, lp, dl, d = tr.preference_loss(l64, yn, cu, r64, beta, kind, eps, margin, average, tau, 0.5)
    _, ls, live = _check_logp(o.logp, l64, yn, tau)
    # a sequence's sum is off by the errors of its log-probabilities
    e_lp = E_LP + 4 * U * (np.abs(lp) + 60 * tau)
    n = np.diff(cu)
    e_s = np.array([e_lp[a:b][live[a:b]].sum() / (max(live[a:b].sum(), 1) if average else 1)
                    for a, b in zip(cu[:-1], cu[1:])])
    assert (np.abs(o.rewards.double().cpu().numpy() - rewards) <= beta * e_s + 2 * U * np.abs(rewards)).all()
    e_d = e_s[0::2] + e_s[1::2]
    delta = (rewards[0::2] - rewards[1::2]) / beta
    if kind == ops.QLORA_PREF_IPO:
        e_loss, e_g = 2 * np.abs(delta - 0.5 / beta) * e_d + e_d ** 2, 2 * e_d
    else:
        z = beta * delta - margin
        assert kind != ops.QLORA_PREF_HINGE or (np.abs(z - 1) > beta * e_d).all()      # no pair on the corner
        e_loss, e_g = beta * e_d, beta ** 2 * e_d * (0 if kind == ops.QLORA_PREF_HINGE else 1)
    assert abs(o.loss.item() - loss) <= e_loss.mean() + 2 * U * abs(loss)
    row_e = np.zeros(M)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        row_e[a:b] = e_g[i // 2] / P * 0.5 / (max(live[a:b].sum(), 1) if average else 1)
    _check_grad(o.dlogits, dl, ls, d, tau, dtype, row_e + 3 * U * np.abs(d))
    if not inplace:
        assert torch.equal(buf, before)
    return o, l, buf, before


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,eps,margin,average", KINDS)
@pytest.mark.parametrize("M,V,P", [(2, 5, 1), (30, 129, 1), (60, 1000, 4), (200, 2048, 9), (70, 32001, 2), (512, 70, 32),
                                   (400, 129, 40), (513, 300, 5), (600, 1003, 33)])
def test_preference(M, V, P, kind, eps, margin, average, dtype):
    _run_preference(M + V + kind, M, V, P, dtype, kind, eps, margin, average)


# more rows than the few-rows kernel takes (M, V, P, type, kind, eps, average, ld, off)
LARGE = [(2100, 16400, 7, "bf16", 0, 0.1, False, 16400, 0), (530, 65537, 3, "bf16", 2, 0.0, True, 65537, 0),
         (4100, 4100, 40, "fp32", 1, 0.0, False, 4103, 1), (600, 32001, 60, "bf16", 0, 0.0, True, 32010, 3)]


# many short rows (a warp each), and rows around the lengths that take one vector a thread or one chunk more
WIDTHS = [(2500, 600, 5, "bf16", 0, 0.0, False, 603, 1), (2500, 5120, 33, "bf16", 1, 0.0, True, 5120, 0),
          (2500, 2559, 33, "fp32", 0, 0.1, False, 2561, 1), (700, 513, 40, "fp32", 2, 0.0, True, 513, 0),
          (600, 5135, 33, "bf16", 0, 0.0, False, 5135, 0), (600, 8200, 33, "bf16", 0, 0.1, False, 8200, 0),
          (600, 12288, 33, "bf16", 2, 0.0, True, 12290, 3), (600, 12297, 33, "bf16", 0, 0.0, False, 12297, 0),
          (600, 6145, 33, "fp32", 1, 0.0, False, 6146, 1)]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("M,V,P,dtype,kind,eps,average,ld,off", WIDTHS)
def test_preference_rows_of_every_width(M, V, P, dtype, kind, eps, average, ld, off, inplace):
    _run_preference(M + V, M, V, P, dtype, kind, eps, 0.0, average, ld=ld, off=off, beta=0.02, inplace=inplace)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("M,V,P,dtype,kind,eps,average,ld,off", LARGE)
def test_preference_large(M, V, P, dtype, kind, eps, average, ld, off, inplace):
    o, l, buf, _ = _run_preference(M, M, V, P, dtype, kind, eps, 0.0, average, ld=ld, off=off, beta=0.02,
                                   inplace=inplace)
    if not inplace:
        again, _, _, _ = _run_preference(M, M, V, P, dtype, kind, eps, 0.0, average, ld=ld, off=off, beta=0.02)
        assert torch.equal(o.dlogits, again.dlogits) and torch.equal(o.loss, again.loss)
        assert torch.equal(o.rewards, again.rewards) and torch.equal(o.logp, again.logp)
    assert ops.qlora_device_status() == 0


def test_preference_large_agrees_with_small_calls():
    """Pairs of 1 to 700 rows, rows in no pair before, and masked rows among them, in one large call, against one
    small call for each pair (its gradient there is P times as large)."""
    V, rng = 16384, np.random.default_rng(3)
    cu = np.array([5, 6, 7, 300, 302, 700, 1400, 1400, 1401, 2100, 2500], np.int32)
    P, M = 5, 2520
    l = (torch.randn((M, V), device="cuda") * 3).bfloat16()
    low = torch.finfo(torch.bfloat16).min
    y = torch.from_numpy(rng.integers(0, V, M)).cuda()
    y[::9] = -100
    l[10] = low                                                 # uniform
    l[11, 7:] = -float("inf")
    y[11] = 3
    l[301, 5:900] = low
    l[400] = float("nan")
    y[400] = -1
    ref = torch.from_numpy(rng.standard_normal(M).astype(np.float32) - 9).cuda()
    o = ops.preference_loss(l, y, torch.from_numpy(cu).cuda(), ref, 0.01)
    losses = []
    for p in range(P):
        a, b = int(cu[2 * p]), int(cu[2 * p + 2])
        c = torch.from_numpy(cu[2 * p:2 * p + 3] - a).cuda()
        s = ops.preference_loss(l[a:b], y[a:b], c, ref[a:b], 0.01)
        losses.append(s.loss.item())
        assert torch.allclose(o.rewards[2 * p:2 * p + 2], s.rewards, rtol=1e-5, atol=0.01 * (b - a) * 2 * E_LP)
        d = (o.dlogits[a:b].float() * P - s.dlogits.float()).abs()
        assert (d <= 2.5 * HALF["bf16"] * s.dlogits.float().abs() + 1e-6).all()
        assert torch.allclose(o.logp[a:b], s.logp, rtol=4 * U, atol=2 * E_LP)
    assert abs(o.loss.item() - np.mean(losses)) <= 0.01 * 700 * 4 * E_LP
    assert (o.dlogits[:5] == 0).all() and (o.dlogits[2500:] == 0).all() and (o.dlogits[400] == 0).all()


def test_preference_large_on_two_streams_and_captured():
    """Two calls at once, each of which fills the GPU, and a captured one: the results of one at a time."""
    M, V = 2200, 16384
    sets = [((torch.randn((M, V), device="cuda") * 3).bfloat16(), torch.randint(0, V, (M,), device="cuda")) for _ in range(2)]
    cu = torch.tensor([0, 500, 900, 1500, 2150], dtype=torch.int32, device="cuda")

    def call(s, **k):
        o = ops.preference_loss(s[0], s[1], cu, None, 0.01, **k)
        return [o.loss, o.rewards, o.logp, o.dlogits]

    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [call(s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    l, y = sets[0][0].clone(), sets[0][1].clone()
    ws = ops.loss_workspace(M)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call((l, y), ws=ws)
    for s, ref in zip(sets, want):
        l.copy_(s[0])
        y.copy_(s[1])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert ops.qlora_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_preference_scaled_reference_free_and_unaligned(dtype):
    _run_preference(3, 50, 777, 3, dtype, 0, 0.0, 0.5, True, ld=781, off=3, tau=1.3, beta=2.0, ref_free=True)
    _run_preference(4, 50, 777, 3, dtype, 0, 0.1, 0.0, False, ld=800, off=5, tau=0.7)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_preference_in_place_leaves_the_padding(dtype):
    """Gradient over the logits: equal to the one written elsewhere, and the columns between V and ld stay."""
    kw = dict(kind=0, eps=0.0, margin=0.0, average=False, ld=1031, off=1)
    a, _, _, _ = _run_preference(8, 40, 1001, 3, dtype, **kw)
    b, l, buf, before = _run_preference(8, 40, 1001, 3, dtype, inplace=True, **kw)
    assert torch.equal(a.dlogits, b.dlogits) and b.dlogits.data_ptr() == l.data_ptr()
    assert (buf[1:].view(40, 1031)[:, 1001:] == 777.0).all() and (buf[:1] == 777.0).all()


def test_gradient_rows_at_another_alignment_than_the_logits():
    M, V = 20, 1003
    g, _, l, y, _, _ = _make(5, M, V, "bf16")
    cu = torch.tensor([0, 8, 20], dtype=torch.int32, device="cuda")
    want = ops.preference_loss(l, y, cu, None, 0.1).dlogits
    out = torch.full((M * 1010 + 1,), 5.0, dtype=torch.bfloat16, device="cuda")
    dl = out.as_strided((M, V), (1010, 1), 1)
    ops.preference_loss(l, y, cu, None, 0.1, dlogits=dl)
    assert torch.equal(dl, want)
    assert (out.as_strided((M - 1, 7), (1010, 1), 1 + V) == 5.0).all() and out[0] == 5.0
    w = torch.rand(M, device="cuda")
    want = ops.policy_loss(l, y, w - 0.5, w, None, None).dlogits
    ops.policy_loss(l, y, w - 0.5, w, None, None, dlogits=dl)
    assert torch.equal(dl, want)
    assert (out.as_strided((M - 1, 7), (1010, 1), 1 + V) == 5.0).all() and out[0] == 5.0


def test_preference_many_short_and_few_long_pairs():
    """More pairs than the warps of the cluster, next to pairs of thousands of tokens (V small: the sums count)."""
    g = np.random.default_rng(12)
    lens = g.integers(0, 6, 2 * 700)
    lens[[3, 500, 501, 1399]] = [3000, 1100, 2500, 5000]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    M, V = int(cu[-1]) + 13, 11
    _, _, l, y, l64, yn = _make(13, M, V, "fp32")
    ref = g.standard_normal(M).astype(np.float32) - 2
    o = ops.preference_loss(l, y, torch.from_numpy(cu).cuda(), torch.from_numpy(ref).cuda(), 0.02)
    loss, rewards, lp, dl, d = tr.preference_loss(l64, yn, cu, ref.astype(np.float64), 0.02, 0)
    # the longest pair's sum moves by at most 5000 E_LP, times beta
    e = 0.02 * 5000 * (E_LP + 1e-6)
    assert (np.abs(o.rewards.double().cpu().numpy() - rewards) <= e + 2 * U * np.abs(rewards)).all()
    assert abs(o.loss.item() - loss) <= 2 * e
    _check_grad(o.dlogits, dl, tr.token_logprob(l64, yn)[1], d, 1.0, "fp32", 0.02 * 2 * e / 700)
    again = ops.preference_loss(l, y, torch.from_numpy(cu).cuda(), torch.from_numpy(ref).cuda(), 0.02)
    for a, b in zip((o.loss, o.rewards, o.logp, o.dlogits), (again.loss, again.rewards, again.logp, again.dlogits)):
        assert torch.equal(a, b)


def test_preference_nothing_in_play():
    """No target anywhere: loss ln 2, no reward, no gradient, NaN logits unread."""
    l = torch.full((6, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = torch.full((6,), -100, device="cuda")
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for average in (False, True):
        o = ops.preference_loss(l, y, cu, torch.full((6,), float("nan"), device="cuda"), 0.1, average=average)
        assert abs(o.loss.item() - np.log(2)) < 1e-6
        assert (o.rewards == 0).all() and (o.logp == 0).all() and (o.dlogits == 0).all()


def test_boundaries_outside_the_rows_are_clamped():
    """cu_seqlens is device data: what it holds cannot lead out of the arrays."""
    M, V = 16, 50
    _, _, l, y, _, _ = _make(2, M, V, "fp32")
    bad = torch.tensor([-5, 4, 2, 9, 100], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 4, 4, 9, 16], dtype=torch.int32, device="cuda")
    a = ops.preference_loss(l, y, bad, None, 0.1)
    b = ops.preference_loss(l, y, good, None, 0.1)
    # pair 0 is rows [0, 4) against nothing in both; pair 1's chosen sequence begins at 2 instead of 4
    assert a.rewards[0] == b.rewards[0] and a.rewards[1] == 0 and a.rewards[3] == b.rewards[3]
    assert torch.isfinite(a.loss) and torch.isfinite(a.dlogits).all()


# ------------------------------------------------------------------ policy
def _run_policy(seed, M, V, dtype, tau=1.0, ld=None, off=0, old=True, ref=True, inplace=False, kl=0.05):
    g, buf, l, y, l64, yn = _make(seed, M, V, dtype, ld, off)
    lp0 = tr.token_logprob(l64, yn, tau)[0]
    # ratios inside, above and below the clipping range, none near its borders
    shift = g.choice([-0.5, -0.1, 0.0, 0.1, 0.5], M)
    oldv = (lp0 - shift).astype(np.float32) if old else None
    refv = (lp0 + 0.3 * g.standard_normal(M)).astype(np.float32) if ref else None
    adv = g.standard_normal(M).astype(np.float32)
    w = (g.random(M) / M).astype(np.float32)
    w[1::6] = 0
    dead = (w == 0) | (yn < 0) | (yn >= V)
    for t in (adv, oldv, refv):
        if t is not None:
            t[dead] = np.nan
    cu = lambda t: None if t is None else torch.from_numpy(t).cuda()  # noqa: E731
    o = ops.policy_loss(l, y, cu(adv), cu(w), cu(oldv), cu(refv), 0.2, 0.28, kl, logit_scale=tau, grad_scale=2.0,
                        dlogits=l if inplace else None)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else np.nan_to_num(t.astype(np.float64))  # noqa: E731
    stats, lp, dl, d = tr.policy_loss(l64, yn, f(adv), w.astype(np.float64), f(oldv), f(refv), 0.2, 0.28, kl, tau, 2.0)
    _check_logp(o.logp, l64, np.where(w != 0, yn, -1), tau)
    ls = tr.token_logprob(l64, np.where(dead, -1, yn), tau)[1]
    e_lp = E_LP + 4 * U * (np.abs(lp) + 60 * tau) + 4 * U
    ed = np.exp(np.where(dead, 0, f(refv) - lp)) if ref else np.zeros(M)
    e_pol = np.where(dead, 0, np.abs(f(adv)) * 1.7 * e_lp)
    e_kl = np.where(dead, 0, ed + 1) * e_lp
    e = np.array([(w * (e_pol + kl * e_kl)).sum(), (w * e_pol).sum(), (w * e_kl).sum(), 0.0]) + 8 * U * w.sum()
    assert (np.abs(o.stats.double().cpu().numpy() - stats) <= e + 4 * U * np.abs(stats)).all()
    _check_grad(o.dlogits, dl, ls, d, tau, dtype, 2 * w * (e_pol + kl * e_kl) + 8 * U * np.abs(d) + 8 * U * w * kl)
    return o, l, buf


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SHAPES)
def test_policy(M, V, dtype):
    _run_policy(M + V, M, V, dtype)


@pytest.mark.parametrize("V", [40, 2100, 9000, 20000, 40000])
def test_policy_every_row_is_taken_once(V):
    """Row counts around what the GPU holds at once, and dozens of times that: every row's log-probability and
    gradient row are those of the row alone."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    base, M0 = _make(V, 64, V, "bf16")[2], 64
    y0 = torch.arange(M0, device="cuda") * 13 % V
    w0 = torch.rand(M0, device="cuda") + 0.5
    w0[::9] = 0
    adv0 = torch.randn(M0, device="cuda")
    want = ops.policy_loss(base, y0, adv0, w0, None, None)
    for M in (sms, 2 * sms + 1, 3 * sms - 1, 6 * sms + 5, 9 * sms, 13 * sms + 1):
        if M * V > 3e8:
            continue
        pick = torch.randint(0, M0, (M,), device="cuda")
        o = ops.policy_loss(base[pick], y0[pick], adv0[pick], w0[pick], None, None)
        # a row may be split over another number of CTAs than in the small call: sums in another order
        assert torch.allclose(o.logp, want.logp[pick], rtol=4 * U, atol=E_LP)
        d = (o.dlogits.float() - want.dlogits[pick].float()).abs()
        g = (w0 * adv0.abs())[pick][:, None]
        assert (d <= 2 * HALF["bf16"] * want.dlogits[pick].float().abs() + 1e-4 * g + 1e-30).all()


@pytest.mark.parametrize("dtype,M,V", [("bf16", 300, 8191), ("bf16", 300, 32767), ("bf16", 300, 32776), ("bf16", 3, 65551),
                                       ("bf16", 3, 131080), ("bf16", 3, 262144), ("fp32", 300, 4095),
                                       ("fp32", 300, 16383), ("fp32", 300, 16391), ("fp32", 3, 32779),
                                       ("fp32", 3, 65543), ("fp32", 3, 131072), ("fp32", 40, 131079),
                                       ("fp32", 3, 262144)])
def test_policy_rows_of_every_width(dtype, M, V):
    """Around the lengths from which a row is shared by one CTA more, up to a cluster of 16, at every
    alignment of a row."""
    _run_policy(V, M, V, dtype, ld=V + 5, off=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("old,ref", [(False, False), (True, False), (False, True)])
def test_policy_without_old_or_reference(old, ref, dtype):
    _run_policy(31, 50, 1500, dtype, tau=1.25, old=old, ref=ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,ld,off", [(1001, 1003, 0), (1001, 1024, 3), (40003, 40007, 7)])
def test_policy_in_place_at_any_alignment(V, ld, off, dtype):
    a, _, _ = _run_policy(77, 30, V, dtype, ld=ld, off=off)
    b, l, buf = _run_policy(77, 30, V, dtype, ld=ld, off=off, inplace=True)
    assert torch.equal(a.dlogits, b.dlogits) and torch.equal(a.stats, b.stats)
    assert (buf[off:].view(30, ld)[:, V:] == 777.0).all() and (buf[:off] == 777.0).all()


def test_policy_nothing_in_play():
    l = torch.full((5, 70), float("nan"), dtype=torch.float32, device="cuda")
    y = torch.zeros(5, dtype=torch.int64, device="cuda")
    nan = torch.full((5,), float("nan"), device="cuda")
    o = ops.policy_loss(l, y, nan, torch.zeros(5, device="cuda"), nan, nan, kl_coef=0.1)
    assert (o.stats == 0).all() and (o.logp == 0).all() and (o.dlogits == 0).all()


# ------------------------------------------------------------------ both
def test_loss_without_gradient():
    _, _, l, y, _, _ = _make(6, 40, 900, "bf16")
    cu = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
    w = torch.rand(40, device="cuda")
    for f in (lambda **k: ops.preference_loss(l, y, cu, None, 0.1, **k), lambda **k: ops.policy_loss(l, y, w, w, None, None, **k)):
        a, b = f(), f(want_grad=False)
        assert b.dlogits is None and torch.equal(a.logp, b.logp)
        assert torch.equal(a.loss, b.loss) if hasattr(a, "loss") else torch.equal(a.stats, b.stats)


@pytest.mark.parametrize("V", [900, 33000])
def test_captured_and_on_two_streams(V):
    """A captured loss replays on new logits; two calls at once on two streams agree with one at a time."""
    M = 40
    sets = [_make(s, M, V, "bf16") for s in (1, 2)]
    cu = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
    w = torch.rand(M, device="cuda")

    def both(l, y, ws, **k):
        a = ops.preference_loss(l, y, cu, None, 0.1, ws=ws, **k)
        b = ops.policy_loss(l, y, w - 0.5, w, None, None, ws=ws, **k)
        return [a.loss, a.rewards, a.logp, a.dlogits, b.stats, b.logp, b.dlogits]

    wss = [ops.loss_workspace(M) for _ in range(2)]
    want = [both(s[2], s[3], ws) for s, ws in zip(sets, wss)]
    torch.cuda.synchronize()
    l, y = sets[0][2].clone(), sets[0][3].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(l, y, wss[0])
    for s, ref in zip(sets, want):
        l.copy_(s[2])
        y.copy_(s[3])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [both(s[2], s[3], None, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_past_32_bit_offsets():
    """A gradient row that begins behind element 2^31 of its array (a wide pitch: few rows are touched)."""
    M, V, ld = 5, 1000, (1 << 29) + 40
    buf = torch.empty(((M - 1) * ld + V,), dtype=torch.bfloat16, device="cuda")
    l = buf.as_strided((M, V), (ld, 1), 0)
    small = torch.randn((M, V), device="cuda").to(torch.bfloat16)
    l.copy_(small)
    y = torch.arange(M, device="cuda") * 7
    w = torch.rand(M, device="cuda")
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    a, b = ops.policy_loss(small, y, w - 0.5, w, None, None), ops.policy_loss(l, y, w - 0.5, w, None, None, dlogits=l)
    assert torch.equal(a.dlogits, b.dlogits) and torch.equal(a.stats, b.stats)
    l.copy_(small)
    a, b = ops.preference_loss(small, y, cu, None, 0.1), ops.preference_loss(l, y, cu, None, 0.1, dlogits=l)
    assert torch.equal(a.dlogits, b.dlogits) and torch.equal(a.loss, b.loss)


def test_refusals_on_the_gpu():
    _, _, l, y, _, _ = _make(1, 4, 64, "bf16")
    w = torch.ones(4, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="targets"):
        ops.token_logprob(l, y[:3])
    with pytest.raises(ValueError, match="targets"):
        ops.token_logprob(l, y.int())
    with pytest.raises(ValueError, match="cu_seqlens"):
        ops.preference_loss(l, y, cu[:2], None, 0.1)
    with pytest.raises(ValueError, match="ref_logp"):
        ops.preference_loss(l, y, cu, w.double(), 0.1)
    with pytest.raises(ValueError, match="dlogits"):
        ops.preference_loss(l, y, cu, None, 0.1, dlogits=l.float())
    with pytest.raises(ValueError, match="weights"):
        ops.policy_loss(l, y, w, w[:3], None, None)
    with pytest.raises(ops.QLoRAError) as e:
        ops.policy_loss(l.expand(4, 64)[:1].expand(4, 64), y, w, w, None, None, dlogits=torch.empty_like(l))
    assert e.value.code == -2                                   # rows 0 elements apart
