"""The operators of one training step used together: two adapted layers (the second the output projection), their
inputs kept as 8-bit checkpoints, a preference or a policy loss on the logits, the backward from the checkpoints and
the 8-bit AdamW step of the adapters -- eager, stage by stage against the definitions in fp64, and as one CUDA graph.

Tolerances: an output rounded to bf16 is off by at most 2^-8 of itself, so a product's relative Frobenius error is
below 2^-8 plus its fp32 accumulation (far below): 5e-3.  Through the whole chain the roundings of Y, the logits and
dX (2^-8 each), of the logits' exponentials (the logits are below 4 in magnitude here: 2^-8 4 = 1.6e-2 of a
probability) and of the 8-bit inputs add up: int8 values are off by at most amax / 128 of their block of 32, which is
at most sqrt(32) / 128 = 4.4e-2 of the block's norm, E4M3 values by 2^-4 of themselves; their sum with the roundings is
below 0.1 and 0.13."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops
from bit_nf4_quantized_quant_b200 import inputs
from oracle import training as tr

pytestmark = pytest.mark.gpu
K, H, V, R, S = 256, 512, 1000, 16, 2.0
CHAIN = {ops.QLORA_ACT8_INT8: 0.1, ops.QLORA_ACT8_E4M3: 0.13}


def _rel(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


class Model:
    def __init__(self, M, seed=0):
        self.M = M
        self.X = inputs.normal(100 + seed, (M, K), 1.0).cuda()
        self.w = [ops.nf4_quantize_dq(inputs.weight(101 + seed + i, 0, n, k, 0.03).cuda())
                  for i, (n, k) in enumerate(((H, K), (V, H)))]
        # adapters in one flat parameter buffer: A1, B1, A2, B2
        shapes = [(R, K), (H, R), (R, H), (V, R)]
        g = torch.Generator().manual_seed(7 + seed)
        self.flat = torch.cat([(torch.rand(s, generator=g) * 0.1 - 0.05).flatten() for s in shapes]).bfloat16().cuda()
        self.grad = torch.zeros_like(self.flat)
        n = [a * b for a, b in shapes]
        self.p = [t.view(s) for t, s in zip(self.flat.split(n), shapes)]
        self.g = [t.view(s) for t, s in zip(self.grad.split(n), shapes)]
        rng = np.random.default_rng(seed)
        y = rng.integers(0, V, M)
        y[::6] = -100
        self.y = torch.from_numpy(y).cuda()
        self.cu = torch.tensor([0, M // 4, M // 2, M - M // 3, M - 1], dtype=torch.int32, device="cuda")
        self.old = torch.from_numpy((-7 + 0.5 * rng.standard_normal(M)).astype(np.float32)).cuda()
        self.adv = torch.from_numpy(rng.standard_normal(M).astype(np.float32)).cuda()
        self.wt = torch.full((M,), 1.0 / M, device="cuda")
        self.state = ops.AdamW8State.zeros(self.flat.numel())

    def step(self, loss, fmt, t=1, update=True):
        A1, B1, A2, B2 = self.p
        T1, T2 = (torch.empty((self.M, R), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        Y = ops.qlora_linear_fwd(self.X, self.w[0], A1, B1, S, T_out=T1)
        logits = ops.qlora_linear_fwd(Y, self.w[1], A2, B2, S, T_out=T2)
        q1, q2 = ops.act8_quantize(self.X, fmt), ops.act8_quantize(Y, fmt)
        keep = logits.clone()                                  # the test's copy: the gradient goes over the logits
        if loss == "preference":
            o = ops.preference_loss(logits, self.y, self.cu, self.old, 0.1, dlogits=logits)
            value = o.loss
        else:
            o = ops.policy_loss(logits, self.y, self.adv, self.wt, self.old, self.old, kl_coef=0.05, dlogits=logits)
            value = o.stats
        dY, _, _ = ops.qlora_linear_bwd_act8(q2, o.dlogits, self.w[1], A2, B2, S, T=T2, dA=self.g[2], dB=self.g[3])
        dX, _, _ = ops.qlora_linear_bwd_act8(q1, dY, self.w[0], A1, B1, S, T=T1, dA=self.g[0], dB=self.g[1])
        if update:
            ops.adamw_8bit_step(self.flat, self.grad, self.state, t, 1e-3)
        return dict(Y=Y, logits=keep, dlogits=o.dlogits, dY=dY, dX=dX, loss=value, q1=q1, q2=q2, T1=T1, T2=T2)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _oracle_loss(m, loss, l64, y):
    old = _f64(m.old)
    if loss == "preference":
        value, _, _, dl, _ = tr.preference_loss(l64, y, m.cu.cpu().numpy(), old, 0.1, 0)
    else:
        value, _, dl, _ = tr.policy_loss(l64, y, _f64(m.adv), _f64(m.wt), old, old, 0.2, 0.2, 0.05)
    return value, dl


@pytest.mark.parametrize("fmt", [ops.QLORA_ACT8_INT8, ops.QLORA_ACT8_E4M3])
@pytest.mark.parametrize("loss", ["preference", "policy"])
@pytest.mark.parametrize("M", [24, 96, 300])
def test_gradients_of_the_step(oracle_mod, M, loss, fmt):
    m = Model(M)
    o = m.step(loss, fmt, update=False)
    torch.cuda.synchronize()
    assert ops.qlora_device_status() == 0
    W = [_f64(ops.nf4_dequant(w)) for w in m.w]
    A1, B1, A2, B2 = (_f64(p) for p in m.p)
    X, y = _f64(m.X), m.y.cpu().numpy()
    # stage by stage, each fed with the stage before as the GPU made it
    value, dl = _oracle_loss(m, loss, _f64(o["logits"]), y)
    assert np.allclose(_f64(o["loss"]), value, rtol=1e-4, atol=1e-5)
    assert _rel(_f64(o["dlogits"]), dl) < 5e-3
    x2 = tr.act8_values(o["q2"].codes.cpu().numpy(), o["q2"].scales.cpu().numpy(), fmt)
    x1 = tr.act8_values(o["q1"].codes.cpu().numpy(), o["q1"].scales.cpu().numpy(), fmt)
    g2, gy = _f64(o["dlogits"]), _f64(o["dY"])
    dY, dA2, _ = oracle_mod.linear_bwd(x2, g2, W[1], A2, B2, S)
    dX, dA1, _ = oracle_mod.linear_bwd(x1, gy, W[0], A1, B1, S)
    for got, ref in ((o["dY"], dY), (m.g[2], dA2), (m.g[3], S * g2.T @ _f64(o["T2"])), (o["dX"], dX), (m.g[0], dA1),
                     (m.g[1], S * gy.T @ _f64(o["T1"]))):
        assert _rel(_f64(got), ref) < 5e-3
    # the whole chain in fp64 from X
    Y, T1 = oracle_mod.linear_fwd(X, W[0], A1, B1, S)
    L, T2 = oracle_mod.linear_fwd(Y, W[1], A2, B2, S)
    assert np.abs(L).max() < 4
    _, dl = _oracle_loss(m, loss, L, y)
    dY, dA2, dB2 = oracle_mod.linear_bwd(Y, dl, W[1], A2, B2, S)
    dX, dA1, dB1 = oracle_mod.linear_bwd(X, dY, W[0], A1, B1, S)
    for got, ref in zip(m.g, (dA1, dB1, dA2, dB2)):
        assert _rel(_f64(got), ref) < CHAIN[fmt]


@pytest.mark.parametrize("loss", ["preference", "policy"])
@pytest.mark.parametrize("M", [24, 300])
def test_two_steps_eager_and_captured(oracle_mod, M, loss):
    """Two updates, eager and as replays of one captured step: the same parameters bit for bit, and those of the
    oracle's AdamW step on the GPU's gradients."""
    fmt = ops.QLORA_ACT8_INT8
    a, b = Model(M), Model(M)
    ref, st = inputs.bf16_bits(a.flat).copy(), oracle_mod.adamw8_state(a.flat.numel())
    for t in (1, 2):
        a.step(loss, fmt, t=1)                                 # the step number is a launch argument: 1 in both
        torch.cuda.synchronize()
        oracle_mod.adamw8_step(ref, inputs.bf16_bits(a.grad).copy(), st, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0)
        assert np.array_equal(inputs.bf16_bits(a.flat), ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Model(M).step(loss, fmt)                               # first calls outside the capture
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step(loss, fmt, t=1)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.flat, b.flat) and torch.equal(a.grad, b.grad)
