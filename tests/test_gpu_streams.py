"""Calls on a stream that is not the current one: what they allocate is not in use anywhere else, before or after."""
import pytest
import torch

from bit_nf4_quantized_quant_b200 import _ops as ops
from bit_nf4_quantized_quant_b200 import inputs

pytestmark = pytest.mark.gpu
M, V, N, K, R = 2000, 64, 256, 512, 16
WAIT = int(1e8)                                  # cycles: some 50 ms, far longer than the host needs to queue a call


def _calls():
    """name -> (call with keyword stream, its outputs as a list, bytes of its workspace)."""
    l = torch.randn((M, V), device="cuda")
    y = torch.arange(M, device="cuda") % V
    w = torch.rand(M, device="cuda")
    adv = w - 0.5
    cu = torch.tensor([0, 700, 1500], dtype=torch.int32, device="cuda")
    X = torch.randn((M, K), device="cuda").bfloat16()
    x8 = ops.act8_quantize(X)
    W = ops.nf4_quantize_dq(inputs.weight(3, 0, N, K, 0.05).cuda())
    A, B = (torch.randn(s, device="cuda").mul_(0.1).bfloat16() for s in ((R, K), (N, R)))
    dY = torch.randn((M, N), device="cuda").bfloat16()
    lw = ops.loss_workspace_bytes(M)

    def pref(**k):
        o = ops.preference_loss(l, y, cu, None, 0.1, **k)
        return [o.loss, o.rewards, o.logp, o.dlogits]

    def policy(**k):
        o = ops.policy_loss(l, y, adv, w, None, None, **k)
        return [o.stats, o.logp, o.dlogits]

    def quantize(**k):
        o = ops.act8_quantize(X, **k)
        return [o.codes, o.scales]

    X1, wt = X[:16], inputs.weight(3, 0, N, K, 0.05).cuda()
    bf, dropped = ops.qlora_workspace_bytes, ops.qlora_dropout_workspace_bytes

    def weight(f):
        def call(**k):
            o = f(**k)
            return [o.packed, o.codes, o.scale, o.mean]
        return call, 0

    older = {"nf4_quantize_dq": weight(lambda **k: ops.nf4_quantize_dq(wt, **k)),
             "quant4_quantize_dq": weight(lambda **k: ops.quant4_quantize_dq(wt, ops.QLORA_QUANT_FP4, **k)),
             "nf4_dequant": (lambda **k: [ops.nf4_dequant(W, **k)], 0),
             "nf4_dequant_merge": (lambda **k: [ops.nf4_dequant_merge(W, A, B, 2.0, **k)], 0),
             "qlora_linear_fwd": (lambda **k: [ops.qlora_linear_fwd(X, W, A, B, 2.0, **k)], bf(M, N, K, R)),
             "qlora_linear_fwd of 16": (lambda **k: [ops.qlora_linear_fwd(X1, W, A, B, 2.0, **k)], bf(16, N, K, R)),
             "qlora_linear_bwd": (lambda **k: list(ops.qlora_linear_bwd(X, dY, W, A, B, 2.0, **k)), bf(M, N, K, R)),
             "qlora_linear_fwd_dropout": (lambda **k: [ops.qlora_linear_fwd_dropout(X, W, A, B, 2.0, 0.1, 1, 0, **k)],
                                          dropped(M, N, K, R)),
             "qlora_linear_bwd_dropout": (lambda **k: list(ops.qlora_linear_bwd_dropout(X, dY, W, A, B, 2.0, 0.1, 1, 0,
                                                                                        **k)), dropped(M, N, K, R))}
    return {**older, "token_logprob": (lambda **k: [ops.token_logprob(l, y, **k)], 0),
            "preference_loss": (pref, lw), "policy_loss": (policy, lw),
            "act8_quantize": (quantize, 0), "act8_dequant": (lambda **k: [ops.act8_dequant(x8, **k)], 0),
            "qlora_linear_bwd_act8": (lambda **k: list(ops.qlora_linear_bwd_act8(x8, dY, W, A, B, 2.0, **k)),
                                      ops.qlora_act8_workspace_bytes(M, N, K, R))}


NAMES = ["token_logprob", "preference_loss", "policy_loss", "act8_quantize", "act8_dequant", "qlora_linear_bwd_act8",
         "nf4_quantize_dq", "quant4_quantize_dq", "nf4_dequant", "nf4_dequant_merge", "qlora_linear_fwd",
         "qlora_linear_fwd of 16", "qlora_linear_bwd", "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout"]


def _blocks(outs, ws):
    """Blocks of the sizes that the call allocates, more of each than the pool is likely to hold."""
    sizes = [t.numel() * t.element_size() for t in outs] + ([ws] if ws else [])
    return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(16)]


@pytest.mark.parametrize("name", NAMES)
def test_blocks_in_use_on_the_current_stream_are_not_taken(name):
    """Blocks are freed on the current stream while it still has to write them; a call on another stream that were
    given one would have its results, or its workspace, overwritten."""
    call, ws = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    for _ in range(2):
        torch.cuda.synchronize()
        blocks = _blocks(want, ws)
        torch.cuda.synchronize()
        torch.cuda._sleep(WAIT)
        for b in blocks:
            b.fill_(0x55)
        del b, blocks
        got = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", NAMES)
def test_workspace_is_not_reused_while_the_call_runs(name):
    """The call waits on its stream; what the current stream allocates and writes meanwhile is not its workspace."""
    call, ws = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(stream=side)
    for b in _blocks(want, ws):
        b.fill_(0x55)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_reused_while_the_current_stream_reads_them(name):
    """Outputs are read on the current stream and dropped; the other stream's next blocks are not theirs until then."""
    call, ws = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    kept = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        for b in _blocks(want, ws):
            b.fill_(0x55)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))
