"""GPU tests of the mixture of experts as it is used: norm, sort, dispatch, the
experts' products, combine and the gradients one after the other, against the
layer in fp32 on the CPU.

Bar: an E4M3 operand is off by 2^-4 at most, 2.6 % in the root mean square; a
product of two such operands by 3.7 % of its norm.  What the experts add to the
stream has three products in a row (gate and up side by side): 6.4 %; the
gradients one or two more quantised operands, about 8 %.  Twice that is allowed.
The gradients of the router and of the weights of its choices are differences
between experts' outputs that are each off by as much: three times."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import moe

pytestmark = pytest.mark.gpu
NAMES = ("w_norm", "b_norm", "router", "w_gate", "w_up", "w_down")


def announce(msg):
    print(f"\n[case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()
    yield
    torch.cuda.synchronize()


def far(a, b):
    a, b = a.detach().float().cpu(), b.detach().float().cpu()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("tokens,G,top_k", [(1, 4, 2), (33, 4, 2), (300, 6, 3), (1000, 3, 1)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_step(tokens, G, top_k, act):
    announce(f"moe step tokens={tokens} G={G} top_k={top_k} {act}")
    H, I = 512, 384
    weights = moe.random_weights(H, I, G, seed=tokens)
    layer = moe.MoEFFN(*weights, top_k=top_k, act=act)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res, dout = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, saved = layer.forward(x, res, save=True)
    dx, grads = layer.backward(saved, dout)
    params = [w.cpu().requires_grad_() for w in weights]
    xr, rr = x.float().cpu().requires_grad_(), res.float().cpu()
    want = moe.reference(*params, xr, rr, saved[2].cpu(), act=act)
    want.backward(dout.float().cpu())
    want, h = want.detach(), (x.float() + res.float()).cpu()
    # the stream is bf16: its rounding, 2^-9 of |h| in the root mean square at most, beside what the experts add
    assert float((out.float().cpu() - want).norm()) <= 0.13 * float((want - h).norm()) + 2.0 ** -8 * float(want.norm())
    assert far(dx, xr.grad) <= 0.16
    for name, p in zip(NAMES, params):
        if name == "router" and top_k == 1:            # one choice has weight 1: no gradient
            assert float(grads[name].abs().max()) == 0
            continue
        assert far(grads[name], p.grad) <= (0.24 if name == "router" else 0.16), name


def test_forward_and_decode_agree():
    """Contiguous segments and fixed rows per expert, tokens together and alone: the same layer."""
    announce("moe forward and decode")
    H, I, G, T = 512, 256, 5, 70
    layer = moe.MoEFFN(*moe.random_weights(H, I, G), top_k=2, training=False)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, _ = layer.forward(x, res)
    both = layer.decode(x, res)
    assert far(both, out) <= 0.01                       # other kernels, other orders of the sums: a code may differ
    for t in (0, 33, T - 1):
        assert far(layer.decode(x[t:t + 1], res[t:t + 1]), out[t:t + 1]) <= 0.01


def test_decode_replays_in_a_graph():
    announce("moe graph")
    H, I, G, T = 512, 256, 5, 8
    layer = moe.MoEFFN(*moe.random_weights(H, I, G), top_k=2, training=False)
    g = torch.Generator(device="cuda").manual_seed(4)
    inputs = [[torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2)] for _ in range(3)]
    want = [layer.decode(*i) for i in inputs]
    x, res = (t.clone() for t in inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(x, res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(x, res)
    for k in (0, 1, 2, 1, 0):
        x.copy_(inputs[k][0])
        res.copy_(inputs[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
        layer.decode(*inputs[2])
        torch.cuda.synchronize()


def test_example_runs(capsys):
    announce("moe example")
    moe.main(tokens=130, H=256, I=256, G=4, top_k=2)
    assert "training step" in capsys.readouterr().out
