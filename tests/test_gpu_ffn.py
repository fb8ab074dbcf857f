"""GPU tests of the feed-forward layer as it is used: its parts one after the
other, forward and backward, against the layer in fp32 on the CPU; and of the
binding's refusals on device tensors, in native code and in Python.

Bar of the layer: an E4M3 operand is off by 2^-4 at most, 2.6 % in the root mean
square; a product of two such operands by 3.7 % of its norm.  out has three
products in a row (gate and up side by side): sqrt(2 * 3.7^2 + 3.7^2) = 6.4 %;
the gradients one or two more quantised operands, about 8 %.  Twice that is
allowed."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import ffn

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("tokens", [1, 33, 128, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_step(tokens, act):
    announce(f"ffn step tokens={tokens} {act}")
    H, I = 512, 384
    weights = ffn.random_weights(H, I, seed=tokens)
    layer = ffn.GatedFFN(*weights, act=act)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res, dout, dres = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(4))
    out, stream, saved = layer.forward(x, res, save=True)
    dx, grads = layer.backward(saved, dout, dh=dres)
    params = [w.cpu().requires_grad_() for w in weights]
    xr = x.float().cpu().requires_grad_()
    want, h = ffn.reference(*params, xr, res.float().cpu(), act=act)
    (want * dout.float().cpu()).sum().add((h * dres.float().cpu()).sum()).backward()
    assert torch.equal(stream, (x.float() + res.float()).bfloat16())
    assert far(out, want) <= 0.13
    assert far(dx, xr.grad) <= 0.16
    for name, p in zip(("w_norm", "w_gate", "w_up", "w_down"), params):
        assert far(grads[name], p.grad) <= 0.16, name


def test_decode_equals_prefill_rows():
    """Rows go through the layer independently of each other: one token at a time gives the rows of the whole."""
    announce("ffn rows")
    H, I, T = 512, 256, 150
    layer = ffn.GatedFFN(*ffn.random_weights(H, I))
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, stream, _ = layer.forward(x, res)
    for r in (0, 77, T - 1):
        one, s, _ = layer.forward(x[r:r + 1], res[r:r + 1])
        assert torch.equal(s, stream[r:r + 1])
        assert far(one, out[r:r + 1]) <= 0.01           # other kernels, other orders of the sums: a code may differ


def test_example_runs(capsys):
    announce("ffn example")
    ffn.main(tokens=130, H=256, I=256)
    assert "training step" in capsys.readouterr().out


def test_layer_replays_in_a_graph():
    """A decode step captured once and replayed with new inputs between eager calls."""
    announce("ffn graph")
    H, I = 512, 256
    layer = ffn.GatedFFN(*ffn.random_weights(H, I))
    g = torch.Generator(device="cuda").manual_seed(4)
    inputs = [[torch.randn(8, H, generator=g, device="cuda").bfloat16() for _ in range(2)] for _ in range(3)]
    want = [layer.forward(*i)[:2] for i in inputs]
    x, res = (t.clone() for t in inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, stream, _ = layer.forward(x, res)
    for k in (0, 1, 2, 1, 0):
        x.copy_(inputs[k][0])
        res.copy_(inputs[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, want[k][1])
        assert torch.equal(out, want[k][0])
        layer.forward(*inputs[2])
        torch.cuda.synchronize()


# ---------------------------------------------------------------- the binding's refusals

@pytest.fixture(params=["native", "python"])
def checks(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(dg, "_native_addresses", lambda *_: None)
    else:
        assert dg._native_addresses.__name__ == "addresses", "the native checks are not built"


def refused(error, match, f, *args, **kw):
    with pytest.raises(error, match=match):
        f(*args, **kw)


def test_refusals_of_device_tensors(checks):
    announce("binding refusals")
    bf = torch.bfloat16
    x, w = torch.zeros((4, 256), dtype=bf, device="cuda"), torch.ones(256, dtype=bf, device="cuda")
    f = dg.rmsnorm_quantize_e4m3_1x128
    f(x, w)
    refused(TypeError, "x", f, x.half(), w)
    refused(TypeError, "weight", f, x, None)
    refused(ValueError, "weight", f, x, w[:128])
    refused(ValueError, "weight", f, x, w.cpu())
    refused(ValueError, "columns", f, x.t(), w)
    refused(ValueError, "residual", f, x, w, residual=x[:2])
    refused(TypeError, "residual_out", f, x, w, residual=x, residual_out=x.float())
    refused(ValueError, "y", f, x, w, y=torch.empty((256, 4), dtype=bf, device="cuda").t())
    refused(ValueError, "residual_out", f, x, w, residual_out=x)
    refused(ValueError, "sf", f, x, w, sf=torch.zeros((3, 4), device="cuda"))
    refused(TypeError, "sf", f, x, w, sf=torch.zeros((1, 4), device="cuda"), scales="ue8m0_packed")
    refused(dg.DGError, "SHAPE", f, x[:, :192], w[:192])
    refused(dg.DGError, "ALIGN", f, torch.zeros((4, 257), dtype=bf, device="cuda")[:, 1:], w)
    refused(dg.DGError, "ARG", f, x, w, eps=-1.0)

    f = dg.rmsnorm_backward
    f(x, x, w)
    refused(TypeError, "dres", f, x, x, w, dres=x.float())
    refused(ValueError, "dw", f, x, x, w, dw=torch.zeros(128, device="cuda"))
    refused(ValueError, "dy", f, x[:1], x, w)
    refused(dg.DGError, "NULL", f, torch.zeros((64, 256), dtype=bf, device="cuda"), torch.zeros((64, 256), dtype=bf, device="cuda"),
            w, workspace=None)
    refused(dg.DGError, "ARG", f, torch.zeros((64, 256), dtype=bf, device="cuda"), torch.zeros((64, 256), dtype=bf, device="cuda"),
            w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))

    a, sfa = torch.zeros((4, 256), dtype=torch.uint8, device="cuda"), torch.ones((2, 4), device="cuda")
    b, sfb = torch.zeros((2, 128, 256), dtype=torch.uint8, device="cuda"), torch.ones((2, 1, 2), device="cuda")
    f = dg.fp8_gated_gemm_nt
    f(a, sfa, b, sfb)
    refused(ValueError, "sfa", f, a, sfa[:1], b, sfb)
    refused(TypeError, "sfb", f, a, sfa, b, sfb.int())
    refused(ValueError, "act", f, a, sfa, b, sfb, act="relu")
    refused(ValueError, "h", f, a, sfa, b, sfb, h=torch.empty((4, 64), dtype=bf, device="cuda"))
    refused(ValueError, "b", f, a, sfa, b.transpose(0, 1), sfb)
    refused(dg.DGError, "SHAPE", f, a, sfa, b[:, :100].contiguous(), sfb, q=True)
    g = dg.m_grouped_fp8_gated_gemm_nt_masked
    refused(TypeError, "masked_m", g, a[None], sfa[None].contiguous(), b[None], sfb[None], torch.zeros(1, device="cuda"))
    c = dg.m_grouped_fp8_gated_gemm_nt_contiguous
    refused(dg.DGError, "SHAPE", c, a, sfa, b[None], sfb[None], torch.zeros(4, dtype=torch.int32, device="cuda"))

    f = dg.gated_backward_quantize_e4m3
    gu, dh = torch.zeros((4, 512), dtype=bf, device="cuda"), torch.zeros((4, 256), dtype=bf, device="cuda")
    f(gu, dh, q=True)
    refused(dg.DGError, "NULL", f, gu, dh)
    refused(ValueError, "gu", f, gu[:, :256].contiguous(), dh, q=True)
    refused(ValueError, "qt", f, gu, dh, qt=torch.zeros((4, 512), dtype=torch.uint8, device="cuda"))
    refused(TypeError, "sft", f, gu, dh, qt=True, sft=torch.zeros((1, 512), dtype=bf, device="cuda"))
