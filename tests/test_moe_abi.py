"""Refusals of the layer norm's and the experts' row operators' entry points
that need no GPU: every invalid argument is found on the host before any HIP
call, and calls that have nothing to do succeed without one."""
import ctypes as ct
import math
import os

import pytest

from moe_grouped_gemm_scaled_amd import binding

P = ct.c_void_p(0x10000)      # 16-byte aligned, never dereferenced
MIS = ct.c_void_p(0x10004)
ODD = ct.c_void_p(0x10002)
OK, NULL, SHAPE, ALIGN, ARG = 0, -1, -2, -3, -4
BIG = 1 << 30
FORMS = ["", "_ue8m0", "_ue8m0_packed"]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from moe_grouped_gemm_scaled_amd import build
        build.build()
    return binding.lib()


class Call:
    """An entry point with valid arguments by name; refuses(status, ..) replaces some."""

    def __init__(self, f, **args):
        self.f, self.args = f, args

    def refuses(self, status, **kw):
        assert set(kw) <= set(self.args), set(kw) - set(self.args)
        got = self.f(*{**self.args, **kw}.values())
        assert got == status, (kw, got)


@pytest.mark.parametrize("form", FORMS)
def test_layernorm(lib, form):
    c = Call(getattr(lib, "dg_layernorm_quantize_e4m3_1x128" + form), x=P, x_type=0, ld_x=256, residual=P, residual_type=0,
             weight=P, bias=P, weight_type=0, eps=1e-6, residual_out=P, y=P, q=P, sf=P, ld_sf=8, rows=5, K=256, stream=None)
    for name in ("x", "sf"):
        c.refuses(NULL, **{name: None})
    c.refuses(NULL, y=None, q=None)
    for kw in (dict(rows=-1), dict(K=0), dict(K=64), dict(K=200), dict(K=16512, ld_x=16512), dict(K=4, q=None, ld_x=8),
               dict(K=12, q=None), dict(K=16392, ld_x=16392, q=None)):
        c.refuses(SHAPE, **kw)
    for kw in (dict(x_type=2), dict(residual_type=-1), dict(weight_type=7), dict(eps=-1.0), dict(eps=math.nan),
               dict(residual=None)):
        c.refuses(ARG, **kw)
    for name in ("x", "residual", "weight", "bias", "residual_out", "y", "q", "sf"):
        c.refuses(ALIGN, **{name: MIS})
    for kw in (dict(ld_x=255), dict(ld_x=260), dict(ld_x=258, x_type=1), dict(ld_sf=4), dict(ld_sf=7)):
        c.refuses(ALIGN, **kw)
    c.refuses(OK, rows=0, x=None, residual=None, residual_out=None, weight=None, bias=None, y=None, q=None, sf=None)


def test_layernorm_backward(lib):
    c = Call(lib.dg_layernorm_backward, dy=P, dy_type=0, h=P, h_type=1, weight=P, weight_type=0, eps=1e-6, dres=P, dx=P,
             dw=P, db=P, rows=5, K=256, workspace=P, workspace_bytes=BIG, stream=None)
    for name in ("dy", "h", "dx"):
        c.refuses(NULL, **{name: None})
    for kw in (dict(rows=-1), dict(K=100), dict(K=0), dict(K=4), dict(K=32768)):
        c.refuses(SHAPE, **kw)
    for kw in (dict(dy_type=2), dict(h_type=-1), dict(weight_type=3), dict(eps=-1e-9), dict(eps=math.nan)):
        c.refuses(ARG, **kw)
    for name in ("dy", "h", "weight", "dres", "dx", "dw", "db", "workspace"):
        c.refuses(ALIGN, **{name: MIS})
    f = lib.dg_get_layernorm_backward_workspace_size
    assert f(-1, 256) == SHAPE and f(4, 100) == SHAPE and f(4, 16392) == SHAPE


def test_sort(lib):
    common = dict(ids=P, T=5, top_k=2, G=8, rows=P, src=P)
    for c in (Call(lib.dg_moe_sort_contiguous, **common, m_indices=P, counts=P, ks=P, M_total=1280, workspace=P,
                   workspace_bytes=0, stream=None),
              Call(lib.dg_moe_sort_masked, **common, masked_m=P, M_cap=4, workspace=P, workspace_bytes=0, stream=None)):
        for name in ("ids", "rows"):
            c.refuses(NULL, **{name: None})
        for kw in (dict(T=-1), dict(top_k=0), dict(G=0), dict(G=1025), dict(T=BIG, top_k=2), dict(T=1 << 25, top_k=3),
                   dict(T=(1 << 31) - 1, top_k=(1 << 31) - 1)):
            c.refuses(SHAPE, **kw)
        for name in ("ids", "rows", "src"):
            c.refuses(ALIGN, **{name: ODD})
        c.refuses(ALIGN, workspace=MIS)
    c.refuses(NULL, masked_m=None)
    c.refuses(ALIGN, masked_m=ODD)
    for kw in (dict(M_cap=0), dict(M_cap=-4), dict(M_cap=1 << 28)):        # 8 * 2^28 rows
        c.refuses(SHAPE, **kw)
    c = Call(lib.dg_moe_sort_contiguous, **common, m_indices=P, counts=P, ks=P, M_total=1280, workspace=P, workspace_bytes=0,
             stream=None)
    for kw in (dict(M_total=100), dict(M_total=-128)):
        c.refuses(SHAPE, **kw)
    c.refuses(ALIGN, m_indices=MIS)
    for name in ("counts", "ks"):
        c.refuses(ALIGN, **{name: ODD})


def test_sort_sizes(lib):
    rows, ws = lib.dg_get_moe_rows, lib.dg_get_moe_sort_workspace_size
    for f in (rows, ws):
        for args in ((-1, 2, 8), (5, 0, 8), (5, 2, 0), (5, 2, 1025), (BIG, 2, 8), ((1 << 26) + 1, 1, 8)):
            assert f(*args) == SHAPE, args
    assert rows(0, 2, 8) == 0 and rows(1, 1, 8) == 128 and rows(1, 8, 64) == 1024 and rows(128, 1, 1) == 128
    # whatever the counts, they fit: `used` experts of 128 b + 1 pairs each are the worst, and what is left fills up
    for n, G in ((1, 1), (127, 3), (129, 2), (1000, 7), (300, 300), (300, 299), (4097, 33)):
        worst = max(128 * (used + (n - used) // 128) for used in range(1, min(n, G) + 1))
        assert worst <= rows(n, 1, G) <= n + 127 * min(n, G), (n, G)
    assert ws(2048, 8, 64) == 0 and ws(2049, 8, 64) == 17 * 64 * 4


def dispatch_calls(lib, form):
    head = dict(x=P, x_type=0, ld_x=256)
    tail = dict(y=P, q=P, sf=P, qt=P, sft=P, T=5, top_k=2, K=256, M_total=1280, stream=None)
    return [Call(getattr(lib, "dg_moe_dispatch_quantize_e4m3_contiguous" + form), **head, weights=P, rows=P, src=P, **tail),
            Call(getattr(lib, "dg_moe_dispatch_quantize_e4m3_masked" + form), **head, weights=P, rows=P, y=P, q=P, sf=P, T=5,
                 top_k=2, K=256, G=4, M_cap=6, stream=None),
            Call(getattr(lib, "dg_moe_combine_backward_quantize_e4m3_contiguous" + form), **head, ye=P, weights=P, rows=P,
                 src=P, dw=P, **tail)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_dispatch(lib, form, which):
    c = dispatch_calls(lib, form)[which]
    outs = [n for n in ("y", "q", "qt", "dw") if n in c.args]
    tensors = [n for n in ("x", "ye", "weights", "rows", "src", "dw", "y", "q", "sf", "qt", "sft") if n in c.args]
    for name in ("x", "rows", "sf") + (("src", "sft") if "src" in c.args else ()) + (("ye",) if which == 2 else ()):
        c.refuses(NULL, **{name: None})
    c.refuses(NULL, **dict.fromkeys(outs))
    rows = [dict(M_total=100), dict(M_total=-128)] if which != 1 else [dict(M_cap=0), dict(G=0), dict(M_cap=1 << 29)]
    for kw in [dict(T=-1), dict(top_k=0), dict(T=BIG, top_k=2), dict(K=0), dict(K=64), dict(K=200),
               dict(K=16512, ld_x=16512)] + rows:
        c.refuses(SHAPE, **kw)
    for t in (-1, 2):
        c.refuses(ARG, x_type=t)
    for name in tensors:
        c.refuses(ALIGN, **{name: ODD})
    for name in set(tensors) - {"weights", "rows", "src", "dw"}:
        c.refuses(ALIGN, **{name: MIS})
    for kw in (dict(ld_x=255), dict(ld_x=260), dict(ld_x=258, x_type=1)):
        c.refuses(ALIGN, **kw)
    nothing = dict.fromkeys(tensors)                   # no tokens, and no rows that qt would have to clear
    c.refuses(OK, T=0, **({**nothing, "M_total": 0} if which != 1 else {**nothing, "y": P}))


@pytest.mark.parametrize("form", ["", "_ue8m0_packed"])
def test_dispatch_codes(lib, form):
    common = dict(q_in=P, sf_in=P, ld_in=8, rows=P, q=P, sf=P, T=5, top_k=2, K=256)
    for c, kws in ((Call(getattr(lib, "dg_moe_dispatch_e4m3_contiguous" + form), **common, M_total=1280, stream=None),
                    [dict(M_total=100), dict(M_total=-128)]),
                   (Call(getattr(lib, "dg_moe_dispatch_e4m3_masked" + form), **common, G=4, M_cap=6, stream=None),
                    [dict(M_cap=0), dict(G=0), dict(M_cap=1 << 29)])):
        for name in ("q_in", "sf_in", "rows", "q", "sf"):
            c.refuses(NULL, **{name: None})
            c.refuses(ALIGN, **{name: ODD})
        for kw in [dict(T=-1), dict(top_k=0), dict(T=BIG, top_k=2), dict(K=0), dict(K=64), dict(K=200)] + kws:
            c.refuses(SHAPE, **kw)
        for kw in (dict(ld_in=4), dict(ld_in=6)):
            c.refuses(ALIGN, **kw)
        c.refuses(OK, T=0, q_in=None, sf_in=None, rows=None, q=None, sf=None)


def test_combine(lib):
    c = Call(lib.dg_moe_combine, y=P, weights=P, rows=P, residual=P, out=P, out_type=0, T=5, top_k=2, K=256, R=1280,
             stream=None)
    for name in ("y", "rows", "out"):
        c.refuses(NULL, **{name: None})
    for kw in (dict(T=-1), dict(R=-1), dict(top_k=0), dict(T=BIG, top_k=2), dict(K=0), dict(K=4), dict(K=100)):
        c.refuses(SHAPE, **kw)
    for t in (-1, 2):
        c.refuses(ARG, out_type=t)
    for name in ("y", "residual", "out"):
        c.refuses(ALIGN, **{name: MIS})
    for name in ("weights", "rows"):
        c.refuses(ALIGN, **{name: ODD})
    c.refuses(OK, T=0, y=None, weights=None, rows=None, residual=None, out=None)


def test_binding():
    """The binding names the argument and raises before the library is called (host tensors are refused too)."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros(256)
    for f, kw in ((binding.layernorm_quantize_e4m3_1x128, dict(x=x, weight=w)),
                  (binding.layernorm_backward, dict(dy=x, h=x)),
                  (binding.moe_sort_contiguous, dict(ids=ids, G=4)),
                  (binding.moe_sort_masked, dict(ids=ids, G=4, M_cap=4)),
                  (binding.moe_dispatch_quantize_e4m3_contiguous, dict(x=x, rows=ids, M_total=512)),
                  (binding.moe_dispatch_quantize_e4m3_masked, dict(x=x, rows=ids, G=4, M_cap=4)),
                  (binding.moe_dispatch_e4m3_contiguous, dict(q_in=x.view(torch.uint8), sf_in=x, rows=ids, M_total=512)),
                  (binding.moe_dispatch_e4m3_masked, dict(q_in=x.view(torch.uint8), sf_in=x, rows=ids, G=4, M_cap=4)),
                  (binding.moe_combine, dict(y=x, rows=ids)),
                  (binding.moe_combine_backward_quantize_e4m3_contiguous, dict(dout=x, y=x, rows=ids))):
        with pytest.raises(ValueError, match="device tensor"):
            f(**kw)
    with pytest.raises(ValueError, match="scales"):
        binding.layernorm_quantize_e4m3_1x128(x, w, scales="fp16")
    with pytest.raises(ValueError, match="scales"):
        binding.moe_dispatch_quantize_e4m3_contiguous(x, ids, 512, scales="fp16")
    with pytest.raises(ValueError, match="columns"):
        binding.moe_dispatch_quantize_e4m3_contiguous(x.t(), ids, 512)
    with pytest.raises(ValueError, match="ids"):
        binding.moe_sort_contiguous(ids[0], 4)
    with pytest.raises(ValueError, match="y\\["):
        binding.moe_combine(w, ids)
    with pytest.raises(ValueError, match="workspace"):
        binding.layernorm_backward(x, x, workspace="none")
    with pytest.raises(binding.DGError, match="SHAPE"):
        binding.get_moe_rows(5, 2, 1025)


def test_sizes_past_32_bits():
    """Sizes whose low 32 bits would make a valid call are refused by name (tensors without memory)."""
    import torch
    n = (1 << 32) + 128
    big = torch.empty((n, 8), dtype=torch.bfloat16, device="meta")
    ids = torch.empty((n, 1), dtype=torch.int32, device="meta")
    few = ids[:4]
    for f, args in ((binding.layernorm_quantize_e4m3_1x128, (big,)), (binding.layernorm_backward, (big, big)),
                    (binding.moe_sort_contiguous, (ids, 4)), (binding.moe_sort_masked, (ids, 4, 4)),
                    (binding.moe_dispatch_quantize_e4m3_contiguous, (big, ids, 128)),
                    (binding.moe_dispatch_quantize_e4m3_contiguous, (big[:4], few, n)),
                    (binding.moe_dispatch_quantize_e4m3_masked, (big[:4], few, 4, n)),
                    (binding.moe_dispatch_e4m3_contiguous, (big, big, ids, 128)),
                    (binding.moe_combine, (big, few)), (binding.moe_combine, (big[:4], ids)),
                    (binding.moe_combine_backward_quantize_e4m3_contiguous, (big[:4], big, few))):
        with pytest.raises(ValueError, match="32 bits"):
            f(*args)
