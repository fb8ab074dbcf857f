"""Measured cases of the FP8 feed-forward layer's operators.

Four operators, in plain torch (own = False) and through the library's entry
points (own = True):
  norm       residual addition + RMS norm + E4M3 quantisation (1x128 scales)
  norm_bwd   its gradient: dx and dw
  gated      gate and up projections (FP8, block scales), act(gate) * up, with
             a bf16 or an E4M3 output and the saved projections; dense, M-grouped
             contiguous and M-grouped masked
  gated_bwd  the gradient of act(gate) * up, quantised for the two gradient GEMMs

Layouts are the library's: codes E4M3, A scales [K/128][ld] with ld a multiple
of 4, B scales one per 128x128 block, packed scales four exponents per int32
along the K blocks.  Sizes: hidden 7168 and expert width 2048 are those of the
library's grouped workloads, 1536 of 2112 columns the query latent of its
projections; the rest are generic.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


def listed():
    return [
        # one decode step of a 64-request batch: the norm before the experts, packed scales
        {"name": "norm decode", "op": "norm", "rows": 64, "K": 7168, "pitch": 7168, "res": True, "x": "bf16",
         "stream": "bf16", "y": False, "scales": "packed"},
        # a prefill chunk of 4096 tokens
        {"name": "norm prefill", "op": "norm", "rows": 4096, "K": 7168, "pitch": 7168, "res": True, "x": "bf16",
         "stream": "bf16", "y": False, "scales": "fp32"},
        # the query latent: the first 1536 of the 2112 columns of a projection, an odd number of rows, bf16 copy kept
        {"name": "norm latent", "op": "norm", "rows": 1111, "K": 1536, "pitch": 2112, "res": False, "x": "bf16",
         "stream": "bf16", "y": True, "scales": "fp32"},
        # a short training sequence with an fp32 residual stream
        {"name": "norm_bwd short", "op": "norm_bwd", "rows": 333, "K": 2048, "stream": "fp32", "dres": True},
        # a long training batch
        {"name": "norm_bwd long", "op": "norm_bwd", "rows": 16384, "K": 7168, "stream": "bf16", "dres": True},
        # a single token through a shared expert
        {"name": "gated one token", "op": "gated", "mode": "dense", "rows": 1, "I": 2048, "K": 7168, "act": "silu",
         "scales": "fp32", "out": "h", "gu": False},
        # a decode batch, the output quantised for the down projection
        {"name": "gated decode", "op": "gated", "mode": "dense", "rows": 64, "I": 2048, "K": 7168, "act": "silu",
         "scales": "packed", "out": "q", "gu": False},
        # prefill / training forward of a dense layer, projections saved for the backward pass
        {"name": "gated prefill", "op": "gated", "mode": "dense", "rows": 4096, "I": 2048, "K": 7168, "act": "silu",
         "scales": "packed", "out": "q", "gu": True},
        # the experts of a training step: ragged token counts, tokens sorted by expert
        {"name": "gated experts", "op": "gated", "mode": "contiguous", "G": 8, "blocks": 72, "I": 2048, "K": 7168,
         "act": "silu", "scales": "fp32", "out": "h", "gu": True},
        # the experts of a decode step: 16 local experts, up to 256 rows each, counts on the device
        {"name": "gated masked", "op": "gated", "mode": "masked", "G": 16, "cap": 256, "I": 2048, "K": 7168,
         "act": "silu", "scales": "packed", "out": "q", "gu": False},
        # backward of a short sequence through a dense layer, tanh-GELU gate
        {"name": "gated_bwd short", "op": "gated_bwd", "mode": "dense", "rows": 200, "I": 2048, "act": "gelu"},
        # backward of the experts of a training step
        {"name": "gated_bwd experts", "op": "gated_bwd", "mode": "contiguous", "G": 8, "blocks": 136, "I": 2048,
         "act": "silu"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gated", "gated", "gated", "gated_bwd"])
    if op in ("norm", "norm_bwd"):
        rows, K = _log(rng, 1, 16384), 128 * _log(rng, 4, 128)
        rows = min(rows, 4096 * 7168 // K if op == "norm" else 16384 * 7168 // K)
        stream = rng.choice(["bf16", "bf16", "fp32"])
        if op == "norm_bwd":
            return {"op": op, "rows": rows, "K": K, "stream": stream, "dres": rng.random() < 0.7}
        return {"op": op, "rows": rows, "K": K, "pitch": K + rng.choice([0, 0, 64, 576]), "res": rng.random() < 0.7,
                "x": rng.choice(["bf16", "bf16", "fp32"]), "stream": stream, "y": rng.random() < 0.5,
                "scales": rng.choice(["fp32", "packed"])}
    act = rng.choice(["silu", "silu", "gelu"])
    if op == "gated_bwd":
        if rng.random() < 0.5:
            return {"op": op, "mode": "dense", "rows": _log(rng, 1, 8192), "I": 128 * _log(rng, 2, 32), "act": act}
        return {"op": op, "mode": "contiguous", "G": rng.randint(2, 8), "blocks": _log(rng, 2, 64),
                "I": 128 * _log(rng, 2, 32), "act": act}
    mode = rng.choice(["dense", "dense", "contiguous", "masked"])
    out = rng.choice(["h", "q"])
    case = {"op": op, "mode": mode, "I": 128 * _log(rng, 2, 32), "K": 128 * _log(rng, 4, 64), "act": act,
            "scales": "packed" if out == "q" else rng.choice(["fp32", "packed"]), "out": out,
            "gu": rng.random() < 0.4}
    if mode == "dense":
        case["rows"] = min(_log(rng, 1, 4096), max(1, 4096 * 2048 * 7168 // (case["I"] * case["K"])))
        if out == "h" and rng.random() < 0.4:
            case["I"] = max(8, case["I"] - rng.randint(1, 100))     # a width that is no multiple of a block
    else:
        case["G"] = rng.randint(2, 16)
        most = 8 if case["G"] <= 8 else 16
        case["I"] = min(case["I"], max(128, 2048 * 7168 // case["K"] * 8 // most // 128 * 128))
        if mode == "contiguous":
            case["G"] = min(case["G"], 8)
            case["blocks"] = _log(rng, 2, 40)
        else:
            case["cap"] = rng.choice([16, 64, 128, 200, 256])
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _type(name):
    return BF16 if name == "bf16" else F32


def _ld(rows):
    return (rows + 3) // 4 * 4


def _pow2_up(s):
    """s rounded up to a power of two (s normal and positive)."""
    u = s.view(torch.int32)
    return torch.where((u & 0x7FFFFF) != 0, (u & 0x7F800000) + 0x800000, u).view(F32)


def _scale(amax, scales):
    s = amax.clamp_min(1e-4) / 448.0
    return _pow2_up(s) if scales == "packed" else s


def _pack(sf):
    """fp32 powers of two [.., blocks, n] -> int32 words [.., ceil(blocks/4), n], four exponents a word."""
    e = (sf.view(torch.int32) >> 23) & 0xFF
    pad = -e.shape[-2] % 4
    if pad:
        e = torch.cat([e, e.new_zeros(*e.shape[:-2], pad, e.shape[-1])], -2)
    e = e.unflatten(-2, (-1, 4))
    return e[..., 0, :] | (e[..., 1, :] << 8) | (e[..., 2, :] << 16) | (e[..., 3, :] << 24)


def _unpack(words, blocks):
    """int32 words [.., w, n] -> fp32 [.., blocks, n]."""
    b = words.contiguous().view(torch.uint8).unflatten(-1, (-1, 4)).movedim(-1, -2).flatten(-3, -2)
    return (b[..., :blocks, :].to(torch.int32) << 23).view(F32)


def _sf_shape(scales, blocks, n):
    return ((blocks + 3) // 4 if scales == "packed" else blocks, n)


def _sf_buffer(scales, lead, blocks, n):
    return torch.zeros(*lead, *_sf_shape(scales, blocks, n), dtype=torch.int32 if scales == "packed" else F32, device=DEV)


def _sf_value(scales, sf):
    """Scales as the values that they stand for."""
    return sf.view(E8M0) if scales == "packed" else sf


def _codes(y, s):
    return (y / s).clamp(-448.0, 448.0).to(E4M3)


def _quant_rows(y, scales, ld):
    """y [.., rows, K] fp32 -> codes, scales [.., K/128, ld] (zeros past the rows), one scale per row and 128 columns."""
    b = y.unflatten(-1, (-1, 128))
    s = _scale(b.abs().amax(-1), scales)
    q = _codes(b, s.unsqueeze(-1)).flatten(-2)
    sf = s.transpose(-1, -2)
    if scales == "packed":
        sf = _pack(sf.contiguous())
    if ld > sf.shape[-1]:
        sf = torch.cat([sf, sf.new_zeros(*sf.shape[:-1], ld - sf.shape[-1])], -1)
    return q, sf.contiguous()


def _quant_cols(y):
    """y [128 t, N] fp32 -> codes [128 t, N], scales [t, N] fp32: one scale per column and 128 rows."""
    b = y.unflatten(0, (-1, 128))
    s = _scale(b.abs().amax(1), "fp32")
    return _codes(b, s.unsqueeze(1)).flatten(0, 1), s


def _quant_blocks(w, scales):
    """w [.., N, K] fp32 -> codes (uint8), scales [.., ceil(N/128), K/128] or their packed words along the last axis."""
    n = w.shape[-2]
    pad = -n % 128
    p = torch.nn.functional.pad(w, (0, 0, 0, pad)) if pad else w
    b = p.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))            # [.., N/128, 128, K/128, 128]
    s = _scale(b.abs().amax((-1, -3)), scales)
    q = _codes(b, s.unsqueeze(-1).unsqueeze(-3)).flatten(-2).flatten(-3, -2)[..., :n, :].contiguous()
    if scales == "packed":
        s = _pack(s.transpose(-1, -2).contiguous()).transpose(-1, -2)
    return q.view(torch.uint8), s.contiguous()


def _counts(case, seed):
    """Rows of each expert: masked, any number up to the capacity; contiguous, `blocks` blocks of 128 rows dealt
    unevenly (an expert may get none), the last block of each expert partly filled."""
    g = torch.Generator().manual_seed(int(seed) * 31 + 5)
    if case["mode"] == "masked":
        return torch.randint(0, case["cap"] + 1, (case["G"],), generator=g).tolist()
    n = case["blocks"]
    cuts = [0] + sorted(torch.randint(0, n + 1, (case["G"] - 1,), generator=g).tolist()) + [n]
    return [max(0, 128 * (b - a) - int(torch.randint(0, 128, (1,), generator=g))) for a, b in zip(cuts, cuts[1:])]


def _indices(counts):
    """Expert of each row, -1 on the rows that pad every expert's segment to 128."""
    parts = [torch.cat([torch.full((c,), e, dtype=torch.int32), torch.full((-c % 128,), -1, dtype=torch.int32)])
             for e, c in enumerate(counts)]
    return torch.cat(parts).to(DEV)


def _activations(g, *shape):
    """Values like a residual stream's: N(0, 1) with a few strong columns."""
    x = _randn(g, *shape)
    x[..., ::97] *= 8.0
    return x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norm":
        rows, K = case["rows"], case["K"]
        full = _activations(g, rows, case["pitch"]).to(_type(case["x"]))
        s = {"case": case, "x": full[:, :K], "w": (1.0 + 0.2 * _randn(g, K)).to(BF16),
             "q": torch.zeros(rows, K, dtype=torch.uint8, device=DEV),
             "sf": _sf_buffer(case["scales"], (), K // 128, _ld(rows))}
        if case["res"]:
            s["res"] = (2.0 * _activations(g, rows, K)).to(_type(case["stream"]))
            s["res_out"] = torch.empty_like(s["res"])
        if case["y"]:
            s["y"] = torch.empty(rows, K, dtype=BF16, device=DEV)
        return s
    if op == "norm_bwd":
        rows, K, t = case["rows"], case["K"], _type(case["stream"])
        s = {"case": case, "dy": (0.1 * _randn(g, rows, K)).to(BF16), "h": _activations(g, rows, K).to(t),
             "w": (1.0 + 0.2 * _randn(g, K)).to(BF16), "dx": torch.empty(rows, K, dtype=t, device=DEV),
             "dw": torch.empty(K, dtype=F32, device=DEV)}
        if case["dres"]:
            s["dres"] = (0.1 * _randn(g, rows, K)).to(t)
        return s
    if op == "gated_bwd":
        I = case["I"]
        s = {"case": case}
        if case["mode"] == "contiguous":
            s["idx"] = _indices(_counts(case, seed))
            rows = s["idx"].numel()
        else:
            rows = case["rows"]
        full = (rows + 127) // 128 * 128
        s["gu"] = _randn(g, rows, 2 * I).to(BF16)
        s["dh"] = (0.05 * _randn(g, rows, I)).to(BF16)
        s["q"] = torch.empty(rows, 2 * I, dtype=torch.uint8, device=DEV)
        s["sf"] = _sf_buffer("fp32", (), 2 * I // 128, _ld(rows))
        s["qt"] = torch.empty(full, 2 * I, dtype=torch.uint8, device=DEV)
        s["sft"] = torch.empty(full // 128, 2 * I, dtype=F32, device=DEV)
        s["ht"] = torch.empty(full, I, dtype=torch.uint8, device=DEV)
        s["sfht"] = torch.empty(full // 128, I, dtype=F32, device=DEV)
        return s
    I, K, scales, mode = case["I"], case["K"], case["scales"], case["mode"]
    s = {"case": case}
    lead, groups = (), ()
    if mode == "contiguous":
        s["idx"] = _indices(_counts(case, seed))
        rows, groups = s["idx"].numel(), (case["G"],)
    elif mode == "masked":
        s["counts"] = torch.tensor(_counts(case, seed), dtype=torch.int32, device=DEV)
        rows, groups = case["cap"], (case["G"],)
        lead = groups
    else:
        rows = case["rows"]
    ld = rows if mode == "contiguous" else _ld(rows)
    a, s["sfa"] = _quant_rows(_activations(g, *lead, rows, K), scales, ld)
    s["a"] = a.view(torch.uint8)
    s["b"], s["sfb"] = _quant_blocks(_randn(g, *groups, 2, I, K) * (K ** -0.5), scales)
    if case["out"] == "q":
        s["q"] = torch.zeros(*lead, rows, I, dtype=torch.uint8, device=DEV)
        s["sf"] = _sf_buffer(scales, lead, I // 128, ld)
    else:
        s["h"] = torch.zeros(*lead, rows, I, dtype=BF16, device=DEV)
    if case["gu"]:
        s["gu"] = torch.zeros(*lead, rows, 2 * I, dtype=BF16, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if c["res"]:
        h = h + s["res"].float()
        out["res_out"] = h.to(s["res"].dtype)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    if c["y"]:
        out["y"] = y.to(BF16)
    out["q"], sf = _quant_rows(y, c["scales"], _ld(c["rows"]))
    out["sf"] = _sf_value(c["scales"], sf)
    return out


def _norm_bwd_plain(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    gw = dy * s["w"].float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    if "dres" in s:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * n).sum(0)}


def _act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _act_grad(x, act):
    if act == "silu":
        t = torch.sigmoid(x)
        return t * (1.0 + x * (1.0 - t))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * x * x)


def _rows_value(s, scales, rows, K, t=F32):
    """A operand [.., rows, K] as numbers."""
    sf = _unpack(s["sfa"], K // 128) if scales == "packed" else s["sfa"]
    v = s["a"].view(E4M3).to(t).unflatten(-1, (-1, 128))
    return (v * sf[..., :rows].transpose(-1, -2).unsqueeze(-1).to(t)).flatten(-2)


def _weights_value(s, scales, I, K, t=F32):
    """B operand [.., 2, I, K] as numbers."""
    sf = s["sfb"]
    if scales == "packed":
        sf = _unpack(sf.transpose(-1, -2), K // 128).transpose(-1, -2)
    sf = sf.repeat_interleave(128, -2)[..., :I, :]
    return (s["b"].view(E4M3).to(t).unflatten(-1, (-1, 128)) * sf.unsqueeze(-1).to(t)).flatten(-2)


def _gated_out(s, gate, up, valid):
    c = s["case"]
    h = _act(gate, c["act"]) * up
    out = {}
    if c["gu"]:
        gu = torch.cat([gate, up], -1).to(BF16)
        out["gu"] = gu if valid is None else gu * valid
    if c["out"] == "h":
        h = h.to(BF16)
        out["h"] = h if valid is None else h * valid
        return out
    q, sf = _quant_rows(h, c["scales"], s["sf"].shape[-1])
    if valid is not None:                     # rows that are not computed keep what the buffers held
        q = torch.where(valid, q.view(torch.uint8), 0).view(E4M3)
        keep = torch.nn.functional.pad(valid.squeeze(-1), (0, sf.shape[-1] - valid.shape[-2])).unsqueeze(-2)
        sf = torch.where(keep, sf, 0)
    out["q"], out["sf"] = q, _sf_value(c["scales"], sf)
    return out


def _gated_plain(s):
    c = s["case"]
    I, K, scales, mode = c["I"], c["K"], c["scales"], c["mode"]
    rows = s["a"].shape[-2]
    a, w = _rows_value(s, scales, rows, K), _weights_value(s, scales, I, K)
    if mode == "dense":
        gu = a @ w.view(2 * I, K).t()
        return _gated_out(s, gu[:, :I], gu[:, I:], None)
    if mode == "masked":
        gu = torch.bmm(a, w.flatten(1, 2).transpose(1, 2))
        valid = (torch.arange(rows, device=DEV)[None] < s["counts"][:, None]).unsqueeze(-1)
        return _gated_out(s, gu[..., :I], gu[..., I:], valid)
    expert = s["idx"][::128].long()                                   # of each 128-row block
    gu = torch.bmm(a.view(-1, 128, K), w.flatten(1, 2)[expert].transpose(1, 2)).view(rows, 2 * I)
    return _gated_out(s, gu[:, :I], gu[:, I:], (s["idx"] >= 0).unsqueeze(-1))


def _gated_bwd_plain(s):
    c = s["case"]
    I, rows = c["I"], s["gu"].shape[0]
    gate, up, dh = s["gu"][:, :I].float(), s["gu"][:, I:].float(), s["dh"].float()
    a = _act(gate, c["act"])
    d = torch.cat([dh * up * _act_grad(gate, c["act"]), dh * a], -1)
    h = a * up
    if "idx" in s:
        live = (s["idx"] >= 0).unsqueeze(-1)
        d, h = torch.where(live, d, 0.0), torch.where(live, h, 0.0)
    q, sf = _quant_rows(d, "fp32", _ld(rows))
    pad = (0, 0, 0, -rows % 128)
    qt, sft = _quant_cols(torch.nn.functional.pad(d, pad))
    ht, sfht = _quant_cols(torch.nn.functional.pad(h, pad))
    return {"q": q, "sf": sf, "qt": qt, "sft": sft, "ht": ht, "sfht": sfht}


# ---------------------------------------------------------------- the library's calls

_SCALES = {"fp32": "fp32", "packed": "ue8m0_packed"}


def _run_own(s):
    from moe_grouped_gemm_scaled_amd import binding as dg
    c = s["case"]
    op = c["op"]
    if op == "norm":
        dg.rmsnorm_quantize_e4m3_1x128(s["x"], s["w"], EPS, residual=s.get("res"), residual_out=s.get("res_out"),
                                       y=s.get("y"), q=s["q"], sf=s["sf"], scales=_SCALES[c["scales"]])
        out = {k: s[k] for k in ("res_out", "y") if k in s}
        return {**out, "q": s["q"].view(E4M3), "sf": _sf_value(c["scales"], s["sf"])}
    if op == "norm_bwd":
        dg.rmsnorm_backward(s["dy"], s["h"], s["w"], EPS, dres=s.get("dres"), dx=s["dx"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "gated_bwd":
        dg.gated_backward_quantize_e4m3(s["gu"], s["dh"], act=c["act"], m_indices=s.get("idx"), q=s["q"], sf=s["sf"],
                                        qt=s["qt"], sft=s["sft"], ht=s["ht"], sfht=s["sfht"])
        return {"q": s["q"].view(E4M3), "sf": s["sf"], "qt": s["qt"].view(E4M3), "sft": s["sft"],
                "ht": s["ht"].view(E4M3), "sfht": s["sfht"]}
    outs = {k: s[k] for k in ("h", "q", "sf", "gu") if k in s}
    if c["mode"] == "dense":
        dg.fp8_gated_gemm_nt(s["a"], s["sfa"], s["b"], s["sfb"], act=c["act"], **outs)
    elif c["mode"] == "contiguous":
        dg.m_grouped_fp8_gated_gemm_nt_contiguous(s["a"], s["sfa"], s["b"], s["sfb"], s["idx"], act=c["act"], **outs)
    else:
        dg.m_grouped_fp8_gated_gemm_nt_masked(s["a"], s["sfa"], s["b"], s["sfb"], s["counts"], act=c["act"], **outs)
    if "q" in outs:
        outs["q"], outs["sf"] = s["q"].view(E4M3), _sf_value(c["scales"], s["sf"])
    return outs


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "gated_bwd":
        return _gated_bwd_plain(state)
    return _gated_plain(state)


# ---------------------------------------------------------------- work and 64-bit values

def _valid(case):
    """(rows held, rows computed, experts read): the expectation over the seeds where counts are drawn."""
    if case.get("mode") == "contiguous":
        n, e = case["blocks"], case["G"] * case["blocks"] / (case["blocks"] + case["G"] - 1)
        return 128 * n, 128 * n - 63.5 * e, e
    if case.get("mode") == "masked":
        return case["G"] * case["cap"], case["G"] * case["cap"] / 2, case["G"] * case["cap"] / (case["cap"] + 1)
    return case["rows"], case["rows"], 1


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "norm":
        n = case["rows"] * case["K"]
        per = size[case["x"]] + 1 + (2 * size[case["stream"]] if case["res"] else 0) + (2 if case["y"] else 0)
        per += (1 if case["scales"] == "packed" else 4) / 128
        return {"bytes": n * per + 2 * case["K"], "flops": 8 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 + size[case["stream"]] * (3 if case["dres"] else 2)) + 6 * case["K"], "flops": 10 * n}
    held, rows, groups = _valid(case)
    I = case["I"]
    if op == "gated_bwd":
        full = (held + 127) // 128 * 128
        return {"bytes": rows * I * 6 + held * 2 * I * (1 + 4 / 128) + full * 3 * I * (1 + 4 / 128),
                "flops": 30 * rows * I}
    K = case["K"]
    per = 1 if case["scales"] == "packed" else 4
    b = rows * K * (1 + per / 128) + groups * 2 * I * K * (1 + per / 16384)
    b += rows * I * (2 if case["out"] == "h" else 1 + per / 128) + (rows * 4 * I if case["gu"] else 0)
    return {"bytes": b, "flops": 4 * rows * I * K}


def _exact_scale(amax, scales):
    s = torch.clamp(amax, min=1e-4) / 448.0
    return torch.exp2(torch.ceil(torch.log2(s))) if scales == "packed" else s


def _exact_rows(y, scales, ld):
    """Quantised rows as 64-bit numbers: values over their scales (not rounded to codes), and the scales' layout."""
    rows, K = y.shape
    amax = y.reshape(rows, K // 128, 128).abs().max(-1).values
    s = _exact_scale(amax, scales)
    q = y / s.repeat_interleave(128, 1)
    if scales == "packed":
        blocks = (K // 128 + 3) // 4 * 4
        sf = torch.full((blocks // 4, ld, 4), 2.0 ** -127, dtype=torch.float64, device=y.device)
        at = torch.zeros(blocks, ld, dtype=torch.float64, device=y.device) + 2.0 ** -127
        at[:K // 128, :rows] = s.t()
        sf[:] = at.reshape(blocks // 4, 4, ld).permute(0, 2, 1)
        return q, sf.reshape(blocks // 4, 4 * ld)
    sf = torch.zeros(K // 128, ld, dtype=torch.float64, device=y.device)
    sf[:, :rows] = s.t()
    return q, sf


def _exact_cols(y):
    rows, n = y.shape
    p = torch.zeros((rows + 127) // 128 * 128, n, dtype=torch.float64, device=y.device)
    p[:rows] = y
    s = _exact_scale(p.reshape(-1, 128, n).abs().max(1).values, "fp32")
    return p / s.repeat_interleave(128, 0), s


def _exact_gate(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e + g * e * (1.0 - e)
    k = (2.0 / math.pi) ** 0.5
    z = k * (g + 0.044715 * g ** 3)
    t = torch.tanh(z)
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * k * (1 + 0.134145 * g ** 2)


def _exact_codes(a, sf, packed):
    """[rows, K] codes with [K/128 (words), ld] scales -> 64-bit numbers."""
    v = a.view(E4M3).double()
    rows, K = v.shape
    if packed:
        w = sf.to(torch.int64) & 0xFFFFFFFF
        sf = torch.stack([torch.exp2(((w[b // 4] >> (8 * (b % 4))) & 0xFF).double() - 127) for b in range(K // 128)])
    return v * sf[:, :rows].t().double().repeat_interleave(128, 1)


def _exact_weights(b, sf, packed):
    """[2, I, K] codes with [2, I/128, K/128 (words)] scales -> 64-bit numbers."""
    v = b.view(E4M3).double()
    I, K = v.shape[1:]
    if packed:
        w = sf.to(torch.int64) & 0xFFFFFFFF
        sf = torch.stack([torch.exp2(((w[..., k // 4] >> (8 * (k % 4))) & 0xFF).double() - 127)
                          for k in range(K // 128)], -1)
    return v * sf.double().repeat_interleave(128, 1)[:, :I].repeat_interleave(128, 2)


def exact(case, seed):
    op = case["op"]
    if op == "gated" and work(case)["flops"] > 8e11:
        return None
    s = prepare(case, seed)
    if op == "norm":
        h = s["x"].double()
        out = {}
        if case["res"]:
            h = h + s["res"].double()
            out["res_out"] = h
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["K"] + EPS) * s["w"].double()
        if case["y"]:
            out["y"] = y
        out["q"], out["sf"] = _exact_rows(y, case["scales"], _ld(case["rows"]))
        return out
    if op == "norm_bwd":
        h, dy, w, K = s["h"].double(), s["dy"].double(), s["w"].double(), case["K"]
        v = h.pow(2).sum(1, keepdim=True) / K + EPS
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = dy * w / v.sqrt() - h * dot / (K * v * v.sqrt())
        if "dres" in s:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dw": (dy * h / v.sqrt()).sum(0)}
    I = case["I"]
    if op == "gated_bwd":
        gu, dh = s["gu"].double(), s["dh"].double()
        a, da = _exact_gate(gu[:, :I], case["act"])
        d = torch.cat([dh * gu[:, I:] * da, dh * a], 1)
        h = a * gu[:, I:]
        if "idx" in s:
            d[s["idx"] < 0] = 0
            h[s["idx"] < 0] = 0
        q, sf = _exact_rows(d, "fp32", _ld(d.shape[0]))
        qt, sft = _exact_cols(d)
        ht, sfht = _exact_cols(h)
        return {"q": q, "sf": sf, "qt": qt, "sft": sft, "ht": ht, "sfht": sfht}
    packed = case["scales"] == "packed"

    def one(a, sfa, b, sfb, ld):
        p = _exact_codes(a, sfa, packed)
        w = _exact_weights(b, sfb, packed)
        gate, up = p @ w[0].t(), p @ w[1].t()
        h = _exact_gate(gate, case["act"])[0] * up
        out = {"gu": torch.cat([gate, up], 1)}
        if case["out"] == "h":
            out["h"] = h
        else:
            out["q"], out["sf"] = _exact_rows(h, case["scales"], ld)
        return out

    names = (["gu"] if case["gu"] else []) + (["h"] if case["out"] == "h" else ["q", "sf"])
    if case["mode"] == "dense":
        got = one(s["a"], s["sfa"], s["b"], s["sfb"], _ld(case["rows"]))
        return {k: got[k] for k in names}
    full = {k: (torch.zeros(s[k].shape, dtype=torch.float64, device=DEV) if k != "sf" else
                _sf_value(case["scales"], s["sf"]).double()) for k in names}
    per = 4 if packed else 1
    if case["mode"] == "masked":
        for e, n in enumerate(s["counts"].tolist()):
            if n:
                ld = s["sfa"].shape[-1]
                got = one(s["a"][e, :n], s["sfa"][e], s["b"][e], s["sfb"][e], ld)
                for k in names:
                    if k == "sf":
                        full[k][e] = got[k]
                    else:
                        full[k][e, :n] = got[k]
        return full
    idx = s["idx"].cpu()
    for e in range(case["G"]):
        at = (idx == e).nonzero().flatten()
        if not at.numel():
            continue
        lo, n = int(at[0]), at.numel()
        got = one(s["a"][lo:lo + n], s["sfa"][:, lo:lo + n], s["b"][e], s["sfb"][e], n)
        for k in names:
            if k == "sf":
                full[k][:, lo * per:(lo + n) * per] = got[k]
            else:
                full[k][lo:lo + n] = got[k]
    return full
