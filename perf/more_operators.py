"""Measured cases of the operators around a mixture of experts: layer norm, and
the tokens' way to the experts' rows and back.

Five operators, in plain torch (own = False) and through the library's entry
points (own = True):
  ln           residual addition + layer norm + E4M3 quantisation (1x128 scales)
  ln_bwd       its gradient: dx, dw and db
  dispatch     token pairs sorted by expert (a row for each token and choice, the
               expert of each row, the counts) and the tokens' values written to
               those rows: quantised along rows, and along columns for a weight
               gradient, or their codes and scales copied
  combine      the experts' rows back to their tokens: weighted sum and residual
               (without weights: the gradient of dispatch)
  combine_bwd  its gradient: the weights' and the rows', quantised in both
               directions for the gradient GEMMs

Layouts are the library's: codes E4M3, A scales [K/128][ld], packed scales four
exponents per int32 along the K blocks, expert segments of 128-row blocks
(contiguous) or of M_cap rows each (masked), column scales [R/128][K].  Hidden
7168 is that of the library's grouped workloads; the rest are generic.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-5
MOST = 8192 * 4 * 7168          # (token, choice, column) triples of the largest listed cases


def listed():
    return [
        # one decode step of a 64-request batch, packed scales
        {"name": "ln decode", "op": "ln", "rows": 64, "K": 7168, "res": True, "x": "bf16", "stream": "bf16",
         "q": True, "y": False, "scales": "packed"},
        # a prefill chunk of 4096 tokens
        {"name": "ln prefill", "op": "ln", "rows": 4096, "K": 7168, "res": True, "x": "bf16", "stream": "bf16",
         "q": True, "y": False, "scales": "fp32"},
        # a short training sequence with an fp32 residual stream
        {"name": "ln_bwd short", "op": "ln_bwd", "rows": 333, "K": 2048, "stream": "fp32", "dres": True},
        # a long training batch
        {"name": "ln_bwd long", "op": "ln_bwd", "rows": 16384, "K": 7168, "stream": "bf16", "dres": True},
        # one token to its 8 of 64 experts: rows of fixed capacity, packed scales
        {"name": "dispatch one token", "op": "dispatch", "T": 1, "k": 8, "G": 64, "K": 7168, "cap": 16, "x": "bf16",
         "scales": "packed", "cols": False, "drop": False},
        # a decode batch of odd size whose norm left codes and packed scales; some experts live elsewhere
        {"name": "dispatch codes", "op": "dispatch", "T": 333, "k": 6, "G": 32, "K": 2048, "cap": 0, "x": "codes",
         "scales": "packed", "cols": False, "drop": True},
        # a prefill chunk: each token quantised once, written to 8 of 64 experts
        {"name": "dispatch prefill", "op": "dispatch", "T": 4096, "k": 8, "G": 64, "K": 7168, "cap": 0, "x": "bf16",
         "scales": "fp32", "cols": False, "drop": False},
        # a training step: also column-scaled, for the weight gradient
        {"name": "dispatch training", "op": "dispatch", "T": 8192, "k": 4, "G": 16, "K": 7168, "cap": 0, "x": "bf16",
         "scales": "fp32", "cols": True, "drop": False},
        # a decode batch back from the experts
        {"name": "combine decode", "op": "combine", "T": 64, "k": 8, "G": 64, "K": 7168, "cap": 32, "weights": True,
         "res": True, "out": "bf16", "drop": False},
        # a prefill chunk back from the experts
        {"name": "combine prefill", "op": "combine", "T": 4096, "k": 8, "G": 64, "K": 7168, "cap": 0, "weights": True,
         "res": True, "out": "bf16", "drop": False},
        # backward of a short sequence of odd length
        {"name": "combine_bwd short", "op": "combine_bwd", "T": 333, "k": 2, "G": 8, "K": 2048, "x": "bf16",
         "cols": True, "scales": "fp32", "drop": True},
        # backward of a training step
        {"name": "combine_bwd training", "op": "combine_bwd", "T": 8192, "k": 4, "G": 16, "K": 7168, "x": "bf16",
         "cols": True, "scales": "fp32", "drop": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "dispatch", "dispatch", "combine", "combine_bwd"])
    if op in ("ln", "ln_bwd"):
        q = rng.random() < 0.7
        rows, K = _log(rng, 1, 16384), 128 * _log(rng, 2, 128)
        if op == "ln_bwd" or not q:
            K -= 8 * rng.choice([0, 0, 1, 5, 14])       # a width that is no multiple of a block
        stream = rng.choice(["bf16", "bf16", "fp32"])
        if op == "ln_bwd":
            return {"op": op, "rows": min(rows, MOST // 4 // K), "K": K, "stream": stream, "dres": rng.random() < 0.7}
        return {"op": op, "rows": min(rows, MOST // 8 // K), "K": K, "res": rng.random() < 0.7,
                "x": rng.choice(["bf16", "bf16", "fp32"]), "stream": stream, "q": q, "y": not q or rng.random() < 0.4,
                "scales": rng.choice(["fp32", "packed"])}
    T, k, G = _log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 2, 256)
    k = min(k, G)
    K = 128 * _log(rng, 2, 56)
    while _rows_bound(T, k, G) * K > MOST:
        T, K = max(1, T * 3 // 4), max(128, K * 3 // 4 // 128 * 128)
    case = {"op": op, "T": T, "k": k, "G": G, "K": K, "drop": rng.random() < 0.3}
    if op == "combine_bwd":
        return {**case, "x": rng.choice(["bf16", "bf16", "fp32"]), "cols": rng.random() < 0.7,
                "scales": rng.choice(["fp32", "ue8m0"])}
    # rows of fixed capacity: roomy or tight (then some pairs find no row)
    case["cap"] = 4 * (T * k // G // 2 + rng.randint(1, 8)) if rng.random() < 0.3 and T <= 1024 else 0
    if op == "combine":
        return {**case, "weights": rng.random() < 0.7, "res": rng.random() < 0.6, "out": rng.choice(["bf16", "fp32"])}
    x = rng.choice(["bf16", "bf16", "fp32", "codes"])
    cols = case["cap"] == 0 and x != "codes" and rng.random() < 0.4
    return {**case, "x": x, "scales": rng.choice(["fp32", "packed"]), "cols": cols}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32)


def _type(name):
    return F32 if name == "fp32" else BF16


def _ld(rows):
    return (rows + 3) // 4 * 4


def _rows_bound(T, k, G):
    """Rows that hold T * k pairs in segments of whole 128-row blocks, however they fall on G experts."""
    n = T * k
    return (n + 127 * min(G, n)) // 128 * 128


def _pow2_up(s):
    """s rounded up to a power of two (s normal and positive)."""
    u = s.view(torch.int32)
    return torch.where((u & 0x7FFFFF) != 0, (u & 0x7F800000) + 0x800000, u).view(F32)


def _scale(amax, scales):
    s = amax.clamp_min(1e-4) / 448.0
    return s if scales == "fp32" else _pow2_up(s)


def _pack(sf):
    """fp32 powers of two [.., blocks, n] -> int32 words [.., ceil(blocks/4), n], four exponents a word."""
    e = (sf.view(torch.int32) >> 23) & 0xFF
    pad = -e.shape[-2] % 4
    if pad:
        e = torch.cat([e, e.new_zeros(*e.shape[:-2], pad, e.shape[-1])], -2)
    e = e.unflatten(-2, (-1, 4))
    return e[..., 0, :] | (e[..., 1, :] << 8) | (e[..., 2, :] << 16) | (e[..., 3, :] << 24)


def _sf_rows(scales, blocks):
    return (blocks + 3) // 4 if scales == "packed" else blocks


def _sf_buffer(scales, lead, blocks, n):
    return torch.zeros(*lead, _sf_rows(scales, blocks), n, dtype=torch.int32 if scales == "packed" else F32, device=DEV)


def _sf_value(scales, sf):
    """Scales as the values that they stand for."""
    return sf.view(E8M0) if scales == "packed" else sf


def _codes(y, s):
    return (y / s).clamp(-448.0, 448.0).to(E4M3)


def _quant(y, scales):
    """y [rows, K] fp32 -> codes, scales [rows, K/128], one scale per row and 128 columns."""
    b = y.unflatten(-1, (-1, 128))
    s = _scale(b.abs().amax(-1), scales)
    return _codes(b, s.unsqueeze(-1)).flatten(-2), s


def _quant_rows(y, scales, ld):
    """The same with the scales laid out [K/128 (words), ld], zeros past the rows."""
    q, s = _quant(y, scales)
    sf = s.t()
    if scales == "packed":
        sf = _pack(sf.contiguous())
    if ld > sf.shape[-1]:
        sf = torch.cat([sf, sf.new_zeros(sf.shape[0], ld - sf.shape[-1])], -1)
    return q, sf.contiguous()


def _quant_cols(y, scales):
    """y [128 t, N] fp32 -> codes [128 t, N], scales [t, N] fp32: one scale per column and 128 rows."""
    b = y.unflatten(0, (-1, 128))
    s = _scale(b.abs().amax(1), scales)
    return _codes(b, s.unsqueeze(1)).flatten(0, 1), s


def _activations(g, *shape):
    """Values like a residual stream's: N(0, 1) about a small mean, with a few strong columns."""
    x = _randn(g, *shape) + 0.25
    x[..., ::97] *= 8.0
    return x


def _choices(case, g):
    """Experts of each token, best first, some experts more popular than others, and their weights; with `drop`, the
    last quarter of the experts lives elsewhere (no row here)."""
    T, k, G = case["T"], case["k"], case["G"]
    total = G + G // 3 if case["drop"] else G
    logits = _randn(g, T, total) + 0.5 * _randn(g, 1, total)
    v, ids = logits.topk(k, dim=1)
    ids = torch.where(ids < G, ids, -1).to(torch.int32)
    return ids.contiguous(), torch.softmax(v, 1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    K = case["K"]
    s = {"case": case}
    if op in ("ln", "ln_bwd"):
        rows = case["rows"]
        s["w"], s["b"] = (1.0 + 0.2 * _randn(g, K)).to(BF16), (0.1 * _randn(g, K)).to(BF16)
        t = _type(case["stream"])
        if op == "ln_bwd":
            s["dy"], s["h"] = (0.1 * _randn(g, rows, K)).to(BF16), _activations(g, rows, K).to(t)
            s["dx"] = torch.empty(rows, K, dtype=t, device=DEV)
            s["dw"], s["db"] = (torch.empty(K, dtype=F32, device=DEV) for _ in range(2))
            if case["dres"]:
                s["dres"] = (0.1 * _randn(g, rows, K)).to(t)
            return s
        s["x"] = _activations(g, rows, K).to(_type(case["x"]))
        if case["res"]:
            s["res"] = (2.0 * _activations(g, rows, K)).to(t)
            s["res_out"] = torch.empty_like(s["res"])
        if case["y"]:
            s["y"] = torch.empty(rows, K, dtype=BF16, device=DEV)
        if case["q"]:
            s["q"] = torch.zeros(rows, K, dtype=torch.uint8, device=DEV)
            s["sf"] = _sf_buffer(case["scales"], (), K // 128, _ld(rows))
        return s
    T, k, G, cap = case["T"], case["k"], case["G"], case.get("cap", 0)
    s["ids"], s["weights"] = _choices(case, g)
    s["R"] = R = G * cap if cap else _rows_bound(T, k, G)
    lead, per, ld = ((G,), cap, _ld(cap)) if cap else ((), R, R)

    def i32(*shape):
        return torch.empty(*shape, dtype=torch.int32, device=DEV)

    if op == "dispatch":
        x = _activations(g, T, K)
        if case["x"] == "codes":
            q, s["sf_in"] = _quant_rows(x, case["scales"], _ld(T))
            s["x"] = q.view(torch.uint8)
        else:
            s["x"] = x.to(_type(case["x"]))
        s["rows"] = i32(T, k)
        s["q"] = torch.zeros(*lead, per, K, dtype=torch.uint8, device=DEV)
        s["sf"] = _sf_buffer(case["scales"], lead, K // 128, ld)
        if cap:
            s["masked_m"] = i32(G)
        else:
            s["m_indices"], s["ks"] = i32(R), i32(G)
        if case["cols"]:
            s["src"] = i32(R)
            s["qt"] = torch.zeros(R, K, dtype=torch.uint8, device=DEV)
            s["sft"] = torch.zeros(R // 128, K, dtype=F32, device=DEV)
        return s
    plan = _plan(s["ids"], G, R, cap)
    s["rows"], s["src"] = plan["rows"], plan["src"]
    s["y"] = (0.5 * _randn(g, *lead, per, K)).to(BF16)
    if op == "combine":
        t = _type(case["out"])
        s["out"] = torch.empty(T, K, dtype=t, device=DEV)
        if case["res"]:
            s["res"] = _activations(g, T, K).to(t)
        return s
    s["dout"] = (0.1 * _randn(g, T, K)).to(_type(case["x"]))
    s["dw"] = torch.empty(T, k, dtype=F32, device=DEV)
    s["q"] = torch.zeros(R, K, dtype=torch.uint8, device=DEV)
    s["sf"] = _sf_buffer(case["scales"], (), K // 128, R)
    if case["cols"]:
        s["qt"] = torch.zeros(R, K, dtype=torch.uint8, device=DEV)
        s["sft"] = torch.zeros(R // 128, K, dtype=F32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _ln_plain(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if c["res"]:
        h = h + s["res"].float()
        out["res_out"] = h.to(s["res"].dtype)
    d = h - h.mean(-1, keepdim=True)
    y = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS) * s["w"].float() + s["b"].float()
    if c["y"]:
        out["y"] = y.to(BF16)
    if c["q"]:
        out["q"], sf = _quant_rows(y, c["scales"], _ld(c["rows"]))
        out["sf"] = _sf_value(c["scales"], sf)
    return out


def _ln_bwd_plain(s):
    h, dy = s["h"].float(), s["dy"].float()
    d = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = d * r
    gw = dy * s["w"].float()
    dx = r * (gw - gw.mean(-1, keepdim=True) - n * (gw * n).mean(-1, keepdim=True))
    if "dres" in s:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * n).sum(0), "db": dy.sum(0)}


def _plan(ids, G, R, cap):
    """Rows of the pairs sorted by expert, in pair order within one: segments of whole 128-row blocks, or of cap rows."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < G), flat, G)
    counts = torch.zeros(G + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))
    order = torch.sort(key, stable=True).indices
    keys = key[order]
    at = torch.arange(n, device=DEV) - (counts.cumsum(0) - counts)[keys]
    if cap:
        start = torch.arange(G, device=DEV) * cap
        room = torch.full((G,), cap, dtype=torch.int64, device=DEV)
    else:
        full = (counts[:G] + 127) // 128 * 128
        start = full.cumsum(0) - full
        room = (R - start).clamp_min(0)
    e = keys.clamp_max(G - 1)
    held = (keys < G) & (at < room[e])
    row = torch.where(held, start[e] + at, R)
    rows = torch.empty(n, dtype=torch.int64, device=DEV)
    rows[order] = torch.where(held, row, -1)
    src = torch.full((R + 1,), -1, dtype=torch.int64, device=DEV)
    src[row] = order
    expert = torch.full((R + 1,), -1, dtype=torch.int64, device=DEV)
    expert[row] = keys
    out = {"rows": rows.view(ids.shape), "src": src[:R].contiguous()}
    if cap:
        out["masked_m"] = torch.minimum(counts[:G], room)
    else:
        out["m_indices"], out["ks"] = expert[:R].contiguous(), torch.minimum(full, room)
    return {k: v.to(torch.int32) for k, v in out.items()}


def _to_rows(y, src, k):
    """[R, ..]: y of the token that each row holds, zeros elsewhere."""
    live = (src >= 0).unsqueeze(-1)
    return torch.where(live, y[(src.long().clamp_min(0) // k)], torch.zeros((), dtype=y.dtype, device=DEV))


def _scales_to_rows(sf, src, k, G, cap):
    """Token scales [T, n] -> the layout's [.., n, ld]."""
    rows = _to_rows(sf, src, k)
    if not cap:
        return rows.t().contiguous()
    out = torch.zeros(G, sf.shape[1], _ld(cap), dtype=sf.dtype, device=DEV)
    out[..., :cap] = rows.view(G, cap, -1).transpose(1, 2)
    return out


def _dispatch_plain(s):
    c = s["case"]
    T, k, G, K, cap, scales = c["T"], c["k"], c["G"], c["K"], c["cap"], c["scales"]
    out = _plan(s["ids"], G, s["R"], cap)
    src = out["src"]
    if c["x"] == "codes":
        q, sf = s["x"], s["sf_in"][:, :T].t()
    else:
        q, sf = _quant(s["x"].float(), scales)
        q = q.view(torch.uint8)
        if scales == "packed":
            sf = _pack(sf.t().contiguous()).t()
    out["q"] = _to_rows(q, src, k).view(s["q"].shape).view(E4M3)
    out["sf"] = _sf_value(scales, _scales_to_rows(sf, src, k, G, cap))
    if c["cols"]:
        out["qt"], out["sft"] = _quant_cols(_to_rows(s["x"].float(), src, k), "fp32")
    else:
        del out["src"]
    return out


def _combine_plain(s):
    c = s["case"]
    K = c["K"]
    out = s["res"].float() if c["res"] else torch.zeros(c["T"], K, dtype=F32, device=DEV)
    y = s["y"].view(-1, K)
    for j in range(c["k"]):
        r = s["rows"][:, j].long()
        v = y[r.clamp_min(0)].float()
        if c["weights"]:
            v = v * s["weights"][:, j:j + 1]
        out = out + torch.where((r >= 0).unsqueeze(-1), v, 0.0)
    return {"out": out.to(_type(c["out"]))}


def _combine_bwd_plain(s):
    c = s["case"]
    k, K = c["k"], c["K"]
    d = s["dout"].float()
    dw = torch.zeros_like(s["weights"])
    for j in range(k):
        r = s["rows"][:, j].long()
        dw[:, j] = torch.where(r >= 0, (d * s["y"][r.clamp_min(0)].float()).sum(1), 0.0)
    src = s["src"]
    w = torch.where(src >= 0, s["weights"].view(-1)[src.long().clamp_min(0)], 0.0)
    dy = _to_rows(d, src, k) * w.unsqueeze(-1)
    live = src >= 0
    q, sf = _quant_rows(dy, c["scales"], s["R"])
    out = {"dw": dw, "q": torch.where(live.unsqueeze(-1), q.view(torch.uint8), 0).view(E4M3),
           "sf": torch.where(live, sf, 0.0)}
    if c["cols"]:
        out["qt"], out["sft"] = _quant_cols(dy, c["scales"])
    return out


# ---------------------------------------------------------------- the library's calls

_SCALES = {"fp32": "fp32", "ue8m0": "ue8m0", "packed": "ue8m0_packed"}


def _run_own(s):
    from moe_grouped_gemm_scaled_amd import binding as dg
    c = s["case"]
    op = c["op"]
    if op == "ln":
        dg.layernorm_quantize_e4m3_1x128(s["x"], s["w"], s["b"], EPS, residual=s.get("res"), residual_out=s.get("res_out"),
                                         y=s.get("y"), q=s.get("q", False), sf=s.get("sf"), scales=_SCALES[c["scales"]])
        out = {k: s[k] for k in ("res_out", "y") if k in s}
        if c["q"]:
            out["q"], out["sf"] = s["q"].view(E4M3), _sf_value(c["scales"], s["sf"])
        return out
    if op == "ln_bwd":
        dg.layernorm_backward(s["dy"], s["h"], s["w"], EPS, dres=s.get("dres"), dx=s["dx"], dw=s["dw"], db=s["db"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "combine":
        dg.moe_combine(s["y"], s["rows"], weights=s["weights"] if c["weights"] else None, residual=s.get("res"),
                       out=s["out"])
        return {"out": s["out"]}
    if op == "combine_bwd":
        cols = {k: s[k] for k in ("src", "qt", "sft") if c["cols"]}
        dg.moe_combine_backward_quantize_e4m3_contiguous(s["dout"], s["y"], s["rows"], s["weights"], dw=s["dw"], q=s["q"],
                                                         sf=s["sf"], scales=_SCALES[c["scales"]], **cols)
        out = {k: s[k] for k in ("dw", "sf", "sft") if k in s}
        return {**out, **{k: s[k].view(E4M3) for k in ("q", "qt") if k in s}}
    cap = c["cap"]
    if cap:
        dg.moe_sort_masked(s["ids"], c["G"], cap, rows=s["rows"], masked_m=s["masked_m"])
    else:
        dg.moe_sort_contiguous(s["ids"], c["G"], s["R"], rows=s["rows"], m_indices=s["m_indices"], ks=s["ks"],
                               src=s.get("src"))
    if c["x"] == "codes":
        if cap:
            dg.moe_dispatch_e4m3_masked(s["x"], s["sf_in"], s["rows"], c["G"], cap, q=s["q"], sf=s["sf"])
        else:
            dg.moe_dispatch_e4m3_contiguous(s["x"], s["sf_in"], s["rows"], s["R"], q=s["q"], sf=s["sf"])
    elif cap:
        dg.moe_dispatch_quantize_e4m3_masked(s["x"], s["rows"], c["G"], cap, q=s["q"], sf=s["sf"],
                                             scales=_SCALES[c["scales"]])
    else:
        cols = {k: s[k] for k in ("src", "qt", "sft") if c["cols"]}
        rows = {"q": s["q"], "sf": s["sf"]}
        if c["cols"] and c["scales"] == "packed":       # a call has one scale format; the weight gradient's is fp32 here
            dg.moe_dispatch_quantize_e4m3_contiguous(s["x"], s["rows"], s["R"], scales="ue8m0_packed", **rows)
            rows = {}
        scales = _SCALES[c["scales"]] if rows else "fp32"
        dg.moe_dispatch_quantize_e4m3_contiguous(s["x"], s["rows"], s["R"], scales=scales, **rows, **cols)
    out = {k: s[k] for k in ("rows", "src", "masked_m", "m_indices", "ks", "sft") if k in s}
    out.update({k: s[k].view(E4M3) for k in ("q", "qt") if k in s})
    out["sf"] = _sf_value(c["scales"], s["sf"])
    return out


_PLAIN = {"ln": _ln_plain, "ln_bwd": _ln_bwd_plain, "dispatch": _dispatch_plain, "combine": _combine_plain,
          "combine_bwd": _combine_bwd_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and 64-bit values

def _live(case):
    """Pairs that have a row (the expectation over the seeds)."""
    n = case["T"] * case["k"]
    if case["drop"]:
        n = n * case["G"] / (case["G"] + case["G"] // 3)
    return min(n, case["G"] * case["cap"]) if case.get("cap") else n


def work(case):
    op, K = case["op"], case["K"]
    size = {"bf16": 2, "fp32": 4, "codes": 1}
    if op == "ln":
        n = case["rows"] * K
        per = size[case["x"]] + (2 * size[case["stream"]] if case["res"] else 0) + (2 if case["y"] else 0)
        if case["q"]:
            per += 1 + (1 if case["scales"] == "packed" else 4) / 128
        return {"bytes": n * per + 4 * K, "flops": 10 * n}
    if op == "ln_bwd":
        n = case["rows"] * K
        return {"bytes": n * (2 + size[case["stream"]] * (3 if case["dres"] else 2)) + 10 * K, "flops": 16 * n}
    T, n, live = case["T"], case["T"] * case["k"], _live(case)
    R = _rows_bound(T, case["k"], case["G"])
    code = 1 + (1 if case.get("scales") == "packed" else 4) / 128       # a code and its share of a scale
    if op == "combine":
        b = live * K * 2 + n * (8 if case["weights"] else 4) + T * K * size[case["out"]] * (2 if case["res"] else 1)
        return {"bytes": b, "flops": 2 * live * K}
    cols = R * K * (1 + 4 / 128) + 4 * R if case["cols"] else 0
    if op == "combine_bwd":
        b = T * K * size[case["x"]] + live * K * 2 + live * K * code + cols + 12 * n
        return {"bytes": b, "flops": live * K * (8 if case["cols"] else 5)}
    b = T * K * (code if case["x"] == "codes" else size[case["x"]]) + live * K * code + cols + 8 * n
    b += 4 * case["G"] + (0 if case["cap"] else 4 * R)
    return {"bytes": b, "flops": 0 if case["x"] == "codes" else 4 * T * K + (4 * live * K if case["cols"] else 0)}


def _exact_scale(amax, scales):
    s = torch.clamp(amax, min=1e-4) / 448.0
    return s if scales == "fp32" else torch.exp2(torch.ceil(torch.log2(s)))


def _exact_quant(y, scales):
    """Values over their scales (not rounded to codes) [n, K] and the scales [n, K/128] in 64 bits."""
    s = _exact_scale(y.reshape(y.shape[0], -1, 128).abs().max(-1).values, scales)
    return y / s.repeat_interleave(128, 1), s


def _exact_cols(y, scales):
    s = _exact_scale(y.reshape(-1, 128, y.shape[1]).abs().max(1).values, scales)
    return y / s.repeat_interleave(128, 0), s


def _exact_layout(s, rows, ld, scales):
    """Scales [n, blocks] (numbers) at columns `rows` of [blocks (words), ld]; a packed word's unused bytes and the
    words of other columns stand for 2^-127 each."""
    blocks = s.shape[1]
    if scales != "packed":
        out = torch.zeros(blocks, ld, dtype=torch.float64, device=DEV)
        out[:, rows] = s.t()
        return out
    words = (blocks + 3) // 4
    out = torch.full((words * 4, ld), 2.0 ** -127, dtype=torch.float64, device=DEV)
    out[:blocks, rows] = s.t()
    return out.reshape(words, 4, ld).permute(0, 2, 1).reshape(words, 4 * ld)


def _exact_plan(ids, G, R, cap):
    """The plan pair by pair on the host."""
    T, k = ids.shape
    lists = [[] for _ in range(G)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < G:
            lists[e].append(p)
    rows, src, expert, held, full = [-1] * (T * k), [-1] * R, [-1] * R, [], []
    lo = 0
    for e, pairs in enumerate(lists):
        if cap:
            lo, room = e * cap, cap
        else:
            room = max(0, R - lo)
        kept = pairs[:room]
        for i, p in enumerate(kept):
            rows[p], src[lo + i], expert[lo + i] = lo + i, p, e
        held.append(len(kept))
        size = -(-len(pairs) // 128) * 128
        full.append(min(size, room))
        if not cap:
            lo += size

    def dev(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    out = {"rows": dev(rows).view(T, k), "src": dev(src)}
    if cap:
        out["masked_m"] = dev(held)
    else:
        out["m_indices"], out["ks"] = dev(expert), dev(full)
    return out


def exact(case, seed):
    op, K = case["op"], case["K"]
    s = prepare(case, seed)
    if op == "ln":
        h = s["x"].double()
        out = {}
        if case["res"]:
            h = h + s["res"].double()
            out["res_out"] = h
        mu = h.sum(1, keepdim=True) / K
        var = (h - mu).pow(2).sum(1, keepdim=True) / K
        y = (h - mu) / torch.sqrt(var + EPS) * s["w"].double() + s["b"].double()
        if case["y"]:
            out["y"] = y
        if case["q"]:
            out["q"], sf = _exact_quant(y, case["scales"])
            out["sf"] = _exact_layout(sf, slice(0, case["rows"]), _ld(case["rows"]), case["scales"])
        return out
    if op == "ln_bwd":
        h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
        c = h - h.sum(1, keepdim=True) / K
        v = c.pow(2).sum(1, keepdim=True) / K + EPS
        gw = dy * w
        dx = (gw - gw.sum(1, keepdim=True) / K) / v.sqrt() - c * (gw * c).sum(1, keepdim=True) / (K * v * v.sqrt())
        if "dres" in s:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dw": (dy * c / v.sqrt()).sum(0), "db": dy.sum(0)}
    T, k, G, cap, R = case["T"], case["k"], case["G"], case.get("cap", 0), s["R"]
    plan = _exact_plan(s["ids"].cpu(), G, R, cap)
    at = (plan["src"] >= 0).nonzero().flatten()             # rows that hold a pair
    pair = plan["src"][at].long()
    token = torch.div(pair, k, rounding_mode="floor")
    if op == "combine":
        out = s["res"].double() if case["res"] else torch.zeros(T, K, dtype=torch.float64, device=DEV)
        v = s["y"].view(-1, K)[at].double()
        if case["weights"]:
            v = v * s["weights"].view(-1)[pair].double().unsqueeze(1)
        return {"out": out.index_add(0, token, v)}
    scales = case["scales"]

    def place(q):
        full = torch.zeros(R, K, dtype=torch.float64, device=DEV)
        full[at] = q
        return full

    def sums(sf):
        if not cap:
            return _exact_layout(sf, at, R, scales)
        ld = _ld(cap)
        return torch.stack([_exact_layout(sf[at // cap == e], at[at // cap == e] % cap, ld, scales) for e in range(G)])

    if op == "dispatch":
        out = {n: plan[n] for n in ("rows", "masked_m", "m_indices", "ks") if n in plan}
        if case["x"] == "codes":
            sf = s["sf_in"]
            if scales == "packed":
                w = sf.to(torch.int64) & 0xFFFFFFFF
                sf = torch.stack([torch.exp2(((w[b // 4] >> (8 * (b % 4))) & 0xFF).double() - 127) for b in range(K // 128)])
            q, sf = s["x"].view(E4M3).double(), sf[:, :T].t().double()
        else:
            q, sf = _exact_quant(s["x"].double(), scales)
        out["q"], out["sf"] = place(q[token]).view(s["q"].shape), sums(sf[token])
        if case["cols"]:
            out["src"] = plan["src"]
            out["qt"], out["sft"] = _exact_cols(place(s["x"].double()[token]), "fp32")
        return out
    d = s["dout"].double()[token]
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[pair] = (d * s["y"][at].double()).sum(1)
    dy = d * s["weights"].view(-1)[pair].double().unsqueeze(1)
    q, sf = _exact_quant(dy, scales)
    out = {"dw": dw.view(T, k), "q": place(q), "sf": sums(sf)}
    if case["cols"]:
        out["qt"], out["sft"] = _exact_cols(place(dy), scales)
    return out
