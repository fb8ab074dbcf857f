"""A mixture of gated feed-forward experts in FP8, put together from the
library's calls.

    h       = x + residual                            (the residual stream)
    n       = layernorm(h)                            layernorm_quantize_e4m3_1x128
    ids, w  = top_k of n R^T, softmax over the chosen (torch)
    rows    = a row for each token and choice         moe_sort_contiguous / moe_sort_masked
    n_e     = n in the experts' rows                  moe_dispatch_..
    a_e     = act(n_e Wg_e^T) * (n_e Wu_e^T)          m_grouped_fp8_gated_gemm_nt_contiguous / _masked
    y_e     = a_e Wd_e^T                              m_grouped_fp8_gemm_nt_contiguous / _masked
    out     = h + sum_j w_j y_e[rows_j]               moe_combine

forward() serves prefill (contiguous segments), decode() a batch of single
tokens (a fixed number of rows per expert, nothing read back by the host);
forward(save=True) and backward() are a training step.

    python -m moe_grouped_gemm_scaled_amd.moe [tokens]

runs one training step and a few decode steps on random weights and prints the
distance to the same layer in fp32.
"""
from __future__ import annotations

import sys

import torch

from . import binding as dg


def _transposed(codes, sf):
    """[G, N, K] codes with [G, N/128, K/128] scales as the weights of the transposed product, [G, K, N]."""
    return codes.transpose(1, 2).contiguous(), sf.transpose(1, 2).contiguous()


class MoEFFN:
    """w_norm, b_norm [H]; router [G, H]; w_gate, w_up [G, I, H]; w_down [G, H, I] (fp32 or bf16, on the device; H and I
    multiples of 128)."""

    def __init__(self, w_norm, b_norm, router, w_gate, w_up, w_down, top_k, act="silu", eps=1e-5, training=True):
        self.w_norm, self.b_norm = w_norm.contiguous(), b_norm.contiguous()
        self.router = router.float().contiguous()
        self.top_k, self.act, self.eps = top_k, act, eps
        self.G, self.I, self.H = w_gate.shape
        G, I, H = self.G, self.I, self.H
        both = torch.stack([w_gate.float(), w_up.float()], 1)                       # [G, 2, I, H]
        q, sf = dg.quantize_e4m3_128x128(both.view(2 * G, I, H))
        self.gu, self.sf_gu = q.view(G, 2, I, H), sf.view(G, 2, I // 128, H // 128)
        self.down, self.sf_down = dg.quantize_e4m3_128x128(w_down.float().contiguous())
        if training:
            # the backward pass multiplies by the same codes, transposed
            self.gu_t, self.sf_gu_t = _transposed(self.gu.view(G, 2 * I, H), self.sf_gu.view(G, 2 * I // 128, H // 128))
            self.down_t, self.sf_down_t = _transposed(self.down, self.sf_down)

    def _route(self, n):
        top, ids = (n.float() @ self.router.t()).topk(self.top_k, dim=1)
        return ids.int(), torch.softmax(top, 1)

    def forward(self, x, residual, save=False):
        """x, residual [T, H] bf16 -> (the new residual stream [T, H] bf16, what backward() needs)."""
        dev, bf16 = x.device, torch.bfloat16
        q, sf, h, n = dg.layernorm_quantize_e4m3_1x128(x, self.w_norm, self.b_norm, self.eps, residual=residual, y=True)
        ids, w = self._route(n)
        rows, src, m_indices, _, ks = dg.moe_sort_contiguous(ids, self.G, src=True if save else None, ks=True if save else None)
        R = m_indices.shape[0]
        # the norm's own codes, of n before its rounding to bf16, whether or not a backward pass follows
        nq, sfn = dg.moe_dispatch_e4m3_contiguous(q, sf, rows, R)
        if save:                                       # n along columns too, for the weight gradient
            _, _, nqt, sfnt, _ = dg.moe_dispatch_quantize_e4m3_contiguous(n, rows, R, src=src, q=False, qt=True)
        _, a, sfa, gu = dg.m_grouped_fp8_gated_gemm_nt_contiguous(nq, sfn, self.gu, self.sf_gu, m_indices, act=self.act, q=True,
                                                                  gu=True if save else None)
        y = torch.empty((R, self.H), dtype=bf16, device=dev)
        dg.m_grouped_fp8_gemm_nt_contiguous(a, sfa, self.down, self.sf_down, y, m_indices)
        out = dg.moe_combine(y, rows, weights=w, residual=h)
        return out, (h, n, ids, w, rows, src, m_indices, ks, nqt, sfnt, gu, y) if save else None

    def decode(self, x, residual, M_cap=None):
        """The same for a batch of single tokens: M_cap rows per expert (T when None: no pair can be left without)."""
        T, dev, bf16 = x.shape[0], x.device, torch.bfloat16
        M_cap = T if M_cap is None else M_cap
        q, sf, h, n = dg.layernorm_quantize_e4m3_1x128(x, self.w_norm, self.b_norm, self.eps, residual=residual, y=True)
        ids, w = self._route(n)
        rows, _, masked_m = dg.moe_sort_masked(ids, self.G, M_cap)
        nq, sfn = dg.moe_dispatch_e4m3_masked(q, sf, rows, self.G, M_cap)
        _, a, sfa, _ = dg.m_grouped_fp8_gated_gemm_nt_masked(nq, sfn, self.gu, self.sf_gu, masked_m, act=self.act, q=True)
        y = torch.empty((self.G, M_cap, self.H), dtype=bf16, device=dev)
        dg.m_grouped_fp8_gemm_nt_masked(a, sfa, self.down, self.sf_down, y, masked_m)
        return dg.moe_combine(y, rows, weights=w, residual=h)

    def backward(self, saved, dout):
        """dout [T, H] bf16: gradient of forward()'s output.  Returns (gradient of x and of the residual, {name: weight
        gradient})."""
        h, n, ids, w, rows, src, m_indices, ks, nqt, sfnt, gu, y = saved
        G, I, H, R, dev, bf16 = self.G, self.I, self.H, y.shape[0], dout.device, torch.bfloat16
        # through the combine: the weights, and the experts' rows in both directions
        dw, _, dyq, sfdy, dyqt, sfdyt = dg.moe_combine_backward_quantize_e4m3_contiguous(dout, y, rows, w, src=src, dw=True,
                                                                                        q=True, qt=True)
        da = torch.empty((R, I), dtype=bf16, device=dev)
        dg.m_grouped_fp8_gemm_nt_contiguous(dyq, sfdy, self.down_t, self.sf_down_t, da, m_indices)
        _, gq, sfg, gqt, sfgt, aqt, sfat = dg.gated_backward_quantize_e4m3(gu, da, act=self.act, m_indices=m_indices, q=True,
                                                                           qt=True, ht=True)
        dn_rows = torch.empty((R, H), dtype=bf16, device=dev)
        dg.m_grouped_fp8_gemm_nt_contiguous(gq, sfg, self.gu_t, self.sf_gu_t, dn_rows, m_indices)
        # weight gradients: the K axis of each expert is its segment of rows
        d_gu = torch.empty((G, 2 * I, H), device=dev)
        dg.k_grouped_fp8_gemm_tn_contiguous(gqt, sfgt, nqt, sfnt, ks, d_gu)
        d_down_t = torch.empty((G, I, H), device=dev)
        dg.k_grouped_fp8_gemm_tn_contiguous(aqt, sfat, dyqt, sfdyt, ks, d_down_t)
        # through the router: softmax over the chosen
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        dlogits = torch.zeros((n.shape[0], G), device=dev).scatter_(1, ids.long(), dl)
        dn = dg.moe_combine(dn_rows, rows, residual=dlogits @ self.router)
        dx, d_norm, db_norm = dg.layernorm_backward(dn, h, self.w_norm, self.eps, dres=dout)
        return dx, {"w_norm": d_norm, "b_norm": db_norm, "router": dlogits.t() @ n.float(), "w_gate": d_gu[:, :I],
                    "w_up": d_gu[:, I:], "w_down": d_down_t.transpose(1, 2)}


def reference(w_norm, b_norm, router, w_gate, w_up, w_down, x, residual, ids, act="silu", eps=1e-5):
    """The same layer in plain torch, with the experts of each token given."""
    h = x + residual
    n = torch.nn.functional.layer_norm(h, h.shape[-1:], w_norm, b_norm, eps)
    ids = ids.long()
    w = torch.softmax((n @ router.t()).gather(1, ids), 1)
    f = torch.nn.functional.silu if act == "silu" else lambda v: torch.nn.functional.gelu(v, approximate="tanh")
    out = h
    for e in range(router.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            y = (f(n[t] @ w_gate[e].t()) * (n[t] @ w_up[e].t())) @ w_down[e].t()
            out = out.index_add(0, t, y * w[t, j].unsqueeze(1))
    return out


def random_weights(H, I, G, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape, scale):
        return torch.randn(*shape, generator=g, device=device) * scale

    return (1 + rand(H, scale=0.1), rand(H, scale=0.1), rand(G, H, scale=H ** -0.5), rand(G, I, H, scale=H ** -0.5),
            rand(G, I, H, scale=H ** -0.5), rand(G, H, I, scale=I ** -0.5))


def main(tokens=300, H=1024, I=512, G=8, top_k=2):
    weights = random_weights(H, I, G)
    layer = MoEFFN(*weights, top_k=top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dout = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, saved = layer.forward(x, res, save=True)
    dx, grads = layer.backward(saved, dout)
    params = [v.clone().requires_grad_() for v in weights]
    xr = x.float().requires_grad_()
    want = reference(*params, xr, res.float(), saved[2])
    want.backward(dout.float())

    def far(a, b):
        a, b = a.detach().float(), b.detach().float()
        return float((a - b).norm() / b.norm())

    h = x.float() + res.float()
    names = ("w_norm", "b_norm", "router", "w_gate", "w_up", "w_down")
    print(f"training step, {tokens} tokens: out - h {far(out.float() - h, want - h):.3f}, dx {far(dx, xr.grad):.3f}, "
          + ", ".join(f"d{k} {far(grads[k], p.grad):.3f}" for k, p in zip(names, params)), flush=True)
    stream = res[:4]
    for step in range(4):
        stream = layer.decode(x[:4], stream)
    print(f"decode: 4 steps of 4 tokens, |stream| {float(stream.float().norm()):.3f}", flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
