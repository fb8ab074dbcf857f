"""A gated feed-forward block in FP8, put together from the library's calls.

    h   = x + residual                        (the residual stream, kept)
    n   = rmsnorm(h) * w_norm                 rmsnorm_quantize_e4m3_1x128
    a   = act(n Wg^T) * (n Wu^T)              fp8_gated_gemm_nt
    out = a Wd^T                              fp8_gemm_nt

forward() serves decode and prefill; forward(save=True) and backward() are a
training step.  Every operand of a matrix product is E4M3 with block scales;
what flows between the products in 8 bits is written there by the operator
before it, so the layer has no separate quantiser pass in its forward.

    python -m moe_grouped_gemm_scaled_amd.ffn [tokens]

runs one training step and a few decode steps on random weights and prints the
distance to the same layer in fp32.
"""
from __future__ import annotations

import sys

import torch

from . import binding as dg


class GatedFFN:
    """w_norm [H]; w_gate, w_up [I, H]; w_down [H, I] (fp32 or bf16, on the device; H and I multiples of 128)."""

    def __init__(self, w_norm, w_gate, w_up, w_down, act="silu", eps=1e-6):
        self.w_norm = w_norm.contiguous()
        self.act, self.eps = act, eps
        self.I, self.H = w_gate.shape
        self.gu, self.sf_gu = dg.quantize_e4m3_128x128(torch.stack([w_gate.float(), w_up.float()]))
        self.down, self.sf_down = dg.quantize_e4m3_128x128(w_down.float().contiguous())
        # the backward pass multiplies by the same codes, transposed (the NN
        # layout); its scales are laid out [N/128][K/128]
        self.sf_gu_t = self.sf_gu.view(2 * self.I // 128, self.H // 128).t().contiguous()
        self.sf_down_t = self.sf_down.t().contiguous()

    def forward(self, x, residual, save=False):
        """x, residual [T, H] bf16 -> (out [T, H] bf16, the new residual stream, what backward() needs)."""
        T = x.shape[0]
        q, sf, h, n = dg.rmsnorm_quantize_e4m3_1x128(x, self.w_norm, self.eps, residual=residual, y=True if save else None)
        _, qa, sfa, gu = dg.fp8_gated_gemm_nt(q, sf, self.gu, self.sf_gu, act=self.act, q=True, gu=True if save else None)
        out = torch.empty((T, self.H), dtype=torch.bfloat16, device=x.device)
        dg.fp8_gemm_nt(qa, sfa, self.down, self.sf_down, out)
        return out, h, (h, n, gu) if save else None

    def backward(self, saved, dout, dh=None):
        """dout [T, H] bf16: gradient of out; dh: gradient of the residual stream (h's type) or None.
        Returns (gradient of x and of the residual, {name: weight gradient})."""
        h, n, gu = saved
        T, dev = dout.shape[0], dout.device
        bf16 = torch.bfloat16
        # d a = dout Wd
        qd, sfd = dg.quantize_e4m3_1x128(dout.float())
        da = torch.empty((T, self.I), dtype=bf16, device=dev)
        dg.fp8_gemm("nn", qd, sfd, self.down, self.sf_down_t, da)
        # through the gate, quantised for the two products below
        _, q, sf, qt, sft, at, sfat = dg.gated_backward_quantize_e4m3(gu, da, act=self.act, q=True, qt=True, ht=True)
        # d n = [d gate, d up] [Wg; Wu]
        dn = torch.empty((T, self.H), dtype=bf16, device=dev)
        dg.fp8_gemm("nn", q, sf, self.gu.view(2 * self.I, self.H), self.sf_gu_t, dn)
        dx, dw_norm = dg.rmsnorm_backward(dn, h, self.w_norm, self.eps, dres=dh)
        # weight gradients: the K axis is the tokens, padded to whole blocks with zeros
        nq, sfn = self._by_blocks(n)
        dw = torch.empty((2 * self.I, self.H), dtype=bf16, device=dev)
        dg.fp8_gemm("tn", qt, sft, nq, sfn, dw)
        dq, sfdq = self._by_blocks(dout)
        dw_down_t = torch.empty((self.I, self.H), dtype=bf16, device=dev)
        dg.fp8_gemm("tn", at, sfat, dq, sfdq, dw_down_t)
        return dx, {"w_norm": dw_norm, "w_gate": dw[:self.I], "w_up": dw[self.I:], "w_down": dw_down_t.t()}

    @staticmethod
    def _by_blocks(x):
        """x [T, N] as codes [T padded to 128, N] with 128x128 scales laid out [N/128][T/128]."""
        pad = -x.shape[0] % 128
        q, sf = dg.quantize_e4m3_128x128(torch.nn.functional.pad(x.float(), (0, 0, 0, pad)))
        return q, sf.t().contiguous()


def reference(w_norm, w_gate, w_up, w_down, x, residual, act="silu", eps=1e-6):
    """The same layer in plain torch: out and the residual stream."""
    h = x + residual
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * w_norm
    gate = n @ w_gate.t()
    a = torch.nn.functional.silu(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
    return (a * (n @ w_up.t())) @ w_down.t(), h


def random_weights(H, I, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    def rand(*shape, scale):
        return torch.randn(*shape, generator=g, device=device) * scale
    return (1 + rand(H, scale=0.1), rand(I, H, scale=H ** -0.5), rand(I, H, scale=H ** -0.5), rand(H, I, scale=I ** -0.5))


def main(tokens=300, H=1024, I=512):
    weights = random_weights(H, I)
    layer = GatedFFN(*weights)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dout = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, stream, saved = layer.forward(x, res, save=True)
    dx, grads = layer.backward(saved, dout)
    params = [w.clone().requires_grad_() for w in weights]
    xr = x.float().requires_grad_()
    want, _ = reference(*params, xr, res.float())
    want.backward(dout.float())
    def far(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())
    print(f"training step, {tokens} tokens: out {far(out, want):.3f}, dx {far(dx, xr.grad):.3f}, "
          + ", ".join(f"d{k} {far(grads[k], p.grad):.3f}" for k, p in zip(("w_norm", "w_gate", "w_up", "w_down"), params)),
          flush=True)
    stream = res[:1]
    y = x[:1]
    for step in range(4):
        y, stream, _ = layer.forward(y, stream)
    print(f"decode: 4 steps of one token, |out| {float(y.float().norm()):.3f}", flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
