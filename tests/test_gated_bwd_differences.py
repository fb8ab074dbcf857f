"""Every element of the gated activation's gradient against central differences
in 64 bits.  h = act(gate) * up is taken element by element, so one pair of
evaluations shifted by t gives the derivative of sum(dh * h) along every gate
at once, and another pair along every up.  The bar is one element's: half a
bf16 ulp, the fp32 arithmetic (2^-20 (2 + 2|g| + 0.1|g|^3) of the factors,
through the logistic function's argument), and the differences' own error: t^2
/ 6 of the third derivative (below 4 for both activations) and the rounding of
two values of size |act|, 2^-52 |act| / t.

On the CPU the same bar is put to gradients with one mistake each, which it has
to refuse."""
import sys

import numpy as np
import pytest
import torch

from layer_helpers import act, act_grad, bf16, check_bf16, f64, logistic, normal

ROWS, I, T = 130, 256, 1e-5


def inputs(kind):
    seed = 70 if kind == "silu" else 80
    return bf16(2 * normal(seed, (ROWS, 2 * I))), bf16(normal(seed + 1, (ROWS, I)))


def check_gradient(dgu, gu, dh, kind, where):
    g, u, d = f64(gu)[:, :I], f64(gu)[:, I:], f64(dh)
    fp32 = 2.0 ** -20 * (2 + 2 * np.abs(g) + 0.1 * np.abs(g) ** 3)
    num = d * u * (act(g + T, kind) - act(g - T, kind)) / (2 * T)
    size = np.abs(d * u)
    check_bf16(dgu[:, :I], num, size * (fp32 + T * T + 2.0 ** -52 * (1 + np.abs(g)) / T), where + " d_gate")
    num = (d * act(g, kind) * (u + T) - d * act(g, kind) * (u - T)) / (2 * T)
    size = np.abs(d * act(g, kind))
    check_bf16(dgu[:, I:], num, size * (fp32 + 2.0 ** -52 * (1 + np.abs(u)) / T), where + " d_up")


def formula(gu, dh, kind):
    g, u, d = f64(gu)[:, :I], f64(gu)[:, I:], f64(dh)
    return d * u * act_grad(g, kind), d * act(g, kind)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_the_bar_accepts_the_formula_and_refuses_mistakes(kind):
    gu, dh = inputs(kind)
    g, u, d = f64(gu)[:, :I], f64(gu)[:, I:], f64(dh)
    dg_, du_ = formula(gu, dh, kind)
    check_gradient(bf16(np.concatenate([dg_, du_], 1)), gu, dh, kind, "formula")
    other = "gelu" if kind == "silu" else "silu"
    v = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    one_term = dg_.copy()
    one_term[0, 0] *= 1.02                                           # one element, 2 % off
    mistakes = {"without the term of the logistic function's slope": (d * u * logistic(v), du_),
                "d_gate 2 % large": (1.02 * dg_, du_), "d_up 2 % small": (dg_, 0.98 * du_),
                "d_up without the activation": (dg_, d * g), "the other activation": (d * u * act_grad(g, other), du_),
                "gate and up exchanged": (du_, dg_), "one element": (one_term, du_)}
    for name, (a, b) in mistakes.items():
        with pytest.raises(AssertionError):
            check_gradient(bf16(np.concatenate([a, b], 1)), gu, dh, kind, name)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_every_element(kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from moe_grouped_gemm_scaled_amd import binding as dg
    print(f"\n[case] gated_bwd, every element against differences, {kind}", file=sys.stderr, flush=True)
    gu, dh = inputs(kind)
    dgu = dg.gated_backward_quantize_e4m3(gu.cuda(), dh.cuda(), kind, dgu=True)[0]
    check_gradient(dgu, gu, dh, kind, "kernel")
