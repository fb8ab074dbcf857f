"""GPU tests of what a mixture of experts answers in training and in
inference: the same layer, whether it keeps what backward() needs or not."""
import sys

import pytest
import torch

from moe_grouped_gemm_scaled_amd import binding as dg
from moe_grouped_gemm_scaled_amd import moe

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


@pytest.mark.parametrize("tokens,G,top_k", [(1, 4, 2), (33, 4, 2), (300, 6, 3), (1000, 3, 1)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_and_inference_answer_the_same(tokens, G, top_k, act):
    announce(f"moe forward with and without save tokens={tokens} G={G} top_k={top_k} {act}")
    H, I = 512, 384
    layer = moe.MoEFFN(*moe.random_weights(H, I, G, seed=tokens), top_k=top_k, act=act)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, res = (torch.randn(tokens, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    kept, saved = layer.forward(x, res, save=True)
    out, nothing = layer.forward(x, res)
    assert nothing is None and saved is not None
    assert torch.equal(kept, out)
