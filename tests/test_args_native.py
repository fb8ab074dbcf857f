"""The binding's native argument checks on tensors whose address torch refuses
to give (fake tensors under torch.vmap, batched tensors): the checks decline,
and the binding raises torch's error, as its checks in Python do.  In a child
process, since an exception that left the C entry would end the interpreter."""
import os
import subprocess
import sys

import pytest

from moe_grouped_gemm_scaled_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from moe_grouped_gemm_scaled_amd import _args, binding as dg

assert dg._native_addresses is _args.addresses
BF16 = 1
with FakeTensorMode():
    x = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")

    def inside(row):
        assert _args.addresses(0, row, BF16, (256,)) is None
        raised = []
        for native in (_args.addresses, lambda *_: None):
            dg._native_addresses = native
            try:
                dg._pointers(0, ("row",), row, BF16, (256,))
            except RuntimeError as e:
                raised.append(type(e))
        assert raised == [RuntimeError, RuntimeError], raised
        return row.clone()

    torch.vmap(inside)(x)
    # the other tensors of a call do not matter, before or after
    torch.vmap(lambda r: (_args.addresses(0, None, BF16, (), r, BF16, (256,), None, BF16, ()) is None or 1 / 0) and r.clone())(x)
assert _args.addresses(0, None, BF16, ()) == (None,)
assert _args.addresses(0, torch.zeros(3), 2, (3,)) is None        # not on the device
print("declined")
"""


@pytest.mark.skipif(not os.path.exists(build.ARGS), reason="the native checks are not built")
def test_tensors_without_an_address():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "declined" in r.stdout, (r.returncode, r.stderr[-2000:])
