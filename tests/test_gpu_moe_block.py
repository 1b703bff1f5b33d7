"""The example block (examples/moe_block.py) against plain torch: bfloat16
paths to 1% (a few roundings of 2^-9 each), the FP8 experts to 13%, twice
what their roundings come to: an e4m3 value is off by 2^-5.3 rms, the gate and
up products each by sqrt 2 of that, their product by 2 of it, and the requantised
result and the last weights by one each: sqrt(6) 2^-5.3 = 6.2%."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_block_against_plain_torch():
    import moe_block
    for name, v in moe_block.main().items():
        assert v < (0.13 if name.startswith("serve") else 0.01), (name, v)


def test_masked_and_contiguous_serve_alike():
    import moe_block
    p = moe_block.make(3)
    x = torch.randn(40, moe_block.H, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    adapter = torch.full((40,), 2, dtype=torch.int32, device="cuda")
    a, b = (moe_block.serve(p, x, adapter, d) for d in (True, False))
    assert moe_block.far(a, b) < 0.01
