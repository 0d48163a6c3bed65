"""The decode step of examples/decode_step.py: append, attention, projection and the
fixed-order fold of W ranks' partial sums, against the layer in 64 bits."""
import os
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("world,dtype", [(1, torch.bfloat16), (2, torch.bfloat16), (4, torch.float16), (2, torch.float32)])
def test_decode_steps_on_ranks(world, dtype):
    import decode_step
    error, apart = decode_step.main(world=world, dtype=dtype)
    # the layer's intermediate values (queries, keys, values, attended heads) are rounded to the type, four times,
    # each by at most its unit roundoff relative to its norm's terms: a handful of roundoffs, taken as eight. The
    # projection in binary32 on tensor or FMA units adds 512 terms' roundings.
    unit = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -17}[dtype]
    assert error < 8 * unit
    # two attentions of the same values, each output rounded once
    assert apart < 2 * unit
