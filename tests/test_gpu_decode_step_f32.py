"""The decode step of examples/decode_step.py in binary32, to binary32's own limits: nothing
on the way may be held in fewer bits."""
import os
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U = 2.0 ** -24


@pytest.mark.parametrize("world", [1, 2, 4])
def test_decode_steps_in_binary32(world):
    import decode_step
    assert not torch.backends.cuda.matmul.allow_tf32 and torch.get_float32_matmul_precision() == "highest"
    error, apart = decode_step.main(world=world, dtype=torch.float32)
    # Errors taken as independent, relative to norms. A chain of n products is off by about sqrt(n / 6) u of its
    # result: 9 u for the 512-term projection to queries, keys and values. Scores have unit size, so they are off by
    # 9 u of the queries' and 9 u of the keys' error and a few u of their own 64 terms: 13 u, which are the weights'
    # relative errors, with 3 u of their exponentials; the values' 9 u beside them. 17 u in all, and the output
    # projection of up to 512 terms and the fold add 9 u: 20 u. The limit is four times that, 4.8e-6. (One
    # rounding to bfloat16 or TF32 on the way is 2^-9 or 2^-12 of something: 2.4e-4 at least.)
    assert error < 80 * U
    # Two attentions of the same values: weights' exponentials are off by (2 + |x|) u, |x| up to 6 or so, sums
    # and joins by a few u, each against another maximum. Independent over the tokens, and the norm averages them:
    # under 8 u. The limit is twice that.
    assert apart < 16 * U
