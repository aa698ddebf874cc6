"""The gated delta rule, the convolution and the norms together, as a model uses them (examples/delta_decode.py)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,most", [("float32", 1e-4), ("bfloat16", 5e-2)])
def test_decode_agrees_with_prefill(cuda_lib, dtype, most):
    """The same tokens one by one and in one prefill.  f32: three layers of sums of up to 1032 f32 terms,
    2^-24 * sqrt(1032) * 10 products in a row is 2e-5, with room to 1e-4; bf16: a rounding of 2^-9 after
    each of about 30 operations in a row, 6e-2 if all added up, sqrt(30) * 2^-9 = 1.1e-2 if independent."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import delta_decode
    tokens, distance = delta_decode.run(getattr(torch, dtype))
    assert tokens.shape == (4, 16)
    assert distance < most
