"""The example model: prompts and single tokens through all the layer operators agree."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,fp8,most", [("float32", False, 1e-4), ("bfloat16", False, 5e-2)])
def test_decode_agrees_with_prefill(cuda_lib, dtype, fp8, most):
    """The same tokens one by one and in one prefill.  f32: four layers of sums of up to 1024 f32 terms,
    2^-24 * sqrt(1024) * 10 products in a row is 2e-5, with room to 1e-4; bf16: a rounding of 2^-9 after
    each of about 40 operations in a row, 40 * 2^-9 = 8e-2 if all added up, sqrt(40) * 2^-9 = 1.2e-2 if
    independent."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mamba_decode
    tokens, distance = mamba_decode.run(getattr(torch, dtype), fp8)
    assert tokens.shape == (4, 16)
    assert distance < most


def test_fp8_norm_in_the_model(cuda_lib):
    """With the norms' outputs in 8 bits the logits keep their direction (e4m3 rounds by up to 2^-4)."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mamba_decode
    tokens, distance = mamba_decode.run(torch.bfloat16, True)
    assert tokens.shape == (4, 16) and distance < 0.5
