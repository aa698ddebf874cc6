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


def _logits(fp8, group, d_model, dtype):
    """Last tokens' logits of one prefill, of a model whose weights and tokens depend on neither fp8 nor group."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mamba_decode
    model = mamba_decode.Mamba(layers=4, d_model=d_model, dtype=getattr(torch, dtype), fp8=fp8, group=group, seed=3)
    g = torch.Generator("cuda").manual_seed(4)
    tokens = torch.randint(0, model.embedding.shape[0], (4, 64), device="cuda", generator=g)
    lens = torch.tensor([37, 5, 64, 1], dtype=torch.int32, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    return model.prefill(tokens, lens, model.new_cache(4), slots)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("group,d_model", [(0, 512), (128, 512), (128, 528)])
def test_fp8_norm_against_the_norm_in_the_models_type(cuda_lib, group, d_model, dtype):
    """The same weights and tokens with the norms' outputs in 8 bits and without.

    e4m3 is off by 2^-3 / sqrt(12) rms in a binade's [1, 2), 0.025 of the value, e say.  A layer's output is a product of
    two branches of its input, so off by 2 (e + d) (added as independent errors) for an input that is off by d; the
    residual is the sum of as many such outputs as there were layers, which gives 0.05, 0.09, 0.13 and 0.17 after four
    layers, and 0.17 for the logits: held to twice that.  Rounding is as often up as down, so the logits' size (their
    projection on those without) moves only with the square of it: held to 0.1, which a scale that is off by that much
    in the last norm alone breaks."""
    want, got = _logits(False, 0, d_model, dtype), _logits(True, group, d_model, dtype)
    assert float((got - want).norm() / want.norm()) < 0.35
    assert abs(float((got * want).sum() / (want * want).sum()) - 1) < 0.1
    assert not (got == want).all()


def test_fp8_groups_decode_agrees_with_prefill(cuda_lib):
    """As test_fp8_norm_in_the_model, with a scale for each 128 columns."""
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mamba_decode
    tokens, distance = mamba_decode.run(torch.bfloat16, True, group=128)
    assert tokens.shape == (4, 16) and distance < 0.5
