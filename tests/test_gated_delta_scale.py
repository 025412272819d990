"""The scale of the gated delta rule's binding: 0 means 1 / sqrt(d_k) to the library, so no value may become it."""
import pytest


@pytest.mark.parametrize("scale", [0.0, -0.0, 0, 1e-50, -1e-46])
def test_a_scale_that_is_zero_in_float32_is_refused(scale):
    import torch
    from linear_recurrent_sequence_amd import retention as R
    with pytest.raises(ValueError, match="scale"):
        R._delta_scale(scale)
    with pytest.raises(ValueError):
        R._delta_scale(torch.tensor(scale))


@pytest.mark.parametrize("scale,want", [(None, 0.0), (1e-40, 1e-40), (1, 1.0), (-0.25, -0.25)])
def test_others_pass(scale, want):
    from linear_recurrent_sequence_amd import retention as R
    assert R._delta_scale(scale) == want
