"""The scale of the gated delta rule: 0 in the C dims stands for the default, so a given scale must stay above 0 in
fp32, and finite."""
import pytest
import torch

from selective_state_space_depthwise_b200 import api, build


@pytest.mark.parametrize("scale", [1e-50, 1e-46, 0.0, -1.0, float("inf"), float("nan"), 1e39])
def test_scales_that_fp32_cannot_hold_are_refused(scale):
    build.build()
    bf = dict(dtype=torch.bfloat16)
    q, v, g = torch.zeros(1, 8, 2, 64, **bf), torch.zeros(1, 8, 4, 64, **bf), torch.zeros(1, 8, 4)
    with pytest.raises(ValueError, match="scale"):
        api._delta_dims(q, q, v, g, g, v, scale, False, 1, 8, 1, 0)


def test_scales_that_fp32_holds_are_passed_on():
    bf = dict(dtype=torch.bfloat16)
    q, v, g = torch.zeros(1, 8, 2, 64, **bf), torch.zeros(1, 8, 4, 64, **bf), torch.zeros(1, 8, 4)
    for scale, want in ((None, 0.0), (1, 1.0), (0.125, 0.125), (1e-38, torch.tensor(1e-38).item())):
        assert api._delta_dims(q, q, v, g, g, v, scale, False, 1, 8, 1, 0).scale == want
