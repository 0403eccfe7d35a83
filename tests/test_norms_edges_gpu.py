"""Edges of the norms around a block: rows of more groups than fit 32-bit thread
numbers. Tolerances as in test_norms_gpu.py.
"""
import pytest
import torch

from selective_state_space_depthwise_b200 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


@pytest.mark.parametrize("group,more", [(1, 27), (8, 29)])
def test_gated_norm_of_rows_with_more_threads_than_32_bits_count(group, more):
    """A team of 32 (8) threads for each of 2^27 (2^29) groups of a row, and three more."""
    groups = (1 << more) + 3
    x = torch.ones(1, groups * group, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(1000 * group, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[0, -tail.numel():] = tail
    w = 0.5 + torch.arange(group, device="cuda") / 16.0
    out = torch.zeros_like(x)
    api.gated_norm(x, None, w, group_size=group, out=out)
    torch.cuda.synchronize()
    t = tail.double().reshape(-1, group)
    want = t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
    got = out[0, -tail.numel():].double().reshape(-1, group)
    assert ((got - want).abs() <= (2.0 ** -8 + 1e-5) * want.abs()).all()
    one = (w.double() / (1 + 1e-5) ** 0.5).bfloat16()
    head = out[0, :-tail.numel()].reshape(-1, group)
    for i in range(group):
        assert (head[:, i] == one[i]).all()
