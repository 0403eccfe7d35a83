"""Edges of the norms around a block: rows of more groups than fit 32-bit thread
numbers, results over inputs, a layer without tokens. Tolerances as in
test_norms_gpu.py.
"""
import pytest
import torch

from selective_state_space_depthwise_b200 import api
from selective_state_space_depthwise_b200 import workloads as W

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


@pytest.mark.parametrize("dim", [64, 771, 2560, 20000])
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_results_over_inputs(dim, post):
    """y over x or over the residual, the sum over the other: as with buffers of their own."""
    gen = torch.Generator().manual_seed(dim)
    x, r = (torch.randn(37, dim, generator=gen).bfloat16().cuda() for _ in range(2))
    w, p = (1 + 0.1 * torch.randn(dim, generator=gen).cuda() for _ in range(2))
    kw = dict(post_weight=p if post else None, residual_scale=0.5)
    want = api.residual_norm(x, r, w, **kw)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        y, s = api.residual_norm(a, b, w, **kw, out=b if swap else a, residual_out=a if swap else b)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(s, want[1])


def test_residual_block_without_tokens_passes_its_caches_on():
    wl = W.Workload("residual_block", batch=2, seqlen=8, d_inner=128, seed=6)
    inp = W.make_block_inputs(wl, 64, device="cuda")
    proj = {k: inp[k] for k in api.PROJ_NAMES}
    x = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    cc, st = torch.randn(2, 3, 128, device="cuda").bfloat16(), torch.randn(2, 128, 16, device="cuda")
    out, r, cc2, st2 = api.residual_block_forward(x, None, inp, proj, torch.ones(64, device="cuda"), conv_cache_in=cc,
                                                  ssm_state_in=st)
    torch.cuda.synchronize()
    assert out.shape == r.shape == (2, 0, 64) and torch.equal(cc2, cc) and torch.equal(st2, st)
