"""Edges of the gated delta rule: values that are not finite in one head of a
pair, decode rows at their default strides, keys and queries whose squares
overflow, packed cuts on their edges, correlated keys. Tolerances as in
test_delta_gpu.py.
"""
import ctypes
import math

import pytest
import torch

from delta_util import inputs, rule
from selective_state_space_depthwise_b200 import _lib, api
from test_delta_gpu import check, state0

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [0, 1])
@pytest.mark.parametrize("what,value", [("g", NAN), ("g", INF), ("g", 100.0), ("beta", NAN), ("beta", INF), ("v", NAN)])
@pytest.mark.parametrize("form", ["one walk", "segments", "packed", "packed cut", "shares"])
def test_a_head_that_is_not_finite_leaves_its_pair_alone(form, what, value, bad):
    """Two heads of 64 value channels on one key group are walked together. A decay, beta or value of one that is not
    finite, or decays that leave the range of fp32 within a chunk, must not reach the other."""
    G, H, dk, dv = 1, 2, 128, 64
    lens = {"one walk": [200], "segments": [2500], "packed": [70, 200, 33], "packed cut": [90, 2500, 130],
            "shares": [1100] * 3}[form]
    if form == "shares":
        H = 160
    packed = form.startswith("packed")
    i = 1 if packed else 0           # the sequence with the bad value
    t = 2 * lens[i] // 3
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    x = inputs(lead, G, H, dk, dv, seed=len(form), decay=0.3, l2norm=True)
    clean = {n: y.clone() for n, y in x.items()}
    row, at = (0, sum(lens[:i]) + t) if packed else (0, t)
    if what == "v":
        x["v"][row, at, bad, 5] = value
    else:
        x[what][row, at, bad] = value
    if packed:
        cu = torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        out, st = api.delta_prefill(**{n: y[0] for n, y in x.items()}, qk_l2norm=True, cu_seqlens=cu)
        out = out[None]
        seqs = [(0, sum(lens[:n]), sum(lens[:n + 1])) for n in range(len(lens))]
    else:
        out, st = api.delta_prefill(**x, qk_l2norm=True)
        seqs = [(n, 0, lens[n]) for n in range(len(lens))]
    torch.cuda.synchronize()
    for n, (b, a, e) in enumerate(seqs):
        want, wst = rule(**{m: y[b:b + 1, a:e] for m, y in clean.items()}, l2norm=True)
        keep = [h for h in range(H) if n != i or h != bad]
        check(out[b:b + 1, a:e, keep], st[n:n + 1, keep], want[:, :, keep], wst[:, keep], f"sequence {n}")
        if n == i and not math.isfinite(value):
            check(out[b:b + 1, a:a + t, bad], torch.zeros(1), want[:, :t, bad], torch.zeros(1), "before the value")
            after, s = out[b, a + t:e, bad], st[n, bad]
            if what == "v":
                after, s = after[:, 5], s[5]
            assert not torch.isfinite(after).any() and not torch.isfinite(s).any()


def test_decode_rows_do_not_follow_the_token_strides():
    """The dims of a prefill out of a fused buffer, given to decode with dense rows: the rows are dense. (The buffers
    are as long as rows at the token strides would be.)"""
    lib = _lib.load()
    b, G, H, dk, dv = 5, 2, 4, 64, 72
    nk, nv, wide = G * dk, H * dv, 2 * G * dk + H * dv
    x = inputs((b, 1), G, H, dk, dv, seed=5)
    d = _lib.SsmDeltaDims(b, 9, H, G, dk, dv, 0.0, 0, wide, 0, wide, 0, wide, 0, wide, 0, H + 4, 0)

    def rows(t, stride):
        buf = torch.full((b * stride + 64,), 7.0, dtype=t.dtype, device="cuda")
        buf[:t.numel()] = t.reshape(-1)
        return buf

    buf = {n: rows(t, H + 4 if n in ("g", "beta") else wide) for n, t in x.items()}
    out = torch.full((b * wide + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(b, H, dv, dk, device="cuda")
    _lib.check(lib.ssm_delta_decode_step(ctypes.byref(d), *(buf[n].data_ptr() for n in ("q", "k", "v", "g", "beta")),
                                         None, b, st.data_ptr(), out.data_ptr(), st.data_ptr(), None))
    torch.cuda.synchronize()
    check(out[:b * nv].reshape(b, 1, H, dv), st, *rule(**x))
    assert (out[b * nv:] == 7).all()


@pytest.mark.parametrize("L", [1, 2, 17, 40, 64, 100, 2500])
@pytest.mark.parametrize("l2norm", [False, True])
@pytest.mark.parametrize("dk", [64, 128])
def test_keys_whose_squares_overflow(L, l2norm, dk):
    """A finite key with a sum of squares beyond fp32: as a key that is not finite, at every length."""
    t, H, dv = 2 * L // 3, 2, 128
    x = inputs((2, L), 1, H, dk, dv, seed=L, decay=0.1, l2norm=l2norm)
    want, wst = rule(**x, l2norm=l2norm)
    x["k"][0, t] = 1e20
    out, st = api.delta_prefill(**x, qk_l2norm=l2norm)
    check(out[:1, :t], torch.zeros(1), want[:1, :t], torch.zeros(1))
    check(out[1:], st[1:], want[1:], wst[1:])
    assert not torch.isfinite(out[0, t:]).any() and not torch.isfinite(st[0]).any()
    if L == 1:
        s0 = torch.zeros(2, H, dv, dk, device="cuda")
        out = api.delta_decode_step(**{n: y[:, 0] for n, y in x.items()}, state=s0, qk_l2norm=l2norm)
        check(out[1:, None], s0[1:], want[1:], wst[1:])
        assert not torch.isfinite(out[0]).any() and not torch.isfinite(s0[0]).any()


@pytest.mark.parametrize("L", [1, 17, 40, 64, 100, 2500])
@pytest.mark.parametrize("dv", [64, 128])
def test_queries_whose_squares_overflow(L, dv):
    """A finite query with a sum of squares beyond fp32 has no norm: its output is not a number, and nothing else."""
    t, H, dk = 2 * L // 3, 2, 128
    x = inputs((2, L), 1, H, dk, dv, seed=L, l2norm=True)
    want, wst = rule(**x, l2norm=True)
    x["q"][0, t] = 1e20
    out, st = api.delta_prefill(**x, qk_l2norm=True)
    assert out[0, t].isnan().all()
    out[0, t], want[0, t] = 0, 0
    check(out, st, want, wst)
    if L == 1:
        s0 = torch.zeros(2, H, dv, dk, device="cuda")
        out = api.delta_decode_step(**{n: y[:, 0] for n, y in x.items()}, state=s0, qk_l2norm=True)
        assert out[0].isnan().all()
        check(out[1:, None], s0, want[1:], wst)


@pytest.mark.parametrize("given", [False, True])
def test_packed_buffers_without_tokens_pass_the_states_on(given):
    x = {n: t[0] for n, t in inputs((1, 0), 1, 2, 64, 128, seed=1).items()}
    s0 = torch.randn(3, 2, 128, 64, device="cuda") if given else None
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, st = api.delta_prefill(**x, cu_seqlens=cu, state_in=s0)
    torch.cuda.synchronize()
    assert out.shape == (0, 2, 128) and torch.equal(st, s0 if given else torch.zeros_like(st))


@pytest.mark.parametrize("lens", [
    [513] * 60 + [8] * 100, [1100] * 9 + [1] * 200, [577, 5, 577, 64] * 20, [4000] + [513] * 30, [512] * 40 + [2100],
])
def test_packed_cuts_stay_inside_their_workspace(lens):
    """Many packed sequences just long enough to be cut, next to shorter ones: results, and nothing behind the
    workspace."""
    T, n, G, H, dk, dv = sum(lens), len(lens), 1, 2, 64, 72
    x = {m: t[0] for m, t in inputs((1, T), G, H, dk, dv, seed=T, decay=0.05).items()}
    at = torch.tensor([0] + lens).cumsum(0)
    need = api.delta_prefill_workspace_bytes(n, T, H, G, dk, dv, packed=True)
    ws = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    s0 = torch.randn(n, H, dv, dk, device="cuda")
    out, st = api.delta_prefill(**x, cu_seqlens=at.int().cuda(), state_in=s0, workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0x5A).all()
    for m in sorted(set(lens)):
        which = [i for i in range(n) if lens[i] == m]
        rows = torch.stack([torch.arange(at[i], at[i] + m) for i in which]).cuda()
        want = rule(**{k: t[rows] for k, t in x.items()}, state=s0[which])
        check(out[rows], st[which], *want, f"length {m}")


@pytest.mark.parametrize("L", [64, 300, 2500])
@pytest.mark.parametrize("noise", [0.0, 0.05, 0.5])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_correlated_keys(L, noise, decay):
    """Keys near plus or minus one direction and beta near 1: the chunk's system is then far from the identity, and its
    inverse's terms cancel."""
    b, G, H, dk, dv = 2, 1, 4, 128, 64
    x = inputs((b, L), G, H, dk, dv, seed=L, decay=decay)
    gen = torch.Generator().manual_seed(L)
    sign = torch.randint(0, 2, (b, L, G, 1), generator=gen) * 2.0 - 1
    k = sign * torch.randn(b, 1, G, dk, generator=gen) / dk ** 0.5
    k = k + noise * torch.randn(b, L, G, dk, generator=gen) / dk ** 0.5
    x["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).bfloat16().cuda()
    x["beta"] = (1 - 0.02 * torch.rand(b, L, H, generator=gen)).cuda()
    s0 = state0(b, H, dv, dk, 9)
    out, st = api.delta_prefill(**x, state_in=s0)
    check(out, st, *rule(**x, state=s0))


@pytest.mark.parametrize("L", [64, 100, 128, 300, 2048])
@pytest.mark.parametrize("noise", [0.0, 0.01, 0.05])
@pytest.mark.parametrize("alternate", [False, True])
def test_keys_alike_and_nothing_forgotten(L, noise, alternate):
    """beta = 1, no decay and keys that are (nearly) one, with either sign: entries of the chunk's system are alike, and
    what its products leave out would add up over the tokens instead of averaging out."""
    b, G, H, dk, dv = 2, 8, 8, 128, 128
    x = inputs((b, L), G, H, dk, dv, seed=L, decay=0.0)
    gen = torch.Generator().manual_seed(7 * L)
    k = torch.randn(b, 1, G, dk, generator=gen) / dk ** 0.5
    if alternate:
        k = k * (torch.randint(0, 2, (b, L, G, 1), generator=gen) * 2.0 - 1)
    k = k + noise * torch.randn(b, L, G, dk, generator=gen) / dk ** 0.5
    x["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).bfloat16().cuda()
    x["beta"].fill_(1.0)
    check(*api.delta_prefill(**x), *rule(**x))
