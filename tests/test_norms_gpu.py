"""Gated group norm and residual norm (ssm_gated_norm, ssm_residual_norm)
against their definitions in float64, and the residual block forward against
its two steps.

Tolerances. An output is rounded once: half a step of its type (2^-8 of the
value in bf16, 2^-24 in fp32). Inside, fp32: the sum of n squares has relative
error at most about sqrt(n) 2^-24 (of either sign; n <= 32768: 1.1e-5, and half
of that in its root), the sigmoid and the root 2^-22 each, a few products 2^-24
each: 1e-5 in all for the longest rows, 3e-6 up to 8192 channels. Relative L2 and
every element are held to half a step plus that.
"""
import numpy as np
import pytest
import torch

from selective_state_space_depthwise_b200 import api
from selective_state_space_depthwise_b200 import workloads as W

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def rnd(*shape, seed, dtype=F32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def close(got, want, inner=1e-5):
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    lim = (HALF_STEP[got.dtype] + inner) * want.abs() + 1e-30
    d = (got.double() - want).abs()
    assert (d <= lim).all(), f"off by up to {float((d / want.abs().clamp_min(1e-30)).max()):.2e} of the value"


def gated(x, z, w, group, first, eps=1e-5):
    x, w = x.double(), w.double()
    gate = 1.0 if z is None else z.double() * torch.sigmoid(z.double())
    t = (x * gate if first else x).unflatten(-1, (-1, group))
    y = t / (t.square().mean(-1, keepdim=True) + eps).sqrt()
    y = y * (w.unflatten(0, (-1, group)) if w.shape[0] == x.shape[-1] else w)
    y = y.flatten(-2)
    return y if first else y * gate


@pytest.mark.parametrize("dim,group", [
    (8, 8), (64, 64), (128, 64), (1280, 80), (1024, 1024), (384, 128), (1000, 1000), (2056, 1028), (2560, 2560),
    (8192, 8192), (15360, 7680), (32768, 32768), (1, 1), (7, 7), (33, 11), (771, 771), (999, 333), (4097, 4097),
    (5001, 5001), (32767, 32767),
])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_sizes(dim, group, dtype, first):
    x, z = rnd(5, dim, seed=dim, dtype=dtype), rnd(5, dim, seed=dim + 1, dtype=dtype)
    for w in (rnd(dim, seed=2), rnd(group, seed=3)):
        close(api.gated_norm(x, z, w, group_size=group, gate_first=first), gated(x, z, w, group, first))


def test_gated_norm_rows_and_no_gate():
    for rows in (1, 2, 63, 1000):
        x, w = rnd(rows, 256, seed=rows, dtype=BF16), rnd(256, seed=1)
        close(api.gated_norm(x, None, w, group_size=64), gated(x, None, w, 64, False))
        close(api.gated_norm(x, None, w, group_size=64, gate_first=True), gated(x, None, w, 64, False))
    x = rnd(0, 256, seed=1)
    assert api.gated_norm(x, x, rnd(256, seed=2)).shape == (0, 256)


@pytest.mark.parametrize("offset", [0, 1, 8])
def test_gated_norm_strides_and_in_place(offset):
    """x and z as halves of a fused buffer [b, L, 2 D + ...] at aligned and unaligned columns; out over x, over z."""
    b, L, D = 2, 9, 192
    buf = rnd(b, L + 1, 2 * D + 16, seed=5, dtype=BF16)
    keep = buf.clone()
    x, z = buf[:, :L, offset:offset + D], buf[:, :L, offset + D:offset + 2 * D]
    w = rnd(D, seed=6)
    want = gated(x, z, w, 64, False)
    close(api.gated_norm(x, z, w, group_size=64), want)
    close(api.gated_norm(x, z, w, group_size=64, out=x), want)
    assert torch.equal(buf[..., :offset], keep[..., :offset]) and torch.equal(buf[:, L:], keep[:, L:])
    assert torch.equal(buf[..., offset + D:], keep[..., offset + D:])
    buf.copy_(keep)
    close(api.gated_norm(x, z, w, group_size=64, out=z), want)


def test_gated_norm_zero_rows_and_extreme_gates():
    """Rows of zeros are normalised by eps alone; gates at the ends of SiLU."""
    x = rnd(4, 128, seed=8)
    z = rnd(4, 128, seed=9)
    x[1] = 0
    z[2] = -200.0
    z[3, :64] = 80.0
    w = rnd(128, seed=10)
    got = api.gated_norm(x, z, w)
    torch.cuda.synchronize()
    assert (got[1] == 0).all() and (got[2].abs() < 1e-30).all()
    close(got[[0, 3]], gated(x, z, w, 128, False)[[0, 3]])
    got = api.gated_norm(x, z, w, gate_first=True)
    torch.cuda.synchronize()
    assert (got[1] == 0).all() and torch.isfinite(got).all()


def residual(x, r, w, post, alpha, eps=1e-5):
    norm = lambda t, u: t / (t.square().mean(-1, keepdim=True) + eps).sqrt() * u.double()  # noqa: E731
    t = x.double()
    if post is not None:
        t = norm(t, post)
    out = alpha * t if r is None else r.double() + alpha * t
    return norm(out, w), out


@pytest.mark.parametrize("dim", [1, 8, 64, 200, 771, 2560, 4097, 8192, 8200, 32760, 32767, 32768])
@pytest.mark.parametrize("io,res", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_sizes(dim, io, res, post):
    """x and the residual on scales where their sum does not cancel to less than a rounding of its terms."""
    x, r, w = rnd(3, dim, seed=dim, dtype=io).abs() + 0.5, rnd(3, dim, seed=dim + 1, dtype=res).abs() + 0.5, rnd(dim, seed=2)
    p = rnd(dim, seed=3).abs() + 0.5 if post else None
    y, ro = api.residual_norm(x, r, w, post_weight=p, residual_scale=0.3)
    wy, wr = residual(x, r, w, p, float(np.float32(0.3)))
    close(y, wy)
    close(ro, wr)
    assert ro.dtype == res and y.dtype == io


def test_residual_norm_first_block_in_place_and_3d():
    x, w = rnd(2, 6, 256, seed=11, dtype=BF16), rnd(256, seed=12)
    y, r = api.residual_norm(x, None, w, residual_dtype=F32)
    wy, wr = residual(x, None, w, None, 1.0)
    close(y, wy), close(r, wr)
    x2, r0 = rnd(2, 6, 256, seed=13, dtype=BF16).abs() + 0.1, r.abs()
    wy, wr = residual(x2, r0, w, None, 1.0)
    y2, r2 = api.residual_norm(x2, r0, w, residual_out=r0, out=x2)
    assert r2.data_ptr() == r0.data_ptr() and y2.data_ptr() == x2.data_ptr()
    close(y2, wy), close(r0, wr)
    x0 = rnd(0, 64, seed=1)
    assert api.residual_norm(x0, x0, rnd(64, seed=1))[0].shape == (0, 64)


@pytest.mark.parametrize("offset", [0, 3])
def test_residual_norm_strides(offset):
    buf, rb = rnd(7, 300, seed=14, dtype=BF16).abs() + 0.1, rnd(7, 280, seed=15).abs() + 0.1
    x, r, w = buf[:, offset:offset + 256], rb[:, offset:offset + 256], rnd(256, seed=16)
    ob = torch.full((7, 272), 5.0, dtype=BF16, device="cuda")
    y, ro = api.residual_norm(x, r, w, out=ob[:, offset:offset + 256])
    wy, wr = residual(x, r, w, None, 1.0)
    close(y, wy), close(ro, wr)
    assert (ob[:, :offset] == 5).all() and (ob[:, offset + 256:] == 5).all()


def test_norms_streams_and_graphs():
    x, z, w, r = rnd(64, 512, seed=17, dtype=BF16), rnd(64, 512, seed=18, dtype=BF16), rnd(512, seed=19), rnd(64, 512, seed=20)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    close(api.gated_norm(x, z, w, group_size=128, stream=s), gated(x, z, w, 128, False))
    graph = torch.cuda.CUDAGraph()
    api.residual_norm(x, r, w)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = api.gated_norm(x, z, w, group_size=128)
        y2, r2 = api.residual_norm(y, r, w)
    x.copy_(rnd(64, 512, seed=21, dtype=BF16))
    graph.replay()
    close(y, gated(x, z, w, 128, False))
    close(y2, residual(y, r, w, None, 1.0)[0], inner=1e-4)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("first", [False, True])
def test_residual_block_equals_its_steps(post, first):
    """The layer is its two calls: bit for bit, the conv cache and the state among it."""
    wl = W.Workload("residual_block", batch=2, seqlen=70, d_inner=128, seed=6)
    inp = W.make_block_inputs(wl, 64, device="cuda")
    proj = {k: inp[k] for k in api.PROJ_NAMES}
    x, w = inp["hidden"], rnd(64, seed=22)
    r = None if first else rnd(2, 70, 64, seed=23)
    p = rnd(64, seed=24) if post else None
    out, ro, cc, st = api.residual_block_forward(x, r, inp, proj, w, post_weight=p, residual_scale=0.5)
    hidden, want_r = api.residual_norm(x, r, w, post_weight=p, residual_scale=0.5, residual_dtype=F32)
    want = api.block_forward(hidden, inp, proj)
    torch.cuda.synchronize()
    assert torch.equal(ro, want_r) and torch.equal(out, want[0])
    assert torch.equal(cc, want[1]) and torch.equal(st, want[2])
    # the next layer, its output over its input and its residual in place
    out2, ro2, _, _ = api.residual_block_forward(out, ro, inp, proj, w, out=out, residual_out=ro)
    hidden, want_r2 = api.residual_norm(want[0], want_r, w)
    want2 = api.block_forward(hidden, inp, proj)
    torch.cuda.synchronize()
    assert torch.equal(ro2, want_r2) and torch.equal(out2, want2[0])


def test_delta_layer_end_to_end():
    """A gated-delta layer as it is used: residual norm, projection, rule, gated norm, projection, over a prompt and
    then token by token, against float64 with bf16 at the same places. Five roundings to bf16 lie between x and out
    (hidden, the projection, the rule's and the norm's output, the last product), each of at most 2^-8, about 2^-9.2 RMS:
    2^-9.2 sqrt(5) < 4e-3, and q, k's rounding enters the rule twice: relative L2 at most 1e-2."""
    from delta_util import rel_l2, rule

    b, L, D, G, H, dk, dv = 2, 90, 256, 2, 4, 64, 64
    nk, nv = G * dk, H * dv
    x, r = rnd(b, L, D, seed=30, dtype=BF16), rnd(b, L, D, seed=31)
    w1, w2 = 1 + 0.1 * rnd(D, seed=32), 1 + 0.1 * rnd(dv, seed=33)
    Win = (rnd(2 * nk + 2 * nv, D, seed=34) * D ** -0.5).to(BF16)
    Wout = (rnd(D, nv, seed=35) * nv ** -0.5).to(BF16)
    g, beta = -0.1 * rnd(b, L, H, seed=36).abs(), torch.sigmoid(rnd(b, L, H, seed=37))

    def layer(x, r, g, beta, state, decode):
        n = x.shape[1]
        hidden, ro = api.residual_norm(x, r, w1)
        p = api.proj_gemm(hidden.reshape(-1, D), Win).reshape(b, n, -1)
        q, k = (p[..., i * nk:(i + 1) * nk].unflatten(-1, (G, dk)) for i in range(2))
        v, z = p[..., 2 * nk:2 * nk + nv].unflatten(-1, (H, dv)), p[..., 2 * nk + nv:]
        if decode:
            o = api.delta_decode_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state, qk_l2norm=True)[:, None]
        else:
            o, state = api.delta_prefill(q, k, v, g, beta, state_in=state, qk_l2norm=True)
        y = api.gated_norm(o.flatten(-2), z, w2, group_size=dv)
        return api.proj_gemm(y.reshape(-1, nv), Wout).reshape(b, n, D), ro, state

    out, ro, state = layer(x[:, :80].contiguous(), r[:, :80].contiguous(), g[:, :80], beta[:, :80], None, False)
    outs, ros = [out], [ro]
    for t in range(80, L):
        o, rr, _ = layer(x[:, t:t + 1].contiguous(), r[:, t:t + 1].contiguous(), g[:, t:t + 1], beta[:, t:t + 1], state, True)
        outs.append(o), ros.append(rr)
    torch.cuda.synchronize()
    hidden, want_r = residual(x, r, w1, None, 1.0)
    p = hidden.to(BF16).double() @ Win.double().T
    p = p.to(BF16).double()
    q, k = (p[..., i * nk:(i + 1) * nk].unflatten(-1, (G, dk)) for i in range(2))
    v, z = p[..., 2 * nk:2 * nk + nv].unflatten(-1, (H, dv)), p[..., 2 * nk + nv:]
    o, st = rule(q, k, v, g, beta, l2norm=True)
    y = gated(o.to(BF16).flatten(-2), z, w2, dv, False).to(BF16)
    want = y.double() @ Wout.double().T
    assert rel_l2(torch.cat(ros, 1), want_r) <= 1e-6
    assert rel_l2(torch.cat(outs, 1), want) <= 1e-2 and rel_l2(state, st) <= 1e-2
