"""Gated delta rule (ssm_delta_prefill, ssm_delta_decode_step) against its
float64 definition, token by token.

Tolerances.
 - out is rounded once to bf16, at most half a step (2^-8 of the value); inside,
   fp32 sums, and operands of two bf16 terms (relative error 2^-16 each, three
   of them): relative L2 at most 2^-8 + 1e-4, and every element within 2^-8 of
   its value plus 1e-3 of the tensor's RMS (cancelled sums).
 - the state is fp32 throughout. A token's update rounds sums of up to 128
   products: about sqrt(128) 2^-24 = 7e-7 of the state, of either sign; over a
   memory of about 100 tokens sqrt(100) times that: relative L2 at most 1e-5.
"""
import pytest
import torch

from delta_util import inputs, rel_l2, rule
from selective_state_space_depthwise_b200 import api

pytestmark = pytest.mark.gpu

TOL_OUT, TOL_STATE = 2.0 ** -8 + 1e-4, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def check(out, state, want_out, want_state, label=""):
    torch.cuda.synchronize()
    api.check_device_error()
    if want_out.numel():
        assert torch.isfinite(out).all(), label
        e = rel_l2(out, want_out)
        assert e <= TOL_OUT, f"{label}: out rel-L2 {e:.2e}"
        d = (out.double() - want_out).abs()
        lim = 2.0 ** -8 * want_out.abs() + 1e-3 * want_out.square().mean().sqrt()
        assert (d <= lim).all(), f"{label}: out off by {float((d - lim).max()):.2e} beyond its bound"
    assert torch.isfinite(state).all(), label
    e = rel_l2(state, want_state)
    assert e <= TOL_STATE, f"{label}: state rel-L2 {e:.2e}"


def state0(b, H, dv, dk, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (0.3 * torch.randn(b, H, dv, dk, generator=g)).cuda()


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 449])
def test_prefill_lengths(L):
    x = inputs((2, L), 2, 4, 128, 128, seed=L)
    s0 = state0(2, 4, 128, 128, L)
    check(*api.delta_prefill(**x, state_in=s0), *rule(**x, state=s0), f"L {L}")


@pytest.mark.parametrize("G,H,dk,dv", [
    (1, 1, 8, 8), (1, 3, 24, 40), (2, 2, 32, 64), (3, 6, 64, 64), (2, 4, 64, 128), (1, 2, 72, 136), (2, 4, 96, 192),
    (2, 2, 120, 8), (1, 5, 128, 64), (4, 4, 128, 256), (2, 2, 56, 384), (2, 8, 128, 64), (1, 6, 40, 64),
])
@pytest.mark.parametrize("l2norm", [False, True])
def test_prefill_shapes(G, H, dk, dv, l2norm):
    x = inputs((2, 150), G, H, dk, dv, seed=dk + dv, l2norm=l2norm)
    check(*api.delta_prefill(**x, qk_l2norm=l2norm), *rule(**x, l2norm=l2norm), f"{G} {H} {dk} {dv}")


def test_prefill_scale_and_zero_norm():
    """A given scale; q and k rows of zeros are normalised by the epsilon alone."""
    x = inputs((1, 90), 1, 2, 64, 64, seed=3, l2norm=True)
    x["q"][:, 5] = 0
    x["k"][:, 7] = 0
    check(*api.delta_prefill(**x, qk_l2norm=True, scale=0.37), *rule(**x, l2norm=True, scale=0.37))


@pytest.mark.parametrize("decay", [0.0, 1.0, 30.0, 1000.0])
def test_prefill_decays(decay):
    """No decay at all, an ordinary one, and decays that underflow within a few tokens."""
    x = inputs((2, 300), 2, 4, 128, 128, seed=11, decay=decay)
    s0 = state0(2, 4, 128, 128, 12)
    check(*api.delta_prefill(**x, state_in=s0), *rule(**x, state=s0), f"decay {decay}")


def test_prefill_resets_and_idle_tokens():
    """g = -inf forgets everything before its token; beta = 0 leaves the state to decay; both at chunk borders too."""
    x = inputs((1, 260), 2, 2, 128, 64, seed=13)
    x["g"][:, [0, 40, 63, 64, 130, 131, 259]] = float("-inf")
    x["beta"][:, 64:70] = 0
    x["beta"][:, 127:129] = 0
    s0 = state0(1, 2, 64, 128, 14)
    check(*api.delta_prefill(**x, state_in=s0), *rule(**x, state=s0))


def test_prefill_repeated_keys():
    """One key for all tokens and beta = 1: every step erases the last value (the inverse within a chunk is then far
    from a sum of few terms)."""
    x = inputs((1, 200), 1, 2, 128, 128, seed=15, decay=0.1)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:] = 1.0
    check(*api.delta_prefill(**x), *rule(**x))


def test_prefill_strides_and_guards():
    """q, k, v as slices of one fused buffer, out inside a larger one whose other columns stay as they were."""
    b, L, G, H, dk, dv = 2, 100, 2, 4, 64, 72
    x = inputs((b, L), G, H, dk, dv, seed=17)
    nk, nv = G * dk, H * dv
    buf = torch.full((b, L + 3, 2 * nk + nv + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = buf[:, :L, 8:8 + nk].unflatten(-1, (G, dk))
    k = buf[:, :L, 8 + nk:8 + 2 * nk].unflatten(-1, (G, dk))
    v = buf[:, :L, 8 + 2 * nk:8 + 2 * nk + nv].unflatten(-1, (H, dv))
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    gb = torch.full((b, L + 1, H + 3), float("nan"), device="cuda")
    g, beta = gb[:, :L, :H], torch.empty_like(gb)[:, :L, :H]
    g.copy_(x["g"]), beta.copy_(x["beta"])
    obuf = torch.full((b, L + 2, nv + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[:, 1:L + 1, 8:8 + nv].unflatten(-1, (H, dv))
    got, st = api.delta_prefill(q, k, v, g, beta, out=out)
    check(got, st, *rule(**x))
    assert (obuf[:, 0] == 7).all() and (obuf[:, L + 1:] == 7).all()
    assert (obuf[..., :8] == 7).all() and (obuf[..., 8 + nv:] == 7).all()


@pytest.mark.parametrize("lens", [[5], [64, 64], [1, 130, 0, 63, 65, 2], [0, 0, 7], [200, 1, 1, 1, 310]])
@pytest.mark.parametrize("dk", [64, 128])
def test_prefill_packed(lens, dk):
    """Packed sequences, empty ones among them, inside a buffer whose other rows hold NaN: each equals its own
    sequence, and rows of no sequence keep what they held."""
    G, H, dv, T = 2, 4, 128, sum(lens)
    x = inputs((1, T), G, H, dk, dv, seed=T, l2norm=True)
    s0 = state0(len(lens), H, dv, dk, T + 1)
    tail = 9
    pad = lambda t: torch.cat([t[0], torch.full_like(t[0, :1], float("nan")).expand(tail, *t.shape[2:])])  # noqa: E731
    p = {n: pad(t).contiguous() for n, t in x.items()}
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    out = torch.full((T + tail, H, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    got, st = api.delta_prefill(**p, cu_seqlens=cu, state_in=s0, qk_l2norm=True, out=out)
    torch.cuda.synchronize()
    assert (got[T:] == 5).all()
    at = 0
    for i, n in enumerate(lens):
        want = rule(**{m: t[:, at:at + n] for m, t in x.items()}, state=s0[i:i + 1], l2norm=True)
        check(got[None, at:at + n], st[i:i + 1], *want, f"sequence {i} of {lens}")
        at += n


def test_packed_neighbours_do_not_leak():
    """NaN in one packed sequence (q, k, v, g, beta) reaches neither its neighbours nor other heads of v."""
    lens, G, H, dk, dv = [70, 30, 100], 1, 2, 128, 128
    x = inputs((1, 200), G, H, dk, dv, seed=23)
    p = {n: t[0].clone() for n, t in x.items()}
    for t in p.values():
        t[70:100] = float("nan")
    cu = torch.tensor([0, 70, 100, 200], dtype=torch.int32, device="cuda")
    got, st = api.delta_prefill(**p, cu_seqlens=cu)
    for i, (a, e) in enumerate(((0, 70), (70, 100), (100, 200))):
        if i == 1:
            assert got[a:e].isnan().all() and st[i].isnan().all()
        else:
            check(got[None, a:e], st[i:i + 1], *rule(**{m: t[:, a:e] for m, t in x.items()}))
    p = {n: t[0].clone() for n, t in x.items()}
    p["v"][10, 0] = float("nan")
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    got, st = api.delta_prefill(**p, cu_seqlens=cu)
    want, wst = rule(**x)
    check(got[None, :, 1], st[:, 1], want[:, :, 1], wst[:, 1])
    assert got[10:, 0].isnan().all() and torch.isfinite(got[:10, 0]).all()


def test_cu_seqlens_are_clamped():
    """Entries past the buffer or decreasing ones: the rows that they name inside it, and no others."""
    x = inputs((1, 80), 1, 2, 64, 64, seed=29)
    p = {n: t[0] for n, t in x.items()}
    cu = torch.tensor([0, 50, 500, 20], dtype=torch.int32, device="cuda")  # 0..50, 50..80, empty
    got, st = api.delta_prefill(**p, cu_seqlens=cu)
    for i, (a, e) in enumerate(((0, 50), (50, 80))):
        check(got[None, a:e], st[i:i + 1], *rule(**{m: t[:, a:e] for m, t in x.items()}))
    torch.cuda.synchronize()
    assert (st[2] == 0).all()


def test_empty_sequences_pass_the_state_on():
    x = inputs((2, 0), 1, 2, 64, 64, seed=31)
    s0 = state0(2, 2, 64, 64, 32)
    out, st = api.delta_prefill(**x, state_in=s0)
    torch.cuda.synchronize()
    assert out.shape == (2, 0, 2, 64) and torch.equal(st, s0)
    out, st = api.delta_prefill(**x)
    torch.cuda.synchronize()
    assert (st == 0).all()


@pytest.mark.parametrize("cut", [1, 64, 100, 191])
def test_pieces_equal_the_whole_and_state_in_place(cut):
    x = inputs((2, 300), 2, 4, 128, 128, seed=37)
    want = rule(**x)
    st = torch.zeros(2, 4, 128, 128, device="cuda")
    outs = []
    for a, e in ((0, cut), (cut, 300)):
        o, got = api.delta_prefill(**{n: t[:, a:e] for n, t in x.items()}, state_in=st, state_out=st)
        assert got.data_ptr() == st.data_ptr()
        outs.append(o)
    check(torch.cat(outs, 1), st, *want, f"cut {cut}")


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (40, 72)])
def test_prefill_then_decode_equals_prefill(dk, dv):
    x = inputs((3, 100), 2, 4, dk, dv, seed=41, l2norm=True)
    want_out, want_state = rule(**x, l2norm=True)
    out, st = api.delta_prefill(**{n: t[:, :80] for n, t in x.items()}, qk_l2norm=True)
    outs = [out]
    for t in range(80, 100):  # token t of [b, T, ...] tensors in place
        outs.append(api.delta_decode_step(*(x[n][:, t] for n in ("q", "k", "v", "g", "beta")), st,
                                          qk_l2norm=True)[:, None])
    check(torch.cat(outs, 1), st, want_out, want_state)


def test_long_sequences():
    """Thousands of tokens, one and two sequences, against the definition."""
    for b, L, H in ((1, 6001, 2), (2, 2500, 4)):
        x = inputs((b, L), 1, H, 128, 128, seed=L)
        s0 = state0(b, H, 128, 128, L)
        check(*api.delta_prefill(**x, state_in=s0), *rule(**x, state=s0), f"{b} x {L}")


@pytest.mark.parametrize("decay", [0.02, 1.0])
@pytest.mark.parametrize("b,L,G,H,dk,dv", [(1, 3000, 2, 2, 128, 128), (1, 9001, 1, 1, 96, 40), (2, 2111, 1, 3, 64, 192),
                                           (1, 4097, 4, 16, 128, 128), (2, 3003, 1, 4, 128, 64), (1, 2500, 1, 2, 64, 64)])
def test_long_sequences_of_few_heads(b, L, G, H, dk, dv, decay):
    """Walked in segments that are joined: decays weak enough that the first state reaches the last segment, and
    state_out over state_in."""
    x = inputs((b, L), G, H, dk, dv, seed=L, decay=decay, l2norm=True)
    s0 = state0(b, H, dv, dk, L)
    want = rule(**x, state=s0, l2norm=True)
    check(*api.delta_prefill(**x, state_in=s0, qk_l2norm=True), *want)
    out, st = api.delta_prefill(**x, state_in=s0, state_out=s0, qk_l2norm=True)
    check(out, st, *want)
    assert st.data_ptr() == s0.data_ptr()


@pytest.mark.parametrize("lens,G,H,dk,dv", [
    ([5000], 1, 2, 128, 128), ([3000, 0, 1, 700, 64], 2, 4, 64, 72), ([130, 4097, 63, 2000], 1, 3, 128, 192),
    ([1] * 40 + [3333] + [70] * 9, 2, 8, 128, 128), ([9] * 299 + [2500], 1, 2, 64, 64), ([0] * 20 + [2100], 1, 1, 128, 8),
    ([130, 2900, 63, 1, 0, 200], 1, 4, 128, 64),
])
def test_long_packed_sequences(lens, G, H, dk, dv):
    """Long packed sequences, cut into segments on the device, next to short and empty ones; more sequences than are
    cut."""
    T, n = sum(lens), len(lens)
    x = inputs((1, T), G, H, dk, dv, seed=T, decay=0.05)
    s0 = state0(n, H, dv, dk, T)
    at = torch.tensor([0] + lens).cumsum(0)
    out, st = api.delta_prefill(**{m: t[0] for m, t in x.items()}, state_in=s0, cu_seqlens=at.int().cuda())
    # the sequences of one length together
    for m in sorted(set(lens)):
        which = [i for i in range(n) if lens[i] == m]
        rows = torch.stack([torch.arange(at[i], at[i] + m) for i in which]).cuda()
        want = rule(**{k: t[0][rows] for k, t in x.items()}, state=s0[which])
        check(out[rows], st[which], *want, f"length {m}")


@pytest.mark.parametrize("L", [17, 130, 200, 2500, 2501])
@pytest.mark.parametrize("what", ["k", "g", "beta", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_behind_their_token(L, what, value):
    """A key, decay, beta or value that is not finite at one token: outputs before it are those of the shorter
    sequence, none from it on is finite (of v: in its row and head), and so is the state."""
    t, H, dv = 2 * L // 3, 2, 64 if L % 4 else 72  # 64: the two heads are walked as a pair
    x = inputs((1, L), 1, H, 128, dv, seed=L, decay=0.1)
    want, _ = rule(**{n: y[:, :t] for n, y in x.items()})
    bad = {n: y.clone() for n, y in x.items()}
    if what == "k":
        bad["k"][0, t, 0, 5] = value
    elif what == "v":
        bad["v"][0, t, 1, 7] = value
    else:
        bad[what][0, t] = value
    out, st = api.delta_prefill(**bad)
    check(out[:, :t], torch.zeros(1), want, torch.zeros(1))
    if what == "v":
        assert not torch.isfinite(out[0, t:, 1, 7]).any() and not torch.isfinite(st[0, 1, 7]).any()
        keep = torch.ones(H, dv, dtype=torch.bool)
        keep[1, 7] = False
        full, wst = rule(**x)
        check(out[:, :, keep], st[:, keep], full[:, :, keep], wst[:, keep])
    else:
        assert not torch.isfinite(out[0, t:]).any() and not torch.isfinite(st).any()


@pytest.mark.parametrize("L", [17, 130, 2500])
def test_a_query_that_is_not_finite_stays_at_its_token(L):
    t = 2 * L // 3
    x = inputs((1, L), 1, 2, 128, 64, seed=L)
    want, wst = rule(**x)
    x["q"][0, t, 0, 3] = float("nan")
    out, st = api.delta_prefill(**x)
    keep = [i for i in range(L) if i != t]
    check(out[:, keep], st, want[:, keep], wst)
    assert out[0, t].isnan().all()


@pytest.mark.parametrize("L", [17, 200, 2500])
def test_a_state_that_is_not_finite_stays_in_its_row(L):
    x = inputs((1, L), 1, 2, 64, 64, seed=L)
    s0 = state0(1, 2, 64, 64, L)
    s0[0, 1, 9, 3] = float("nan")
    out, st = api.delta_prefill(**x, state_in=s0)
    s0[0, 1, 9, 3] = 0
    want, wst = rule(**x, state=s0)
    keep = torch.ones(2, 64, dtype=torch.bool)
    keep[1, 9] = False
    check(out[:, :, keep], st[:, keep], want[:, :, keep], wst[:, keep])
    assert not torch.isfinite(out[0, :, 1, 9]).any() and not torch.isfinite(st[0, 1, 9]).any()


def test_many_units():
    """More (sequence, head) units than SMs, two slices of d_value."""
    x = inputs((5, 140), 8, 32, 64, 256, seed=43)
    check(*api.delta_prefill(**x), *rule(**x))


def test_calls_are_deterministic():
    x = inputs((2, 500), 2, 8, 128, 128, seed=47)
    a = api.delta_prefill(**x)
    for _ in range(3):
        b = api.delta_prefill(**x)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_graphs():
    """A call on another stream, two calls at once, and captured calls replayed on new inputs."""
    xs = [inputs((1, 333), 2, 4, 128, 128, seed=50 + i) for i in range(2)]
    want = [rule(**x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    torch.cuda.synchronize()
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append(api.delta_prefill(**x))
    for (o, st), w in zip(got, want):
        check(o, st, *w)
    o, st = api.delta_prefill(**xs[0], stream=streams[1])
    check(o, st, *want[0])

    buf = {n: t.clone() for n, t in xs[0].items()}
    dec = {n: t[:, 0].clone() for n, t in xs[0].items()}
    pool = state0(1, 4, 128, 128, 60)
    out = torch.zeros(1, 333, 4, 128, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(1, 4, 128, 128, device="cuda")
    api.delta_prefill(**buf, out=out, state_out=state)  # loads the kernels before the capture
    api.delta_decode_step(**dec, state=pool.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.delta_prefill(**buf, out=out, state_out=state)
        dec_out = api.delta_decode_step(**dec, state=state)
    for x, w in zip(xs, want):
        for n, t in x.items():
            buf[n].copy_(t)
            dec[n].copy_(t[:, 0])
        graph.replay()
        both = rule(**{n: torch.cat([t, t[:, :1]], 1) for n, t in x.items()})
        check(torch.cat([out, dec_out[:, None]], 1), state, *both)


# ------------------------------------------------------------------- decode ---
@pytest.mark.parametrize("b", [1, 3, 70])
@pytest.mark.parametrize("G,H,dk,dv", [(1, 1, 8, 8), (2, 4, 64, 128), (2, 6, 128, 128), (1, 4, 96, 40), (4, 4, 128, 264)])
def test_decode_shapes(b, G, H, dk, dv):
    x = inputs((b, 1), G, H, dk, dv, seed=b + dv, l2norm=True)
    s0 = state0(b, H, dv, dk, b)
    st = s0.clone()
    out = api.delta_decode_step(**{n: t[:, 0] for n, t in x.items()}, state=st, qk_l2norm=True)
    check(out[:, None], st, *rule(**x, state=s0, l2norm=True))


def test_decode_state_index_and_padding():
    """Rows name states of a pool; padded rows (negative or past the pool) leave their output and every state alone;
    with another state_out, states that no row names stay as they were there."""
    b, G, H, dk, dv, slots = 6, 2, 4, 128, 64, 9
    x = inputs((b, 1), G, H, dk, dv, seed=61)
    one = {n: t[:, 0] for n, t in x.items()}
    pool = state0(slots, H, dv, dk, 62)
    index = torch.tensor([7, -1, 0, 3, 9, -2147483648], dtype=torch.int32, device="cuda")
    live = [0, 2, 3]
    want_out, want_state = rule(**{n: t[live] for n, t in x.items()}, state=pool[[7, 0, 3]])
    for other in (False, True):
        st = pool.clone()
        dst = torch.full_like(st, 3.0) if other else None
        out = torch.full((b, H, dv), 5.0, dtype=torch.bfloat16, device="cuda")
        api.delta_decode_step(**one, state=st, state_index=index, out=out, state_out=dst)
        got = dst if other else st
        check(out[live][:, None], got[[7, 0, 3]], want_out, want_state)
        assert (out[[1, 4, 5]] == 5).all()
        rest = [i for i in range(slots) if i not in (7, 0, 3)]
        assert (got[rest] == 3).all() if other else torch.equal(got[rest], pool[rest])
        if other:
            assert torch.equal(st, pool)


def test_decode_offsets_past_32_bits():
    """The last state of a pool of more than 2^31 elements and 2^32 bytes."""
    H, dv, dk = 32, 128, 128
    slots = (1 << 31) // (H * dv * dk) + 2
    pool = torch.empty(slots, H, dv, dk, device="cuda")
    x = inputs((1, 1), 1, H, dk, dv, seed=67)
    s0 = state0(1, H, dv, dk, 68)
    pool[-1:] = s0
    index = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    out = api.delta_decode_step(**{n: t[:, 0] for n, t in x.items()}, state=pool, state_index=index)
    check(out[:, None], pool[-1:], *rule(**x, state=s0))


def test_offsets_that_do_not_ascend_stay_inside_their_buffers():
    """Offsets that name the whole buffer again and again are no valid packing, and their rows' results are not
    specified; the call still ends, writes nothing behind its workspace, outputs and states, and leaves the next call
    its results."""
    T, n, G, H, dk, dv = 2100, 41, 1, 2, 128, 64
    x = {m: t[0] for m, t in inputs((1, T), G, H, dk, dv, seed=77).items()}
    cu = torch.tensor([T * (i % 2) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    need = api.delta_prefill_workspace_bytes(n, T, H, G, dk, dv, packed=True)
    room = 1 << 20
    ws = torch.full((need + room,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 64, H, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((n + 8, H, dv, dk), 5.0, device="cuda")
    api.delta_prefill(**x, cu_seqlens=cu, workspace=ws[:need], out=out[:T], state_out=st[:n])
    api.check_device_error()
    assert (ws[need:] == 0x5A).all() and (out[T:] == 5).all() and (st[n:] == 5).all()
    assert (st[1:n:2] == 0).all()  # the empty ones
    lens = [T - 100, 100]
    cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
    got, st = api.delta_prefill(**x, cu_seqlens=cu, workspace=ws[:need])
    at = 0
    for i, m in enumerate(lens):
        check(got[None, at:at + m], st[i:i + 1], *rule(**{k: t[None, at:at + m] for k, t in x.items()}))
        at += m


@pytest.mark.parametrize("L", [300, 2500])
def test_buffers_belong_to_the_calls_stream(L):
    """With stream=, workspace and results are that stream's memory: what the current stream allocates right after the
    call, while it still waits on its stream, is none of it."""
    x = inputs((1, L), 1, 2, 128, 128, seed=L)
    want = rule(**x)
    api.delta_prefill(**x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = api.delta_prefill_workspace_bytes(1, L, 2, 1, 128, 128)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    out, st = api.delta_prefill(**x, stream=s)
    for n in (ws, out.numel() * 2, st.numel() * 4):
        for _ in range(4):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # the current stream writes over what it is given
    torch.cuda.synchronize()
    check(out, st, *want)


@pytest.mark.parametrize("b,L,G,H,dk,dv", [
    (3, 1100, 8, 64, 64, 128), (2, 1500, 1, 160, 128, 64), (11, 1024, 5, 15, 64, 72), (1, 1027, 3, 150, 32, 8),
    (3, 2000, 2, 50, 128, 136), (1, 12000, 8, 32, 128, 128), (1, 12000, 2, 40, 64, 64),
])
def test_more_walks_than_sms(b, L, G, H, dk, dv):
    """Walks that the blocks share: those cut between two of them continue from the state that the first leaves, with
    a state given and updated in place, and call after call alike."""
    x = inputs((b, L), G, H, dk, dv, seed=L + H, decay=0.05)
    s0 = state0(b, H, dv, dk, L)
    want = rule(**x, state=s0)
    st = s0.clone()
    out, _ = api.delta_prefill(**x, state_in=st, state_out=st)
    api.check_device_error()
    check(out, st, *want)
    for _ in range(3):
        again, st2 = api.delta_prefill(**x, state_in=s0)
        assert torch.equal(again, out) and torch.equal(st2, st)


def test_shared_walks_at_once_and_replayed():
    """Three calls with more walks than SMs at once, each on its own stream, and one captured and replayed while
    another runs: blocks of one call wait for each other's states, never for another call."""
    xs = [inputs((3, 1100), 8, 64, 64, 128, seed=90 + i, decay=0.05) for i in range(3)]
    want = [api.delta_prefill(**x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(4):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(api.delta_prefill(**x))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for o, st in g:
            assert torch.equal(o, w[0]) and torch.equal(st, w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, st = api.delta_prefill(**xs[0])
    for _ in range(3):
        o.zero_(), st.zero_()
        with torch.cuda.stream(streams[1]):
            streams[1].wait_stream(torch.cuda.current_stream())
            o1, st1 = api.delta_prefill(**xs[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0][0]) and torch.equal(st, want[0][1])
        assert torch.equal(o1, want[1][0]) and torch.equal(st1, want[1][1])
    api.check_device_error()


def test_packed_on_the_edges_of_a_cut():
    """Packed buffers where the first length to be cut, and 256 and 257 sequences, are just met."""
    for lens in ([64 * 32 - 1], [64 * 31], [64 * 32, 64 * 8 + 1], [8] * 255 + [2100], [8] * 256 + [2100]):
        T, H, dk, dv = sum(lens), 2, 64, 128
        x = inputs((1, T), 1, H, dk, dv, seed=T, decay=0.05)
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        out, st = api.delta_prefill(**{m: t[0] for m, t in x.items()},
                                    cu_seqlens=torch.tensor(at, dtype=torch.int32, device="cuda"))
        for i in (0, len(lens) - 1):
            want = rule(**{m: t[:, at[i]:at[i + 1]] for m, t in x.items()})
            check(out[None, at[i]:at[i + 1]], st[i:i + 1], *want, f"sequence {i} of {len(lens)}")
