"""CPU checks of the gated delta rule's and the norms' entry points: arguments
that are refused are refused on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from selective_state_space_depthwise_b200 import _lib, api, build

FAKE = 0x10000  # 16-byte-aligned, never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def delta_dims(**kw):
    d = _lib.SsmDeltaDims()
    d.batch, d.seqlen, d.nheads, d.ngroups, d.d_key, d.d_value = 2, 64, 4, 2, 64, 128
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def delta_call(lib, d, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, cu=None, sin=None, out=2 * FAKE, sout=FAKE, work=FAKE,
             nbytes=1 << 40)
    a.update(kw)
    return lib.ssm_delta_prefill(ctypes.byref(d) if d else None, a["q"], a["k"], a["v"], a["g"], a["beta"], a["cu"],
                                 a["sin"], a["out"], a["sout"], a["work"], a["nbytes"], None)


def decode_call(lib, d, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, index=None, n=2, sin=FAKE, out=2 * FAKE, sout=FAKE)
    a.update(kw)
    return lib.ssm_delta_decode_step(ctypes.byref(d) if d else None, a["q"], a["k"], a["v"], a["g"], a["beta"],
                                     a["index"], a["n"], a["sin"], a["out"], a["sout"], None)


BAD_DIMS = [
    ("batch", 0, _lib.SSM_ERR_INVALID_ARG), ("batch", 1 << 40, _lib.SSM_ERR_INVALID_ARG),
    ("nheads", 3, _lib.SSM_ERR_INVALID_ARG), ("nheads", 0, _lib.SSM_ERR_INVALID_ARG),
    ("ngroups", 0, _lib.SSM_ERR_INVALID_ARG), ("d_key", 60, _lib.SSM_ERR_UNSUPPORTED),
    ("d_key", 136, _lib.SSM_ERR_UNSUPPORTED), ("d_key", 0, _lib.SSM_ERR_UNSUPPORTED),
    ("d_value", 12, _lib.SSM_ERR_UNSUPPORTED), ("d_value", 4104, _lib.SSM_ERR_UNSUPPORTED),
    ("scale", -1.0, _lib.SSM_ERR_INVALID_ARG), ("scale", float("nan"), _lib.SSM_ERR_INVALID_ARG),
    ("qk_l2norm", 2, _lib.SSM_ERR_INVALID_ARG), ("q_tok_stride", 132, _lib.SSM_ERR_INVALID_ARG),
    ("k_tok_stride", 64, _lib.SSM_ERR_INVALID_ARG), ("v_tok_stride", 8, _lib.SSM_ERR_INVALID_ARG),
    ("out_tok_stride", -512, _lib.SSM_ERR_INVALID_ARG), ("v_seq_stride", -8, _lib.SSM_ERR_INVALID_ARG),
    ("out_seq_stride", 4, _lib.SSM_ERR_INVALID_ARG), ("gb_tok_stride", 3, _lib.SSM_ERR_INVALID_ARG),
    ("gb_seq_stride", -4, _lib.SSM_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("field,value,status", BAD_DIMS)
def test_delta_rejects_bad_dims(lib, field, value, status):
    d = delta_dims(**{field: value})
    assert delta_call(lib, d) == status
    assert decode_call(lib, d, n=1 << 50) == status
    assert lib.ssm_last_error()


def test_delta_rejects_bad_pointers(lib):
    d = delta_dims()
    assert delta_call(lib, None) == _lib.SSM_ERR_INVALID_ARG
    assert decode_call(lib, None) == _lib.SSM_ERR_INVALID_ARG
    for n in ("q", "k", "v", "g", "beta", "out", "sout"):
        assert delta_call(lib, d, **{n: None}) == _lib.SSM_ERR_INVALID_ARG, n
        assert decode_call(lib, d, **{n: None}) == _lib.SSM_ERR_INVALID_ARG, n
        assert delta_call(lib, d, **{n: FAKE + 2}) == _lib.SSM_ERR_INVALID_ARG, n
    assert delta_call(lib, d, out=FAKE) == _lib.SSM_ERR_INVALID_ARG  # over q
    assert delta_call(lib, d, sin=FAKE + 4) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, d, cu=FAKE + 2) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, delta_dims(seqlen=-1)) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, delta_dims(seqlen=1 << 31)) == _lib.SSM_ERR_INVALID_ARG
    need = lib.ssm_delta_prefill_workspace_bytes(ctypes.byref(d), 0)
    packed = lib.ssm_delta_prefill_workspace_bytes(ctypes.byref(d), 1)
    assert need == 2 * packed // 3 > 0  # two sequences of one chunk; 64 rows in two sequences: up to three chunks
    assert need == api.delta_prefill_workspace_bytes(2, 64, 4, 2, 64, 128)
    assert delta_call(lib, d, nbytes=need - 1) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, d, cu=FAKE, nbytes=packed - 1) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, d, work=None) == _lib.SSM_ERR_INVALID_ARG
    assert delta_call(lib, d, work=FAKE + 16) == _lib.SSM_ERR_INVALID_ARG
    assert lib.ssm_delta_prefill_workspace_bytes(ctypes.byref(delta_dims(seqlen=1)), 0) == 0
    assert lib.ssm_delta_prefill_workspace_bytes(ctypes.byref(delta_dims(seqlen=0)), 1) == 0
    assert lib.ssm_delta_prefill_workspace_bytes(ctypes.byref(delta_dims(d_key=12)), 0) == 0
    assert lib.ssm_delta_prefill_workspace_bytes(None, 0) == 0
    assert decode_call(lib, d, sin=None) == _lib.SSM_ERR_INVALID_ARG
    assert decode_call(lib, d, n=0) == _lib.SSM_ERR_INVALID_ARG
    assert decode_call(lib, d, n=1) == _lib.SSM_ERR_INVALID_ARG  # fewer states than rows, no index
    assert decode_call(lib, d, index=FAKE + 1) == _lib.SSM_ERR_INVALID_ARG


def test_delta_binding_refuses_what_it_cannot_express(lib):
    bf = dict(dtype=torch.bfloat16)
    q, v, g = torch.zeros(1, 8, 2, 64, **bf), torch.zeros(1, 8, 4, 64, **bf), torch.zeros(1, 8, 4)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        api.delta_prefill(q, q, v, g, g)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        api.delta_decode_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(1, 4, 64, 64))
    with pytest.raises(ValueError, match="with cu_seqlens"):
        api.delta_prefill(q[0], q[0], v[0], g[0], g[0])
    with pytest.raises(ValueError, match="expanded"):
        api._stride("q", q[:, :1].expand(1, 8, 2, 64), 1)
    assert api._stride("q", q, 0) == 0 and api._stride("q", q, 1) == 128
    with pytest.raises(ValueError, match="contiguous"):
        api._dense_heads("q", q.transpose(2, 3))


def gated_dims(**kw):
    d = _lib.SsmGatedNormDims()
    d.batch, d.seqlen, d.dim, d.group, d.eps, d.io_dtype = 2, 3, 128, 64, 1e-5, _lib.SSM_BF16
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_gated_norm_rejects_bad_arguments(lib):
    def call(d, x=FAKE, z=FAKE, w=FAKE, y=FAKE):
        return lib.ssm_gated_norm(ctypes.byref(d) if d else None, x, z, w, y, None)

    assert call(None) == _lib.SSM_ERR_INVALID_ARG
    for kw in (dict(batch=-1), dict(seqlen=-1), dict(dim=0), dict(group=0), dict(group=48), dict(io_dtype=7),
               dict(eps=-1.0), dict(eps=float("nan")), dict(gate_first=2), dict(shared_weight=-1),
               dict(x_tok_stride=64), dict(z_seq_stride=-1), dict(batch=1 << 40, seqlen=1 << 20)):
        assert call(gated_dims(**kw)) == _lib.SSM_ERR_INVALID_ARG, kw
    assert call(gated_dims(dim=65536, group=65536)) == _lib.SSM_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 1), dict(z=FAKE + 1), dict(w=FAKE + 2)):
        assert call(gated_dims(), **kw) == _lib.SSM_ERR_INVALID_ARG, kw
    assert call(gated_dims(batch=0), x=None) == _lib.SSM_OK  # no rows


def test_residual_norm_rejects_bad_arguments(lib):
    def call(x=FAKE, r=FAKE, w=FAKE, p=None, y=FAKE, ro=FAKE, none=False, **kw):
        d = _lib.SsmResidualNormDims()
        d.rows, d.dim, d.eps, d.residual_scale, d.io_dtype, d.residual_dtype = 4, 128, 1e-5, 1.0, 1, 0
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.ssm_residual_norm(None if none else ctypes.byref(d), x, r, w, p, y, ro, None)

    assert call(none=True) == _lib.SSM_ERR_INVALID_ARG
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(eps=-1.0), dict(io_dtype=3),
               dict(residual_dtype=-1), dict(x_stride=64), dict(y_stride=-128), dict(residual_in_stride=1),
               dict(residual_out_stride=1), dict(x=None), dict(w=None), dict(y=None), dict(r=FAKE + 2),
               dict(p=FAKE + 1)):
        assert call(**kw) == _lib.SSM_ERR_INVALID_ARG, kw
    assert call(dim=32769) == _lib.SSM_ERR_UNSUPPORTED
    assert call(rows=0, x=None) == _lib.SSM_OK


def test_residual_norm_refuses_one_buffer_for_both_results(lib):
    """Both are bf16 here: the norm would be written over the sum."""
    d = _lib.SsmResidualNormDims()
    d.rows, d.dim, d.eps, d.residual_scale, d.io_dtype, d.residual_dtype = 4, 128, 1e-5, 1.0, 1, 1
    st = lib.ssm_residual_norm(ctypes.byref(d), FAKE, FAKE, FAKE, None, 2 * FAKE, 2 * FAKE, None)
    assert st == _lib.SSM_ERR_INVALID_ARG


def test_packed_workspace_holds_32_segments_a_sequence_at_most(lib):
    """The workspace of few long packed sequences grows with their chunks' tiles, not with their possible cuts."""
    H, dk, dv = 4, 128, 128
    chunk = 26496 * H  # tiles of 64 tokens
    sizes = [api.delta_prefill_workspace_bytes(2, 64 * n, H, H, dk, dv, packed=True) for n in (4096, 8192)]
    assert sizes[1] - sizes[0] == 4096 * chunk


def test_norm_bindings_refuse_host_tensors_and_odd_rows(lib):
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        api.gated_norm(x, x, w)
    with pytest.raises(RuntimeError, match="CUDA tensor"):
        api.residual_norm(x, x, w)
    t = torch.zeros(2, 8, 64)[:, :4]
    with pytest.raises(ValueError, match="one stride"):
        api._row_stride("x", t)
    assert api._row_stride("x", torch.zeros(3, 1, 64)) == 64
    assert api._row_stride("x", torch.zeros(1, 5, 80)[..., :64]) == 80
    with pytest.raises(ValueError, match="expanded"):
        api._row_stride("x", torch.zeros(1, 64).expand(4, 64))


def test_residual_block_rejects_bad_arguments(lib):
    w = _lib.SsmWeights(*([FAKE] * 6))
    pw = _lib.SsmBlockWeights(FAKE, FAKE, FAKE)
    d = api.make_block_dims(2, 64, 32, 64)
    need = lib.ssm_residual_block_workspace_bytes(ctypes.byref(d))
    assert need == lib.ssm_block_workspace_bytes(ctypes.byref(d)) + 2 * 64 * 32 * 2

    def call(dims=d, proj=pw, norm=None, x=FAKE, r=FAKE, ro=2 * FAKE, out=3 * FAKE, ws=FAKE, nbytes=need,
             norm_w=FAKE, res=0, drop_norm=False):
        n = _lib.SsmBlockNorm(norm_w, None, 1e-5, 1.0, res)
        return lib.ssm_residual_block_forward(ctypes.byref(dims) if dims else None, ctypes.byref(w),
                                              ctypes.byref(proj) if proj else None,
                                              None if drop_norm else ctypes.byref(n), x, r, None, None, ro, out, FAKE,
                                              FAKE, ws, nbytes, None)

    for kw in (dict(dims=None), dict(drop_norm=True), dict(proj=None), dict(x=None), dict(norm_w=None), dict(res=9),
               dict(ro=None), dict(out=None), dict(out=FAKE), dict(out=2 * FAKE), dict(ws=None), dict(ws=FAKE + 16),
               dict(nbytes=need - 1), dict(proj=_lib.SsmBlockWeights(FAKE, None, FAKE))):
        assert call(**kw) == _lib.SSM_ERR_INVALID_ARG, kw


def test_a_workspace_must_be_contiguous():
    """An expanded workspace has fewer bytes than elements."""
    with pytest.raises(ValueError, match="contiguous"):
        api._workspace(torch.empty(1, dtype=torch.uint8).expand(1024), 1024, torch.device("cpu"), None)
    w = torch.empty(64, dtype=torch.uint8)
    assert api._workspace(w, 64, w.device, None) is w and api._workspace(w, 65, w.device, None).numel() == 65


def test_packed_workspace_holds_states_of_cut_sequences_only(lib):
    """256 sequences of 128 tokens: at most 63 of more than 512 tokens lie in so many rows, with one segment each and
    one more for 512 tokens; none of the others has a segment's state and matrix."""
    b, H, dk, dv = 256, 32, 128, 128
    L = b * 128
    tiles = 26496 * H * (L // 64 + b)
    cut = min(b, L // 513)
    states = (cut + (L // 64 + cut) // 8) * H * (dv * dk + dk * dk) * 4
    got = api.delta_prefill_workspace_bytes(b, L, H, H, dk, dv, packed=True)
    assert tiles + states <= got <= tiles + states + (1 << 14)


def test_norms_refuse_a_result_over_an_input_at_another_stride_or_type(lib):
    """Rows of a result written over rows of an input that other blocks still read."""
    def residual(x=FAKE, r=2 * FAKE, y=3 * FAKE, ro=4 * FAKE, **kw):
        d = _lib.SsmResidualNormDims()
        d.rows, d.dim, d.eps, d.residual_scale, d.io_dtype, d.residual_dtype = 4, 128, 1e-5, 1.0, 1, 1
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.ssm_residual_norm(ctypes.byref(d), x, r, FAKE, None, y, ro, None)

    for kw in (dict(y=FAKE, y_stride=136), dict(y=FAKE, x_stride=136), dict(y=2 * FAKE, residual_dtype=0),
               dict(y=2 * FAKE, residual_in_stride=256), dict(ro=FAKE, residual_dtype=0),
               dict(ro=FAKE, residual_out_stride=144), dict(ro=2 * FAKE, residual_in_stride=256),
               dict(y=2 * FAKE, residual_dtype=0, rows=1)):
        assert residual(**kw) == _lib.SSM_ERR_INVALID_ARG, kw

    def gated(x=FAKE, z=2 * FAKE, y=3 * FAKE, **kw):
        return lib.ssm_gated_norm(ctypes.byref(gated_dims(**kw)), x, z, FAKE, y, None)

    for kw in (dict(y=FAKE, y_tok_stride=136), dict(y=FAKE, x_seq_stride=512), dict(y=2 * FAKE, z_tok_stride=256),
               dict(y=2 * FAKE, y_seq_stride=1024)):
        assert gated(**kw) == _lib.SSM_ERR_INVALID_ARG, kw
