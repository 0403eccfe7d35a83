"""Cases for the operators of a gated-delta layer around the block core: the
gated delta rule over whole sequences (dense or packed) and over one token, the
gated group norm behind a scan, and the residual norm between two blocks.

`run` computes a case in its plain form (elementary torch operations in fp32)
or, with `own` set, through the framework's entry points; `exact` computes the
same outputs in float64 from the definitions.

Gated delta rule, per sequence and head, S in R^{dv x dk}, a_t = exp(g_t):
    S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   o_t = scale S_t q_t.
Gated norm, per group of channels:
    y = x / rms(x) w SiLU(z),   or with the gate first   t = x SiLU(z), y = t / rms(t) w.
Residual norm, per row:
    t = x (or x / rms(x) w_post),   r' = r + alpha t,   y = r' / rms(r') w,
with rms(x) = sqrt(mean(x^2) + eps).
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CHUNK = 64  # tokens per step of the plain form's recurrence


# ------------------------------------------------------------------- cases ---
def _prefill(name, batch, seqlen, groups, heads, dk, dv, state=False, l2norm=False, packed=False):
    c = dict(op="delta_prefill", batch=batch, seqlen=seqlen, groups=groups, heads=heads, dk=dk, dv=dv, state=state,
             l2norm=l2norm, packed=packed)
    return dict(c, name=name) if name else c


def _decode(name, batch, groups, heads, dk, dv, slots=0, padded=0, l2norm=False):
    c = dict(op="delta_decode", batch=batch, groups=groups, heads=heads, dk=dk, dv=dv, slots=slots, padded=padded,
             l2norm=l2norm)
    return dict(c, name=name) if name else c


def _gated(name, rows, dim, group, io, gate_first=False, shared_weight=False, fused=False):
    c = dict(op="gated_norm", rows=rows, dim=dim, group=group, io=io, gate_first=gate_first,
             shared_weight=shared_weight, fused=fused)
    return dict(c, name=name) if name else c


def _residual(name, rows, dim, io, res, alpha=1.0, post=False):
    c = dict(op="residual_norm", rows=rows, dim=dim, io=io, res=res, alpha=alpha, post=post)
    return dict(c, name=name) if name else c


def listed():
    return [
        # A short odd prompt that meets an empty state: latency of one call.
        _prefill("prefill prompt 33", 1, 33, 16, 32, 128, 128, l2norm=True),
        # The layer shape of the block core (E = 7680 as 60 heads of 128) at its prompt length.
        _prefill("prefill layer 2048", 1, 2048, 60, 60, 128, 128),
        # The batched chunk-scan shape: 8 sequences, 80 heads of 64 sharing one group.
        _prefill("prefill batch 8x4096", 8, 4096, 1, 80, 128, 64),
        # Prompts of a serving queue in one packed buffer, lengths from one token to thousands, continuing states.
        _prefill("prefill packed ragged", 13, 16001, 8, 32, 128, 128, state=True, l2norm=True, packed=True),
        # One long context in a continued state, 16 key heads for 32 value heads.
        _prefill("prefill long 32768", 1, 32768, 16, 32, 128, 128, state=True, l2norm=True),
        # A single user's next token.
        _decode("decode one token", 1, 16, 32, 128, 128, l2norm=True),
        # The full decode batch of the block core.
        _decode("decode batch 256", 256, 60, 60, 128, 128),
        # A padded batch over a pool of state slots, narrower keys.
        _decode("decode slots", 45, 8, 24, 64, 128, slots=96, padded=4, l2norm=True),
        # Per-head norm behind the scan, z inside the fused projection buffer.
        _gated("gated heads 16384", 16384, 7680, 128, "bf16", shared_weight=True, fused=True),
        # Whole-row norm with the gate first, one decode batch.
        _gated("gated row 256", 256, 5120, 5120, "bf16", gate_first=True),
        # The residual stream in fp32 between the blocks of a long prompt.
        _residual("residual 65536", 65536, 2560, "bf16", "f32"),
        # One token between two blocks, with the norm behind the block and a residual scale.
        _residual("residual one token", 1, 2560, "bf16", "bf16", alpha=0.22, post=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("delta_prefill", "delta_prefill", "delta_decode", "gated_norm", "residual_norm"))
    if op == "delta_prefill":
        groups = rng.choice((1, 2, 3, 4, 8, 16))
        heads = groups * rng.choice((1, 2, 3, 4))
        dk, dv = rng.choice((32, 64, 96, 128, 128)), rng.choice((40, 64, 128, 128, 192, 256))
        packed = rng.random() < 0.4
        batch = rng.randint(1, 12) if packed else rng.choice((1, 1, 2, 3, 4, 8))
        most = min(32768, 32768 * 32 * 128 * 128 // (heads * dk * dv))
        if packed:
            seqlen = _log_int(rng, max(16, 4 * batch), most)
        else:
            seqlen = _log_int(rng, 1, max(2, most // batch))
        return _prefill(None, batch, seqlen, groups, heads, dk, dv, rng.random() < 0.5, rng.random() < 0.5, packed)
    if op == "delta_decode":
        groups = rng.choice((1, 2, 4, 8, 15, 16))
        heads = groups * rng.choice((1, 2, 4))
        dk, dv = rng.choice((32, 64, 96, 128)), rng.choice((40, 64, 128, 256))
        batch = _log_int(rng, 1, min(256, 256 * 60 * 128 * 128 // (heads * dk * dv)))
        slots = batch + rng.randint(1, 40) if rng.random() < 0.5 else 0
        padded = rng.randint(0, batch // 3) if slots else 0
        return _decode(None, batch, groups, heads, dk, dv, slots, padded, rng.random() < 0.5)
    io = rng.choice(("bf16", "bf16", "f32"))
    if op == "gated_norm":
        group = rng.choice((64, 80, 128, 256, 1000, 2560, 5120))
        dim = group * rng.randint(1, max(1, 8192 // group))
        rows = _log_int(rng, 1, min(65536, 120_000_000 // dim))
        return _gated(None, rows, dim, group, io, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    dim = rng.choice((64, 200, 771, 1024, 2560, 4097, 5120, 7680, 8192))
    rows = _log_int(rng, 1, min(65536, 120_000_000 // dim))
    res = "f32" if io == "f32" else rng.choice(("f32", "bf16"))
    return _residual(None, rows, dim, io, res, rng.choice((1.0, 0.22, 0.5)), rng.random() < 0.5)


# ------------------------------------------------------------------ inputs ---
def _lengths(case, seed):
    """Lengths of a packed batch, their sum the case's seqlen: each at least one token, spread over the logarithm."""
    rng = random.Random(seed * 7919 + case["batch"])
    n, total = case["batch"], case["seqlen"]
    weight = [math.exp(rng.uniform(0.0, math.log(max(2.0, total / 4)))) for _ in range(n)]
    lens = [max(1, int(total * w / sum(weight))) for w in weight]
    if n > 2:
        lens[rng.randrange(n)] = 1
    at = max(range(n), key=lambda i: lens[i])
    lens[at] += total - sum(lens)
    return lens


def _io(case):
    return BF16 if case["io"] == "bf16" else F32


def _delta_inputs(case, lead, gen):
    """q, k, v, g, beta with leading sizes `lead`: q and k after SiLU (normalised here unless the operator does it),
    g = -softplus step times a rate in [1, 16] as a layer's decay, beta = sigmoid."""
    G, H, dk, dv = case["groups"], case["heads"], case["dk"], case["dv"]
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    u = lambda *s: torch.rand(s, device="cuda", generator=gen)  # noqa: E731
    silu = lambda t: t / (1 + torch.exp(-t))  # noqa: E731
    q, k = silu(r(*lead, G, dk)), silu(r(*lead, G, dk))
    if not case["l2norm"]:
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    v = r(*lead, H, dv)
    dt = torch.exp(u(H) * math.log(100.0) + math.log(1e-3))  # [1e-3, 1e-1], as the block core's steps
    g = -(dt * torch.exp(0.5 * r(*lead, H))) * (1 + 15 * u(H))
    beta = torch.sigmoid(r(*lead, H))
    return dict(q=q.to(BF16), k=k.to(BF16), v=v.to(BF16), g=g, beta=beta)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    r = lambda *n: torch.randn(n, device="cuda", generator=gen)  # noqa: E731
    if case["op"] == "delta_prefill":
        b, H, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
        if case["packed"]:
            s["lens"] = _lengths(case, seed)
            lead = (case["seqlen"],)
            at = [0]
            for n in s["lens"]:
                at.append(at[-1] + n)
            s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        else:
            lead = (b, case["seqlen"])
            s["cu"] = None
        s.update(_delta_inputs(case, lead, gen))
        s["state_in"] = 0.3 * r(b, H, dv, dk) if case["state"] else None
        s["out"] = torch.zeros(*lead, H, dv, dtype=BF16, device="cuda")
        s["state_out"] = torch.zeros(b, H, dv, dk, device="cuda")
    elif case["op"] == "delta_decode":
        b, H, dk, dv = case["batch"], case["heads"], case["dk"], case["dv"]
        s.update(_delta_inputs(case, (b,), gen))
        slots = case["slots"] or b
        s["state"] = 0.3 * r(slots, H, dv, dk)
        s["state_out"] = torch.zeros_like(s["state"])
        s["out"] = torch.zeros(b, H, dv, dtype=BF16, device="cuda")
        s["index"] = None
        if case["slots"]:
            index = torch.argsort(torch.rand(slots, device="cuda", generator=gen))[:b].to(torch.int32)
            if case["padded"]:
                index[b - case["padded"]:] = -1
            s["index"] = index
    elif case["op"] == "gated_norm":
        n, d, io = case["rows"], case["dim"], _io(case)
        if case["fused"]:  # x and z as a fused projection leaves them
            xz = r(n, 2 * d).to(io)
            s["x"], s["z"] = xz[:, :d], xz[:, d:]
        else:
            s["x"], s["z"] = r(n, d).to(io), r(n, d).to(io)
        s["w"] = 1 + 0.1 * r(case["group"] if case["shared_weight"] else d)
        s["out"] = torch.zeros(n, d, dtype=io, device="cuda")
    else:
        n, d, io = case["rows"], case["dim"], _io(case)
        res = BF16 if case["res"] == "bf16" else F32
        s["x"], s["r"] = r(n, d).to(io), (3 * r(n, d)).to(res)
        s["w"] = 1 + 0.1 * r(d)
        s["post"] = 1 + 0.1 * r(d) if case["post"] else None
        s["out"], s["r_out"] = torch.zeros(n, d, dtype=io, device="cuda"), torch.zeros(n, d, dtype=res, device="cuda")
    return s


# -------------------------------------------------------------- plain form ---
def _padded_index(s, length):
    """[n, length] rows of the packed buffer, and which of them are tokens of the sequence."""
    cu = s["cu"].long()
    pos = torch.arange(length, device="cuda")
    real = pos < (cu[1:] - cu[:-1])[:, None]
    return torch.where(real, cu[:-1, None] + pos, 0), real


def _l2(t):
    return t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6)


def _plain_prefill(s):
    """The rule in chunks: within a chunk (I + A) U = beta (V - e^G K S), A_ij = beta_i e^{G_i - G_j} k_i.k_j below
    the diagonal, G the running sum of g; then O = e^G Q S + (Q K^T e^{G_i - G_j}) U and S = e^G_C S + K^T e^{G_C - G} U."""
    case = s["case"]
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    q, k, v, g, beta = s["q"], s["k"], s["v"], s["g"], s["beta"]
    if case["packed"]:
        index, real = _padded_index(s, max(s["lens"]))
        q, k, v, g, beta = (t[index] for t in (q, k, v, g, beta))
    else:
        real = None
    b, L = g.shape[:2]
    nc = -(-L // CHUNK)
    rep = H // case["groups"]

    def chunks(t):  # [b, L, h, ...] -> fp32 [b, h, nc, CHUNK, ...], zeros behind the last token
        t = t.to(F32)
        if real is not None:
            t = torch.where(real.reshape(real.shape + (1,) * (t.dim() - 2)), t, torch.zeros((), device="cuda"))
        t = torch.cat([t, t.new_zeros((b, nc * CHUNK - L) + t.shape[2:])], 1)
        return t.reshape((b, nc, CHUNK) + t.shape[2:]).transpose(2, 3).transpose(1, 2)

    q, k = (_l2(t.to(F32)) if case["l2norm"] else t for t in (q, k))
    q, k, v, g, beta = (chunks(t) for t in (q, k, v, g, beta))
    q, k = (t.repeat_interleave(rep, 1) for t in (q, k))
    q = q * dk ** -0.5
    G = torch.cumsum(g.double(), -1)
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda"))
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).to(F32)
    eG, eC = torch.exp(G).to(F32)[..., None], torch.exp(G[..., -1:] - G).to(F32)[..., None]
    A = torch.tril(beta[..., None] * D * (k @ k.transpose(-1, -2)), -1)
    T = torch.eye(CHUNK, device="cuda").expand_as(A).contiguous()
    for i in range(1, CHUNK):  # (I + A)^-1 row by row
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    del A
    U0, W = T @ (beta[..., None] * v), T @ (beta[..., None] * eG * k)
    del T
    P, q, k = (q @ k.transpose(-1, -2)) * D, q * eG, (k * eC).transpose(-1, -2)
    S = s["state_in"].transpose(-1, -2) if s["state_in"] is not None else torch.zeros(b, H, dk, dv, device="cuda")
    O = torch.empty_like(v)
    for c in range(nc):
        U = U0[:, :, c] - W[:, :, c] @ S
        O[:, :, c] = q[:, :, c] @ S + P[:, :, c] @ U
        S = eG[:, :, c, -1:] * S + k[:, :, c] @ U
    O = O.transpose(1, 2).transpose(2, 3).reshape(b, nc * CHUNK, H, dv)[:, :L].to(BF16)
    if case["packed"]:
        s["out"][index[real]] = O[real]
        O = s["out"]
    return {"out": O, "state": S.transpose(-1, -2).contiguous()}


def _plain_decode(s):
    case = s["case"]
    rep = case["heads"] // case["groups"]
    rows = slice(None) if s["index"] is None else torch.nonzero(s["index"] >= 0)[:, 0]
    at = rows if s["index"] is None else s["index"][rows].long()
    q, k, v, g, beta = (s[n][rows].to(F32) for n in ("q", "k", "v", "g", "beta"))
    if case["l2norm"]:
        q, k = _l2(q), _l2(k)
    q, k = q.repeat_interleave(rep, 1) * case["dk"] ** -0.5, k.repeat_interleave(rep, 1)
    S = s["state"][at] * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (S * k[:, :, None]).sum(-1))
    S = S + u[..., None] * k[:, :, None]
    s["out"][rows] = (S * q[:, :, None]).sum(-1).to(BF16)
    s["state_out"][at] = S
    return {"out": s["out"], "state": s["state_out"]}


def _plain_gated(s):
    case = s["case"]
    x, z, w = s["x"].to(F32), s["z"].to(F32), s["w"]
    n, d, group = case["rows"], case["dim"], case["group"]
    gate = z / (1 + torch.exp(-z))
    if case["shared_weight"]:
        w = w.repeat(d // group)
    if case["gate_first"]:
        x = x * gate
    y = x.reshape(n, d // group, group)
    y = (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-5)).reshape(n, d) * w
    return {"out": (y if case["gate_first"] else y * gate).to(_io(case))}


def _plain_residual(s):
    case = s["case"]
    norm = lambda t, w: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-5) * w  # noqa: E731
    t = s["x"].to(F32)
    if s["post"] is not None:
        t = norm(t, s["post"])
    r = s["r"].to(F32) + case["alpha"] * t
    return {"out": norm(r, s["w"]).to(_io(case)), "residual": r.to(s["r"].dtype)}


# -------------------------------------------------------- the framework's ---
def _own(s):
    from selective_state_space_depthwise_b200 import api

    case = s["case"]
    if case["op"] == "delta_prefill":
        out, state = api.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], state_in=s["state_in"],
                                       qk_l2norm=case["l2norm"], cu_seqlens=s["cu"], out=s["out"],
                                       state_out=s["state_out"])
        return {"out": out, "state": state}
    if case["op"] == "delta_decode":
        out = api.delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], state_index=s["index"],
                                    qk_l2norm=case["l2norm"], out=s["out"], state_out=s["state_out"])
        return {"out": out, "state": s["state_out"]}
    if case["op"] == "gated_norm":
        return {"out": api.gated_norm(s["x"], s["z"], s["w"], group_size=case["group"], eps=1e-5,
                                      gate_first=case["gate_first"], out=s["out"])}
    out, r = api.residual_norm(s["x"], s["r"], s["w"], post_weight=s["post"], residual_scale=case["alpha"], eps=1e-5,
                               out=s["out"], residual_out=s["r_out"])
    return {"out": out, "residual": r}


def run(state):
    if own:
        return _own(state)
    return {"delta_prefill": _plain_prefill, "delta_decode": _plain_decode, "gated_norm": _plain_gated,
            "residual_norm": _plain_residual}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work ---
def work(case):
    if case["op"] in ("delta_prefill", "delta_decode"):
        G, H, dk, dv = case["groups"], case["heads"], case["dk"], case["dv"]
        if case["op"] == "delta_prefill":
            tokens = case["seqlen"] if case["packed"] else case["batch"] * case["seqlen"]
            states = case["batch"] * (2 if case["state"] else 1)
        else:
            tokens = case["batch"] - case["padded"]
            states = 2 * tokens
        per_token = 2 * (2 * G * dk + 2 * H * dv) + 8 * H
        return {"bytes": tokens * per_token + states * 4 * H * dv * dk, "flops": 6 * tokens * H * dk * dv}
    n = case["rows"] * case["dim"]
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "gated_norm":
        return {"bytes": 3 * n * e + 4 * (case["group"] if case["shared_weight"] else case["dim"]), "flops": 8 * n}
    return {"bytes": n * (2 * e + 2 * (2 if case["res"] == "bf16" else 4)) + 4 * case["dim"] * (1 + case["post"]),
            "flops": (10 if case["post"] else 6) * n}


# ------------------------------------------------------------------- exact ---
def _exact_rule(q, k, v, g, beta, S, scale):
    """Token by token in float64: q, k [n, L, H, dk], v [n, L, H, dv], g, beta [n, L, H], S [n, H, dv, dk]."""
    out = []
    decay = torch.exp(g)
    for t in range(g.shape[1]):
        S = S * decay[:, t, :, None, None]
        kt, qt = k[:, t, :, :, None], q[:, t, :, :, None]
        u = beta[:, t, :, None, None] * (v[:, t, :, :, None] - S @ kt)
        S = S + u * kt.transpose(-1, -2)
        out.append((S @ qt)[..., 0] * scale)
    return torch.stack(out, 1), S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("delta_prefill", "delta_decode"):
        H, dk, dv = case["heads"], case["dk"], case["dv"]
        q, k, v, g, beta = (s[n].to(F64) for n in ("q", "k", "v", "g", "beta"))
        if case["l2norm"]:
            q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
        head = torch.arange(H, device="cuda") // (H // case["groups"])
        q, k = q[..., head, :], k[..., head, :]
        if case["op"] == "delta_decode":
            one = [t[:, None] for t in (q, k, v, g, beta)]
            index = torch.arange(case["batch"], device="cuda") if s["index"] is None else s["index"].long()
            live = index >= 0
            o, S = _exact_rule(*(t[live] for t in one), s["state"][index[live]].to(F64), dk ** -0.5)
            out, state = s["out"].to(F64), s["state_out"].to(F64)
            out[live], state[index[live]] = o[:, 0], S
            return {"out": out, "state": state}
        S = s["state_in"].to(F64) if s["state_in"] is not None else torch.zeros(case["batch"], H, dv, dk, dtype=F64,
                                                                               device="cuda")
        if not case["packed"]:
            out, S = _exact_rule(q, k, v, g, beta, S, dk ** -0.5)
            return {"out": out, "state": S}
        start = [sum(s["lens"][:i]) for i in range(case["batch"])]
        # The sequences run together, padded to the longest with tokens that change nothing (g = 0, beta = 0).
        longest = max(s["lens"])
        pad = lambda t: torch.stack([torch.cat([t[a:a + n], t.new_zeros((longest - n,) + t.shape[1:])])  # noqa: E731
                                     for a, n in zip(start, s["lens"])])
        o, S = _exact_rule(*(pad(t) for t in (q, k, v, g, beta)), S, dk ** -0.5)
        return {"out": torch.cat([o[i, :n] for i, n in enumerate(s["lens"])]), "state": S}
    x, w = s["x"].to(F64), s["w"].to(F64)
    if case["op"] == "gated_norm":
        gate = s["z"].to(F64) * torch.sigmoid(s["z"].to(F64))
        x = (x * gate if case["gate_first"] else x).unflatten(-1, (-1, case["group"]))
        y = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        y = (y * w if case["shared_weight"] else y * w.unflatten(0, (-1, case["group"]))).flatten(-2)
        return {"out": y if case["gate_first"] else y * gate}
    if s["post"] is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * s["post"].to(F64)
    r = s["r"].to(F64) + case["alpha"] * x
    return {"out": r / (r.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w, "residual": r}
