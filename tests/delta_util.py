"""Float64 definition of the gated delta rule and its inputs, for the tests."""
from __future__ import annotations

import math

import torch


def inputs(lead, G, H, dk, dv, *, seed, l2norm=False, device="cuda", decay=1.0):
    """Token tensors with leading sizes `lead`: q, k after SiLU (normalised here
    unless the operator does it), v normal, g = -(steps of a few thousandths to
    tenths) * decay, beta in (0, 1)."""
    gen = torch.Generator(device="cpu").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = torch.nn.functional.silu(r(*lead, G, dk)), torch.nn.functional.silu(r(*lead, G, dk))
    if not l2norm:
        q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    g = -torch.exp(math.log(3e-2) + 1.2 * r(*lead, H)) * decay
    t = dict(q=q.bfloat16(), k=k.bfloat16(), v=r(*lead, H, dv).bfloat16(), g=g, beta=torch.sigmoid(r(*lead, H)))
    return {n: x.to(device) for n, x in t.items()}


def rule(q, k, v, g, beta, state=None, scale=None, l2norm=False):
    """Token by token in float64: q, k [b, L, G, dk], v [b, L, H, dv], g, beta
    [b, L, H], state [b, H, dv, dk]. Returns (out, state)."""
    b, L, G, dk = q.shape
    H, dv = v.shape[2:]
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    if l2norm:
        q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    S = torch.zeros(b, H, dv, dk, dtype=torch.float64, device=q.device) if state is None else state.double()
    scale = dk ** -0.5 if scale is None else scale
    out = torch.empty(b, L, H, dv, dtype=torch.float64, device=q.device)
    for t in range(L):
        S = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhvk,bhk->bhv", S, k[:, t]))
        S = S + u[..., None] * k[:, t, :, None, :]
        out[:, t] = scale * torch.einsum("bhvk,bhk->bhv", S, q[:, t])
    return out, S


def rel_l2(got, want):
    d, n = float((got.double() - want.double()).norm()), float(want.double().norm())
    return d / n if n else d
