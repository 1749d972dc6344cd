"""Plain 64-bit forms of the gated delta rule and the block plan, and inputs for
their tests (CPU; nothing here uses the CUDA library)."""
from __future__ import annotations

import math

import torch

BF16, F32 = torch.bfloat16, torch.float32


def unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)


def tokens(lead, Hk, H, dk, dv, dtype, seed, rate=(0.01, 2.0)):
    """q, k (unit rows), v, g (log-decays, one rate per head), beta of ``lead`` tokens."""
    gen = torch.Generator().manual_seed(seed)
    q = unit(torch.randn(*lead, Hk, dk, generator=gen)).to(dtype)
    k = unit(torch.randn(*lead, Hk, dk, generator=gen)).to(dtype)
    v = torch.randn(*lead, H, dv, generator=gen).to(dtype)
    lo, hi = math.log(rate[0]), math.log(rate[1])
    r = torch.exp(torch.rand(H, generator=gen) * (hi - lo) + lo)
    g = -r * torch.nn.functional.softplus(torch.randn(*lead, H, generator=gen))
    beta = torch.sigmoid(torch.randn(*lead, H, generator=gen))
    return dict(q=q, k=k, v=v, g=g, beta=beta)


def pool(rows, H, dk, dv, seed, std=0.2):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(rows, H, dk, dv, generator=gen) * std


def cu_of(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)


def step(S, q, k, v, g, beta, scale):
    """One token on S [H, dk, dv] (float64): the section's equations, literally."""
    Sb = torch.exp(g)[:, None, None] * S
    seen = torch.einsum("hkv,hk->hv", Sb, k)
    S = Sb + beta[:, None, None] * k[:, :, None] * (v - seen)[:, None, :]
    return S, scale * torch.einsum("hkv,hk->hv", S, q)


def reference(x, spans, H, scale, state, src, dst, ctx=None, table=None, block=0, update=True):
    """Token by token in float64.  ``spans``: (first token, tokens) per sequence into
    x's flat [tokens, heads, d] tensors.  Returns (o float64, pool float64); rows of o
    that no sequence covers are NaN."""
    rep = H // x["q"].shape[-2]
    f = {n: t.double() for n, t in x.items()}
    q, k = f["q"].repeat_interleave(rep, 1), f["k"].repeat_interleave(rep, 1)
    dv = x["v"].shape[-1]
    o = torch.full((x["v"].shape[0], H, dv), float("nan"), dtype=torch.float64)
    old = state.double() if state is not None else None
    new = old.clone() if state is not None else None
    P = 0 if state is None else state.shape[0]
    for n, (t0, length) in enumerate(spans):
        s = -1 if src is None else int(src[n])
        S = old[s].clone() if 0 <= s < P else torch.zeros(H, q.shape[-1], dv, dtype=torch.float64)
        c0 = 0 if ctx is None else int(ctx[n])
        for t in range(t0, t0 + length):
            S, o[t] = step(S, q[t], k[t], f["v"][t], f["g"][t], f["beta"][t], scale)
            pos = c0 + t - t0 + 1
            if block and pos % block == 0 and pos // block <= table.shape[1]:
                r = int(table[n, pos // block - 1])
                if 0 <= r < P and update:
                    new[r] = S
        d = -1 if dst is None else int(dst[n])
        if 0 <= d < P and update:
            new[d] = S
    return o, new


def plan_reference(new, ctx, free, head, table, bs, T):
    """The block plan by plain loops; returns the outputs as lists (table included)."""
    table = [list(r) for r in table]
    M = len(table[0]) if table else 0
    cu, src, dst, pos, slots = [0], [], [], [], []
    head = max(head, 0)
    for n, b in enumerate(new):
        b, a = max(b, 0), 0 if ctx is None else max(ctx[n], 0)
        for j in range(-(-a // bs), -(-(a + b) // bs)):
            if j < M:
                table[n][j] = free[head] if head < len(free) else -1
            head += 1
        cu.append(cu[-1] + b)

        def at(j):
            return table[n][j] if j < M else -1
        src.append(at((a - 1) // bs) if a else -1)
        dst.append(at((a + b - 1) // bs) if a + b else -1)
        for p in range(a, a + b):
            pos.append(p)
            slots.append(at(p // bs) * bs + p % bs if at(p // bs) >= 0 else -1)
    pos, slots = (x[:T] + [-1] * (T - len(x)) for x in (pos, slots))
    return cu, pos, slots, src, dst, head, table


def max_err(got, ref):
    """max |got - ref| / max |ref|; a NaN anywhere in got is infinite error."""
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape
    if got.numel() == 0:
        return 0.0
    if not torch.isfinite(got).all():
        return float("inf")
    return float((got - ref).abs().max() / ref.abs().max().clamp_min(1e-30))
