"""Latent attention in 64 bits, written from the formulas of include/coli_mla.h, with the tolerances of its tests.

Tolerances count roundings, each off by at most u = eps / 2 of its type relative to the value rounded.  Products and
sums run in binary32 (u32 = 2^-24) and are bounded by the length of the sum times u32 times the sum of magnitudes."""
from __future__ import annotations

import math

import torch

ROPE = 64
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}   # a step of the subnormals
U32 = 2.0 ** -24


def cumulative(lens, device):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(device)


def rotate(x, positions, inv_freq, halves):
    """x [n, ..., 64] in 64 bits."""
    a = positions.double().view(-1, *([1] * (x.dim() - 1))) * inv_freq.double()
    c, s = a.cos(), a.sin()
    x = x.double()
    p, q = (x[..., :32], x[..., 32:]) if halves else (x[..., 0::2], x[..., 1::2])
    p, q = p * c - q * s, q * c + p * s
    return torch.cat([p, q], -1) if halves else torch.stack([p, q], -1).flatten(-2)


def norm(x, g, eps):
    x = x.double()
    return x if g is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * g.double()


def rows_of(pages, scale, rank, dtype):
    """Latents and keys of every slot in 64 bits."""
    flat = pages.reshape(-1, pages.shape[-1])
    if scale is None:
        return flat[:, :rank].double(), flat[:, rank:].double()
    lat = flat[:, :rank].contiguous().view(torch.float8_e4m3fn).double() * scale.double()[:, None]
    return lat, flat[:, rank:].contiguous().view(dtype).double()


def slots_of(table, b, n, page):
    t = torch.arange(n, device=table.device)
    return table[b].long()[t // page] * page + t % page


def attend(s, v):
    """s [rows, keys] (-inf: not seen), v [keys, width]: output, lse and sum of |p v| (for the tolerance)."""
    if s.shape[1] == 0:
        z = torch.zeros(s.shape[0], v.shape[1], dtype=torch.float64, device=s.device)
        return z, torch.full((s.shape[0],), -math.inf, dtype=torch.float64, device=s.device), z
    lse = torch.logsumexp(s, -1)
    p = torch.where(lse[:, None] == -math.inf, 0.0, (s - lse[:, None]).exp())
    finite = torch.where(v.isfinite(), v, 0.0)
    out = p @ finite
    # a value that is not finite reaches the rows that see it, and no other
    seen = (p > 0).double()
    up, down, nan = (seen @ w.double() > 0 for w in (v == math.inf, v == -math.inf, v.isnan()))
    out = torch.where(up, math.inf, torch.where(down, -math.inf, out))
    return torch.where(nan | (up & down), math.nan, out), lse, p @ finite.abs()


def decode(q_lat, q_pe, lat, key, table, lens, n_q, page, scale):
    n, h, rank = q_lat.shape
    out = torch.zeros(n, h, rank, dtype=torch.float64, device=q_lat.device)
    mag = torch.zeros_like(out)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=q_lat.device)
    smag = torch.zeros_like(lse)
    for b, m in enumerate(lens):
        at = slots_of(table, b, m, page)
        for j in range(n_q):
            seen = m - n_q + 1 + j
            if seen > 0:
                r = b * n_q + j
                c, k = lat[at[:seen]], key[at[:seen]]
                q, qp = q_lat[r].double(), q_pe[r].double()
                out[r], lse[r], mag[r] = attend((q @ c.t() + qp @ k.t()) * scale, c)
                smag[r] = ((q.abs() @ c.abs().t() + qp.abs() @ k.abs().t()) * scale).amax(-1)
    return out, lse, mag, smag


def prefill(q, k_nope, k_pe, v, q_lens, k_lens, causal, scale):
    n, h, wide = q.shape
    nope = wide - ROPE
    out = torch.zeros(n, h, v.shape[-1], dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=q.device)
    smag = torch.zeros_like(lse)
    q0 = k0 = 0
    for a, m in zip(q_lens, k_lens):
        hidden = torch.zeros((a, m), dtype=torch.bool, device=q.device)
        if causal:
            hidden = torch.arange(m, device=q.device)[None] > torch.arange(a, device=q.device)[:, None] + m - a
        for i in range(h):
            x, kn, kp = q[q0:q0 + a, i].double(), k_nope[k0:k0 + m, i].double(), k_pe[k0:k0 + m].double()
            s = (x[:, :nope] @ kn.t() + x[:, nope:] @ kp.t()) * scale
            if a and m:
                sm = (x[:, :nope].abs() @ kn.abs().t() + x[:, nope:].abs() @ kp.abs().t()) * scale
                smag[q0:q0 + a, i] = sm.masked_fill(hidden, 0.0).amax(-1)
            o, l, g = attend(s.masked_fill(hidden, -math.inf), v[k0:k0 + m, i].double())
            out[q0:q0 + a, i], lse[q0:q0 + a, i], mag[q0:q0 + a, i] = o, l, g
        q0, k0 = q0 + a, k0 + m
    return out, lse, mag, smag


def close(got, want, tol, what):
    """|got - want| <= tol element by element; non-finite values have to agree."""
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {float(got[at])!r}, "
                             f"want {float(want[at])!r}, tolerance {float(torch.as_tensor(tol).expand_as(want)[at])!r}")


def attend_tol(out, mag, smag, width, keys, dtype):
    """Tolerances of (out, lse).

    A score is a sum of `width` products in binary32 (width * u32 * its magnitude sum smag, and the scaling and the
    exponent's own argument: 8 u32 * smag more); exp turns its error into a relative one of the weight, on the weights
    and on their sum: twice.  The weights are rounded to 16 bits before their product (u), which weighs sum |p v|; the
    sums over the keys are in binary32 (keys * u32, twice); the result is rounded (u)."""
    ds = (width + 8) * U32 * smag
    rel = 2 * ds + 2 * (keys + 16) * U32 + U[dtype] * (1 + 2.0 ** -6)
    return rel[..., None] * mag + U[dtype] * out.abs() * (1 + 2.0 ** -6) + TINY[dtype], ds + (keys + 16) * U32 + 2 * U32 * 128
