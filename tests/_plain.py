"""Plain 64-bit forms of the rotary, chunk-attention and page operators, for their tests."""
from __future__ import annotations

import math

import torch

LATENT, ROPE = 512, 64
BF16 = 2.0 ** -8            # half a BF16 step, relative
F16 = 2.0 ** -11


def make_cache(n_slots, row, gen, rope=True, outliers=False):
    """A cache of valid rows: random codes without NaN, random positive scales, BF16 tails (CPU, uint8)."""
    c = torch.zeros((n_slots, row), dtype=torch.uint8)
    lat = torch.randn((n_slots, LATENT), generator=gen)
    if outliers:
        lat = torch.where(torch.rand(lat.shape, generator=gen) < 0.01, 20 * lat, lat)
    lat = lat.to(torch.bfloat16).float().view(n_slots, 4, 128)
    sc = lat.abs().amax(-1) / 448.0
    c[:, :512] = (lat / sc[..., None]).to(torch.float8_e4m3fn).view(n_slots, 512).view(torch.uint8)
    c[:, 512:528] = sc.contiguous().view(torch.uint8)
    if row == 656 and rope:
        c[:, 528:] = torch.randn((n_slots, ROPE), generator=gen).to(torch.bfloat16).view(torch.uint8)
    return c


def dequant(rows):
    """uint8 [n, row] -> (latent fp64 [n, 512], rope fp64 [n, 64] or None)."""
    lat = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    sc = rows[:, 512:528].contiguous().view(torch.float32).double()
    lat = lat * sc.repeat_interleave(128, 1)
    rope = rows[:, 528:].contiguous().view(torch.bfloat16).double() if rows.shape[1] == 656 else None
    return lat, rope


def chunk(q, cache, q_start, kv_len, table, page, scale, causal=True):
    """fp64 reference on the CPU: (out, lse, tol_out, tol_lse), NaN / -inf / 0 where the definition says so; tokens
    outside every sequence are NaN in tol_out.

    The tolerances follow from the kernel's roundings: P, the f16 scale ratio and their product are each off by
    at most half an f16 step (3 x 2^-11 of sum p|v|), the output by half a BF16 step, P below the f16 normal range by
    2^-25 of the largest value each; q.K is exact before fp32 accumulation, each of at most 64 additions
    losing 2^-23 of the sum of absolute products."""
    T, H, d = q.shape
    out = torch.zeros((T, H, LATENT), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    to = torch.full((T, H, LATENT), math.nan, dtype=torch.float64)
    tl = torch.zeros((T, H), dtype=torch.float64)
    qd = q.double()
    top = 0
    for s in range(len(kv_len)):
        a, b, L = int(q_start[s]), int(q_start[s + 1]), max(0, int(kv_len[s]))
        n = b - a
        taken = a >= top and a <= b <= T
        top = max(top, a)
        if not taken or n == 0:
            continue
        cap = table.shape[1] * page
        pos = torch.arange(min(L, cap))
        pg = table[s].long()[pos // page]
        slot = pg * page + pos % page
        ok = (pg >= 0) & (slot > 0) & (slot < cache.shape[0])
        pos, slot = pos[ok], slot[ok]
        lat, rope = dequant(cache[slot])
        bad = ~torch.isfinite(lat).all(1)
        key = lat
        if d == 576:
            bad |= ~torch.isfinite(rope).all(1)
            key = torch.cat([lat, rope], 1)
        key = torch.where(bad[:, None], torch.zeros_like(key), key)
        lat = torch.where(bad[:, None], torch.zeros_like(lat), lat)
        for i in range(n):
            last = L - n + i if causal else L - 1
            m = pos <= last
            to[a + i] = 1e-30
            if not m.any():
                continue
            if bad[m].any():
                out[a + i] = math.nan
                lse[a + i] = math.nan
                continue
            K, V = key[m], lat[m]
            sc = qd[a + i] @ K.t() * scale
            big = (qd[a + i].abs() @ K.abs().t()).amax(-1) * abs(scale)
            l = torch.logsumexp(sc, -1)
            p = torch.exp(sc - l[:, None])
            out[a + i] = p @ V
            lse[a + i] = l
            pv = p @ V.abs()
            n_keys = int(m.sum())
            to[a + i] = (3 * F16 + BF16) * pv + n_keys * 2.0 ** -24 * V.abs().max() + 64 * 2.0 ** -23 * big[:, None] * pv
            tl[a + i] = 64 * 2.0 ** -23 * big + 2.0 ** -20 * (1 + l.abs())
    return out, lse, to, tl


def check_chunk(out, lse, ref):
    ro, rl, to, tl = ref
    o, l = out.double().cpu(), lse.double().cpu()
    covered = ~torch.isnan(to[..., 0])
    nan = torch.isnan(rl) & covered
    assert torch.isnan(o[nan]).all() and torch.isnan(l[nan]).all(), "an attended non-finite row must give NaN"
    empty = torch.isneginf(rl) & covered
    assert (o[empty] == 0).all() and torch.isneginf(l[empty]).all(), "a token that attends nothing: 0 and -inf"
    ok = covered & ~nan & ~empty
    assert torch.isfinite(o[ok]).all() and torch.isfinite(l[ok]).all()
    eo = ((o - ro).abs() / to)[ok]
    el = ((l - rl).abs() / tl.clamp(min=1e-30))[ok]
    if eo.numel():
        assert eo.max() <= 1, f"out off by {eo.max():.3g} of its tolerance"
        assert el.max() <= 1, f"lse off by {el.max():.3g} of its tolerance"


def rotate(x, pos, inv_freq, axis, interleaved, scale=1.0, inverse=False):
    """x fp64 [n, heads, 64]; returns (y, sum of absolute products) in fp64."""
    y = torch.empty_like(x)
    mag = torch.empty_like(x)
    pos = pos if pos.dim() == 2 else pos[None]
    for i in range(32):
        ang = pos[axis[i]].double() * inv_freq[i] * (-1 if inverse else 1)
        c, s = (torch.cos(ang) * scale)[:, None], (torch.sin(ang) * scale)[:, None]
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
        mag[..., lo] = mag[..., hi] = (a.abs() + b.abs()) * abs(scale)
    return y, mag
