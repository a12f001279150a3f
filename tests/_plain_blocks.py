"""Plain 64-bit forms of the block-sparse and tree operators, and the batches that their tests take."""
from __future__ import annotations

import math

import torch

import _plain as P


def batch(seqs, H, d_qk, page, row, seed=0, extra=2, tail_tokens=0, head_tokens=0):
    """seqs: (new tokens, context length). Pages in random order, page 0 unused; tokens before the first sequence and
    behind the last."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-L // page) for _, L in seqs]
    total = sum(pages) + 3
    cache = P.make_cache(total * page, row, g, rope=d_qk == 576)
    order = torch.randperm(total - 1, generator=g).to(torch.int32) + 1
    table = torch.full((len(seqs), max(pages + [0]) + extra), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(pages):
        table[i, :k] = order[at:at + k]
        at += k
    start = [head_tokens]
    for n, _ in seqs:
        start.append(start[-1] + n)
    T = start[-1] + tail_tokens
    q = torch.randn((T, H, d_qk), generator=g).to(torch.bfloat16)
    return dict(q=q, cache=cache, q_start=torch.tensor(start, dtype=torch.int32),
                kv_len=torch.tensor([L for _, L in seqs], dtype=torch.int32), table=table, page=page,
                scale=1.0 / math.sqrt(d_qk), T=T, pages=total)


def tokens(b):
    """(token, sequence, index within it, position) of every token that is in a sequence; the position at most the
    table's last."""
    cap = b["table"].shape[1] * b["page"]
    for s in range(len(b["kv_len"])):
        a, e, L = int(b["q_start"][s]), int(b["q_start"][s + 1]), max(0, int(b["kv_len"][s]))
        for t in range(a, e):
            yield t, s, t - a, min(L - (e - a) + t - a, cap - 1)


def attend(b, sees):
    """fp64 on the CPU: out, lse and their tolerances (as in _plain.chunk, whose derivation holds: the
    arithmetic is the same). sees[t]: the positions that token t attends, whether they are there or not."""
    q, cache, table, page = b["q"], b["cache"], b["table"], b["page"]
    T, H, d = q.shape
    out = torch.zeros((T, H, 512), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    to = torch.full((T, H, 512), math.nan, dtype=torch.float64)
    tl = torch.zeros((T, H), dtype=torch.float64)
    lat, rope = P.dequant(cache)
    bad = ~torch.isfinite(lat).all(1)
    key = lat
    if d == 576:
        bad |= ~torch.isfinite(rope).all(1)
        key = torch.cat([lat, rope], 1)
    for t, s, _, _ in tokens(b):
        pos = torch.as_tensor(sees[t], dtype=torch.long)
        pos = pos[(pos >= 0) & (pos < table.shape[1] * page)]
        pg = table[s].long()[pos // page]
        slot = pg * page + pos % page
        slot = slot[(pg >= 0) & (slot > 0) & (slot < cache.shape[0])]
        to[t] = 1e-30
        if not slot.numel():
            continue
        if bad[slot].any():
            out[t] = lse[t] = math.nan
            continue
        K, V = key[slot], lat[slot]
        qd = q[t].double()
        sc = qd @ K.t() * b["scale"]
        big = (qd.abs() @ K.abs().t()).amax(-1) * abs(b["scale"])
        l = torch.logsumexp(sc, -1)
        p = torch.exp(sc - l[:, None])
        pv = p @ V.abs()
        out[t], lse[t] = p @ V, l
        to[t] = (3 * P.F16 + P.BF16) * pv + slot.numel() * 2.0 ** -24 * V.abs().max() + 64 * 2.0 ** -23 * big[:, None] * pv
        tl[t] = 64 * 2.0 ** -23 * big + 2.0 ** -20 * (1 + l.abs())
    return out, lse, to, tl


def block_positions(b, blocks):
    """Per token the positions up to its own of its blocks."""
    sees = [[] for _ in range(b["T"])]
    for t, _, _, pos in tokens(b):
        mine = {int(x) for x in blocks[t] if 0 <= int(x) < b["table"].shape[1]}
        sees[t] = [p for x in sorted(mine) for p in range(x * b["page"], min((x + 1) * b["page"], pos + 1))]
    return sees


def mean_keys(b, d_qk, num_keys):
    """{page: (key fp64, tolerance)} of the pages that the batch's tokens complete: fp32 sums of up to `rows` terms lose at
    most 2^-24 of the running sum of sizes each, the quotient half an fp32 step, the key half a BF16 step."""
    lat, rope = P.dequant(b["cache"])
    key = lat if d_qk == 512 else torch.cat([lat, rope], 1)
    page, done = b["page"], {}
    for s in range(len(b["kv_len"])):
        n, L = int(b["q_start"][s + 1] - b["q_start"][s]), max(0, int(b["kv_len"][s]))
        if n == 0:
            continue
        for k in range(max(0, L - n) // page, min(L // page, b["table"].shape[1])):
            phys = int(b["table"][s, k])
            if phys < 0 or phys >= num_keys:
                continue
            slots = [x for x in range(phys * page, (phys + 1) * page) if 0 < x < key.shape[0]]
            rows = key[slots]
            m = rows.sum(0) / max(1, len(slots))
            size = rows.abs().sum(0) / max(1, len(slots))
            done[phys] = (m, P.BF16 * m.abs() + (len(slots) + 10) * 2.0 ** -24 * size + 1e-38)
    return done


def block_scores(b, keys, num_keys=None):
    """(scores fp64 [T, max_pages], tolerance; NaN in the tolerance where nothing is written). A score's exponentials are
    off by twice the largest error of a logit (64 additions losing 2^-23 of the sum of absolute products, and the
    product with the scale), their sums by 2^-24 a term."""
    T, H, _ = b["q"].shape
    page, table = b["page"], b["table"]
    num_keys = keys.shape[0] if num_keys is None else num_keys
    sc = torch.zeros((T, table.shape[1]), dtype=torch.float64)
    tol = torch.full((T, table.shape[1]), math.nan, dtype=torch.float64)
    k64 = keys.double()
    for t, s, _, pos in tokens(b):
        n = pos // page if pos >= 0 else 0
        pg = table[s, :n].long()
        ok = (pg >= 0) & (pg < num_keys)
        sc[t, :n] = -math.inf
        tol[t, :n] = 0.0
        if not ok.any():
            continue
        K, q = k64[pg[ok]], b["q"][t].double()
        x = q @ K.t() * b["scale"]
        off = (64 * 2.0 ** -23 * (q.abs() @ K.abs().t()) * abs(b["scale"]) + 2.0 ** -22 * x.abs()).amax(-1, keepdim=True)
        p = torch.softmax(x, -1)
        at = torch.arange(n)[ok]
        sc[t, at] = p.sum(0)
        tol[t, at] = (p * (2 * off + (n + H + 8) * 2.0 ** -24 + 2.0 ** -20)).sum(0) + 1e-30
    return sc, tol


def select(b, scores, width, sink, local):
    """Row by row, in plain Python; None where a token is in no sequence."""
    rows = [None] * b["T"]
    for t, _, _, pos in tokens(b):
        own = pos // b["page"] if pos >= 0 else -1
        forced = [x for x in range(own + 1) if x < sink or x > own - local]
        row = scores[t].tolist()
        rest = [x for x in range(own + 1) if x not in set(forced) and row[x] > -math.inf]
        rest.sort(key=lambda x: (-row[x], x))
        got = sorted(forced + rest[:width - len(forced)])
        rows[t] = got + [-1] * (width - len(got))
    return rows


def ancestors(b, parent):
    """Per token the indices (within its sequence) of itself and its ancestors; a parent that does not come before
    its child is none."""
    up = [[] for _ in range(b["T"])]
    for t, _, i, _ in tokens(b):
        p = int(parent[t])
        up[t] = [i] + (up[t - i + p] if 0 <= p < i else [])
    return up


def mask_bits(rows, T, words):
    m = torch.zeros((T, words), dtype=torch.int64)
    for t, r in enumerate(rows):
        for j in r:
            if j < 32 * words:
                m[t, j // 32] |= 1 << (j % 32)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32)


def tree_positions(b, rows):
    """Per token the context's positions and those of the drafted tokens rows[t]."""
    sees = [[] for _ in range(b["T"])]
    for t, s, _, _ in tokens(b):
        n, L = int(b["q_start"][s + 1] - b["q_start"][s]), max(0, int(b["kv_len"][s]))
        sees[t] = list(range(max(0, L - n))) + [L - n + j for j in sorted(set(rows[t])) if 0 <= L - n + j and j < n]
    return sees
