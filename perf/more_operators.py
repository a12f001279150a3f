"""Cases that measure block-sparse attention over the paged FP8 MLA cache and the attention of drafted trees.

Blocks are the cache's pages: ``mla_block_keys`` (a mean key for each page that new tokens completed),
``mla_block_scores`` (how much each token's heads want each complete block before its own), ``mla_block_select`` (the
blocks that it attends) and ``mla_block_attention`` (over their positions). Trees: ``mla_tree_mask`` and
``mla_tree_attention`` (drafted tokens that attend the context and their ancestors), ``mla_tree_commit`` (the accepted
path's rows moved together).

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, by the calls
a user makes of the library. ``exact`` restates each operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

LATENT, ROPE, TILE = 512, 64, 128
ROW, ROW_NOPE = 656, 528
DEV = "cuda"


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 256 sequences: about four of them complete a page of 64 with their new token.
        dict(name="keys_decode_256", kind="keys", seqs=256, new=1, ragged_new=False, ctx=1500, page=64, d_qk=576, row=ROW,
             shape=1),
        # Four prompts of up to 16,384 tokens written whole: the keys of all their pages.
        dict(name="keys_prompts_16384", kind="keys", seqs=4, new=16384, ragged_new=True, ctx=16384, page=64, d_qk=576,
             row=ROW, shape=2),

        # A decode step of 32 sequences with all 128 heads and contexts of up to 65,536: 1,024 blocks each.
        dict(name="scores_decode_h128", kind="scores", seqs=32, new=1, ragged_new=False, heads=128, d_qk=576, ctx=65536,
             page=64, shape=3),
        # A prefill chunk of 4,096 tokens behind a prefix of 12,288, 16 heads.
        dict(name="scores_prefill_4096", kind="scores", seqs=1, new=4096, ragged_new=False, heads=16, d_qk=576, ctx=16384,
             page=64, shape=0),

        # The selection for one decode step of 64 long sequences: 48 of up to 2,048 blocks.
        dict(name="select_decode_64", kind="select", seqs=64, new=1, ragged_new=False, ctx=131072, page=64, width=48,
             sink=1, local=2, ties=False, shape=4),
        # For the prefill chunk: 32 of up to 256 blocks, scores that tie.
        dict(name="select_prefill_4096", kind="select", seqs=1, new=4096, ragged_new=False, ctx=16384, page=64, width=32,
             sink=1, local=2, ties=True, shape=0),

        # Single new tokens of 64 sequences, each over 32 blocks of 64 at most (serving, ragged), 16 heads.
        dict(name="blocks_decode_64", kind="blocks", seqs=64, new=1, ragged_new=False, heads=16, d_qk=576, ctx=16384,
             page=64, row=ROW, width=32, shape=5),
        # The prefill chunk of 4,096 tokens, each over its own 32 blocks: the largest.
        dict(name="blocks_prefill_4096", kind="blocks", seqs=1, new=4096, ragged_new=False, heads=16, d_qk=576, ctx=16384,
             page=64, row=ROW, width=32, shape=0),

        # Trees of up to 31 drafted tokens of 16 sequences, NoPE rows, pages of 16.
        dict(name="tree_31_nope", kind="tree", seqs=16, new=31, ragged_new=True, heads=16, d_qk=512, ctx=8192, page=16,
             row=ROW_NOPE, reach=8, shape=6),
        # Trees of 60 drafted tokens of 8 sequences with all 128 heads.
        dict(name="tree_60_h128", kind="tree", seqs=8, new=60, ragged_new=False, heads=128, d_qk=576, ctx=16384, page=64,
             row=ROW, reach=12, shape=7),

        # The accepted paths of the small trees: at most 6 tokens of each.
        dict(name="commit_16", kind="commit", seqs=16, new=31, ragged_new=True, ctx=900, page=16, row=ROW_NOPE, path=6,
             shape=8),
        # Of 256 sequences' trees.
        dict(name="commit_256", kind="commit", seqs=256, new=60, ragged_new=False, ctx=300, page=64, row=ROW, path=9,
             shape=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["keys", "scores", "select", "blocks", "blocks", "tree", "tree", "commit"])
    c = dict(kind=kind, shape=rng.randint(1, 1 << 30), page=rng.choice([16, 32, 48, 64, 128]),
             ragged_new=rng.choice([True, False]))
    rope = rng.choice([True, True, False])
    d_qk, row = 576 if rope else 512, ROW if rope else rng.choice([ROW, ROW_NOPE])
    heads = rng.choice([5, 16, 16, 32, 64, 128])
    if kind == "keys":
        new = _log(rng, 1, 8192)
        return dict(c, seqs=max(1, min(256, _log(rng, 1, 65536) // new)), new=new, ctx=_log(rng, 1, 16384), d_qk=d_qk, row=row)
    if kind == "scores":
        new, ctx, seqs = _log(rng, 1, 2048), _log(rng, 4 * c["page"], 65536), _log(rng, 1, 48)
        # products at most about the largest listed scores', keys at most half a million
        while new * seqs > 1 and (new * heads * seqs * (max(new, ctx) // c["page"] + 1) > 1.5e7 or new * heads * seqs > 65536):
            seqs, new = (seqs + 1) // 2, new if seqs > 1 else (new + 1) // 2
        return dict(c, seqs=seqs, new=new, heads=heads, d_qk=d_qk, ctx=ctx)
    if kind == "select":
        # (the longest context has more blocks than are chosen: otherwise its scores would not matter)
        new, ctx, seqs = _log(rng, 1, 2048), _log(rng, 16 * c["page"], 131072), _log(rng, 1, 64)
        while new * seqs > 1 and new * seqs * (max(new, ctx) // c["page"] + 1) > 1000000:
            seqs, new = (seqs + 1) // 2, new if seqs > 1 else (new + 1) // 2
        sink, local = rng.randint(0, 3), rng.randint(1, 3)
        return dict(c, seqs=seqs, new=new, ctx=ctx, width=sink + local + _log(rng, 1, min(100, ctx // c["page"] // 2)), sink=sink, local=local,
                    ties=rng.choice([True, False]))
    if kind == "blocks":
        many = rng.choice([True, False])
        new, ctx = _log(rng, 33, 2048) if many else rng.choice([1, 1, 2, 4]), _log(rng, 1, 16384)
        seqs = rng.randint(1, 4) if many else _log(rng, 1, 64)
        width = _log(rng, 3, 3000 // c["page"])
        # at most about a quarter of the largest listed case's
        while seqs * new > 1 and (new * heads * max(new, ctx) * seqs > 2.5e8 or new * seqs * width * c["page"] > 1000000):
            seqs, new = (seqs + 1) // 2, new if seqs > 1 else (new + 1) // 2
        return dict(c, seqs=seqs, new=new, heads=heads, d_qk=d_qk, ctx=ctx, row=row, width=width)
    new = _log(rng, 1, 100)
    if kind == "commit":
        return dict(c, seqs=_log(rng, 1, 256), new=new, ctx=_log(rng, 1, 1000), row=row, path=rng.randint(1, 12))
    ctx, seqs = _log(rng, 1, 16384), _log(rng, 1, 32)
    while seqs > 1 and new * heads * max(new, ctx) * seqs > 2.5e8:
        seqs = (seqs + 1) // 2
    return dict(c, seqs=seqs, new=new, heads=heads, d_qk=d_qk, ctx=ctx, row=row, reach=rng.choice([1, 4, 12, 100]))


# What a case's own numbers say about its shape, on the host, without the seed.

def _shape(c):
    """Per sequence: new tokens and context length (the new ones included)."""
    r = random.Random(c["shape"])
    new = [r.randint(1, c["new"]) if c["ragged_new"] and c["seqs"] > 1 else c["new"] for _ in range(c["seqs"])]
    ctx = [max(n, r.randint(1, c["ctx"])) for n in new]
    ctx[0] = max(ctx[0], c["ctx"])
    if c["kind"] == "keys":
        ctx[0] = c["page"] * -(-ctx[0] // c["page"])      # one that completes a page, at least
    return new, ctx


def _paths(c):
    """Per sequence: the accepted drafted tokens, ascending."""
    r = random.Random(c["shape"] + 1)
    return [sorted(r.sample(range(n), r.randint(0, min(n, c["path"])))) for n in _shape(c)[0]]


def _before(n, L, page):
    """Sum over a sequence's new tokens of the complete blocks before each one's own."""
    return sum((L - n + i) // page for i in range(n))


def work(case):
    c = case
    new, ctx = _shape(c)
    page, T = c["page"], sum(new)
    if c["kind"] == "keys":
        done = sum(L // page - (L - n) // page for n, L in zip(new, ctx))
        return {"bytes": done * (page * (ROW if c["d_qk"] == 576 else ROW_NOPE) + 2 * c["d_qk"]) + 12 * len(new),
                "flops": done * page * (c["d_qk"] + LATENT)}
    if c["kind"] in ("scores", "select"):
        pairs = sum(_before(n, L, page) for n, L in zip(new, ctx))
        if c["kind"] == "select":
            return {"bytes": 4 * pairs + 4 * T * c["width"], "flops": 0}
        b = T * c["heads"] * 2 * c["d_qk"] + sum((L - 1) // page for L in ctx) * (2 * c["d_qk"] + 4) + 4 * pairs
        return {"bytes": b, "flops": 2.0 * pairs * c["heads"] * c["d_qk"]}
    if c["kind"] == "commit":
        moved = sum(1 for p in _paths(c) for j, i in enumerate(p) if i != j)
        return {"bytes": moved * (2 * c["row"] + 4) + 12 * len(new), "flops": 0}
    rope = c["d_qk"] == 576
    if c["kind"] == "blocks":
        rows = flops = 0
        for n, L in zip(new, ctx):
            pos = range(L - n, L)
            seen = sum(min(p // page, c["width"] - 1) * page + p % page + 1 for p in pos)
            rows += min(L, seen)
            flops += seen
        ints = T * c["width"]
    else:
        # the tree's part by its average depth is small beside the context
        rows, flops, ints = sum(ctx), sum(n * (L - n + min(n, 4)) for n, L in zip(new, ctx)), 2 * T
    b = rows * (ROW if rope else ROW_NOPE) + T * c["heads"] * (2 * c["d_qk"] + 2 * LATENT + 4) + 4 * ints
    return {"bytes": b, "flops": 2.0 * flops * c["heads"] * (c["d_qk"] + LATENT)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6947 + 29)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _cache(slots, row, g):
    """Rows as the writer leaves them: amax of each 128 over 448 as the scale, values over that to the nearest E4M3."""
    cache = torch.empty((slots, row), dtype=torch.uint8, device=DEV)
    step = 1 << 18
    for a in range(0, slots, step):
        x = _randn((min(step, slots - a), LATENT), g).float().view(-1, 4, TILE)
        scale = x.abs().amax(-1) / 448.0
        parts = [(x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, LATENT),
                 scale.contiguous().view(torch.uint8)]
        if row == ROW:
            parts.append(_randn((x.shape[0], ROPE), g).view(torch.uint8))
        cache[a:a + step] = torch.cat(parts, 1)
    return cache


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    new, ctx = _shape(c)
    page, T, S = c["page"], sum(new), len(new)
    pages = [-(-L // page) for L in ctx]
    total = sum(pages) + 1 + max(1, sum(pages) // 16)
    order = torch.randperm(total - 1, generator=g, device=DEV).to(torch.int32) + 1
    table = torch.full((S, max(pages) + 2), -1, dtype=torch.int32, device=DEV)
    first = 0
    for i, k in enumerate(pages):
        table[i, :k] = order[first:first + k]
        first += k
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"case": c, "table": table, "q_start": _ints(start), "kv_len": _ints(ctx), "n_tokens": T}
    # where each token stands: its sequence, its place among the new ones, its position
    s["seq"] = torch.tensor([i for i, n in enumerate(new) for _ in range(n)], device=DEV)
    s["place"] = torch.tensor([i for n in new for i in range(n)], device=DEV)
    s["pos"] = s["kv_len"].long()[s["seq"]] - torch.tensor(new, device=DEV)[s["seq"]] + s["place"]
    if c["kind"] in ("keys", "blocks", "tree", "commit"):
        s["cache"] = _cache(total * page, c["row"], g)
    if c["kind"] == "keys":
        s["keys"] = torch.zeros((total, c["d_qk"]), dtype=torch.bfloat16, device=DEV)
    if c["kind"] in ("scores", "blocks", "tree"):
        s["q"] = _randn((T, c["heads"], c["d_qk"]), g)
        s["scale"] = 1.0 / math.sqrt(c["d_qk"])
    if c["kind"] in ("blocks", "tree"):
        s["out"] = torch.empty((T, c["heads"], LATENT), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((T, c["heads"]), dtype=torch.float32, device=DEV)
    if c["kind"] == "scores":
        s["keys"] = _randn((total, c["d_qk"]), g)
        s["scores"] = torch.zeros(T, table.shape[1], device=DEV)
    if c["kind"] in ("select", "blocks"):
        # what the heads want of a block changes slowly from token to token
        taste = torch.randn((S, T // 64 + 1, table.shape[1]), generator=g, device=DEV)
        noise = torch.randn((T, table.shape[1]), generator=g, device=DEV)
        want = (1.5 * taste[s["seq"], torch.arange(T, device=DEV) // 64] + 0.5 * noise).softmax(-1)
        if c.get("ties"):
            want = (want * 4096).round() / 4096
            # blocks whose pages are not there
            want = torch.where(torch.rand(want.shape, generator=g, device=DEV) < 0.02, torch.full_like(want, -math.inf), want)
        s["scores"] = want
        s["blocks"] = torch.zeros((T, c["width"]), dtype=torch.int32, device=DEV)
        if c["kind"] == "blocks":
            s["blocks"] = _plain_select({**s, "case": dict(c, sink=1, local=1)})
            del s["scores"]
    if c["kind"] == "tree":
        r = random.Random(c["shape"] + 7 * seed)
        s["parent"] = _ints([r.randint(max(-1, i - c["reach"]), i - 1) for n in new for i in range(n)])
        s["words"] = -(-max(new) // 32)
        s["mask"] = torch.zeros((T, s["words"]), dtype=torch.int32, device=DEV)
        s["rotary"] = torch.zeros(T, dtype=torch.int32, device=DEV)
    if c["kind"] == "commit":
        paths = _paths(c)
        s["path"] = _ints([p + [0] * (c["path"] - len(p)) for p in paths])
        s["path_len"] = _ints([len(p) for p in paths])
        s["len_out"] = torch.zeros(S, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _views(cache):
    """A cache as the values it holds: E4M3 codes, tile scales, rotary values."""
    v = {"codes": cache[:, :LATENT].view(torch.float8_e4m3fn), "scales": cache[:, 512:528].view(torch.float32)}
    return v if cache.shape[1] == ROW_NOPE else {**v, "rope": cache[:, 528:].view(torch.bfloat16)}


def _widened(rows, d_qk):
    """Cache rows as 32-bit keys [..., d_qk]."""
    k = rows[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, TILE))
    k = (k * rows[..., 512:528].contiguous().view(torch.float32)[..., None]).flatten(-2)
    if d_qk == 576:
        k = torch.cat([k, rows[..., 528:].contiguous().view(torch.bfloat16).float()], -1)
    return k


def _plain_keys(s):
    c, page = s["case"], s["case"]["page"]
    done = (s["pos"] + 1) % page == 0                       # tokens that complete a page
    pg = s["table"].long()[s["seq"][done], s["pos"][done] // page]
    slots = pg[:, None] * page + torch.arange(page, device=DEV)
    s["keys"][pg] = _widened(s["cache"][slots], c["d_qk"]).mean(1).to(torch.bfloat16)
    return {"keys": s["keys"]}


def _plain_scores(s):
    c, table = s["case"], s["table"].long()
    k = s["keys"][table.clamp(min=0)].float()                                       # [S, blocks, d]
    q = torch.zeros((k.shape[0], max(_shape(c)[0]), c["heads"], c["d_qk"]), device=DEV)
    q[s["seq"], s["place"]] = s["q"].float()
    a = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, (-1, c["heads"]))[s["seq"], s["place"]] * s["scale"]
    b = torch.arange(table.shape[1], device=DEV)
    seen = b < (s["pos"] // c["page"])[:, None]
    a = torch.where(seen[:, None], a, torch.full_like(a, -math.inf))
    top = a.amax(-1, keepdim=True)
    p = (a - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    s["scores"] = torch.where(seen, p.sum(1), s["scores"])
    return {"scores": s["scores"]}


def _plain_select(s):
    c = s["case"]
    width, sc = c["width"], s["scores"]
    at = torch.arange(sc.shape[1], device=DEV)
    mine = (s["pos"] // c["page"])[:, None]
    always = (at <= mine) & ((at < c["sink"]) | (at > mine - c["local"]))
    may = (at <= mine) & (sc > -math.inf)
    rank = torch.where(always, torch.full_like(sc, math.inf), torch.where(may, sc, torch.full_like(sc, -math.inf)))
    value, got = torch.sort(rank, dim=-1, descending=True, stable=True)
    none = sc.shape[1]
    got = torch.where(value > -math.inf, got, torch.full_like(got, none))[:, :width]
    got = torch.sort(got, -1).values
    got = torch.where(got < none, got, torch.full_like(got, -1))
    blocks = torch.full((sc.shape[0], width), -1, dtype=torch.int32, device=DEV)
    blocks[:, :got.shape[1]] = got.int()
    return blocks


def _attend(q, k, seen, scale):
    """q [B, R, d], k [B, N, d], seen [B, R or 1, N] -> out [B, R, 512], lse [B, R]."""
    a = torch.matmul(q, k.transpose(1, 2)) * scale
    a = torch.where(seen, a, torch.full_like(a, -math.inf))
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (a - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, k[..., :LATENT])
    return torch.where(total > 0, o / total, torch.zeros_like(o)), (top + total.log())[..., 0]


def _context(s):
    """All positions of each sequence: keys [S, longest, d] and whether they are there."""
    c, page = s["case"], s["case"]["page"]
    at = torch.arange(max(_shape(c)[1]), device=DEV)
    slot = s["table"].long()[:, at // page] * page + at % page
    there = at < s["kv_len"].long()[:, None]
    k = _widened(s["cache"][torch.where(there, slot, torch.zeros_like(slot))], c["d_qk"])
    return at, torch.where(there[..., None], k, torch.zeros_like(k)), there


def _by_sequence(s, at, k, seen):
    """Attention of all tokens over their sequence's positions; seen [T, positions]."""
    c, H = s["case"], s["case"]["heads"]
    most = max(_shape(c)[0])
    q = torch.zeros((k.shape[0], most, H, c["d_qk"]), device=DEV)
    q[s["seq"], s["place"]] = s["q"].float()
    m = torch.zeros((k.shape[0], most, at.numel()), dtype=torch.bool, device=DEV)
    m[s["seq"], s["place"]] = seen
    m = m[:, :, None].expand(-1, -1, H, -1).flatten(1, 2)
    o, lse = _attend(q.flatten(1, 2), k, m, s["scale"])
    return {"out": o.unflatten(1, (-1, H))[s["seq"], s["place"]].to(torch.bfloat16),
            "lse": lse.unflatten(1, (-1, H))[s["seq"], s["place"]]}


def _plain_blocks(s):
    c, page, blocks = s["case"], s["case"]["page"], s["blocks"].long()
    if c["new"] > 32:
        # many tokens share most of the context: dense, with the other blocks masked
        at, k, _ = _context(s)
        wide = torch.zeros((blocks.shape[0], s["table"].shape[1] + 1), dtype=torch.bool, device=DEV)
        wide[:, :-1].scatter_(1, blocks.clamp(min=0), blocks >= 0)
        wide[:, 0] = (blocks == 0).any(1)
        return _by_sequence(s, at, k, wide[:, at // page] & (at <= s["pos"][:, None]))
    p = blocks[..., None] * page + torch.arange(page, device=DEV)
    pg = s["table"].long()[s["seq"][:, None], blocks.clamp(min=0)]
    seen = (blocks >= 0)[..., None] & (p <= s["pos"][:, None, None])
    slot = torch.where(seen, pg[..., None] * page + p % page, torch.zeros_like(p)).flatten(1)
    k = _widened(s["cache"][slot], c["d_qk"])
    o, lse = _attend(s["q"].float(), torch.where(seen.flatten(1)[..., None], k, torch.zeros_like(k)), seen.flatten(1)[:, None],
                     s["scale"])
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_tree(s):
    c = s["case"]
    n = s["q_start"][1:] - s["q_start"][:-1]
    most = max(_shape(c)[0])
    # each token reaches itself and its parent; squaring doubles how far
    reach = torch.zeros((c["seqs"], most, most + 1), device=DEV)
    reach[s["seq"], s["place"], s["place"]] = 1
    reach[s["seq"], s["place"], torch.where(s["parent"] < 0, torch.full_like(s["parent"], most), s["parent"]).long()] = 1
    reach = reach[..., :most]
    for _ in range(most.bit_length()):
        reach = (torch.matmul(reach, reach) > 0).float()
    bits = (reach[s["seq"], s["place"]] > 0)
    wide = torch.zeros((bits.shape[0], 32 * s["words"]), dtype=torch.int64, device=DEV)
    wide[:, :most] = bits
    word = (wide.unflatten(1, (-1, 32)) << torch.arange(32, device=DEV)).sum(-1)
    mask = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
    prefix = (s["kv_len"] - n).long()[s["seq"]]
    rotary = (prefix + bits.sum(-1) - 1).int()
    at, k, _ = _context(s)
    j = at - prefix[:, None]
    inside = torch.gather(bits, 1, j.clamp(0, most - 1)) & (j >= 0) & (j < most)
    return {"mask": mask, "rotary": rotary, **_by_sequence(s, at, k, (j < 0) | inside)}


def _plain_commit(s):
    c, page = s["case"], s["case"]["page"]
    n = s["q_start"][1:] - s["q_start"][:-1]
    prefix = (s["kv_len"] - n).long()[:, None]
    j = torch.arange(c["path"], device=DEV)
    ok = j < s["path_len"][:, None]
    src, dst = prefix + s["path"].long(), prefix + j
    row = torch.arange(c["seqs"], device=DEV)[:, None]
    table = s["table"].long()
    slot = lambda p: (table[row, p // page] * page + p % page)[ok]  # noqa: E731
    s["cache"][slot(torch.where(ok, dst, prefix))] = s["cache"][slot(torch.where(ok, src, prefix))]
    s["len_out"].copy_(prefix[:, 0] + s["path_len"])
    return {"len": s["len_out"], **_views(s["cache"])}


def _own_run(s):
    from fp8_mla_kv_gb300 import mlasparse as M
    c, where = s["case"], (s["q_start"], s["kv_len"], s["table"], s["case"]["page"])
    if c["kind"] == "keys":
        M.mla_block_keys(s["cache"], *where, s["keys"], s["n_tokens"])
        return {"keys": s["keys"]}
    if c["kind"] == "scores":
        M.mla_block_scores(s["q"], s["keys"], *where, s["scale"], scores=s["scores"])
        return {"scores": s["scores"]}
    if c["kind"] == "select":
        M.mla_block_select(s["scores"], s["q_start"], s["kv_len"], c["page"], c["width"], sink=c["sink"], local=c["local"],
                           blocks=s["blocks"])
        return {"blocks": s["blocks"]}
    if c["kind"] == "blocks":
        if "ws" not in s:
            s["ws"] = M.alloc_block_workspace(s["n_tokens"], c["heads"], c["width"])
        M.mla_block_attention(s["q"], s["cache"], s["blocks"], *where, s["scale"], out=s["out"], lse=s["lse"],
                              workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "tree":
        if "ws" not in s:
            s["ws"] = M.alloc_chunk_workspace(s["n_tokens"], c["heads"], c["seqs"])
        M.mla_tree_mask(s["parent"], s["q_start"], s["kv_len"], mask=s["mask"], positions=s["rotary"])
        M.mla_tree_attention(s["q"], s["cache"], *where, s["scale"], s["mask"], out=s["out"], lse=s["lse"],
                             workspace=s["ws"])
        return {"mask": s["mask"], "rotary": s["rotary"], "out": s["out"], "lse": s["lse"]}
    M.mla_tree_commit(s["cache"], *where, s["path"], s["path_len"], kv_len_out=s["len_out"])
    return {"len": s["len_out"], **_views(s["cache"])}


def run(state):
    if own:
        return _own_run(state)
    kind = state["case"]["kind"]
    if kind == "select":
        state["blocks"].copy_(_plain_select(state))
        return {"blocks": state["blocks"]}
    return {"keys": _plain_keys, "scores": _plain_scores, "blocks": _plain_blocks, "tree": _plain_tree,
            "commit": _plain_commit}[kind](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, i, L):
    """Keys of the first L positions of sequence i."""
    page = s["case"]["page"]
    p = torch.arange(L, device=DEV)
    rows = s["cache"][s["table"][i].long()[p // page] * page + p % page]
    k = rows[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double()
    k = k * rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(TILE, 1)
    return k if s["case"]["d_qk"] == 512 else torch.cat([k, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def exact(case, seed):
    c = case
    if c["kind"] in ("select", "commit"):
        return None                                       # whole numbers, and bytes that move
    s = prepare(c, seed)
    new, ctx = _shape(c)
    page = c["page"]
    if c["kind"] == "keys":
        keys = torch.zeros_like(s["keys"], dtype=torch.float64)
        for i, (n, L) in enumerate(zip(new, ctx)):
            first, last = (L - n) // page, L // page
            if last > first:
                k = _exact_rows(s, i, last * page)[first * page:].reshape(last - first, page, -1)
                keys[s["table"][i, first:last].long()] = k.sum(1) / page
        return {"keys": keys}
    H, at = c["heads"], 0
    if c["kind"] == "scores":
        scores = torch.zeros(s["scores"].shape, dtype=torch.float64, device=DEV)
        for i, (n, L) in enumerate(zip(new, ctx)):
            nb = (L - 1) // page
            k = s["keys"][s["table"][i, :nb].long()].double()
            for a in range(0, n, 256):
                q = s["q"][at + a:at + min(n, a + 256)].double()
                x = (q.reshape(-1, c["d_qk"]) @ k.t()).reshape(q.shape[0], H, nb) * s["scale"]
                full = (L - n + a + torch.arange(q.shape[0], device=DEV)) // page
                hidden = torch.arange(nb, device=DEV) >= full[:, None]
                x.masked_fill_(hidden[:, None], -math.inf)
                w = torch.nan_to_num(torch.softmax(x, -1)).sum(1)
                scores[at + a:at + a + q.shape[0], :nb] = w.masked_fill(hidden, 0.0)
            at += n
        return {"scores": scores}
    pairs = sum(n * L for n, L in zip(new, ctx)) * H * (c["d_qk"] + LATENT)
    if pairs > 1.3e12:
        return None
    out = torch.zeros((sum(new), H, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.full((sum(new), H), -math.inf, dtype=torch.float64, device=DEV)
    parent = s["parent"].tolist() if c["kind"] == "tree" else None
    for i, (n, L) in enumerate(zip(new, ctx)):
        k = _exact_rows(s, i, L)
        step = max(1, (1 << 27) // (H * L))
        for a in range(0, n, step):
            m = min(n, a + step) - a
            see = torch.zeros((m, L), dtype=torch.bool)
            if c["kind"] == "blocks":
                lists = s["blocks"][at + a:at + a + m].tolist()
                for x in range(m):
                    for b in lists[x]:
                        if b >= 0:
                            see[x, b * page:min((b + 1) * page, L - n + a + x + 1)] = True
            else:
                see[:, :L - n] = True
                for x in range(m):
                    up = a + x
                    while up >= 0:
                        see[x, L - n + up] = True
                        up = parent[at + up]
            v = (s["q"][at + a:at + a + m].double().reshape(m * H, -1) @ k.t()).reshape(m, H, L) * s["scale"]
            v.masked_fill_(~see.to(DEV)[:, None], -math.inf)
            total = torch.logsumexp(v, -1)
            w = torch.where(total[..., None] == -math.inf, torch.zeros_like(v), torch.exp(v - total[..., None]))
            out[at + a:at + a + m] = (w.reshape(m * H, L) @ k[:, :LATENT]).reshape(m, H, LATENT)
            lse[at + a:at + a + m] = total
        at += n
    return {"out": out, "lse": lse} if c["kind"] == "blocks" else {"mask": None, "rotary": None, "out": out, "lse": lse}
