"""Cases that measure the operators around the paged FP8 MLA cache: the rotary
positions fused with the cache write (``mla_rope_kv_write``), the attention of a
chunk of new tokens over the paged cache (``mla_chunk_attention``), and the cache's
pages (``mla_page_copy``, ``mla_page_fork``, ``mla_page_free``, ``mla_page_compact``).

``run`` computes a case either in its plain form (elementary torch operations in 32
bits, 64 where 32 lose what matters) or, where ``own`` is true, by the calls a user
makes of the library. ``exact`` restates each operator's definition in 64 bits.
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
        # One decode step of one sequence on a 16-head shard: one new row, text only (one axis).
        dict(name="rope_write_1", kind="write", rows=1, heads=16, axes=1, interleaved=True, pad=0, far=131072,
             slots=4096),
        # A decode step of 67 sequences with all 128 heads on one GPU, a few of them padding.
        dict(name="rope_write_67_h128", kind="write", rows=67, heads=128, axes=1, interleaved=True, pad=5,
             far=1000000, slots=16384),
        # An image's tokens in a prefill chunk: time, height and width positions, halves layout.
        dict(name="rope_write_1024_3d", kind="write", rows=1024, heads=16, axes=3, interleaved=False, pad=0,
             far=32768, slots=65536),
        # The largest prefill step of the writer benchmark (8,192 rows, a quarter aimed at the reserved slot), video.
        dict(name="rope_write_8192_3d", kind="write", rows=8192, heads=64, axes=3, interleaved=False, pad=2048,
             far=131072, slots=65536),

        # Single new tokens of four sequences, short contexts: the smallest decode step, where latency counts.
        dict(name="chunk_decode_4", kind="chunk", seqs=4, new=1, ragged_new=False, heads=16, d_qk=576, ctx=700,
             shape=1, page=64, row=ROW, causal=True, outliers=False),
        # Single new tokens of 64 sequences with contexts of 1..16,384 (serving, ragged), 16 heads.
        dict(name="chunk_decode_64", kind="chunk", seqs=64, new=1, ragged_new=False, heads=16, d_qk=576, ctx=16384,
             shape=2, page=64, row=ROW, causal=True, outliers=False),
        # Two tokens each (a draft token verified) with all 128 heads, 1 % outliers of x20 in the cache.
        dict(name="chunk_verify_h128", kind="chunk", seqs=24, new=2, ragged_new=False, heads=128, d_qk=576, ctx=16384,
             shape=3, page=64, row=ROW, causal=True, outliers=True),
        # NoPE rows of 528 bytes, pages of 16, odd chunk lengths: a mixed batch of short prefills and decodes.
        dict(name="chunk_mixed_nope", kind="chunk", seqs=9, new=131, ragged_new=True, heads=16, d_qk=512, ctx=1900,
             shape=4, page=16, row=ROW_NOPE, causal=True, outliers=False),
        # A prefill chunk of 4,096 tokens behind a prefix of 12,288: the largest.
        dict(name="chunk_prefill_4096", kind="chunk", seqs=1, new=4096, ragged_new=False, heads=16, d_qk=576,
             ctx=16384, shape=0, page=64, row=ROW, causal=True, outliers=False),

        # A step of parallel sampling: 32 children dropped and forked anew from 8 parents.
        dict(name="pages_fork_32", kind="fork", pages=2048, page=64, parents=8, forks=32, length=5000, shape=5),
        # Pages handed from one cache to another (a finished prefill to the decode's cache), shuffled.
        dict(name="pages_copy_1500", kind="copy", pages=4096, page=64, moved=1500, shape=6),
        # The 1,048,576-slot cache half empty after a burst: live pages moved to the front.
        dict(name="pages_compact_16384", kind="compact", pages=16384, page=64, seqs=64, live=0.5, shape=7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["write", "write", "chunk", "chunk", "chunk", "fork", "copy", "compact"])
    if kind == "write":
        rows = _log(rng, 1, 8192)
        return dict(kind=kind, rows=rows, heads=rng.choice([1, 7, 16, 32, 64]), axes=rng.choice([1, 2, 3]),
                    interleaved=rng.choice([True, False]), pad=rng.randint(0, rows // 4), far=_log(rng, 100, 1000000),
                    slots=65536)
    if kind == "chunk":
        rope = rng.choice([True, True, False])
        heads = rng.choice([5, 16, 16, 32, 64, 128])
        new = _log(rng, 1, 2048)
        ctx = _log(rng, 1, 16384)
        seqs = _log(rng, 1, 48)
        # at most about a third of the largest listed case's products
        while new * heads * max(new, ctx) * seqs > 3.5e8:
            if seqs > 1:
                seqs = (seqs + 1) // 2
            else:
                new = (new + 1) // 2
        return dict(kind=kind, seqs=seqs, new=new, ragged_new=rng.choice([True, False]), heads=heads,
                    d_qk=576 if rope else 512, ctx=ctx, shape=rng.randint(0, 1 << 30), page=rng.choice([1, 16, 48, 64, 128]),
                    row=ROW if rope else rng.choice([ROW, ROW_NOPE]), causal=rng.choice([True, True, False]),
                    outliers=rng.choice([False, False, True]))
    page = rng.choice([16, 32, 64])
    if kind == "fork":
        parents = _log(rng, 1, 16)
        forks = _log(rng, 1, 64)
        length = _log(rng, 1, 6000)
        return dict(kind=kind, pages=(parents + 2) * (length // page + 2) + 2 * forks + rng.randint(2, 300), page=page,
                    parents=parents, forks=forks, length=length, shape=rng.randint(0, 1 << 30))
    if kind == "copy":
        pages = _log(rng, 16, 4096)
        return dict(kind=kind, pages=pages, page=page, moved=_log(rng, 1, pages - 1), shape=rng.randint(0, 1 << 30))
    return dict(kind=kind, pages=_log(rng, 64, 12000), page=page, seqs=_log(rng, 1, 64),
                live=rng.uniform(0.05, 0.9), shape=rng.randint(0, 1 << 30))


# What a case's own numbers say about its shape, on the host, without the seed.

def _chunk_shape(c):
    """Per sequence: new tokens and context length (the chunk included)."""
    r = random.Random(c["shape"])
    if c["seqs"] == 1:
        return [c["new"]], [c["ctx"]]
    new = [r.randint(1, c["new"]) if c["ragged_new"] else c["new"] for _ in range(c["seqs"])]
    # contexts from one token on; a chunk is never longer than its context, but for one sequence in the
    # ragged mixes whose first tokens have nothing to attend
    ctx = [max(n, r.randint(1, c["ctx"])) for n in new]
    if c["ragged_new"] and new[-1] > 1:
        ctx[-1] = new[-1] - 1
    ctx[0] = max(ctx[0], c["ctx"])
    return new, ctx


def _attended(c):
    """Sum over tokens of the positions each attends."""
    new, ctx = _chunk_shape(c)
    if not c["causal"]:
        return sum(n * L for n, L in zip(new, ctx))
    return sum(max(0, L - n + i + 1) for n, L in zip(new, ctx) for i in range(n))


def _fork_shape(c):
    r = random.Random(c["shape"])
    lens = [max(1, r.randint(c["length"] // 2, c["length"])) for _ in range(c["parents"])]
    parent = [r.randrange(c["parents"]) for _ in range(c["forks"])]
    return lens, parent


def _compact_moves(c):
    """Which pages are live (page 0 never), and how many of them have to move."""
    r = random.Random(c["shape"])
    live = [False] + [r.random() < c["live"] for _ in range(c["pages"] - 1)]
    n = sum(live)
    return live, sum(live[n + 1:])


def work(case):
    c = case
    if c["kind"] == "write":
        kept = c["rows"] - c["pad"]
        b = c["rows"] * 8 + kept * (2 * LATENT + 2 * ROPE + ROW) + c["rows"] * 4 * c["axes"]
        b += c["rows"] * c["heads"] * 2 * 2 * ROPE
        return {"bytes": b, "flops": c["rows"] * (c["heads"] + 1) * 3 * ROPE + kept * 4 * LATENT}
    if c["kind"] == "chunk":
        new, ctx = _chunk_shape(c)
        T, rope = sum(new), c["d_qk"] == 576
        b = sum(ctx) * (ROW if rope else ROW_NOPE) + T * c["heads"] * (2 * c["d_qk"] + 2 * LATENT + 4)
        b += sum((L + c["page"] - 1) // c["page"] for L in ctx) * 4
        return {"bytes": b, "flops": 2.0 * _attended(c) * c["heads"] * (c["d_qk"] + LATENT)}
    row = ROW
    if c["kind"] == "fork":
        lens, parent = _fork_shape(c)
        rem = sum(lens[p] % c["page"] for p in parent)
        entries = sum(-(-lens[p] // c["page"]) for p in parent)
        return {"bytes": 2 * rem * row + 4 * entries * 5, "flops": 0}
    if c["kind"] == "copy":
        return {"bytes": c["moved"] * (2 * c["page"] * row + 8), "flops": 0}
    live, moves = _compact_moves(c)
    return {"bytes": 2 * moves * c["page"] * row + 3 * 4 * c["pages"] + 8 * sum(live), "flops": 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(shape, g, outliers=False):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if outliers:
        x = torch.where(torch.rand(shape, generator=g, device=DEV) < 0.01, 20 * x, x)
    return x.to(torch.bfloat16)


def _quantised(latent):
    """Rows of codes and of scales: amax of each 128 over 448, values over that, to the nearest E4M3."""
    x = latent.float().view(-1, 4, TILE)
    amax = x.abs().amax(-1)
    # 448 as a tensor: a Python number would be turned into a product with its reciprocal
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    codes = (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(-1, LATENT), scale


def _cache_rows(latent, rope, row):
    codes, scale = _quantised(latent)
    parts = [codes, scale.contiguous().view(torch.uint8)]
    if row == ROW:
        parts.append(torch.zeros((codes.shape[0], 128), dtype=torch.uint8, device=DEV) if rope is None
                     else rope.contiguous().view(torch.uint8))
    return torch.cat(parts, 1)


def _frequencies(c):
    """Radians a position for each of the 32 pairs, and the axis whose position turns it (contiguous sections)."""
    inv = [10000.0 ** (-2.0 * i / ROPE) for i in range(32)]
    cut = {1: [32], 2: [16, 16], 3: [8, 12, 12]}[c["axes"]]
    return inv, [a for a, n in enumerate(cut) for _ in range(n)]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "write":
        n, H = c["rows"], c["heads"]
        slots = torch.randperm(c["slots"] - 1, generator=g, device=DEV)[:n] + 1
        if c["pad"]:
            slots[torch.randperm(n, generator=g, device=DEV)[:c["pad"]]] = 0
        s["slots"] = slots
        s["latent"] = _randn((n, LATENT), g)
        s["k_pe"] = _randn((n, ROPE), g)
        s["pos"] = torch.randint(0, c["far"], (c["axes"], n), generator=g, device=DEV, dtype=torch.int32)
        # the query projection's output [n, H, 128 + 64]: its last 64 values are the ones to rotate
        s["q_proj"] = _randn((n, H, 192), g)
        s["q"] = torch.zeros((n, H, LATENT + ROPE), dtype=torch.bfloat16, device=DEV)
        s["cache"] = torch.zeros((c["slots"], ROW), dtype=torch.uint8, device=DEV)
        return s
    if c["kind"] == "chunk":
        new, ctx = _chunk_shape(c)
        page, row, H, T = c["page"], c["row"], c["heads"], sum(new)
        pages = [-(-L // page) for L in ctx]
        total = sum(pages) + 1 + max(1, sum(pages) // 16)
        slots = total * page
        cache = torch.empty((slots, row), dtype=torch.uint8, device=DEV)
        step = 1 << 18
        for a in range(0, slots, step):
            k = min(step, slots - a)
            rope = _randn((k, ROPE), g, c["outliers"]) if c["d_qk"] == 576 else None
            cache[a:a + k] = _cache_rows(_randn((k, LATENT), g, c["outliers"]), rope, row)
        order = torch.randperm(total - 1, generator=g, device=DEV).to(torch.int32) + 1
        width = max(pages) + 2
        table = torch.full((len(new), width), -1, dtype=torch.int32, device=DEV)
        first = 0
        for i, k in enumerate(pages):
            table[i, :k] = order[first:first + k]
            first += k
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        s["cache"], s["table"] = cache, table
        s["q"] = _randn((T, H, c["d_qk"]), g)
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(c["d_qk"])
        # where each token stands: its sequence and its place in the chunk
        s["seq"] = torch.tensor([i for i, n in enumerate(new) for _ in range(n)], device=DEV)
        s["place"] = torch.tensor([i for n in new for i in range(n)], device=DEV)
        s["out"] = torch.empty((T, H, LATENT), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device=DEV)
        return s
    page, P = c["page"], c["pages"]
    s["cache"] = torch.randint(0, 127, (P * page, ROW), generator=g, device=DEV, dtype=torch.uint8)
    order = torch.randperm(P - 1, generator=g, device=DEV).to(torch.int32) + 1
    if c["kind"] == "fork":
        lens, parent = _fork_shape(c)
        pages = [-(-L // page) for L in lens]
        width = max(pages) + 3
        rows = c["parents"] + c["forks"]
        table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
        refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        first = 0
        for i, k in enumerate(pages):
            table[i, :k] = order[first:first + k]
            first += k
        refs[order[:first].long()] = 1
        # children of an earlier step: each holds one page of its own and shares nothing
        table[c["parents"]:, 0] = order[first:first + c["forks"]]
        refs[order[first:first + c["forks"]].long()] = 1
        s["table"], s["refs"] = table, refs
        s["parent"] = torch.tensor(parent, dtype=torch.int32, device=DEV)
        s["child"] = torch.arange(c["parents"], rows, dtype=torch.int32, device=DEV)
        s["lens"] = torch.tensor([lens[p] for p in parent], dtype=torch.int32, device=DEV)
        return s
    if c["kind"] == "copy":
        s["into"] = torch.zeros_like(s["cache"])
        s["src"] = order[:c["moved"]].clone()
        s["dst"] = (torch.randperm(P - 1, generator=g, device=DEV).to(torch.int32) + 1)[:c["moved"]].clone()
        return s
    live, _ = _compact_moves(c)
    at = torch.tensor([i for i, v in enumerate(live) if v], dtype=torch.int32, device=DEV)
    at = at[torch.randperm(at.numel(), generator=g, device=DEV)]
    n, S = at.numel(), c["seqs"]
    width = -(-n // S) + 1
    table = torch.full((S * width,), -1, dtype=torch.int32, device=DEV)
    i = torch.arange(n, device=DEV)
    table[(i % S) * width + i // S] = at
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[at.long()] = 1
    s["table"], s["refs"] = table.view(S, width), refs
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(refs)
    s["map"] = torch.empty_like(refs)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _views(cache):
    """A cache as the values it holds: E4M3 codes, tile scales, rotary values."""
    return {"codes": cache[:, :LATENT].view(torch.float8_e4m3fn), "scales": cache[:, 512:528].view(torch.float32),
            "rope": cache[:, 528:].view(torch.bfloat16)}


def _plain_rotate(x, pos, c):
    """x [n, heads, 64] turned by its positions; angles in 64 bits (far positions), products in 32."""
    inv, axis = _frequencies(c)
    ang = pos.double()[axis].t() * torch.tensor(inv, dtype=torch.float64, device=DEV)     # [n, 32]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(torch.bfloat16)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(torch.bfloat16)


def _plain_write(s):
    c = s["case"]
    s["q"][..., LATENT:] = _plain_rotate(s["q_proj"][..., 128:], s["pos"], c)
    k = _plain_rotate(s["k_pe"][:, None], s["pos"], c)[:, 0]
    rows = _cache_rows(s["latent"], k, ROW)
    # a padding row writes back what the reserved slot holds
    keep = (s["slots"] > 0)[:, None]
    s["cache"][s["slots"]] = torch.where(keep, rows, s["cache"][s["slots"]])
    return {"q": s["q"], **_views(s["cache"])}


def _plain_chunk(s):
    c = s["case"]
    table, kv_len, page = s["table"].long(), s["kv_len"].long(), c["page"]
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    longest, H = max(_chunk_shape(c)[1]), c["heads"]
    at = torch.arange(longest, device=DEV)
    pg = table[:, at // page]
    slot = pg * page + at % page
    present = (pg >= 0) & (slot > 0) & (slot < s["cache"].shape[0]) & (at < kv_len[:, None])
    rows = s["cache"][torch.where(present, slot, torch.zeros_like(slot))]
    k = rows[..., :LATENT].view(torch.float8_e4m3fn).float().unflatten(-1, (4, TILE))
    k = (k * rows[..., 512:528].contiguous().view(torch.float32)[..., None]).flatten(-2)
    if c["d_qk"] == 576:
        k = torch.cat([k, rows[..., 528:].contiguous().view(torch.bfloat16).float()], -1)
    k = torch.where(present[..., None], k, torch.zeros_like(k))
    q = torch.zeros((len(new), max(_chunk_shape(c)[0]), H, c["d_qk"]), device=DEV)
    q[s["seq"], s["place"]] = s["q"].float()
    sc = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).unflatten(1, (-1, H)) * s["scale"]
    place = torch.arange(q.shape[1], device=DEV)
    last = (kv_len - new)[:, None] + place if c["causal"] else (kv_len - 1)[:, None].expand(-1, q.shape[1])
    seen = present[:, None] & (at <= last[..., None])
    sc = torch.where(seen[:, :, None], sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (sc - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(1, 2), k[..., :LATENT]).unflatten(1, (-1, H))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    return {"out": o[s["seq"], s["place"]].to(torch.bfloat16), "lse": lse[s["seq"], s["place"]]}


def _plain_fork(s):
    c, table, refs, page = s["case"], s["table"], s["refs"], s["case"]["page"]
    child, parent, lens = s["child"].long(), s["parent"].long(), s["lens"].long()
    # the children of the step before let go of their pages
    old = table[child]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).int().flatten())
    # whole pages are shared; a last page that is not full gets a page of its own, the lowest free ones in order
    col = torch.arange(table.shape[1], device=DEV)
    whole, rest = lens // page, lens % page
    got = torch.where(col < whole[:, None], table[parent], torch.full_like(table[parent], -1))
    refs.index_add_(0, got.clamp(min=0).flatten().long(), (got >= 0).int().flatten())
    empty = refs == 0
    empty[0] = False
    vacant = torch.argsort((~empty).int(), stable=True)
    needs = rest > 0
    fresh = vacant[(needs.int().cumsum(0) - 1).clamp(min=0)]
    table[child] = torch.where((col == whole[:, None]) & needs[:, None], fresh[:, None].int(), got)
    refs.index_add_(0, torch.where(needs, fresh, torch.zeros_like(fresh)), needs.int())
    pages = s["cache"].view(c["pages"], page, ROW)
    had = table[parent, whole.clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    part = (torch.arange(page, device=DEV) < rest[:, None])[..., None]
    to = torch.where(needs, fresh, torch.zeros_like(fresh))
    pages[to] = torch.where(part, pages[had], pages[to])
    return {"table": table, "refs": refs, "cache": s["cache"]}


def _plain_copy(s):
    c = s["case"]
    s["into"].view(c["pages"], c["page"], ROW)[s["dst"].long()] = s["cache"].view(c["pages"], c["page"], ROW)[s["src"].long()]
    return {"cache": s["into"]}


def _plain_compact(s):
    c, refs, table = s["case"], s["refs"], s["table"]
    live = refs > 0
    live[0] = False
    n = live.sum()
    at = torch.arange(c["pages"], device=DEV)
    high = (live & (at > n)).nonzero()[:, 0]
    low = (~live & (at <= n) & (at > 0)).nonzero()[:, 0]
    to = torch.where(live | (at == 0), at, torch.full_like(at, -1))
    to[high] = low
    new = refs.clone()
    new[low] = refs[high]
    new[high] = 0
    pages = s["cache"].view(c["pages"], c["page"], ROW)
    pages[low] = pages[high]
    s["refs_out"].copy_(new)
    s["map"].copy_(to)
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["map"], "cache": s["cache"]}


def _own_run(s):
    from fp8_mla_kv_gb300 import mlasparse as M
    c = s["case"]
    if c["kind"] == "write":
        if "rope" not in s:
            inv, axis = _frequencies(c)
            s["rope"] = M.rope_spec(inv, axis, interleaved=c["interleaved"])
        M.mla_rope_kv_write(s["cache"], s["slots"], s["latent"], s["k_pe"], s["pos"], s["rope"],
                            q_pe=s["q_proj"][..., 128:], q_out=s["q"][..., LATENT:])
        return {"q": s["q"], **_views(s["cache"])}
    if c["kind"] == "chunk":
        if "ws" not in s:
            s["ws"] = M.alloc_chunk_workspace(s["q"].shape[0], c["heads"], c["seqs"])
        M.mla_chunk_attention(s["q"], s["cache"], s["q_start"], s["kv_len"], s["table"], c["page"], s["scale"],
                              causal=c["causal"], out=s["out"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "fork":
        if "ws" not in s:
            s["ws"] = M.alloc_page_workspace(c["pages"], c["forks"])
        M.mla_page_free(s["refs"], s["table"], s["child"])
        M.mla_page_fork(s["cache"], c["page"], s["refs"], s["table"], s["parent"], s["child"], s["lens"],
                        workspace=s["ws"])
        return {"table": s["table"], "refs": s["refs"], "cache": s["cache"]}
    if c["kind"] == "copy":
        M.mla_page_copy(s["into"], s["cache"], c["page"], s["dst"], s["src"])
        return {"cache": s["into"]}
    if "ws" not in s:
        s["ws"] = M.alloc_page_workspace(c["pages"], 0)
    M.mla_page_compact(s["cache"], c["page"], s["refs"], s["table"], refcount_out=s["refs_out"],
                       table_out=s["table_out"], page_map=s["map"], workspace=s["ws"])
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["map"], "cache": s["cache"]}


def run(state):
    if own:
        return _own_run(state)
    return {"write": _plain_write, "chunk": _plain_chunk, "fork": _plain_fork, "copy": _plain_copy,
            "compact": _plain_compact}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_code(v):
    """The E4M3 value nearest to each v (ties to even), |v| at most 448: steps of 2^(e-3), of 2^-9 below 2^-6."""
    e = torch.frexp(v)[1].double() - 1.0
    step = torch.pow(2.0, e.clamp(min=-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_rotate(x, pos, c):
    inv, axis = _frequencies(c)
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for i in range(32):
        ang = pos[axis[i]].double() * inv[i]
        lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + 32)
        a, b = x[..., lo].double(), x[..., hi].double()
        co, si = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        out[..., lo] = a * co - b * si
        out[..., hi] = b * co + a * si
    return out


def exact(case, seed):
    c = case
    if c["kind"] in ("fork", "copy", "compact"):
        return None                                   # whole numbers only
    if c["kind"] == "chunk" and 2.0 * _attended(c) * c["heads"] * (c["d_qk"] + LATENT) > 1.0e13:
        return None
    s = prepare(c, seed)
    if c["kind"] == "write":
        q = s["q"].double()
        q[..., LATENT:] = _exact_rotate(s["q_proj"][..., 128:], s["pos"], c)
        codes = torch.zeros((c["slots"], LATENT), dtype=torch.float64, device=DEV)
        scales = torch.zeros((c["slots"], 4), dtype=torch.float64, device=DEV)
        rope = torch.zeros((c["slots"], ROPE), dtype=torch.float64, device=DEV)
        kept = s["slots"] != 0
        x = s["latent"][kept].double().reshape(-1, 4, TILE)
        sc = x.abs().max(-1).values / 448.0
        sc = torch.where(sc > 0, sc, torch.ones_like(sc))
        slots = s["slots"][kept]
        # by definition the scale is held in 32 bits, and so is the quotient that is rounded to a code
        codes[slots] = _exact_code((x / sc.float().double()[..., None]).float().double()).reshape(-1, LATENT)
        scales[slots] = sc
        rope[slots] = _exact_rotate(s["k_pe"][:, None], s["pos"], c)[:, 0][kept]
        return {"q": q, "codes": codes, "scales": scales, "rope": rope}
    new, ctx = _chunk_shape(c)
    T, H, page = sum(new), c["heads"], c["page"]
    out = torch.zeros((T, H, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for i, (n, L) in enumerate(zip(new, ctx)):
        p = torch.arange(L, device=DEV)
        slot = s["table"][i, p // page].long() * page + p % page
        rows = s["cache"][slot]
        k = rows[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double()
        sc = rows[:, 512:528].contiguous().view(torch.float32).double()
        k = k * sc.repeat_interleave(TILE, 1)
        key = torch.cat([k, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1) if c["d_qk"] == 576 else k
        q = s["q"][first:first + n].double().reshape(n * H, c["d_qk"])
        a = (q @ key.t()).reshape(n, H, L) * s["scale"]
        if c["causal"]:
            own_place = L - n + torch.arange(n, device=DEV)
            a.masked_fill_((p > own_place[:, None])[:, None], -math.inf)
        b = torch.logsumexp(a, -1)
        w = torch.where(b[..., None] == -math.inf, torch.zeros_like(a), torch.exp(a - b[..., None]))
        out[first:first + n] = (w.reshape(n * H, L) @ k).reshape(n, H, LATENT)
        lse[first:first + n] = b
        first += n
    return {"out": out, "lse": lse}
