"""mla_chunk_attention at the ends of its ranges: small queries, scales far apart, contexts near 2^31 positions. Every
case for few query rows (one token a sequence) and for many."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"
MANY = 8_000_000                     # pairs of query rows and positions that are many for the choice of the kernel


def batch(seqs, H, d_qk, page, row, seed):
    """seqs: (new tokens, context length). Random pages, a table wide enough for the kernel for many rows where the
    rows are many."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-L // page) for _, L in seqs]
    cache = P.make_cache((sum(pages) + 2) * page, row, g, rope=d_qk == 576)
    order = torch.randperm(sum(pages) + 1, generator=g).to(torch.int32) + 1
    T = sum(n for n, _ in seqs)
    width = max(pages) + 2
    if T * H >= 64 * len(seqs):
        width = max(width, MANY // (T * H * page) + 1)
    table = torch.full((len(seqs), width), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(pages):
        table[i, :k] = order[at:at + k]
        at += k
    start = torch.tensor([0] + [n for n, _ in seqs], dtype=torch.int32).cumsum(0).to(torch.int32)
    return dict(q=torch.randn((T, H, d_qk), generator=g).to(torch.bfloat16), cache=cache, q_start=start,
                kv_len=torch.tensor([L for _, L in seqs], dtype=torch.int32), table=table, page=page,
                scale=1.0 / math.sqrt(d_qk))


def call(b, causal=True):
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    out, lse = M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], t["page"], t["scale"],
                                     causal=causal)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    return out, lse


def ref(b, causal=True):
    return P.chunk(b["q"], b["cache"], b["q_start"], b["kv_len"], b["table"], b["page"], b["scale"], causal)


def run(b, causal=True):
    P.check_chunk(*call(b, causal), ref(b, causal))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 528)])
@pytest.mark.parametrize("log2", [-10, -14, -20, -24, -40, -90])
def test_small_query_rows(n, d_qk, row, log2):
    """Every query row small, and a softmax scale that makes its scores as large as usual."""
    b = batch([(n, 300), (n, 77)], 16, d_qk, 16, row, seed=1)
    b["q"] = (b["q"].double() * 2.0 ** log2).to(torch.bfloat16)
    b["scale"] = 2.0 ** -log2 / 24
    run(b)


@pytest.mark.parametrize("n", [1, 40])
def test_rows_of_equal_scores_at_any_size(n):
    """Powers of two that q and the softmax scale give and take change nothing, bit for bit."""
    b = batch([(n, 300)], 16, 576, 16, 656, seed=2)
    # (f16's range holds these values exactly at every one of the sizes)
    b["q"] = torch.where(b["q"].abs() < 2.0 ** -9, torch.zeros_like(b["q"]), b["q"])
    want = call(b)
    q, scale = b["q"], b["scale"]
    for log2 in (-60, -24, -8, 3, 20):
        b["q"], b["scale"] = (q.double() * 2.0 ** log2).to(torch.bfloat16), scale * 2.0 ** -log2
        out, lse = call(b)
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


@pytest.mark.parametrize("n", [1, 4])                   # 16 and 64 query rows: both kernels
@pytest.mark.parametrize("less", [0, 1000])
def test_contexts_near_2_to_31_positions(n, less):
    """A table of nothing but a few pages, at the context's start, within it and at its end, where the end of the last
    piece, rounded up to whole blocks, passes 2^31."""
    page = 4093
    g = torch.Generator().manual_seed(3)
    cache = P.make_cache(6 * page, 656, g)
    width = ((1 << 31) - 4097) // page
    L = width * page - less
    table = torch.full((1, width), -1, dtype=torch.int32)
    at = [0, width // 3, width - 700, width - 2, width - 1]
    for i, k in enumerate(at):
        table[0, k] = i + 1
    q = torch.randn((n, 16, 576), generator=g).to(torch.bfloat16)
    out, lse = M.mla_chunk_attention(q.to(D), cache.to(D), torch.tensor([0, n], dtype=torch.int32, device=D),
                                     torch.tensor([L], dtype=torch.int32, device=D), table.to(D), page, 1 / 24)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    # the formula over the positions that are there, as a context of their own
    pos = torch.cat([torch.arange(k * page, (k + 1) * page) for k in at])
    slot = torch.arange(page, 6 * page)[pos < L]
    rows = torch.cat([cache[:1], cache[slot]])
    P.check_chunk(out, lse, P.chunk(q, rows, torch.tensor([0, n]), torch.tensor([len(slot)]),
                                    torch.arange(1, len(slot) + 1, dtype=torch.int32)[None], 1, 1 / 24))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("some", [False, True])
def test_negative_scales(n, some):
    """A scale's sign is the values' (the writer makes none; a cache from elsewhere may): all negative, or every third
    and those eight times as large."""
    b = batch([(n, 300), (n, 33)], 16, 576, 16, 656, seed=4)
    sc = b["cache"][:, 512:528].contiguous().view(torch.float32)
    sign = torch.where((torch.arange(sc.numel()) % 3 == 0) | (not some), -8.0 if some else -1.0, 1.0).view(sc.shape)
    b["cache"][:, 512:528] = (sc * sign).contiguous().view(torch.uint8)
    run(b)


def rows_of(lat, rope):
    """Cache rows as the writer makes them (a tile of zeros has the scale 1)."""
    t = lat.to(torch.bfloat16).float().view(-1, 4, 128)
    amax = t.abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (t / sc[..., None]).to(torch.float8_e4m3fn).view(-1, 512).view(torch.uint8)
    return torch.cat([codes, sc.contiguous().view(torch.uint8), rope.to(torch.bfloat16).view(torch.uint8)], 1)


def held_to(n_keys, scale):
    """What values lose beside a tile scale: their own scale is off by at most 2^-25 of the larger one, codes are at
    most 448, and few rows' P (at least 16 at the largest score) times the ratio is held to 2^-25 too, per position."""
    return (1 + n_keys / 16) * 449 * 2.0 ** -25 * scale


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("which", ["first", "middle", "last", "tiles"])
@pytest.mark.parametrize("log2", [0, -6, -12])
def test_rows_of_zeros_beside_small_values(n, which, log2):
    """Tiles of zeros have the scale 1."""
    L = 200
    b = batch([(n, L)], 16, 576, 1, 656, seed=5)
    g = torch.Generator().manual_seed(5)
    lat = torch.randn((L, 512), generator=g) * 2.0 ** log2
    if which == "first":
        lat[:70] = 0
    elif which == "middle":
        lat[100] = 0
        lat[133:136] = -0.0
    elif which == "last":
        lat[-1] = 0
    else:
        lat.view(L, 4, 128)[torch.rand((L, 4), generator=g) < 0.1] = 0
    b["cache"][b["table"][0, :L].long()] = rows_of(lat, torch.randn((L, 64), generator=g))
    out, lse = call(b)
    ro, rl, to, tl = ref(b)
    P.check_chunk(out, lse, (ro, rl, to + held_to(L, 1.0), tl))


@pytest.mark.parametrize("n,H", [(3, 5), (40, 16)])
@pytest.mark.parametrize("log2", [6, 12, 20])
def test_a_large_scale_in_the_last_token_only(n, H, log2):
    """The tokens before it do not attend its row, but share a tile with it."""
    b = batch([(n, 100)], H, 576, 16, 656, seed=6)
    slot = int(b["table"][0, 99 // 16]) * 16 + 99 % 16
    sc = b["cache"][slot, 512:528].view(torch.float32) * 2.0 ** log2
    b["cache"][slot, 512:528] = sc.view(torch.uint8)
    b["q"] = b["q"] * 2.0 ** -10                        # the last token's own score stays within reach
    out, lse = call(b)
    ro, rl, to, tl = ref(b)
    P.check_chunk(out, lse, (ro, rl, to + held_to(100, sc.double().repeat_interleave(128)), tl))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("which", ["first", "middle", "last", "tiles", "most"])
@pytest.mark.parametrize("log2", [-6, -24])
def test_rows_of_zeros_take_no_bits(n, which, log2):
    """Tiles of zeros do not count, whatever the others' size; rows whose scale is 1 because their largest value is 448
    count like any."""
    L = 500
    b = batch([(n, L)], 16, 576, 1, 656, seed=5)
    g = torch.Generator().manual_seed(5)
    lat = torch.randn((L, 512), generator=g) * 2.0 ** log2
    if which == "first":
        lat[:150] = 0
    elif which == "middle":
        lat[200] = 0
        lat[401:404] = -0.0
    elif which == "last":
        lat[-1] = 0
    elif which == "tiles":
        lat.view(L, 4, 128)[torch.rand((L, 4), generator=g) < 0.1] = 0
    else:
        lat[torch.rand(L, generator=g) < 0.97] = 0
    b["cache"][b["table"][0, :L].long()] = rows_of(lat, torch.randn((L, 64), generator=g))
    run(b)
    # a row that is not zeros but has the scale 1 in one tile: a value of 448
    lat[:, 128:256] = lat[:, 128:256].sign() * 0.25
    lat[77, 200] = 448.0
    b["cache"][b["table"][0, :L].long()] = rows_of(lat, torch.randn((L, 64), generator=g))
    assert b["cache"][int(b["table"][0, 77]), 516:520].view(torch.float32) == 1.0
    run(b)


@pytest.mark.parametrize("n,H", [(1, 16), (3, 5), (40, 16)])
@pytest.mark.parametrize("d_qk,row", [(512, 528), (512, 656), (576, 656)])
@pytest.mark.parametrize("where", [(0,), (31, 32, 63), (64, 65, 66, 67), "block", "all"], ids=str)
def test_rows_that_are_not_finite_anywhere(n, H, d_qk, row, where):
    """Several in a block, a whole block of them, nothing else; by codes and by scales of different tiles, beside rows
    of zeros; the second sequence has none."""
    L = 200
    b = batch([(n, L), (n, L)], H, d_qk, 1, row, seed=7)
    at = range(96, 128) if where == "block" else range(L) if where == "all" else where
    cache = b["cache"]
    for i, p in enumerate(at):
        r = int(b["table"][0, p])
        if i % 3 == 0:
            cache[r, (131 * i) % 512] = 0xFF if i % 2 else 0x7F
        elif i % 3 == 1:
            cache[r, 512 + 4 * (i % 4):516 + 4 * (i % 4)] = torch.tensor([math.nan if i % 2 else -math.inf]).view(torch.uint8)
        elif d_qk == 576:
            cache[r, 528 + 2 * (i % 64):530 + 2 * (i % 64)] = torch.tensor([math.inf], dtype=torch.bfloat16).view(torch.uint8)
        else:
            cache[r, 511] = 0x7F
    for p in (5, 97, 150):
        if p not in at:
            r = int(b["table"][0, p])
            cache[r, :512], cache[r, 512:528] = 0, torch.ones(4).view(torch.uint8)
    run(b)
    b["kv_len"][0] = 160
    run(b)
