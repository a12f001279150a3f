"""Drafted trees (mla_tree_mask, _attention, _commit) against plain forms."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P
import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"


def dev(b):
    return {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}


def some_parents(b, reach, seed=0):
    g = torch.Generator().manual_seed(seed + 31)
    parent = torch.full((b["T"],), -1, dtype=torch.int32)
    for t, _, i, _ in B.tokens(b):
        lo = max(-1, i - reach)
        parent[t] = int(torch.randint(lo, i, (1,), generator=g)) if i > lo else -1
    return parent


SEQS = [(1, 1), (0, 9), (31, 60), (33, 33), (1, 300), (64, 500), (65, 66), (200, 333), (7, 3)]


# ---- mask ----

@pytest.mark.parametrize("reach", [1, 3, 1000])
@pytest.mark.parametrize("words", [0, 1, 2, 7, 9])
def test_mask(words, reach):
    b = B.batch(SEQS, 1, 512, 16, 528, seed=words, tail_tokens=2, head_tokens=1)
    parent = some_parents(b, reach, words)
    parent[parent == -1] = torch.randint(-5, 0, (int((parent == -1).sum()),), dtype=torch.int32)     # any negative one
    up = B.ancestors(b, parent)
    mask = torch.full((b["T"], words), 77, dtype=torch.int32, device=D)
    pos = torch.full((b["T"],), 55, dtype=torch.int32, device=D)
    M.mla_tree_mask(parent.to(D), b["q_start"].to(D), b["kv_len"].to(D), mask=mask, positions=pos)
    assert M.mla_get_error() == (M.MLA_ERR_CHUNK_RANGE if 0 < words < 7 else 0)
    want = B.mask_bits(up, b["T"], words)
    inside = [t for t, _, _, _ in B.tokens(b)]
    outside = [t for t in range(b["T"]) if t not in set(inside)]
    assert torch.equal(mask.cpu()[inside], want[inside]) and (mask.cpu()[outside] == 77).all()
    for t, s, i, p in B.tokens(b):
        assert int(pos[t]) == p - i + len(up[t]) - 1
    assert (pos.cpu()[outside] == 55).all()


def test_mask_of_parents_out_of_order():
    b = B.batch([(10, 20), (5, 9)], 1, 512, 16, 528, seed=3)
    parent = some_parents(b, 4, 3)
    parent[4], parent[6], parent[12] = 4, 9, 100        # itself, a later one, none of the tokens
    mask, pos = M.mla_tree_mask(parent.to(D), b["q_start"].to(D), b["kv_len"].to(D), words=1)
    assert M.mla_get_error() == M.MLA_ERR_CHUNK_RANGE
    up = B.ancestors(b, parent)
    assert torch.equal(mask.cpu(), B.mask_bits(up, 15, 1))


def test_mask_of_many_sequences():
    b = B.batch([(i % 7, 50) for i in range(700)], 1, 512, 64, 528, seed=5)
    parent = some_parents(b, 3)
    mask, _ = M.mla_tree_mask(parent.to(D), b["q_start"].to(D), b["kv_len"].to(D), words=1)
    assert M.mla_get_error() == 0 and torch.equal(mask.cpu(), B.mask_bits(B.ancestors(b, parent), b["T"], 1))


# ---- attention ----

def check(b, rows, words, error=0):
    """rows[t]: the drafted tokens that token t's bits name."""
    t = dev(b)
    H = b["q"].shape[1]
    out = torch.full((b["T"], H, 512), 3.0, dtype=torch.bfloat16, device=D)
    lse = torch.full((b["T"], H), 5.0, device=D)
    M.mla_tree_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], b["page"], b["scale"],
                         B.mask_bits(rows, b["T"], words).to(D), out=out, lse=lse)
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    ref = B.attend(b, B.tree_positions(b, [[j for j in r if j < 32 * words] for r in rows]))
    P.check_chunk(out, lse, ref)
    outside = torch.isnan(ref[2][..., 0])
    assert (out.cpu()[outside] == 3.0).all() and (lse.cpu()[outside] == 5.0).all()
    return out, lse


# a table much wider than the contexts sends batches of 36 rows a sequence and more to the kernel for many rows
def wide(T, H, page, many):
    return 8_000_000 // (T * H * page) + 2 if many else 2


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("H,d_qk,row,page", [(16, 576, 656, 64), (5, 512, 528, 16), (128, 576, 656, 48)])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(3, 40), (1, 33)], [(31, 31), (31, 500), (20, 129)], [(60, 700)], [(33, 20), (7, 90)]],
                         ids=str)
def test_attention(seqs, H, d_qk, row, page, many):
    n = sum(x for x, _ in seqs)
    b = B.batch(seqs, H, d_qk, page, row, seed=H + n, extra=wide(n, H, page, many), tail_tokens=2)
    up = B.ancestors(b, some_parents(b, 6, n))
    check(b, up, 2)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("H", [1, 2, 3, 7, 16, 31, 64, 100])
def test_attention_heads(H, many):
    b = B.batch([(37, 150), (40, 40), (64, 90)], H, 576, 32, 656, seed=H, extra=wide(141, H, 32, many))
    check(b, B.ancestors(b, some_parents(b, 20, H)), 2)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("n_seq", [1, 9, 31, 32, 33])
def test_attention_split_tiles_of_unlike_lengths(n_seq, many):
    """Contexts that are cut into pieces, of one to two waves and more; a sequence without tokens, one without positions."""
    g = torch.Generator().manual_seed(n_seq)
    seqs = [(int(torch.randint(1, 13, (1,), generator=g)), int(torch.randint(14, 2600, (1,), generator=g))) for _ in range(n_seq)]
    if n_seq > 8:
        seqs[3], seqs[7] = (0, 50), (2, 0)
    T = sum(n for n, _ in seqs)
    b = B.batch(seqs, 16, 512, 16, 528, seed=n_seq, extra=wide(T, 16, 16, many))
    check(b, B.ancestors(b, some_parents(b, 4, n_seq)), 1)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("page", [1, 31, 128])
def test_attention_pages_that_end_inside_a_tile(page, many):
    b = B.batch([(35, 333), (32, 70), (12, 64)], 16, 512, page, 528, seed=page, extra=wide(79, 16, page, many))
    check(b, B.ancestors(b, some_parents(b, 5, page)), 2)


@pytest.mark.parametrize("many", [False, True])
def test_attention_by_any_mask(many):
    """Bits of later tokens, rows without any, more tokens than the mask has bits, tokens before the first position."""
    b = B.batch([(70, 300), (20, 20), (40, 25), (3, 0)], 16, 576, 16, 656, seed=6, extra=wide(133, 16, 16, many))
    g = torch.Generator().manual_seed(2)
    rows = [torch.randperm(75, generator=g)[:int(torch.randint(0, 30, (1,), generator=g))].tolist() for _ in range(b["T"])]
    rows[71] = rows[5] = []
    check(b, rows, 1)
    check(b, rows, 3)
    check(b, rows, 0)


@pytest.mark.parametrize("many", [False, True])
def test_attention_a_chain_is_chunk_attention(many):
    b = B.batch([(33, 200), (40, 40)], 16, 576, 16, 656, seed=7, extra=wide(73, 16, 16, many))
    check(b, [list(range(i + 1)) for _, _, i, _ in B.tokens(b)], 2)
    t = dev(b)
    mask = B.mask_bits([list(range(i + 1)) for _, _, i, _ in B.tokens(b)], b["T"], 2).to(D)
    out, lse = M.mla_tree_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 16, b["scale"], mask)
    P.check_chunk(out, lse, P.chunk(b["q"], b["cache"], b["q_start"], b["kv_len"], b["table"], 16, b["scale"]))


@pytest.mark.parametrize("many", [False, True])
def test_attention_holes_and_rows_that_are_not_finite(many):
    b = B.batch([(40, 200), (40, 100)], 16, 576, 16, 656, seed=8, extra=wide(80, 16, 16, many))
    b["table"][0, 3] = -1
    b["table"][1, 5] = 0
    b["cache"][0] = 0xFF
    # a drafted token of the first sequence is NaN: its descendants' outputs and no others
    slot = int(b["table"][0, 170 // 16]) * 16 + 170 % 16
    b["cache"][slot, 3] = 0x7F
    parent = some_parents(b, 3, 1)
    up = B.ancestors(b, parent)
    assert sum(10 in r for r in up[:40]) not in (0, 40)
    check(b, up, 2)
    b["table"][0, 2] = 1 << 26
    check(b, up, 2, error=M.MLA_ERR_DECODE_INDEX_RANGE)


def test_attention_lengths_past_the_table():
    # (the last 6 positions are past the table: absent)
    b = B.batch([(20, 64)], 16, 576, 16, 656, seed=9, extra=0)
    b["kv_len"][0] = 70
    check(b, B.ancestors(b, some_parents(b, 4)), 1, error=M.MLA_ERR_CHUNK_RANGE)


# ---- commit ----

def commit(b, paths, max_path=None, error=0, alias=False):
    """paths: what is asked. Returns nothing; checks every byte of the cache and the lengths."""
    S, page = len(b["kv_len"]), b["page"]
    max_path = max([len(p) for p in paths] + [1]) if max_path is None else max_path
    path = torch.zeros((S, max_path), dtype=torch.int32)
    for s, p in enumerate(paths):
        path[s, :min(len(p), max_path)] = torch.tensor(p[:max_path], dtype=torch.int32)
    t = dev(b)
    cache, lens = t["cache"].clone(), t["kv_len"].clone()
    out = lens if alias else torch.full((S,), -3, dtype=torch.int32, device=D)
    M.mla_tree_commit(cache, t["q_start"], lens, t["table"], page, path.to(D),
                      torch.tensor([len(p) for p in paths], dtype=torch.int32, device=D), kv_len_out=out)
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    want, old = b["cache"].clone(), b["cache"]
    for s, p in enumerate(paths):
        n, L = int(b["q_start"][s + 1] - b["q_start"][s]), int(b["kv_len"][s])
        if L < n or L > b["table"].shape[1] * page:
            assert int(out[s]) == L
            continue
        good = []
        for x in p[:max_path]:
            if not 0 <= x < n or (good and x <= good[-1]):
                break
            good.append(x)

        def slot(pos):
            phys = int(b["table"][s, pos // page])
            at = phys * page + pos % page
            return at if phys >= 0 and 0 < at < old.shape[0] else None

        for j, x in enumerate(good):
            a, c = slot(L - n + x), slot(L - n + j)
            if x != j and a is not None and c is not None:
                want[c] = old[a]
        assert int(out[s]) == L - n + len(good)
    assert torch.equal(cache.cpu(), want)


@pytest.mark.parametrize("page,row", [(16, 656), (64, 528), (1, 656), (33, 656)])
def test_commit(page, row):
    b = B.batch([(n, max(n, L)) for n, L in SEQS], 1, 512, page, row, seed=page)
    g = torch.Generator().manual_seed(page)
    for most in (0, 1, 5, 8, 9, 200):
        paths = [sorted(torch.randperm(n, generator=g)[:int(torch.randint(0, min(n, most) + 1, (1,), generator=g))].tolist())
                 for n, _ in SEQS]
        commit(b, paths, alias=most == 5)
    commit(b, [list(range(n)) for n, _ in SEQS])         # everything accepted: nothing moves
    commit(b, [list(range(n - n // 2, n)) for n, _ in SEQS])      # each row moves to where another one was


def test_commit_paths_out_of_order():
    b = B.batch([(10, 40), (10, 40), (10, 40), (10, 40), (5, 5)], 1, 512, 16, 656, seed=1)
    commit(b, [[1, 3, 3, 5], [2, 10], [4, 2], [-1, 2], [1, 2]], error=M.MLA_ERR_CHUNK_RANGE)
    commit(b, [[1, 3, 5], [2, 4, 6, 8], [], [0], [1]], max_path=3, error=M.MLA_ERR_CHUNK_RANGE)


def test_commit_lengths_and_pages_out_of_range():
    b = B.batch([(10, 40), (10, 8), (10, 48)], 1, 512, 16, 656, seed=2, extra=0)
    b["kv_len"][2] = 60
    commit(b, [[1, 3, 5], [1, 2], [3]], error=M.MLA_ERR_CHUNK_RANGE)
    b = B.batch([(20, 40), (20, 40)], 1, 512, 16, 656, seed=2, extra=0)
    b["table"][0, 1] = -1
    b["table"][1, 2] = 1 << 27
    commit(b, [[1, 15, 19], [2, 15, 19]], error=M.MLA_ERR_PAGE_RANGE)
    b["table"][1, 2] = 0                                 # holds the reserved slot
    b["table"][0, 1] = 3
    commit(b, [[1], [2, 12, 19]], error=M.MLA_ERR_PAGE_RANGE)


def test_commit_without_lengths_out():
    b = dev(B.batch([(4, 9)], 1, 512, 16, 656, seed=3))
    M.mla_tree_commit(b["cache"], b["q_start"], b["kv_len"], b["table"], 16, torch.tensor([[2]], dtype=torch.int32, device=D),
                      torch.tensor([1], dtype=torch.int32, device=D))
    assert M.mla_get_error() == 0 and int(b["kv_len"][0]) == 9
    page = int(b["table"][0, 0]) * 16
    assert torch.equal(b["cache"][page + 5], b["cache"][page + 7])
