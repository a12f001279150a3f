"""Block-sparse attention (mla_block_keys, _scores, _select, _attention) against the formulas in 64 bits."""
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


def where(t):
    return t["q_start"], t["kv_len"], t["table"], t["page"]


# ---- mean keys ----

def check_keys(b, d_qk, num_keys=None, error=0):
    t = dev(b)
    num_keys = b["pages"] if num_keys is None else num_keys
    keys = torch.full((num_keys, d_qk), 7.0, dtype=torch.bfloat16, device=D)
    M.mla_block_keys(t["cache"], *where(t), keys, b["T"])
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    got, want = keys.double().cpu(), B.mean_keys(b, d_qk, num_keys)
    for p in range(num_keys):
        if p not in want:
            assert (got[p] == 7.0).all(), f"page {p} was not completed"
            continue
        m, tol = want[p]
        fine = torch.isfinite(m)
        assert torch.equal(fine, torch.isfinite(got[p])) and torch.equal(m.isnan(), got[p].isnan())
        assert ((got[p] - m).abs()[fine] <= tol[fine]).all()
    return keys


@pytest.mark.parametrize("page", [1, 2, 7, 16, 33, 64, 500])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 656), (512, 528)])
def test_keys(page, d_qk, row):
    check_keys(B.batch([(1, 64), (1, 63), (5, 5), (0, 128), (130, 700), (64, 1000), (1, 1), (1000, 1000)], 1, d_qk, page, row,
                       seed=page, tail_tokens=3, head_tokens=2), d_qk)


def test_keys_of_many_sequences():
    check_keys(B.batch([(1 + i % 3, 1 + i) for i in range(600)], 1, 576, 16, 656, seed=1), 576)


@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 528)])
def test_keys_of_many_pages(d_qk, row):
    """More than a GPU's worth: several pages a CTA."""
    b = B.batch([(9, 20), (2900, 2900), (0, 40), (2500, 2600), (1, 7)], 1, d_qk, 1, row, seed=6)
    b["table"][1, 17] = -1
    check_keys(b, d_qk)


def test_keys_page_0_holes_and_pages_out_of_range():
    b = B.batch([(200, 200), (100, 250)], 1, 576, 16, 656, seed=2)
    b["table"][0, 3] = 0                                # the reserved slot is no row
    b["cache"][0] = 0xFF
    b["table"][0, 5] = -1
    check_keys(b, 576)
    b["table"][1, 12] = b["pages"] + 5                  # no key there
    check_keys(b, 576, error=M.MLA_ERR_PAGE_RANGE)
    b["table"][1, 12] = 1
    check_keys(b, 576, num_keys=b["pages"] - 4, error=M.MLA_ERR_PAGE_RANGE)
    b = B.batch([(32, 32)], 1, 512, 16, 528, seed=3)
    b["cache"] = b["cache"][:int(b["table"][0, 1]) * 16 + 5]    # a page that ends past the cache, or pages past it
    check_keys(b, 512, error=M.MLA_ERR_PAGE_RANGE)


def test_keys_more_tokens_than_positions_and_lengths_past_the_table():
    b = B.batch([(40, 33), (3, 0), (20, 64)], 1, 576, 16, 656, seed=4, extra=0)
    b["kv_len"][1] = -5
    check_keys(b, 576)
    b["kv_len"][2] = 100
    check_keys(b, 576, error=M.MLA_ERR_CHUNK_RANGE)


def test_keys_of_rows_that_are_not_finite():
    b = B.batch([(64, 64)], 1, 576, 16, 656, seed=5)
    slot = int(b["table"][0, 2]) * 16 + 3
    b["cache"][slot, 17] = 0x7F                          # a NaN code
    b["cache"][slot + 1, 530:532] = torch.tensor([0x80, 0x7F], dtype=torch.uint8)     # an infinite RoPE value
    check_keys(b, 576)


# ---- scores ----

def check_scores(b, keys, error=0):
    t = dev(b)
    scores = torch.full((b["T"], b["table"].shape[1]), 5.0, device=D)
    M.mla_block_scores(t["q"], keys.to(D), *where(t), b["scale"], scores=scores)
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    want, tol = B.block_scores(b, keys)
    got, written = scores.double().cpu(), ~tol.isnan()
    assert (got[~written] == 5.0).all(), "columns that are no block before the token's own"
    gone = written & torch.isneginf(want)
    assert torch.isneginf(got[gone]).all()
    ok = written & ~gone
    off = ((got - want).abs() / tol)[ok]
    if off.numel():
        assert off.max() <= 1, f"off by {off.max():.3g} of the tolerance"
    return scores


def some_keys(b, d_qk, seed=0):
    g = torch.Generator().manual_seed(seed + 99)
    return torch.randn((b["pages"], d_qk), generator=g).to(torch.bfloat16)


SCORE_SHAPES = [[(1, 1)], [(1, 64)], [(1, 65)], [(1, 700), (1, 3)], [(3, 5000)], [(9, 9)], [(40, 300), (0, 90), (7, 1000)],
                [(130, 400), (1, 1), (33, 33), (65, 129)]]


@pytest.mark.parametrize("seqs", SCORE_SHAPES, ids=str)
@pytest.mark.parametrize("H,d_qk,page", [(16, 576, 16), (128, 512, 64), (5, 576, 1)])
def test_scores(seqs, H, d_qk, page):
    b = B.batch(seqs, H, d_qk, page, 656, seed=H + len(seqs), tail_tokens=2, head_tokens=1)
    check_scores(b, some_keys(b, d_qk))


@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 31, 32, 33, 63, 64, 65, 96, 100, 127, 128])
def test_scores_heads(H):
    b = B.batch([(70, 333), (1, 90), (5, 41), (1, 1500)], H, 576, 16, 656, seed=H)
    check_scores(b, some_keys(b, 576))


@pytest.mark.parametrize("d_qk", [512, 576])
def test_scores_of_a_single_row(d_qk):
    b = B.batch([(1, 20)], 1, d_qk, 1, 656, seed=2)     # fewer query rows than a copy takes
    check_scores(b, some_keys(b, d_qk))
    keys = some_keys(b, d_qk)[:1]                       # one key, and blocks past it
    b["table"][0, :19] = 0
    check_scores(b, keys)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("blocks", [127, 128, 129, 255, 257, 511, 512, 513, 1025, 2100, 4097, 5000])
def test_scores_of_many_blocks(blocks, n):
    b = B.batch([(n, blocks + 1), (2, 7)], 4, 512, 1, 528, seed=blocks)
    check_scores(b, some_keys(b, 512))


def test_scores_large_and_small_products():
    b = B.batch([(20, 400)], 16, 576, 16, 656, seed=6)
    keys = some_keys(b, 576)
    b["q"][3] *= 100                                    # one block takes all
    b["q"][4] *= 2.0 ** -60
    b["q"][5] = 0
    keys[int(b["table"][0, 4])] *= 30
    check_scores(b, keys)


def test_scores_holes_and_pages_out_of_range():
    b = B.batch([(30, 400), (2, 200)], 16, 576, 16, 656, seed=7)
    keys = some_keys(b, 576)
    b["table"][0, 3] = b["table"][1, 0] = -1
    b["table"][0, 7] = 0                                # page 0 has a key
    check_scores(b, keys)
    b["table"][0, 20] = b["pages"] + 1
    check_scores(b, keys, error=M.MLA_ERR_PAGE_RANGE)
    b["table"][1, :] = -1                               # nothing there at all
    check_scores(b, keys, error=M.MLA_ERR_PAGE_RANGE)


def test_scores_lengths():
    b = B.batch([(10, 4), (3, 0), (40, 64)], 16, 576, 16, 656, seed=8, extra=0)
    b["kv_len"][1] = -7
    check_scores(b, some_keys(b, 576))
    b["kv_len"][2] = 1000
    check_scores(b, some_keys(b, 576), error=M.MLA_ERR_CHUNK_RANGE)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_scores_a_key_that_is_not_finite_reaches_only_those_who_see_it(value):
    b = B.batch([(40, 400), (1, 100)], 16, 576, 16, 656, seed=9)
    keys = some_keys(b, 576)
    want, tol = B.block_scores(b, keys)
    keys[int(b["table"][0, 23]), 5] = value             # block 23: seen from position 384 on
    t = dev(b)
    got = M.mla_block_scores(t["q"], keys.to(D), *where(t), b["scale"]).double().cpu()
    assert M.mla_get_error() == 0
    for tok, s, _, pos in B.tokens(b):
        if s == 1 or pos < 384:
            n = pos // 16
            assert ((got[tok, :n] - want[tok, :n]).abs() <= tol[tok, :n]).all()


# ---- selection ----

def check_select(b, scores, width, sink, local, error=0):
    t = dev(b)
    blocks = torch.full((b["T"], width), -9, dtype=torch.int32, device=D)
    M.mla_block_select(scores.to(D), t["q_start"], t["kv_len"], b["page"], width, sink=sink, local=local, blocks=blocks)
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    got = blocks.cpu().tolist()
    for row, want in zip(got, B.select(b, scores, width, sink, local)):
        assert row == ([-9] * width if want is None else want)


def some_scores(b, seed=0, ties=False):
    g = torch.Generator().manual_seed(seed + 5)
    sc = torch.randn((b["T"], b["table"].shape[1]), generator=g)
    return (sc * 4).round() / 4 if ties else sc


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("width,sink,local", [(1, 0, 1), (8, 1, 1), (32, 2, 3), (33, 0, 33), (40, 39, 1), (300, 1, 2)])
@pytest.mark.parametrize("page,extra", [(16, 0), (3, 300), (1, 2), (1, 1500), (1, 7000), (1, 9000)])
def test_select(page, extra, width, sink, local, ties):
    b = B.batch([(1, 1), (1, 700), (50, 400), (0, 9), (9, 9), (20, 3), (1, 64)], 1, 512, page, 528, seed=width, extra=extra,
                tail_tokens=2, head_tokens=3)
    check_select(b, some_scores(b, width, ties), width, sink, local)


@pytest.mark.parametrize("blocks", [255, 256, 257, 1024, 1025, 2048, 2049, 8192, 8193, 20000])
def test_select_from_many(blocks):
    b = B.batch([(2, blocks), (1, blocks // 3)], 1, 512, 1, 528, seed=blocks, extra=0)
    for width, ties in ((1, False), (64, True), (min(blocks, 1000), False)):
        check_select(b, some_scores(b, blocks, ties), width, 0, 1)


@pytest.mark.parametrize("width,sink,local", [(1, 0, 1), (2, 0, 1), (7, 3, 4), (31, 1, 2), (64, 0, 1), (200, 7, 9)])
@pytest.mark.parametrize("blocks", [31, 32, 33, 256, 511, 512, 513])
def test_select_close_scores(blocks, width, sink, local):
    """Scores that differ in their last bits, in their sign, or not at all; most of them absent."""
    b = B.batch([(6, blocks), (1, 5), (4, blocks)], 1, 512, 1, 528, seed=blocks + width, extra=0)
    g = torch.Generator().manual_seed(blocks)
    sc = torch.randint(0, 3, (b["T"], b["table"].shape[1]), generator=g).float()
    last = (torch.tensor([1.0]).view(torch.int32) + sc.int()).view(torch.float32)       # 1 and the two values after it
    sc[0] = last[0]
    sc[1] = -last[1]
    sc[2] = 1.0
    sc[3] = (sc[3] - 1.0) * 3.4028234663852886e38
    sc[4, torch.rand(sc.shape[1], generator=g) < 0.8] = -math.inf
    sc[8, torch.rand(sc.shape[1], generator=g) < 0.95] = -math.inf
    sc[9] = last[9] * 2.0 ** torch.randint(-60, 60, sc.shape[1:], generator=g)
    check_select(b, sc, width, sink, local)


def test_select_special_values():
    b = B.batch([(6, 600)], 1, 512, 4, 528, seed=10)
    sc = some_scores(b, 3)
    sc[0, ::2] = -math.inf
    sc[0, 1::4] = math.nan
    sc[1, :] = -math.inf
    sc[1, 70] = 3.4028234663852886e38
    sc[2, ::3] = math.inf
    sc[3, :] = 0.0
    sc[3, ::2] = -0.0                                   # equal to 0
    sc[4, :] = -1e-40                                   # below the normal range
    sc[4, 9] = 1e-40
    sc[5, :] = math.nan
    for width in (3, 20, 140):
        check_select(b, sc, width, 1, 1)


def test_select_lengths_past_the_table():
    b = B.batch([(5, 64)], 1, 512, 16, 528, seed=11, extra=0)
    b["kv_len"][0] = 70
    check_select(b, some_scores(b), 3, 1, 1, error=M.MLA_ERR_CHUNK_RANGE)


# ---- attention ----

def some_blocks(b, width, seed=0):
    """Lists as they may come: in any order, holes, doubles, blocks past the token's own."""
    g = torch.Generator().manual_seed(seed + 17)
    blocks = torch.full((b["T"], width), -1, dtype=torch.int32)
    for t, s, _, pos in B.tokens(b):
        own = max(0, pos) // b["page"]
        blocks[t] = torch.randint(-1, own + 2, (width,), generator=g).clamp(max=b["table"].shape[1] - 1).to(torch.int32)
        blocks[t, int(torch.randint(0, width, (1,), generator=g))] = own
    return blocks


def check_attention(b, blocks, error=0, **kw):
    t = dev(b)
    out = torch.full((b["T"], b["q"].shape[1], 512), 3.0, dtype=torch.bfloat16, device=D)
    lse = torch.full((b["T"], b["q"].shape[1]), 5.0, device=D)
    M.mla_block_attention(t["q"], t["cache"], blocks.to(D), *where(t), b["scale"], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    ref = B.attend(b, B.block_positions(b, blocks))
    P.check_chunk(out, lse, ref)
    outside = torch.isnan(ref[2][..., 0])
    assert (out.cpu()[outside] == 3.0).all() and (lse.cpu()[outside] == 5.0).all()
    return out, lse


# few query rows: one kernel; many: the other
SHAPES = [([(1, 1)], 3), ([(1, 2), (1, 33)], 2), ([(1, 700), (1, 129), (1, 65)], 6), ([(7, 7), (2, 2)], 4), ([(17, 333), (1, 5)], 9),
          ([(1, 3000)], 40), ([(300, 700)], 70), ([(150, 150), (129, 900), (3, 4), (200, 411)], 64)]


@pytest.mark.parametrize("seqs,width", SHAPES, ids=str)
@pytest.mark.parametrize("H,d_qk,row,page", [(16, 576, 656, 64), (5, 512, 528, 16), (64, 576, 656, 48), (16, 512, 656, 16)])
def test_attention(seqs, width, H, d_qk, row, page):
    if sum(n for n, _ in seqs) * H > 6000:
        seqs = [(n // 4 + 1, L) for n, L in seqs]
    b = B.batch(seqs, H, d_qk, page, row, seed=H + width, tail_tokens=3, head_tokens=2)
    check_attention(b, some_blocks(b, width, H))


@pytest.mark.parametrize("H", [1, 2, 3, 4, 15, 16, 17, 24, 31, 33, 63, 64, 65, 100, 128])
@pytest.mark.parametrize("many", [False, True])
def test_attention_heads(H, many):
    # many: rows x (width x page) past what the kernel for many rows is taken from
    b = B.batch([(9, 150), (1, 40), (20, 90)], H, 576, 32, 656, seed=H, extra=8_000_000 // (30 * H * 32) if many else 2)
    check_attention(b, some_blocks(b, 8_000_000 // (30 * H * 32) if many else 5, H))


@pytest.mark.parametrize("page", [1, 2, 31, 32, 33, 128, 1000])
@pytest.mark.parametrize("many", [False, True])
def test_attention_pages_that_end_inside_a_tile(page, many):
    b = B.batch([(5, 333), (1, 70), (12, 64)], 16, 576, page, 656, seed=page, extra=16000 // page + 2 if many else 2)
    check_attention(b, some_blocks(b, 16000 // page if many else 7, page))


@pytest.mark.parametrize("many", [False, True])
def test_attention_empty_rows_and_lists(many):
    b = B.batch([(0, 50), (3, 0), (10, 4), (0, 0), (4, 4), (33, 70)], 16, 576, 16, 656, seed=1, tail_tokens=3, head_tokens=5,
                extra=400 if many else 2)
    blocks = some_blocks(b, 300 if many else 4, 3)
    blocks[20:30] = -1                                  # nothing listed
    blocks[31] = b["table"].shape[1] - 1                # only a block past its own
    check_attention(b, blocks)
    check_attention(b, blocks[:, :0])


@pytest.mark.parametrize("many", [False, True])
def test_attention_holes_reserved_slot_and_pages_past_the_cache(many):
    b = B.batch([(12, 400), (12, 90)], 16, 576, 16, 656, seed=3, extra=700 if many else 2)
    width = 700 if many else 26
    blocks = torch.arange(width, dtype=torch.int32).repeat(b["T"], 1)
    b["table"][0, 3] = -1
    b["table"][0, 5] = 0
    b["table"][1, 1] = -7
    b["cache"][0] = 0xFF
    check_attention(b, blocks)
    b["table"][1, 2] = 1 << 26                          # past the cache
    check_attention(b, blocks, error=M.MLA_ERR_DECODE_INDEX_RANGE)
    b["table"][1, 2] = b["pages"] - 1                   # a page that ends past it
    b["cache"] = b["cache"][:-7]
    check_attention(b, blocks, error=M.MLA_ERR_DECODE_INDEX_RANGE if (b["table"] >= 0).any() else 0)
    blocks[1, 0] = b["table"].shape[1]                  # past the table
    check_attention(b, blocks, error=M.MLA_ERR_DECODE_INDEX_RANGE)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what", ["code", "scale_inf", "rope_nan"])
def test_attention_rows_that_are_not_finite_reach_only_those_who_list_them(many, what):
    b = B.batch([(24, 200), (24, 200)], 16, 576, 16, 656, seed=4, extra=700 if many else 2)
    blocks = some_blocks(b, 700 if many else 5, 8)
    blocks[blocks == 2] = 3
    blocks[[5, 20, 40], 1] = 2                          # three tokens list block 2
    slot = int(b["table"][0, 2]) * 16 + 9
    if what == "code":
        b["cache"][slot, 300] = 0xFF
    elif what == "scale_inf":
        b["cache"][slot, 516:520] = torch.tensor([0, 0, 0x80, 0x7F], dtype=torch.uint8)
    else:
        b["cache"][slot, 600:602] = torch.tensor([0xC1, 0x7F], dtype=torch.uint8)
    out, _ = check_attention(b, blocks)
    assert torch.isnan(out[5].float()).all() and torch.isnan(out[20].float()).all() and not torch.isnan(out[40].float()).any()


def test_attention_blocks_past_65536_of_them():
    """The lists are made 65,536 blocks at a time."""
    g = torch.Generator().manual_seed(12)
    n, L = 6, 140000
    cache = P.make_cache(L + 5, 528, g, rope=False)
    b = dict(q=torch.randn((n, 16, 512), generator=g).to(torch.bfloat16), cache=cache, T=n,
             q_start=torch.tensor([0, 4, 6], dtype=torch.int32), kv_len=torch.tensor([L, 70000], dtype=torch.int32),
             table=torch.stack([torch.randperm(L + 4, generator=g)[:L].to(torch.int32) + 1 for _ in range(2)]), page=1,
             scale=0.05)
    blocks = torch.randint(-1, L, (n, 400), generator=g).to(torch.int32)
    blocks[:, 7] = torch.tensor([65535, 65536, 131072, 139999, 65536, 69999], dtype=torch.int32)
    check_attention(b, blocks)


def test_attention_lengths_past_the_table():
    b = B.batch([(20, 64)], 16, 576, 16, 656, seed=13, extra=0)
    b["kv_len"][0] = 70
    check_attention(b, torch.tensor([[0, 1, 2, 3]] * 20, dtype=torch.int32), error=M.MLA_ERR_CHUNK_RANGE)


def test_all_blocks_listed_is_chunk_attention():
    for many in (False, True):
        b = B.batch([(33, 333), (1, 77)], 16, 576, 16, 656, seed=14, extra=700 if many else 2)
        t = dev(b)
        blocks = torch.arange(b["table"].shape[1], dtype=torch.int32, device=D).repeat(b["T"], 1)
        out, lse = M.mla_block_attention(t["q"], t["cache"], blocks, *where(t), b["scale"])
        ref = P.chunk(b["q"], b["cache"], b["q_start"], b["kv_len"], b["table"], b["page"], b["scale"])
        P.check_chunk(out, lse, ref)


def test_a_workspace_of_any_contents_gives_the_same_bits():
    b = B.batch([(1, 3000), (2, 900)], 16, 576, 16, 656, seed=15)
    t, blocks = dev(b), some_blocks(b, 180, 1).to(D)
    got = []
    for byte in (0, 0xFF):
        ws = torch.full((M.mla_block_attention_workspace_bytes(3, 16, 180),), byte, dtype=torch.uint8, device=D)
        got.append(M.mla_block_attention(t["q"], t["cache"], blocks, *where(t), b["scale"], workspace=ws))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
