"""Forms of the block operators that only some sizes take: scores of more columns than a CTA has at once, for each kind of
heads, and the attention of one to three heads in the kernel for many rows."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P
import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"
ROUND = 256                                             # columns that a CTA has at once


def dev(b):
    return {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}


def check_scores(b, d_qk, holes=0):
    g = torch.Generator().manual_seed(b["T"])
    keys = torch.randn((b["pages"], d_qk), generator=g).to(torch.bfloat16)
    if holes:
        b["table"][0, torch.randperm(b["table"].shape[1], generator=g)[:holes]] = -1
    t = dev(b)
    scores = torch.full((b["T"], b["table"].shape[1]), 5.0, device=D)
    M.mla_block_scores(t["q"], keys.to(D), t["q_start"], t["kv_len"], t["table"], b["page"], b["scale"], scores=scores)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    want, tol = B.block_scores(b, keys)
    got, written = scores.double().cpu(), ~tol.isnan()
    gone = written & torch.isneginf(want)
    assert (got[~written] == 5.0).all() and torch.isneginf(got[gone]).all()
    ok = written & ~gone
    off = ((got - want).abs() / tol)[ok]
    assert off.max() <= 1, f"off by {off.max():.3g} of the tolerance"


# beyond 8 CTAs' columns; and where a table is taken to be less full than it is
@pytest.mark.parametrize("blocks", [1025, 1300, 2047, 2048, 2049, 2305, 4095, 4096, 4097, 4500])
@pytest.mark.parametrize("H,d_qk", [(1, 576), (4, 512), (16, 576), (16, 512), (32, 576), (48, 576), (128, 512), (128, 576)])
def test_scores_in_rounds(blocks, H, d_qk):
    b = B.batch([(9, blocks + 1), (2, 7), (3, blocks - 300)], H, d_qk, 1, 656, seed=blocks + H, tail_tokens=1)
    check_scores(b, d_qk, holes=blocks // 9)


# as many tiles as there are SMs: a CTA a tile
@pytest.mark.parametrize("blocks", [257, 300, 341])
@pytest.mark.parametrize("H", [8, 16, 30, 32, 40, 128])
def test_scores_in_rounds_of_many_tiles(blocks, H):
    tokens = 4 * (32 // H) if H <= 32 else 2 if H <= 64 else 1
    n = 160 * tokens
    b = B.batch([(n, blocks * 16 + 5)], H, 576, 16, 656, seed=blocks, extra=0)
    assert blocks > ROUND and b["table"].shape[1] * 3 // 4 <= ROUND
    check_scores(b, 576, holes=11)


@pytest.mark.parametrize("H", [1, 2, 3])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 528)])
def test_attention_of_few_heads_and_many_rows(H, d_qk, row):
    page, seqs = 32, [(61, 300), (3, 40), (80, 120), (64, 64)]
    positions = (4 << 20) // (sum(n for n, _ in seqs) * H) + 1
    b = B.batch(seqs, H, d_qk, page, row, seed=H, extra=positions // page + 1, tail_tokens=3, head_tokens=2)
    width = min(b["table"].shape[1], positions // page + 1)
    # (what the kernel for many rows is taken from)
    assert b["T"] * H >= 36 * len(seqs) and b["T"] * H * width * page >= 4 << 20
    g = torch.Generator().manual_seed(H)
    blocks = torch.full((b["T"], width), -1, dtype=torch.int32)
    for t, _, _, pos in B.tokens(b):
        blocks[t, :40] = torch.randint(-1, pos // page + 1, (40,), generator=g).to(torch.int32)
        blocks[t, 17] = pos // page
    t = dev(b)
    out = torch.full((b["T"], H, 512), 3.0, dtype=torch.bfloat16, device=D)
    lse = torch.full((b["T"], H), 5.0, device=D)
    M.mla_block_attention(t["q"], t["cache"], blocks.to(D), t["q_start"], t["kv_len"], t["table"], page, b["scale"], out=out, lse=lse)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    ref = B.attend(b, B.block_positions(b, blocks))
    P.check_chunk(out, lse, ref)
    outside = torch.isnan(ref[2][..., 0])
    assert (out.cpu()[outside] == 3.0).all() and (lse.cpu()[outside] == 5.0).all()
