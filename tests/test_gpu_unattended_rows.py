"""Rows of a listed page, and drafted rows, that no token attends have no part in any output, whatever they hold."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P
import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"


def fill(b, s, positions, what):
    """Rows of sequence s become others: of far larger scales, or of values that are not finite."""
    for p in positions:
        slot = int(b["table"][s, p // b["page"]]) * b["page"] + p % b["page"]
        if what == "large":
            b["cache"][slot, 512:528] = torch.full((4,), 1e30).view(torch.uint8)
        else:
            b["cache"][slot] = 0xFF


def dev(b):
    return {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}


def same(x, y):
    return all(torch.equal(a.contiguous().view(torch.uint8), c.contiguous().view(torch.uint8)) for a, c in zip(x, y))


# heads of few rows in groups, of few rows alone, of many rows
@pytest.mark.parametrize("H,seqs,width", [(1, [(40, 333), (2, 37)], 9), (5, [(9, 100), (7, 250)], 12), (16, [(1, 70), (1, 130)], 3),
                                          (16, [(300, 1001), (150, 203)], 60), (2, [(900, 2500)], 80), (128, [(70, 700)], 40)])
@pytest.mark.parametrize("what", ["large", "nan"])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 528)])
def test_rows_past_a_token_in_its_own_block(H, seqs, width, what, d_qk, row):
    b = B.batch(seqs, H, d_qk, 32, row, seed=H + width, extra=1)
    g = torch.Generator().manual_seed(width)
    blocks = torch.full((b["T"], width), -1, dtype=torch.int32)
    for t, _, _, pos in B.tokens(b):
        blocks[t, 1:] = torch.randint(0, pos // 32 + 1, (width - 1,), generator=g).to(torch.int32)
        blocks[t, 0] = pos // 32
    blocks[0] = blocks[0].clamp(max=0)
    ref = B.attend(b, B.block_positions(b, blocks))

    def run():
        t = dev(b)
        got = M.mla_block_attention(t["q"], t["cache"], blocks.to(D), t["q_start"], t["kv_len"], t["table"], 32, b["scale"])
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        return got

    before = run()
    P.check_chunk(*before, ref)
    for s, (_, L) in enumerate(seqs):
        fill(b, s, range(L, -(-L // 32) * 32), what)    # past the context, in its last page
    after = run()
    P.check_chunk(*after, ref)
    assert same(before, after)


@pytest.mark.parametrize("H,wide", [(1, 2), (5, 2), (16, 2), (16, 2000), (2, 20000), (128, 600)])
@pytest.mark.parametrize("what", ["large", "nan"])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 528)])
def test_drafted_rows_that_no_mask_names(H, wide, what, d_qk, row):
    seqs = [(31, 90), (60, 300), (33, 33)]
    b = B.batch(seqs, H, d_qk, 32, row, seed=H, extra=wide)
    rows = [[j for j in (i, i // 2, 3) if j % 5 != 4] for _, _, i, _ in B.tokens(b)]
    ref = B.attend(b, B.tree_positions(b, rows))

    def run():
        t = dev(b)
        got = M.mla_tree_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 32, b["scale"],
                                   B.mask_bits(rows, b["T"], 2).to(D))
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        return got

    before = run()
    P.check_chunk(*before, ref)
    for s, (n, L) in enumerate(seqs):
        fill(b, s, [L - n + j for j in range(4, n, 5)], what)
    after = run()
    P.check_chunk(*after, ref)
    assert same(before, after)
