"""Lists that a CTA of mla_block_attention reads itself (tokens that share their tile with none), at their longest and in any
order, on sizes where the first rows are copied as soon as the list is there."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P
import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"


def attention(b, blocks, error=0):
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    out, lse = M.mla_block_attention(t["q"], t["cache"], blocks.to(D), t["q_start"], t["kv_len"], t["table"], b["page"], b["scale"])
    torch.cuda.synchronize()
    assert M.mla_get_error() == error
    return out, lse


@pytest.mark.parametrize("H,d_qk,row", [(1, 576, 656), (16, 512, 528), (40, 576, 656)])
@pytest.mark.parametrize("page", [1, 3, 32])
@pytest.mark.parametrize("width", [191, 192, 193, 511, 512, 513])
def test_long_lists_in_any_order(width, page, H, d_qk, row):
    b = B.batch([(1, 600 * page), (1, 200 * page + page // 2), (1, 7)], H, d_qk, page, row, seed=width + page)
    g = torch.Generator().manual_seed(width)
    blocks = torch.full((3, width), -1, dtype=torch.int32)
    up = torch.randperm(600, generator=g)[:width].sort().values.to(torch.int32)
    blocks[0, :len(up)] = up                            # ascending
    blocks[1] = torch.randint(-2, 201, (width,), generator=g).to(torch.int32)      # any order, doubles, none
    blocks[2] = torch.arange(width, dtype=torch.int32).flip(0)                     # its own are the last ones
    out, lse = attention(b, blocks)
    P.check_chunk(out, lse, B.attend(b, B.block_positions(b, blocks)))


def test_the_same_lists_give_the_same_bits():
    b = B.batch([(1, 4000)] * 6, 16, 576, 16, 656, seed=5)
    blocks = torch.arange(32, dtype=torch.int32).repeat(6, 1) * 7
    first = attention(b, blocks)
    for _ in range(20):
        again = attention(b, blocks)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
