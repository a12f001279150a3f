"""Caches and key arrays of more than 2^32 bytes (and 2^31 values): the same rows in far slots give the same bits."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("many", [False, True])
def test_far_slots_give_the_bits_of_near_ones(page, many):
    b = B.batch([(40, 300), (1, 90), (33, 150)], 16, 576, page, 656, seed=page, extra=9000 // page if many else 2)
    near = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    pages = 7_000_000 // page
    shift = pages - b["pages"]
    far = dict(near)
    far["cache"] = torch.zeros((pages * page, 656), dtype=torch.uint8, device=D)
    far["cache"][shift * page:] = near["cache"]
    far["table"] = torch.where(near["table"] >= 0, near["table"] + shift, near["table"])
    assert far["cache"].numel() > 1 << 32
    g = torch.Generator().manual_seed(3)
    width = 9000 // page if many else 12
    blocks = torch.full((b["T"], width), -1, dtype=torch.int32)
    for t, _, _, pos in B.tokens(b):
        blocks[t, :12] = torch.randint(-1, pos // page + 1, (12,), generator=g).to(torch.int32)
        blocks[t, 5] = pos // page
    blocks = blocks.to(D)
    parent = torch.full((b["T"],), -1, dtype=torch.int32)
    for t, _, i, _ in B.tokens(b):
        parent[t] = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
    parent = parent.to(D)
    path = torch.tensor([[1, 5, 20, 33], [0, 0, 0, 0], [0, 4, 30, 0]], dtype=torch.int32, device=D)
    path_len = torch.tensor([4, 0, 3], dtype=torch.int32, device=D)

    def run(t, keys, start):
        w = (t["q_start"], t["kv_len"], t["table"], page)
        M.mla_block_keys(t["cache"], *w, keys, t["T"])
        scores = M.mla_block_scores(t["q"], keys, *w, t["scale"])
        out, lse = M.mla_block_attention(t["q"], t["cache"], blocks, *w, t["scale"])
        mask, _ = M.mla_tree_mask(parent, *w[:2], words=2)
        tree, tree_lse = M.mla_tree_attention(t["q"], t["cache"], *w, t["scale"], mask)
        M.mla_tree_commit(t["cache"], *w, path, path_len)
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        return keys[start:start + b["pages"]], scores, out, lse, tree, tree_lse, t["cache"][start * page:]

    few = run(near, torch.zeros((b["pages"], 576), dtype=torch.bfloat16, device=D), 0)
    keys = torch.zeros((pages, 576), dtype=torch.bfloat16, device=D)
    assert page > 1 or keys.numel() > 1 << 31
    for x, y in zip(few, run(far, keys, shift)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
