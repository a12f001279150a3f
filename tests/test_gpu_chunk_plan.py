"""mla_chunk_attention around the sizes at which its plan changes: 512 sequences (up to there the plan holds them in
shared memory, a thread each, and sorts them when there is more than a wave of pieces), 36 query rows a sequence (from
there the kernel for many rows runs, where the table is wide), contexts at the shortest piece."""

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"


def run(seqs, H, page=16, capacity=0, seed=0):
    """seqs: (new tokens, context length); a table for contexts of at least `capacity` positions."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-L // page) for _, L in seqs]
    cache = P.make_cache((sum(pages) + 2) * page, 656, g)
    order = torch.randperm(sum(pages) + 1, generator=g).to(torch.int32) + 1
    table = torch.full((len(seqs), max(max(pages) + 1, -(-capacity // page))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(pages):
        table[i, :k] = order[at:at + k]
        at += k
    start = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    q = torch.randn((int(start[-1]), H, 576), generator=g).to(torch.bfloat16)
    got = []
    for _ in range(2):
        got.append(M.mla_chunk_attention(q.to(D), cache.to(D), start.to(D), lens.to(D), table.to(D), page, 1 / 24))
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    P.check_chunk(*got[0], P.chunk(q, cache, start, lens, table[:, :max(pages) + 1], page, 1 / 24))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("n_seq", [511, 512, 513, 1024, 1025])
@pytest.mark.parametrize("H,capacity", [(3, 0), (40, 100000)])          # few rows, many rows
def test_many_sequences_and_a_split_one(n_seq, H, capacity):
    """A tile or more for each sequence (more than a wave), short ones, empty ones, and long ones first, last and in
    between, which are cut."""
    g = torch.Generator().manual_seed(n_seq + H)
    seqs = [(int(torch.randint(0, 4, (1,), generator=g)) or 1, int(torch.randint(1, 60, (1,), generator=g))) for _ in range(n_seq)]
    seqs[7], seqs[n_seq - 9] = (0, 20), (0, 0)
    for s, L in ((0, 2500), (n_seq // 2, 6000), (n_seq - 1, 3100)):
        seqs[s] = (1, L)
    run(seqs, H, capacity=capacity, seed=n_seq)


@pytest.mark.parametrize("n_seq", [512, 513])
@pytest.mark.parametrize("H,capacity", [(3, 0), (40, 100000)])
def test_sequences_that_are_all_alike(n_seq, H, capacity):
    run([(1, 33)] * n_seq, H, capacity=capacity, seed=1)


@pytest.mark.parametrize("n,H", [(35, 1), (36, 1), (7, 5), (3, 12), (1, 35), (1, 36), (2, 18)])
@pytest.mark.parametrize("capacity", [0, 200000])
def test_around_36_rows_a_sequence(n, H, capacity):
    run([(n, 300), (n, 41), (n, n), (n, 1000)], H, capacity=capacity, seed=n)


@pytest.mark.parametrize("L", [127, 128, 129, 255, 256, 257, 4096, 4097])
@pytest.mark.parametrize("n,H", [(1, 16), (4, 16), (9, 16)])
def test_contexts_around_the_shortest_piece(L, n, H):
    run([(n, L)], H, capacity=70000 if n > 1 else 0, seed=L)
