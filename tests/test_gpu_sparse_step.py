"""The block-sparse and tree operators as a server uses them, one after the other: prompts are written in chunks with their
rotary positions, the pages' keys kept, every token attends the blocks selected for it; trees are drafted, written,
attended and committed; sequences fork. Everything is held against the 64-bit formulas over the rows each sequence has."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P
import _plain_blocks as B

pytestmark = pytest.mark.gpu
D = "cuda:0"
INV = [10000.0 ** (-2.0 * i / 64) for i in range(32)]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=D)


class Server:
    def __init__(self, page=16, pages=260, rows=6, width=40, H=16):
        self.page, self.H, self.width, self.scale = page, H, width, 1 / math.sqrt(576)
        self.cache = torch.full((pages * page, 656), 0xFF, dtype=torch.uint8, device=D)
        self.keys = torch.full((pages, 576), float("nan"), dtype=torch.bfloat16, device=D)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=D)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=D)
        self.len = [0] * rows
        self.g = torch.Generator().manual_seed(5)
        self.spec = M.rope_spec(INV)

    def grow(self, r, n):
        table, refs = self.table[r].cpu(), self.refs.cpu()
        for k in range(-(-(self.len[r] + n) // self.page)):
            if table[k] < 0:
                table[k] = int((refs[1:] == 0).nonzero()[0]) + 1
                refs[table[k]] = 1
        self.table[r], self.refs[:] = table.to(D), refs.to(D)

    def write(self, new, positions=None):
        """Rows for new[r] tokens of each sequence, and their queries."""
        seqs = sorted(new)
        slots, starts, pos = [], [0], []
        for r in seqs:
            self.grow(r, new[r])
            t = self.table[r].tolist()
            at = range(self.len[r], self.len[r] + new[r])
            slots += [t[p // self.page] * self.page + p % self.page for p in at]
            pos += list(at)
            starts.append(len(slots))
            self.len[r] += new[r]
        n = len(slots)
        lat, k = (torch.randn((n, d), generator=self.g).to(torch.bfloat16).to(D) for d in (512, 64))
        q = (1.5 * torch.randn((n, self.H, 576), generator=self.g)).to(torch.bfloat16).to(D)
        self.where = (ints(starts), ints([self.len[r] for r in seqs]), self.table[seqs].contiguous(), self.page)
        pos = ints(pos) if positions is None else positions(self.where)
        M.mla_rope_kv_write(self.cache, torch.tensor(slots, device=D), lat, k, pos, self.spec, q_pe=q[..., 512:])
        return q

    def plain(self, q):
        start, lens, table, page = (x.cpu() if isinstance(x, torch.Tensor) else x for x in self.where)
        return dict(q=q.cpu(), cache=self.cache.cpu(), q_start=start, kv_len=lens, table=table, page=page, scale=self.scale,
                    T=q.shape[0], pages=self.keys.shape[0])

    def sparse(self, new, width=6):
        q = self.write(new)
        M.mla_block_keys(self.cache, *self.where, self.keys, q.shape[0])
        scores = M.mla_block_scores(q, self.keys, *self.where, self.scale)
        blocks = M.mla_block_select(scores, *self.where[:2], self.page, width, sink=1, local=2)
        out, lse = M.mla_block_attention(q, self.cache, blocks, *self.where, self.scale)
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        b = self.plain(q)
        for p, (m, tol) in B.mean_keys(b, 576, b["pages"]).items():
            assert ((self.keys[p].double().cpu() - m).abs() <= tol).all()
        want, tol = B.block_scores(b, self.keys.cpu())
        ok = ~tol.isnan()
        assert ((scores.double().cpu() - want).abs()[ok] <= tol[ok]).all()
        for row, w in zip(blocks.cpu().tolist(), B.select(b, scores.cpu(), width, 1, 2)):
            assert row == w
        P.check_chunk(out, lse, B.attend(b, B.block_positions(b, blocks.cpu())))

    def speculate(self, new, keep):
        """new[r] drafted tokens of each sequence, of which a path of at most `keep` is accepted."""
        seqs = sorted(new)
        parent = []
        for r in seqs:
            parent += [int(torch.randint(max(-1, i - 4), i, (1,), generator=self.g)) if i else -1 for i in range(new[r])]
        made = {}

        def positions(where):
            made["mask"], pos = M.mla_tree_mask(ints(parent), *where[:2], words=1)
            return pos

        q = self.write(new, positions)
        out, lse = M.mla_tree_attention(q, self.cache, *self.where, self.scale, made["mask"])
        b = self.plain(q)
        up = B.ancestors(b, torch.tensor(parent))
        P.check_chunk(out, lse, B.attend(b, B.tree_positions(b, up)))
        paths, path_len = torch.zeros((len(seqs), keep), dtype=torch.int32), []
        for i, r in enumerate(seqs):
            a, e = int(b["q_start"][i]), int(b["q_start"][i + 1])
            leaf = max(range(e - a), key=lambda j: len(up[a + j]))
            path = sorted(up[a + leaf])[:keep]
            paths[i, :len(path)] = torch.tensor(path)
            path_len.append(len(path))
        before = [torch.stack([self.row(r, self.len[r] - new[r] + int(j)) for j in paths[i, :path_len[i]]])
                  for i, r in enumerate(seqs)]
        lens = self.where[1].clone()
        M.mla_tree_commit(self.cache, self.where[0], lens, self.where[2], self.page, paths.to(D), ints(path_len), kv_len_out=lens)
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        for i, r in enumerate(seqs):
            self.len[r] += path_len[i] - new[r]
            assert int(lens[i]) == self.len[r]
            after = torch.stack([self.row(r, self.len[r] - path_len[i] + j) for j in range(path_len[i])])
            assert torch.equal(before[i], after)
        # the accepted rows' pages may be complete now
        M.mla_block_keys(self.cache, ints([0] + torch.tensor(path_len).cumsum(0).tolist()), lens, self.where[2], self.page,
                         self.keys, sum(path_len))

    def row(self, r, p):
        return self.cache[int(self.table[r, p // self.page]) * self.page + p % self.page].clone()


def test_prompt_decode_speculate_fork_and_go_on():
    s = Server()
    s.sparse({0: 100, 1: 260, 2: 5})
    s.sparse({0: 1, 1: 1, 2: 1})
    s.speculate({0: 20, 1: 32, 2: 9}, 6)
    s.sparse({0: 1, 1: 30, 2: 1})
    s.speculate({1: 12, 2: 25}, 5)
    s.sparse({0: 60, 1: 1, 2: 1})
    # a fork shares whole pages, and their keys
    M.mla_page_fork(s.cache, s.page, s.refs, s.table, ints([1]), ints([3]), ints([s.len[1]]))
    s.len[3] = s.len[1]
    s.sparse({1: 1, 3: 2})
    s.speculate({1: 7, 3: 16}, 4)
    s.sparse({0: 1, 1: 1, 2: 1, 3: 1})


def test_keys_made_anew_are_those_kept():
    s = Server()
    s.sparse({0: 100, 1: 260, 2: 5})
    s.sparse({0: 1, 1: 1, 2: 1})
    s.sparse({0: 13, 1: 7, 2: 40})
    total = [s.len[r] for r in range(3)]
    again = torch.full_like(s.keys, float("nan"))
    M.mla_block_keys(s.cache, ints([0] + torch.tensor(total).cumsum(0).tolist()), ints(total), s.table[:3].contiguous(), s.page, again,
                     sum(total))
    assert M.mla_get_error() == 0 and torch.equal(again.view(torch.int16), s.keys.view(torch.int16))


def step(q, cache, keys, parent, where, T, scale, ws, tree_ws):
    M.mla_block_keys(cache, *where, keys, T)
    scores = M.mla_block_scores(q, keys, *where, scale)
    blocks = M.mla_block_select(scores, *where[:2], where[3], 8, sink=1, local=1)
    sparse = M.mla_block_attention(q, cache, blocks, *where, scale, workspace=ws)
    mask, pos = M.mla_tree_mask(parent, *where[:2], words=2)
    tree = M.mla_tree_attention(q, cache, *where, scale, mask, workspace=tree_ws)
    return (keys, scores, blocks, *sparse, mask, pos, *tree)


@pytest.mark.parametrize("seqs", [[(1, 300), (3, 77), (0, 40), (50, 120)], [(40, 600), (60, 60)]], ids=str)
def test_captured_steps_serve_other_lengths(seqs):
    """One graph, replayed with other lengths, tables, queries and lists than it was captured with, gives the bits of calls;
    two graphs may share a workspace as long as they run one after the other."""
    total, H, page = max(sum(n for n, _ in seqs), 100), 16, 16
    made = []
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        mine = [(n, max(n, int(L * (1 - 0.2 * seed)))) for n, L in seqs] if seed < 2 else [(n, n) for n, _ in seqs]
        b = B.batch(mine, H, 576, page, 656, seed=seed)
        b["q"] = torch.randn((total, H, 576), generator=g).to(torch.bfloat16)
        parent = torch.full((total,), -1, dtype=torch.int32)
        for t, _, i, _ in B.tokens(b):
            parent[t] = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        made.append((b, parent))
    slots = max(b["cache"].shape[0] for b, _ in made)
    width = max(b["table"].shape[1] for b, _ in made)

    def padded(b, parent):
        cache = torch.zeros((slots, 656), dtype=torch.uint8)
        cache[:b["cache"].shape[0]] = b["cache"]
        table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        table[:, :b["table"].shape[1]] = b["table"]
        return [x.to(D) for x in (b["q"], cache, parent, b["q_start"], b["kv_len"], table)]

    ws = M.alloc_block_workspace(total, H, 8)
    tree_ws = M.alloc_chunk_workspace(total, H, len(seqs))
    live = padded(*made[0])
    keys = torch.zeros((slots // page, 576), dtype=torch.bfloat16, device=D)

    def run(a, k):
        q, cache, parent, start, lens, table = a
        return step(q, cache, k, parent, (start, lens, table, page), total, 1 / 24, ws, tree_ws)

    run(live, keys)                                     # (the first call of a process prepares its kernels)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run(live, keys)
        graphs.append((graph, outs))
    for b, parent in made + made[:1]:
        other = padded(b, parent)
        fresh = torch.zeros_like(keys)
        want = run(other, fresh)
        for x, y in zip(live, other):
            x.copy_(y)
        for graph, outs in graphs:
            keys.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(outs, want):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert M.mla_get_error() == 0


def test_two_calls_at_once_with_workspaces_of_their_own():
    sets = []
    for seed in range(2):
        b = B.batch([(1, 900), (2, 300), (33, 200)], 16, 576, 16, 656, seed=seed)
        t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
        g = torch.Generator().manual_seed(seed)
        blocks = torch.randint(0, 20, (b["T"], 12), generator=g).to(torch.int32).to(D)
        parent = torch.full((b["T"],), -1, dtype=torch.int32, device=D)
        sets.append((t, blocks, parent))

    def run(t, blocks, parent, stream=None):
        w = (t["q_start"], t["kv_len"], t["table"], 16)
        keys = torch.zeros((t["pages"], 576), dtype=torch.bfloat16, device=D)
        if stream is not None:
            torch.cuda.current_stream().synchronize()
        M.mla_block_keys(t["cache"], *w, keys, t["T"], stream=stream)
        scores = M.mla_block_scores(t["q"], keys, *w, 1 / 24, stream=stream)
        lists = M.mla_block_select(scores, *w[:2], 16, 5, stream=stream)
        a = M.mla_block_attention(t["q"], t["cache"], blocks, *w, 1 / 24, stream=stream)
        mask, pos = M.mla_tree_mask(parent, *w[:2], words=2, stream=stream)
        c = M.mla_tree_attention(t["q"], t["cache"], *w, 1 / 24, mask, stream=stream)
        return (keys, scores, lists, *a, mask, pos, *c)

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(run(*s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for p, q in zip(x, y):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    # the stream by its argument: what the call makes is made there
    with torch.cuda.stream(streams[0]):
        got = run(*sets[0], stream=streams[1])
    streams[1].synchronize()
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    for p, q in zip(got, want[0]):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("start", [[0, 9, 5, 20], [4, 2, 0, -3], [0, 30, 10, 25], [-5, 6, 12, 20], [3, 3, 99, 20], [20, 20, 20, 20]], ids=str)
@pytest.mark.parametrize("many", [False, True])
def test_starts_out_of_order_are_flagged_and_nothing_else_is_touched(start, many):
    b = B.batch([(5, 60), (7, 90), (8, 33)], 16, 576, 16, 656, seed=1, extra=20000 if many else 2)
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    T, width = 20, 20000 if many else 6
    w = (ints(start), t["kv_len"], t["table"], 16)
    flagged = start != [20, 20, 20, 20]

    def guarded(shape, dtype):
        flat = torch.zeros(64 + math.prod(shape) + 64, dtype=dtype, device=D)
        return flat, flat[64:-64].view(shape)

    keep = []
    for make in (lambda: M.mla_block_keys(t["cache"], *w, one((b["pages"], 576), torch.bfloat16), T),
                 lambda: M.mla_block_scores(t["q"], torch.zeros((b["pages"], 576), dtype=torch.bfloat16, device=D), *w, 0.04,
                                            scores=one((T, b["table"].shape[1]), torch.float32)),
                 lambda: M.mla_block_select(torch.zeros((T, b["table"].shape[1]), device=D), *w[:2], 16, 6, blocks=one((T, 6), torch.int32)),
                 lambda: M.mla_block_attention(t["q"], t["cache"], torch.zeros((T, width), dtype=torch.int32, device=D), *w, 0.04,
                                               out=one((T, 16, 512), torch.bfloat16), lse=one((T, 16), torch.float32)),
                 lambda: M.mla_tree_mask(torch.full((T,), -1, dtype=torch.int32, device=D), *w[:2], mask=one((T, 1), torch.int32),
                                         positions=one((T,), torch.int32)),
                 lambda: M.mla_tree_attention(t["q"], t["cache"], *w, 0.04, torch.zeros((T, 1), dtype=torch.int32, device=D),
                                              out=one((T, 16, 512), torch.bfloat16), lse=one((T, 16), torch.float32)),
                 lambda: M.mla_tree_commit(t["cache"].clone(), *w, torch.zeros((3, 2), dtype=torch.int32, device=D), ints([0, 0, 0]))):
        def one(shape, dtype):
            flat, view = guarded(shape, dtype)
            keep.append(flat)
            return view
        make()
        torch.cuda.synchronize()
        assert (M.mla_get_error() & M.MLA_ERR_CHUNK_RANGE != 0) == flagged
    for flat in keep:
        assert (flat[:64] == 0).all() and (flat[-64:] == 0).all()
