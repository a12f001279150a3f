"""The operators as a server uses them: chunks are written with their rotary positions turned, attended over the paged
cache, a sequence is forked for parallel sampling, children drop out, the pool is compacted, decoding goes on. The
whole is held against the 64-bit formulas over the tokens each sequence has, whatever pages they are in."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"
INV = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
AXIS = [0] * 8 + [1] * 12 + [2] * 12


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=D)


class Server:
    def __init__(self, page=16, pages=200, rows=8, width=20, H=16):
        self.page, self.H, self.width = page, H, width
        self.cache = torch.full((pages * page, 656), 0xFF, dtype=torch.uint8, device=D)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=D)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=D)
        self.len = [0] * rows
        self.rows = [[] for _ in range(rows)]       # per sequence: its tokens' cache rows, as they were written
        self.g = torch.Generator().manual_seed(11)
        self.spec = M.rope_spec(INV, AXIS)

    def grow(self, r, n):
        """Pages for n more tokens (the host's own allocator: any free page)."""
        table, refs = self.table[r].cpu(), self.refs.cpu()
        for k in range(-(-(self.len[r] + n) // self.page)):
            if table[k] < 0:
                vacant = [p for p in range(1, refs.numel()) if refs[p] == 0]
                table[k] = vacant[int(torch.randint(0, len(vacant), (1,), generator=self.g))]
                refs[table[k]] = 1
        self.table[r], self.refs[:] = table.to(D), refs.to(D)

    def step(self, new):
        """new: {row: tokens}. Writes them, attends, checks."""
        seqs = sorted(new)
        slots, starts = [], [0]
        for r in seqs:
            self.grow(r, new[r])
            t = self.table[r].tolist()
            slots += [t[p // self.page] * self.page + p % self.page for p in range(self.len[r], self.len[r] + new[r])]
            starts.append(len(slots))
        n = len(slots)
        lat = torch.randn((n, 512), generator=self.g).to(torch.bfloat16).to(D)
        k = torch.randn((n, 64), generator=self.g).to(torch.bfloat16).to(D)
        pos = torch.randint(0, 5000, (3, n), generator=self.g).to(torch.int32).to(D)
        proj = torch.randn((n, self.H, 192), generator=self.g).to(torch.bfloat16).to(D)
        q = torch.randn((n, self.H, 576), generator=self.g).to(torch.bfloat16).to(D)
        slot_t = torch.tensor(slots, device=D)
        M.mla_rope_kv_write(self.cache, slot_t, lat, k, pos, self.spec, q_pe=proj[..., 128:], q_out=q[..., 512:])
        for i, r in enumerate(seqs):
            self.rows[r] = self.rows[r] + list(self.cache[slot_t[starts[i]:starts[i + 1]]].cpu())
            self.len[r] += new[r]
        out, lse = M.mla_chunk_attention(q, self.cache, ints(starts), ints([self.len[r] for r in seqs]),
                                         self.table[seqs].contiguous(), self.page, 1 / math.sqrt(576))
        torch.cuda.synchronize()
        assert M.mla_get_error() == 0
        # the reference over the tokens as they were written, laid out one after the other
        host = torch.cat([torch.zeros((self.width * self.page, 656), dtype=torch.uint8)] +
                         [torch.cat([torch.stack(self.rows[r]),
                                     torch.zeros((self.width * self.page - self.len[r], 656), dtype=torch.uint8)])
                          for r in seqs])
        table = torch.arange(self.width * (len(seqs) + 1), dtype=torch.int32).view(-1, self.width)[1:]
        ref = P.chunk(q.cpu(), host, torch.tensor(starts), torch.tensor([self.len[r] for r in seqs]), table, self.page,
                      1 / math.sqrt(576))
        P.check_chunk(out, lse, ref)

    def fork(self, parent, child):
        M.mla_page_fork(self.cache, self.page, self.refs, self.table, ints([parent] * len(child)), ints(child),
                        ints([self.len[parent]] * len(child)))
        for c in child:
            self.len[c], self.rows[c] = self.len[parent], list(self.rows[parent])

    def free(self, rows):
        M.mla_page_free(self.refs, self.table, ints(rows))
        for r in rows:
            self.len[r], self.rows[r] = 0, []


def test_prefill_fork_sample_drop_compact_and_go_on():
    s = Server()
    s.step({0: 37, 1: 150, 2: 5})
    s.step({0: 1, 1: 20, 2: 1})
    s.fork(1, [3, 4, 5])
    s.step({1: 1, 3: 1, 4: 2, 5: 1})                # siblings go apart: their last pages are their own
    s.free([0, 4])
    s.step({1: 1, 2: 30, 3: 1, 5: 1})
    M.mla_page_compact(s.cache, s.page, s.refs, s.table)
    live = int((s.refs > 0).sum())
    assert (s.refs[1:live + 1] > 0).all() and int(s.table.max()) == live
    s.step({1: 1, 2: 1, 3: 3, 5: 1})
    s.fork(5, [0])
    s.step({0: 9, 5: 1, 6: 12})
    # moved to another cache: the same pages there
    other = torch.zeros_like(s.cache)
    used = torch.arange(1, s.refs.numel(), dtype=torch.int32, device=D)
    M.mla_page_copy(other, s.cache, s.page, used, used)
    s.cache = other
    s.step({0: 1, 1: 1, 6: 1})
    # everything let go: nothing counted
    s.free([0, 1, 2, 3, 5, 6])
    assert M.mla_get_error() == 0 and (s.refs == 0).all() and (s.table == -1).all()
