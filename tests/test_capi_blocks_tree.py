"""Refusals of the block-sparse and tree entry points: decided on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from fp8_mla_kv_gb300 import build as B
from fp8_mla_kv_gb300 import mlasparse as M

P = ctypes.c_void_p
A = P(256)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load()


def refuse(call, ok, invalid, unsupported=()):
    for v in ok:
        assert call(**v) == M.MLA_OK, v
    for v in invalid:
        assert call(**v) == M.MLA_EINVAL, v
    for v in unsupported:
        assert call(**v) == M.MLA_EUNSUPPORTED, v


KV = M.KVCache(256, 64, 656)
BATCH_INVALID = [dict(ns=-1), dict(mp=-1), dict(ps=0), dict(ps=-4), dict(qs=None), dict(kl=None), dict(bt=None), dict(qs=P(258)),
                 dict(kl=P(257)), dict(bt=P(259))]
BATCH_UNSUPPORTED = [dict(mp=1 << 20, ps=1 << 11), dict(mp=2, ps=1 << 30), dict(mp=1, ps=(1 << 31) - 4096)]


def test_keys(lib):
    def call(kv=KV, d=576, qs=A, kl=A, bt=A, ns=1, mp=2, ps=16, T=4, keys=A, nk=4):
        return lib.mla_block_keys(kv, d, qs, kl, bt, ns, mp, ps, T, keys, nk, None)

    refuse(call, [dict(T=0), dict(ns=0), dict(mp=0)],
           BATCH_INVALID + [dict(T=-1), dict(nk=-1), dict(keys=None), dict(keys=P(264)), dict(kv=M.KVCache(None, 64, 656)),
                            dict(kv=M.KVCache(264, 64, 656)), dict(kv=M.KVCache(256, -1, 656)), dict(kv=M.KVCache(256, 64, 600))],
           BATCH_UNSUPPORTED + [dict(d=500), dict(kv=M.KVCache(256, 64, 528))])


def test_scores(lib):
    def call(q=A, T=4, H=16, d=576, keys=A, nk=4, qs=A, kl=A, bt=A, ns=1, mp=2, ps=16, sc=0.1, out=A):
        return lib.mla_block_scores(q, T, H, d, keys, nk, qs, kl, bt, ns, mp, ps, sc, out, None)

    refuse(call, [dict(T=0), dict(ns=0), dict(mp=0)],
           BATCH_INVALID + [dict(T=-1), dict(nk=-1), dict(sc=float("nan")), dict(sc=float("inf")), dict(q=None), dict(keys=None),
                            dict(out=None), dict(q=P(264)), dict(keys=P(264)), dict(out=P(258))],
           BATCH_UNSUPPORTED + [dict(d=500), dict(H=0), dict(H=129), dict(T=1 << 30, H=128)])


def test_select(lib):
    def call(sc=A, T=4, cols=8, qs=A, kl=A, ns=1, ps=16, sink=1, local=1, width=4, out=A):
        return lib.mla_block_select(sc, T, cols, qs, kl, ns, ps, sink, local, width, out, None)

    refuse(call, [dict(T=0), dict(ns=0), dict(cols=0)],
           [dict(T=-1), dict(ns=-1), dict(cols=-1), dict(ps=0), dict(sink=-1), dict(local=0), dict(width=1), dict(sink=4),
            dict(width=-1), dict(sink=(1 << 31) - 1, local=(1 << 31) - 1), dict(sc=None), dict(out=None), dict(qs=None), dict(kl=None),
            dict(sc=P(258)), dict(out=P(257))],
           [dict(cols=1 << 20, ps=1 << 11)])


def test_attention(lib):
    def call(q=A, T=1, H=16, d=576, kv=KV, bl=A, w=4, qs=A, kl=A, bt=A, ns=1, mp=2, ps=16, sc=0.1, out=A, lse=A, ws=None, wb=0):
        return lib.mla_block_attention(q, T, H, d, kv, bl, w, qs, kl, bt, ns, mp, ps, sc, out, lse, ws, wb, None)

    refuse(call, [dict(T=0), dict(ns=0)],
           BATCH_INVALID + [dict(T=-1), dict(w=-1), dict(sc=float("nan")), dict(q=None), dict(bl=None), dict(out=None), dict(lse=None),
                            dict(q=P(264)), dict(out=P(264)), dict(lse=P(257)), dict(bl=P(257)), dict(kv=M.KVCache(None, 64, 656)),
                            dict(kv=M.KVCache(264, 64, 656)), dict(kv=M.KVCache(256, -1, 656)), dict(kv=M.KVCache(256, 64, 600))],
           BATCH_UNSUPPORTED + [dict(d=500), dict(H=0), dict(H=129), dict(kv=M.KVCache(256, 64, 528)), dict(T=1 << 30, H=128)])
    for T, H, w in ((0, 16, 1), (1, 0, 1), (1, 129, 1), (1, 16, -1)):
        assert lib.mla_block_attention_workspace_bytes(T, H, w) == 0


def test_tree(lib):
    def mask(p=A, T=4, qs=A, kl=A, ns=1, m=A, w=2, pos=A):
        return lib.mla_tree_mask(p, T, qs, kl, ns, m, w, pos, None)

    refuse(mask, [dict(T=0), dict(ns=0)], [dict(T=-1), dict(ns=-1), dict(w=-1), dict(p=None), dict(m=None), dict(qs=None), dict(kl=None),
                                           dict(p=P(258)), dict(m=P(257)), dict(pos=P(258))])

    def attention(q=A, T=1, H=16, d=576, kv=KV, qs=A, kl=A, bt=A, ns=1, mp=2, ps=16, m=A, w=2, sc=0.1, out=A, lse=A, ws=None, wb=0):
        return lib.mla_tree_attention(q, T, H, d, kv, qs, kl, bt, ns, mp, ps, m, w, sc, out, lse, ws, wb, None)

    refuse(attention, [dict(T=0), dict(ns=0)],
           BATCH_INVALID + [dict(T=-1), dict(w=-1), dict(m=None), dict(m=P(258)), dict(sc=float("inf")), dict(q=None), dict(out=None),
                            dict(lse=None), dict(q=P(264)), dict(kv=M.KVCache(None, 64, 656))],
           BATCH_UNSUPPORTED + [dict(d=500), dict(H=0), dict(H=129), dict(kv=M.KVCache(256, 64, 528))])

    def commit(kv=KV, qs=A, kl=A, bt=A, ns=1, mp=2, ps=16, p=A, pl=A, most=3, out=A):
        return lib.mla_tree_commit(kv, qs, kl, bt, ns, mp, ps, p, pl, most, out, None)

    refuse(commit, [dict(ns=0)],
           BATCH_INVALID + [dict(most=-1), dict(p=None), dict(pl=None), dict(p=P(258)), dict(pl=P(258)), dict(out=P(257)),
                            dict(kv=M.KVCache(None, 64, 656)), dict(kv=M.KVCache(264, 64, 656)), dict(kv=M.KVCache(256, -1, 656)),
                            dict(kv=M.KVCache(256, 64, 600))], BATCH_UNSUPPORTED)


def test_the_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((1, 2), dtype=torch.int32)
    c = torch.zeros((64, 656), dtype=torch.uint8)
    q = torch.zeros((1, 16, 576), dtype=torch.bfloat16)
    k = torch.zeros((4, 576), dtype=torch.bfloat16)
    one = i[:1]
    for f in (lambda: M.mla_block_keys(c, i, one, t, 16, k, 1), lambda: M.mla_block_scores(q, k, i, one, t, 16, 0.1),
              lambda: M.mla_block_select(torch.zeros(1, 2), i, one, 16, 4), lambda: M.mla_block_attention(q, c, t, i, one, t, 16, 0.1),
              lambda: M.mla_tree_mask(one, i, one), lambda: M.mla_tree_attention(q, c, i, one, t, 16, 0.1, t),
              lambda: M.mla_tree_commit(c, i, one, t, 16, t, one)):
        with pytest.raises(ValueError):
            f()
