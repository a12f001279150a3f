"""Refusals of the rotary, chunk-attention and page entry points: decided on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from fp8_mla_kv_gb300 import build as B
from fp8_mla_kv_gb300 import mlasparse as M

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load()


def spec(**kw):
    return M.rope_spec([1.0 / (i + 1) for i in range(32)], **kw)


def test_rope(lib):
    r = spec()
    f = lib.mla_rope
    a16 = P(256)
    ok = dict(x=a16, xr=64, xh=64, y=a16, yr=64, yh=64, n=0, h=1, pos=a16, ps=0, r=ctypes.byref(r))

    def call(**kw):
        v = {**ok, **kw}
        return f(v["x"], v["xr"], v["xh"], v["y"], v["yr"], v["yh"], v["n"], v["h"], v["pos"], v["ps"], v["r"], None)

    assert call() == M.MLA_OK and call(n=4, h=0) == M.MLA_OK
    for bad in (dict(n=-1), dict(h=-1), dict(ps=-1), dict(r=None), dict(n=2, x=None), dict(n=2, y=None),
                dict(n=2, pos=None), dict(n=2, x=P(264)), dict(n=2, y=P(258)), dict(n=2, xr=60), dict(n=2, h=2, yh=4),
                dict(n=2, pos=P(257))):
        assert call(**bad) == M.MLA_EINVAL, bad
    for field, value in (("n_axes", 0), ("n_axes", 5), ("scale", float("nan"))):
        s = spec()
        setattr(s, field, value)
        assert call(r=ctypes.byref(s)) == M.MLA_EINVAL
    s = spec()
    s.axis[3] = 1
    assert call(r=ctypes.byref(s)) == M.MLA_EINVAL              # an axis that is not there
    s = spec()
    s.inv_freq[31] = float("inf")
    assert call(r=ctypes.byref(s)) == M.MLA_EINVAL
    s = spec(axis=[i % 3 for i in range(32)])
    assert call(n=5, ps=4, r=ctypes.byref(s)) == M.MLA_EINVAL   # axes overlap
    with pytest.raises(ValueError):
        M.rope_spec([1.0] * 31)
    with pytest.raises(ValueError):
        M.rope_spec([1.0] * 32, axis=[4] * 32)


def test_rope_kv_write(lib):
    r = ctypes.byref(spec())
    kv = M.KVCache(256, 16, 656)

    def call(kv=kv, n=2, slots=P(256), lat=P(256), k=P(256), pos=P(256), r=r, q=None, qr=0, qh=0, qo=None, qor=0, qoh=0, h=0):
        return lib.mla_rope_kv_write(kv, slots, lat, k, n, 0, pos, 0, r, q, qr, qh, qo, qor, qoh, h, None)

    assert call(n=0) == M.MLA_OK
    for bad in (dict(n=-1), dict(h=-1), dict(kv=M.KVCache(256, 16, 528)), dict(kv=M.KVCache(256, -1, 656)),
                dict(kv=M.KVCache(None, 16, 656)), dict(kv=M.KVCache(264, 16, 656)), dict(slots=None), dict(slots=P(260)),
                dict(lat=None), dict(lat=P(264)), dict(k=None), dict(k=P(258)), dict(pos=None), dict(r=None),
                dict(q=P(256), h=1), dict(qo=P(256), h=1), dict(q=P(256), qo=P(264), qr=64, qor=64, h=1),
                dict(q=P(256), qo=P(256), qr=63, qor=64, h=1)):
        assert call(**bad) == M.MLA_EINVAL, bad


def test_chunk_attention(lib):
    kv = M.KVCache(256, 16, 656)

    def call(q=P(256), T=1, H=16, d=576, kv=kv, qs=P(256), kl=P(256), bt=P(256), ns=1, mp=1, ps=16, sc=0.1, out=P(256),
             lse=P(256), ws=None, wb=0):
        return lib.mla_chunk_attention(q, T, H, d, kv, qs, kl, bt, ns, mp, ps, 1, sc, out, lse, ws, wb, None)

    assert call(T=0) == M.MLA_OK and call(ns=0) == M.MLA_OK
    for bad in (dict(T=-1), dict(ns=-1), dict(mp=-1), dict(ps=0), dict(sc=float("nan")), dict(sc=float("inf")),
                dict(kv=M.KVCache(256, -1, 656)), dict(kv=M.KVCache(256, 16, 600)), dict(q=None), dict(out=None),
                dict(lse=None), dict(qs=None), dict(kl=None), dict(bt=None), dict(kv=M.KVCache(None, 16, 656)),
                dict(q=P(264)), dict(out=P(264)), dict(kv=M.KVCache(264, 16, 656)), dict(lse=P(257)), dict(qs=P(257)),
                dict(kl=P(257)), dict(bt=P(257))):
        assert call(**bad) == M.MLA_EINVAL, bad
    for bad in (dict(d=300), dict(H=0), dict(H=129), dict(kv=M.KVCache(256, 16, 528)), dict(T=1 << 30, H=128),
                dict(mp=1 << 20, ps=1 << 11), dict(mp=2, ps=1 << 30)):
        assert call(**bad) == M.MLA_EUNSUPPORTED, bad
    for T, H, n in ((0, 16, 1), (1, 0, 1), (1, 129, 1), (1, 16, 0)):
        assert lib.mla_chunk_attention_workspace_bytes(T, H, n) == 0


def test_pages(lib):
    kv, kv5 = M.KVCache(256, 64, 656), M.KVCache(256, 64, 528)
    a = P(256)
    f = lib.mla_page_copy
    assert f(kv, kv, 16, None, None, 0, None) == M.MLA_OK
    for args in ((kv, kv, 16, a, a, -1), (kv, kv, 0, a, a, 1), (kv, kv5, 16, a, a, 1), (kv, kv, 16, None, a, 1),
                 (kv, kv, 16, a, None, 1), (M.KVCache(None, 64, 656), kv, 16, a, a, 1),
                 (kv, M.KVCache(264, 64, 656), 16, a, a, 1), (M.KVCache(256, 64, 600), kv, 16, a, a, 1),
                 (kv, kv, 16, P(257), a, 1)):
        assert f(*args, None) == M.MLA_EINVAL
    f = lib.mla_page_free
    assert f(a, 4, a, 2, 2, a, 0, None) == M.MLA_OK
    for args in ((a, 0, a, 2, 2, a, 1), (a, 4, a, 0, 2, a, 1), (a, 4, a, 2, 0, a, 1), (a, 4, a, 2, 2, a, -1),
                 (None, 4, a, 2, 2, a, 1), (a, 4, None, 2, 2, a, 1), (a, 4, a, 2, 2, None, 1), (P(258), 4, a, 2, 2, a, 1)):
        assert f(*args, None) == M.MLA_EINVAL
    need = lib.mla_page_workspace_bytes(4, 3)
    assert need > 0 and lib.mla_page_workspace_bytes(0, 3) == 0 and lib.mla_page_workspace_bytes(4, -1) == 0

    def fork(kv=kv, ps=16, refs=a, P_=4, t=a, ns=2, mp=2, p=a, c=a, l=a, n=3, ws=a, wb=need):
        return lib.mla_page_fork(kv, ps, refs, P_, t, ns, mp, p, c, l, n, ws, wb, None)

    assert fork(n=0) == M.MLA_OK
    for bad in (dict(n=-1), dict(ps=0), dict(P_=0), dict(P_=5), dict(ns=0), dict(mp=0), dict(kv=M.KVCache(None, 64, 656)),
                dict(refs=None), dict(t=None), dict(p=None), dict(c=None), dict(l=None), dict(l=P(257))):
        assert fork(**bad) == M.MLA_EINVAL, bad
    for bad in (dict(ws=None), dict(wb=need - 1), dict(ws=P(264))):
        assert fork(**bad) == M.MLA_ENOWORKSPACE, bad

    def compact(kv=kv, ps=16, r=a, ro=a, P_=4, t=a, to=a, ns=2, mp=2, m=None, ws=a, wb=1 << 30):
        return lib.mla_page_compact(kv, ps, r, ro, P_, t, to, ns, mp, m, ws, wb, None)

    for bad in (dict(ps=0), dict(P_=0), dict(P_=5), dict(ns=-1), dict(mp=-1), dict(r=None), dict(ro=None), dict(t=None),
                dict(to=None), dict(kv=M.KVCache(None, 64, 656)), dict(m=P(258)), dict(to=P(258))):
        assert compact(**bad) == M.MLA_EINVAL, bad
    for bad in (dict(ws=None), dict(wb=16), dict(ws=P(264))):
        assert compact(**bad) == M.MLA_ENOWORKSPACE, bad


def test_the_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    c = torch.zeros((64, 656), dtype=torch.uint8)
    for f in (lambda: M.mla_page_copy(c, c, 16, i, i), lambda: M.mla_page_free(i, i.view(2, 2), i),
              lambda: M.mla_page_compact(c, 16, i, i.view(2, 2)),
              lambda: M.mla_rope(torch.zeros((4, 64), dtype=torch.bfloat16), i, spec())):
        with pytest.raises(ValueError):
            f()
