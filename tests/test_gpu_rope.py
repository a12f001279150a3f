"""mla_rope and mla_rope_kv_write against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"
INV = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
AXES = {1: [0] * 32, 2: [i % 2 for i in range(32)], 3: [0] * 8 + [1] * 12 + [2] * 12, 4: [i // 8 for i in range(32)]}


def close(y, ref, mag):
    # one BF16 rounding, and fp32 angles (off by less than 2^-23 rad) and products
    err = (y.double().cpu() - ref).abs()
    assert (err <= P.BF16 * ref.abs() + 2.0 ** -21 * mag + 1e-38).all(), err.max()


@pytest.mark.parametrize("n,heads", [(1, 1), (1, 128), (3, 5), (33, 16), (67, 40), (257, 7), (1000, 64)])
@pytest.mark.parametrize("axes,interleaved", [(1, True), (3, False), (2, True), (4, False)])
def test_rope_matches(n, heads, axes, interleaved):
    g = torch.Generator().manual_seed(n * 131 + heads)
    proj = torch.randn((n, heads, 192), generator=g).to(torch.bfloat16)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (axes, n), generator=g).to(torch.int32)
    if n > 2:
        pos[:, 0], pos[:, 1] = 0, (1 << 31) - 1
    spec = M.rope_spec(INV, AXES[axes], interleaved=interleaved, scale=1.25)
    x = proj.to(D)
    out = torch.full((n, heads, 576), 7.0, dtype=torch.bfloat16, device=D)
    M.mla_rope(x[..., 128:], pos.to(D), spec, out=out[..., 512:])
    torch.cuda.synchronize()
    # far positions: the reference's own angle is a product in 64 bits, off by 2^31 * 2^-53
    ref, mag = P.rotate(proj[..., 128:].double(), pos, INV, AXES[axes], interleaved, 1.25)
    close(out[..., 512:], ref, mag)
    assert (out[..., :512] == 7.0).all(), "only the rotary values are written"
    assert torch.equal(x.cpu(), proj)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_in_place_and_back(interleaved):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((50, 20, 64), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (3, 50), generator=g).to(torch.int32)
    fwd, back = (M.rope_spec(INV, AXES[3], interleaved=interleaved, inverse=v) for v in (False, True))
    y = x.to(D)
    M.mla_rope(y, pos.to(D), fwd, out=y)
    ref, mag = P.rotate(x.double(), pos, INV, AXES[3], interleaved)
    close(y, ref, mag)
    z = M.mla_rope(y, pos.to(D), back)
    ref2, mag2 = P.rotate(y.double().cpu(), pos, INV, AXES[3], interleaved, inverse=True)
    close(z, ref2, mag2)
    # two BF16 roundings of a rotation, which keeps lengths
    pair = (x.double().view(50, 20, 32, 2) if interleaved else x.double().view(50, 20, 2, 32).transpose(2, 3))
    length = pair.norm(dim=-1, keepdim=True).expand_as(pair)
    length = length.reshape(50, 20, 64) if interleaved else length.transpose(2, 3).reshape(50, 20, 64)
    assert ((z.double().cpu() - x.double()).abs() <= (2 * P.BF16 * 1.5 + 2.0 ** -18) * length + 1e-30).all()


def test_rope_inverse_is_the_gradient():
    """d(sum w . rope(x)) / dx is the inverse rotation of w; checked by differences of the 64-bit formula."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn((4, 3, 64), generator=g).double()
    w = torch.randn((4, 3, 64), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 5000, (2, 4), generator=g).to(torch.int32)
    dx = M.mla_rope(w.to(D), pos.to(D), M.rope_spec(INV, AXES[2], interleaved=True, inverse=True)).double().cpu()
    for idx in [(0, 0, 0), (1, 2, 17), (3, 1, 63), (2, 0, 40)]:
        e = torch.zeros_like(x)
        e[idx] = 0.5
        f = [(P.rotate(v, pos, INV, AXES[2], True)[0] * w.double()).sum() for v in (x + e, x - e)]   # linear: exact
        lo = idx[2] & ~1
        mag = w[idx[0], idx[1], lo:lo + 2].double().abs().sum()
        assert abs(dx[idx] - (f[0] - f[1])) <= P.BF16 * abs(f[0] - f[1]) + 2.0 ** -21 * mag + 1e-12


@pytest.mark.parametrize("n,heads,pad", [(1, 16, 0), (1, 0, 0), (2, 128, 1), (61, 16, 7), (300, 5, 0), (2048, 3, 500)])
@pytest.mark.parametrize("axes,interleaved", [(1, True), (3, False)])
def test_rope_kv_write(n, heads, pad, axes, interleaved):
    g = torch.Generator().manual_seed(n + heads)
    slots_n = 4096
    slots = torch.randperm(slots_n - 1, generator=g)[:n] + 1
    lat = torch.randn((n, 512), generator=g).to(torch.bfloat16)
    k = torch.randn((n, 64), generator=g).to(torch.bfloat16)
    drop = torch.randperm(n, generator=g)[:pad]
    slots[drop] = torch.tensor([0, -1, -5])[torch.arange(pad) % 3]
    lat[drop] = float("nan")
    k[drop] = float("nan")
    pos = torch.randint(0, 200000, (axes, n), generator=g).to(torch.int32)
    q = torch.randn((n, max(heads, 1), 192), generator=g).to(torch.bfloat16)
    spec = M.rope_spec(INV, AXES[axes], interleaved=interleaved)
    cache = torch.full((slots_n, 656), 0xA5, dtype=torch.uint8, device=D)
    qo = torch.zeros((n, max(heads, 1), 576), dtype=torch.bfloat16, device=D)
    kw = dict(q_pe=q.to(D)[..., 128:], q_out=qo[..., 512:]) if heads else {}
    M.mla_rope_kv_write(cache, slots.to(D), lat.to(D), k.to(D), pos.to(D), spec, **kw)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    # bit for bit what mla_kv_write makes of the rotated values, which the oracle knows
    turned = M.mla_rope(torch.nan_to_num(k).to(D), pos.to(D), spec)
    ref, mag = P.rotate(torch.nan_to_num(k).double()[:, None], pos, INV, AXES[axes], interleaved)
    close(turned[:, None], ref, mag)
    want = np.full((slots_n, 656), 0xA5, np.uint8)
    oracle.kv_write(want, slots.numpy(), lat, turned.cpu())
    assert np.array_equal(cache.cpu().numpy(), want)
    if heads:
        rq, mq = P.rotate(q[..., 128:].double(), pos, INV, AXES[axes], interleaved)
        close(qo[..., 512:], rq, mq)
        assert (qo[..., :512] == 0).all()


def test_rope_kv_write_flags_a_slot_past_the_cache():
    cache = torch.zeros((16, 656), dtype=torch.uint8, device=D)
    one = torch.ones((1, 64), dtype=torch.bfloat16, device=D)
    spec = M.rope_spec(INV)
    M.mla_rope_kv_write(cache, torch.tensor([16], device=D), torch.ones((1, 512), dtype=torch.bfloat16, device=D), one,
                        torch.zeros(1, dtype=torch.int32, device=D), spec)
    assert M.mla_get_error() == M.MLA_ERR_WRITE_SLOT_RANGE
    assert (cache == 0).all()


def test_rope_refuses_bad_views():
    spec = M.rope_spec(INV, AXES[3])
    x = torch.zeros((4, 2, 72), dtype=torch.bfloat16, device=D)
    pos = torch.zeros((3, 4), dtype=torch.int32, device=D)
    with pytest.raises(M.MlaError):
        M.mla_rope(x[..., 4:68], pos, spec, out=torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=D))   # 8-byte aligned
    with pytest.raises(M.MlaError):
        odd = torch.zeros((4, 2, 68), dtype=torch.bfloat16, device=D)[..., :64]                            # head stride 68
        M.mla_rope(odd, pos, spec)
    with pytest.raises(ValueError):
        M.mla_rope(x[..., :64], pos[:2], spec)                                                              # axes missing
    with pytest.raises(ValueError):
        M.mla_rope(x[..., :64].cpu(), pos, spec)
    with pytest.raises(ValueError):
        M.mla_rope(x[..., :60], pos, spec)


def test_rope_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((40, 16, 64), generator=g).to(torch.bfloat16).to(D)
    pos = torch.randint(0, 9000, (1, 40), generator=g).to(torch.int32).to(D)
    spec = M.rope_spec(INV, interleaved=True)
    want = M.mla_rope(x, pos, spec)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(want)
    M.mla_rope(x, pos, spec, out=got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        M.mla_rope(x, pos, spec, out=got)
    pos.add_(7)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, M.mla_rope(x, pos, spec))


def test_nothing_to_do_and_one_dimensional_positions():
    spec = M.rope_spec(INV)
    pos = torch.arange(5, dtype=torch.int32, device=D)
    assert M.mla_rope(torch.empty((0, 3, 64), dtype=torch.bfloat16, device=D), pos[:0], spec).shape == (0, 3, 64)
    assert M.mla_rope(torch.empty((5, 0, 64), dtype=torch.bfloat16, device=D), pos, spec).shape == (5, 0, 64)
    x = torch.randn((5, 64), device=D).to(torch.bfloat16)
    y = M.mla_rope(x, pos, spec)
    ref, mag = P.rotate(x.cpu().double()[:, None], pos.cpu(), INV, AXES[1], False)
    close(y[:, None], ref, mag)
    cache = torch.zeros((16, 656), dtype=torch.uint8, device=D)
    M.mla_rope_kv_write(cache, torch.empty(0, dtype=torch.int64, device=D), torch.empty((0, 512), dtype=torch.bfloat16, device=D),
                        torch.empty((0, 64), dtype=torch.bfloat16, device=D), pos[:0], spec)
    assert (cache == 0).all()
