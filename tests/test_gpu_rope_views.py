"""mla_rope and mla_rope_kv_write on positions and views that are not laid out row after row."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"
INV = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
AXIS3 = [0] * 8 + [1] * 12 + [2] * 12


@pytest.mark.parametrize("n", [1, 2, 33, 1000])
@pytest.mark.parametrize("interleaved", [True, False])
def test_one_row_of_positions_for_all_axes(n, interleaved):
    """pos.expand(3, n), as text has them in a model with three axes, against the same rows spelled out."""
    g = torch.Generator().manual_seed(n)
    spec = M.rope_spec(INV, AXIS3, interleaved=interleaved)
    x = torch.randn((n, 5, 64), generator=g).to(torch.bfloat16)
    # others' positions lie behind the row
    pos = torch.randint(0, 100000, (4, n), generator=g).to(torch.int32).to(D)
    row = pos[0].expand(3, n)
    assert row.stride(0) == 0
    got = M.mla_rope(x.to(D), row, spec)
    assert torch.equal(got, M.mla_rope(x.to(D), row.contiguous(), spec))
    ref, mag = P.rotate(x.double(), row.cpu(), INV, AXIS3, interleaved)
    assert ((got.double().cpu() - ref).abs() <= P.BF16 * ref.abs() + 2.0 ** -21 * mag + 1e-38).all()
    slots = (torch.randperm(2 * n, generator=g)[:n] + 1).to(D)
    lat = torch.randn((n, 512), generator=g).to(torch.bfloat16).to(D)
    k = torch.randn((n, 64), generator=g).to(torch.bfloat16).to(D)
    made = []
    for p in (row, row.contiguous()):
        cache = torch.zeros((2 * n + 1, 656), dtype=torch.uint8, device=D)
        q = torch.zeros((n, 5, 64), dtype=torch.bfloat16, device=D)
        M.mla_rope_kv_write(cache, slots, lat, k, p, spec, q_pe=x.to(D), q_out=q)
        made.append((cache, q))
    assert M.mla_get_error() == 0
    assert torch.equal(made[0][0], made[1][0]) and torch.equal(made[0][1], made[1][1])
    assert torch.equal(made[0][1], got)


def test_a_column_of_a_wider_table_of_positions():
    """One decode step: [axes, 1] out of [axes, many], and its transposed storage."""
    spec = M.rope_spec(INV, AXIS3)
    pos = torch.randint(0, 100000, (3, 40), generator=torch.Generator().manual_seed(1)).to(torch.int32).to(D)
    x = torch.randn((1, 16, 64), device=D).to(torch.bfloat16)
    want = M.mla_rope(x, pos[:, 7:8].contiguous(), spec)
    for p in (pos[:, 7:8], pos.t().contiguous().t()[:, 7:8]):
        assert torch.equal(M.mla_rope(x, p, spec), want)


def test_views_with_heads_outside_rows_and_heads_that_repeat():
    g = torch.Generator().manual_seed(2)
    spec = M.rope_spec(INV)
    n, heads = 37, 6
    pos = torch.randint(0, 9000, (n,), generator=g).to(torch.int32).to(D)
    x = torch.randn((n, heads, 64), generator=g).to(torch.bfloat16).to(D)
    want = M.mla_rope(x, pos, spec)
    # heads first; in wider buffers; rows with room behind them
    for out in (torch.zeros((heads, n, 64), dtype=torch.bfloat16, device=D).transpose(0, 1),
                torch.zeros((n, heads, 128), dtype=torch.bfloat16, device=D)[..., 64:],
                torch.zeros((heads, n, 200), dtype=torch.bfloat16, device=D)[..., 8:72].transpose(0, 1),
                torch.as_strided(torch.zeros(40000, dtype=torch.bfloat16, device=D), (n, heads, 64), (7 * 64, 64, 1))):
        assert torch.equal(M.mla_rope(x, pos, spec, out=out), want)
    # 3 rows 256 apart, 2 heads 384 apart: neither lies within the other's, and nothing overlaps
    buf = torch.zeros(2048, dtype=torch.bfloat16, device=D)
    out = torch.as_strided(buf, (3, 2, 64), (256, 384, 1))
    assert torch.equal(M.mla_rope(x[:3, :2], pos[:3], spec, out=out), want[:3, :2])
    one = x[:, :1].expand(n, heads, 64)
    assert torch.equal(M.mla_rope(one, pos, spec), want[:, :1].expand(n, heads, 64))
    with pytest.raises(M.MlaError):
        M.mla_rope(one, pos, spec, out=one)
    cache = torch.zeros((64, 656), dtype=torch.uint8, device=D)
    args = (cache, torch.arange(1, n + 1, device=D), torch.zeros((n, 512), dtype=torch.bfloat16, device=D),
            torch.zeros((n, 64), dtype=torch.bfloat16, device=D), pos, spec)
    with pytest.raises(M.MlaError):
        M.mla_rope_kv_write(*args, q_pe=one)
    got = torch.empty((n, heads, 64), dtype=torch.bfloat16, device=D)
    M.mla_rope_kv_write(*args, q_pe=one, q_out=got)
    assert torch.equal(got, want[:, :1].expand(n, heads, 64))


@pytest.mark.parametrize("interleaved", [True, False])
def test_the_inverse_turns_back_by_the_same_angle(interleaved):
    """At any position, near and far: the inverse, the negative frequency and the negative position are one rotation,
    bit for bit."""
    g = torch.Generator().manual_seed(3)
    n = 4000
    x = torch.randn((n, 8, 64), generator=g).to(torch.bfloat16).to(D)
    pos = torch.randint(-(1 << 31) + 1, (1 << 31) - 1, (3, n), generator=g).to(torch.int32)
    pos[:, :100] = torch.arange(100, dtype=torch.int32)
    pos = pos.to(D)
    kw = dict(interleaved=interleaved, scale=0.75)
    want = M.mla_rope(x, -pos, M.rope_spec(INV, AXIS3, **kw))
    assert torch.equal(M.mla_rope(x, pos, M.rope_spec(INV, AXIS3, inverse=True, **kw)), want)
    assert torch.equal(M.mla_rope(x, pos, M.rope_spec([-f for f in INV], AXIS3, **kw)), want)
    assert torch.equal(M.mla_rope(x, -pos, M.rope_spec([-f for f in INV], AXIS3, inverse=True, **kw)), want)
