"""mla_chunk_attention against the formula in 64 bits, at the sizes and masks where it can go wrong."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"


WIDE = False


@pytest.fixture(params=["narrow", "wide"], autouse=True)
def table_width(request):
    """A batch with 48 rows a sequence goes to the kernel for many rows only where its contexts' capacity is large, so
    every test runs with a table just wide enough and with one of many unused columns."""
    global WIDE
    WIDE = request.param == "wide"


def batch(seqs, H, d_qk, page, row, seed=0, extra=2, tail_tokens=0, outliers=False):
    """seqs: (new tokens, context length). Pages in random order, page 0 unused."""
    rows = (sum(n for n, _ in seqs) + tail_tokens) * H
    if WIDE and extra and rows >= 48 * len(seqs):
        extra += 8_000_000 // (rows * page) + 1
    g = torch.Generator().manual_seed(seed)
    pages = [-(-L // page) for _, L in seqs]
    total = sum(pages) + 3
    cache = P.make_cache(total * page, row, g, rope=d_qk == 576, outliers=outliers)
    order = torch.randperm(total - 1, generator=g).to(torch.int32) + 1
    table = torch.full((len(seqs), max(pages + [0]) + extra), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(pages):
        table[i, :k] = order[at:at + k]
        at += k
    start = [0]
    for n, _ in seqs:
        start.append(start[-1] + n)
    T = start[-1] + tail_tokens
    q = torch.randn((T, H, d_qk), generator=g).to(torch.bfloat16)
    return dict(q=q, cache=cache, q_start=torch.tensor(start, dtype=torch.int32),
                kv_len=torch.tensor([L for _, L in seqs], dtype=torch.int32), table=table, page=page,
                scale=1.0 / math.sqrt(d_qk))


def call(b, causal=True, **kw):
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    out, lse = M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], t["page"], t["scale"],
                                     causal=causal, **kw)
    torch.cuda.synchronize()
    return out, lse


def ref(b, causal=True):
    return P.chunk(b["q"], b["cache"], b["q_start"], b["kv_len"], b["table"], b["page"], b["scale"], causal)


def run(b, causal=True, error=0):
    out, lse = call(b, causal)
    assert M.mla_get_error() == error
    P.check_chunk(out, lse, ref(b, causal))
    return out, lse


SHAPES = [
    [(1, 1)], [(1, 2)], [(1, 31)], [(1, 32)], [(1, 33)], [(1, 64), (1, 1)], [(1, 129), (1, 700), (1, 65)],
    [(2, 2)], [(7, 7)], [(8, 8), (9, 9)], [(16, 300)], [(17, 33), (1, 5), (40, 41)], [(33, 200), (64, 64)],
    [(1, 3000)], [(3, 1500), (1, 257)],
]


@pytest.mark.parametrize("seqs", SHAPES, ids=str)
@pytest.mark.parametrize("H,d_qk,row,page", [(16, 576, 656, 64), (5, 512, 528, 16), (128, 576, 656, 48)])
def test_shapes(seqs, H, d_qk, row, page):
    run(batch(seqs, H, d_qk, page, row, seed=len(seqs) * 7 + H))


@pytest.mark.parametrize("H", [1, 3, 16, 31, 64, 100])
@pytest.mark.parametrize("causal", [True, False])
def test_heads(H, causal):
    run(batch([(9, 150), (1, 40), (20, 90)], H, 576, 32, 656, seed=H), causal)


@pytest.mark.parametrize("page", [1, 2, 31, 32, 33, 128, 1000])
@pytest.mark.parametrize("d_qk,row", [(576, 656), (512, 656), (512, 528)])
def test_pages_that_end_inside_a_tile(page, d_qk, row):
    run(batch([(5, 333), (1, 70), (12, 64)], 16, d_qk, page, row, seed=page))


@pytest.mark.parametrize("causal", [True, False])
def test_empty_sequences_rows_and_tokens_outside(causal):
    # no new tokens, no context, fewer positions than tokens (the first rows attend nothing), tokens behind the last
    b = batch([(0, 50), (3, 0), (10, 4), (0, 0), (4, 4), (130, 3)], 16, 576, 16, 656, seed=1, tail_tokens=3)
    out = torch.full((b["q"].shape[0], 16, 512), 3.0, dtype=torch.bfloat16, device=D)
    lse = torch.full((b["q"].shape[0], 16), 5.0, device=D)
    call(b, causal, out=out, lse=lse)
    assert M.mla_get_error() == 0
    P.check_chunk(out, lse, ref(b, causal))
    assert (out[-3:] == 3.0).all() and (lse[-3:] == 5.0).all()


@pytest.mark.parametrize("n_seq", [33, 64, 65, 130, 700])
@pytest.mark.parametrize("H", [2, 64])
def test_many_sequences(n_seq, H):
    """Around the batch sizes that are planned in each CTA (64) and by a kernel of their own."""
    g = torch.Generator().manual_seed(n_seq)
    seqs = [(int(torch.randint(0, 3, (1,), generator=g)), int(torch.randint(0, 120, (1,), generator=g))) for _ in range(n_seq)]
    seqs[n_seq // 2] = (2, 2000)                            # one long context among short ones
    run(batch(seqs, H, 576, 16, 656, seed=n_seq))


def test_nothing_in_the_table():
    b = batch([(2, 100), (70, 300)], 16, 576, 64, 656, seed=2)
    b["table"][:] = -1
    out, lse = run(b)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("n", [1, 12, 40])
def test_holes_reserved_slot_and_slots_past_the_cache(n):
    b = batch([(n, 400), (n, 90)], 16, 576, 16, 656, seed=3)
    b["table"][0, 3] = -1                                   # a hole
    b["table"][0, 5] = 0                                    # holds the reserved slot: slots 1..15 are rows like others
    b["table"][1, 1] = -7
    b["cache"][0] = 0xFF                                    # the reserved slot holds NaN
    run(b)
    b["table"][1, 2] = 1 << 28                              # past the cache: absent and flagged
    run(b, error=M.MLA_ERR_DECODE_INDEX_RANGE)


@pytest.mark.parametrize("n,L", [(1, 200), (24, 200), (70, 200)])
@pytest.mark.parametrize("what", ["code", "scale_inf", "scale_nan", "rope_inf", "rope_nan"])
def test_rows_that_are_not_finite(n, L, what):
    b = batch([(n, L), (n, L)], 16, 576, 16, 656, seed=4)
    bad = []
    for s, p in ((0, L - max(1, n // 2)), (1, 0)):          # seen by half the tokens; by all of them
        slot = int(b["table"][s, p // 16]) * 16 + p % 16
        bad.append(slot)
        if what == "code":
            b["cache"][slot, 77] = 0x7F
        elif what.startswith("scale"):
            b["cache"][slot, 516:520] = torch.tensor([math.inf if "inf" in what else math.nan]).view(torch.uint8)
        else:
            b["cache"][slot, 540:542] = torch.tensor([-math.inf if "inf" in what else math.nan],
                                                     dtype=torch.bfloat16).view(torch.uint8)
    run(b)
    # behind the context: no trace
    b["kv_len"][0] = L - max(1, n // 2)
    run(b)
    # rows of no sequence hold anything at all
    used = set((int(p) * 16 + i) for p in b["table"].flatten().tolist() if p >= 0 for i in range(16))
    rest = [i for i in range(b["cache"].shape[0]) if i not in used]
    b["cache"][rest] = 0xFF
    run(b)


def test_masked_positions_do_not_change_a_bit():
    b = batch([(40, 200), (1, 90)], 16, 576, 16, 656, seed=5)
    out, lse = call(b)
    # the pages' rows behind each context
    for s, L in ((0, 200), (1, 90)):
        for p in range(L, -(-L // 16) * 16):
            b["cache"][int(b["table"][s, p // 16]) * 16 + p % 16] = 0xFF
    o2, l2 = call(b)
    assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


@pytest.mark.parametrize("n", [1, 30])
def test_outliers_and_scores_that_climb(n):
    b = batch([(n, 900)], 16, 576, 64, 656, seed=6, outliers=True)
    b["q"] *= 4
    run(b)
    # each position's score above the last one's, so that the running maximum moves block after block
    b = batch([(n, 900)], 16, 512, 64, 528, seed=7)
    lat = torch.ones((900, 512)) * torch.linspace(0.01, 3.0, 900)[:, None]
    sc = lat.view(900, 4, 128).amax(-1) / 448.0
    for p in range(900):
        slot = int(b["table"][0, p // 64]) * 64 + p % 64
        b["cache"][slot, :512] = (lat[p].view(4, 128) / sc[p][:, None]).to(torch.float8_e4m3fn).view(-1).view(torch.uint8)
        b["cache"][slot, 512:528] = sc[p].contiguous().view(torch.uint8)
    b["q"] = b["q"].abs()
    run(b)


@pytest.mark.parametrize("n", [1, 40])
def test_scales_far_apart(n):
    """Tile scales from 2^-40 to 2^40 in one context, and large queries."""
    b = batch([(n, 150)], 16, 512, 16, 528, seed=8)
    g = torch.Generator().manual_seed(8)
    e = torch.randint(-40, 10, (b["cache"].shape[0], 4), generator=g).double()
    b["cache"][:, 512:528] = torch.pow(2.0, e).float().contiguous().view(torch.uint8)
    b["q"] = (b["q"].double() * 2.0 ** -12).to(torch.bfloat16)
    run(b)


def test_lengths_past_the_table_and_bad_starts_are_flagged():
    b = batch([(4, 64), (70, 64)], 16, 576, 16, 656, seed=9, extra=0)
    b["kv_len"][0] = 70                                     # the table ends at 64: causal limits count from 70
    b["kv_len"][1] = 64
    run(b, error=M.MLA_ERR_CHUNK_RANGE)
    b["kv_len"][0] = -3
    run(b)
    b["q_start"] = torch.tensor([4, 2, 74], dtype=torch.int32)
    out, lse = call(b)
    assert M.mla_get_error() == M.MLA_ERR_CHUNK_RANGE
    P.check_chunk(out, lse, ref(b))
    for starts in ([0, 4, 75], [-1, 4, 74], [0, 74, 0], [5, 4, 74]):
        b["q_start"] = torch.tensor(starts, dtype=torch.int32)
        out, lse = call(b)
        assert M.mla_get_error() == M.MLA_ERR_CHUNK_RANGE
        P.check_chunk(out, lse, ref(b))


def test_starts_that_overlap_are_refused():
    """[0, T, 0, T, ...] names T tokens again and again: only the first is taken."""
    b = batch([(40, 64)], 16, 576, 16, 656, seed=14, extra=0)
    n = 600
    b["q_start"] = torch.tensor([0, 40] * (n // 2) + [40], dtype=torch.int32)
    b["kv_len"] = torch.full((n,), 64, dtype=torch.int32)
    b["table"] = b["table"].expand(n, -1).contiguous()
    out, lse = call(b)
    assert M.mla_get_error() == M.MLA_ERR_CHUNK_RANGE
    P.check_chunk(out, lse, ref(b))


def test_one_graph_serves_other_lengths_and_a_dirty_workspace():
    b = batch([(1, 700), (1, 90), (20, 60)], 16, 576, 16, 656, seed=10)
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    T = t["q"].shape[0]
    ws = M.alloc_chunk_workspace(T, 16, 3)
    out, lse = torch.empty((T, 16, 512), dtype=torch.bfloat16, device=D), torch.empty((T, 16), device=D)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 16, t["scale"], out=out, lse=lse,
                              workspace=ws)
    for lens, starts in (([700, 90, 60], [0, 1, 2, 22]), ([5, 90, 20], [0, 1, 2, 22]), ([650, 0, 40], [0, 15, 15, 22]),
                         ([700, 90, 60], [0, 0, 22, 22])):
        b["kv_len"], b["q_start"] = torch.tensor(lens, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32)
        t["kv_len"].copy_(b["kv_len"])
        t["q_start"].copy_(b["q_start"])
        got = []
        for fill in (0xFF, 0x00):
            ws.fill_(fill)
            out.fill_(math.nan)
            lse.fill_(math.nan)
            gr.replay()
            torch.cuda.synchronize()
            got.append((out.clone(), lse.clone()))
        assert M.mla_get_error() == 0
        P.check_chunk(*got[0], ref(b))
        assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])


def test_agrees_with_the_sparse_decode():
    """One new token per sequence is the sparse decode with every position listed."""
    b = batch([(1, 200), (1, 77), (1, 1)], 16, 576, 16, 656, seed=11)
    out, lse = call(b)
    topk = torch.full((3, 200), -1, dtype=torch.int32)
    for s, L in enumerate((200, 77, 1)):
        topk[s, :L] = torch.arange(L, dtype=torch.int32)
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    o2, l2 = M.mla_sparse_decode_paged(t["q"], t["cache"], topk.to(D), t["table"], 16, t["scale"],
                                       token_seq=torch.arange(3, dtype=torch.int32, device=D))
    _, _, to, tl = ref(b)
    assert ((out.double() - o2.double()).abs().cpu() <= 2 * to).all()
    assert ((lse - l2).abs().double().cpu() <= 2 * tl).all()


def test_on_another_stream():
    b = batch([(3, 500), (1, 90)], 16, 576, 16, 656, seed=12)
    out, lse = call(b)
    s = torch.cuda.Stream()
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    ws = M.alloc_chunk_workspace(4, 16, 2)
    s.wait_stream(torch.cuda.current_stream())
    M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 16, t["scale"], out=o2, lse=l2,
                          workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


def test_a_stream_of_its_own_for_what_the_call_makes():
    """Without out, lse and workspace the call makes them on its stream, behind nothing of the current one."""
    b = batch([(3, 500), (60, 90)], 16, 576, 16, 656, seed=17)
    want, wlse = call(b)
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)                           # the current stream is busy meanwhile
    for stream in (s, s.cuda_stream):
        out, lse = M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 16, t["scale"], stream=stream)
        s.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wlse)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_a_query_row_that_is_not_finite_is_alone(n, value):
    b = batch([(n, 300), (n, 200)], 16, 576, 16, 656, seed=15)
    out, lse = call(b)
    b["q"][n // 2, 3, 100] = value
    o2, l2 = call(b)
    assert M.mla_get_error() == 0
    keep = torch.ones(out.shape[:2], dtype=torch.bool)
    keep[n // 2, 3] = False
    assert torch.equal(out.cpu()[keep].view(torch.int16), o2.cpu()[keep].view(torch.int16))
    assert torch.equal(lse.cpu()[keep], l2.cpu()[keep])
    if math.isnan(value):
        assert torch.isnan(o2[n // 2, 3]).all() and torch.isnan(l2[n // 2, 3])


@pytest.mark.parametrize("n", [1, 40])
def test_query_rows_of_very_different_sizes(n):
    """q rows scaled from 2^-30 to 2^40: each row's exponent shift is its own."""
    b = batch([(n, 300)], 16, 576, 16, 656, seed=16)
    e = torch.linspace(-30, 40, n * 16).view(n, 16, 1).round()
    b["q"] = (b["q"].double() * torch.pow(2.0, e.double())).to(torch.bfloat16)
    b["scale"] = 2.0 ** -12
    run(b)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dim", [5, 300, 570])
@pytest.mark.parametrize("log2", [8, 12, 16, 24])
def test_one_large_value_in_every_query_row(n, dim, log2):
    """Values far below their row's largest: what the many-rows kernel rounds of them (2^-21 of the largest, where
    they are below 2^-13 of it) is within the bound, which is relative to the sum of |q| |K|."""
    b = batch([(n, 300)], 16, 576, 16, 656, seed=17)
    q = b["q"].double()
    q[..., dim] = torch.where(q[..., dim] < 0, -1.0, 1.0) * 2.0 ** log2
    b["q"] = q.to(torch.bfloat16)
    b["scale"] = 2.0 ** -max(5, log2 - 4)
    run(b)


def test_a_cache_whose_offsets_pass_32_bits():
    """Rows beyond 4 GiB of the cache (7 million slots of 656 bytes)."""
    slots, page = 7_000_000, 64
    g = torch.Generator().manual_seed(13)
    cache = torch.zeros((slots, 656), dtype=torch.uint8, device=D)
    rows = P.make_cache(10 * page, 656, g)
    first = slots // page - 10
    cache[first * page:(first + 10) * page] = rows.to(D)
    table = torch.randperm(10, generator=g).to(torch.int32)
    q = torch.randn((50, 16, 576), generator=g).to(torch.bfloat16)
    start, lens = torch.tensor([0, 1, 50], dtype=torch.int32), torch.tensor([300, 320], dtype=torch.int32)
    small = torch.stack([table[:5], table[5:]])
    out, lse = M.mla_chunk_attention(q.to(D), cache, start.to(D), lens.to(D), (small + first).to(D), page, 0.04)
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    # the reference on the ten pages alone, one page further on so that none is the reserved one
    host = torch.cat([torch.zeros((page, 656), dtype=torch.uint8), rows])
    P.check_chunk(out, lse, P.chunk(q, host, start, lens, small + 1, page, 0.04))


def test_refusals():
    b = batch([(1, 20)], 16, 576, 16, 656)
    t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    args = (t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"])
    with pytest.raises(M.MlaError) as e:
        M.mla_chunk_attention(*args, 16, math.nan)
    assert e.value.code == M.MLA_EINVAL
    with pytest.raises(M.MlaError) as e:
        M.mla_chunk_attention(*args, 0, 0.1)
    assert e.value.code == M.MLA_EINVAL
    with pytest.raises(M.MlaError) as e:
        M.mla_chunk_attention(*args, 16, 0.1, workspace=torch.empty(64, dtype=torch.uint8, device=D))
    assert e.value.code == M.MLA_ENOWORKSPACE
    with pytest.raises(ValueError):
        M.mla_chunk_attention(t["q"].cpu(), *args[1:], 16, 0.1)
    with pytest.raises(AssertionError):
        M.mla_chunk_attention(t["q"].repeat(1, 1, 2)[..., :576], *args[1:], 16, 0.1)


@pytest.mark.parametrize("seqs", [[(40, 9000)], [(3, 20000), (40, 700)], [(1, 30000), (1, 5), (9, 12000)]], ids=str)
@pytest.mark.parametrize("row,d_qk", [(656, 576), (528, 512)])
def test_long_contexts_cut_into_pieces(seqs, row, d_qk):
    run(batch(seqs, 16, d_qk, 64, row, seed=18))


@pytest.mark.parametrize("n", [1, 40])
def test_one_high_score_over_many_low_ones(n):
    """Half of the softmax in one position, the other half spread over thousands, each 2^-12 of it and less."""
    b = batch([(n, 4000)], 16, 576, 64, 656, seed=19)
    b["q"] = torch.zeros_like(b["q"])
    b["q"][..., 512] = 1.0
    rope = b["cache"][:, 528:].view(torch.bfloat16)
    rope[:, 0] = 0.0
    page = int(b["table"][0, 20])
    rope[page * 64 + 11, 0] = math.log(4000.0)              # the position 20 * 64 + 11
    b["scale"] = 1.0
    run(b, causal=False)


def test_two_calls_at_once():
    """Many and few rows on two streams over one cache, a workspace each, again and again."""
    b = batch([(40, 900), (40, 1100)], 16, 576, 64, 656, seed=20)
    want = call(b)
    few = dict(b, q=b["q"][:2].contiguous(), q_start=torch.tensor([0, 1, 2], dtype=torch.int32))
    want_few = call(few)
    calls = []
    for c, w in ((b, want), (few, want_few)):
        t = {k: v.to(D) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
        calls.append((torch.cuda.Stream(), t, M.alloc_chunk_workspace(t["q"].shape[0], 16, 2), w, []))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, t, ws, _, got in calls:
            got.append(M.mla_chunk_attention(t["q"], t["cache"], t["q_start"], t["kv_len"], t["table"], 64, t["scale"],
                                             workspace=ws, stream=s))
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    for _, _, _, (wo, wl), got in calls:
        for o, l in got:
            assert torch.equal(o.view(torch.int16), wo.view(torch.int16)) and torch.equal(l, wl)
