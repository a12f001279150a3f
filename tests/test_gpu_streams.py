"""Where a call without outputs and workspace makes them: on the stream that it is given."""
import math

import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

import _plain as P

pytestmark = pytest.mark.gpu
D = "cuda:0"


def test_the_stream_given_is_the_one_memory_is_made_on():
    side = torch.cuda.Stream()
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            for stream, handle in ((None, current.cuda_stream), (0, 0), (torch.cuda.default_stream(), 0),
                                   (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
                with M._on(stream):
                    assert torch.cuda.current_stream().cuda_stream == handle
                assert M._stream(stream) == handle


def test_the_default_stream_by_its_handle_0():
    """From within another stream, while the default one is busy: nothing overtakes, and tokens outside every
    sequence are zeros."""
    g = torch.Generator().manual_seed(1)
    cache = P.make_cache(20 * 16, 656, g)
    table = torch.arange(1, 19, dtype=torch.int32).view(2, 9)
    q = torch.randn((9, 16, 576), generator=g).to(torch.bfloat16)
    start, lens = torch.tensor([0, 1, 7], dtype=torch.int32), torch.tensor([140, 99], dtype=torch.int32)
    args = [t.to(D) for t in (q, cache, start, lens, table)]
    x, pos = torch.randn((50, 64), device=D).to(torch.bfloat16), torch.arange(50, dtype=torch.int32, device=D)
    spec = M.rope_spec([10000.0 ** (-i / 32) for i in range(32)])
    want = M.mla_rope(x, pos, spec)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(3):
            with torch.cuda.stream(torch.cuda.default_stream()):
                torch.cuda._sleep(5_000_000)
            out, lse = M.mla_chunk_attention(*args, 16, 1 / 24, stream=0)
            y = M.mla_rope(x, pos, spec, stream=0)
            torch.cuda.default_stream().synchronize()
            P.check_chunk(out, lse, P.chunk(q, cache, start, lens, table, 16, 1 / 24))
            assert (out[7:] == 0).all() and (lse[7:] == -math.inf).all()
            assert torch.equal(y, want)
