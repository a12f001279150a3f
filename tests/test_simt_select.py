"""mla_block_select's kernels run on the CPU from their own source, thread by thread, with the warps of a CTA in orders in which
one is as far ahead of the others, or behind them, as its barriers allow."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import _plain_blocks as B
from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_mla_kv_gb300", "csrc")
SIMT = os.path.join(ROOT, "tests", "simt")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    # The sources beside a device header that stands in for the library's.
    d = tmp_path_factory.mktemp("simt")
    for f in (os.path.join(CSRC, "mla_block.cu"), os.path.join(CSRC, "mla_seq.cuh"), os.path.join(SIMT, "mla_device.cuh")):
        shutil.copy(f, d)
    (d / "all.cpp").write_text('#include "mla_block.cu"\n' + open(os.path.join(SIMT, "run.cpp")).read())
    so = str(d / "libselect.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-w", "-I", os.path.join(ROOT, "include"), str(d / "all.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so)


def select(lib, b, scores, width, sink, local, order):
    blocks = torch.full((b["T"], width), -9, dtype=torch.int32)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    lib.simt_order(order)
    rc = lib.mla_block_select(p(scores), b["T"], scores.shape[1], p(b["q_start"]), p(b["kv_len"]), b["kv_len"].numel(), b["page"],
                              sink, local, width, p(blocks), None)
    assert rc == 0, "warps that wait for each other at different barriers"
    assert lib.simt_error() == 0
    return blocks.tolist()


def lists(b, scores, width, sink, local):
    return [[-9] * width if r is None else r for r in B.select(b, scores, width, sink, local)]


# 0, 1: warps in ascending or descending order; 2 + k: warp k last
@pytest.mark.parametrize("order", [0, 1, 2, 4])
@pytest.mark.parametrize("blocks", [300, 513, 1024, 1100, 4100])
@pytest.mark.parametrize("ties", [False, True])
def test_no_order_of_warps_changes_a_list(lib, blocks, order, ties):
    b = B.batch([(2, blocks), (1, blocks // 3), (1, 3)], 1, 512, 1, 528, seed=blocks, extra=0, tail_tokens=1)
    g = torch.Generator().manual_seed(blocks)
    scores = torch.randn((b["T"], blocks), generator=g)
    # each warp of a CTA (32 neighbouring columns) has scores of a size of its own: their bits that differ are others
    scores *= 2.0 ** ((torch.arange(blocks) // 32) % 4 * 9 - 20)
    if ties:
        scores = torch.where(scores.abs() < 1e-4, torch.zeros_like(scores), scores.sign())
    for width, sink, local in ((1, 0, 1), (48, 1, 2), (200, 0, 1)):
        assert select(lib, b, scores, width, sink, local, order) == lists(b, scores, width, sink, local)


@pytest.mark.parametrize("order", [0, 1, 5])
def test_no_order_of_warps_changes_a_list_that_is_read_again(lib, order):
    blocks = 8200                                       # past what the CTA's registers hold
    b = B.batch([(1, blocks)], 1, 512, 1, 528, seed=3, extra=0)
    scores = torch.randn((1, blocks), generator=torch.Generator().manual_seed(4))
    assert select(lib, b, scores, 64, 1, 2, order) == lists(b, scores, 64, 1, 2)


@pytest.mark.parametrize("per", [1, 8, 128, 8192, 268435520, 2 ** 31 - 4097])
@pytest.mark.parametrize("n", [0, 1, 127, 128, 129, 8193, 2 ** 31 - 8192, 2 ** 31 - 4097])
def test_parts_of_the_longest_tables(lib, n, per):
    """Chunks of a token's blocks, CTAs of a tile's: tables may have up to 2^31 - 4097 blocks (of one position)."""
    assert lib.simt_parts(n, per) == -(-n // per)
