"""Paged cache on the CPU: layouts whose rows share memory are refused where the
call writes them, and layouts that only look unusual are taken (refused by nothing
but the absence of a GPU)."""
import itertools

import pytest

import block_sparse_local_b200 as sta
from block_sparse_local_b200 import build as sta_build
from tests.test_kv_host import _append, _attend, _i64


@pytest.fixture(scope="module")
def L():
    sta_build.build()
    return sta.lib()


IN = (1 << 20, 1 << 14, 128)


def _overlaps(strides, sizes, inner):
    """Whether two rows of `inner` elements share one, by listing all of them."""
    at = sorted(sum(i * s for i, s in zip(idx, strides))
                for idx in itertools.product(*map(range, sizes)))
    return any(b - a < inner for a, b in zip(at, at[1:]))


# q_out and out, [B = 2, hq = 8, S = 3] rows of 128
OUT = [
    (1 << 20, 128, 128), (128, 3 * 128, 128), (8 * 128, 128, 128), (128, 256, 1920),
    (3 * 8 * 128 - 128, 3 * 128, 128), (1 << 20, 256, 128), (1 << 20, 128, 7 * 128),
    (1 << 62, 1 << 62, 128 + (1 << 62)),
]


@pytest.mark.parametrize("st", OUT, ids=str)
def test_rows_of_the_output_that_share_memory_are_refused(L, st):
    if max(st) < 1 << 60:
        assert _overlaps(st, (2, 8, 3), 128)
    assert _append(L, st=_i64(*IN * 3, *st)) == 1
    assert _attend(L, st=_i64(*IN, *st)) == 1


# blocks and heads of the cache, [20][8] of 64 x 128
CACHE = [(8192, 8192), (8192, 16384), (7 * 8192, 8192), (8192, 19 * 8192)]


@pytest.mark.parametrize("operand", [0, 1])
@pytest.mark.parametrize("st", CACHE, ids=str)
def test_append_refuses_blocks_that_share_memory(L, st, operand):
    assert _overlaps(st, (20, 8), 8192)
    good = (1 << 16, 8192)
    cst = _i64(*(st + good if operand == 0 else good + st))
    assert _append(L, cst=cst) == 1


GOOD_OUT = [(3 * 8 * 128, 128, 8 * 128), (3 * 8 * 128, 3 * 128, 128), (128, 6 * 128, 256),
            (128, 256, 16 * 128), (3 * 128, 6 * 128, 128), (1 << 40, 1 << 36, 136)]
GOOD_CACHE = [(8 * 8192, 8192), (8192, 20 * 8192), (2 * 8 * 8192, 2 * 8192), (1 << 17, 8208)]


@pytest.fixture
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers")


def test_layouts_without_overlap_are_taken(L, no_gpu):
    for st in GOOD_OUT:
        assert not _overlaps(st, (2, 8, 3), 128)
        assert _append(L, st=_i64(*IN * 3, *st)) == 3       # STA_ERR_CUDA: no device here
        assert _attend(L, st=_i64(*IN, *st)) == 3
    for st in GOOD_CACHE:
        assert not _overlaps(st, (20, 8), 8192)
        assert _append(L, cst=_i64(*st, *st)) == 3
        assert _attend(L, cst=_i64(*st, *st)) == 3
    # what is only read may repeat itself: inputs, and a dimension of one is free
    assert _append(L, st=_i64(0, 0, 0, 0, 128, 0, 0, 0, 0, *IN)) == 3
    assert _append(L, S=1, st=_i64(*IN * 3, 1 << 14, 128, 0), width=8) == 3
    assert _attend(L, st=_i64(0, 0, 0, *IN)) == 3
