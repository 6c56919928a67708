"""The sizes up to which the expert-grouped products take a call (CPU: refused before CUDA is touched)."""
import ctypes

import pytest
import torch

from masked_optimizer_step_b200 import binding as b
from tests.test_grouped_validation import UNSUPPORTED, _problem, lib  # noqa: F401

MOST = 2 ** 30


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device pointers: host validation only")
@pytest.mark.parametrize("call", ["sf_grouped_forward", "sf_grouped_dx", "sf_grouped_dw"])
@pytest.mark.parametrize("kw", [dict(T=MOST + 1), dict(T=2 ** 31 - 1), dict(T=2 ** 31 - 2 ** 22), dict(T=1, C=MOST + 8, ld_a=MOST + 8, ld_w=MOST + 8),
                                dict(T=1, R=MOST + 8, ld_y=MOST + 8), dict(T=1, R=2 ** 31 - 8, ld_y=2 ** 31)])
def test_counts_that_do_not_round_up_in_32_bits(lib, call, kw):  # noqa: F811
    f = dict(E=1, R=8, C=8, ld_a=8, ld_w=8, ld_y=8)
    f.update(kw)
    args = [ctypes.byref(_problem(**f))] + ([0] if call == "sf_grouped_dw" else []) + [None, None]
    assert getattr(lib, call)(*args) == UNSUPPORTED


@pytest.mark.parametrize("T,R,C", [(MOST + 1, 8, 8), (2 ** 31 - 1, 8, 8), (8, MOST + 8, 8), (8, 8, MOST + 8)])
def test_the_binding_refuses_them(T, R, C):
    def meta(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="meta")
    off = torch.zeros(2, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="at most 2\\^30"):
        b.grouped_problem(meta(T, C), meta(1, R, C), meta(T, R), off)


def _tile_tokens(cnt, most, step):
    tiles = -(-cnt // most)
    return (-(-cnt // tiles) + step - 1) // step * step


@pytest.mark.parametrize("cnt", [1, 511, MOST - 1, MOST])
@pytest.mark.parametrize("most", [16, 64, 512])
def test_tiles_of_the_largest_counts_fit_32_bits(cnt, most):
    """What the kernels add up on the way to an expert's tiles, each below 2^31."""
    tiles = -(-cnt // most)
    tile = _tile_tokens(cnt, most, 16 if most < 64 else 32)
    n = -(-cnt // tile)
    for x in (cnt + most - 1, cnt + tiles - 1, tile + 31, cnt + tile - 1, cnt + 63, n * tile, n * (tile // 32 + 4)):
        assert x < 2 ** 31
    assert tile <= most and n <= tiles


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device pointers: host validation only")
def test_the_kernels_query_refuses_what_the_calls_refuse(lib):  # noqa: F811
    from tests.test_grouped_validation import REFUSED
    for product in (0, 1, 2):
        for case, kw, code in REFUSED:
            assert lib.sf_grouped_kernel(ctypes.byref(_problem(**kw)), product, 0) == code, case
        assert lib.sf_grouped_kernel(None, product, 0) == -1
    assert lib.sf_grouped_kernel(ctypes.byref(_problem()), 3, 0) == -1
    assert lib.sf_grouped_kernel(ctypes.byref(_problem()), 2, 1) == -1
    assert lib.sf_grouped_kernel(ctypes.byref(_problem(T=0)), 0, 0) == b.SF_GROUPED_NONE
