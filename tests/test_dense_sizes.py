"""The sizes up to which the dense step and its norm take a call (CPU: refused before CUDA is touched)."""
import ctypes

import pytest
import torch

from masked_optimizer_step_b200 import binding as b
from tests.test_dense_validation import P, _dense, _step, lib  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device pointers: host validation only")

UNSUPPORTED = -3


@pytest.mark.parametrize("lengths", [[2 ** 40 + 1], [5, 2 ** 40 - 4], [2 ** 39, 2 ** 39, 1], [2 ** 62, 2 ** 62, 2 ** 62]])
def test_more_than_two_to_the_40_elements_are_refused_whole(lib, lengths):  # noqa: F811
    """Before any launch: the first tensors, with fp32 moments, would be launched ahead of the last ones with 8-bit moments."""
    ts = [_dense(n=n, state_type=3 if i == len(lengths) - 1 else 0) for i, n in enumerate(lengths)]
    assert _step(lib, ts) == UNSUPPORTED
    arr = (b.sf_dense * len(ts))(*ts)
    need = lib.sf_grad_norm_ws_bytes(arr, len(ts))
    assert lib.sf_grad_norm(arr, len(ts), 1.0, 1.0, P, P, need, None, None) == UNSUPPORTED
