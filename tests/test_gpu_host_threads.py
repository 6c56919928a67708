"""Calls from other host threads than the first, alone and several at once."""
import threading

import pytest
import torch

from tests.test_gpu_grouped import check_dw, check_dx, check_forward, normal, offsets

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


# single CTAs and CTA pairs of each
@pytest.mark.parametrize("E,T,R,C", [(2, 6, 264, 1032), (2, 700, 2056, 1032)])
@pytest.mark.parametrize("product", ["forward", "dx", "dw"])
def test_the_first_call_of_a_thread(sf, product, E, T, R, C):
    """A new thread has no CUDA context until a call makes the device's own current."""
    A, W, Y, off = normal((T, C), BF, 1), normal((E, R, C), BF, 2, 0.05), normal((T, R), BF, 3), offsets([T // 2, T // 2])
    G = torch.zeros((E, R, C), device=DEV)
    p = sf.grouped_problem(A, G if product == "dw" else W, Y, off)
    stream, errors = torch.cuda.current_stream(), []

    def work():
        try:
            getattr(sf, "sf_grouped_" + product)(p, stream=stream)
        except Exception as e:
            errors.append(e)
    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors
    if product == "forward":
        check_forward(A, W, Y, off, Y, BF)
    elif product == "dx":
        check_dx(A, W, Y, off, A, BF)
    else:
        check_dw(A, G, Y, off, None, F32)
