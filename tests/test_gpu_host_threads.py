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


def at_once(workers, calls):
    """Runs every worker `calls` times in a thread and on a stream of its own; the errors they raised. A call drops Python's
    lock while it is in the library, so one thread may be between a kernel's set-up and its launch while another sets up."""
    errors, start = [], threading.Barrier(len(workers))

    def loop(work):
        stream = torch.cuda.Stream(device=DEV)
        stream.synchronize()
        start.wait()
        try:
            for _ in range(calls):
                work(stream)
        except Exception as e:
            errors.append(e)
        stream.synchronize()
    threads = [threading.Thread(target=loop, args=(w,)) for w in workers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


# one kernel with twice the shared memory for the first shape of each pair: few units, so a CTA has its SM to itself
@pytest.mark.parametrize("shapes", [((1, 2, 256, 2048), (1, 2, 4096, 4096)), ((1, 60, 64, 4096), (2, 100, 2048, 2048))])
def test_forward_calls_with_different_shared_memory(sf, shapes):
    sets = []
    for i, (E, T, R, C) in enumerate(shapes):
        x = normal((T, C), BF, i), normal((E, R, C), BF, i + 5, 0.05), torch.zeros((T, R), dtype=BF, device=DEV), offsets([T // E] * E)
        sets.append((x, sf.grouped_problem(*x)))
    torch.cuda.synchronize()
    assert not at_once([lambda s, p=p: sf.sf_grouped_forward(p, stream=s) for _, p in sets], 4000)
    for (A, W, Y, off), _ in sets:
        check_forward(A, W, Y, off, Y, BF)


def test_weight_gradients_with_different_shared_memory(sf):
    sets = []
    for i, (T, R, C) in enumerate(((40, 128, 256), (40, 2048, 4096))):
        x = normal((T, C), BF, i), torch.zeros((1, R, C), device=DEV), normal((T, R), BF, i + 5), offsets([T])
        sets.append((x, sf.grouped_problem(*x)))
    torch.cuda.synchronize()
    assert not at_once([lambda s, p=p: sf.sf_grouped_dw(p, stream=s) for _, p in sets], 4000)
    for (A, W, Y, off), _ in sets:
        check_dw(A, W, Y, off, None, F32)


def test_updates_with_different_shared_memory(sf):
    """The update parks a row in shared memory: 44 KB for 11,008 columns, 64 KB for 16,384."""
    sets = []
    for C in (11008, 16384):
        m = sf.Matrix(32, C, 32, DEV)
        sf.sf_mask_init(m.mask)
        sf.sf_quantize_init(normal((32, C), F32, C), m)
        sf.sf_mask_update([m.mask], [sf.make_src(sf.SF_SRC_WORDS, torch.full((1,), -1, dtype=torch.int32, device=DEV))], 0.01)
        m.grad.zero_()
        sets.append((m, [sf.matrix_struct(m)], sf.AdamParams(lr=1e-3), sf.status_word()))
    torch.cuda.synchronize()
    assert not at_once([lambda s, x=x: sf.sf_sparse_update(x[1], x[2], x[3], stream=s) for x in sets], 4000)
    assert all(int(x[3]) == 0 for x in sets)
