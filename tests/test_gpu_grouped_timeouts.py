"""Bounded waits of the expert-grouped products. With SF_TEST_GROUPED_WITHHOLD set, the barrier of CTA 0's first pipeline stage
expects one arrival too many: the waits for that stage run out after their limit (2 s), what depends on it is not stored, the call reports
SF_STATUS_WAIT_TIMEOUT, and the next call on the same context is right again."""
import time

import pytest
import torch

from tests.test_gpu_grouped import check_dw, check_dx, check_forward, normal, offsets, rounding, spans

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def right(got, ref, size, n, dt):
    """Where `got` is within the tolerance of test_gpu_grouped.py."""
    slack = (n / 16 + 32) * 2.0 ** -23 * size
    return (got.double() - ref).abs() <= slack + rounding(ref.abs() + slack, dt)


def withheld(monkeypatch, sf, call):
    """A call whose waits run out, from start to end; then the next one, on a status word of its own."""
    monkeypatch.setenv("SF_TEST_GROUPED_WITHHOLD", "1")
    status, t0 = sf.status_word(), time.perf_counter()
    call(status)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    monkeypatch.delenv("SF_TEST_GROUPED_WITHHOLD")
    assert int(status) == sf.SF_STATUS_WAIT_TIMEOUT and 1.5 < took < 30.0


# single CTAs: whole sums, several units to a CTA, sums in slices; slices over clusters; CTA pairs
@pytest.mark.parametrize("counts,R,C", [([12] * 8, 4104, 2568), ([64] * 64, 1024, 1024), ([30] * 3, 4104, 264), ([2], 256, 4096),
                                        ([100, 0, 90], 264, 2568), ([160] * 8, 2568, 2056)])
def test_forward(sf, monkeypatch, counts, R, C):
    T = sum(counts)
    A, W, Y = normal((T, C), BF, 1), normal((len(counts), R, C), BF, 2, 0.05), normal((T, R), BF, 3)
    off, before = offsets(counts), Y.clone()
    p = sf.grouped_problem(A, W, Y, off)
    withheld(monkeypatch, sf, lambda status: sf.sf_grouped_forward(p, status))
    left = Y == before
    for e, a, b in spans(off):
        x, w = A[a:b].double(), W[e].double().t()
        assert bool((left[a:b] | right(Y[a:b], x @ w, x.abs() @ w.abs(), C, BF)).all())
    assert bool(left[:, :32].all(1).any()) and not bool(left.all())         # CTA 0 has the first rows of an expert
    status = sf.status_word()
    sf.sf_grouped_forward(p, status)
    check_forward(A, W, Y, off, before, BF)
    assert int(status) == 0


@pytest.mark.parametrize("counts,R,C", [([2], 4096, 256), ([160] * 8, 2056, 2568)])
def test_dx(sf, monkeypatch, counts, R, C):
    T = sum(counts)
    A, W, Y = normal((T, C), BF, 1), normal((len(counts), R, C), BF, 2, 0.05), normal((T, R), BF, 3)
    off, before = offsets(counts), A.clone()
    p = sf.grouped_problem(A, W, Y, off)
    withheld(monkeypatch, sf, lambda status: sf.sf_grouped_dx(p, status))
    left = A == before
    for e, a, b in spans(off):
        y, w = Y[a:b].double(), W[e].double()
        assert bool((left[a:b] | right(A[a:b], y @ w, y.abs() @ w.abs(), R, BF)).all())
    assert bool(left[:, :32].all(1).any()) and not bool(left.all())
    status = sf.status_word()
    sf.sf_grouped_dx(p, status)
    check_dx(A, W, Y, off, before, BF)
    assert int(status) == 0


# single CTAs: whole sums, slices over clusters (one and several rounds of them); CTA pairs: many tokens, few of them (the
# withheld stage is one whose last rows are cleared), added to in shared memory
@pytest.mark.parametrize("counts,R,C,add", [([40], 2048, 2048, False), ([8192], 64, 512, True), ([65001], 128, 128, False),
                                            ([160] * 8, 2568, 2056, False), ([60] * 8, 2568, 2056, False), ([160] * 8, 2568, 2056, True)])
def test_dw(sf, monkeypatch, counts, R, C, add):
    T = sum(counts)
    A, Y, W = normal((T, C), BF, 1), normal((T, R), BF, 2, 0.05), normal((len(counts), R, C), F32, 3)
    off, before = offsets(counts), W.clone()
    p = sf.grouped_problem(A, W, Y, off)
    withheld(monkeypatch, sf, lambda status: sf.sf_grouped_dw(p, status, accumulate=add))
    left = W == before
    for e, a, b in spans(off):
        y, x = Y[a:b].double(), A[a:b].double()
        ref, size = y.t() @ x + add * before[e].double(), y.abs().t() @ x.abs() + add * before[e].double().abs()
        assert bool((left[e] | right(W[e], ref, size, b - a, F32)).all())
    assert bool(left[:, :32, :64].flatten(1).all(1).any()) and not bool(left.all())
    W.copy_(before)
    status = sf.status_word()
    sf.sf_grouped_dw(p, status, accumulate=add)
    check_dw(A, W, Y, off, before if add else None, F32)
    assert int(status) == 0
