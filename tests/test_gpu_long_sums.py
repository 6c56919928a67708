"""Weight gradients in 16 bits over many tokens: the tensor cores add with truncation, so that a sum that is not cut drifts by
more than its rounding."""
import pytest
import torch

from tests.test_gpu_grouped import normal, offsets

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16
ROWS = 2 ** 16                                 # the tokens are the same again and again


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("counts,R,C,kernel", [
    ([2 ** 26], 8, 8, "CLUSTERS"), ([2 ** 23], 64, 136, "CLUSTERS"), ([2 ** 22, 0, 5, 2 ** 22 + 2 ** 16], 264, 392, "SLICES"),
    ([2 ** 21 + 2 ** 20], 1032, 520, "PAIRS"), ([3 * 2 ** 16, 2 ** 17] + [0] * 200, 72, 264, "PAIRS")])
def test_sums_of_one_sign(sf, counts, R, C, kernel, dt):
    """All products are positive. A sum of up to 8,192 tokens is off by a step (2^-23) for each of its 512 additions at most, the sums
    of those (and of 32 slices) by one for each of theirs, and the result by half a step of its type."""
    T, E = sum(counts), len(counts)
    a, y = normal((ROWS, C), dt, 1, 0.1).abs(), normal((ROWS, R), dt, 2, 0.1).abs()
    A, Y, W = a.repeat(-(-T // ROWS), 1)[:T], y.repeat(-(-T // ROWS), 1)[:T], torch.zeros((E, R, C), dtype=dt, device=DEV)
    if dt == HF:
        A.mul_(2.0 ** -8)                      # the sums stay below 65,504
        a.mul_(2.0 ** -8)
    off, status = offsets(counts), sf.status_word()
    p = sf.grouped_problem(A, W, Y, off)
    assert sf.sf_grouped_kernel(p, sf.SF_GROUPED_DW) == getattr(sf, "SF_GROUPED_" + kernel)
    sf.sf_grouped_dw(p, status)
    once, at = y.double().t() @ a.double(), 0
    for e, n in enumerate(counts):
        rest = torch.arange(at + n // ROWS * ROWS, at + n, device=DEV) % ROWS      # any ROWS tokens in a row sum to the same
        ref = once * (n // ROWS) + y[rest].double().t() @ a[rest].double()
        at += n
        tol = (512 + 32 + (n / 960 if kernel == "PAIRS" else n / 32 / 8192) + 2) * 2.0 ** -23 + torch.finfo(dt).eps / 2
        tiny = torch.finfo(dt).tiny * torch.finfo(dt).eps / 2
        off_by = (W[e].double() - ref).abs()
        assert bool((off_by <= tol * ref + tiny).all()), f"off by {float((off_by / ref.clamp(min=1e-30)).max()):.3g}, {tol:.3g} allowed"
    assert int(status) == 0
