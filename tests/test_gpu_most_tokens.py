"""The expert-grouped products over as many tokens as a call takes, 2^30 of them, in the narrowest rows."""
import pytest
import torch

from tests.test_gpu_grouped import check, normal, offsets

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
T, N, ROWS = 2 ** 30, 8, 2 ** 18                 # the tokens are the same 2^18 again and again


def again(base):
    return base.repeat(T // ROWS, 1)


def all_like_the_first(x):
    first = x[:ROWS].reshape(1, -1)
    return all(bool((part == first).all()) for part in x.view(T // ROWS, -1).split(512))


def test_two_to_the_30_tokens(sf):
    a, y, W = normal((ROWS, N), BF, 1), normal((ROWS, N), BF, 2), normal((1, N, N), BF, 3)
    off, status, w = offsets([T]), sf.status_word(), W[0].double()
    A, Y = again(a), torch.zeros((T, N), dtype=BF, device=DEV)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off), status)
    check(Y[:ROWS], a.double() @ w.t(), a.double().abs() @ w.t().abs(), N, BF)
    assert all_like_the_first(Y)                # a row's sum is the same wherever it lies
    Y.copy_(again(y))
    A.zero_()
    sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off), status)
    check(A[:ROWS], y.double() @ w, y.double().abs() @ w.abs(), N, BF)
    assert all_like_the_first(A)
    A.copy_(again(a))
    for G in (torch.zeros((1, N, N), device=DEV), torch.ones((1, N, N), device=DEV)):
        add = bool(G.any())
        sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off), status, accumulate=add)
        ref, size = y.double().t() @ a.double() * (T // ROWS) + int(add), y.double().abs().t() @ a.double().abs() * (T // ROWS) + int(add)
        # sums of 960 tokens (60 additions on the tensor cores), 32 slices of tokens whose sums are added for each 960 of a slice:
        # every addition is off by one step (2^-23) of what it has added so far, at most
        assert bool(((G[0].double() - ref).abs() <= (60 + 32 + T / 32 / 960 + 2) * 2.0 ** -23 * size).all())
    assert int(status) == 0
