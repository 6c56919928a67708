"""sf_grouped_forward, sf_grouped_dx and sf_grouped_dw against the sums of include/sf.h in 64 bits.

Tolerance. A product of two 16-bit values is exact in fp32. The tensor core adds 16 of them at a time into an fp32
accumulator; each such addition, and each fp32 addition of partial sums behind it, is off by less than one fp32 step
(2^-23) of the magnitudes it has added so far, which the sum S of the products' magnitudes bounds. So a sum of n products is off
by less than (n / 16 + 32) 2^-23 S, and its rounding to 16 bits by half a step of the result.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def offsets(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def normal(shape, dt, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def rounding(ref, dt):
    return torch.finfo(dt).eps / 2 * ref.abs() + torch.finfo(dt).tiny * torch.finfo(dt).eps / 2


def check(got, ref, size, n, dt):
    """|got - ref| within the module's tolerance; size: the sum of the products' magnitudes."""
    slack = (n / 16 + 32) * 2.0 ** -23 * size
    tol = slack + rounding(ref.abs() + slack, dt)
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol).max()):.3g} of the tolerance"


def spans(off):
    o = off.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def check_forward(A, W, Y, off, before, dt):
    o = off.tolist()
    for e, a, b in spans(off):
        if a < b:
            w = W[e].double()
            x = A[a:b].double()
            check(Y[a:b], x @ w.t(), x.abs() @ w.t().abs(), W.shape[2], dt)
    assert torch.equal(Y[:o[0]], before[:o[0]]) and torch.equal(Y[o[-1]:], before[o[-1]:])


def check_dx(A, W, Y, off, before, dt):
    o = off.tolist()
    for e, a, b in spans(off):
        if a < b:
            w = W[e].double()
            y = Y[a:b].double()
            check(A[a:b], y @ w, y.abs() @ w.abs(), W.shape[1], dt)
    assert torch.equal(A[:o[0]], before[:o[0]]) and torch.equal(A[o[-1]:], before[o[-1]:])


def check_dw(A, W, Y, off, before, out_dt):
    for e, a, b in spans(off):
        ref = Y[a:b].double().t() @ A[a:b].double()
        size = Y[a:b].double().abs().t() @ A[a:b].double().abs()
        if before is not None:
            ref = ref + before[e].double()
            size = size + before[e].double().abs()
        check(W[e], ref, size, max(b - a, 1), out_dt)


# counts by expert, R, C: few tokens (K split over clusters), a token box that an expert overflows, pairs of CTAs
# with one and several token tiles, odd widths, empty experts in front, between and behind
CASES = [
    ([1], 8, 8), ([1], 256, 512), ([1, 0, 1], 136, 1024), ([0, 0, 3], 264, 4096), ([2, 5, 0, 1], 1000, 72),
    ([16, 17, 15], 128, 640), ([40, 1, 0, 0, 3], 392, 200), ([90, 60, 95], 264, 520), ([0, 200, 1, 31], 152, 136),
    ([128], 128, 64), ([255, 257], 256, 256), ([700], 520, 328), ([1025, 3, 512], 264, 1096), ([96, 97, 98, 300], 8, 2056),
    ([0, 1000, 33, 500, 0], 776, 24), ([2100, 17], 136, 72),
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("counts,R,C", CASES)
def test_forward(sf, counts, R, C, dt):
    T = sum(counts)
    A, W = normal((T, C), dt, 1), normal((len(counts), R, C), dt, 2, 0.05)
    Y = normal((T, R), dt, 3)
    off, status, before = offsets(counts), sf.status_word(), Y.clone()
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off), status)
    check_forward(A, W, Y, off, before, dt)
    assert int(status[0]) == 0


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("counts,R,C", CASES)
def test_dx(sf, counts, R, C, dt):
    T = sum(counts)
    Y, W = normal((T, R), dt, 1), normal((len(counts), R, C), dt, 2, 0.05)
    A = normal((T, C), dt, 3)
    off, status, before = offsets(counts), sf.status_word(), A.clone()
    sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off), status)
    check_dx(A, W, Y, off, before, dt)
    assert int(status[0]) == 0


@pytest.mark.parametrize("dt,out,add", [(BF, F32, False), (BF, F32, True), (HF, F32, False), (BF, BF, False),
                                        (HF, HF, False)])
@pytest.mark.parametrize("counts,R,C", CASES)
def test_dw(sf, counts, R, C, dt, out, add):
    T = sum(counts)
    A, Y = normal((T, C), dt, 1), normal((T, R), dt, 2, 0.05)
    W = normal((len(counts), R, C), out, 3)
    off, status, before = offsets(counts), sf.status_word(), W.clone() if add else None
    sf.sf_grouped_dw(sf.grouped_problem(A, W, Y, off), status, accumulate=add)
    check_dw(A, W, Y, off, before, out)
    assert int(status[0]) == 0


@pytest.mark.parametrize("out,add", [(F32, False), (F32, True), (BF, False)])
@pytest.mark.parametrize("counts,R,C", [([700, 301], 2056, 1544), ([1, 0, 1100, 960], 1288, 1800), ([2111], 2312, 2568),
                                        ([64, 0, 961, 1025, 16], 1032, 1352)])
def test_dw_of_many_tiles(sf, counts, R, C, out, add):
    """Enough tokens and tiles for the pairs' kernel: whole and ragged last stages, empty experts, several chunks."""
    test_dw(sf, counts, R, C, BF, out, add)


@pytest.mark.parametrize("counts", [[5000], [3000, 0, 1999, 70]])
@pytest.mark.parametrize("R,C", [(72, 136), (264, 200), (520, 712)])
def test_dw_of_few_tiles_and_long_sums(sf, counts, R, C):
    """Few tiles and many tokens: sums in slices, several chunks of each."""
    test_dw(sf, counts, R, C, HF, F32, True)
    test_dw(sf, counts, R, C, BF, BF, False)


def strided(shape, dt, seed, pad, lead=0):
    """A view whose rows are pad elements further apart than they are long."""
    big = normal((*shape[:-1], shape[-1] + pad), dt, seed)
    return big[..., :shape[-1]]


@pytest.mark.parametrize("counts", [[3, 0, 9], [300, 150, 0, 451]])
def test_strided_operands_and_outer_rows(sf, counts):
    """Rows further apart than they are long, experts further apart than their rows, rows before the first expert
    and behind the last: what lies between and around stays as it was."""
    E, R, C, lead, trail = len(counts), 264, 392, 5, 7
    T = lead + sum(counts) + trail
    off = offsets(counts, lead)
    A, Y = strided((T, C), BF, 1, 24), strided((T, R), BF, 2, 8)
    W = normal((E, R + 3, C + 16), BF, 3, 0.05)[:, :R, :C]
    before = Y._base.clone()
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off))
    check_forward(A, W, Y, off, before[:, :R], BF)
    assert torch.equal(Y._base[:, R:], before[:, R:])
    before = A._base.clone()
    sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off))
    check_dx(A, W, Y, off, before[:, :C], BF)
    assert torch.equal(A._base[:, C:], before[:, C:])
    G = normal((E, R + 3, C + 4), F32, 4)
    before = G.clone()
    sf.sf_grouped_dw(sf.grouped_problem(A, G[:, :R, :C], Y, off), accumulate=True)
    check_dw(A, G[:, :R, :C], Y, off, before[:, :R, :C], F32)
    assert torch.equal(G[:, R:], before[:, R:]) and torch.equal(G[:, :, C:], before[:, :, C:])


@pytest.mark.parametrize("counts", [[5, 3, 9], [113, 70, 301], [17, 0, 260]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_with_its_sums(sf, counts, bad):
    """A row that is all NaN or infinite spoils its own outputs and its own expert's weight gradient, nothing else."""
    E, R, C = len(counts), 136, 328
    T = sum(counts) + 4
    off = offsets(counts)
    A, W, Y = normal((T, C), BF, 1), normal((E, R, C), BF, 2, 0.05), normal((T, R), BF, 3)
    t = counts[0] + counts[1]                       # the first row of the last expert
    A[t], A[T - 1] = bad, bad                       # and a row behind all of them
    out = torch.zeros((T, R), dtype=BF, device=DEV)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, out, off))
    fine = torch.isfinite(out).all(1)
    assert not bool(fine[t]) and int((~fine).sum()) == 1
    Y[t], Y[T - 1] = bad, bad
    dx = torch.zeros((T, C), dtype=BF, device=DEV)
    sf.sf_grouped_dx(sf.grouped_problem(dx, W, Y, off))
    fine = torch.isfinite(dx).all(1)
    assert not bool(fine[t]) and int((~fine).sum()) == 1
    G = torch.zeros((E, R, C), device=DEV)
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off))
    assert not bool(torch.isfinite(G[-1]).any()) and bool(torch.isfinite(G[:-1]).all())
    # a weight of one expert reaches that expert's tokens alone
    W[0, 5, 7] = bad
    A[t] = A[T - 1] = 1.0
    sf.sf_grouped_forward(sf.grouped_problem(A, W, out, off))
    rows = ~torch.isfinite(out)
    assert bool(rows[:counts[0], 5].all()) and int(rows.sum()) == counts[0]


@pytest.mark.parametrize("off", [[0, 5, 3, 10], [-1, 2, 3, 4], [0, 2, 3, 11], [4, 3, 2, 1], [0, 2 ** 31 - 1, 5, 6]])
@pytest.mark.parametrize("wide", [False, True])
def test_bad_offsets_compute_nothing(sf, off, wide):
    R, C, T = 136, 72, 10
    A, W, Y = normal((T, C), BF, 1), normal((3, R, C), BF, 2), normal((T, R), BF, 3)
    G = normal((3, R, C), F32, 4)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    if wide:                                                     # the pair kernels
        A, Y = normal((1000, C), BF, 1), normal((1000, R), BF, 3)
        o[1:] = torch.where(o[1:] == 11, 1001, o[1:])
    for call, x, w, out in ((sf.sf_grouped_forward, A, W, Y), (sf.sf_grouped_dx, A, W, A), (sf.sf_grouped_dw, A, G, G)):
        status, before = sf.status_word(), out.clone()
        call(sf.grouped_problem(A, w, Y, o), status)
        assert int(status[0]) == sf.SF_STATUS_BAD_OFFSET
        assert torch.equal(out, before)


def test_no_tokens(sf):
    for T in (0, 6):
        A, W, Y = normal((T, 72), BF, 1), normal((3, 136, 72), BF, 2), normal((T, 136), BF, 3)
        off = offsets([0, 0, 0])
        y, a = Y.clone(), A.clone()
        sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off))
        sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off))
        assert torch.equal(y, Y) and torch.equal(a, A)
        G = normal((3, 136, 72), F32, 4)
        g = G.clone()
        sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off), accumulate=True)
        assert torch.equal(g, G)
        sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off))
        assert int(torch.count_nonzero(G)) == 0


@pytest.mark.parametrize("E", [33, 193, 1024])
def test_many_experts(sf, E):
    counts = [(7 * e) % 5 for e in range(E)]
    R, C, T = 24, 40, sum(counts)
    A, W, Y = normal((T, C), HF, 1), normal((E, R, C), HF, 2), torch.zeros((T, R), dtype=HF, device=DEV)
    off = offsets(counts)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off))
    check_forward(A, W, Y, off, Y, HF)
    sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off))
    check_dx(A, W, Y, off, A, HF)
    G = torch.empty((E, R, C), device=DEV)
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off))
    check_dw(A, G, Y, off, None, F32)


@pytest.mark.parametrize("counts", [[3, 1, 0, 4], [400, 100, 0, 250]])
def test_repeats_bit_for_bit_and_replays_with_new_offsets(sf, counts):
    """The same call gives the same bits; a captured call reads the offsets of the moment."""
    R, C, T = 264, 1032, sum(counts)
    A, W = normal((T, C), BF, 1), normal((len(counts), R, C), BF, 2, 0.05)
    Y, dA, G = torch.zeros((T, R), dtype=BF, device=DEV), torch.zeros((T, C), dtype=BF, device=DEV), torch.zeros_like(W, dtype=F32)
    off = offsets(counts)
    fwd, dx, dw = (sf.grouped_problem(*x, off) for x in ((A, W, Y), (dA, W, Y), (A, G, Y)))

    def run():
        sf.sf_grouped_forward(fwd)
        sf.sf_grouped_dx(dx)
        sf.sf_grouped_dw(dw)
        torch.cuda.synchronize()
        return Y.clone(), dA.clone(), G.clone()
    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            sf.sf_grouped_forward(fwd)
            sf.sf_grouped_dx(dx)
            sf.sf_grouped_dw(dw)
    off.copy_(offsets(counts[::-1]))
    want = run()
    for x in (Y, dA, G):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (Y, dA, G)))
    check_forward(A, W, Y, off, Y, BF)


def test_two_streams_at_once(sf):
    """Calls on two streams share nothing."""
    sets = []
    for i, counts in enumerate(([300, 212, 4], [2, 1, 3])):
        T, R, C = sum(counts), 520, 1032
        sets.append((normal((T, C), BF, i), normal((3, R, C), BF, i + 9, 0.05), torch.zeros((T, R), dtype=BF, device=DEV),
                     offsets(counts)))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, x in zip(streams, sets):
            sf.sf_grouped_forward(sf.grouped_problem(*x), stream=st)
    torch.cuda.synchronize()
    for x in sets:
        check_forward(x[0], x[1], x[2], x[3], x[2], BF)


def test_long_sums_keep_fp32_accuracy(sf):
    """A weight gradient over 20,000 tokens whose products all have one sign: the sum of each 1,024 tokens is added in
    fp32, so the relative error stays that of short sums (64 additions, then 20)."""
    T, R, C = 20000, 40, 72
    A, Y = normal((T, C), BF, 1).abs(), normal((T, R), BF, 2).abs()
    G = torch.empty((1, R, C), device=DEV)
    off = offsets([T])
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off))
    ref = Y.double().t() @ A.double()
    assert float(((G[0].double() - ref).abs() / ref).max()) <= (64 + 20 + 32) * 2.0 ** -23


def test_refusals(sf):
    A, W, Y = normal((6, 72), BF, 1), normal((3, 136, 72), BF, 2), normal((6, 136), BF, 3)
    off = offsets([1, 2, 3])
    ok = sf.grouped_problem(A, W, Y, off)
    bads = [lambda: sf.grouped_problem(A, W[:, :, :64], Y, off), lambda: sf.grouped_problem(A, W, Y[:5], off),
            lambda: sf.grouped_problem(A.half(), W, Y, off), lambda: sf.grouped_problem(A, W.half(), Y, off),
            lambda: sf.grouped_problem(A, W, Y, off[:3]), lambda: sf.grouped_problem(A, W, Y, off.long()),
            lambda: sf.grouped_problem(A.cpu(), W, Y, off), lambda: sf.grouped_problem(A, W, Y.t().contiguous().t(), off),
            lambda: sf.grouped_problem(A.float(), W, Y, off)]
    for b in bads:
        with pytest.raises(ValueError):
            b()
    with pytest.raises(RuntimeError, match="invalid argument"):
        sf.sf_grouped_dw(ok, accumulate=True)                    # bf16 gradients are not added to
    with pytest.raises(RuntimeError, match="invalid argument"):
        sf.sf_grouped_forward(sf.grouped_problem(A, W.float(), Y, off))
    with pytest.raises(RuntimeError, match="invalid argument"):
        sf.sf_grouped_forward(sf.grouped_problem(A[:, :68], W[:, :, :68], Y, off))
    big = normal((6, 81), BF, 1)
    with pytest.raises(RuntimeError, match="misaligned"):
        sf.sf_grouped_forward(sf.grouped_problem(big[:, 1:73], W, Y, off))
