"""The dense step and the expert-grouped products at the ends of what their calls allow: operands beyond 2^31 elements,
single rows, padding that holds NaN, two streams, status words given by address, captured chains, refused aliases.

Tolerances as in test_gpu_grouped.py: a sum of n products whose magnitudes add up to S is off by less than
(n / 16 + 32) 2^-23 S, and its rounding by half a step of the result."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def offsets(counts):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def normal(*shape, dt=BF, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dt)


def check(got, a, b):
    """got = a @ b for 64-bit a and b."""
    ref, size, n = a @ b, a.abs() @ b.abs(), a.shape[1]
    slack = (n / 16 + 32) * 2.0 ** -23 * size
    tol = slack + torch.finfo(got.dtype).eps / 2 * (ref.abs() + slack) + torch.finfo(got.dtype).tiny
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("T,E", [(70001, 2), (530, 3), (40, 4)])
def test_operands_beyond_two_to_the_31(sf, T, E):
    """Rows so far apart that A, W and Y each span more than 2^31 elements; what lies between the rows is NaN."""
    R, C = 264, 136
    ld = (2 ** 31 + 2 ** 20) // (T - 1) // 8 * 8 + 8
    gap = (2 ** 31 + 2 ** 20) // (E - 1) // 8 * 8 + 8
    buf = torch.full((max((T - 1) * ld + R, (E - 1) * gap + R * C),), float("nan"), dtype=BF, device=DEV)
    assert buf.numel() > 2 ** 31
    wide = buf.clone()
    A, W = buf.as_strided((T, C), (ld, 1)), wide.as_strided((E, R, C), (gap, C, 1))
    A.copy_(normal(T, C, seed=1))
    W.copy_(normal(E, R, C, seed=2))
    counts = [T - 5 * (E - 1)] + [5] * (E - 1)
    off, status = offsets(counts), sf.status_word()
    spans = list(zip(off.tolist(), off.tolist()[1:]))
    Y = torch.full_like(buf, float("nan")).as_strided((T, R), (ld, 1))
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off), status)
    for e, (a, b) in enumerate(spans):
        for part in (slice(a, min(a + 64, b)), slice(max(b - 64, a), b)):
            check(Y[part], A[part].double(), W[e].double().t())
    before, W16 = A.clone(), W.clone()
    sf.sf_grouped_dx(sf.grouped_problem(A, W, Y, off), status)
    for e, (a, b) in enumerate(spans):
        for part in (slice(a, min(a + 64, b)), slice(max(b - 64, a), b)):
            check(A[part], Y[part].double(), W16[e].double())
    A.copy_(before)
    sf.sf_grouped_dw(sf.grouped_problem(A, W, Y, off), status)
    for e, (a, b) in enumerate(spans):
        check(W[e], Y[a:b].double().t(), A[a:b].double())
    assert int(status) == 0
    assert bool(buf[C:ld].isnan().all()) and bool(wide[R * C:gap].isnan().all())       # nothing beside the operands was written


def test_a_tensor_beyond_two_to_the_31(sf):
    """Its last elements step like a short tensor of the same values, bit for bit; a block's scale is its own."""
    n, k = 2 ** 31 + 1000, 1000                            # 2^31 is a whole number of blocks
    hp = sf.AdamParams(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1)
    big = sf.Dense(torch.zeros(n, dtype=BF, device=DEV), torch.zeros(n, dtype=BF, device=DEV), sf.SF_TYPE_E4M3)
    small = sf.Dense(normal(k, seed=3), normal(k, seed=4), sf.SF_TYPE_E4M3)
    big.p[-k:] = small.p
    big.g[-k:] = small.g
    out, status = torch.zeros(2, device=DEV), sf.status_word()
    ts = sf.DenseTensors([big])
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts, DEV), 1.0, status=status)
    # each sum of eight squares is off by 8 half steps of fp32 at most, and the result's rounding is one more
    want = float(small.g.double().square().sum().sqrt())
    assert abs(float(out[0]) - want) <= 9 * 2.0 ** -24 * want
    for d in (big, small):
        step, one = sf.step_words(), sf.DenseTensors([d])
        for _ in range(2):
            sf.sf_adamw_step(one, hp, step, status=status)
    assert torch.equal(big.p[-k:], small.p)
    for a, b in ((big.m, small.m), (big.v, small.v)):
        assert torch.equal(a[-k:].view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(big.m_scale[-4:], small.m_scale) and torch.equal(big.v_scale[-4:], small.v_scale)
    assert not bool(big.p[:-k].any()) and int(status) == 0


@pytest.mark.parametrize("R,C", [(8, 8), (136, 72), (2056, 264)])
def test_a_single_strided_row(sf, R, C):
    """A slice of one row keeps the stride of what it was cut from, which need not suit the calls."""
    A, Y = normal(3, C + 5, seed=5)[0:1, :C], torch.zeros(3, R + 3, dtype=BF, device=DEV)[0:1, :R]
    W, off, status = normal(2, R, C, seed=6), offsets([0, 1]), sf.status_word()
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off), status)
    check(Y, A.double(), W[1].double().t())
    G = torch.zeros(2, R, C, device=DEV)
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off), status)
    check(G[1], Y.double().t(), A.double())
    assert not bool(G[0].any()) and int(status) == 0


@pytest.mark.parametrize("counts", [[130] * 24, [128, 0, 257, 64, 1, 390, 127, 129, 96, 33, 512, 500], [2000, 90, 95, 100, 97]])
@pytest.mark.parametrize("dt", [BF, torch.float16])
def test_tiles_of_every_width(sf, counts, dt):
    """Token tiles of up to 128, 256 and 512 rows, ragged ends among them, over more units than there are SMs."""
    R, C = 2568, 2056
    off, T, E, status = offsets(counts), sum(counts), len(counts), sf.status_word()
    A, W, Y = normal(T, C, dt=dt, seed=7), normal(E, R, C, dt=dt, seed=8), torch.zeros(T, R, dtype=dt, device=DEV)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off), status)
    dY, dA = normal(T, R, dt=dt, seed=9), torch.zeros_like(A)
    sf.sf_grouped_dx(sf.grouped_problem(dA, W, dY, off), status)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        if a < b:
            check(Y[a:b], A[a:b].double(), W[e].double().t())
            check(dA[a:b], dY[a:b].double(), W[e].double())
    assert int(status) == 0


@pytest.mark.parametrize("counts,M,K", [([1], 64, 4096), ([16], 72, 4104), ([42], 248, 7912), ([100], 520, 11008), ([3, 0, 9, 4], 64, 4096),
                                        ([2, 2], 1032, 4096), ([100, 0, 90], 264, 2568), ([2], 4096, 4096), ([0, 1, 0], 8, 8200),
                                        ([10, 22, 1, 0, 30, 64, 17, 8], 64, 2056), ([17] * 32, 64, 2048),
                                        ([232, 232], 184, 3784), ([541], 1472, 5608), ([1000], 64, 4096), ([300, 0, 700, 129], 72, 2056)])
@pytest.mark.parametrize("dt", [BF, torch.float16])
def test_few_rows_and_long_sums(sf, counts, M, K, dt):
    """Few results over a long K, whose slices are spread over SMs."""
    off, T, E, status = offsets(counts), sum(counts), len(counts), sf.status_word()
    A, W, Y = normal(T, K, dt=dt, seed=10), normal(E, M, K, dt=dt, seed=11), torch.full((T + 2, M), 7.0, dtype=dt, device=DEV)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y[:T], off), status)
    dY, Wt, dA = normal(T, K, dt=dt, seed=12), normal(E, K, M, dt=dt, seed=13), torch.full((T + 2, M), 7.0, dtype=dt, device=DEV)
    sf.sf_grouped_dx(sf.grouped_problem(dA[:T], Wt, dY, off), status)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        if a < b:
            check(Y[a:b], A[a:b].double(), W[e].double().t())
            check(dA[a:b], dY[a:b].double(), Wt[e].double())
    assert bool((Y[T:] == 7).all()) and bool((dA[T:] == 7).all()) and int(status) == 0


@pytest.mark.parametrize("counts,R,C", [([8192], 64, 512), ([65001], 128, 128), ([9000, 0, 3], 72, 136), ([5, 20011], 8, 264), ([0, 4500], 64, 64)])
@pytest.mark.parametrize("out,add", [(F32, False), (F32, True), (BF, False)])
def test_few_weights_and_many_tokens(sf, counts, R, C, out, add):
    """Small weight gradients over many tokens, whose slices are spread over SMs."""
    off, T, E, status = offsets(counts), sum(counts), len(counts), sf.status_word()
    A, Y, G = normal(T, C, seed=14), normal(T, R, seed=15), normal(E, R, C, dt=out, seed=16)
    before = G.double() if add else torch.zeros_like(G, dtype=torch.float64)
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off), status, accumulate=add)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        y, x = Y[a:b].double(), A[a:b].double()
        ref, size = y.t() @ x + before[e], y.abs().t() @ x.abs() + before[e].abs()
        slack = ((b - a) / 16 + 32) * 2.0 ** -23 * size
        assert bool(((G[e].double() - ref).abs() <= slack + torch.finfo(out).eps / 2 * (ref.abs() + slack)).all())
        if out == F32 and not add and b - a > 4000:        # far from the bound: chunks keep sums of any length this near
            assert float((G[e].double() - ref).norm()) < 1e-6 * float(ref.norm())
    assert int(status) == 0


@pytest.mark.parametrize("counts", [[5, 0, 64, 16, 1, 33, 127, 100], [1] * 20, [300, 2, 0, 9, 31, 80, 200, 17]])
@pytest.mark.parametrize("out,add", [(F32, False), (F32, True), (BF, False)])
def test_large_weight_gradients_of_few_tokens(sf, counts, out, add):
    """Many tiles of W to a handful of tokens: what counts is the results' way out, tile by tile."""
    R, C = 1288, 1800
    off, T, E, status = offsets(counts), sum(counts), len(counts), sf.status_word()
    A, Y, G = normal(T, C, seed=17), normal(T, R, seed=18), normal(E, R + 8, C + 16, dt=out, seed=19)
    old = G.clone()
    sf.sf_grouped_dw(sf.grouped_problem(A, G[:, :R, :C], Y, off), status, accumulate=add)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        before = old[e, :R, :C].double() if add else torch.zeros(R, C, dtype=torch.float64, device=DEV)
        y, x = Y[a:b].double(), A[a:b].double()
        ref, size = y.t() @ x + before, y.abs().t() @ x.abs() + before.abs()
        slack = ((b - a) / 16 + 32) * 2.0 ** -23 * size
        assert bool(((G[e, :R, :C].double() - ref).abs() <= slack + torch.finfo(out).eps / 2 * (ref.abs() + slack)).all())
    assert torch.equal(G[:, R:], old[:, R:]) and torch.equal(G[:, :, C:], old[:, :, C:]) and int(status) == 0


@pytest.mark.parametrize("counts,R,C", [([700, 301, 64], 2112, 1600), ([1300, 0, 977], 1856, 2048), ([40, 3, 0, 120], 2112, 1600), ([130] * 8, 1088, 960),
                                        ([5, 64, 31, 0, 128, 1], 832, 1344), ([2000], 320, 4160), ([130] * 8, 1088, 968), ([700, 301], 2120, 1600)])
@pytest.mark.parametrize("out,add", [(F32, False), (F32, True), (BF, False)])
def test_weight_gradients_of_whole_and_broken_chunks(sf, counts, R, C, out, add):
    """Columns in whole chunks of 64, and not, with last tiles of every width; rows that are views of wider ones."""
    off, T, E, status = offsets(counts), sum(counts), len(counts), sf.status_word()
    wide_a, wide_y = torch.full((T + 1, C + 72), float("nan"), dtype=BF, device=DEV), torch.full((T + 1, R + 8), float("nan"), dtype=BF, device=DEV)
    A, Y, G = wide_a[:T, :C], wide_y[:T, :R], normal(E, R, C, dt=out, seed=22)
    A.copy_(normal(T, C, seed=20))
    Y.copy_(normal(T, R, seed=21))
    old = G.double() if add else torch.zeros(E, R, C, dtype=torch.float64, device=DEV)
    sf.sf_grouped_dw(sf.grouped_problem(A, G, Y, off), status, accumulate=add)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        y, x = Y[a:b].double(), A[a:b].double()
        ref, size = y.t() @ x + old[e], y.abs().t() @ x.abs() + old[e].abs()
        slack = ((b - a) / 16 + 32) * 2.0 ** -23 * size
        assert bool(((G[e].double() - ref).abs() <= slack + torch.finfo(out).eps / 2 * (ref.abs() + slack)).all())
    assert int(status) == 0


def chain(sf, T=700, E=5, R=520, C=264, seed=0):
    """Forward, gradients, norm and step of one expert projection: every call reads what the one before wrote."""
    W, A, dY = normal(E, R, C, dt=F32, seed=seed) * 0.05, normal(T, C, seed=seed + 1), normal(T, R, seed=seed + 2) * 0.01
    Y, dA = torch.zeros(T, R, dtype=BF, device=DEV), torch.zeros(T, C, dtype=BF, device=DEV)
    grad = torch.zeros_like(W)
    d = sf.Dense(W, grad, sf.SF_TYPE_E4M3, live=True)
    ts, out, step, status = sf.DenseTensors([d]), torch.zeros(2, device=DEV), sf.step_words(), sf.status_word()
    ws, hp = sf.grad_norm_workspace(ts, DEV), sf.AdamParams(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.01)
    off = offsets([T - 3 * (T // 4), T // 4, 0, T // 4, T // 4])

    def run():
        sf.sf_grouped_forward(sf.grouped_problem(A, d.live, Y, off), status)
        sf.sf_grouped_dw(sf.grouped_problem(A, grad, Y, off), status)
        sf.sf_grouped_dw(sf.grouped_problem(A, grad, dY, off), status, accumulate=True)
        sf.sf_grouped_dx(sf.grouped_problem(dA, d.live, Y, off), status)
        sf.sf_grad_norm(ts, out, ws, 1.0, status=status)
        sf.sf_adamw_step(ts, hp, step, out, status)
        A.copy_(dA)
        A.mul_(0.01)

    return run, lambda: [t.clone() for t in (W, d.live, d.m.view(torch.uint8), d.v.view(torch.uint8), Y, dA, grad, out, step, status)]


@pytest.mark.parametrize("T", [12, 700, 6000])
def test_a_captured_chain_equals_the_calls(sf, T):
    run, state = chain(sf, T)
    for _ in range(4):
        run()
    torch.cuda.synchronize()
    want = state()
    run, state = chain(sf, T)
    run()                                                  # the first call also sets the kernels up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = state()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and int(got[-1]) == 0 and int(got[-2][0]) == 4


def test_two_chains_on_two_streams(sf):
    alone = []
    for seed in (0, 50):
        run, state = chain(sf, 900, seed=seed)
        for _ in range(6):
            run()
        torch.cuda.synchronize()
        alone.append(state())
    pair = [chain(sf, 900, seed=seed) for seed in (0, 50)]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, (run, _) in zip(streams, pair):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for want, (_, state) in zip(alone, pair):
        assert all(torch.equal(a, b) for a, b in zip(state(), want))


def test_a_status_word_given_by_its_address(sf):
    status = sf.status_word()
    d = sf.Dense(torch.ones(300, device=DEV), torch.full((300,), float("nan"), device=DEV))
    ts, out, hp = sf.DenseTensors([d]), torch.zeros(2, device=DEV), sf.AdamParams(lr=1e-2)
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts, DEV), 1.0, status=status.data_ptr())
    assert int(status) == sf.SF_STATUS_NONFINITE
    status.zero_()
    sf.sf_adamw_step(ts, hp, sf.step_words(), out, status.data_ptr())
    assert int(status) == sf.SF_STATUS_NONFINITE
    status.zero_()
    A, W, Y = normal(4, 16), normal(2, 24, 16), torch.zeros(4, 24, dtype=BF, device=DEV)
    sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, offsets([5, 4])), status.data_ptr())
    assert int(status) == sf.SF_STATUS_BAD_OFFSET and not bool(Y.any())


def test_shared_buffers_are_refused(sf):
    a, b = (sf.Dense(torch.ones(64, device=DEV), torch.ones(64, device=DEV)) for _ in range(2))
    with pytest.raises(ValueError, match="twice"):
        sf.DenseTensors([a, b, a])
    b.p = a.p
    with pytest.raises(ValueError, match="twice"):
        sf.DenseTensors([a, b])
    c = sf.Dense(torch.ones(64, device=DEV), a.g)          # a shared gradient is only read
    sf.DenseTensors([a, c])
    X = normal(16, 16)
    with pytest.raises(RuntimeError, match="sf_grouped_forward"):
        sf.sf_grouped_forward(sf.grouped_problem(X, normal(2, 16, 16), X, offsets([8, 8])))


def test_bf16_weights_as_their_own_live_copy(sf):
    hp, step = sf.AdamParams(lr=1e-2), [sf.step_words() for _ in range(2)]
    two = [sf.Dense(normal(1003, seed=1), normal(1003, seed=2)) for _ in range(2)]
    two[0].live = two[0].p
    two[1].live = two[1].p.clone()
    for d, st in zip(two, step):
        sf.sf_adamw_step(sf.DenseTensors([d]), hp, st)
    assert torch.equal(two[0].p, two[1].p) and torch.equal(two[1].live, two[1].p)
