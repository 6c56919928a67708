"""What the expert-grouped products promise, on every kernel that a call may take: bad offsets compute nothing, a bad value stays
with its sums, rows around the experts and between the operands' rows stay as they were, repeats are the same bit for bit, a
captured call reads the offsets of the moment. The kernels are asked for by name, so that a shape that no longer reaches its
own fails here. Tolerances as in test_gpu_grouped.py."""
import pytest
import torch

from tests.test_gpu_grouped import check_dw, check_dx, check_forward, normal, offsets, spans

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
RAGGED = [130, 0, 257, 64, 1, 390, 127, 311]

# kernel: tokens by expert, width of the results, length of the sums (forward: R, C; dx: C, R)
PRODUCT = {
    "SINGLE": ([12, 3, 20, 0, 16, 17, 5, 23], 4104, 2568),
    "ROUNDS": ([(37 * e) % 97 for e in range(64)], 1032, 1032),
    "SLICES": ([30, 0, 31, 29], 4104, 264),
    "CLUSTERS": ([100, 0, 90], 264, 2568),
    "PAIRS": (RAGGED, 2568, 2056),
}
# kernel: tokens by expert, R, C, whether it adds
DW = {
    "SINGLE": ([40, 3, 0, 21], 1032, 1032, False),
    "SINGLE, added": ([40, 3, 0, 21], 1032, 1032, True),
    "SLICES": ([300, 0, 451, 150], 264, 392, False),
    "SLICES, added": ([300, 0, 451, 150], 264, 392, True),
    "CLUSTERS": ([9000, 0, 3], 72, 136, False),
    "CLUSTERS, added": ([9000, 0, 3], 72, 136, True),
    "PAIRS": ([160, 0, 257, 64, 1, 390, 127, 311], 1288, 1800, False),
    "PAIRS, added": ([700, 301, 900], 1288, 1800, True),
    "PAIRS_FEW": ([100, 0, 257, 64, 1, 90, 127, 33], 1288, 1800, False),
    "PAIRS_ADD": ([160, 0, 257, 64, 1, 390, 127, 311], 1288, 1800, True),
}


class Call:
    """One product's operands with rows before the first expert and behind the last, all rows further apart than they are long."""

    def __init__(self, sf, which, name, dt=BF, lead=0, trail=0, pad=0, seed=1):
        self.sf, self.which, self.kernel = sf, which, getattr(sf, "SF_GROUPED_" + name.split(",")[0])
        if which == "dw":
            self.counts, R, C, self.add = DW[name]
        else:
            self.counts, M, K = PRODUCT[name]
            (R, C), self.add = ((M, K) if which == "forward" else (K, M)), False
        self.dt, E, T = dt, len(self.counts), lead + sum(self.counts) + trail
        self.wide = {"A": normal((T, C + pad), dt, seed), "Y": normal((T, R + pad), dt, seed + 1),
                     "W": normal((E, R + pad // 8, C + pad), F32 if which == "dw" else dt, seed + 2, 1.0 if which == "dw" else 0.05)}
        self.A, self.Y, self.W = self.wide["A"][:, :C], self.wide["Y"][:, :R], self.wide["W"][:, :R, :C]
        self.off, self.status = offsets(self.counts, lead), sf.status_word()
        self.written = {"forward": "Y", "dx": "A", "dw": "W"}[which]
        self.out, self.out_wide = getattr(self, self.written), self.wide[self.written]
        self.before, self.before_wide = self.out.clone(), self.out_wide.clone()
        self.problem = sf.grouped_problem(self.A, self.W, self.Y, self.off)
        product = {"forward": sf.SF_GROUPED_FORWARD, "dx": sf.SF_GROUPED_DX, "dw": sf.SF_GROUPED_DW}[which]
        assert sf.sf_grouped_kernel(self.problem, product, self.add) == self.kernel

    def __call__(self):
        extra = {"accumulate": self.add} if self.which == "dw" else {}
        getattr(self.sf, "sf_grouped_" + self.which)(self.problem, self.status, **extra)

    def restore(self):
        self.out_wide.copy_(self.before_wide)

    def check(self):
        if self.which == "forward":
            check_forward(self.A, self.W, self.Y, self.off, self.before, self.dt)
        elif self.which == "dx":
            check_dx(self.A, self.W, self.Y, self.off, self.before, self.dt)
        else:
            check_dw(self.A, self.W, self.Y, self.off, self.before if self.add else None, F32)


PATHS = [(w, n) for w in ("forward", "dx") for n in PRODUCT] + [("dw", n) for n in DW]


@pytest.mark.parametrize("which,name", PATHS)
def test_bad_offsets_compute_nothing(sf, which, name):
    c = Call(sf, which, name)
    good, E, T = c.off.tolist(), len(c.counts), c.A.shape[0]
    for e, value in ((0, -1), (E, T + 1), (E // 2, T + 1), (E // 2, good[E // 2 - 1] - 1), (E, 2 ** 31 - 1), (1, -2 ** 31)):
        off = list(good)
        off[e] = value
        c.off.copy_(torch.tensor(off, dtype=torch.int32))
        c.status.zero_()
        c()
        assert int(c.status) == sf.SF_STATUS_BAD_OFFSET and torch.equal(c.out_wide, c.before_wide)
    c.off.copy_(torch.tensor(good, dtype=torch.int32))
    c.status.zero_()
    c()
    c.check()
    assert int(c.status) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which,name", PATHS)
def test_a_bad_value_stays_with_its_sums(sf, which, name, bad):
    """A row of an expert that is all bad, and rows before and behind the experts: the sums they are in, and no others."""
    c = Call(sf, which, name, lead=3, trail=2)
    T = c.A.shape[0]
    busy = [(e, a, b) for e, a, b in spans(c.off) if b > a]
    e, a, b = busy[len(busy) // 2]
    for t in {a, b - 1}:                         # next to the experts before and behind
        for x in (c.A, c.Y):
            if x is not c.out:
                for row in (0, 2, t, T - 2, T - 1):
                    x[row] = bad
    c()
    assert int(c.status) == 0
    fine = torch.isfinite(c.out)
    if which == "dw":
        assert not bool(fine[e].any()) and bool(fine[:e].all()) and bool(fine[e + 1:].all())
        return
    rows = {a, b - 1}
    assert bool((~fine).any(1).nonzero().flatten().eq(torch.tensor(sorted(rows), device=DEV)).all())
    # a weight reaches its own expert's tokens and, of them, one result each
    c = Call(sf, which, name, lead=3, trail=2)
    r, k = c.W.shape[1] - 1, c.W.shape[2] - 1
    c.W[e, r, k] = bad
    c()
    fine, col = torch.isfinite(c.out), r if which == "forward" else k
    assert not bool(fine[a:b, col].any()) and int((~fine).sum()) == b - a


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("which,name", PATHS)
def test_rows_around_and_between_stay(sf, which, name, dt):
    c = Call(sf, which, name, dt, lead=5, trail=7, pad=24)
    c()
    c.check()
    after = c.out_wide.clone()
    if which == "dw":
        after[:, :c.out.shape[1], :c.out.shape[2]] = c.before
    else:
        first, last = int(c.off[0]), int(c.off[-1])
        after[first:last, :c.out.shape[1]] = c.before[first:last]
    assert torch.equal(after, c.before_wide) and int(c.status) == 0


@pytest.mark.parametrize("which,name", PATHS)
def test_repeats_and_replays(sf, which, name):
    c = Call(sf, which, name)
    c()
    first = c.out.clone()
    c.check()
    for _ in range(3):
        c.restore()
        c()
        assert torch.equal(c.out, first)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            c()
    for counts in (c.counts[::-1], c.counts):
        c.off.copy_(offsets(counts))
        c.restore()
        c()
        want = c.out.clone()
        c.restore()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
        c.check()
    assert torch.equal(c.out, first) and int(c.status) == 0


@pytest.mark.parametrize("which", ["forward", "dx"])
@pytest.mark.parametrize("counts", [[600, 530], [1024, 1100], [2048, 0, 777], [513, 512, 511, 520, 560]])
@pytest.mark.parametrize("K", [8, 64, 72, 128, 136, 192, 200, 256, 320])
def test_pairs_of_short_sums(sf, which, counts, K):
    """One to five steps of K under tiles of more than 256 tokens, whose two halves' first steps run one behind the other."""
    M, T, E = 4104, sum(counts), len(counts)
    R, C = (M, K) if which == "forward" else (K, M)
    A, W, Y = normal((T, C), BF, 1), normal((E, R, C), BF, 2, 0.05), normal((T, R), BF, 3)
    off, status, p = offsets(counts), sf.status_word(), None
    p = sf.grouped_problem(A, W, Y, off)
    assert sf.sf_grouped_kernel(p, sf.SF_GROUPED_FORWARD if which == "forward" else sf.SF_GROUPED_DX) == sf.SF_GROUPED_PAIRS
    if which == "forward":
        sf.sf_grouped_forward(p, status)
        check_forward(A, W, Y, off, Y, BF)
    else:
        sf.sf_grouped_dx(p, status)
        check_dx(A, W, Y, off, A, BF)
    assert int(status) == 0


def test_what_a_call_takes(sf):
    """Calls that take nothing, and the refusals."""
    c = Call(sf, "forward", "PAIRS")
    none = sf.grouped_problem(c.A[:0], c.W, c.Y[:0], c.off)
    assert sf.sf_grouped_kernel(none, sf.SF_GROUPED_FORWARD) == sf.sf_grouped_kernel(none, sf.SF_GROUPED_DX) == sf.SF_GROUPED_NONE
    assert sf.sf_grouped_kernel(none, sf.SF_GROUPED_DW) != sf.SF_GROUPED_NONE               # writes zeros
    for product, add in ((3, False), (-1, False), (sf.SF_GROUPED_DW, True)):
        with pytest.raises(RuntimeError, match="invalid argument"):
            sf.sf_grouped_kernel(c.problem, product, add)                                   # bf16 gradients are not added to
