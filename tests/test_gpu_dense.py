"""sf_grad_norm and sf_adamw_step against the formulas of include/sf.h in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 256
DEV = "cuda:0"
EPS32 = 2.0 ** -24                       # half a step of fp32, relative


def half_step(dt):
    return torch.finfo(dt).eps / 2


def e4m3(y):
    """Nearest e4m3 value of float64 magnitudes up to 448 (ties to even)."""
    grain = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.rint(y / grain) * grain


class Ref:
    """One tensor's AdamW state in 64 bits."""

    def __init__(self, p, m, v):
        self.p, self.m, self.v = (x.double().cpu().numpy().ravel() for x in (p, m, v))

    def step(self, g, t, hp, decay, factor=1.0):
        b1, b2, lr, eps, wd, clip = (float(np.float32(x)) for x in (hp.beta1, hp.beta2, hp.lr, hp.eps, hp.wd, hp.clip))
        g = g.double().cpu().numpy().ravel() * factor
        if clip > 0:
            g = np.clip(g, -clip, clip)
        self.m = b1 * self.m + (1 - b1) * g
        self.v = b2 * self.v + (1 - b2) * g * g
        u = (self.m / (1 - b1 ** t)) / (np.sqrt(self.v / (1 - b2 ** t)) + eps)
        self.p = self.p - lr * u - lr * wd * decay * self.p


def make(sf, n, p_dt, g_dt, state, live, seed, decay=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    p = (torch.randn(n, generator=gen, device=DEV) * 0.02).to(p_dt)
    g = (torch.randn(n, generator=gen, device=DEV) * 1e-3).to(g_dt)
    return sf.Dense(p, g, state, live, decay)


def decoded(d):
    """(m, sqrt(v)) of a Dense in float64."""
    if d.m_scale is None:
        return d.m.double().cpu().numpy().ravel(), np.sqrt(d.v.double().cpu().numpy().ravel())
    out = []
    for code, sc in ((d.m, d.m_scale), (d.v, d.v_scale)):
        s = sc.double().cpu().numpy().repeat(BLOCK)[:code.numel()]
        out.append(code.float().double().cpu().numpy().ravel() * s)
    return tuple(out)


LENGTHS = [1, 7, 8, 9, 255, 256, 257, 2048, 5003, 70001]


@pytest.mark.parametrize("g_dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("p_dt", [torch.float32, torch.bfloat16])
def test_fp32_moments_follow_the_formula(sf, p_dt, g_dt):
    """Three steps over odd lengths. Each fp32 operation is off by at most 2^-24 of its result. The moments are
    sums of at most 3 terms of 3 roundings: 12 x 2^-24 of the largest term. p moves by at most ~lr a step, its
    own roundings are 3 a step (2^-24 of p) or one to bf16 (2^-9 of p plus the drift of earlier roundings)."""
    hp = sf.AdamParams(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1)
    ds = [make(sf, n, p_dt, g_dt, sf.SF_TYPE_F32, True, n, decay=float(n % 2)) for n in LENGTHS]
    refs = [Ref(d.p, d.m, d.v) for d in ds]
    step, status = sf.step_words(), sf.status_word()
    ts = sf.DenseTensors(ds)
    for t in range(1, 4):
        sf.sf_adamw_step(ts, hp, step, status=status)
        for d, r in zip(ds, refs):
            r.step(d.g, t, hp, d.decay)
            if p_dt == torch.bfloat16:                       # compare each step from the same weights
                p_got = d.p.double().cpu().numpy()
                tol = (half_step(p_dt) + 8 * EPS32) * np.abs(r.p) + 16 * EPS32 * hp.lr
                assert np.all(np.abs(p_got - r.p) <= tol)
                r.p = p_got
    assert step.tolist() == [3, 0] and int(status[0]) == 0
    for d, r in zip(ds, refs):
        g = np.abs(d.g.double().cpu().numpy())
        assert np.all(np.abs(d.m.double().cpu().numpy() - r.m) <= 12 * EPS32 * np.maximum(np.abs(r.m), g * 0.3))
        assert np.all(np.abs(d.v.double().cpu().numpy() - r.v) <= 12 * EPS32 * r.v + 1e-45)
        p = d.p.double().cpu().numpy()
        if p_dt == torch.float32:
            # u: m, v, bias corrections, root, product, quotient: 24 x 2^-24 of |u| <= ~1 times lr, three steps
            assert np.all(np.abs(p - r.p) <= 9 * EPS32 * np.abs(r.p) + 3 * 40 * EPS32 * hp.lr)
            live = d.live.double().cpu().numpy()
            assert np.all(np.abs(live - p) <= half_step(torch.bfloat16) * np.abs(p))
        else:
            assert torch.equal(d.live, d.p)


@pytest.mark.parametrize("p_dt,g_dt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float16)])
def test_8bit_moments_one_step_from_any_state(sf, p_dt, g_dt):
    """From the codes held, a step's moments are the formula's values rounded to the block's e4m3 grid: within
    half a step of it, 2^-4 of the value (or 2^-10 of the scale below 2^-6), plus the fp32 operations before
    the rounding (8 x 2^-24, which can also tip a tie: it is then half a step off, still within)."""
    hp = sf.AdamParams(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
    ds = [make(sf, n, p_dt, g_dt, sf.SF_TYPE_E4M3, True, n) for n in LENGTHS]
    step, status, ts = sf.step_words(), sf.status_word(), sf.DenseTensors(ds)
    for t in range(1, 5):
        befores = [(d.p.clone(), *decoded(d)) for d in ds]
        for i, d in enumerate(ds):                           # other gradients each step, some blocks all zero
            d.g.copy_(torch.randn(d.g.numel(), generator=torch.Generator(device=DEV).manual_seed(100 * t + i), device=DEV) * 10.0 ** -t)
            d.g[512:768] = 0
        sf.sf_adamw_step(ts, hp, step, status=status)
        for d, (p0, m0, r0) in zip(ds, befores):
            r = Ref(p0, torch.from_numpy(m0), torch.from_numpy(r0 * r0))
            r.step(d.g, t, hp, d.decay)
            m1, r1 = decoded(d)
            for got, want, sc in ((m1, r.m, d.m_scale), (r1, np.sqrt(r.v), d.v_scale)):
                n = want.size
                pad = np.zeros(-(-n // BLOCK) * BLOCK)
                pad[:n] = np.abs(want)
                scale = np.maximum(pad.reshape(-1, BLOCK).max(1) / 448, 2.0 ** -100)
                s = sc.double().cpu().numpy()
                assert np.all(np.abs(s - scale) <= 10 * EPS32 * scale)
                at = scale.repeat(BLOCK)[:n]
                assert np.all(np.abs(got - want) <= (2.0 ** -4 + 16 * EPS32) * np.abs(want) + 2.0 ** -10 * at)
                # nearly all are exactly the nearest code
                exact = e4m3(want / at) * s.repeat(BLOCK)[:n]
                tiny = (want > 0) & (exact == 0)
                assert np.mean(np.abs(got - exact)[~tiny] <= 1e-6 * np.abs(exact)[~tiny]) > 0.995 if n > 255 else True
            assert np.all((r1 > 0) == (r.v > 0))             # a positive root keeps a positive code
            tol = (half_step(p_dt) + 6 * EPS32) * np.abs(r.p) + 40 * EPS32 * hp.lr
            # |u| can pass 1 here: 40 roundings of it
            tol = tol + 40 * EPS32 * np.abs(r.p - p0.double().cpu().numpy())
            assert np.all(np.abs(d.p.double().cpu().numpy() - r.p) <= tol)
    assert step.tolist() == [4, 0] and int(status[0]) == 0


def test_the_root_is_correctly_rounded(sf):
    """A block with one gradient g has the scale fp32(sqrt(v) * fp32(1 / 448)) with v = fp32(fp32(g g) (1 - beta2)): over
    100,000 values of all sizes it is, bit for bit, what the correctly rounded root gives, down to v = 2^-100. Below, the
    root's residual r r - v is a multiple of 2^-149 that was rounded by up to 2^-150, and enters the root times 1 / (2 sqrt(v)):
    2^-151 / v of it, before the two roundings (2^-24 each) of root and scale and those of the value it is compared with."""
    n = 100_000
    hp = sf.AdamParams(lr=0.0, beta1=0.9, beta2=0.95)
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(n, generator=gen, device=DEV) * torch.exp2(torch.randint(-58, 58, (n,), generator=gen, device=DEV).float())
    g = torch.zeros((n, BLOCK), device=DEV)
    g[torch.arange(n), torch.arange(n) % BLOCK] = x
    d = sf.Dense(torch.zeros(n * BLOCK, device=DEV), g.view(-1), sf.SF_TYPE_E4M3)
    sf.sf_adamw_step(sf.DenseTensors([d]), hp, sf.step_words())
    v = x.cpu().numpy() ** 2 * np.float32(hp.one_minus_b2)
    assert v.dtype == np.float32
    got, want = d.v_scale.cpu().numpy(), np.maximum(np.sqrt(v) * np.float32(1 / 448), np.float32(2.0 ** -100))
    small = v < 2.0 ** -100
    assert np.array_equal(got[~small], want[~small])
    w = want[small].astype(np.float64)
    assert np.all(np.abs(got[small] - w) <= w * (2.0 ** -151 / np.maximum(v[small].astype(np.float64), 2.0 ** -149) + 4 * EPS32))


def test_a_decaying_block_keeps_decaying(sf):
    """Without gradients v falls by beta2 a step although 1 - beta2 is far below a code's step: the scale
    carries it, and the codes stay."""
    hp = sf.AdamParams(lr=0.0, beta1=0.9, beta2=0.999)
    d = make(sf, 512, torch.float32, torch.float32, sf.SF_TYPE_E4M3, False, 3)
    ts, step = sf.DenseTensors([d]), sf.step_words()
    sf.sf_adamw_step(ts, hp, step)
    _, r0 = decoded(d)
    d.g.zero_()
    for _ in range(200):
        sf.sf_adamw_step(ts, hp, step)
    _, r1 = decoded(d)
    # the block's largest is exact to 200 x 4 roundings; 2^-4 for a code that moved to its neighbour once
    assert np.all(np.abs(r1 / r0 - 0.999 ** 100) <= 2.0 ** -3)
    big = r0.reshape(2, BLOCK).argmax(1)
    for b, k in enumerate(big):
        assert abs(r1.reshape(2, BLOCK)[b, k] / r0.reshape(2, BLOCK)[b, k] - float(np.float32(0.999)) ** 100) <= 800 * EPS32


@pytest.mark.parametrize("count", [1, 383, 385, 800])
def test_many_tensors_in_one_call(sf, count):
    """More tensors than a launch takes, empty ones among them; one step count for all."""
    hp = sf.AdamParams(lr=1e-3, wd=0.0)
    lengths = [0 if i % 7 == 3 else 1 + (37 * i) % 600 for i in range(count)]
    ds = [make(sf, n, torch.float32, torch.float32, sf.SF_TYPE_E4M3 if i % 2 else sf.SF_TYPE_F32, False, i)
          for i, n in enumerate(lengths)]
    refs = [Ref(d.p, d.m.float(), d.v.float()) for d in ds]
    ts, step, out = sf.DenseTensors(ds), sf.step_words(), torch.zeros(2, device=DEV)
    ws = sf.grad_norm_workspace(ts)
    for t in (1, 2):
        sf.sf_grad_norm(ts, out, ws, max_norm=0.01)
    norm = math.sqrt(sum(float(d.g.double().square().sum()) for d in ds))
    # squares in fp32, eight to a sum: 8 roundings, then fp64; the root halves them
    assert abs(float(out[0]) - norm) <= 6 * EPS32 * norm
    assert abs(float(out[1]) - min(1.0, 0.01 / (norm + 1e-6))) <= 10 * EPS32
    sf.sf_adamw_step(ts, hp, step, factor=out)
    f = float(out[1])
    for d, r in zip(ds, refs):
        r.step(d.g, 1, hp, 1.0, f)
        assert np.all(np.abs(d.p.double().cpu().numpy() - r.p) <= 4 * EPS32 * np.abs(r.p) + 40 * EPS32 * hp.lr)
    assert step.tolist() == [1, 0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_non_finite_gradient_skips_the_step(sf, bad):
    ds = [make(sf, 1000, torch.float32, torch.float16, sf.SF_TYPE_E4M3, True, i) for i in range(3)]
    ds[1].g[777] = bad
    ts, step, out, status = sf.DenseTensors(ds), sf.step_words(), torch.zeros(2, device=DEV), sf.status_word()
    before = [[x.clone() for x in (d.p, d.m.view(torch.uint8), d.v.view(torch.uint8), d.m_scale, d.live)] for d in ds]
    ws = sf.grad_norm_workspace(ts)
    sf.sf_grad_norm(ts, out, ws, max_norm=1.0)
    sf.sf_adamw_step(ts, sf.AdamParams(), step, factor=out, status=status)
    assert float(out[1]) == 0.0 and step.tolist() == [0, 0] and int(status[0]) == sf.SF_STATUS_NONFINITE
    for d, b in zip(ds, before):
        for x, y in zip((d.p, d.m.view(torch.uint8), d.v.view(torch.uint8), d.m_scale, d.live), b):
            assert torch.equal(x, y)
    ds[1].g[777] = 0.5                                        # the workspace is ready for the next call
    sf.sf_grad_norm(ts, out, ws, max_norm=1.0)
    sf.sf_adamw_step(ts, sf.AdamParams(), step, factor=out)
    assert float(out[1]) > 0.0 and step.tolist() == [1, 0]


def test_loss_scale_and_element_clip(sf):
    """inv_scale undoes a loss scale before norm, clip and step."""
    hp = sf.AdamParams(lr=1e-2, clip=5e-4)
    a = make(sf, 3000, torch.float32, torch.float32, sf.SF_TYPE_F32, False, 1)
    b = sf.Dense(a.p.clone(), a.g * 1024.0)
    out = torch.zeros(2, device=DEV)
    ts = sf.DenseTensors([b])
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts), max_norm=0.0, inv_scale=2.0 ** -10)
    sf.sf_adamw_step(ts, hp, sf.step_words(), factor=out)
    sf.sf_adamw_step(sf.DenseTensors([a]), hp, sf.step_words())
    assert float(out[1]) == 2.0 ** -10
    assert torch.equal(a.p, b.p) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)


def test_non_finite_results_are_reported(sf):
    d = make(sf, 300, torch.float32, torch.float32, sf.SF_TYPE_E4M3, False, 1)
    d.g[5] = float("nan")
    status = sf.status_word()
    sf.sf_adamw_step(sf.DenseTensors([d]), sf.AdamParams(), sf.step_words(), status=status)
    assert int(status[0]) == sf.SF_STATUS_NONFINITE
    assert math.isnan(float(d.p[5])) and bool(torch.isfinite(d.p[6:]).all())
    assert math.isnan(float(d.m_scale[0])) and bool(torch.isfinite(d.m_scale[1:]).all())


def test_captured_step_replays(sf):
    """Norm and step in a CUDA graph: each replay is a step (the count is on the device)."""
    hp = sf.AdamParams(lr=1e-3, wd=0.1)
    mk = lambda: [make(sf, n, torch.float32, torch.bfloat16, s, True, n) for n in (300, 5000) for s in (sf.SF_TYPE_F32, sf.SF_TYPE_E4M3)]  # noqa: E731
    runs = []
    for graph in (False, True):
        ds = mk()
        ts, step, out = sf.DenseTensors(ds), sf.step_words(), torch.zeros(2, device=DEV)
        ws = sf.grad_norm_workspace(ts)

        def once():
            sf.sf_grad_norm(ts, out, ws, max_norm=0.01)
            sf.sf_adamw_step(ts, hp, step, factor=out)
        if graph:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    once()
            for _ in range(5):
                g.replay()
        else:
            for _ in range(5):
                once()
        torch.cuda.synchronize()
        runs.append((ds, step.tolist(), out.clone()))
    assert runs[0][1] == runs[1][1] == [5, 0] and torch.equal(runs[0][2], runs[1][2])
    for a, b in zip(runs[0][0], runs[1][0]):
        assert torch.equal(a.p, b.p) and torch.equal(a.live, b.live)
        assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))


def test_empty_call_counts_a_step(sf):
    step = sf.step_words()
    sf.sf_adamw_step(sf.DenseTensors([]), sf.AdamParams(), step)
    d = make(sf, 0, torch.float32, torch.float32, sf.SF_TYPE_F32, False, 0)
    ts, out = sf.DenseTensors([d]), torch.ones(2, device=DEV)
    sf.sf_adamw_step(ts, sf.AdamParams(), step)
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts), max_norm=1.0)
    assert step.tolist() == [2, 0] and out.tolist() == [0.0, 1.0]


def test_refusals(sf):
    d = make(sf, 512, torch.float32, torch.float32, sf.SF_TYPE_E4M3, False, 0)
    with pytest.raises(ValueError):
        sf.dense_tensor(d.p, d.g, d.m, d.v)                               # no scales
    with pytest.raises(ValueError):
        sf.dense_tensor(d.p, d.g[:511], d.m, d.v, m_scale=d.m_scale, v_scale=d.v_scale)
    with pytest.raises(ValueError):
        sf.dense_tensor(d.p.double(), d.g, d.m, d.v, m_scale=d.m_scale, v_scale=d.v_scale)
    with pytest.raises(ValueError):
        sf.dense_tensor(d.p, d.g.cpu(), d.m, d.v, m_scale=d.m_scale, v_scale=d.v_scale)
    off = torch.zeros(520, device=DEV)[1:513]
    t = sf.DenseTensors([sf.dense_tensor(off, d.g, d.m, d.v, m_scale=d.m_scale, v_scale=d.v_scale)])
    with pytest.raises(RuntimeError, match="misaligned"):
        sf.sf_adamw_step(t, sf.AdamParams(), sf.step_words())
    ts = sf.DenseTensors([d])
    with pytest.raises(ValueError):
        sf.sf_adamw_step(ts, sf.AdamParams(), torch.zeros(2, device=DEV))  # step words must be int32
    with pytest.raises(RuntimeError, match="invalid argument"):
        sf.sf_grad_norm(ts, torch.zeros(2, device=DEV), torch.zeros(8, dtype=torch.uint8, device=DEV))
