"""The dense step and its norm on values at the ends of what the types hold: not finite, beyond the squares' range, below it."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_dense import EPS32, Ref, half_step, make

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("g_dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("at", [5, 290])                     # in a whole block, and in the last, short one
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_bad_gradient_under_an_element_clip(sf, bad, at, state8, g_dt):
    """A NaN passes the clamp and spoils its own element (with 8-bit moments its block's moments); an infinity becomes the
    clip's value. Both are reported. Tolerances of one step as in test_gpu_dense.py: 4 roundings of p, 40 of an update of lr."""
    hp = sf.AdamParams(lr=1e-2, clip=5e-4)
    d = make(sf, 300, torch.float32, g_dt, sf.SF_TYPE_E4M3 if state8 else sf.SF_TYPE_F32, True, 1)
    status, step = sf.status_word(), sf.step_words()
    clean = make(sf, 300, torch.float32, g_dt, sf.SF_TYPE_E4M3 if state8 else sf.SF_TYPE_F32, True, 1)
    sf.sf_adamw_step(sf.DenseTensors([clean]), hp, sf.step_words(), status=status)
    assert int(status) == 0
    d.g[at] = bad
    ref = Ref(d.p, d.m.float(), d.v.float())
    ref.step(d.g, 1, hp, 1.0)
    sf.sf_adamw_step(sf.DenseTensors([d]), hp, step, status=status)
    assert int(status) == sf.SF_STATUS_NONFINITE and step.tolist() == [1, 0]
    got = d.p.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref.p)) and int(np.isnan(got).sum()) == int(math.isnan(bad))
    fine = ~np.isnan(ref.p)
    assert np.all(np.abs(got - ref.p)[fine] <= (4 * EPS32 * np.abs(ref.p) + 40 * EPS32 * hp.lr)[fine])
    assert torch.equal(d.live.isnan(), d.p.isnan())
    if state8:
        assert torch.equal(d.m_scale.isnan().cpu(), torch.tensor([b == at // 256 and math.isnan(bad) for b in range(2)]))
    else:
        assert torch.equal(d.m.isnan(), d.p.isnan()) and torch.equal(d.v.isnan(), d.p.isnan())


@pytest.mark.parametrize("factor", [1.0, 0.25])
def test_a_clip_through_the_plan_without_a_norm(sf, factor):
    """The plan's own path to it: no norm, no loss scale, an element clip in the hyper-parameters."""
    from masked_optimizer_step_b200.model import DensePlan
    d = make(sf, 600, torch.float32, torch.float32, sf.SF_TYPE_F32, False, 2)
    d.g[7] = NAN
    plan, status = DensePlan([d], sf.AdamParams(lr=1e-2, clip=1e-3 * factor)), sf.status_word()
    plan.step(status)
    assert int(status) == sf.SF_STATUS_NONFINITE and bool(d.p[7].isnan()) and int(d.p.isnan().sum()) == 1


@pytest.mark.parametrize("g_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e25, 3e19, 1e-19, 1e-25, 1e-38])
@pytest.mark.parametrize("n", [1, 8, 300, 70001])
def test_the_norm_of_values_whose_squares_leave_fp32(sf, n, size, g_dt):
    """Alone, and among values of ordinary size. Eight squares to a sum: 8 roundings, which the root halves, and those of
    the result."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    g = (torch.randn(n, generator=gen, device=DEV).double() * size).to(g_dt)
    mixed = (torch.randn(n, generator=gen, device=DEV) * torch.where(torch.arange(n, device=DEV) % 3 == 0, size, 1.0)).to(g_dt)
    zeros = torch.zeros(n, dtype=g_dt, device=DEV)
    zeros[-1] = -0.0
    for tensors in ([g], [mixed], [zeros, g, zeros]):
        ds = [sf.Dense(torch.zeros(x.numel(), device=DEV), x) for x in tensors]
        ts, out, status = sf.DenseTensors(ds), torch.zeros(2, device=DEV), sf.status_word()
        sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts), max_norm=1.0, inv_scale=0.5, status=status)
        want = 0.5 * math.sqrt(sum(float(x.double().square().sum()) for x in tensors))
        assert want < 3e38
        # below 2^-126 the result itself is a multiple of 2^-149
        assert abs(float(out[0]) - want) <= 6 * EPS32 * want + 2.0 ** -150
        f = 0.5 * min(1.0, 1.0 / (want + 1e-6))
        assert abs(float(out[1]) - f) <= 10 * EPS32 * f + 2.0 ** -150 and int(status) == 0


@pytest.mark.parametrize("n", [1, 300])
def test_a_norm_beyond_fp32_skips_the_step(sf, n):
    ds = [sf.Dense(torch.ones(n, device=DEV), torch.full((n,), 3e38, device=DEV)) for _ in range(2)]
    ts, out, status, step = sf.DenseTensors(ds), torch.zeros(2, device=DEV), sf.status_word(), sf.step_words()
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts), max_norm=1.0, status=status)
    sf.sf_adamw_step(ts, sf.AdamParams(), step, out)
    assert out.tolist() == [INF, 0.0] and int(status) == sf.SF_STATUS_NONFINITE and step.tolist() == [0, 0]
    assert all(bool((d.p == 1).all()) for d in ds)


@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_bad_value_in_the_norm(sf, bad):
    """Beside values that take the fp64 sums."""
    d = sf.Dense(torch.ones(300, device=DEV), torch.full((300,), 1e25, device=DEV))
    d.g[290] = bad
    ts, out, status = sf.DenseTensors([d]), torch.zeros(2, device=DEV), sf.status_word()
    sf.sf_grad_norm(ts, out, sf.grad_norm_workspace(ts), max_norm=1.0, status=status)
    assert not math.isfinite(float(out[0])) and float(out[1]) == 0.0 and int(status) == sf.SF_STATUS_NONFINITE


@pytest.mark.parametrize("p_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("at", [5, 290])
@pytest.mark.parametrize("size", [1e20, -3e30])
def test_a_square_beyond_fp32_leaves_the_weight_finite(sf, size, at, state8, p_dt):
    """The root moment becomes infinite and the update m / v zero: the weight decays and no more, as the formula has it. The
    moment is reported. One step: 4 roundings of p, 40 of an update of lr, and half a step of the weights' type."""
    hp = sf.AdamParams(lr=1e-2, wd=0.1)
    d = make(sf, 300, p_dt, torch.float32, sf.SF_TYPE_E4M3 if state8 else sf.SF_TYPE_F32, True, 3)
    d.g[at] = size
    status, before = sf.status_word(), d.p.double().clone()
    ref = Ref(d.p, d.m.float(), d.v.float())
    ref.step(d.g, 1, hp, 1.0)
    ref.p[at] = float(before[at]) * (1 - float(np.float32(hp.lr)) * float(np.float32(hp.wd)))
    sf.sf_adamw_step(sf.DenseTensors([d]), hp, sf.step_words(), status=status)
    assert int(status) == sf.SF_STATUS_NONFINITE and bool(d.p.isfinite().all()) and bool(d.live.isfinite().all())
    tol = (4 * EPS32 + half_step(p_dt)) * np.abs(ref.p) + 40 * EPS32 * hp.lr
    assert np.all(np.abs(d.p.double().cpu().numpy() - ref.p) <= tol)
    assert int((~(d.v_scale if state8 else d.v).isfinite()).sum()) == 1


def test_a_loss_scale_that_is_set_later(sf):
    """A plan made without one takes it from the next step on; a power of two changes no bit."""
    from masked_optimizer_step_b200.model import DensePlan
    a = make(sf, 3000, torch.float32, torch.float32, sf.SF_TYPE_E4M3, True, 4)
    b = sf.Dense(a.p.clone(), a.g * 1024.0, sf.SF_TYPE_E4M3, True)
    plans = [DensePlan([d], sf.AdamParams(lr=1e-2)) for d in (a, b)]
    plans[1].inv_scale = 2.0 ** -10
    for _ in range(2):
        for plan in plans:
            plan.step()
    assert torch.equal(a.p, b.p) and torch.equal(a.live, b.live) and torch.equal(a.m_scale, b.m_scale)
