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
