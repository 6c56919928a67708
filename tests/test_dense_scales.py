"""The norm's limit and the loss scale of a DensePlan (CPU: which calls a step makes)."""
from types import SimpleNamespace

import pytest
import torch

from masked_optimizer_step_b200 import model as M

HP = SimpleNamespace(bc1=torch.ones(2))
NAN = float("nan")


@pytest.mark.parametrize("max_norm,inv_scale", [(NAN, 1.0), (NAN, 0.5), (1.0, 0.0), (1.0, -1.0), (0.0, NAN)])
def test_a_limit_or_scale_that_is_none_is_refused(max_norm, inv_scale):
    with pytest.raises(ValueError, match="inv_scale"):
        M.DensePlan([], HP, max_norm, inv_scale)


def test_they_may_be_changed_from_step_to_step(monkeypatch):
    log = []
    monkeypatch.setattr(M.sf, "sf_grad_norm", lambda t, out, ws, max_norm, inv_scale, status, stream: log.append((max_norm, inv_scale)))
    monkeypatch.setattr(M.sf, "sf_adamw_step", lambda t, hp, steps, factor, status, stream: log.append(factor is not None))
    plan = M.DensePlan([], HP)
    for max_norm, inv_scale in ((0.0, 1.0), (0.0, 2.0 ** -10), (1.0, 1.0), (-1.0, 1.0), (NAN, 1.0)):
        plan.max_norm, plan.inv_scale = max_norm, inv_scale
        plan.step()
    assert str(log) == str([False, (0.0, 2.0 ** -10), True, (1.0, 1.0), True, False, (NAN, 1.0), True])    # the call refuses a NaN
