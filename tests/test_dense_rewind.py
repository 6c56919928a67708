"""A rewind takes the dense tensors back with the int8 matrices: the host's side of it (CPU)."""
from types import SimpleNamespace

from masked_optimizer_step_b200 import helix as hx
from tests.test_helix import _FakeBinding, _FakeMat

LOSSES = [2.0, 1.95, 1.9] + [2.3] * 10                     # 2.3 > 1.15 * 1.9: the watch ends in a rewind


def _rewinder(dense):
    rw = hx.Rewinder.__new__(hx.Rewinder)
    rw.sf, rw.mats = _FakeBinding(), [_FakeMat(64, 32, 8)]
    rw.policy, rw.helix, rw.saved = hx.RewindPolicy(), hx.Helix(), False
    rw.ckpts = [rw.sf.Checkpoint(8, 32, "cpu")]
    rw.dense = dense
    return rw


def test_the_dense_state_is_saved_and_restored_with_the_matrices():
    for stream, given in ((None, 0), (0, 0), (77, 77)):    # no stream is the default one, as for the matrices
        log = []
        rw = _rewinder(SimpleNamespace(save=lambda s: log.append(("save", s)), restore=lambda s: log.append(("restore", s))))
        acts = [rw.before_step(L, None, stream) for L in LOSSES]
        assert log == [(name, given) for name, _ in rw.sf.calls]
        assert [a.event for a in acts][-1] == "rewind" and log[-1][0] == "restore" and log.count(("restore", given)) == 1


def test_a_rewind_without_a_checkpoint_touches_nothing():
    log = []
    rw = _rewinder(SimpleNamespace(save=lambda s: log.append("save"), restore=lambda s: log.append("restore")))
    rw.policy.ckpt_loss = 1.0                              # the policy thinks of one; none was saved
    assert not rw.before_step(float("nan")).skip and log == []


def test_the_trainer_gives_its_plan_to_the_rewinder():
    from masked_optimizer_step_b200.model import Trainer
    log = []
    dense = SimpleNamespace(reserve=lambda: log.append("reserve"))
    tr = Trainer(SimpleNamespace(all_mats=[], device="cpu"), [], None, None, dense=dense)
    assert tr.rewinder.dense is dense and log == ["reserve"]
    assert Trainer(SimpleNamespace(all_mats=[], device="cpu"), [], None, None).rewinder.dense is None
