"""The host side of the dense tensors in the training loop (CPU)."""
from types import SimpleNamespace

from masked_optimizer_step_b200 import model as M


def _trainer(skip):
    t = M.Trainer.__new__(M.Trainer)
    log = []
    act = SimpleNamespace(event="rewind" if skip else "", skip=skip)
    t.stream = SimpleNamespace(cuda_stream=7)
    t.status = 99
    t.rewinder = SimpleNamespace(before_step=lambda *a: act)
    t.helix = SimpleNamespace(coefficients=lambda: SimpleNamespace(c_self=1.0, c_partner={}))
    t.pipes = [SimpleNamespace(set_mix=lambda *a: None, set_tokens=lambda *a: None,
                               step=lambda hp, st, s: log.append(("sparse", st, s)))]
    t.hp, t.events = None, {}
    t.dense = SimpleNamespace(step=lambda st, s: log.append(("dense", st, s)))
    return t, log


def test_dense_step_follows_the_sparse_one_on_its_stream():
    t, log = _trainer(False)
    t.step(0, 1.0)
    assert log == [("sparse", 99, t.stream), ("dense", 99, t.stream)]


def test_a_rewound_step_leaves_the_dense_tensors_out():
    t, log = _trainer(True)
    t.step(0, 1.0)
    assert log == []


def test_without_dense_tensors_nothing_changes():
    t, log = _trainer(False)
    t.dense = None
    t.step(0, 1.0)
    assert log == [("sparse", 99, t.stream)]
