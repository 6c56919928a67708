"""A rewind takes the dense tensors back with the int8 matrices, byte for byte, and training goes on from there."""
import pytest
import torch

from tests.test_gpu_grouped import normal, offsets

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16
LOSSES = [3.0, 2.9, 2.8] + [3.3] * 10 + [2.8, 2.8]         # 3.3 > 1.15 * 2.8: a rewind, then on


def bits(t):
    return t.reshape(-1).view(torch.uint8).clone()


def build(sf):
    from masked_optimizer_step_b200 import model as M
    from masked_optimizer_step_b200 import synth
    model = M.SparseModel(1, vocab=256, hidden=64, ffn=96, layer_shapes=(("q", 64, 64), ("o", 64, 64)), emb_slots=256)
    model.init(0)
    toks = torch.from_numpy(synth.zipf_ids(synth.rng(0, "tokens"), 64, 256)).to(DEV)
    inputs = dict(tokens=toks, dY=normal((64, 64), BF, 1), Y=[normal((64, 64), BF, 2 + i) for i in range(2)],
                  dX=[normal((64, 64), BF, 4 + i) for i in range(2)], A=[normal((64, 64), BF, 6 + i) for i in range(2)])
    ws = torch.zeros(sf.sf_embed_grad_ws_bytes(64, model.emb.mask.slot_cap) // 4, dtype=torch.int32, device=DEV)
    pipe = M.Pipeline(model, inputs, ws, chunks=1)
    proj = M.ExpertProjection(normal((3, 72, 136), torch.float32, 20, 0.05), sf.SF_TYPE_E4M3)
    gain = sf.Dense(torch.ones(65, device=DEV), torch.zeros(65, device=DEV), decay=0.0)
    head = sf.Dense(normal((300,), BF, 21), torch.zeros(300, dtype=BF, device=DEV), live=True)
    plan = M.DensePlan([proj.dense, gain, head], sf.AdamParams(lr=1e-2), max_norm=1.0)
    off = offsets([5, 0, 7])

    def grads(k):
        proj.backward(normal((12, 136), BF, 30 + k), normal((12, 72), BF, 60 + k), off)
        gain.g.copy_(normal((65,), torch.float32, 90 + k))
        head.g.copy_(normal((300,), BF, 120 + k))
    return model, pipe, plan, grads


@pytest.mark.parametrize("side", [False, True])
def test_a_rewind_restores_the_dense_state(sf, side):
    from masked_optimizer_step_b200 import model as M
    model, pipe, plan, grads = build(sf)
    stream = torch.cuda.Stream() if side else None
    trainer = M.Trainer(model, [pipe], sf.AdamParams(lr=1e-2), sf.status_word(), stream=stream, dense=plan)
    assert len(plan.state()) == 6 + 3 + 3 + 1              # p, m, v, scales, live of the experts; of the gain; of the head; steps
    saved = stepped = None
    torch.cuda.synchronize()
    for k, loss in enumerate(LOSSES):
        before = [bits(t) for t in plan.state()]
        grads(k)
        torch.cuda.synchronize()
        act = trainer.step(k, loss)
        torch.cuda.synchronize()
        if act.save:
            saved = before
        if act.restore:
            assert act.skip and not all(torch.equal(a, b) for a, b in zip(before, saved))
            assert all(torch.equal(bits(t), b) for t, b in zip(plan.state(), saved))
            stepped = int(plan.steps[0])
        elif stepped is not None:
            stepped += 1
            assert plan.steps.tolist() == [stepped, 0]
    # the small model's rows outgrow their moment slots, which is the matrices' own affair
    assert stepped is not None and int(trainer.status) & ~sf.SF_STATUS_SLOT_OVERFLOW == 0


def test_the_steps_after_a_restore_are_those_after_the_save(sf):
    _, _, plan, grads = build(sf)
    runs = []
    for k in range(2):
        grads(k)
        plan.step()
    with pytest.raises(RuntimeError, match="nothing was saved"):
        plan.restore()
    plan.save()
    for run in range(2):
        for k in range(2, 5):
            grads(k)
            plan.step()
        runs.append([bits(t) for t in plan.state()])
        plan.restore()
    assert all(torch.equal(a, b) for a, b in zip(*runs)) and plan.steps.tolist() == [2, 0]


@pytest.mark.parametrize("state8", [False, True])
def test_many_tensors_of_every_size_come_back(sf, state8):
    from masked_optimizer_step_b200.model import DensePlan
    lengths = [0, 1, 7, 255, 4096, 2 ** 18 - 1, 2 ** 18, 2 ** 18 + 5, 1_000_003] + [64] * 150
    ds = [sf.Dense(normal((n,), torch.float32 if i % 2 else BF, i), normal((n,), BF, 500 + i), sf.SF_TYPE_E4M3 if state8 else sf.SF_TYPE_F32,
                   live=i % 3 == 0) for i, n in enumerate(lengths)]
    plan = DensePlan(ds, sf.AdamParams(lr=1e-2))
    plan.step()
    saved = [bits(t) for t in plan.state()]
    plan.save()
    plan.step()
    assert not all(torch.equal(bits(t), b) for t, b in zip(plan.state(), saved))
    plan.restore()
    assert all(torch.equal(bits(t), b) for t, b in zip(plan.state(), saved))
