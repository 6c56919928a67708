"""The dense-tensor and expert-grouped calls together, as a training step uses them: routed tokens through an expert
projection, its gradients, the clipped AdamW step that writes the live weights, the next forward pass. Every call is
held to the formulas in 64 bits, from what the calls before it left."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_dense import EPS32, Ref, half_step
from tests.test_gpu_grouped import check_dw, check_dx, check_forward, normal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


def route(scores, k):
    """The k best experts of every token: the tokens' rows by expert, and the experts' offsets (all on the device)."""
    E = scores.shape[1]
    e = scores.topk(k, dim=1).indices.flatten()
    order = torch.argsort(e, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=scores.device)
    off[1:] = torch.bincount(e, minlength=E).cumsum(0)
    return order // k, off


@pytest.mark.parametrize("state8", [False, True])
@pytest.mark.parametrize("E,T,R,C", [(4, 37, 72, 136), (8, 300, 520, 264), (3, 1500, 264, 520)])
def test_training_steps_of_an_expert_projection(sf, E, T, R, C, state8):
    from masked_optimizer_step_b200.model import DensePlan, ExpertProjection
    hp = sf.AdamParams(lr=1e-3, beta1=0.9, beta2=0.95, wd=0.1)
    proj = ExpertProjection(normal((E, R, C), torch.float32, 1, 0.05), sf.SF_TYPE_E4M3 if state8 else sf.SF_TYPE_F32)
    gain = sf.Dense(torch.ones(C, device=DEV), torch.zeros(C, device=DEV), decay=0.0)
    plan = DensePlan([proj.dense, gain], hp, max_norm=1.0)
    status = sf.status_word()
    for t in range(1, 4):
        x, want = normal((T, C), torch.float32, 10 * t), normal((2 * T, R), torch.float32, 10 * t + 1)
        rows, off = route(normal((T, E), torch.float32, 10 * t + 2), 2)
        A = (x * gain.p)[rows].to(BF)
        Y, dA = torch.zeros((2 * T, R), dtype=BF, device=DEV), torch.zeros((2 * T, C), dtype=BF, device=DEV)
        live, before = proj.live.clone(), (proj.dense.p.clone(), proj.dense.m.float().clone())
        proj.forward(A, Y, off, status)
        check_forward(A, live, Y, off, Y, BF)
        dY = ((Y.float() - want) / T).to(BF)
        half = int(off[E // 2])                                  # two micro-batches: the experts' rows in two calls
        first, second = off.clamp(max=half), off.clamp(min=half)
        proj.backward(A, dY, first, dA, status=status)
        proj.backward(A, dY, second, dA, accumulate=True, status=status)
        check_dw(A, proj.grad, dY, off, None, torch.float32)
        check_dx(dA, live, dY, off, dA, BF)
        gain.g.zero_().index_add_(0, torch.arange(C, device=DEV), (dA.float() * x[rows]).sum(0))
        ref_gain = Ref(gain.p, gain.m, gain.v)
        if not state8:
            ref = Ref(before[0], before[1], proj.dense.v)
        plan.step(status)
        norm = math.sqrt(float(proj.grad.double().square().sum() + gain.g.double().square().sum()))
        assert abs(float(plan.norm[0]) - norm) <= 6 * EPS32 * norm
        f = float(plan.norm[1])
        assert abs(f - min(1.0, 1.0 / (norm + 1e-6))) <= 10 * EPS32 * f
        ref_gain.step(gain.g, t, hp, 0.0, f)
        assert np.all(np.abs(gain.p.double().cpu().numpy() - ref_gain.p) <= 4 * EPS32 * np.abs(ref_gain.p) + 40 * EPS32 * hp.lr)
        p = proj.dense.p.double().cpu().numpy().ravel()
        if not state8:
            ref.step(proj.grad, t, hp, 1.0, f)
            assert np.all(np.abs(p - ref.p) <= 4 * EPS32 * np.abs(ref.p) + 80 * EPS32 * hp.lr)
        new = proj.live.double().cpu().numpy().ravel()
        assert np.all(np.abs(new - p) <= half_step(BF) * np.abs(p))
        assert not torch.equal(proj.live, live)
    assert plan.steps.tolist() == [3, 0] and int(status[0]) == 0


def test_gradients_against_differences(sf):
    """d(sum of G * Y) / dW and / dA by central differences in the forward call itself. Y is linear in W and in A, so the
    difference of two forward calls is the derivative but for their roundings: each output is off by half a step of bf16
    (2^-9) of its size, twice, and the gradient by its own rounding."""
    E, T, R, C = 3, 23, 40, 72
    off = torch.tensor([0, 9, 9, 23], dtype=torch.int32, device=DEV)
    A, W, G = normal((T, C), BF, 1), normal((E, R, C), BF, 2, 0.1), normal((T, R), BF, 3)
    dW, dA = torch.zeros((E, R, C), device=DEV), torch.zeros((T, C), dtype=BF, device=DEV)
    sf.sf_grouped_dw(sf.grouped_problem(A, dW, G, off))
    sf.sf_grouped_dx(sf.grouped_problem(dA, W, G, off))

    def loss(A, W):
        Y = torch.zeros((T, R), dtype=BF, device=DEV)
        sf.sf_grouped_forward(sf.grouped_problem(A, W, Y, off))
        return float((G.double() * Y.double()).sum()), float((G.double() * Y.double()).abs().sum())
    h = 4.0                                                      # a step far above the roundings; exact in bf16 to add to
    for e, r, c in ((0, 0, 0), (0, 39, 71), (1, 7, 9), (2, 13, 64), (2, 38, 33)):
        up, down = W.clone(), W.clone()
        up[e, r, c], down[e, r, c] = h, -h
        (a, sa), (b, sb) = loss(A, up), loss(A, down)
        assert abs((a - b) / (2 * h) - float(dW[e, r, c])) <= 2.0 ** -9 * (sa + sb) / (2 * h) + 1e-5
    for t, c in ((0, 0), (8, 71), (9, 3), (22, 64)):
        up, down = A.clone(), A.clone()
        up[t, c], down[t, c] = h, -h
        (a, sa), (b, sb) = loss(up, W), loss(down, W)
        g = float(dA[t, c])
        assert abs((a - b) / (2 * h) - g) <= 2.0 ** -9 * (sa + sb) / (2 * h) + 2.0 ** -8 * abs(g) + 1e-5


def test_trainer_steps_its_dense_tensors(sf):
    """A Trainer with a DensePlan steps it behind the sparse step and counts with it."""
    from masked_optimizer_step_b200 import model as M
    from masked_optimizer_step_b200 import synth
    model = M.SparseModel(1, vocab=256, hidden=64, ffn=96, layer_shapes=(("q", 64, 64), ("o", 64, 64)), emb_slots=256)
    model.init(0)
    toks = torch.from_numpy(synth.zipf_ids(synth.rng(0, "tokens"), 64, 256)).to(DEV)
    inputs = dict(tokens=toks, dY=normal((64, 64), BF, 1), Y=[normal((64, 64), BF, 2 + i) for i in range(2)],
                  dX=[normal((64, 64), BF, 4 + i) for i in range(2)], A=[normal((64, 64), BF, 6 + i) for i in range(2)])
    ws = torch.zeros(sf.sf_embed_grad_ws_bytes(64, model.emb.mask.slot_cap) // 4, dtype=torch.int32, device=DEV)
    status = sf.status_word()
    pipe = M.Pipeline(model, inputs, ws, chunks=1)
    hp = sf.AdamParams(lr=1e-2)
    gain = sf.Dense(torch.ones(64, device=DEV), torch.full((64,), 0.5, device=DEV))
    plan = M.DensePlan([gain], hp)
    trainer = M.Trainer(model, [pipe], hp, status, dense=plan)
    for k in range(3):
        trainer.step(k, 1.0)
    torch.cuda.synchronize()
    assert plan.steps.tolist() == [3, 0]
    # a constant gradient: every step moves by lr but for roundings (m and v corrections cancel)
    assert float((gain.p - (1.0 - 3e-2)).abs().max()) <= 3 * 40 * EPS32 * 1e-2 + 3 * EPS32
