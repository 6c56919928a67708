"""Host-side argument checks of sf_grad_norm and sf_adamw_step (CPU: every case is refused before CUDA is touched)."""
import ctypes

import pytest
import torch

from masked_optimizer_step_b200 import binding as b

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device pointers: host validation only")

ARG, ALIGN = -1, -2
P = 0x7F0000000000            # 16-byte aligned placeholder address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return b.load()


def _dense(**kw):
    f = dict(n=1000, p=P, g=P, m=P, v=P, m_scale=P, v_scale=P, live=None, decay=1.0, p_type=0, g_type=1, state_type=3)
    f.update(kw)
    return b.sf_dense(*[f[k] for k, _ in b.sf_dense._fields_])


def _hp(**kw):
    f = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, one_minus_b1=0.1, one_minus_b2=0.001, wd=0.0, clip=0.0,
             bc1=P, bc2=P, t_max=100)
    f.update(kw)
    return b.sf_adam(*[f[k] for k, _ in b.sf_adam._fields_])


def _step(lib, ts, hp=None, step=P, factor=None, n=None):
    arr = (b.sf_dense * max(len(ts), 1))(*ts)
    hp = _hp() if hp is None else hp
    return lib.sf_adamw_step(arr, len(ts) if n is None else n, ctypes.byref(hp), step, factor, None, None)


@pytest.mark.parametrize("case,kw,code", [
    ("negative length", dict(n=-1), ARG),
    ("no weights", dict(p=None), ARG),
    ("no gradient", dict(g=None), ARG),
    ("no first moment", dict(m=None), ARG),
    ("no second moment", dict(v=None), ARG),
    ("8-bit moments without scales", dict(m_scale=None), ARG),
    ("8-bit moments without root scales", dict(v_scale=None), ARG),
    ("fp16 weights", dict(p_type=2), ARG),
    ("8-bit gradient", dict(g_type=3), ARG),
    ("bf16 moments", dict(state_type=1), ARG),
    ("unknown gradient type", dict(g_type=9), ARG),
    ("weights off 16 bytes", dict(p=P + 8), ALIGN),
    ("gradient off 16 bytes", dict(g=P + 2), ALIGN),
    ("codes off 16 bytes", dict(m=P + 8), ALIGN),
    ("root codes off 16 bytes", dict(v=P + 1), ALIGN),
    ("live copy off 16 bytes", dict(live=P + 4), ALIGN),
    ("scales off 4 bytes", dict(m_scale=P + 2), ALIGN),
])
def test_adamw_step_rejects(lib, case, kw, code):
    assert _step(lib, [_dense(), _dense(**kw)]) == code, case


@pytest.mark.parametrize("case,kw", [("no tables", dict(bc1=None)), ("no second table", dict(bc2=None)),
                                     ("empty tables", dict(t_max=0))])
def test_adamw_step_rejects_hyper_parameters(lib, case, kw):
    assert _step(lib, [_dense()], hp=_hp(**kw)) == ARG, case


def test_adamw_step_rejects_call(lib):
    assert _step(lib, [_dense()], step=None) == ARG
    assert _step(lib, [_dense()], step=P + 2) == ALIGN
    assert _step(lib, [_dense()], factor=P + 1) == ALIGN
    assert _step(lib, [_dense()], n=-1) == ARG
    hp = _hp()
    assert lib.sf_adamw_step(None, 1, ctypes.byref(hp), P, None, None, None) == ARG
    assert lib.sf_adamw_step(None, 1, None, P, None, None, None) == ARG


def test_grad_norm_rejects(lib):
    arr = (b.sf_dense * 1)(_dense())
    need = lib.sf_grad_norm_ws_bytes(arr, 1)
    assert need >= 16 + 148 * 8

    def call(inv=1.0, mx=1.0, out=P, ws=P, nbytes=need, a=arr):
        return lib.sf_grad_norm(a, 1, inv, mx, out, ws, nbytes, None, None)
    assert call(nbytes=need - 1) == ARG
    assert call(ws=None) == ARG
    assert call(out=None) == ARG
    assert call(inv=0.0) == ARG
    assert call(inv=float("nan")) == ARG
    assert call(mx=float("nan")) == ARG
    assert call(ws=P + 8) == ALIGN
    assert call(out=P + 2) == ALIGN
    assert call(a=(b.sf_dense * 1)(_dense(g=P + 8))) == ALIGN
    assert call(a=(b.sf_dense * 1)(_dense(g_type=3))) == ARG
    assert lib.sf_grad_norm_ws_bytes(None, 3) == 0


def test_norm_workspace_has_a_place_for_every_launch(lib):
    one = lib.sf_grad_norm_ws_bytes((b.sf_dense * 1)(_dense()), 1)
    many = (b.sf_dense * 800)(*[_dense() for _ in range(800)])
    assert lib.sf_grad_norm_ws_bytes(many, 800) - 16 == 3 * (one - 16)       # 384 tensors to a launch


def test_binding_struct_follows_the_header():
    from tests.test_abi import _c_struct_fields
    assert [f[0] for f in b.sf_dense._fields_] == _c_struct_fields("sf_dense")


def test_binding_refuses_host_tensors():
    x = torch.zeros(8)
    with pytest.raises(ValueError):
        b.dense_tensor(x, x, x, x)
    with pytest.raises(ValueError):
        b.dense_tensor(x, x, x.half(), x.half())
