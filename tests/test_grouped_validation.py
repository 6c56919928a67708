"""Host-side argument checks of the expert-grouped products (CPU: every case is refused before CUDA is touched)."""
import ctypes

import pytest
import torch

from masked_optimizer_step_b200 import binding as b

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device pointers: host validation only")

ARG, ALIGN, UNSUPPORTED = -1, -2, -3
P = 0x7F0000000000            # 16-byte aligned placeholder address, never dereferenced
BF, HF, F32 = b.SF_TYPE_BF16, b.SF_TYPE_F16, b.SF_TYPE_F32


@pytest.fixture(scope="module")
def lib():
    return b.load()


def _problem(**kw):
    f = dict(A=P, ld_a=512, W=P, ld_w=512, stride_w=256 * 512, Y=P, ld_y=256, offsets=P, E=4, T=100, R=256, C=512,
             type=BF, w_type=BF)
    f.update(kw)
    return b.sf_grouped(*[f[k] for k, _ in b.sf_grouped._fields_])


REFUSED = [
    ("no experts", dict(E=0), ARG),
    ("negative tokens", dict(T=-1), ARG),
    ("no rows", dict(R=0), ARG),
    ("rows not a multiple of 8", dict(R=252), ARG),
    ("columns not a multiple of 8", dict(C=508), ARG),
    ("fp32 tokens", dict(type=F32, w_type=F32), ARG),
    ("unknown type", dict(type=7, w_type=7), ARG),
    ("weights of the other 16-bit type", dict(w_type=HF), ARG),
    ("no weights", dict(W=None), ARG),
    ("no offsets", dict(offsets=None), ARG),
    ("no inputs", dict(A=None), ARG),
    ("no outputs", dict(Y=None), ARG),
    ("input rows overlap", dict(ld_a=504), ARG),
    ("output rows overlap", dict(ld_y=248), ARG),
    ("weight rows overlap", dict(ld_w=504), ARG),
    ("experts overlap", dict(stride_w=255 * 512 + 504), ARG),
    ("inputs off 16 bytes", dict(A=P + 2), ALIGN),
    ("outputs off 16 bytes", dict(Y=P + 8), ALIGN),
    ("weights off 16 bytes", dict(W=P + 4), ALIGN),
    ("offsets off 4 bytes", dict(offsets=P + 2), ALIGN),
    ("input row stride off 16 bytes", dict(ld_a=516), ALIGN),
    ("output row stride off 16 bytes", dict(ld_y=260), ALIGN),
    ("weight row stride off 16 bytes", dict(ld_w=516, stride_w=256 * 516 + 4), ALIGN),
    ("expert stride off 16 bytes", dict(stride_w=256 * 512 + 4), ALIGN),
    ("too many experts", dict(E=1025), UNSUPPORTED),
    ("a stride beyond a tensor map's", dict(ld_a=1 << 39), UNSUPPORTED),
    ("too many tiles", dict(T=(1 << 31) - 1, R=1 << 20, ld_y=1 << 20, stride_w=1 << 30), UNSUPPORTED),
]


@pytest.mark.parametrize("call", ["sf_grouped_forward", "sf_grouped_dx", "sf_grouped_dw"])
@pytest.mark.parametrize("case,kw,code", REFUSED)
def test_rejects(lib, call, case, kw, code):
    p = _problem(**kw)
    args = [ctypes.byref(p)] + ([0] if call == "sf_grouped_dw" else []) + [None, None]
    assert getattr(lib, call)(*args) == code, case


def test_fp32_weights_are_for_gradients_only(lib):
    p = _problem(w_type=F32)
    assert lib.sf_grouped_forward(ctypes.byref(p), None, None) == ARG
    assert lib.sf_grouped_dx(ctypes.byref(p), None, None) == ARG
    p = _problem(w_type=F32, ld_w=514, stride_w=256 * 514)
    assert lib.sf_grouped_dw(ctypes.byref(p), 0, None, None) == ALIGN


def test_16bit_gradients_are_not_accumulated(lib):
    p = _problem()
    assert lib.sf_grouped_dw(ctypes.byref(p), 1, None, None) == ARG


@pytest.mark.parametrize("call", ["sf_grouped_forward", "sf_grouped_dx", "sf_grouped_dw"])
@pytest.mark.parametrize("same", [dict(Y=P, W=P + 16), dict(W=P, Y=P + 16), dict(W=P + 16, Y=P + 16)])
def test_operands_do_not_share_an_address(lib, call, same):
    extra = (0,) if call == "sf_grouped_dw" else ()
    assert getattr(lib, call)(ctypes.byref(_problem(**same)), *extra, None, None) == ARG


def test_null_problem(lib):
    assert lib.sf_grouped_forward(None, None, None) == ARG
    assert lib.sf_grouped_dx(None, None, None) == ARG
    assert lib.sf_grouped_dw(None, 0, None, None) == ARG


def test_binding_struct_follows_the_header():
    from tests.test_abi import _c_struct_fields
    assert [f[0] for f in b.sf_grouped._fields_] == _c_struct_fields("sf_grouped")


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((2, 8, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.grouped_problem(x, w, x, torch.zeros(3, dtype=torch.int32))


def test_binding_refuses_sizes_beyond_32_bits():
    def meta(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="meta")
    off = torch.zeros(3, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="32-bit"):
        b.grouped_problem(meta(2 ** 32 + 8, 8), meta(2, 16, 8), meta(2 ** 32 + 8, 16), off)
