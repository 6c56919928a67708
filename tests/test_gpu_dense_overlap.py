"""Tensors of one step that share memory: refused where the step writes it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def parts(sf, n=600):
    """Two tensors' buffers, all in one."""
    flat = torch.zeros(12 * n, device=DEV)
    return flat, [sf.dense_tensor(*(flat[(4 * i + k) * n:(4 * i + k + 1) * n] for k in range(4))) for i in range(2)], n


def test_neighbours_and_shared_gradients_are_taken(sf):
    flat, (a, b), n = parts(sf)
    sf.DenseTensors([a, b])
    sf.DenseTensors([b, a])
    g = a.refs[1]
    c = sf.dense_tensor(b.refs[0], g, b.refs[2], b.refs[3])
    sf.DenseTensors([a, c])                                # one gradient for two tensors is only read
    half = sf.dense_tensor(*(x[:n // 2] for x in (b.refs[0], g, b.refs[2], b.refs[3])))
    sf.DenseTensors([a, half])


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("other", range(4))
@pytest.mark.parametrize("shift", [0, 4, -4, 300, 596])
def test_overlaps_are_refused(sf, which, other, shift):
    """The second tensor's weights, gradient or moments over the first one's, whole or by four elements."""
    flat, (a, b), n = parts(sf)
    refs = list(b.refs[:4])
    start = (other * n + shift) % flat.numel()
    if start + n > flat.numel():
        start = 0
    refs[which] = flat[start:start + n]
    clash = sf.dense_tensor(*refs)
    spans = [(x.data_ptr(), x.data_ptr() + 4 * n, k != 1) for d in (a, clash) for k, x in enumerate(d.refs[:4])]
    bad = any(p < r and q < o and (w or v) for i, (p, o, w) in enumerate(spans) for q, r, v in spans[i + 1:])
    if bad:
        with pytest.raises(ValueError, match="twice"):
            sf.DenseTensors([a, clash])
    else:
        sf.DenseTensors([a, clash])


def test_weights_as_their_own_gradient_are_refused(sf):
    flat, (a, b), n = parts(sf)
    with pytest.raises(ValueError, match="gradient"):
        sf.DenseTensors([sf.dense_tensor(a.refs[0], a.refs[0], a.refs[2], a.refs[3])])
