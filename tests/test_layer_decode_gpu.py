"""moe_mlp where the few-token kernels do not apply (groups of 96 codes, x off 16 bytes): by
the products' decode kernels f32 values keep their bits, and infinities and NaN reach the
results of their token alone."""

import numpy as np
import pytest
import torch

import moe_expert_routed_b200 as M
from tests import layer_ref as LR
from tests.test_layer_gpu import build, check, inputs
from workloads.gen import DT_BF16, DT_F16, DT_F32, FMT_AFFINE

pytestmark = pytest.mark.gpu


def layer_of(m, x_dtype, gs=96, **kw):
    return LR.Layer(m=m, hidden=480, inter=192, top_k=2, E=40, fmt=FMT_AFFINE, bits=4, gs=gs, x_dtype=x_dtype, seed=m, **kw)


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16, DT_F32])
@pytest.mark.parametrize("m", [1, 3, 40])
def test_non_finite_values_reach_the_results(m, x_dtype):
    L = layer_of(m, x_dtype)
    layer = build(L, out_dtype=DT_F32)
    x, ids, w = inputs(L)
    want = layer(x, ids, w)
    check(L, want, DT_F32)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2 = x.clone()
        x2[m // 2, 7] = bad
        out = layer(x2, ids, w)
        keep = [t for t in range(m) if t != m // 2]
        assert torch.equal(out[keep], want[keep])
        assert not torch.isfinite(out[m // 2]).any()


@pytest.mark.parametrize("m", [1, 40])
def test_infinite_h_reaches_the_results(m):
    """gate * up past f32's largest value."""
    L = layer_of(m, DT_F32)
    layer = build(L, out_dtype=DT_F32)
    x, ids, w = inputs(L)
    x = x.clone()
    x[0] *= 2.0**80
    out = layer(x, ids, w)
    assert not torch.isfinite(out[0]).any() and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("gs,off", [(96, 0), (64, 4)])
@pytest.mark.parametrize("m", [1, 5, 40])
def test_f32_values_keep_their_bits(m, gs, off):
    """By the norm: sums of f32 products in f32, or of 24-bit fixed point (480 and 192 terms, a few 2^-24
    each of their root mean square), the activation's 4e-6 of the few values that cancel: below
    2^-20."""
    L = layer_of(m, DT_F32, gs=gs) if gs == 96 else LR.Layer(m=m, hidden=512, inter=192, top_k=2, E=40, fmt=FMT_AFFINE,
                                                               bits=4, gs=gs, x_dtype=DT_F32, seed=m)
    layer = build(L, out_dtype=DT_F32)
    x, ids, w = inputs(L)
    if off:  # x a word off a 16-byte boundary: not for the few-token kernels
        x = torch.cat([torch.zeros(off // 4, device="cuda"), x.flatten()])[off // 4:].view(m, -1)
        assert x.data_ptr() % 16 == off
    got = layer(x, ids, w).cpu().double().numpy()
    ref = L.reference(DT_F32)[0]
    assert np.linalg.norm(got - ref) <= 2.0**-20 * np.linalg.norm(ref)
    assert M.poll_error(layer.workspace) == 0
