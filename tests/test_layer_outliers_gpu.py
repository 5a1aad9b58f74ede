"""moe_mlp with affine groups whose codes lie close together, as an outlier leaves them: code
times scale and bias are each many times the weight, so a rounding of h must meet their
difference, not one of them."""

import numpy as np
import pytest
import torch

from tests import layer_ref as LR
from tests import numpy_ref as R
from tests.test_layer_gpu import build, check, inputs
from workloads.gen import DT_BF16, DT_F16, FMT_AFFINE, Problem, bf16_bits

pytestmark = pytest.mark.gpu

# bits: (codes around the zero point, group)
NARROW = {4: (np.array([7, 8, 9]), 64), 6: (np.arange(29, 36), 32), 8: (np.arange(125, 132), 32)}


def narrow(P: Problem, rng) -> Problem:
    codes, _ = NARROW[P.bits]
    c = codes[rng.integers(0, len(codes), (P.num_experts, P.n, P.k))].astype(np.uint32)
    if P.bits == 8:
        packed = c.astype(np.uint8)
    elif P.bits == 4:
        packed = (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)
    else:  # 4 codes in 3 bytes
        word = c[..., 0::4] | c[..., 1::4] << 6 | c[..., 2::4] << 12 | c[..., 3::4] << 18
        packed = np.stack([word & 255, word >> 8 & 255, word >> 16], -1).astype(np.uint8).reshape(P.num_experts, P.n, -1)
    s = torch.from_numpy(P.scales.view(np.int16)).view(torch.bfloat16).float().numpy()
    return Problem(**{**P.__dict__, "packed": packed, "aux": bf16_bits(-np.float32(1 << (P.bits - 1)) * s)})


@pytest.mark.parametrize("dtype", [DT_BF16, DT_F16])
@pytest.mark.parametrize("m", [1, 7, 60])
@pytest.mark.parametrize("bits", sorted(NARROW))
def test_roundings_of_h_meet_the_weights(bits, m, dtype):
    """Besides the result's own rounding, h's to 11 bits: uniform, independent, at most half a step,
    2^-11 of the value: 2^-11 / sqrt(3) of it by the root of the mean square. With weights w and
    pair weights p these leave 2^-11 / sqrt(3) of the root of the sum of (p w h)^2. A tenth
    more for the chance in some thousand of them and for all sums in f32 (2^-23 of the sums of
    the codes' products, which are up to 50 times those of the weights)."""
    L = LR.Layer(m=m, hidden=256, inter=192, top_k=3, E=6, fmt=FMT_AFFINE, bits=bits, gs=NARROW[bits][1], x_dtype=dtype,
                 seed=bits + m)
    rng = np.random.default_rng(m)
    L.dn = narrow(L.dn, rng)
    out = build(L, out_dtype=dtype)(*inputs(L))
    check(L, out, dtype)
    X, G, D = R.x_f64(L.gu), R.dequant_dense(L.gu), R.dequant_dense(L.dn)
    y, S = np.zeros((m, L.hidden)), 0.0
    for t in range(m):
        for s in range(L.top_k):
            e, p = L.gu.ids[t, s], float(L.w[t, s])
            gu = G[e] @ X[t]
            h = LR.act(L.act, gu[:L.inter]) * gu[L.inter:]
            y[t] += p * (D[e] @ h)
            S += p * p * (D[e]**2 @ h**2).sum()
    err = np.linalg.norm(out.cpu().double().numpy() - y)
    own = LR.HALF_STEP[dtype] * np.linalg.norm(y)
    assert err <= 1.1 / np.sqrt(3) * np.sqrt(own**2 + (2.0**-11)**2 * S)
