"""moe_mlp where a token's largest value meets weights of zero and the others lie far below
it, at the end of the range in which 16-bit x is exact; layers called from two threads."""

import threading

import numpy as np
import pytest
import torch

from tests import layer_ref as LR
from tests.test_layer_gpu import build, check, inputs
from workloads.gen import DT_BF16, DT_F16, DT_F32, FMT_AFFINE, FMT_CODEBOOK, FMT_MXFP4, FMT_NVFP4, Problem

pytestmark = pytest.mark.gpu

FORMATS = dict(aff4=(FMT_AFFINE, 4, 32), aff8=(FMT_AFFINE, 8, 32), cb3=(FMT_CODEBOOK, 3, 32), nvfp4=(FMT_NVFP4, 4, 16),
               mxfp4=(FMT_MXFP4, 4, 32))


def without_first_unit(P: Problem) -> Problem:
    """Weights of the first 32 columns set to zero."""
    new = {n: P.__dict__[n].copy() for n in ("packed", "scales", "aux")}
    if P.fmt in (FMT_NVFP4, FMT_MXFP4):
        new["packed"][..., :16] = 0
    else:
        new["scales"][..., 0] = 0
        if P.fmt == FMT_AFFINE:
            new["aux"][..., 0] = 0
    return Problem(**{**P.__dict__, **new})


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("m,E,k", [(5, 8, 2), (60, 6, 3), (300, 4, 2)])  # the three ways
def test_values_far_below_the_largest(fmt, m, E, k):
    """bf16 values (8 bits) down to 2^-31 of the token's largest, 2^-27 where every second pair of
    4-bit affine codes meets a sixteenth: exact, so within the bounds of x of any size."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=256, inter=96, top_k=k, E=E, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16, seed=m)
    L.gu = without_first_unit(L.gu)
    g = torch.Generator().manual_seed(m)
    low = -27 if fmt == "aff4" else -31
    x = torch.exp2(low + 1.9 * torch.rand(m, 256, generator=g, dtype=torch.float64))
    x *= 1.0 - 2.0 * (torch.rand(m, 256, generator=g) < 0.5)
    x[:, 5] = 1.0  # the largest
    x *= 2.0**29   # h of ordinary size
    L.gu = L.gu.with_x(x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))
    check(L, build(L, out_dtype=DT_BF16)(*inputs(L)), DT_BF16)


def test_layers_called_from_two_threads():
    """Layers of different sizes, each with a stream and a thread of its own: kernels in common
    that need different amounts of shared memory."""
    Ls = [LR.Layer(m=m, hidden=hidden, inter=inter, top_k=4, E=8, fmt=FMT_AFFINE, bits=4, gs=64, x_dtype=dt, seed=m)
          for m, hidden, inter, dt in ((2, 2048, 256, DT_F16), (3, 256, 64, DT_F16))]
    layers = [build(L, out_dtype=L.x_dtype) for L in Ls]
    ins = [inputs(L) for L in Ls]
    torch.cuda.synchronize()
    outs, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(50):
                    outs[i].append(layers[i](*ins[i]))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 -- reported by the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for L, out in zip(Ls, outs):
        check(L, out[0], L.x_dtype)
        assert all(torch.equal(o, out[0]) for o in out)


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F32])
@pytest.mark.parametrize("fmt", ["aff4", "aff8", "nvfp4", "mxfp4", "cb3"])
@pytest.mark.parametrize("m", [3, 60])
def test_large_values_stay_finite(fmt, m, x_dtype):
    """x of about 2^100 against weights 2^-96 times as large (2^-11 where f16 scales hold no less):
    sums of 32 products with the bare codes stay in f32's range."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=128, inter=64, top_k=2, E=8, fmt=f, bits=bits, gs=gs, x_dtype=x_dtype, seed=m)
    P, down = L.gu, 0
    if f == FMT_AFFINE:
        down = 96
        half = {n: (torch.from_numpy(P.__dict__[n].view(np.int16)).view(torch.bfloat16) * 2.0**-down).view(torch.int16)
                .numpy().view(np.uint16) for n in ("scales", "aux")}
        L.gu = Problem(**{**P.__dict__, **half})
    elif f == FMT_NVFP4:
        down = 96
        L.gu = Problem(**{**P.__dict__, "aux": P.aux * np.float32(2.0**-down)})
    elif f == FMT_MXFP4:
        down = 96
        L.gu = Problem(**{**P.__dict__, "scales": (P.scales - down).astype(np.uint8)})
    else:
        down = 40  # x alone is large, gate and up with it
    x = torch.randn(m, 128, generator=torch.Generator().manual_seed(m), dtype=torch.float64) * 2.0**(down + 4)
    t = x.to(LR.TORCH_DT[x_dtype])
    L.gu = L.gu.with_x(t.numpy() if x_dtype == DT_F32 else t.view(torch.int16).numpy().view(np.uint16))
    check(L, build(L, out_dtype=x_dtype)(*inputs(L)), x_dtype)
