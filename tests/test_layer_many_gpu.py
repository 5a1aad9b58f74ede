"""moe_mlp with a hundred pairs an expert and more (tiles of 256 pairs, the f16 image of x,
routing shared by the two products) against 64 bits: every format, biases, ids out of
range, experts of more than one tile and of none; weights far outside f16's range."""

import numpy as np
import pytest
import torch

import moe_expert_routed_b200 as M
from tests import layer_ref as LR
from tests.test_layer_gpu import build, check, inputs
from workloads.gen import (DT_BF16, DT_F16, DT_F32, FMT_AFFINE, FMT_CODEBOOK, FMT_MXFP4, FMT_NVFP4, Problem, bf16_bits,
                           f16_bits)

pytestmark = pytest.mark.gpu

FORMATS = dict(aff4=(FMT_AFFINE, 4, 32), aff6=(FMT_AFFINE, 6, 32), aff8=(FMT_AFFINE, 8, 32), cb2=(FMT_CODEBOOK, 2, 32),
               cb3=(FMT_CODEBOOK, 3, 32), cb4=(FMT_CODEBOOK, 4, 32), nvfp4=(FMT_NVFP4, 4, 16), mxfp4=(FMT_MXFP4, 4, 32))
ACTS = ("silu", "gelu_tanh", "gelu_erf")
M_TOKENS, E = 300, 4


def layer_of(fmt, x_dtype, bias=False, act="silu", hidden=352, inter=224, seed=3, bad=()):
    """300 tokens: 300 pairs of expert 0 (a tile of 256 and one of 44), 190 of expert 1, 110 of
    expert 2, none of expert 3."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=M_TOKENS, hidden=hidden, inter=inter, top_k=2, E=E, fmt=f, bits=bits, gs=gs, x_dtype=x_dtype, act=act,
                 seed=seed, bias=bias)
    ids = np.zeros((M_TOKENS, 2), dtype=np.uint32)
    ids[:, 1] = 1 + (np.arange(M_TOKENS) % 30 >= 19)
    ids[::7] = ids[::7, ::-1]
    for t, s, v in bad:
        ids[t, s] = v
    L.gu = L.gu.with_ids(ids)
    if L.bias:  # the down bias is given as bf16 values
        L.bias = (L.bias[0], torch.from_numpy(L.bias[1]).to(torch.bfloat16).float().numpy())
    return L


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_many_pairs_an_expert(fmt, x_dtype):
    bad = [(0, 1, E), (17, 0, 0xFFFFFFFF), (299, 0, 9), (299, 1, E)]
    act = ACTS[sorted(FORMATS).index(fmt) % 3]
    L = layer_of(fmt, x_dtype, bias=True, act=act, bad=bad)
    x, ids, w = inputs(L)
    w = w.clone()
    for t, s, _ in bad:
        w[t, s] = float("nan")  # not read into the sum
    res = torch.from_numpy(L.res).to(LR.TORCH_DT[x_dtype]).cuda()
    layer = build(L, out_dtype=x_dtype, max_tokens=M_TOKENS + 40)
    layer.workspace[4:] = 255  # what lies in it does not matter (NaN in every type), but for the error word
    out = layer(x, ids, w, residual=res)
    assert M.poll_error(layer.workspace) == 5
    check(L, out, x_dtype, res.double().cpu().numpy())
    assert torch.equal(out, layer(x, ids, w, residual=res))
    assert torch.equal(out[299], res[299])


@pytest.mark.parametrize("x_dtype,out_dtype", [(DT_F32, DT_F32), (DT_BF16, DT_F32), (DT_F16, DT_BF16), (DT_F32, DT_F16)])
@pytest.mark.parametrize("fmt", ["aff4", "nvfp4"])
def test_many_pairs_other_types(fmt, x_dtype, out_dtype):
    L = layer_of(fmt, x_dtype, hidden=96, inter=64)
    check(L, build(L, out_dtype=out_dtype)(*inputs(L)), out_dtype)


def scaled(P: Problem, power: float) -> Problem:
    """Weights times a power of two (scales, and affine biases; the codebook stays)."""
    new = dict(P.__dict__)
    if P.fmt == FMT_AFFINE:
        for n in ("scales", "aux"):
            v = torch.from_numpy(new[n].view(np.int16)).view(torch.bfloat16).float().numpy()
            new[n] = bf16_bits(v * np.float32(power))
    else:
        new["scales"] = f16_bits(new["scales"].view(np.float16).astype(np.float32) * np.float32(power))
    return Problem(**new)


@pytest.mark.parametrize("which", ["gate_up", "down"])
@pytest.mark.parametrize("power", [2.0**21, 2.0**-14, 2.0**-24])
@pytest.mark.parametrize("fmt", ["aff4", "aff6", "aff8", "cb2", "cb3", "cb4"])
def test_weights_outside_the_range_of_f16(fmt, power, which):
    """bf16 tokens: weights from 2^16 up to 2^22 (f16 ends at 65,504) and down to 2^-30 (its last step
    is 2^-24). x makes up for large gates, so that h stays as it is."""
    if FORMATS[fmt][0] == FMT_CODEBOOK and power < 2.0**-14:
        power = 2.0**-17  # what f16 scales can hold
    L = layer_of(fmt, DT_BF16, hidden=128, inter=96)
    if which == "gate_up":
        L.gu = scaled(L.gu, power)
        if power > 1:
            x = torch.from_numpy(L.gu.x.view(np.int16)).view(torch.bfloat16) * 2.0**-21
            L.gu = L.gu.with_x(x.view(torch.int16).numpy().view(np.uint16))
    else:
        L.dn = scaled(L.dn, power)
    check(L, build(L, out_dtype=DT_BF16)(*inputs(L)), DT_BF16)


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16])
@pytest.mark.parametrize("fmt", ["aff4", "cb3", "nvfp4"])
def test_f32_results_of_narrow_tokens(fmt, x_dtype):
    """f32 results keep more than h in bf16 would (2^-9 each, 2^-9.8 of the norm): by the norm, the
    roundings of two-term operands, 2^-16 each of gate (slopes of the activation up to 1.2), up,
    h, down and the remainders' product, 5.2 * 2^-16, and the f32 sums and the activation, 2^-17
    together: below 2^-13."""
    L = layer_of(fmt, x_dtype, hidden=256, inter=160)
    got = build(L, out_dtype=DT_F32)(*inputs(L)).cpu().double().numpy()
    ref = L.reference(DT_F32)[0]
    assert np.linalg.norm(got - ref) <= 2.0**-13 * np.linalg.norm(ref)


@pytest.mark.parametrize("m,top_k,E_", [(5, 2, 8), (60, 3, 6), (300, 2, 4)])  # the three ways
@pytest.mark.parametrize("fmt", ["aff4", "nvfp4"])
def test_no_pair_left(fmt, m, top_k, E_):
    """Every id out of range: the residual alone, or zeros."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=128, inter=64, top_k=top_k, E=E_, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16, seed=m)
    layer = build(L, out_dtype=DT_BF16)
    x, ids, w = inputs(L)
    res = torch.from_numpy(L.res).to(torch.bfloat16).cuda()
    none = torch.full_like(ids, E_)
    assert torch.equal(layer(x, none, w, residual=res), res)
    assert torch.count_nonzero(layer(x, none, w)) == 0 and M.poll_error(layer.workspace) == 5
    check(L, layer(x, ids, w), DT_BF16)
    assert M.poll_error(layer.workspace) == 0


@pytest.mark.parametrize("fmt,x_dtype", [("nvfp4", DT_BF16), ("cb3", DT_F16), ("aff4", DT_BF16)])
def test_many_pairs_captured_and_replayed_with_other_inputs(fmt, x_dtype):
    Ls = [layer_of(fmt, x_dtype, hidden=96, inter=64, seed=s) for s in (3, 3)]
    rng = np.random.default_rng(1)
    Ls[1].gu = Ls[1].gu.with_ids(rng.integers(0, E, (M_TOKENS, 2)).astype(np.uint32)).with_x(Ls[0].gu.x[::-1].copy())
    layer = build(Ls[0], out_dtype=x_dtype)
    x, ids, w = (t.clone() for t in inputs(Ls[0]))
    layer(x, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, ids, w)
    for L in (Ls[1], Ls[0]):
        for to, t in zip((x, ids, w), inputs(L)):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        check(L, out, x_dtype)
