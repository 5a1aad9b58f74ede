"""The operators around the product (moe_gate_topk, moe_mlp, moe_combine) on the GPU
against 64-bit references: the router's choice to the bit, the sums within bounds
derived from the roundings each path makes."""

import numpy as np
import pytest
import torch

import moe_expert_routed_b200 as M
from tests import layer_ref as LR
from workloads.gen import (DT_BF16, DT_F16, DT_F32, FMT_AFFINE, FMT_CODEBOOK, FMT_MXFP4, FMT_NVFP4)
from workloads.torch_io import to_device

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------- gate


def gate_tol(l, k):
    """f32 softmax: exp within 2 units in the last place of an argument off by
    |l - max| 2^-24, a sum of at most E terms in a tree, one division, one product."""
    span = float(np.nanmax(l[np.isfinite(l)]) - np.nanmin(l[np.isfinite(l)])) if np.isfinite(l).any() else 0.0
    return (2 * 2 + 2 * span + 37 + 3) * 2.0**-24


@pytest.mark.parametrize("dtype", [DT_F32, DT_BF16, DT_F16])
@pytest.mark.parametrize("m,E,k", [(1, 128, 8), (1, 1, 1), (3, 8, 8), (257, 160, 6), (5, 31, 4), (2, 33, 32),
                                   (1000, 256, 8), (7, 1000, 16), (4, 1024, 32), (9, 64, 1), (6, 512, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "bias"])
def test_gate_choice_and_weights(m, E, k, score, dtype):
    rng = np.random.default_rng(m * 7 + E + k)
    t = torch.from_numpy(rng.standard_normal((m, E)).astype(np.float32) * 2).to(LR.TORCH_DT[dtype])
    b = rng.standard_normal(E).astype(np.float32) * 0.1 if score == "bias" else None
    name = "sigmoid" if score == "bias" else score
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        ids, w = M.gate_topk(t.cuda(), k, score=name, renormalize=renorm, scale=scale,
                             select_bias=torch.from_numpy(b).cuda() if b is not None else None)
        l = t.double().numpy()
        ri, rw = LR.gate(l, k, name, b, renorm, scale)
        assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), ri)
        assert np.all(np.abs(w.cpu().double().numpy() - rw) <= gate_tol(l, k) * np.abs(rw) + 1e-38)


def test_gate_ties_go_to_the_lowest_expert():
    l = torch.zeros(4, 100)
    l[1, 50:] = 1.0
    l[2, ::3] = -0.0          # -0 and +0 tie
    l[3] = torch.arange(100) // 10
    ids, w = M.gate_topk(l.cuda(), 12)
    want = LR.gate(l.double().numpy(), 12, "softmax")[0]
    assert np.array_equal(ids.cpu().numpy(), want)
    assert ids[2].tolist() == list(range(12)) and ids[3].tolist()[:3] == [90, 91, 92]
    ids, _ = M.gate_topk(l.cuda(), 12, score="sigmoid", select_bias=torch.zeros(100).cuda())
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("near", [1, 12, 40, 300])
def test_gate_selection_bias_decided_in_64_bits(near):
    """Scores that 32 bits cannot tell apart, a few of them and more than a warp holds, at
    the cut and above it; selection biases that are large, infinite and NaN."""
    rng = np.random.default_rng(near)
    m, E, k = 9, 400, 10
    l = rng.standard_normal((m, E)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for t in range(m):
        at = rng.permutation(E)[:near]
        l[t, at] = 18 + rng.permutation(near) * 2.0**-7  # sigmoid within 2^-26 of 1
        b[at] = 1.0
    b[:4] = [1e6, -1e6, np.inf, -np.inf]
    ids, _ = M.gate_topk(torch.from_numpy(l).cuda(), k, score="sigmoid", select_bias=torch.from_numpy(b).cuda())
    assert np.array_equal(ids.cpu().numpy(), LR.gate(l, k, "sigmoid", b)[0])
    b[5] = np.nan
    ids, _ = M.gate_topk(torch.from_numpy(l).cuda(), k, score="sigmoid", select_bias=torch.from_numpy(b).cuda())
    b[5] = -np.inf  # NaN below every number, and no -inf among the first k
    assert np.array_equal(ids.cpu().numpy(), LR.gate(l, k, "sigmoid", b)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_masked_and_non_finite_logits(score):
    inf, nan = float("inf"), float("nan")
    l = torch.randn(6, 40, generator=torch.Generator().manual_seed(3))
    l[0, 5:] = -inf            # fewer left than chosen
    l[1] = -inf                # nothing left
    l[2, ::2] = -inf
    l[3, 7] = nan              # ranks below everything
    l[4, :] = torch.finfo(torch.float32).min
    for renorm in (True, False):
        ids, w = (v.cpu() for v in M.gate_topk(l.cuda(), 8, score=score, renormalize=renorm))
        assert sorted(ids[0, :5].tolist()) == [0, 1, 2, 3, 4] and ids[0, 5:].tolist() == [5, 6, 7]
        assert (w[0, 5:] == 0).all() and (w[0, :5] > 0).all()
        assert (not renorm) or abs(float(w[0].sum()) - 1) < 1e-6
        assert ids[1].tolist() == list(range(8)) and (w[1] == 0).all()
        assert (ids[2] % 2 == 1).all() and torch.isfinite(w[2]).all()
        assert 7 not in ids[3].tolist()
        if score == "softmax" and not renorm:
            assert torch.isnan(w[3]).all()
        else:
            assert torch.isfinite(w[3]).all()
        assert ids[4].tolist() == list(range(8))
        if score == "softmax":
            assert torch.allclose(w[4], torch.full((8,), 1 / 8 if renorm else 1 / 40), rtol=1e-6)
        assert torch.isfinite(w[5]).all()


def test_gate_sigmoid_far_below_zero_still_renormalises():
    l = torch.full((1, 16), -200.0)
    l[0, 3] = -199.0
    ids, w = M.gate_topk(l.cuda(), 2, score="sigmoid")
    assert ids[0].tolist() == [3, 0]
    e = np.exp(1.0)
    assert np.allclose(w.cpu().double().numpy()[0], [e / (1 + e), 1 / (1 + e)], rtol=1e-6, atol=0)


def test_gate_writes_given_outputs_and_nothing_else():
    l = torch.randn(5, 24).cuda()
    buf_i = torch.full((7, 3), -5, dtype=torch.int32, device="cuda")
    buf_w = torch.full((7, 3), 9.0, device="cuda")
    ids, w = M.gate_topk(l, 3, ids=buf_i[1:6], weights=buf_w[1:6])
    assert ids.data_ptr() == buf_i[1:].data_ptr()
    assert (buf_i[[0, 6]] == -5).all() and (buf_w[[0, 6]] == 9.0).all() and (buf_i[1:6] >= 0).all()


# ------------------------------------------------------------------- combine


@pytest.mark.parametrize("dz", [DT_F32, DT_BF16, DT_F16])
@pytest.mark.parametrize("do", [DT_F32, DT_BF16, DT_F16])
@pytest.mark.parametrize("m,S,n", [(1, 8, 2816), (77, 6, 1001), (3, 1, 1), (5, 16, 64), (1, 2, 7), (300, 4, 130)])
def test_combine_matches_the_sum(m, S, n, dz, do):
    rng = np.random.default_rng(m + S + n)
    z = torch.from_numpy(rng.standard_normal((m, S, n)).astype(np.float32)).to(LR.TORCH_DT[dz])
    w = torch.from_numpy(rng.standard_normal((m, S)).astype(np.float32))
    r = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(LR.TORCH_DT[do])
    ids = torch.from_numpy(rng.integers(0, 5, (m, S)).astype(np.int32))
    for res, idt in ((None, None), (r, None), (r, ids), (None, ids)):
        zz, wd = z.clone(), w.double()
        if idt is not None:  # pairs left out are not read, whatever they hold
            wd = torch.where(idt < 4, wd, 0.0)
            zz[idt >= 4] = float("nan")
        out = M.combine(zz.cuda(), w.cuda(), ids=idt.cuda() if idt is not None else None,
                        num_experts=4 if idt is not None else None,
                        residual=res.cuda() if res is not None else None, out_dtype=LR.TORCH_DT[do])
        terms = wd.numpy()[:, :, None] * z.double().numpy()
        ref, mag = terms.sum(1), np.abs(terms).sum(1)
        if res is not None:
            ref, mag = ref + res.double().numpy(), mag + np.abs(res.double().numpy())
        tol = (S + 1) * 2.0**-24 * mag
        tol += LR.HALF_STEP[do] * (np.abs(ref) + tol) + LR.TINY[do]
        assert np.all(np.abs(out.cpu().double().numpy() - ref) <= tol)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_combine_unaligned_rows_and_in_place_residual(off):
    """Views off a 16-byte boundary; the residual may be the output itself; the
    elements around the output stay as they were."""
    g = torch.Generator().manual_seed(5)
    zb = torch.randn(off + 4 * 3 * 96, generator=g).to(torch.bfloat16).cuda()
    z = zb[off:].view(4, 3, 96)
    w = torch.rand(4, 3, generator=g).cuda()
    ob = torch.randn(off + 4 * 96 + 8, generator=g).to(torch.bfloat16).cuda()
    before = ob.clone()
    out = ob[off:off + 4 * 96].view(4, 96)
    want = out.double() + (w.double()[:, :, None] * z.double()).sum(1)
    mag = out.double().abs() + (w.double()[:, :, None] * z.double()).abs().sum(1)
    M.combine(z, w, residual=out, out=out)
    assert ((out.double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-20 * mag).all()
    assert torch.equal(ob[:off], before[:off]) and torch.equal(ob[off + 4 * 96:], before[off + 4 * 96:])


# ----------------------------------------------------------------------- mlp


def build(L, *, out_dtype, max_tokens=None, path="auto", workspace=None):
    gu, dn = to_device(L.gu), to_device(L.dn)
    b = L.bias
    return M.MoeMlp(
        M.ExpertWeights(gu["packed"], gu["scales"], gu["aux"], fmt=L.gu.fmt, bits=L.gu.bits,
                        group_size=L.gu.group_size, bias=torch.from_numpy(b[0]).cuda() if b else None),
        M.ExpertWeights(dn["packed"], dn["scales"], dn["aux"], fmt=L.dn.fmt, bits=L.dn.bits,
                        group_size=L.dn.group_size,
                        bias=torch.from_numpy(b[1]).cuda().to(torch.bfloat16).float() if b else None),
        hidden=L.hidden, inter=L.inter, num_experts=L.E, n_expert_used=L.top_k, max_tokens=max_tokens or L.m,
        x_dtype=LR.TORCH_DT[L.x_dtype], out_dtype=LR.TORCH_DT[out_dtype], act=L.act, path=path, workspace=workspace)


def inputs(L):
    d = to_device(L.gu)
    return d["x"], d["ids"], torch.from_numpy(L.w).cuda()


def check(L, out, out_dtype, residual=None):
    ref, tol, rms = L.reference(out_dtype, residual)
    got = out.detach().cpu().double().numpy()
    if out_dtype == DT_F16:  # values from 65520 on round to infinity
        over = np.isinf(got) & (got * ref > 0) & (np.abs(ref) + tol >= 65520)
        got = np.where(over, ref, got)
    err = np.abs(got - ref)
    assert np.isfinite(err).all() and np.all(err <= tol), f"worst err / bound {np.max(err / tol):.3g}"
    assert np.linalg.norm(err) <= np.linalg.norm(rms), f"{np.linalg.norm(err) / np.linalg.norm(rms):.3g} of the norm"


AFF4, AFF6, AFF8 = (FMT_AFFINE, 4, 64), (FMT_AFFINE, 6, 64), (FMT_AFFINE, 8, 32)
CB2, CB3, CB4 = (FMT_CODEBOOK, 2, 64), (FMT_CODEBOOK, 3, 32), (FMT_CODEBOOK, 4, 32)
NVFP4, MXFP4 = (FMT_NVFP4, 4, 16), (FMT_MXFP4, 4, 32)
FORMATS = dict(aff4=AFF4, aff4g32=(FMT_AFFINE, 4, 32), aff4g128=(FMT_AFFINE, 4, 128), aff6=AFF6, aff8=AFF8,
               cb2=CB2, cb3=CB3, cb4=CB4, nvfp4=NVFP4, mxfp4=MXFP4)


@pytest.mark.parametrize("m", [1, 2, 5, 40])
@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16, DT_F32])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_mlp_matches_the_layer(fmt, x_dtype, m):
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=384, inter=256, top_k=4, E=12, fmt=f, bits=bits, gs=gs, x_dtype=x_dtype, seed=m)
    od = DT_F32 if m == 2 else x_dtype
    x, ids, w = inputs(L)
    layer = build(L, out_dtype=od)
    check(L, layer(x, ids, w), od)
    assert M.poll_error(layer.workspace) == 0


SHAPES = [  # m, hidden, inter, top_k, E, format, down's format
    (1, 2816, 704, 8, 16, AFF4, None), (3, 1376, 352, 3, 10, (FMT_AFFINE, 4, 32), None),
    (1, 64, 32, 1, 1, (FMT_AFFINE, 4, 32), None), (6, 32, 32, 2, 3, (FMT_AFFINE, 4, 32), None),
    (8, 1024, 160, 8, 8, NVFP4, None), (4, 544, 96, 2, 5, MXFP4, None), (2, 200, 48, 2, 4, (FMT_AFFINE, 8, 8), None),
    (7, 256, 128, 3, 6, AFF4, AFF6), (5, 512, 256, 4, 9, CB3, NVFP4), (33, 256, 64, 6, 20, AFF4, None),
    (24, 512, 64, 2, 64, NVFP4, MXFP4), (130, 256, 128, 4, 8, AFF4, AFF8), (16, 96, 64, 4, 4, (FMT_AFFINE, 4, 32), None),
    (64, 256, 64, 8, 40, NVFP4, None), (63, 160, 96, 8, 200, (FMT_AFFINE, 4, 32), None), (40, 128, 64, 12, 16, CB3, CB4),
    (65, 128, 64, 2, 70, AFF6, None), (17, 192, 64, 16, 300, AFF8, CB2), (2, 4096, 128, 1, 3, CB2, AFF8),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(v) for v in s[:5]))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf"])
def test_mlp_shapes_biases_residual(shape, act):
    m, hidden, inter, k, E, (f, bits, gs), down = shape
    L = LR.Layer(m=m, hidden=hidden, inter=inter, top_k=k, E=E, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16,
                 act=act, seed=hidden, down=down, bias=act != "silu")
    if L.bias:  # the down bias is given as bf16 values
        L.bias = (L.bias[0], torch.from_numpy(L.bias[1]).to(torch.bfloat16).float().numpy())
    x, ids, w = inputs(L)
    res = torch.from_numpy(L.res).to(torch.bfloat16).cuda()
    layer = build(L, out_dtype=DT_BF16, max_tokens=m + 3)
    r64 = res.double().cpu().numpy()
    check(L, layer(x, ids, w, residual=res), DT_BF16, r64)
    layer(x, ids, w, residual=res, out=res)  # in place
    check(L, res, DT_BF16, r64)


@pytest.mark.parametrize("path", ["decode", "grouped"])
@pytest.mark.parametrize("m", [3, 24, 64])
@pytest.mark.parametrize("fmt", ["aff4", "aff4g32", "nvfp4", "cb3", "aff6"])
def test_mlp_paths_agree_with_the_layer(fmt, m, path):
    """Both ways at many pairs an expert (several passes of the few-token kernels)."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=256, inter=192, top_k=3, E=4, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16, seed=m + 40)
    layer = build(L, out_dtype=DT_BF16, path=path)
    check(L, layer(*inputs(L)), DT_BF16)


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16, DT_F32])
@pytest.mark.parametrize("m", [1, 6])
def test_mlp_wide_range_of_x(x_dtype, m):
    """Units of very different sizes, zeros and subnormals: each unit has a scale of its own."""
    L = LR.Layer(m=m, hidden=512, inter=128, top_k=4, E=8, fmt=FMT_AFFINE, bits=4, gs=64, x_dtype=x_dtype, seed=70)
    x = torch.randn(m, 512, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    x *= torch.exp2(torch.linspace(-30 if x_dtype != DT_F16 else -12, 6, 16)).repeat_interleave(32)
    x[:, 64:96] = 0
    x[:, 100:104] = 2.0**-24
    t = x.to(LR.TORCH_DT[x_dtype])
    bits_ = t.float().numpy() if x_dtype == DT_F32 else t.view(torch.int16).numpy().view(np.uint16)
    L.gu = L.gu.with_x(bits_)
    layer = build(L, out_dtype=DT_F32)
    check(L, layer(*inputs(L)), DT_F32)


@pytest.mark.parametrize("fmt,most", [("aff4", 58), ("aff4g32", 58), ("aff6", 56), ("aff8", 54), ("nvfp4", 59),
                                      ("cb3", 59)])
@pytest.mark.parametrize("m", [2, 40])
def test_mlp_huge_and_tiny_values(fmt, most, m):
    """h up to about 2^120, and about 2^-85: the factors of its units stay in f32's range."""
    f, bits, gs = FORMATS[fmt]
    for scale in (2.0**most, 2.0**-45):
        L = LR.Layer(m=m, hidden=256, inter=128, top_k=2, E=8, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16, seed=77)
        x = torch.randn(m, 256, generator=torch.Generator().manual_seed(4), dtype=torch.float64) * scale
        L.gu = L.gu.with_x(x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))
        L.w = (L.w * 2.0**-12).astype(np.float32)
        check(L, build(L, out_dtype=DT_BF16)(*inputs(L)), DT_BF16)


@pytest.mark.parametrize("x_dtype", [DT_BF16, DT_F16])
@pytest.mark.parametrize("fmt", sorted(FORMATS))
def test_mlp_tens_of_pairs_an_expert(fmt, x_dtype):
    """Sizes between the few-token kernels and the grouped products: tiles of every number
    of blocks of 8 pairs, more than one tile an expert, an expert without pairs, rows of
    weights and of values that end inside a step; values of very different sizes."""
    f, bits, gs = FORMATS[fmt]
    hidden, inter = (320, 224) if gs < 64 else (320, 192) if gs == 64 else (384, 128)
    L = LR.Layer(m=60, hidden=hidden, inter=inter, top_k=3, E=6, fmt=f, bits=bits, gs=gs, x_dtype=x_dtype, seed=5,
                 bias=True)
    ids = np.tile(np.arange(3), (60, 1))
    ids[:50, 2] = 3 + (np.arange(50) >= 11)  # 60, 60, 10, 11 and 39 pairs, none
    L.gu = L.gu.with_ids(ids.astype(np.uint32))
    x = torch.randn(60, hidden, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    x[7] *= torch.exp2(torch.linspace(-12, 6, hidden // 32)).repeat_interleave(32)
    x[9] = 0
    t = x.to(LR.TORCH_DT[x_dtype])
    L.gu = L.gu.with_x(t.view(torch.int16).numpy().view(np.uint16))
    L.bias = (L.bias[0], torch.from_numpy(L.bias[1]).to(torch.bfloat16).float().numpy())
    res = torch.from_numpy(L.res).to(t.dtype).cuda()
    layer = build(L, out_dtype=x_dtype, max_tokens=61)
    out = layer(*inputs(L), residual=res)
    check(L, out, x_dtype, res.double().cpu().numpy())
    assert torch.equal(out, layer(*inputs(L), residual=res))
    assert M.poll_error(layer.workspace) == 0


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("m", [1, 7])
def test_mlp_few_tokens_keep_32_bits(fmt, m):
    """f32 results of the few-token kernels against 64 bits, by the 2-norm.

    A unit's 32 products and their sums are cut 23 bits below the largest term, which is
    up to three times the terms' root mean square s: 34 cuts, each uniform over a step of
    2^-23 * 3 s with either sign (0.58 of a step), against a sum of about sqrt(32) s:
    sqrt(34) * 0.58 * 3 / sqrt(32) * 2^-23 = 1.8 * 2^-23. gate and up (each 1.8, and slopes
    up to 1.2 of the activation: 2.8) and down (1.8) make 3.3 * 2^-23; x and h, split into two
    f16 terms, add 2^-24 each, the f32 sums of the units and the activation's 4e-6 of the
    few that cancel less than the rest: below 8 * 2^-23."""
    f, bits, gs = FORMATS[fmt]
    L = LR.Layer(m=m, hidden=512, inter=256, top_k=4, E=9, fmt=f, bits=bits, gs=gs, x_dtype=DT_F32, seed=90 + m)
    got = build(L, out_dtype=DT_F32, path="decode")(*inputs(L)).cpu().double().numpy()
    ref = L.reference(DT_F32)[0]
    assert np.linalg.norm(got - ref) <= 2.0**-20 * np.linalg.norm(ref)


def test_mlp_rows_do_not_mix():
    """A token with NaN and one with infinities leave the other tokens' results alone."""
    L = LR.Layer(m=6, hidden=256, inter=128, top_k=2, E=2, fmt=FMT_AFFINE, bits=4, gs=32, x_dtype=DT_BF16, seed=12)
    layer = build(L, out_dtype=DT_BF16)
    x, ids, w = inputs(L)
    want = layer(x, ids, w)
    x = x.clone()
    x[1, 3] = float("nan")
    x[4, 200] = float("inf")
    out = layer(x, ids, w)
    keep = [0, 2, 3, 5]
    assert torch.equal(out[keep], want[keep])
    assert not torch.isfinite(out[1]).any() and not torch.isfinite(out[4]).any()


def test_mlp_leaves_other_rows_of_out_alone():
    L = LR.Layer(m=3, hidden=128, inter=64, top_k=2, E=5, fmt=FMT_MXFP4, bits=4, gs=32, x_dtype=DT_F32, seed=13)
    layer = build(L, out_dtype=DT_F32, max_tokens=9)
    x, ids, w = inputs(L)
    buf = torch.full((5, 128), 7.0, device="cuda")
    layer(x, ids, w, out=buf[1:4])
    check(L, buf[1:4], DT_F32)
    assert (buf[[0, 4]] == 7.0).all()


@pytest.mark.parametrize("m", [1, 4, 60])
@pytest.mark.parametrize("fmt", ["aff4", "nvfp4", "cb3"])
def test_mlp_ids_out_of_range_are_left_out(fmt, m):
    f, bits, gs = FORMATS[fmt]
    bad = [(0, 1, 12)] + ([(m - 1, s, 0xFFFFFFFF) for s in range(4)] if m > 1 else [])
    L = LR.Layer(m=m, hidden=256, inter=128, top_k=4, E=12, fmt=f, bits=bits, gs=gs, x_dtype=DT_BF16, seed=9,
                 bad_ids=bad)
    x, ids, w = inputs(L)
    w = w.clone()
    for t, s, _ in bad:
        w[t, s] = float("nan")  # not read into the sum
    layer = build(L, out_dtype=DT_BF16)
    out = layer(x, ids, w)
    assert M.poll_error(layer.workspace) == 5
    check(L, out, DT_BF16)
    if m > 1:
        assert (out[m - 1] == 0).all()


def test_mlp_repeated_experts_in_a_token():
    """The same expert in several slots of a token counts each time."""
    L = LR.Layer(m=5, hidden=256, inter=128, top_k=4, E=6, fmt=FMT_AFFINE, bits=4, gs=64, x_dtype=DT_BF16, seed=4)
    i = L.gu.ids.copy()
    i[0] = 2
    i[1, 1] = i[1, 0]
    i[3] = i[4]
    L.gu = L.gu.with_ids(i)
    layer = build(L, out_dtype=DT_BF16)
    check(L, layer(*inputs(L)), DT_BF16)


@pytest.mark.parametrize("m", [20, 64])
def test_mlp_all_tokens_on_one_expert(m):
    L = LR.Layer(m=m, hidden=256, inter=96, top_k=2, E=40, fmt=FMT_AFFINE, bits=4, gs=32, x_dtype=DT_F16, seed=5)
    i = L.gu.ids.copy()
    i[:, 0], i[:, 1] = 7, 31
    L.gu = L.gu.with_ids(i)
    layer = build(L, out_dtype=DT_F16)
    check(L, layer(*inputs(L)), DT_F16)


def test_layer_run_together_and_in_a_graph():
    """Router, layer and a later combine as one program: eager, on another stream,
    and captured with other inputs at each replay."""
    m, E, k = 4, 16, 4
    L = LR.Layer(m=m, hidden=512, inter=128, top_k=k, E=E, fmt=FMT_AFFINE, bits=4, gs=64, x_dtype=DT_BF16, seed=6)
    layer = build(L, out_dtype=DT_BF16)
    x = inputs(L)[0]
    logits = torch.randn(m, E, generator=torch.Generator().manual_seed(1)).cuda()

    def program(x, logits, out):
        ids, w = M.gate_topk(logits, k)
        return layer(x, ids, w, residual=x, out=out)

    def want(x, logits):
        ids, w = LR.gate(logits.cpu().double().numpy(), k, "softmax")
        L.gu = L.gu.with_ids(ids.astype(np.uint32)).with_x(x.view(torch.int16).cpu().numpy().view(np.uint16))
        L.w = w.astype(np.float32)
        return x.double().cpu().numpy()

    out = torch.empty_like(x)
    program(x, logits, out)
    check(L, out, DT_BF16, want(x, logits))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out2 = torch.empty_like(x)
        program(x, logits, out2)
    s.synchronize()
    assert torch.equal(out, out2)
    graph = torch.cuda.CUDAGraph()
    gx, gl, go = x.clone(), logits.clone(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        program(gx, gl, go)
    for seed in (11, 12):
        g = torch.Generator().manual_seed(seed)
        gx.copy_(torch.randn(m, 512, generator=g).to(torch.bfloat16))
        gl.copy_(torch.randn(m, E, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        check(L, go, DT_BF16, want(gx, gl))
    # and by parts: the products of qmm_id, combined
    ids, w = M.gate_topk(gl, k)
    gu, dn = to_device(L.gu), to_device(L.dn)
    h = M.qmm_id(gx, ids, gu["packed"], gu["scales"], gu["aux"], n=256, group_size=64, bits=4, fmt=FMT_AFFINE,
                 num_experts=E, act="silu", out_dtype=torch.float32)
    z = M.qmm_id(h.view(m * k, 128), ids.view(m * k, 1), dn["packed"], dn["scales"], dn["aux"], n=512,
                 group_size=64, bits=4, fmt=FMT_AFFINE, num_experts=E)
    out3 = M.combine(z.view(m, k, 512), w, residual=gx, out_dtype=torch.bfloat16)
    check(L, out3, DT_BF16, want(gx, gl))


def test_two_layers_on_two_streams():
    """Layers with workspaces of their own overlap freely."""
    Ls = [LR.Layer(m=3, hidden=512, inter=256, top_k=4, E=8, fmt=FMT_AFFINE, bits=4, gs=64, x_dtype=DT_BF16,
                   seed=20 + i) for i in range(2)]
    layers = [build(L, out_dtype=DT_BF16) for L in Ls]
    ins = [inputs(L) for L in Ls]
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(layers[i](*ins[i]))
    torch.cuda.synchronize()
    for i, L in enumerate(Ls):
        check(L, outs[i][0], DT_BF16)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])


@pytest.mark.parametrize("m,E,k", [(700, 256, 8), (300, 1024, 8), (128, 4, 1), (129, 4, 1), (90, 1, 1)])
def test_mlp_many_experts_and_pairs(m, E, k):
    """More pairs than one CTA routes, the most experts, the last size of tens of pairs an
    expert and the first of the next way, one expert."""
    L = LR.Layer(m=m, hidden=64, inter=32, top_k=k, E=E, fmt=FMT_AFFINE, bits=4, gs=32, x_dtype=DT_BF16, seed=m)
    layer = build(L, out_dtype=DT_BF16, max_tokens=m + 200)
    out = layer(*inputs(L))
    check(L, out, DT_BF16)
    assert torch.equal(out, layer(*inputs(L)))


def test_layers_of_tens_of_pairs_overlap_and_replay():
    """Two layers on two streams, eager and captured at once, one of them also at fewer
    tokens in between: the same results as alone."""
    Ls = [LR.Layer(m=48, hidden=256, inter=160, top_k=4, E=8, fmt=f, bits=b, gs=g, x_dtype=DT_BF16, seed=30 + b)
          for f, b, g in ((FMT_AFFINE, 8, 32), (FMT_CODEBOOK, 3, 32))]
    layers = [build(L, out_dtype=DT_BF16) for L in Ls]
    ins = [inputs(L) for L in Ls]
    want = [layer(*i) for layer, i in zip(layers, ins)]
    few = layers[0](ins[0][0][:2], ins[0][1][:2], ins[0][2][:2])
    for L, w in zip(Ls, want):
        check(L, w, DT_BF16)
    graphs, gout = [], []
    for layer, i in zip(layers, ins):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gout.append(layer(*i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((want[n], layers[n](*ins[n])))
                if n == 0:
                    outs.append((few, layers[0](ins[0][0][:2], ins[0][1][:2], ins[0][2][:2])))
                gout[n].zero_()
                graphs[n].replay()
                outs.append((want[n], gout[n].clone()))
    torch.cuda.synchronize()
    assert all(torch.equal(w, o) for w, o in outs)


def test_mlp_tens_of_pairs_rows_do_not_mix():
    """A token with NaN, one with infinities and one without an expert leave the other
    tokens' results alone."""
    L = LR.Layer(m=40, hidden=256, inter=128, top_k=2, E=4, fmt=FMT_AFFINE, bits=4, gs=32, x_dtype=DT_BF16, seed=12)
    layer = build(L, out_dtype=DT_BF16)
    x, ids, w = inputs(L)
    want = layer(x, ids, w)
    x2, ids2 = x.clone(), ids.clone()
    x2[3] = float("nan")
    x2[17, 5] = float("inf")
    ids2[30] = 4
    out = layer(x2, ids2, w)
    keep = [t for t in range(40) if t not in (3, 17, 30)]
    assert torch.equal(out[keep], want[keep])
    assert out[3].isnan().all() and not out[17].isfinite().any()
    assert torch.count_nonzero(out[30]) == 0 and M.poll_error(layer.workspace) != 0


def test_mlp_refusals():
    L = LR.Layer(m=3, hidden=128, inter=64, top_k=2, E=4, fmt=FMT_AFFINE, bits=4, gs=32, x_dtype=DT_BF16, seed=8)
    layer = build(L, out_dtype=DT_BF16)
    x, ids, w = inputs(L)
    for bad in (lambda: layer(x[:0], ids[:0], w[:0]),                 # no tokens
                lambda: layer(torch.cat([x, x]), torch.cat([ids, ids]), torch.cat([w, w])),  # over max_tokens
                lambda: layer(x.float(), ids, w), lambda: layer(x, ids.long(), w), lambda: layer(x, ids, w.half()),
                lambda: layer(x[:, :64].contiguous(), ids, w), lambda: layer(x.t().contiguous().t(), ids, w),
                lambda: layer(x, ids, w, residual=x.float()), lambda: layer(x, ids, w, out=x.float()),
                lambda: layer(x.cpu(), ids, w)):
        with pytest.raises(ValueError):
            bad()
    check(L, layer(x, ids, w), DT_BF16)
