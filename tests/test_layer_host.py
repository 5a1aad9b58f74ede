"""The layer's operators without a GPU: their C entry points refuse bad arguments
before any CUDA call, and the binding's checks raise."""

import ctypes

import pytest
import torch

import moe_expert_routed_b200 as M


def _gate(**kw):
    a = dict(logits=16, bias=None, ids=16, weights=16, m=4, E=8, k=2, dt=0, score=0, renorm=1, scale=1.0)
    a.update(kw)
    return M.lib().moe_gate_topk(a["logits"], a["bias"], a["ids"], a["weights"], a["m"], a["E"], a["k"], a["dt"],
                                 a["score"], a["renorm"], a["scale"], None)


@pytest.mark.parametrize("kw", [dict(m=0), dict(E=0), dict(k=0), dict(k=9), dict(dt=3), dict(dt=-1), dict(score=2),
                                dict(score=-1), dict(logits=0), dict(ids=0), dict(weights=0), dict(bias=16),
                                dict(logits=18), dict(logits=17, dt=1), dict(ids=18), dict(weights=17),
                                dict(bias=18, score=1)])
def test_gate_refuses_before_cuda(kw):
    assert _gate(**kw) == 1


def test_gate_limits():
    assert _gate(E=1025) == 2
    assert _gate(E=64, k=33) == 2
    assert _gate(m=0x80000000) == 2


def _combine(**kw):
    a = dict(z=16, w=16, ids=None, res=None, out=16, m=4, S=2, n=8, E=0, dz=0, do=0)
    a.update(kw)
    return M.lib().moe_combine(a["z"], a["w"], a["ids"], a["res"], a["out"], a["m"], a["S"], a["n"], a["E"], a["dz"],
                               a["do"], None)


@pytest.mark.parametrize("kw", [dict(m=0), dict(S=0), dict(n=0), dict(z=0), dict(w=0), dict(out=0), dict(dz=3),
                                dict(do=-1), dict(ids=16, E=0), dict(z=18), dict(z=17, dz=1), dict(out=18),
                                dict(res=18), dict(w=18), dict(ids=18, E=4)])
def test_combine_refuses_before_cuda(kw):
    assert _combine(**kw) == 1


def test_combine_limits():
    assert _combine(m=1 << 30, S=4) == 2


def _mlp(gu=None, dn=None, **kw):
    a = dict(x=16, ids=16, weights=16, res=None, out=16, m=4, H=128, I=64, S=2, E=8, xd=1, od=1, act=0, ws=4096,
             wsb=1 << 24, path=0)
    a.update(kw)

    def struct(w):
        f = dict(packed=16, scales=16, aux=16, bias=None, group_size=32, bits=4, fmt=0, bias_dtype=0)
        f.update(w or {})
        return M._WeightsStruct(*(f[n] for n, _ in M._WeightsStruct._fields_))
    s1, s2 = struct(gu), struct(dn)
    p1 = None if gu == "null" else ctypes.addressof(s1)
    return M.lib().moe_mlp(a["x"], a["ids"], a["weights"], p1, ctypes.addressof(s2), a["res"], a["out"], a["m"],
                           a["H"], a["I"], a["S"], a["E"], a["xd"], a["od"], a["act"], a["ws"], a["wsb"], a["path"],
                           None)


@pytest.mark.parametrize("kw", [dict(m=0), dict(H=0), dict(I=0), dict(S=0), dict(E=0), dict(xd=3), dict(od=-1),
                                dict(act=3), dict(act=-1), dict(path=3), dict(path=0x100), dict(x=0), dict(ids=0),
                                dict(weights=0), dict(out=0), dict(ws=0), dict(ws=4097), dict(x=17), dict(out=17),
                                dict(res=17), dict(ids=18), dict(weights=18), dict(gu=dict(bits=5)),
                                dict(gu=dict(packed=None)), dict(gu=dict(scales=None)), dict(gu=dict(aux=None)),
                                dict(dn=dict(fmt=4)), dict(dn=dict(group_size=0)),
                                dict(dn=dict(bias=16, bias_dtype=3)), dict(dn=dict(fmt=2, group_size=32))])
def test_mlp_refuses_before_cuda(kw):
    assert _mlp(**kw) == 1


def test_mlp_null_weights_struct():
    a = M.lib().moe_mlp(16, 16, 16, None, None, None, 16, 4, 128, 64, 2, 8, 1, 1, 0, 4096, 1 << 24, 0, None)
    assert a == 1


def test_mlp_limits_and_workspace():
    assert _mlp(gu=dict(group_size=48)) == 2                  # hidden % group_size
    need = M.lib().moe_mlp_workspace_bytes(4, 128, 64, 2, 8, 1)
    assert need > 0 and _mlp(wsb=need - 1) == 3
    assert M.lib().moe_mlp_workspace_bytes(0, 128, 64, 2, 8, 1) == 0
    assert M.lib().moe_mlp_workspace_bytes(4, 128, 64, 2, 8, 3) == 0


@pytest.mark.parametrize("sizes", [(2816, 704, 8, 128), (4096, 768, 8, 128), (256, 64, 2, 4)])
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_mlp_workspace_of_more_tokens_serves_fewer(sizes, dt):
    H, I, S, E = sizes
    sizes = [M.lib().moe_mlp_workspace_bytes(m, H, I, S, E, dt) for m in range(1, 3000, 7)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_binding_checks():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        M.gate_topk(x, 2)
    with pytest.raises(ValueError, match="\\[m, num_experts\\]"):
        M.gate_topk(x[0], 2)
    with pytest.raises(ValueError, match="CUDA"):
        M.combine(torch.zeros(2, 3, 8), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="n_expert_used"):
        M.combine(x, x)
    w = M.ExpertWeights(x, x, x, fmt=0, bits=4, group_size=32)
    kw = dict(hidden=128, inter=64, num_experts=4, n_expert_used=2, max_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        M.MoeMlp(w, w, **kw)
    for bad in (dict(hidden=0), dict(max_tokens=0), dict(act="relu"), dict(path="fast"), dict(x_dtype=torch.int8)):
        with pytest.raises(ValueError, match="MoeMlp"):
            M.MoeMlp(w, w, **{**kw, **bad})
