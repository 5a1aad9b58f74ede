"""The routing, expert-layer and combine operators: cases, inputs, their plain forms and their calls.

Three operators of an expert-routed layer, as a serving program calls them:

  gate     router logits -> the experts of each token and their weights
  mlp      tokens, experts and weights -> the gated expert MLP, summed over a token's experts
  combine  rows of all (token, slot) pairs -> their weighted sum, one row a token

With ``own`` false, ``run`` computes them in elementary torch operations; with
``own`` true it calls ``moe_expert_routed_b200``.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
# name: (format code of the library, bits)
FORMATS = {"affine4": (0, 4), "affine6": (0, 6), "affine8": (0, 8), "codebook2": (1, 2), "codebook3": (1, 3),
           "codebook4": (1, 4), "nvfp4": (2, 4), "mxfp4": (3, 4)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the router of one decode step
        dict(name="gate_token", op="gate", m=1, e=128, k=8, score="softmax", bias=False, renorm=True, t="f32"),
        # an odd batch, sigmoid scores with a load-balancing selection bias
        dict(name="gate_bias", op="gate", m=257, e=160, k=6, score="sigmoid", bias=True, renorm=True, t="bf16"),
        # the router of a long prefill
        dict(name="gate_prefill", op="gate", m=8192, e=256, k=8, score="softmax", bias=False, renorm=True, t="f32"),
        # one decode step of the benchmark's decode layer
        dict(name="mlp_token", op="mlp", m=1, e=128, k=8, h=2816, i=704, fmt="affine4", gs=64, t="bf16", act="silu"),
        # the same layer, eight sequences decoded together
        dict(name="mlp_batch", op="mlp", m=8, e=128, k=8, h=2816, i=704, fmt="affine4", gs=64, t="bf16", act="silu"),
        # a few sequences on NVFP4 weights, the prefill workload's layer
        dict(name="mlp_nvfp4", op="mlp", m=5, e=128, k=8, h=4096, i=768, fmt="nvfp4", gs=16, t="bf16", act="silu"),
        # a small layer with odd sizes, in 32 bits
        dict(name="mlp_odd", op="mlp", m=3, e=40, k=3, h=1376, i=352, fmt="affine4", gs=32, t="f32", act="gelu_tanh"),
        # a 256-token block through 3-bit codebook experts
        dict(name="mlp_canvas", op="mlp", m=256, e=128, k=8, h=2816, i=704, fmt="codebook3", gs=32, t="f16", act="silu"),
        # a long prefill
        dict(name="mlp_prefill", op="mlp", m=4096, e=128, k=8, h=4096, i=768, fmt="nvfp4", gs=16, t="bf16", act="silu"),
        # the sum over a single token's experts
        dict(name="combine_token", op="combine", m=1, k=8, n=2816, tz="f32", t="bf16", res=True),
        # an odd batch of narrow rows
        dict(name="combine_odd", op="combine", m=77, k=6, n=1001, tz="f16", t="f16", res=False),
        # the sum over the experts of a prefill, into the residual stream
        dict(name="combine_prefill", op="combine", m=4096, k=8, n=4096, tz="bf16", t="bf16", res=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "mlp", "mlp", "combine"])
    if op == "gate":
        e = _log(rng, 8, 1024)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, m=_log(rng, 1, 8192), e=e, k=rng.randint(1, min(16, e)), score=score,
                    bias=score == "sigmoid" and rng.random() < 0.5, renorm=rng.random() < 0.7,
                    t=rng.choice(["f32", "bf16", "f16"]))
    if op == "combine":
        k = rng.randint(1, 16)
        n = _log(rng, 33, 8192)
        tz = rng.choice(["f32", "bf16", "f16"])
        return dict(op=op, m=_log(rng, 1, max(1, min(8192, (1 << 27) // (k * n)))), k=k, n=n, tz=tz,
                    t=rng.choice([tz, "bf16"]), res=rng.random() < 0.5)
    fmt = rng.choice(sorted(FORMATS))
    gs = {"nvfp4": 16, "mxfp4": 32}.get(fmt) or rng.choice([32, 64, 128])
    step = max(32, gs)
    e = _log(rng, 4, 192)
    h = step * rng.randint(max(1, 512 // step), 4096 // step)
    i = step * rng.randint(max(1, 128 // step), 1024 // step)
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    # 32-bit rows are used for few tokens
    m = _log(rng, 1, 12 if t == "f32" else 2048)
    return dict(op=op, m=m, e=e, k=rng.randint(1, min(8, e)), h=h, i=i, fmt=fmt, gs=gs, t=t,
                act=rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf"]))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _row_bytes(fmt, bits, k):
    if fmt == 0 and bits == 6:
        return (k + 3) // 4 * 3
    if fmt in (0, 1):
        per = 32 // bits
        return (k + per - 1) // per * 4
    return k // 2


def _weights(g, c, n, k):
    """One projection of all experts: packed codes, scales and the format's third array."""
    fmt, bits = FORMATS[c["fmt"]]
    e, groups = c["e"], k // c["gs"]
    packed = torch.randint(0, 256, (e, n, _row_bytes(fmt, bits, k)), generator=g, device="cuda", dtype=torch.uint8)
    u = torch.rand((e, n, groups), generator=g, device="cuda")
    if fmt == 0:
        scales = (0.002 + 0.008 * u).to(torch.bfloat16)
        aux = (-(2 ** (bits - 1)) * scales.float() + 0.002 * torch.randn((e, n, groups), generator=g, device="cuda")).to(torch.bfloat16)
        if bits > 4:  # the same range of weights with more codes
            scales, aux = (scales.float() / 2 ** (bits - 4)).to(torch.bfloat16), (aux.float() / 2 ** (bits - 4)).to(torch.bfloat16)
    elif fmt == 1:
        scales = (0.01 + 0.04 * u).to(torch.float16)
        p = (torch.arange(1 << bits, device="cuda", dtype=torch.float64) + 0.5) / (1 << bits)
        aux = torch.special.ndtri(p).to(torch.float16)
    elif fmt == 2:
        scales = (0.2 + 0.35 * u).to(torch.float8_e4m3fn).view(torch.uint8)
        aux = torch.full((e,), 1.0 / 28.0, device="cuda") * (0.5 + torch.rand(e, generator=g, device="cuda"))
    else:
        scales = (117 + 4 * u).to(torch.uint8)
        aux = torch.zeros(1, device="cuda")
    return packed, scales, aux


def prepare(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "gate":
        logits = (1.5 * torch.randn((c["m"], c["e"]), generator=g, device="cuda")).to(DT[c["t"]])
        bias = 0.05 * torch.randn(c["e"], generator=g, device="cuda") if c["bias"] else None
        return dict(case=c, logits=logits, bias=bias,
                    ids=torch.empty((c["m"], c["k"]), dtype=torch.int32, device="cuda"),
                    weights=torch.empty((c["m"], c["k"]), device="cuda"))
    if c["op"] == "combine":
        z = torch.randn((c["m"], c["k"], c["n"]), generator=g, device="cuda").to(DT[c["tz"]])
        w = torch.rand((c["m"], c["k"]), generator=g, device="cuda") + 0.05
        res = torch.randn((c["m"], c["n"]), generator=g, device="cuda").to(DT[c["t"]]) if c["res"] else None
        return dict(case=c, z=z, weights=w / w.sum(1, keepdim=True), residual=res,
                    out=torch.empty((c["m"], c["n"]), dtype=DT[c["t"]], device="cuda"))
    x = torch.randn((c["m"], c["h"]), generator=g, device="cuda").to(DT[c["t"]])
    ids = torch.rand((c["m"], c["e"]), generator=g, device="cuda").topk(c["k"], dim=1).indices.to(torch.int32)
    w = torch.rand((c["m"], c["k"]), generator=g, device="cuda") + 0.05
    return dict(case=c, x=x, ids=ids, weights=w / w.sum(1, keepdim=True),
                gate_up=_weights(g, c, 2 * c["i"], c["h"]), down=_weights(g, c, c["h"], c["i"]),
                out=torch.empty((c["m"], c["h"]), dtype=DT[c["t"]], device="cuda"))


# ------------------------------------------------------------------ plain forms


def _plain_gate(s):
    c = s["case"]
    # the choice is between values that can lie closer than 32 bits tell apart
    l = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        choice = l
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
        choice = p + s["bias"].double() if s["bias"] is not None else l
    # descending, ties to the lowest expert
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _plain_combine(s):
    y = (s["weights"][:, :, None] * s["z"].float()).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[s["case"]["t"]])


def _codes(packed, fmt, bits, k):
    """Packed bytes [..., row_bytes] -> whole codes [..., k]."""
    b = packed
    if fmt == 0 and bits == 6:  # 4 codes in 3 bytes
        b = b.unflatten(-1, (-1, 3)).to(torch.int32)
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        at = 6 * torch.arange(4, device=b.device, dtype=torch.int32)
    elif fmt in (2, 3) or (bits in (2, 4)):  # whole codes in each byte
        word = b
        at = bits * torch.arange(8 // bits, device=b.device, dtype=torch.uint8)
    elif bits == 8:
        return b[..., :k]
    else:  # 10 codes in a 32-bit word
        word = b.view(torch.int32)
        at = 3 * torch.arange(10, device=b.device, dtype=torch.int32)
    return ((word[..., None] >> at) & ((1 << bits) - 1)).flatten(-2)[..., :k]


def _dequantised(proj, experts, c, k):
    """f32 weights [len(experts), n, k] of the given experts."""
    fmt, bits = FORMATS[c["fmt"]]
    packed, scales, aux = proj
    code = _codes(packed[experts], fmt, bits, k)
    groups = k // c["gs"]
    code = code.unflatten(-1, (groups, c["gs"]))
    s = scales[experts]
    if fmt == 0:
        w = code.float().mul_(s.float()[..., None]).add_(aux[experts].float()[..., None])
    elif fmt == 1:
        w = aux.float()[code.int()].mul_(s.float()[..., None])
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
        if fmt == 2:
            s = s.view(torch.float8_e4m3fn).float() * aux[experts][:, None, None]
        else:
            s = torch.exp2(s.float() - 127.0)
        w = table[code.int()].mul_(s[..., None])
    return w.flatten(-2)


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return 0.5 * v * (1.0 + torch.erf(v / math.sqrt(2.0)))


def _plain_mlp(s):
    c = s["case"]
    m, e, k, h, i = c["m"], c["e"], c["k"], c["h"], c["i"]
    pairs = m * k
    # pairs in expert order, in tiles of `rows` pairs of one expert: at most pairs / rows + e tiles
    rows = 1
    while rows < 128 and rows * e < pairs:
        rows *= 2
    tiles = min(pairs, pairs // rows + e)
    flat = s["ids"].long().flatten()
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(e, dtype=torch.long, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    first = torch.cumsum(count, 0) - count
    of = (count + rows - 1) // rows
    tile_first = torch.cumsum(of, 0) - of
    place = torch.arange(pairs, device=flat.device) - first[flat[order]]
    at = (tile_first[flat[order]] + place // rows) * rows + place % rows
    tile = torch.arange(tiles, device=flat.device)
    expert = (torch.searchsorted(tile_first + of, tile, right=True)).clamp_(max=e - 1)
    xs = torch.zeros((tiles * rows, h), device=flat.device)
    xs[at] = s["x"].float()[order // k]
    y = torch.bmm(xs.view(tiles, rows, h), _dequantised(s["gate_up"], expert, c, h).transpose(1, 2))
    hidden = _act(c["act"], y[..., :i]) * y[..., i:]
    z = torch.bmm(hidden, _dequantised(s["down"], expert, c, i).transpose(1, 2)).view(tiles * rows, h)
    back = torch.empty_like(order)
    back[order] = at
    out = (s["weights"][:, :, None] * z[back].view(m, k, h)).sum(1)
    return out.to(DT[c["t"]])


# --------------------------------------------------------------------- the calls


def _own_gate(M, s):
    c = s["case"]
    return M.gate_topk(s["logits"], c["k"], score=c["score"], select_bias=s["bias"], renormalize=c["renorm"],
                       ids=s["ids"], weights=s["weights"])


def _own_combine(M, s):
    return M.combine(s["z"], s["weights"], residual=s["residual"], out=s["out"])


def _own_mlp(M, s):
    # the layer's handle: sizes, formats and workspace bound once, kept with the weights
    if "layer" not in s:
        c = s["case"]
        fmt, bits = FORMATS[c["fmt"]]
        kind = dict(fmt=fmt, bits=bits, group_size=c["gs"])
        s["layer"] = M.MoeMlp(M.ExpertWeights(*s["gate_up"], **kind), M.ExpertWeights(*s["down"], **kind),
                              hidden=c["h"], inter=c["i"], num_experts=c["e"], n_expert_used=c["k"],
                              max_tokens=c["m"], x_dtype=DT[c["t"]], out_dtype=DT[c["t"]], act=c["act"])
    return s["layer"](s["x"], s["ids"], s["weights"], out=s["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        import moe_expert_routed_b200 as M

        return {"gate": _own_gate, "combine": _own_combine, "mlp": _own_mlp}[op](M, state)
    return {"gate": _plain_gate, "combine": _plain_combine, "mlp": _plain_mlp}[op](state)


# ------------------------------------------------------------- work and 64 bits


def work(case):
    c = case
    if c["op"] == "gate":
        return {"bytes": c["m"] * (c["e"] * SIZE[c["t"]] + 8 * c["k"]) + (4 * c["e"] if c["bias"] else 0),
                "flops": 6 * c["m"] * c["e"]}
    if c["op"] == "combine":
        rows = c["m"] * c["n"]
        return {"bytes": rows * (c["k"] * SIZE[c["tz"]] + SIZE[c["t"]] * (2 if c["res"] else 1)) + 4 * c["m"] * c["k"],
                "flops": 2 * rows * c["k"]}
    fmt, bits = FORMATS[c["fmt"]]
    per = {0: 4, 1: 2, 2: 1, 3: 1}[fmt]

    def rows(n, k):
        return n * (_row_bytes(fmt, bits, k) + per * (k // c["gs"]))

    touched = c["e"] * (1.0 - (1.0 - c["k"] / c["e"]) ** c["m"])  # experts that some token of a uniform draw takes
    weights = touched * (rows(2 * c["i"], c["h"]) + rows(c["h"], c["i"]))
    return {"bytes": weights + c["m"] * (2 * c["h"] * SIZE[c["t"]] + 8 * c["k"]),
            "flops": 6 * c["m"] * c["k"] * c["h"] * c["i"]}


def _exact_weight(proj, e, c, n, k):
    """One expert's weights in 64 bits, code by code from the bit string of its rows."""
    fmt, bits = FORMATS[c["fmt"]]
    packed, scales, aux = proj
    raw = packed[e].to(torch.int64)
    j = torch.arange(k, device=raw.device)
    if fmt == 1 and bits == 3:
        bit = (j // 10) * 32 + (j % 10) * 3
    else:
        bit = j * bits
    low = raw[:, bit // 8] >> (bit % 8)
    high = raw[:, (bit // 8 + 1).clamp(max=raw.shape[1] - 1)] << (8 - bit % 8)
    code = (low | high) & ((1 << bits) - 1)
    of = j // c["gs"]
    if fmt == 0:
        return code.double() * scales[e].double()[:, of] + aux[e].double()[:, of]
    if fmt == 1:
        return aux.double()[code] * scales[e].double()[:, of]
    mag = code & 7
    ex, man = mag >> 1, mag & 1
    v = torch.where(ex == 0, 0.5 * man.double(), (1.0 + 0.5 * man.double()) * torch.exp2(ex.double() - 1.0))
    v = torch.where(code >= 8, -v, v)
    if fmt == 2:
        return v * scales[e].view(torch.float8_e4m3fn).double()[:, of] * aux[e].double()
    return v * torch.exp2(scales[e].double() - 127.0)[:, of]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gate":
        l = s["logits"].cpu().double()
        if c["score"] == "softmax":
            p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        else:
            p = torch.special.expit(l)
        choice = p + s["bias"].cpu().double() if s["bias"] is not None else l
        n = choice.numpy()
        import numpy as np

        ids = torch.from_numpy(np.argsort(-n, axis=1, kind="stable")[:, : c["k"]].copy())
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return ids.to(torch.int32), w
    if c["op"] == "combine":
        y = torch.einsum("tk,tkn->tn", s["weights"].double(), s["z"].double())
        return y + s["residual"].double() if s["residual"] is not None else y
    x, ids, w = s["x"].double(), s["ids"].long(), s["weights"].double()
    y = torch.zeros((c["m"], c["h"]), dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        t, slot = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ _exact_weight(s["gate_up"], e, c, 2 * c["i"], c["h"]).T
        a, u = gu[:, : c["i"]], gu[:, c["i"] :]
        if c["act"] == "silu":
            a = a * torch.special.expit(a)
        elif c["act"] == "gelu_tanh":
            a = a * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a**3))
        else:
            a = a * torch.special.ndtr(a)
        y.index_add_(0, t, w[t, slot][:, None] * ((a * u) @ _exact_weight(s["down"], e, c, c["h"], c["i"]).T))
    return y
