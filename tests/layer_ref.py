"""The expert layer (router choice, gated MLP, weighted sum) in 64 bits on the host,
with the error bound of each output, for the GPU tests of the layer's operators."""

from __future__ import annotations

import numpy as np
import torch
from scipy.special import expit, ndtr

from tests import numpy_ref as R
from workloads.gen import DT_BF16, DT_F16, DT_F32, make_problem

TORCH_DT = {DT_F32: torch.float32, DT_BF16: torch.bfloat16, DT_F16: torch.float16}
# half a step of each type, relative to the value
HALF_STEP = {DT_F32: 2.0**-24, DT_BF16: 2.0**-8, DT_F16: 2.0**-11}
TINY = {DT_F32: 2.0**-149, DT_BF16: 2.0**-133, DT_F16: 2.0**-24}


def gate(logits: np.ndarray, k: int, score: str, bias=None, renormalize=True, scale=1.0):
    """(ids, weights) of float64 logits [m, E]; NaN and all-masked rows are the tests' own."""
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        if score == "softmax":
            p = np.exp(l - l.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            choice = l
        else:
            p = expit(l)
            choice = p + bias.astype(np.float64) if bias is not None else l
        ids = np.argsort(-choice, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(p, ids, 1)
        if renormalize:
            w = w / w.sum(1, keepdims=True)
    return ids, scale * w


def act(name: str, v: np.ndarray) -> np.ndarray:
    if name == "silu":
        return v * expit(v)
    if name == "gelu_tanh":
        return v * expit(2.0 * np.sqrt(2.0 / np.pi) * (v + 0.044715 * v**3))
    return v * ndtr(v)


def tau(k: int) -> float:
    """Error of a product of k terms relative to sum |w||x|: f32 sums (k 2^-24), and the
    tensor-core path's split of each operand into two bf16 terms. The first term is off
    by at most half a step, 2^-8 of the value; the second, a rounding of that remainder,
    leaves 2^-8 of it: 2^-16 for each operand, and 2^-8 * 2^-8 for the product of the
    two remainders, which is left out."""
    return k * 2.0**-24 + 3 * 2.0**-16


class Layer:
    """A random layer: two Problems (gate_up: x [m, hidden]; down), weights of the sum."""

    def __init__(self, *, m, hidden, inter, top_k, E, fmt, bits, gs, x_dtype, act="silu", seed=1, down=None,
                 bias=False, bad_ids=()):
        down = down or (fmt, bits, gs)
        self.act, self.m, self.hidden, self.inter, self.top_k, self.E = act, m, hidden, inter, top_k, E
        kw = dict(n_expert_used=top_k, num_experts=E, x_dtype=x_dtype, out_dtype=DT_F32, scale_range=(0.01, 0.03))
        self.gu = make_problem("gate_up", fmt=fmt, bits=bits, group_size=gs, m=m, k=hidden, n=2 * inter,
                               seed=seed, scale2=1 / 30.0, mx_sigma=0.1, **kw)
        self.dn = make_problem("down", fmt=down[0], bits=down[1], group_size=down[2], m=1, k=inter, n=hidden,
                               seed=seed + 1, scale2=1 / 30.0, mx_sigma=0.1, **kw)
        ids = self.gu.ids.copy()
        for t, s, v in bad_ids:
            ids[t, s] = v
        self.gu = self.gu.with_ids(ids)
        rng = np.random.default_rng(seed + 2)
        self.w = (rng.random((m, top_k)) + 0.05).astype(np.float32)
        self.res = rng.standard_normal((m, hidden)).astype(np.float32)
        self.bias = None
        if bias:
            self.bias = (rng.standard_normal((E, 2 * inter)).astype(np.float32) * 0.3,
                         rng.standard_normal((E, hidden)).astype(np.float32) * 0.3)

    @property
    def x_dtype(self):
        return self.gu.x_dtype

    def reference(self, out_dtype, residual=None):
        """(out, bound, rms) [m, hidden] in float64: the layer, the largest error of each
        element, and the root of the sum of the squares of every rounding's largest
        error: independent roundings keep the 2-norm of all errors below that of rms."""
        X, ids = R.x_f64(self.gu), self.gu.ids.astype(np.int64)
        m, I, H = self.m, self.inter, self.hidden
        G, D = R.dequant_dense(self.gu), R.dequant_dense(self.dn)
        hs = HALF_STEP[DT_BF16] if self.x_dtype == DT_BF16 else HALF_STEP[DT_F32]  # h's type
        out, bound = np.zeros((m, H)), np.zeros((m, H))
        mag, var = np.zeros((m, H)), np.zeros((m, H))
        # Splits of tau(): the weights' (2^-16) and the dropped product (2^-16) differ from
        # row to row. The split of a 32-bit x does not: every row of gate and up meets
        # the same error of x[k], so its effect is that of the derivative of the whole
        # layer by x[k], taken before the sum over k. (Narrower x is not split.)
        split = 2.0**-15
        by_x = np.zeros((m, H, H if self.x_dtype == DT_F32 else 0))
        for t in range(m):
            for s in range(self.top_k):
                e = ids[t, s]
                if not 0 <= e < self.E:
                    continue
                y, a = G[e] @ X[t], np.abs(G[e]) @ np.abs(X[t])
                if self.bias:
                    y = y + self.bias[0][e]
                    a = a + np.abs(self.bias[0][e])
                g, u, dg, du = y[:I], y[I:], tau(H) * a[:I], tau(H) * a[I:]
                ag = act(self.act, g)
                h = ag * u
                # activation: slope at most 1.2, second derivative at most 0.8; its own f32
                # evaluation 4e-6 relative, 1e-6 |g| where 1 + tanh or 1 + erf cancels
                dh = 1.2 * np.abs(u) * dg + np.abs(ag) * du + 1.2 * dg * du + 0.4 * dg**2 * (np.abs(u) + du)
                dh += 4e-6 * np.abs(h) + 1e-6 * np.abs(g) * np.abs(u)
                dh += hs * (np.abs(h) + dh)
                sy = (split + H * 2.0**-24) * np.sqrt(G[e]**2 @ X[t]**2)
                vh = (1.2 * u * sy[:I])**2 + (ag * sy[I:])**2 + ((hs + 4e-6) * h)**2 + (1e-6 * g * u)**2
                vz = D[e]**2 @ vh + (1.5 * split + I * 2.0**-24)**2 * (D[e]**2 @ h**2)
                if self.x_dtype == DT_F32:
                    slope = (act(self.act, g + 1e-6) - act(self.act, g - 1e-6)) / 2e-6
                    J = D[e] @ ((slope * u)[:, None] * G[e][:I] + ag[:, None] * G[e][I:])
                    by_x[t] += float(self.w[t, s]) * J
                z, az = D[e] @ h, np.abs(D[e]) @ np.abs(h)
                dz = np.abs(D[e]) @ dh + tau(I) * az
                if self.bias:
                    z = z + self.bias[1][e]
                    az = az + np.abs(self.bias[1][e])
                w = float(self.w[t, s])
                out[t] += w * z
                bound[t] += abs(w) * dz
                mag[t] += abs(w) * az
                var[t] += w * w * vz + (self.top_k * 2.0**-24 * w * z)**2
        if residual is not None:
            out = out + residual
            mag = mag + np.abs(residual)
        bound += (self.top_k + 2) * 2.0**-24 * mag
        bound += HALF_STEP[out_dtype] * (np.abs(out) + bound) + TINY[out_dtype]
        if self.x_dtype == DT_F32:
            var += (2.0**-16 * by_x)**2 @ X[:, :, None]**2 @ np.ones(1)
        rms = np.sqrt(var + (HALF_STEP[out_dtype] * out)**2 + TINY[out_dtype]**2)
        return out, bound, rms
