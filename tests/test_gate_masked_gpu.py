"""moe_gate_topk: experts masked by a logit of -inf where a selection bias is given. They
come after every other expert whatever their bias, and before NaN logits."""

import numpy as np
import pytest
import torch
from scipy.special import expit

import moe_expert_routed_b200 as M

pytestmark = pytest.mark.gpu

INF = np.float32(np.inf)
DTYPES = (torch.float32, torch.bfloat16, torch.float16)


def choice(l, b, k):
    """The first k of each row of 64-bit logits: live experts by sigmoid(l) + b descending,
    then the masked, then NaN; ties to the lowest expert."""
    out = []
    for row in l:
        score = expit(row) + b.astype(np.float64)
        last = np.where(np.isnan(row), 2, np.where(row == -INF, 1, 0))
        out.append(np.lexsort((np.arange(len(row)), np.where(last > 0, 0.0, -score), last))[:k])
    return np.array(out)


def run(t, b, k, renorm=True):
    ids, w = M.gate_topk(t.cuda(), k, score="sigmoid", select_bias=torch.from_numpy(b).cuda(), renormalize=renorm)
    return ids.cpu().numpy(), w.cpu().double().numpy()


def test_masked_expert_loses_to_a_live_one():
    ids, w = run(torch.tensor([[-np.inf, -3.0]]), np.array([0, -0.1], dtype=np.float32), 1)
    assert ids.tolist() == [[1]] and w.tolist() == [[1.0]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,E,k", [(5, 8, 3), (9, 33, 8), (70, 160, 6), (33, 256, 8), (4, 400, 32), (3, 1024, 16)])
@pytest.mark.parametrize("shift", [0.5, -0.5, 3.0, -3.0])
def test_choice_with_masked_experts(m, E, k, shift, dtype):
    """Masked experts with biases above and below the live ones', some of them infinite."""
    rng = np.random.default_rng(E + k)
    t = torch.from_numpy(rng.standard_normal((m, E)).astype(np.float32) * 2)
    masked = rng.random((m, E)) < np.linspace(0.0, 1.0, m)[:, None]  # none in the first row, all in the last
    t[torch.from_numpy(masked)] = -float("inf")
    t = t.to(dtype)
    b = rng.standard_normal(E).astype(np.float32) * 0.1
    b[::2] += shift
    b[1], b[E // 2] = INF, -INF
    l = t.double().numpy()
    for renorm in (True, False):
        ids, w = run(t, b, k, renorm)
        assert np.array_equal(ids, choice(l, b, k))
        gone = np.isneginf(np.take_along_axis(l, ids.astype(np.int64), 1))
        assert (w[gone] == 0).all() and (w[~gone] > 0).all()


@pytest.mark.parametrize("live", [0, 1, 5, 8, 40])
def test_fewer_live_experts_than_chosen(live):
    """The live ones first, then the masked by their number; NaN logits after those."""
    E, k = 200, 12
    rng = np.random.default_rng(live)
    l = np.full((6, E), -INF, dtype=np.float32)
    for row in l:
        row[rng.permutation(E)[:live]] = rng.standard_normal(live)
    l[3, :3] = np.nan
    l[4, 3:] = np.nan  # at most three that are not NaN
    b = rng.standard_normal(E).astype(np.float32)
    ids, _ = run(torch.from_numpy(l), b, k)
    assert np.array_equal(ids, choice(l.astype(np.float64), b, k))


def test_masked_among_scores_that_tie():
    """More experts at the cut than a warp holds: the choice among all of them."""
    E, k = 300, 20
    l = np.zeros((3, E), dtype=np.float32)
    l[0, ::3] = -INF
    l[1, 5:] = -INF
    l[2, 7:290] = -INF
    b = np.zeros(E, dtype=np.float32)
    b[::2] = 1.0
    ids, _ = run(torch.from_numpy(l), b, k)
    assert np.array_equal(ids, choice(l.astype(np.float64), b, k))
