"""route_experts where the chosen experts' scores lie near or below what binary32 holds: the
weights are those of the definition's scores, not of what is left of them in binary32.

A weight is a score of binary32 or, where it is small, of binary64: below 2^-16 relative in either
case (tests/test_gpu_experts.py), and 2^-126 absolute, what binary32 does not hold."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._experts import DEV, f32, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def check(x, top_k, score, bias=None, groups=1, top_groups=1):
    x = np.asarray(x, np.float32)
    for renormalize, scale in ((True, 1.0), (True, 2.5), (False, 1.0), (False, 1e30)):
        got, w = kvq.route_experts(f32(x), top_k, score=score, bias=None if bias is None else f32(bias), groups=groups,
                                   top_groups=top_groups, renormalize=renormalize, scale=scale)
        want, weight = ref.route(x, top_k, score, bias, groups, top_groups, renormalize, scale)
        assert np.array_equal(got.cpu().numpy(), want)
        assert np.all(np.abs(w.cpu().numpy() - weight) <= 2.0 ** -16 * np.abs(weight) + 2.0 ** -126)


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_sigmoids_far_below_one(biased, groups, top_groups):
    rng = np.random.default_rng(1)
    bias = (rng.standard_normal(16) * 0.1).astype(np.float32) if biased else None
    check(np.full((1, 16), -100.0), 2, "sigmoid", bias, groups, top_groups)
    x = np.stack([m + rng.standard_normal(16) for m in (-20, -60, -69, -75, -87, -88.7, -94.5, -103, -150, -400, -690)])
    check(x, 5, "sigmoid", bias, groups, top_groups)
    x[:, ::3] = -np.inf                       # masked among small ones
    check(x, 8, "sigmoid", bias, groups, top_groups)
    x[:, 1::3] = np.finfo(np.float32).min     # the type's lowest value
    check(x, 8, "sigmoid", bias, groups, top_groups)
    x[:, 2] = 3.0                             # one of ordinary size
    check(x, 8, "sigmoid", bias, groups, top_groups)


@pytest.mark.parametrize("experts", [8, 40, 64])
@pytest.mark.parametrize("below", [60.0, 80.0, 100.0, 200.0, 600.0])
def test_softmax_with_a_bias_for_experts_far_below_the_largest(below, experts):
    """Fewer experts of ordinary scores than are chosen, or none: the bias puts others in front."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, experts))
    x[:, :experts // 2] -= below
    bias = np.zeros(experts, np.float32)
    bias[:experts // 2] = 2.0
    check(x, 4, "softmax", bias)
    check(x, experts // 2 + 1, "softmax", bias) if experts <= 32 else check(x, 30, "softmax", bias)
    check(x, 3, "softmax", bias, 4, 2)


def test_scores_of_zero_stay_zero():
    x = np.full((3, 8), -np.inf)
    x[1] = np.finfo(np.float32).min
    x[2] = -1e4
    for score in ("sigmoid", "softmax"):
        check(x, 3, score)
    got, w = kvq.route_experts(f32(x), 3, score="sigmoid")
    assert torch.all(w == 0) and w.device == DEV
