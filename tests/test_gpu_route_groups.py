"""route_experts where the two largest keys of a group nearly cancel: the error of their sum in
binary32 is that of the keys, not of the sum. Equal to the definition in binary64 for every token."""
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


def route(x, top_k, score, bias, groups, top_groups):
    """The choice by the definition, all tokens at once."""
    x = x.astype(np.float64)
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-x))
    else:
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    key = s + bias.astype(np.float64)
    value = np.sort(key.reshape(len(x), groups, -1))[..., -2:].sum(2)
    order = np.argsort(-value, 1, kind="stable")[:, :top_groups]
    taken = np.zeros((len(x), groups), bool)
    np.put_along_axis(taken, order, True, 1)
    key[~np.repeat(taken, x.shape[1] // groups, 1)] = -np.inf
    return np.argsort(-key, 1, kind="stable")[:, :top_k]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("experts,groups,top_groups", [(64, 8, 4), (60, 5, 2), (256, 8, 4)])
@pytest.mark.parametrize("size,spread", [(64.0, 0.01), (1e3, 1.0), (1e4, 1.0), (1e5, 1.0), (1e7, 1.0)])
def test_groups_whose_two_largest_cancel(size, spread, experts, groups, top_groups, score):
    rng = np.random.default_rng(int(size) + experts)
    x = (rng.standard_normal((20000, experts)) * spread).astype(np.float32)
    bias = np.full(experts, -size, np.float32)
    bias[::experts // groups] = size  # one expert of each group
    got, _ = kvq.route_experts(f32(x), 6, score=score, bias=f32(bias), groups=groups, top_groups=top_groups)
    want = route(x, 6, score, bias, groups, top_groups)
    wrong = np.nonzero((got.cpu().numpy() != want).any(1))[0]
    assert len(wrong) == 0, f"{len(wrong)} tokens, the first {wrong[:5]}"
    few = ref.route(x[:40], 6, score, bias, groups, top_groups, True, 1.0)[0]
    assert np.array_equal(want[:40], few)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_one_group_of_large_keys_among_small_ones(score):
    """Groups of keys of every size, some of which cancel."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20000, 64)).astype(np.float32)
    bias = (rng.standard_normal(64) * 0.1).astype(np.float32)
    for g, size in enumerate((0.0, 30.0, 1e3, 0.0, 1e5, 1e2, 0.0, 1e4)):
        if size:
            bias[8 * g:8 * g + 8] = -size
            bias[8 * g + g] = size
    got, _ = kvq.route_experts(f32(x), 6, score=score, bias=f32(bias), groups=8, top_groups=4)
    assert np.array_equal(got.cpu().numpy(), route(x, 6, score, bias, 8, 4))
    assert torch.equal(got, kvq.route_experts(f32(x).to(DEV), 6, score=score, bias=f32(bias), groups=8, top_groups=4)[0])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_beyond_binary32(score):
    """Two keys whose sum binary32 does not hold, of groups that differ by less than it tells apart."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((500, 64)).astype(np.float32)
    for sizes in ((3.4e38, -3.4e38), (3.4e38, 3.399e38, -3.4e38, -3.399e38, 0.0), (-3.4e38, -3.399e38, -1.7e38)):
        for _ in range(10):
            bias = rng.choice(np.array(sizes, np.float32), 64)
            got, _ = kvq.route_experts(f32(x), 6, score=score, bias=f32(bias), groups=8, top_groups=4)
            assert np.array_equal(got.cpu().numpy(), route(x, 6, score, bias, 8, 4))
