"""route_experts, sort_by_expert, combine_experts against their 64-bit definitions, and the whole
layer of experts as a decoder layer runs it.

Choices and places are equal to the oracle's. A weight is a score in binary32: the exponential of a
rounded difference (arguments up to 88: 88 * 2^-24, and 2^-22), a sum of up to 1024 in 37 roundings,
quotients and products, below 2^-16 in all. A combined value is a sum of at most 33 terms in
binary32, 33 * 2^-24 of their magnitudes, and half a step of its type."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._experts import (DEV, DTYPES, HALF_STEP, SUMS, call_over_freed_blocks, check_gated, codes, dev,
                            e4m3_decode, f32, host, i64, ref, u8, weights)

pytestmark = pytest.mark.gpu

LOGITS = dict(DTYPES, fp32=torch.float32)


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    # the fill that call_over_freed_blocks queues: loading its kernel waits for the device
    torch.empty(1, dtype=torch.uint8, device=DEV).fill_(0x55)


def check_route(logits, top_k, dtype="fp32", bias=None, score="softmax", groups=1, top_groups=1, renormalize=True,
                scale=1.0):
    x = torch.from_numpy(logits.astype(np.float32)).to(LOGITS[dtype])
    got, w = kvq.route_experts(x.to(DEV), top_k, score=score, bias=None if bias is None else f32(bias), groups=groups,
                               top_groups=top_groups, renormalize=renormalize, scale=scale)
    want, weight = ref.route(x.float().numpy(), top_k, score, bias, groups, top_groups, renormalize, scale)
    assert np.array_equal(got.cpu().numpy(), want)
    assert np.all(np.abs(w.cpu().numpy() - weight) <= 2.0 ** -16 * np.abs(weight) + 2.0 ** -126)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k,groups,top_groups", [
    (1, 1, 1, 1, 1), (3, 8, 8, 1, 1), (9, 31, 4, 1, 1), (17, 33, 32, 1, 1), (40, 64, 6, 1, 1), (33, 64, 5, 8, 3),
    (7, 60, 4, 4, 2), (12, 160, 6, 8, 3), (65, 256, 8, 8, 4), (5, 384, 10, 1, 1), (6, 100, 7, 5, 2), (9, 1024, 16, 32, 4),
    (4, 1024, 32, 1, 1), (8, 1000, 9, 4, 1), (3, 64, 2, 32, 32), (6, 1008, 5, 21, 3)])
def test_route(tokens, experts, top_k, groups, top_groups, score, dtype):
    rng = np.random.default_rng(tokens * experts)
    x = rng.standard_normal((tokens, experts)) * 2
    for bias in (None, (rng.standard_normal(experts) * 0.1).astype(np.float32)):
        check_route(x, top_k, dtype, bias, score, groups, top_groups, renormalize=bias is None, scale=2.5)
        check_route(x, top_k, dtype, bias, score, groups, top_groups, renormalize=bias is not None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2), (6, 2)])
def test_ties_go_to_the_lower_index(score, groups, top_groups):
    rng = np.random.default_rng(1)
    x = rng.integers(-1, 2, (50, 96)).astype(np.float64)
    x[:5] = 0.5
    x[5] = np.where(np.arange(96) % 2, 0.0, -0.0)
    same = np.full(96, 0.25, np.float32)
    for bias in (None, same, same * rng.integers(0, 2, 96).astype(np.float32)):
        check_route(x, 7, "fp32", bias, score, groups, top_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3), (3, 1)])
def test_keys_that_binary32_cannot_tell_apart(score, groups, top_groups):
    """Scores and biases whose sums lie within a few 2^-27 of each other: binary32 gives many of
    them one value, in another order than their own."""
    rng = np.random.default_rng(2)
    experts = 96
    x = (rng.standard_normal((200, experts)) * 1e-3).astype(np.float32)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-x.astype(np.float64))) if score == "sigmoid" else \
            np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum(1, keepdims=True)
    bias = (0.7 - s[0]).astype(np.float32)  # in the first row, every key is next to 0.7
    x[1:] = x[0] + (rng.standard_normal((199, experts)) * 1e-7).astype(np.float32)
    check_route(x, 9, "fp32", bias, score, groups, top_groups)


def test_large_biases():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((60, 64))
    for size in (1e3, 1e6, 1e30):
        check_route(x, 6, "fp32", (rng.integers(-2, 3, 64) * size).astype(np.float32), "sigmoid")
        check_route(x, 6, "fp32", (rng.integers(-2, 3, 64) * size).astype(np.float32), "softmax", 8, 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups", [(40, 1, 1), (256, 8, 4), (60, 4, 2)])
def test_biases_that_are_not_finite(score, experts, groups, top_groups):
    """-inf: behind all others, chosen where too few others are; NaN, +inf: experts that exist."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((70, experts)).astype(np.float32)
    for out in (0.1, 0.9, 1.0):
        bias = np.where(rng.random(experts) < out, -np.inf, rng.standard_normal(experts) * 0.1).astype(np.float32)
        check_route(x, 7, "fp32", bias, score, groups, top_groups)
    for value in (np.nan, np.inf):
        for share in (0.1, 1.0):
            bias = np.where(rng.random(experts) < share, value, 0.0).astype(np.float32)
            got, w = kvq.route_experts(f32(x), 7, score=score, bias=f32(bias), groups=groups, top_groups=top_groups)
            assert torch.all((got >= 0) & (got < experts)) and torch.all(torch.isfinite(w))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_masked_and_special_logits(score, bias, groups, top_groups):
    """Rows with few or no finite logits, infinities, NaN, the type's lowest value."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((12, 40)).astype(np.float32)
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, ::2] = np.nan
    x[3] = np.nan
    x[4, 7] = x[4, 3] = np.inf
    x[5] = np.finfo(np.float32).min
    x[6, 5] = np.finfo(np.float32).max
    x[7] *= 1e30
    x[8] = 200 * np.sign(x[8])
    x[9, :39] = -np.inf
    b = (rng.standard_normal(40) * 0.1).astype(np.float32) if bias else None
    check_route(x, 6, "fp32", b, score, groups, top_groups)
    check_route(x, 6, "fp32", b, score, groups, top_groups, renormalize=False)


def test_many_tokens_and_strided_logits():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3001, 64)).astype(np.float32)
    wide = torch.full((3001, 70), float("nan"), device=DEV)
    wide[:, 3:67] = f32(x)
    got, w = kvq.route_experts(wide[:, 3:67], 6)
    want, weight = ref.route(x, 6, "softmax", None, 1, 1, True, 1.0)
    assert np.array_equal(got.cpu().numpy(), want)
    row = f32(x[:1]).expand(5, 64)  # one row for all tokens
    got, _ = kvq.route_experts(row, 6)
    assert np.array_equal(got.cpu().numpy(), np.repeat(want[:1], 5, 0))
    assert kvq.route_experts(f32(x[:0]), 6)[0].shape == (0, 6)


def test_rows_beyond_32_bits():
    """Logits, and rows to combine, further apart than 32 bits reach."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((40, 64)).astype(np.float32)
    at = torch.empty(40 << 25, device=DEV).as_strided((40, 64), (1 << 25, 1)).copy_(f32(x))
    want, weight = ref.route(x, 6, "softmax", None, 1, 1, True, 1.0)
    assert np.array_equal(kvq.route_experts(at, 6)[0].cpu().numpy(), want)
    y = at.bfloat16().double().cpu().numpy()
    rows = torch.empty(40 << 26, dtype=torch.bfloat16, device=DEV).as_strided((40, 64), (1 << 26, 1)).copy_(at)
    places = rng.integers(0, 40, (9, 3))
    out = torch.empty(9 << 28, dtype=torch.bfloat16, device=DEV).as_strided((9, 64), (1 << 28, 1))
    got = kvq.combine_experts(rows, i64(places), f32(weight[:9, :3]), out=out)
    sums, mass = ref.combine(y, places, weight[:9, :3].astype(np.float32), None)
    assert np.all(np.abs(got.double().cpu().numpy() - sums) <= 2.0 ** -8 * np.abs(sums) + 33 * 2.0 ** -24 * mass)


# ------------------------------------------------------------------- sort ---

@pytest.mark.parametrize("tokens,top_k,experts", [
    (1, 1, 1), (5, 3, 4), (24, 6, 64), (33, 32, 1024), (100, 41, 7), (512, 8, 160), (513, 8, 16), (4097, 1, 3),
    (1500, 8, 1024), (20000, 2, 33)])
@pytest.mark.parametrize("kind", ["any", "outside", "one"])
def test_sort(tokens, top_k, experts, kind):
    rng = np.random.default_rng(tokens + experts)
    chosen = rng.integers(0, experts, (tokens, top_k))
    if kind == "outside":
        chosen = rng.integers(-2, experts + 2, (tokens, top_k))
        chosen.reshape(-1)[::7] = 1 << 40
    if kind == "one":
        chosen[:] = experts - 1
    got = kvq.sort_by_expert(i64(chosen), experts)
    for g, w in zip(got, ref.sort_by_expert(chosen, experts)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_of_nothing():
    offsets, rows, places = kvq.sort_by_expert(i64(np.zeros((0, 4))), 5)
    assert torch.all(offsets == 0) and rows.shape == (0,) and places.shape == (0, 4)


# ---------------------------------------------------------------- combine ---

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,top_k,n,base", [(1, 1, 8, False), (7, 6, 264, True), (24, 8, 4096, False),
                                                 (33, 9, 2056, True), (5, 32, 7168, True)])
def test_combine(tokens, top_k, n, base, dtype):
    rng = np.random.default_rng(n)
    rows = tokens * top_k + 3
    places = rng.permutation(rows)[:tokens * top_k].reshape(tokens, top_k)
    places[0, 0] = places[-1, -1]  # the same row twice
    places[tokens // 2, ::2] = rng.choice([-1, rows, 1 << 40, -(1 << 50)])
    y = dev(rng.standard_normal((rows, n)), dtype)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    b = dev(rng.standard_normal((tokens, n)), dtype) if base else None
    got = kvq.combine_experts(y, i64(places), f32(w), base=b)
    want, mass = ref.combine(y.double().cpu().numpy(), places, w, b.double().cpu().numpy() if base else None)
    d = np.abs(got.double().cpu().numpy() - want)
    assert np.all(d <= HALF_STEP[dtype] * np.abs(want) + 1.01 * 33 * 2.0 ** -24 * mass + 2.0 ** -25)
    if base:  # in place
        kvq.combine_experts(y, i64(places), f32(w), base=b, out=b)
        assert torch.equal(b, got)


def test_combine_from_and_into_host_memory():
    rng = np.random.default_rng(3)
    y, b = (torch.from_numpy(rng.standard_normal((9, 512)).astype(np.float32)).half().pin_memory() for _ in range(2))
    places, w = i64(rng.integers(0, 9, (9, 4))), f32(rng.random((9, 4)))
    want = kvq.combine_experts(y.to(DEV), places, w, base=b.to(DEV))
    out = torch.empty((9, 512), dtype=torch.float16).pin_memory()
    kvq.combine_experts(y, places, w, base=b, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())


def test_combine_leaves_rows_outside_alone():
    """A place outside adds nothing, whatever its weight; gaps between rows stay."""
    y = torch.full((2, 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = torch.full((3, 24), 9.0, dtype=torch.bfloat16, device=DEV)
    w = f32([[float("nan"), float("inf")]] * 3)
    kvq.combine_experts(y, i64([[-1, 2]] * 3), w, out=out[:, :16])
    assert torch.all(out[:, :16] == 0) and torch.all(out[:, 16:] == 9)
    kvq.combine_experts(y[:0], i64([[0, 1]] * 3), w, out=out[:, :16])
    assert torch.all(out[:, :16] == 0)
    wide = torch.zeros((4, 40), dtype=torch.float16, device=DEV)
    wide[:, 8:24] = 3
    got = kvq.combine_experts(wide[:, 8:24], i64([[1, 3]]), f32([[0.5, 2.0]]))
    assert torch.all(got == 7.5)


# -------------------------------------------------------------- the layer ---

def layer(seed, tokens, hidden, inner, experts):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    logits = f32(rng.standard_normal((tokens, experts)) * 2)
    gate_up, gs = weights(rng, (experts, 2 * inner, hidden))
    down, ds = weights(rng, (experts, hidden, inner))
    return x, logits, gate_up, gs * 8, down, ds


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k,groups", [
    (1, 256, 128, 8, 2, 1), (24, 512, 256, 32, 6, 4), (300, 256, 128, 4, 2, 1), (700, 384, 256, 16, 4, 2)])
def test_a_layer_of_experts_behind_its_norm(tokens, hidden, inner, experts, top_k, groups):
    """Norm, routing, both products and the sum; each step against the oracle on what it was given."""
    x, logits, gate_up, gs, down, ds = layer(tokens, tokens, hidden, inner, experts)
    weight = torch.ones(hidden, dtype=torch.bfloat16, device=DEV)
    x8, xs, residual = kvq.add_rmsnorm_fp8(x, weight, 1e-6, residual=x, group=128)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (x8, xs, logits, u8(gate_up), f32(gs), u8(down), f32(ds), top_k)
    more = dict(groups=groups, top_groups=max(1, groups // 2), score="sigmoid", base=residual, status=st)
    out = kvq.fp8_expert_layer(*args, **more)
    assert st.item() == 0 and out.dtype == torch.bfloat16
    chosen, w = kvq.route_experts(logits, top_k, score="sigmoid", groups=groups, top_groups=max(1, groups // 2))
    offsets, rows, places = kvq.sort_by_expert(chosen, experts)
    z, zs = kvq.fp8_expert_gated_matmul(x8, xs, args[3], args[4], offsets, rows=rows)
    y = kvq.fp8_expert_matmul(z, zs, args[5], args[6], offsets)
    assert torch.equal(out, kvq.combine_experts(y, places, w, base=residual))
    h = host(x8), xs.cpu().numpy()
    o, r = offsets.cpu().numpy(), rows.cpu().numpy()
    check_gated((z, zs), *ref.by_expert(*h, gate_up, gs, o, r, tokens * top_k))
    want_y, mass = ref.by_expert(host(z), zs.cpu().numpy(), down, ds, o, None, tokens * top_k)
    assert np.all(np.abs(y.double().cpu().numpy() - want_y) <= 2.0 ** -8 * np.abs(want_y) + 1.01 * SUMS * mass + 2.0 ** -25)
    want, mass = ref.combine(y.double().cpu().numpy(), places.cpu().numpy(), w.cpu().numpy(),
                             residual.double().cpu().numpy())
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 33 * 2.0 ** -24 * mass)
    # without a status word, on another stream, and captured
    assert torch.equal(kvq.fp8_expert_layer(*args, **dict(more, status=None)), out)
    got = call_over_freed_blocks(lambda s: kvq.fp8_expert_layer(*args, **dict(more, stream=s)), [out])
    assert torch.equal(got, out)
    graph, again = torch.cuda.CUDAGraph(), torch.empty_like(out)
    with torch.cuda.graph(graph):
        kvq.fp8_expert_layer(*args, **dict(more, out=again))
    for _ in range(2):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)


def test_a_layer_refuses_other_numbers_of_tokens_or_experts():
    x, logits, gate_up, gs, down, ds = layer(9, 40, 256, 128, 8)
    x8, xs, _ = kvq.add_rmsnorm_fp8(x, torch.ones(256, dtype=torch.bfloat16, device=DEV), 1e-6, group=128)
    args = u8(gate_up), f32(gs), u8(down), f32(ds), 3
    wide = torch.cat([logits, logits], 1)
    for bad in (lambda: kvq.fp8_expert_layer(x8, xs, wide, *args),
                lambda: kvq.fp8_expert_layer(x8, xs, logits[:, :7], *args),
                lambda: kvq.fp8_expert_layer(x8, xs, logits[:39], *args),
                lambda: kvq.fp8_expert_layer(x8, xs, logits, *args[:2], args[2][:7], args[3][:7], 3),
                lambda: kvq.fp8_expert_layer(x8, xs, logits, args[0][0], args[1][0], *args[2:])):
        with pytest.raises(ValueError):
            bad()


def test_experts_of_another_rank():
    """Pairs of experts that are not here have no place, no product, no share in the sum."""
    x, logits, gate_up, gs, down, ds = layer(9, 40, 256, 128, 8)
    weight = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    x8, xs, _ = kvq.add_rmsnorm_fp8(x, weight, 1e-6, group=128)
    chosen, w = kvq.route_experts(logits, 3)
    parts = []
    for first in (0, 4):
        offsets, rows, places = kvq.sort_by_expert(chosen - first, 4)
        here = slice(first, first + 4)
        z, zs = kvq.fp8_expert_gated_matmul(x8, xs, u8(gate_up[here]), f32(gs[here]), offsets, rows=rows)
        y = kvq.fp8_expert_matmul(z, zs, u8(down[here]), f32(ds[here]), offsets)
        parts.append(kvq.combine_experts(y, places, w).float())
    whole = kvq.fp8_expert_layer(x8, xs, logits, u8(gate_up), f32(gs), u8(down), f32(ds), 3)
    mass = parts[0].abs() + parts[1].abs()
    assert torch.all((parts[0] + parts[1] - whole.float()).abs() <= 2.0 ** -6 * mass)


def test_values_of_codes():
    """The oracle's decode is that of torch's type."""
    c = torch.arange(256, dtype=torch.uint8)
    v = c.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(e4m3_decode(c.numpy()), v, equal_nan=True)
