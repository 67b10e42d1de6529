"""add_rmsnorm_fp8 against the 64-bit definition.

Tolerances, relative to the exact value: a binary32 sum of H squares in a tree
of at most 32 sequential additions per thread and 10 levels is within 2^-18,
so is its root (half of that) and the products after it (3 roundings): 2^-18 in
all for y and the scales (a largest value's own error, one division). A code is
the nearest of y / scale, so code * scale is within half an E4M3 step of y, 2^-4
of it or (below the smallest normal code, 2^-6) 2^-10 * scale, plus 2^-17 from
the errors of y and the scale. The stored sum is one binary32 addition of two
exact values and one rounding: half a step of its type plus 2^-24."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._fp8 import (DEV, DTYPES, HALF_STEP, call_over_freed_blocks, dev, host, ref, rows)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def inputs(seed, tokens, hidden, dtype, residual):
    rng = np.random.default_rng(seed)
    x = rows(rng, (tokens, hidden), dtype, 2.0)
    r = rows(rng, (tokens, hidden), dtype) if residual else None
    w = torch.from_numpy(rng.uniform(0.5, 1.5, hidden).astype(np.float32)).to(DTYPES[dtype])
    return x, r, w.float().numpy()


def check(x, r, w, dtype, group, got, eps=1e-6):
    out, scales, total = got
    y, want_s, h = ref.add_rmsnorm(x, r, w, eps, group)
    s = scales.cpu().double().numpy()
    assert np.all(np.abs(s - want_s) <= 2.0 ** -18 * want_s)
    g = group or x.shape[1]
    full = np.repeat(s, g, 1)
    value = ref.e4m3_decode(host(out)) * full
    assert np.all(np.abs(value - y) <= (2.0 ** -4 + 2.0 ** -17) * np.abs(y) + 2.0 ** -10 * full)
    if r is not None:
        d = np.abs(total.cpu().double().numpy() - h)
        assert np.all(d <= (HALF_STEP[dtype] + 2.0 ** -23) * np.abs(h) + 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("tokens,hidden,group", [
    (1, 8, 0), (3, 16, 0), (2, 128, 128), (7, 1000, 0), (5, 1152, 128), (33, 4096, 128),
    (8, 4096, 0), (4, 7168, 128), (3, 8200, 0), (2, 16384, 128), (2, 32768, 0), (1, 32640, 128)])
def test_sizes(tokens, hidden, group, residual, dtype):
    x, r, w = inputs(tokens + hidden, tokens, hidden, dtype, residual)
    got = kvq.add_rmsnorm_fp8(dev(x, dtype), dev(w, dtype), 1e-6,
                              residual=dev(r, dtype) if residual else None, group=group)
    check(x, r, w, dtype, group, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("tokens,hidden,group", [
    (401, 8, 0), (400, 128, 128), (333, 1000, 0), (310, 4224, 128), (350, 8192, 0), (309, 8200, 0)])
def test_several_vectors_a_thread(tokens, hidden, group, residual, dtype):
    x, r, w = inputs(tokens + hidden, tokens, hidden, dtype, residual)
    got = kvq.add_rmsnorm_fp8(dev(x, dtype), dev(w, dtype), 1e-6,
                              residual=dev(r, dtype) if residual else None, group=group)
    check(x, r, w, dtype, group, got)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("tokens,hidden,group", [(5, 4096, 0), (400, 1024, 0), (400, 1024, 128)])
def test_codes_round_the_exact_quotient(tokens, hidden, group, residual):
    """Above the floor y / scale is 448 u / max |u| with u = h w, formed with
    four roundings of 2^-24 each (u, the maximum, the factor, the product), six
    with a residual (h, in u and in the maximum): where a code is not the exact
    quotient's, the quotient lies that close to the border between two."""
    x, r, w = inputs(3, tokens, hidden, "fp16", residual)
    got = kvq.add_rmsnorm_fp8(dev(x, "fp16"), dev(w, "fp16"), 1e-6,
                              residual=dev(r, "fp16") if residual else None, group=group)
    g = group or hidden
    u = ((x.astype(np.float64) + (r if residual else 0)) * w).reshape(tokens, -1, g)
    u = (448 * u / np.abs(u).max(-1, keepdims=True)).reshape(tokens, hidden)
    off = (6 if residual else 4) * 2.0 ** -24 * (1 + 2.0 ** -20)
    have = ref.e4m3_decode(host(got[0]))
    low, high = (ref.e4m3_decode(ref.e4m3_encode(u * (1 + s * off))) for s in (-1, 1))
    assert np.all((have == low) | (have == high))


def test_many_tokens():
    x, r, w = inputs(1, 3001, 512, "bf16", True)
    got = kvq.add_rmsnorm_fp8(dev(x, "bf16"), dev(w, "bf16"), 1e-6, residual=dev(r, "bf16"))
    check(x, r, w, "bf16", 0, got)


def test_zero_rows_and_small_values():
    """A zero row, and one whose squares vanish, keep the floor's scale and
    codes of zero; a lone value takes the largest code."""
    x = np.zeros((3, 256), np.float32)
    x[1] = 2.0 ** -100
    x[2, 0] = 1.0
    w = np.ones(256, np.float32)
    out, scales, _ = kvq.add_rmsnorm_fp8(dev(x, "bf16"), dev(w, "bf16"), 1e-6, group=128)
    s, c = scales.cpu().numpy(), host(out)
    assert np.all(c[:2] == 0) and np.all(s[:2] == np.float32(1e-4) / np.float32(448))
    assert np.all(c[2, 1:] == 0) and c[2, 0] == 0x7E


def test_strides_in_place_and_given_outputs():
    x, r, w = inputs(5, 9, 640, "bf16", True)
    wide = torch.zeros((9, 704), dtype=torch.bfloat16, device=DEV)
    wide[:, :640] = dev(x, "bf16")
    res = torch.full((9, 656), 3.0, dtype=torch.bfloat16, device=DEV)
    res[:, :640] = dev(r, "bf16")
    out = torch.full((9, 648), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((9, 7), -1.0, device=DEV)
    got = kvq.add_rmsnorm_fp8(wide[:, :640], dev(w, "bf16"), 1e-6, residual=res[:, :640], group=128,
                              out=out[:, :640], scales=scales[:, :5], residual_out=res[:, :640])
    check(x, r, w, "bf16", 128, got)
    assert torch.all(res[:, 640:] == 3.0) and torch.all(out[:, 640:] == 0x55)
    assert torch.all(scales[:, 5:] == -1.0)
    # the sum over x itself
    xd = dev(x, "bf16")
    got = kvq.add_rmsnorm_fp8(xd, dev(w, "bf16"), 1e-6, residual=dev(r, "bf16"), residual_out=xd)
    check(x, r, w, "bf16", 0, got)


def test_nan_and_infinity_stay_in_their_row():
    x, _, w = inputs(6, 4, 256, "bf16", False)
    clean = kvq.add_rmsnorm_fp8(dev(x, "bf16"), dev(w, "bf16"), 1e-6)
    x[1, 7], x[2, 9] = np.nan, np.inf
    got = kvq.add_rmsnorm_fp8(dev(x, "bf16"), dev(w, "bf16"), 1e-6)
    for i in (0, 3):
        assert torch.equal(got[0][i].view(torch.uint8), clean[0][i].view(torch.uint8))
        assert torch.equal(got[1][i], clean[1][i])
    assert np.all((host(got[0])[1] & 0x7F) == 0x7F)  # NaN rows are NaN codes


def test_no_tokens_another_stream_and_a_captured_graph():
    got = kvq.add_rmsnorm_fp8(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                              torch.ones(64, dtype=torch.bfloat16, device=DEV), 1e-6)
    assert got[0].shape == (0, 64)
    x, r, w = inputs(7, 6, 512, "bf16", True)
    xd, rd, wd = dev(x, "bf16"), dev(r, "bf16"), dev(w, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(x, r, w, "bf16", 0, kvq.add_rmsnorm_fp8(xd, wd, 1e-6, residual=rd, stream=s))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kvq.add_rmsnorm_fp8(xd, wd, 1e-6, residual=rd)
    g.replay()
    torch.cuda.synchronize()
    check(x, r, w, "bf16", 0, got)


def test_outputs_made_for_another_stream():
    """They take no block that work on the current stream still writes."""
    x, r, w = inputs(8, 6, 512, "bf16", True)
    xd, rd, wd = dev(x, "bf16"), dev(r, "bf16"), dev(w, "bf16")
    want = kvq.add_rmsnorm_fp8(xd, wd, 1e-6, residual=rd)
    got = call_over_freed_blocks(
        lambda s: kvq.add_rmsnorm_fp8(xd, wd, 1e-6, residual=rd, stream=s), want)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
