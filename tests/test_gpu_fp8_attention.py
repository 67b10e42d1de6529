"""fp8_paged_attention against the 64-bit oracle.

Tolerance for an output element, from the arithmetic: the probabilities enter
the second product as fp16, a relative 2^-11 each, so 2^-11 * mass with mass =
sum_j softmax_j |v_j|. A score is a binary32 sum of exact products; summed in
any order, with the tensor core's truncation of each partial sum counted as a
whole step, it is off by at most dx = 2^-19 * spread, spread the sum of the
products' magnitudes, and exp turns that into a relative 2 dx of p and of the
normaliser; exp2 itself and the binary32 sums of at most 2^17 terms in trees of
short chains stay within 2^-18. A probability below 2^-24 of fp16 is flushed:
at most 2^-30 of the row's largest, times 448 * 2**(the largest value scale),
for each key. Then half a step of the output's type. The log-sum-exp is off by
dx + 2^-18, and half a step of binary32 (2^-24) of itself, doubled for its two
roundings."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._fp8 import (DEV, DTYPES, HALF_STEP, cache_dev, call_over_freed_blocks, dev, make_table,
                        random_cache, ref, rows, starts_of, to_dev)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def case(seed, news, totals, heads=4, kv_heads=2, dim=64, page=16, dtype="bf16", causal=True,
         window=0, spread=1.0, q_size=1.0, sm_scale=None):
    rng = np.random.default_rng(seed)
    news, totals = np.array(news), np.array(totals)
    table, pages = make_table(rng, totals, page)
    t = int(news.sum()) + 3                      # rows behind the last sequence
    ck, sk = random_cache(rng, pages, kv_heads, page, dim, spread)
    cv, sv = random_cache(rng, pages, kv_heads, page, dim, spread)
    # slots behind a sequence and pages that no sequence has hold NaN
    used = np.zeros((pages, page), bool)
    for b, n in enumerate(totals):
        for j in range(-(-int(n) // page)):
            used[table[b, j], :min(page, int(n) - j * page)] = True
    for c in (ck, cv):
        c.transpose(0, 2, 1, 3)[~used] = 0x7F
    q = rows(rng, (t, heads, dim), dtype) * q_size
    q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    return dict(news=news, totals=totals.astype(np.int64), starts=starts_of(news), table=table,
                q=q.float().numpy(), caches=[ck, cv], scales=[sk, sv], dtype=dtype, causal=causal,
                window=window, sm_scale=1 / np.sqrt(dim) if sm_scale is None else sm_scale,
                max_query_len=int(news.max()))


def launch(c, layout="hnd", **more):
    q = dev(c["q"], c["dtype"])
    out = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(out=out, lse=lse, status=status, causal=c["causal"], window=c["window"])
    args.update(more)
    got = kvq.fp8_paged_attention(
        q, *[cache_dev(x, layout) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
        to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
        c["sm_scale"], **args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return got


def compare(c, got):
    want, lse, mass, spread = ref.attention(c["q"], c["caches"], c["scales"], c["table"],
                                            c["totals"], c["starts"], c["sm_scale"], c["causal"],
                                            c["window"])
    out, glse = got[0].cpu().double().numpy(), got[1].cpu().double().numpy()
    n = int(c["starts"][-1])
    assert np.all(out[n:] == 5.0) and np.all(glse[n:] == 5.0)
    want, lse, mass, spread, out, glse = (x[:n] for x in (want, lse, mass, spread, out, glse))
    scale = c["scales"][1].astype(np.int64)
    vmax = 448 * 2.0 ** (scale[scale < 255].max() - 127)
    dx = 2.0 ** -19 * spread[..., None]
    bound = (2.0 ** -11 + 2 * dx + 2.0 ** -18) * mass + HALF_STEP[c["dtype"]] * np.abs(want) + \
        c["totals"].max() * 2.0 ** -30 * vmax + 2.0 ** -24
    assert np.array_equal(np.isnan(out), np.isnan(want))
    fine = ~np.isnan(want)
    bad = np.abs(out - want)[fine] > bound[fine]
    assert not bad.any(), (bad.sum(), np.abs(out - want)[fine][bad].max())
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(glse), empty)
    assert np.all(out[empty] == 0)
    fine = np.isfinite(lse)
    assert np.array_equal(np.isfinite(glse), fine)
    d = np.abs(glse[fine] - lse[fine])
    assert np.all(d <= dx[..., 0][fine] + 2.0 ** -18 + 2.0 ** -23 * np.abs(lse[fine]))


def check(c, layout="hnd", **more):
    compare(c, launch(c, layout, **more))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_single_tokens(dim, page, dtype):
    check(case(1, [1] * 9, [1, 2, 15, 16, 17, 100, 333, 512, 1025], dim=dim, page=page, dtype=dtype))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 2), (3, 1), (5, 1), (8, 1), (9, 1), (16, 1),
                                            (17, 1), (20, 4), (33, 1), (64, 8), (128, 1), (160, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_head_groups(dim, heads, kv_heads):
    check(case(2, [1, 1, 1], [40, 200, 131], heads=heads, kv_heads=kv_heads, dim=dim))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 7, 40, 1000])
@pytest.mark.parametrize("news", [[2, 1, 4, 0, 3], [9, 30, 1, 0, 70]])
def test_short_and_mixed_runs(news, window, causal):
    check(case(3, news, [2, 80, 300, 50, 129], heads=6, kv_heads=2, causal=causal, window=window))
    check(case(4, news, [9, 80, 300, 0, 100], heads=4, kv_heads=4, dim=128, page=64, causal=causal,
               window=window, dtype="fp16"))


@pytest.mark.parametrize("dim,page,heads,kv_heads", [(128, 64, 8, 2), (64, 16, 4, 4), (128, 32, 5, 1),
                                                     (64, 256, 12, 2)])
def test_whole_prompts(dim, page, heads, kv_heads):
    for n in (127, 128, 129, 300, 513):
        check(case(n, [n], [n], dim=dim, page=page, heads=heads, kv_heads=kv_heads))


@pytest.mark.parametrize("window", [0, 100, 128, 257])
def test_chunks_behind_contexts(window):
    check(case(5, [200, 1, 64, 300, 129], [700, 900, 64, 301, 1500], heads=4, kv_heads=2, dim=128,
               page=64, window=window))
    check(case(6, [200, 1, 64, 300], [700, 900, 64, 301], heads=4, kv_heads=2, dim=64, page=16,
               window=window, causal=False, dtype="fp16"))


def test_empty_sequences_and_rows_without_keys():
    check(case(7, [1, 1, 0, 2], [0, 5, 7, 0]))
    # more queries than keys: the first stand before the first key
    check(case(8, [4, 9, 40], [2, 9, 3]))
    check(case(9, [300], [200], dim=128, page=64))
    check(case(9, [300], [200], dim=128, page=64, causal=False))
    check(case(10, [1], [0]))


def test_many_sequences():
    rng = np.random.default_rng(0)
    check(case(11, [1] * 700, rng.integers(0, 90, 700)))
    check(case(12, rng.integers(0, 30, 200), rng.integers(0, 90, 200)))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give what they give
    alone: prompts, single tokens and mixtures side by side."""
    cases = [case(41, [150, 1, 40], [400, 3000, 90], dim=128, page=64),
             case(42, [1] * 9, [3000, 20, 500, 1, 64, 7, 2000, 90, 1000], dim=64, page=16)]
    alone = [launch(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = []
    for c in cases:
        q = dev(c["q"], c["dtype"])
        args.append((q, *[cache_dev(x) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
                     to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]),
                     c["max_query_len"], c["sm_scale"]))
    ws = [torch.empty(64 << 20, dtype=torch.uint8, device=DEV) for _ in cases]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [[torch.empty_like(a[0]) for _ in range(8)] for a in args]
    torch.cuda.synchronize()
    for i in range(8):
        for a, w, s, o in zip(args, ws, streams, outs):
            kvq.fp8_paged_attention(*a, out=o[i], workspace=w, status=status, stream=s)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for c, want, o in zip(cases, alone, outs):
        n = int(c["starts"][-1])
        assert all(torch.equal(x[:n], want[0][:n]) for x in o)


def test_no_new_tokens():
    """Tokens, but in no sequence: nothing is written."""
    c = case(39, [0, 0], [40, 7])
    out, lse = launch(dict(c, max_query_len=0))[:2]
    assert torch.all(out == 5.0) and torch.all(lse == 5.0)


@pytest.mark.parametrize("news", [[1, 1, 2], [90, 1, 33]])
def test_pinned_host_memory(news):
    """All arguments in page-locked host memory give the same bits."""
    c = case(40, news, [290, 200, 400], dim=128, page=32)
    n = int(c["starts"][-1])
    want = launch(c)

    def pin(a):
        return torch.from_numpy(np.ascontiguousarray(a)).pin_memory()

    q = torch.from_numpy(c["q"]).to(DTYPES[c["dtype"]]).pin_memory()
    got = kvq.fp8_paged_attention(q, *[pin(x) for x in c["caches"]], *[pin(x) for x in c["scales"]],
                                  pin(c["table"]), pin(c["totals"]), pin(c["starts"]),
                                  c["max_query_len"], c["sm_scale"])
    torch.cuda.synchronize()
    assert not got[0].is_cuda and torch.equal(got[0][:n], want[0][:n].cpu())


def test_many_sequences_of_several_tiles():
    """More sequences than are put in order by length; and few, of equal
    lengths and without rows among them."""
    rng = np.random.default_rng(1)
    news = rng.integers(0, 5, 300)
    check(case(34, news, news + rng.integers(0, 60, 300), heads=32, kv_heads=2))
    check(case(35, [40, 0, 40, 90, 40, 1], [150, 300, 150, 90, 150, 150], heads=8, kv_heads=1,
               dim=128, page=64))


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("news", [[2, 1, 2, 2], [2, 0, 1, 5]])
def test_two_passes_of_rows(news, dim, page):
    """Up to 32 rows to a key head, whose second 16 are a unit of their own;
    in the second batch a longer run takes the tile kernel."""
    check(case(37, news, [700, 3, 90, 1500], heads=24, kv_heads=2, dim=dim, page=page))
    check(case(38, news, [700, 3, 90, 1500], heads=32, kv_heads=2, dim=dim, page=page, window=70))


@pytest.mark.parametrize("dim,kv_heads", [(128, 2), (64, 1)])
def test_parts_of_a_long_context(dim, kv_heads):
    """Few rows behind long contexts: each row tile's keys are split over
    blocks whose results are joined; one sequence is too short to be split."""
    check(case(36, [60, 100, 20], [5003, 3000, 70], heads=4 * kv_heads, kv_heads=kv_heads, dim=dim,
               page=32))


def test_one_long_sequence():
    check(case(13, [1], [20011], heads=8, kv_heads=1, dim=128, page=64))
    check(case(14, [3], [9000], heads=16, kv_heads=4, dim=64, page=16))
    check(case(15, [3], [9000], heads=16, kv_heads=4, dim=64, page=16, window=4096))
    check(case(15, [150], [9000], heads=2, kv_heads=1, dim=128, page=128))


def test_layouts_and_strides():
    for layout in ("nhd", "gaps"):
        check(case(16, [1, 1, 50, 2], [40, 200, 131, 9], dim=128, page=32), layout)
    c = case(17, [1, 2, 50], [40, 200, 131], heads=6, kv_heads=2, dim=64)
    t = c["q"].shape[0]
    wide = torch.zeros((t, 6, 80), dtype=torch.bfloat16, device=DEV)
    wide[:, :, :64] = dev(c["q"], "bf16")
    outw = torch.full((t, 7, 72), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((t, 6), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = kvq.fp8_paged_attention(
        wide[:, :, :64], *[cache_dev(x) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
        to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]), 50, c["sm_scale"],
        out=outw[:, :6, :64], lse=lse, status=status)
    compare(c, got)
    assert torch.all(outw[:, 6] == 5.0) and torch.all(outw[:, :, 64:] == 5.0)


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [150, 40]])
def test_pages_outside_the_cache_are_dropped(news):
    c = case(18, news, [300, 200], dim=128, page=32)
    c["table"][0, 1], c["table"][0, 3], c["table"][1, 0] = -1, 1 << 40, c["caches"][0].shape[0]
    check(c)
    c["table"][1, :] = -7
    check(c)
    # lengths past the table and below zero
    c = case(19, news, [300, 200], dim=64, page=16)
    c["table"] = c["table"][:, :9].copy()
    c["totals"] = np.array([1 << 50, -3], np.int64)
    check(c)


@pytest.mark.parametrize("news,heads", [([1, 1], 4), ([3, 2], 4), ([150, 40], 4), ([2, 1], 40)])
def test_nan_reaches_only_the_rows_that_see_it(news, heads):
    """NaN codes in keys and values of the newest tokens, which later rows see
    and earlier rows do not; NaN far back, outside some rows' window."""
    c = case(20, news, [290, 200], heads=heads, dim=128, page=32)
    for which in (0, 1):
        for b in (0, 1):
            p = int(c["totals"][b]) - 1
            c["caches"][which][c["table"][b, p // 32], 0, p % 32, 3 + which] = 0xFF
            p = int(c["totals"][b]) - news[b] // 2 - 1
            c["caches"][which][c["table"][b, p // 32], 1, p % 32, 77] = 0x7F
    check(c)
    c["window"] = 64
    for b in (0, 1):
        p = int(c["totals"][b]) - 65
        c["caches"][1][c["table"][b, p // 32], 0, p % 32, :] = 0x7F
    check(c)


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [150, 40]])
def test_scales_far_apart(news):
    """Pages whose scales differ by many powers of two, the largest and the
    smallest byte and the NaN byte among them."""
    c = case(21, news, [290, 200], dim=128, page=16, spread=8.0)
    check(c)
    c = case(22, news, [290, 200], dim=64, page=32)
    c["scales"][1][c["table"][0, 0], 0] = 60
    c["scales"][0][c["table"][0, 1], 0] = 1
    c["scales"][1][c["table"][1, 2], 1] = 0
    c["scales"][0][c["table"][1, 1], 1] = 0
    check(c)
    c["scales"][0][c["table"][0, 3], 1] = 255
    c["scales"][1][c["table"][1, 0], 0] = 255
    check(c)
    # a NaN page that the window hides from some rows
    c["window"] = 150
    check(c)


@pytest.mark.parametrize("news", [[1, 1], [150, 40]])
def test_large_and_small_queries(news):
    check(case(23, news, [290, 200], q_size=2.0 ** 12, sm_scale=2.0 ** -12))
    check(case(24, news, [290, 200], q_size=2.0 ** -60, sm_scale=2.0 ** 57))
    check(case(25, news, [290, 200], sm_scale=0.0))
    check(case(26, news, [290, 200], q_size=30.0))    # sharp: one key takes nearly all
    c = case(27, news, [290, 200])
    c["q"][0] = 0
    c["q"][1, 1, 5] = np.nan
    check(c)


def test_growing_scores_and_values():
    """Scores and value scales that grow along the sequence, so that every
    tile raises the references."""
    for news in ([1], [140]):
        c = case(28, news, [1000], dim=128, page=16, kv_heads=1)
        for j in range(-(-1000 // 16)):
            g = c["table"][0, j]
            c["scales"][0][g] = 118 + j // 8
            c["scales"][1][g] = 100 + j // 2
        check(c)


@pytest.mark.parametrize("news", [[1, 1, 1], [90, 1, 33]])
def test_streams_graphs_workspaces_and_repeats(news):
    c = case(29, news, [290, 200, 4000], dim=128, page=32)
    want = launch(c)
    compare(c, want)
    again = launch(c)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = launch(c, stream=s)
    assert torch.equal(want[0], other[0])
    # no outputs given, no log-sum-exp
    got, none = launch(c, out=None, lse=None)
    n = int(c["starts"][-1])
    assert none is None and torch.equal(got[:n], want[0][:n])
    # a captured graph follows its inputs; a garbage workspace, the smallest one
    q = dev(c["q"], c["dtype"])
    args = [*[cache_dev(x) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
            to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
            c["sm_scale"]]
    size = kvq.fp8_paged_attention_workspace_size(3, q.shape[0], q.shape[1], 2, 128,
                                                  c["max_query_len"])
    assert size <= 64 << 20
    ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    two = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.fp8_paged_attention(q, *args, out=out, workspace=ws, status=status)
        kvq.fp8_paged_attention(q, *args, out=two, workspace=ws, status=status)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:n], want[0][:n]) and torch.equal(two[:n], want[0][:n])
    q.mul_(0.5)
    c["q"] = c["q"] * 0.5
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:n], launch(c)[0][:n])


def test_append_then_attend_as_a_layer_does():
    """Norm, a projection, append and attention over four steps of a ragged
    batch: a prompt, another behind it, then single tokens."""
    rng = np.random.default_rng(30)
    heads, kv_heads, dim, page, hidden = 8, 2, 64, 16, 256
    cache = kvq.fp8_kv_cache(40, kv_heads, page, dim)
    table = np.stack([rng.permutation(20), 20 + rng.permutation(20)]).astype(np.int64)
    a = np.arange(320)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    cos_sin = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    proj = (torch.randn((hidden, (heads + 2 * kv_heads) * dim), device=DEV) / 16).bfloat16()
    weight = torch.ones(hidden, dtype=torch.bfloat16, device=DEV)
    codes = [host_codes(x) for x in cache[:2]]
    scales = [x.view(torch.uint8).cpu().numpy() for x in cache[2:]]
    lens = np.zeros(2, np.int64)
    for step, news in enumerate(([37, 20], [70, 0], [1, 1], [1, 1])):
        t = sum(news)
        x = torch.randn((t, hidden), device=DEV).bfloat16()
        h, s, _ = kvq.add_rmsnorm_fp8(x, weight, 1e-6)
        qkv = ((h.float() * s) @ proj.float()).bfloat16()
        q = qkv[:, :heads * dim].view(t, heads, dim)
        k = qkv[:, heads * dim:(heads + kv_heads) * dim].view(t, kv_heads, dim)
        v = qkv[:, (heads + kv_heads) * dim:].view(t, kv_heads, dim)
        starts = starts_of(news)
        qr = kvq.rope_fp8_kv_append(k, v, *cache, to_dev(table), to_dev(lens), to_dev(starts),
                                    cos_sin=to_dev(cos_sin), q=q)
        want_q, _ = ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), codes, scales, table,
                               lens, starts, cos_sin, dim, True, q=q.float().cpu().numpy())
        lens = lens + np.array(news)
        for have, want in zip(cache[:2], codes):
            assert np.array_equal(host_codes(have), want), step
        assert torch.equal(qr.cpu(), torch.from_numpy(want_q).bfloat16())
        c = dict(q=qr.float().cpu().numpy(), caches=codes, scales=scales, table=table, totals=lens,
                 starts=starts, sm_scale=dim ** -0.5, causal=True, window=0, dtype="bf16",
                 max_query_len=max(news))
        lse = torch.empty((t, heads), device=DEV)
        got = kvq.fp8_paged_attention(qr, *cache, to_dev(table), to_dev(lens), to_dev(starts),
                                      max(news), dim ** -0.5, lse=lse)
        compare(c, got)


def host_codes(t):
    return t.view(torch.uint8).cpu().numpy().copy()


def test_offsets_past_32_bits():
    """A page whose bytes lie past 2**32 of the cache."""
    heads, page, dim = 2, 256, 128
    pages = (1 << 32) // (heads * page * dim) + 2
    c = case(31, [2], [250], heads=4, kv_heads=heads, dim=dim, page=page)
    k, v = (torch.full((pages, heads, page, dim), 0x7F, dtype=torch.uint8, device=DEV)
            for _ in range(2))
    ks, vs = (torch.full((pages, heads), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    g = int(c["table"][0, 0])
    for big, small in zip((k, v, ks, vs), (*c["caches"], *c["scales"])):
        big[-1] = torch.from_numpy(small[g]).to(DEV)
    q = dev(c["q"], "bf16")
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device=DEV)
    got = kvq.fp8_paged_attention(q, k, v, ks, vs, to_dev(np.array([[pages - 1]], np.int64)),
                                  to_dev(c["totals"]), to_dev(c["starts"]), 2, c["sm_scale"],
                                  out=out, lse=lse)
    compare(c, got)


@pytest.mark.parametrize("news", [[1, 1, 2], [90, 1, 33]])
def test_expanded_block_table_and_scales(news):
    """Several sequences over one row of the block table, and one page's scales
    for all pages, give what copies of them give."""
    c = case(43, news, [290, 200, 400], dim=128, page=32)
    c["table"] = np.repeat(c["table"][2:], 3, 0)
    for s in c["scales"]:
        s[:] = s[0]
    want = launch(c)
    compare(c, want)
    q = dev(c["q"], c["dtype"])
    scales = [to_dev(x)[:1].expand(x.shape) for x in c["scales"]]
    table = to_dev(c["table"])[:1].expand(c["table"].shape)
    assert table.stride(0) == 0 and scales[0].stride(0) == 0
    got = kvq.fp8_paged_attention(q, *[cache_dev(x) for x in c["caches"]], *scales, table,
                                  to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
                                  c["sm_scale"])[0]
    n = int(c["starts"][-1])
    assert torch.equal(got[:n], want[0][:n])
    with pytest.raises(kvq.KvqError):  # rows that overlap
        kvq.fp8_paged_attention(q, *[cache_dev(x) for x in c["caches"]], *scales,
                                table.contiguous().as_strided(table.shape, (1, 1)),
                                to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
                                c["sm_scale"])


@pytest.mark.parametrize("handle", [True, False])
def test_a_call_without_status_ends_behind_its_kernels(handle):
    """On the default stream by its handle 0, and on another stream by its own:
    without a status word the call returns when its kernels have run."""
    c = case(44, [90, 1, 33], [290, 200, 400], dim=128, page=32)
    q = dev(c["q"], c["dtype"])
    args = (q, *[cache_dev(x) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
            to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
            c["sm_scale"])
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = torch.full_like(q, 5.0)
    torch.cuda.synchronize()
    for s in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
            done = torch.cuda.Event()
            done.record()
        got = kvq.fp8_paged_attention(*args, out=out, lse=lse, stream=s.cuda_stream if handle else s)
        assert done.query() and s.query()
        compare(c, got)


@pytest.mark.parametrize("news,total", [([1, 1, 1], 4000), ([20, 1, 33], 4000)])
def test_outputs_and_scratch_made_for_another_stream(news, total):
    """They take no block that work on the current stream still writes: neither
    the outputs nor, with rows and tiles in parts, the workspace and status."""
    c = case(45, news, [290, 200, total], dim=128, page=32)
    q = dev(c["q"], c["dtype"])
    args = (q, *[cache_dev(x) for x in c["caches"]], *[to_dev(x) for x in c["scales"]],
            to_dev(c["table"]), to_dev(c["totals"]), to_dev(c["starts"]), c["max_query_len"],
            c["sm_scale"])
    want, _ = kvq.fp8_paged_attention(*args)
    size = kvq.fp8_paged_attention_workspace_size(3, q.shape[0], q.shape[1], 2, 128,
                                                  c["max_query_len"])
    assert size > 0
    got, _ = call_over_freed_blocks(lambda s: kvq.fp8_paged_attention(*args, stream=s), [want],
                                    (size, 4))
    n = int(c["starts"][-1])
    assert torch.equal(got[:n], want[:n])


@pytest.mark.parametrize("news", [[1, 1], [150, 40]])
def test_outputs_with_the_heads_outermost(news):
    c = case(46, news, [290, 200], dim=64, page=32)
    want = launch(c)
    t, heads, dim = c["q"].shape
    out = torch.full((heads, t, dim), 5.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    got = launch(c, out=out)
    assert torch.equal(got[0], want[0])
    with pytest.raises(kvq.KvqError):
        launch(c, out=torch.empty((t, heads, dim), dtype=torch.bfloat16, device=DEV)
               .as_strided((t, heads, dim), (dim, dim, 1)))
