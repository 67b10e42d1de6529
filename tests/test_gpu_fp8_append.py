"""rope_fp8_kv_append against the oracle, byte for byte: every page of both
caches with its scales, untouched bytes included, and the rotated queries."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._fp8 import (DEV, DTYPES, cache_dev, call_over_freed_blocks, dev, host, make_table,
                        random_cache, ref, rows, starts_of, to_dev)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def table_of(rng, n, rot):
    a = rng.uniform(0, 2 * np.pi, (n, max(rot // 2, 1)))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def case(seed, news, ctxs, heads=4, kv_heads=2, dim=64, page=16, rot=None, interleaved=True,
         dtype="bf16", spread=3.0):
    rng = np.random.default_rng(seed)
    rot = dim if rot is None else rot
    news, ctxs = np.array(news), np.array(ctxs)
    table, pages = make_table(rng, ctxs + news, page)
    t = int(news.sum()) + 2                      # two rows behind the last sequence
    c = dict(news=news, ctxs=ctxs.astype(np.int64), starts=starts_of(news), table=table,
             q=rows(rng, (t, heads, dim), dtype), k=rows(rng, (t, kv_heads, dim), dtype, spread),
             v=rows(rng, (t, kv_heads, dim), dtype, spread), rot=rot, interleaved=interleaved,
             dtype=dtype, cos_sin=table_of(rng, int((ctxs + news).max()) + 1, rot), positions=None)
    ck, sk = random_cache(rng, pages, kv_heads, page, dim, 3.0)
    cv, sv = random_cache(rng, pages, kv_heads, page, dim, 3.0)
    c["caches"], c["scales"] = [ck, cv], [sk, sv]
    return c


def launch(c, layout="hnd", with_q=True, in_place=False, stream=None):
    caches = [cache_dev(x, layout) for x in c["caches"]]
    scales = [to_dev(x) for x in c["scales"]]
    q = dev(c["q"], c["dtype"]) if with_q else None
    q_out = q if in_place else (torch.full_like(q, 7.0) if with_q else None)
    got = kvq.rope_fp8_kv_append(
        dev(c["k"], c["dtype"]), dev(c["v"], c["dtype"]), *caches, *scales, to_dev(c["table"]),
        to_dev(c["ctxs"]), to_dev(c["starts"]),
        cos_sin=to_dev(c["cos_sin"]) if c["rot"] else None, rotary_dim=c["rot"],
        interleaved=c["interleaved"],
        positions=to_dev(c["positions"]) if c["positions"] is not None else None, q=q, q_out=q_out,
        stream=stream)
    return caches, scales, got


def check(c, layout="hnd", with_q=True, in_place=False):
    want_c, want_s = [x.copy() for x in c["caches"]], [x.copy() for x in c["scales"]]
    want_q, written = ref.append(c["k"], c["v"], want_c, want_s, c["table"], c["ctxs"], c["starts"],
                                 c["cos_sin"], c["rot"], c["interleaved"], c["positions"], c["q"])
    caches, scales, got = launch(c, layout, with_q, in_place)
    for which in (0, 1):
        assert np.array_equal(host(scales[which]), want_s[which]), which
        have = host(caches[which])
        # the sign of a NaN says nothing
        nan = (want_c[which] & 0x7F) == 0x7F
        assert np.array_equal((have & 0x7F) == 0x7F, nan)
        assert np.array_equal(have[~nan], want_c[which][~nan]), which
    if with_q:
        # rows that are skipped, and those behind the last sequence, are left
        before = torch.from_numpy(c["q"]) if in_place else torch.full(c["q"].shape, 7.0)
        want = torch.where(torch.from_numpy(written)[:, None, None], torch.from_numpy(want_q), before)
        same = torch.equal(got.cpu().nan_to_num(9.0),
                           want.to(DTYPES[c["dtype"]]).nan_to_num(9.0))
        assert same


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_sequences(page, dtype, interleaved):
    check(case(1, [1, 37, 0, 5, 2 * page + 3, page], [0, 9, 20, page - 1, page - 2, 3 * page],
               page=page, dtype=dtype, interleaved=interleaved))


@pytest.mark.parametrize("dim,rot", [(16, 16), (32, 16), (48, 0), (64, 32), (80, 48), (96, 96),
                                     (128, 128), (128, 64), (256, 128), (240, 240)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_head_dims_and_partial_rotation(dim, rot, interleaved):
    check(case(2, [3, 1, 40], [14, 0, 33], dim=dim, rot=rot, interleaved=interleaved))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (20, 5), (64, 8), (128, 1), (17, 17)])
def test_head_counts(heads, kv_heads):
    check(case(3, [1, 1, 18], [5, 16, 30], heads=heads, kv_heads=kv_heads, dim=128))


def test_single_tokens_of_many_sequences():
    rng = np.random.default_rng(4)
    check(case(5, [1] * 300, rng.integers(0, 200, 300), page=16))


@pytest.mark.parametrize("count", [31, 32, 33, 63, 1024, 1025, 2100])
def test_queries_find_their_sequence(count):
    """Runs of none to three tokens: a token's sequence is searched 32 ends at
    a time."""
    rng = np.random.default_rng(count)
    check(case(22, rng.integers(0, 4, count), rng.integers(0, 40, count), heads=2, kv_heads=1,
               page=16))


def test_one_token_and_nothing_before():
    check(case(6, [1], [0], page=64, dim=128))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dim,rot,page", [(64, 32, 16), (80, 80, 16), (128, 128, 64), (256, 64, 256),
                                          (240, 240, 128)])
def test_many_pages(dim, rot, page, interleaved):
    """More pages than the resident teams take at once, sequences that start
    inside a page and sequences without new tokens among them."""
    rng = np.random.default_rng(20)
    news = rng.integers(0, (16 if page == 16 else 4) * page, 24)
    news[[3, 4, 23]] = [0, 1, page]
    c = case(21, news, rng.integers(0, 2 * page, 24), heads=2, kv_heads=7, dim=dim, rot=rot,
             page=page, interleaved=interleaved)
    check(c, with_q=dim == 64)


def test_token_by_token_grows_the_scale():
    """Values that grow token by token: every append moves the page's earlier
    codes; zeros and values below the floor among them."""
    c = case(7, [1], [0], page=16, spread=0.0)
    caches, scales = [x.copy() for x in c["caches"]], [x.copy() for x in c["scales"]]
    for step in range(20):
        c["ctxs"] = np.array([step], np.int64)
        c["table"] = np.array([[1, 2]], np.int64)
        f = 0.0 if step == 0 else 2.0 ** (step - 10)
        c["k"] = (rows(np.random.default_rng(step), c["k"].shape, "bf16") * f).astype(np.float32)
        c["cos_sin"] = table_of(np.random.default_rng(0), 32, 64)
        c["caches"], c["scales"] = caches, scales
        check(c)
        ref.append(c["k"], c["v"], caches, scales, c["table"], c["ctxs"], c["starts"],
                   c["cos_sin"], c["rot"], c["interleaved"])


def test_layouts_and_strided_inputs():
    for layout in ("nhd", "gaps"):
        check(case(8, [5, 30, 1], [10, 17, 0], dim=128, page=32), layout)
    # q, k, v as slices of one projection
    c = case(9, [5, 30, 1], [10, 17, 0], heads=6, kv_heads=2, dim=64)
    t = c["k"].shape[0]
    qkv = dev(np.concatenate([c["q"], c["k"], c["v"]], 1).reshape(t, -1), "bf16")
    q = qkv[:, :384].view(t, 6, 64)
    k, v = qkv[:, 384:512].view(t, 2, 64), qkv[:, 512:].view(t, 2, 64)
    caches, scales = [cache_dev(x) for x in c["caches"]], [to_dev(x) for x in c["scales"]]
    got = kvq.rope_fp8_kv_append(k, v, *caches, *scales, to_dev(c["table"]), to_dev(c["ctxs"]),
                                 to_dev(c["starts"]), cos_sin=to_dev(c["cos_sin"]), q=q)
    want, _, want_q = launch(c)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, want))
    n = int(c["starts"][-1])
    assert torch.equal(got[:n], want_q[:n])


def test_queries_in_place_and_absent():
    c = case(10, [5, 30, 1], [10, 17, 0])
    check(c, in_place=True)
    check(c, with_q=False)


def test_positions_other_than_the_caches():
    c = case(11, [5, 30, 1], [10, 17, 0])
    rng = np.random.default_rng(0)
    c["positions"] = rng.integers(0, c["cos_sin"].shape[0], c["k"].shape[0]).astype(np.int64)
    check(c)


def test_special_values():
    """Zeros, infinities, NaN, the type's largest and smallest values, and a
    magnitude exactly on a power of two times 448."""
    c = case(12, [20, 4, 3], [0, 30, 5], spread=0.0)
    c["k"][0, 0, 5], c["k"][1, 1, :] = np.nan, np.nan
    c["v"][2, 0, 3], c["v"][3, 1, 4] = np.inf, -np.inf
    c["v"][4:20] = 0.0
    c["k"][21, 0, :8] = np.float32(torch.finfo(torch.bfloat16).max)
    c["v"][22, 0, :] = 448.0 * 2 ** 3
    c["v"][22, 1, :] = 1e-30
    c["v"][24:27, :, :] = 2.0 ** -22
    check(c)


def test_tokens_outside_the_table_or_the_cache_are_skipped():
    c = case(13, [6, 10, 20], [14, 5, 40])
    c["positions"] = np.arange(c["k"].shape[0], dtype=np.int64)
    c["positions"][[2, 8]] = [-1, 1 << 40]
    c["positions"][7:9] = -5
    c["cos_sin"] = table_of(np.random.default_rng(1), 60, 64)
    c["table"][0, 1] = -1
    c["table"][1, 0] = 1 << 50
    check(c)
    # past the last column, with a context behind it or below zero
    c = case(14, [6, 10], [14, 30])
    c["table"] = c["table"][:, :2].copy()
    check(c)
    c["ctxs"] = np.array([1 << 60, -4], np.int64)
    check(c)


def test_no_tokens():
    c = case(15, [0, 0], [14, 30])
    check(c)


def test_offsets_past_32_bits():
    """A page whose bytes lie past 2**32 of the cache."""
    heads, page, dim = 2, 256, 128
    pages = (1 << 32) // (heads * page * dim) + 2
    k_cache = torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=DEV)
    v_cache = torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=DEV)
    scales = [torch.full((pages, heads), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
    rng = np.random.default_rng(1)
    k, v = rows(rng, (3, heads, dim), "bf16"), rows(rng, (3, heads, dim), "bf16")
    table = np.array([[pages - 1, 0]], np.int64)
    kvq.rope_fp8_kv_append(dev(k, "bf16"), dev(v, "bf16"), k_cache, v_cache, *scales,
                           to_dev(table), to_dev(np.array([200], np.int64)),
                           to_dev(np.array([0, 3], np.int64)))
    want = [np.zeros((1, heads, page, dim), np.uint8) for _ in range(2)]
    ws = [np.full((1, heads), 127, np.uint8) for _ in range(2)]
    ref.append(k, v, want, ws, np.array([[0, -1]]), [200], [0, 3], None, 0, True)
    assert np.array_equal(host(k_cache[-1]), want[0][0])
    assert np.array_equal(host(v_cache[-1]), want[1][0])
    assert int(k_cache[:-1].max()) == 0


def test_another_stream_and_a_captured_graph():
    c = case(16, [1, 1, 1], [15, 16, 40])
    want, want_s, want_q = launch(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _, _ = launch(c, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    args = [dev(c["k"], "bf16"), dev(c["v"], "bf16"), *[cache_dev(x) for x in c["caches"]],
            *[to_dev(x) for x in c["scales"]], to_dev(c["table"]), to_dev(c["ctxs"]),
            to_dev(c["starts"])]
    q, cs = dev(c["q"], "bf16"), to_dev(c["cos_sin"])
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.rope_fp8_kv_append(*args, cos_sin=cs, q=q, q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[2].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(args[4], want_s[0])
    n = int(c["starts"][-1])
    assert torch.equal(out[:n], want_q[:n])


def test_expanded_tables_and_scales():
    """Sequences at different places of one row of pages; scales that would be
    written from several places, and a rotation table of one row, are refused."""
    c = case(23, [5, 16, 3], [0, 16, 40])
    c["table"] = np.repeat(np.random.default_rng(23).permutation(c["caches"][0].shape[0])[None, :3], 3, 0)
    want, want_s, want_q = launch(c)
    caches, scales = [cache_dev(x) for x in c["caches"]], [to_dev(x) for x in c["scales"]]
    k, v, q = (dev(c[x], "bf16") for x in "kvq")
    lens, starts, cs = to_dev(c["ctxs"]), to_dev(c["starts"]), to_dev(c["cos_sin"])
    table = to_dev(c["table"])[:1].expand(c["table"].shape)
    assert table.stride(0) == 0
    got_q = kvq.rope_fp8_kv_append(k, v, *caches, *scales, table, lens, starts, cos_sin=cs, q=q)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(caches + scales, want + want_s))
    n = int(c["starts"][-1])
    assert torch.equal(got_q[:n], want_q[:n])
    one = [x[:1].expand(x.shape) for x in scales]
    with pytest.raises(kvq.KvqError):
        kvq.rope_fp8_kv_append(k, v, *caches, *one, table, lens, starts, cos_sin=cs, q=q)
    with pytest.raises(kvq.KvqError):
        kvq.rope_fp8_kv_append(k, v, *caches, *scales, table, lens, starts,
                               cos_sin=cs[:1].expand(cs.shape), q=q)


def test_queries_made_for_another_stream():
    """They take no block that work on the current stream still writes."""
    c = case(24, [5, 30, 1], [10, 17, 0])
    args = [dev(c["k"], "bf16"), dev(c["v"], "bf16"), *[cache_dev(x) for x in c["caches"]],
            *[to_dev(x) for x in c["scales"]], to_dev(c["table"]), to_dev(c["ctxs"]),
            to_dev(c["starts"])]
    q, cs = dev(c["q"], "bf16"), to_dev(c["cos_sin"])
    want = kvq.rope_fp8_kv_append(*args, cos_sin=cs, q=q)
    got = call_over_freed_blocks(
        lambda s: kvq.rope_fp8_kv_append(*args, cos_sin=cs, q=q, stream=s), [want])
    n = int(c["starts"][-1])
    assert torch.equal(got[:n], want[:n])


def test_written_places_lie_apart():
    """Queries with the heads outermost; expanded caches and overlapping queries
    are refused."""
    c = case(25, [5, 30, 1], [10, 17, 0])
    want, want_s, want_q = launch(c)
    caches, scales = [cache_dev(x) for x in c["caches"]], [to_dev(x) for x in c["scales"]]
    more = to_dev(c["table"]), to_dev(c["ctxs"]), to_dev(c["starts"]), to_dev(c["cos_sin"])
    k, v, q = (dev(c[x], "bf16") for x in "kvq")
    t, heads, dim = q.shape
    out = torch.empty((heads, t, dim), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    kvq.rope_fp8_kv_append(k, v, *caches, *scales, *more, q=q.transpose(0, 1).contiguous().transpose(0, 1),
                           q_out=out)
    n = int(c["starts"][-1])
    assert torch.equal(out[:n], want_q[:n])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, want))
    for bad in (dict(caches=[x[:1].expand(x.shape) for x in caches]),
                dict(caches=[x[:, :1].expand(x.shape) for x in caches]),
                dict(q_out=torch.empty_like(q).as_strided(q.shape, (dim, dim, 1)))):
        with pytest.raises(kvq.KvqError):
            kvq.rope_fp8_kv_append(k, v, *bad.get("caches", caches), *scales, *more, q=q,
                                   q_out=bad.get("q_out"))
