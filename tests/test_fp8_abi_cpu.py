"""Host-side refusals of the operators on the paged E4M3 cache, with addresses
that nothing reads: every case is rejected, or returns for an empty batch,
before any launch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from oracle import fp8_paged as ref

A, B = 0x7F0000000000, 0x7F0000100000
NAMES = ("add_rmsnorm_fp8", "rope_fp8_kv_append", "fp8_paged_attention",
         "fp8_paged_attention_workspace_size", "fp8_paged_attention_waits")
WORDS = ("add_rmsnorm_fp8_words", "rope_fp8_kv_append_words", "fp8_paged_attention_words")


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return kvq.lib()


def refused(f, ok, bad):
    keys = list(ok)
    for k, v in bad:
        a = dict(ok)
        a.update(k if isinstance(k, dict) else {k: v})
        assert f(*[a[x] for x in keys]) == -1, (k, v)


def test_declared_names_are_exported(L):
    header = os.path.join(os.path.dirname(__graft_entry__.__file__), "include", "kvq_fp8.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = re.findall(r"^(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(NAMES + WORDS)
    raw = ctypes.CDLL(kvq.LIBRARY_PATH)
    for n in names:
        assert ctypes.cast(getattr(raw, n), ctypes.c_void_p).value
    for n in NAMES[:-1] + ("fp8_kv_cache",):
        assert callable(getattr(kvq, n)) and n in kvq.__all__


def test_words_take_the_arguments_in_order(L):
    """Each call as words gives what the call itself gives: 0 for an empty
    batch, a refusal for any word that the call refuses, or of another count."""
    def call(f, words, *rest):
        a = (ctypes.c_int64 * len(words))(*[w or 0 for w in words])
        return f(a, len(words), *rest, None)

    norm = [A, 256, A, 256, A, 0, 0, 256, 128, B, 256, B, 2, A, 256]
    page = [16, 64, 64 * 128 * 8, 64 * 128, 128]
    append = [A, 1024, 128] * 2 + [A, 4096, 128] * 2 + [0, 0, 32, 8, 128, A, 128, 10, 128, 1, 0,
                                                      A, B] + page + [A, B, 8, A, 4, 4, A, A, 2]
    attention = [A, 4096, 128, B, 4096, 128, 0, 0, 32, 8, 128, 1, A, B] + page + [
        A, B, 8, A, 4, 4, A, A, 2, 1, 0, A, A, A, 1 << 26]
    for f, words, rest, wide in ((L.add_rmsnorm_fp8_words, norm, (1e-6,), (5, 8)),
                                 (L.rope_fp8_kv_append_words, append, (), (12, 21)),
                                 (L.fp8_paged_attention_words, attention, (0.1,), (6, 28))):
        assert call(f, words, *rest) == 0
        assert call(f, words + [0], *rest) == call(f, words[:-1], *rest) == -1
        assert f(None, len(words), *rest, None) == -1
        for i in wide:  # a 32-bit argument is not cut down to its low bits
            assert call(f, words[:i] + [1 << 32] + words[i + 1:], *rest) == -1, i


def test_norm_refusals(L):
    ok = dict(x=A, xs=256, res=A, rs=256, w=A, eps=1e-6, dtype=0, tokens=4, hidden=256, group=128,
              out=B, os=256, scales=B, ss=2, ro=A, ros=256, stream=None)
    f = L.add_rmsnorm_fp8
    empty = dict(ok, tokens=0, x=None)
    assert f(*empty.values()) == 0
    nan, inf = float("nan"), float("inf")
    refused(f, ok, [("tokens", -1), ("tokens", 1 << 31), ("dtype", 2), ("hidden", 0),
                    ("hidden", 250), ("hidden", 32776), ("group", 64), ("hidden", 264),
                    ("eps", -1.0), ("eps", nan), ("eps", inf), ("xs", 248), ("xs", 260),
                    ("xs", 1 << 60), ("rs", 128), ("os", 252), ("os", 248), ("ss", 1), ("ros", 8),
                    ("x", None), ("w", None), ("out", None), ("scales", None), ("res", None),
                    ("x", A + 8), ("w", A + 2), ("out", B + 4), ("scales", B + 2), ("res", A + 8),
                    ("ro", A + 8), (dict(ro=A, ros=264), 0)])


APPEND = dict(k=A, kt=256, kh=64, v=A, vt=256, vh=64, q=A, qt=256, qh=64, qo=B, qot=256, qoh=64,
              dtype=0, tokens=4, heads=4, kv_heads=2, dim=64, cs=A, cstride=64, crows=10, rot=64,
              inter=1, pos=None, kc=B, vc=B, pages=4, page=16, ps=2048, hs=1024, ss=64, ks=B, vs=B,
              sps=2, table=A, ts=3, maxp=3, lens=A, starts=A, seqs=2, stream=None)


def test_append_refusals(L):
    f, ok = L.rope_fp8_kv_append, APPEND
    for e in (dict(ok, tokens=0, k=None), dict(ok, seqs=0, table=None)):
        assert f(*e.values()) == 0
    refused(f, ok, [("tokens", -1), ("tokens", 1 << 31), ("seqs", -1), ("seqs", 1 << 21),
                    ("dtype", 2), ("inter", 2), ("dim", 8), ("dim", 72), ("dim", 272), ("rot", 8),
                    ("rot", 80), ("rot", -16), ("pages", 0), ("page", 8), ("page", 24),
                    ("page", 512), ("kv_heads", 0), ("kv_heads", 70000), ("maxp", -1), ("ts", 2),
                    ("ss", 48), ("ss", 72), ("hs", 1000), ("hs", -16), ("ps", 2040),
                    ("ps", 1 << 62), ("sps", 1), ("kt", 252), ("kh", 60), ("kt", -8),
                    ("kh", 32), ("vt", 1 << 60), ("heads", 0), ("qo", None), ("qt", 4),
                    ("qot", 32), (dict(qo=A, qot=512), 0), ("crows", 0), ("cstride", 48),
                    ("cstride", 66), ("k", None), ("v", None), ("kc", None), ("vc", None),
                    ("ks", None), ("vs", None), ("lens", None), ("starts", None), ("table", None),
                    ("cs", None), ("k", A + 8), ("v", A + 2), ("q", A + 8), ("qo", B + 8),
                    ("kc", B + 8), ("cs", A + 8), ("pos", A + 4), ("table", A + 4),
                    ("lens", A + 4), ("starts", A + 4)])


ATTEND = dict(q=A, qt=256, qh=64, out=B, ot=256, oh=64, dtype=0, tokens=4, heads=4, kv_heads=2,
              dim=64, maxq=3, kc=B, vc=B, pages=4, page=16, ps=2048, hs=1024, ss=64, ks=B, vs=B,
              sps=2, table=A, ts=3, maxp=3, lens=A, starts=A, seqs=2, scale=0.1, causal=1, window=0,
              lse=None, status=None, ws=A, wsb=64 << 20, stream=None)


def test_attention_refusals(L):
    f, ok = L.fp8_paged_attention, ATTEND
    for e in (dict(ok, tokens=0, q=None), dict(ok, seqs=0, table=None)):
        assert f(*e.values()) == 0
    refused(f, ok, [("tokens", -1), ("tokens", 1 << 31), ("seqs", -1), ("seqs", 1 << 21),
                    ("dtype", 2), ("heads", 5), ("heads", 1), ("heads", 70000), ("kv_heads", 0),
                    ("dim", 96), ("dim", 256), ("maxq", -1), ("pages", 0), ("page", 8),
                    ("page", 24), ("page", 512), ("maxp", -1), ("ts", 2), ("ss", 48), ("ss", 72),
                    ("hs", 1000), ("ps", 2040), ("sps", 1), ("qt", 252), ("qh", 60), ("qt", -8),
                    ("ot", 32), ("oh", 32), ("ot", 1 << 60), ("scale", -0.1),
                    ("scale", float("nan")), ("scale", float("inf")), ("causal", 2),
                    ("window", -1), ("q", None), ("out", None), ("out", A), ("kc", None),
                    ("vc", None), ("ks", None), ("vs", None), ("table", None), ("lens", None),
                    ("starts", None), ("ws", None), ("q", A + 8), ("out", B + 8), ("kc", B + 4),
                    ("vc", B + 8), ("table", A + 4), ("lens", A + 4), ("starts", A + 4),
                    ("lse", A + 2), ("status", A + 2), ("ws", A + 128), ("wsb", 0)])


def test_workspace_size(L):
    g = L.fp8_paged_attention_workspace_size
    for bad in ((-1, 4, 4, 2, 64, 1), (2, -1, 4, 2, 64, 1), (2, 4, 5, 2, 64, 1),
                (2, 4, 4, 0, 64, 1), (2, 4, 4, 2, 96, 1), (2, 4, 4, 2, 64, -1)):
        assert g(*bad) == -1
    assert g(0, 4, 4, 2, 64, 1) == 0 and g(2, 0, 4, 2, 64, 1) == 0
    for shapes in ((1, 1, 1, 1, 64, 1), (64, 64, 32, 8, 128, 1), (1000, 9000, 128, 1, 128, 2000),
                   (1 << 20, 1 << 30, 65535, 1, 128, 1 << 30)):
        assert 0 <= g(*shapes) <= 64 << 20
    assert g(1, 1, 1, 1, 64, 1) > 0 and g(64, 64, 32, 8, 128, 1) > 0


def test_which_calls_can_time_out(L):
    """Those with more than 32 rows (queries x heads) to a key head."""
    w = L.fp8_paged_attention_waits
    assert w(64, 32, 8, 1) == 0 and w(64, 32, 8, 8) == 0 and w(3, 16, 1, 9) == 1
    assert w(64, 32, 8, 9) == 1 and w(64, 66, 2, 1) == 1 and w(1, 32, 1, 5) == 0


def test_places_in_lse_are_counted_in_64_bits():
    """num_tokens * num_heads may pass 2**31 (275 GB of outputs, which no test
    has room for): every access goes through lse_place, whose width its own
    static_assert checks."""
    csrc = os.path.join(os.path.dirname(kvq.__file__), "csrc")
    uses = 0
    for name in ("fp8_attention_rows.cu", "fp8_attention_tiles.cu"):
        text = open(os.path.join(csrc, name)).read()
        found = re.findall(r"p\.lse(?:\[| \+)\s*(\w+)", text)
        uses += len(found)
        assert set(found) == {"lse_place"}
    assert uses == 6
    assert "static_assert(lse_place(1 << 20, 4096, 7) ==" in open(os.path.join(csrc, "fp8_attention.cuh")).read()


def test_binding_refusals():
    """Wrong types and shapes raise before the library is called."""
    bf = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kvq.add_rmsnorm_fp8(torch.zeros((4, 64)), torch.zeros(64), 1e-6)
    with pytest.raises(TypeError):   # pageable host memory
        kvq.add_rmsnorm_fp8(bf[:, 0], bf[0, 0], 1e-6, out=torch.zeros((4, 64), dtype=torch.uint8),
                            scales=torch.zeros((4, 1)))
    with pytest.raises(ValueError):
        kvq.add_rmsnorm_fp8(bf[:, 0], bf[0, 0], 1e-6, group=64)
    with pytest.raises(ValueError):
        kvq.add_rmsnorm_fp8(bf, bf[0, 0], 1e-6)
    cache = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    scales = torch.zeros((3, 2), dtype=torch.uint8)
    i = torch.zeros((1, 2), dtype=torch.int64)
    with pytest.raises(TypeError):
        kvq.rope_fp8_kv_append(bf.float(), bf, cache, cache, scales, scales, i, i[0, :1], i[0])
    with pytest.raises(TypeError):
        kvq.rope_fp8_kv_append(bf, bf, cache.float(), cache, scales, scales, i, i[0, :1], i[0])
    with pytest.raises(ValueError):
        kvq.rope_fp8_kv_append(bf, bf, cache, cache, scales, scales, i, i[0, :1], i[0],
                               rotary_dim=64)
    with pytest.raises(TypeError):
        kvq.fp8_paged_attention(bf.double(), cache, cache, scales, scales, i, i[0, :1], i[0], 1, 1.0)
    with pytest.raises(ValueError):
        kvq.fp8_paged_attention(bf[0], cache, cache, scales, scales, i, i[0, :1], i[0], 1, 1.0)


def test_strides_of_expanded_rows_reach_the_library():
    """The binding passes the strides that the tensors have, 0 for expanded and
    less than a row for overlapping rows; only a single row's is made up."""
    def cache_args(scales, table):
        cache = torch.zeros((scales.shape[0], 2, 16, 64), dtype=torch.uint8)
        a = kvq._fp8_cache_args(cache, cache, scales, scales, table, 2, 64)
        return a[9], a[11]

    scales, table = torch.zeros((40, 2), dtype=torch.uint8), torch.zeros((5, 8), dtype=torch.int64)
    assert cache_args(scales, table) == (2, 8)
    assert cache_args(scales[:1].expand(40, 2), table[:1].expand(5, 8)) == (0, 0)
    assert cache_args(scales.as_strided((40, 2), (1, 1)), table.as_strided((5, 8), (3, 1))) == (1, 3)
    assert cache_args(scales[:, :2].as_strided((4, 2), (6, 1)), table[::2]) == (6, 16)
    # one row, whatever its stride
    assert cache_args(scales.as_strided((1, 2), (0, 1)), table.as_strided((1, 8), (0, 1))) == (2, 8)
    assert cache_args(scales.as_strided((1, 2), (9, 1)), table.as_strided((1, 8), (3, 1))) == (2, 8)


def test_strides_of_the_rotation_table_reach_the_library(monkeypatch):
    words = []
    monkeypatch.setattr(kvq, "_tensors", lambda *_: 0)
    monkeypatch.setattr(kvq, "_call", lambda *a: words.append(a[4]))
    bf = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache, scales = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2), dtype=torch.uint8)
    i = torch.zeros((1, 2), dtype=torch.int64)
    cs = torch.zeros((10, 64))
    for table, stride in ((cs, 64), (cs[:1].expand(10, 64), 0), (cs.as_strided((9, 64), (32, 1)), 32),
                          (torch.zeros((10, 80)), 80), (cs.as_strided((1, 64), (0, 1)), 64),
                          (torch.zeros((1, 70)), 64)):
        kvq.rope_fp8_kv_append(bf, bf, cache, cache, scales, scales, i, i[0, :1], i[0], cos_sin=table)
        assert words[-1][18] == stride


def test_strides_that_only_reading_allows(L):
    """One row of the block table for all sequences, in both operators; one
    page's scales for all pages in attention, while an append would write them
    from several places at once."""
    assert L.rope_fp8_kv_append(*dict(APPEND, tokens=0, ts=0).values()) == 0
    assert L.fp8_paged_attention(*dict(ATTEND, tokens=0, ts=0, sps=0).values()) == 0
    refused(L.rope_fp8_kv_append, APPEND, [("sps", 0), ("ts", -1), ("cstride", 0)])
    refused(L.fp8_paged_attention, ATTEND, [("sps", -1), ("ts", -1)])


def test_the_handle_0_is_the_default_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    assert kvq._raw_stream(0, "cuda:0") == ("default", "cuda:0")
    assert kvq._raw_stream(A, "cuda:0") == (A, "cuda:0")


def test_what_is_written_may_not_overlap_itself(L):
    """Rows, heads, slots and pages that lie on each other, in any order of the
    dimensions; the same strides are fine to read, and dimensions of one do not
    count."""
    append, attend = L.rope_fp8_kv_append, L.fp8_paged_attention
    pages = [dict(ps=0), dict(hs=0), dict(ps=1024), dict(hs=512), dict(ps=2048, hs=64, ss=64),
             dict(ps=64, hs=1024, ss=64)]
    refused(append, APPEND, [(x, 0) for x in pages])
    for x in pages + [dict(kt=0), dict(vt=0, vh=64)]:
        assert attend(*{**ATTEND, "tokens": 0, **{k: v for k, v in x.items() if k in ATTEND}}.values()) == 0
    refused(append, APPEND, [(dict(qot=64, qoh=64), 0), (dict(qot=192, qoh=64), 0),
                             (dict(qot=64, qoh=192), 0), (dict(qot=0), 0)])
    refused(attend, ATTEND, [(dict(ot=64, oh=64), 0), (dict(ot=192, oh=64), 0),
                             (dict(ot=64, oh=192), 0), (dict(ot=0), 0), (dict(oh=0), 0)])
    # slots first, heads first, gaps, one page, one head (these pass every check
    # that comes before that of a pointer)
    for x in (dict(ps=2048, hs=64, ss=128), dict(ps=1024, hs=4096), dict(ps=4096, hs=2000 // 16 * 16),
              dict(pages=1, ps=0), dict(kv_heads=1, hs=0, sps=1)):
        assert append(*dict(APPEND, tokens=0, **x).values()) == 0
    for x in (dict(qot=64, qoh=256), dict(qot=264, qoh=64), dict(heads=1, qoh=0)):
        assert append(*dict(APPEND, tokens=0, **x).values()) == 0
    for x in (dict(ot=64, oh=256), dict(ot=264, oh=64)):
        assert attend(*dict(ATTEND, tokens=0, **x).values()) == 0


def test_oracle_codes_are_the_nearest():
    """The oracle's E4M3 against brute force over all finite codes."""
    values = ref.e4m3_decode(np.arange(127, dtype=np.uint8))
    mids = (values[1:] + values[:-1]) / 2
    x = np.concatenate([values, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), [449.0, 1e30]])
    x = np.concatenate([x, -x])
    got = ref.e4m3_encode(x)
    near = np.abs(np.minimum(np.abs(x), 448.0)[:, None] - values[None])
    best = near.min(1)
    for c, n, b, v in zip(got, near, best, x):
        ties = np.nonzero(n == b)[0]
        want = ties[0] if len(ties) == 1 or ties[0] % 2 == 0 else ties[1]
        assert (c & 0x7F) == want and (c >> 7) == np.signbit(v)
    assert ref.e4m3_encode(np.array([np.nan]))[0] == 0x7F


def test_oracle_append_is_nearly_independent_of_the_chunks():
    """A page filled at once and token by token has the same scale; codes differ
    only where an earlier rounding below the normal range is rounded again."""
    rng = np.random.default_rng(0)
    k = rng.standard_normal((16, 1, 32)).astype(np.float32)
    one = [np.zeros((1, 1, 16, 32), np.uint8) for _ in range(2)], [np.zeros((1, 1), np.uint8) for _ in range(2)]
    two = [x.copy() for x in one[0]], [x.copy() for x in one[1]]
    table = np.zeros((1, 1), np.int64)
    ref.append(k, k, *one, table, [0], [0, 16], None, 0, True)
    for i in range(16):
        ref.append(k[i:i + 1], k[i:i + 1], *two, table, [i], [0, 1], None, 0, True)
    assert np.array_equal(one[1][0], two[1][0])
    a, b = ref.e4m3_decode(one[0][0]), ref.e4m3_decode(two[0][0])
    assert np.all(np.abs(a - b) <= np.where(np.abs(a) < 2.0 ** -6, 2.0 ** -9, 0))


def test_oracle_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(1)
    codes = [rng.integers(0, 127, (2, 1, 16, 64)).astype(np.uint8) for _ in range(2)]
    scales = [np.full((2, 1), 130, np.uint8) for _ in range(2)]
    q = rng.standard_normal((1, 3, 64))
    out, lse, mass, _ = ref.attention(q, codes, scales, np.array([[1]]), [1], [0, 1], 0.125)
    v = ref.e4m3_decode(codes[1][1, 0, 0]) * 8
    assert np.allclose(out[0], v) and np.allclose(mass[0], np.abs(v))
    assert np.allclose(lse[0], q[0] @ ref.e4m3_decode(codes[0][1, 0, 0]))
