"""Host-side refusals of the 8-bit products and the operators around a layer of experts, with
addresses that nothing reads: every case is rejected, or returns for an empty batch, before any
launch. And the oracle against small cases worked out by hand."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from oracle import experts as ref
from oracle.fp8_paged import e4m3_encode

A, B = 0x7F0000000000, 0x7F0000100000
NAMES = ("fp8_matmul", "fp8_gated_matmul", "route_experts", "sort_by_expert", "combine_experts")


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
    header = os.path.join(os.path.dirname(__graft_entry__.__file__), "include", "kvq_experts.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = re.findall(r"^(?:const\s+)?\w+\**\s+\**(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(NAMES) | {n + "_words" for n in NAMES} | {"sort_by_expert_workspace_size"}
    raw = ctypes.CDLL(kvq.LIBRARY_PATH)
    for n in names:
        assert ctypes.cast(getattr(raw, n), ctypes.c_void_p).value
    for n in NAMES + ("fp8_expert_matmul", "fp8_expert_gated_matmul", "fp8_expert_layer"):
        assert callable(getattr(kvq, n)) and n in kvq.__all__


DENSE = dict(a=A, a_stride=256, sa=A, sa_stride=2, a_groups=2, a_rows=4, b=A, b_stride=256, b_expert=0, sb=A,
             sb_stride=2, sb_expert=0, n=128, k=256, experts=0, offsets=None, rows=None, num_rows=4, out=B,
             out_stride=128, dtype=0, status=None, stream=None)
EXPERTS = dict(DENSE, b_expert=65536, sb_expert=4, experts=3, offsets=A, rows=A, num_rows=9)


def gated(case):
    d = {k: v for k, v in case.items() if k not in ("dtype", "status", "stream")}
    return dict(d, out_scales=B, os_stride=1, status=None, stream=None)


def test_matmul_refusals(L):
    bad = [("a_rows", -1), ("num_rows", -1), ("num_rows", 1 << 31), ("a_rows", 1 << 31), ("n", 0), ("n", 1 << 25), ("k", 0),
           ("k", 250), ("k", 264), ("k", 1 << 25), ("a_groups", 0), ("a_groups", 3), ("a_stride", 240), ("a_stride", 264),
           ("a_stride", 1 << 31), ("sa_stride", -1), ("b_stride", 240), ("b_stride", 264), ("sb_stride", -1),
           ("out_stride", 127), ("out_stride", 1 << 31), ("a", None), ("sa", None), ("b", None), ("sb", None), ("out", None),
           ("a", A + 8), ("b", A + 8), ("sa", A + 2), ("sb", A + 2), ("status", A + 2)]
    for f, case, own in ((L.fp8_matmul, DENSE, [("dtype", 2), ("dtype", -1), ("out", B + 1)]),
                         (L.fp8_gated_matmul, gated(DENSE), [("n", 64), ("n", 200), ("out", B + 8), ("out_scales", None),
                                                             ("out_scales", B + 2), ("out_stride", 136), ("os_stride", 0)])):
        refused(f, case, bad + own + [("num_rows", 3), ("offsets", A), ("rows", A), ("experts", -1)])
        assert f(*dict(case, num_rows=0, a_rows=0, a=None, out=None).values()) == 0
    for f, case in ((L.fp8_matmul, EXPERTS), (L.fp8_gated_matmul, gated(EXPERTS))):
        refused(f, case, bad + [("a_rows", 0), ("experts", 1025), ("offsets", None), ("offsets", A + 4), ("rows", A + 4),
                                ("b_expert", 0), ("b_expert", 65544), ("b_expert", 1 << 40), ("sb_expert", -1)])
        assert f(*dict(case, num_rows=0, a_rows=0, a=None, offsets=None).values()) == 0


ROUTE = dict(logits=A, stride=64, dtype=2, tokens=4, experts=64, top_k=6, score=0, bias=A, groups=8, top_groups=2, renorm=1,
             scale=1.0, chosen=B, weights=B, stream=None)


def test_route_refusals(L):
    f, nan, inf = L.route_experts, float("nan"), float("inf")
    assert f(*dict(ROUTE, tokens=0, logits=None).values()) == 0
    refused(f, ROUTE, [("tokens", -1), ("tokens", 1 << 31), ("dtype", 3), ("dtype", -1), ("experts", 0), ("experts", 1032),
                       ("experts", 60), ("top_k", 0), ("top_k", 17), ("top_k", 33), ("score", 2), ("groups", 0),
                       ("groups", 64), ("groups", 33), ("top_groups", 0), ("top_groups", 9), ("renorm", 2), ("scale", nan),
                       ("scale", inf), ("stride", -1), ("stride", 1 << 31), ("logits", None), ("chosen", None),
                       ("weights", None), ("logits", A + 2), ("bias", A + 2), ("chosen", B + 4), ("weights", B + 2),
                       (dict(groups=32, experts=32, top_k=1), 0)])


SORT = dict(chosen=A, tokens=4000, top_k=2, experts=8, offsets=B, rows=B, places=B, ws=A, wsb=256, stream=None)
COMBINE = dict(y=A, ys=64, rows=9, places=A, weights=A, tokens=4, top_k=2, base=A, bs=64, out=B, os=64, n=64, dtype=0,
               stream=None)


def test_sort_and_combine_refusals(L):
    refused(L.sort_by_expert, SORT, [("tokens", -1), ("tokens", 1 << 31), ("top_k", 0), (dict(tokens=1 << 20, top_k=1 << 12), 0),
                                     ("experts", 0), ("experts", 1025), ("chosen", None), ("offsets", None), ("rows", None),
                                     ("places", None), ("chosen", A + 4), ("offsets", B + 4), ("rows", B + 4),
                                     ("places", B + 4), ("ws", None), ("ws", A + 2), ("wsb", 255)])
    size = L.sort_by_expert_workspace_size
    assert size(4000, 2, 8) == 256 and size(256, 8, 1024) == size(0, 1, 4) == 0
    assert size(-1, 1, 4) == size(1, 0, 4) == size(1 << 20, 1 << 12, 4) == size(1, 1, 0) == size(1, 1, 1025) == -1
    assert all(0 < size(t, k, 1024) <= 1 << 20 for t, k in ((4097, 1), (1 << 20, 32), ((1 << 31) - 1025, 1)))
    f = L.combine_experts
    assert f(*dict(COMBINE, tokens=0, y=None).values()) == 0
    refused(f, COMBINE, [("tokens", -1), ("tokens", 1 << 31), ("rows", -1), ("top_k", 0), ("top_k", 33), ("n", 0), ("n", 12),
                         ("n", 1 << 25), ("dtype", 2), ("ys", 60), ("ys", -8), ("os", 56), ("os", 60), ("os", 1 << 31),
                         ("bs", 4), ("y", None), ("places", None), ("weights", None), ("out", None), ("y", A + 8),
                         ("places", A + 4), ("weights", A + 2), ("base", A + 8), ("out", B + 8),
                         (dict(base=B, bs=72), 0)])


def test_words_take_the_arguments_in_order(L):
    """Each call as words gives what the call itself gives: 0 for an empty batch, a refusal for any
    word that the call refuses, or of another count."""
    def call(f, words, *rest):
        a = (ctypes.c_int64 * len(words))(*[w or 0 for w in words])
        return f(a, len(words), *rest, None)

    cases = ((L.fp8_matmul_words, dict(DENSE, a_rows=0, num_rows=0), (), ("dtype",)),
             (L.fp8_gated_matmul_words, gated(dict(DENSE, a_rows=0, num_rows=0)), (), ()),
             (L.route_experts_words, dict(ROUTE, tokens=0), (1.0,), ("dtype", "score", "renorm")),
             (L.combine_experts_words, dict(COMBINE, tokens=0), (), ("dtype",)))
    for f, case, rest, wide in cases:
        keys = [k for k in case if k not in ("stream", "scale")]
        words = [case[k] for k in keys]
        assert call(f, words, *rest) == 0
        assert call(f, words + [0], *rest) == call(f, words[:-1], *rest) == -1
        assert f(None, len(words), *rest, None) == -1
        for k in wide:  # a 32-bit argument is not cut down to its low bits
            w = list(words)
            w[keys.index(k)] += 1 << 32
            assert call(f, w, *rest) == -1, k
    for f, case, rest, bad in (
            (L.fp8_matmul_words, EXPERTS, (), [("k", 250), ("offsets", None), ("b_expert", 8), ("out_stride", 1), ("status", 2)]),
            (L.fp8_gated_matmul_words, gated(EXPERTS), (), [("n", 100), ("os_stride", 0), ("out_scales", None)]),
            (L.route_experts_words, ROUTE, (1.0,), [("top_groups", 9), ("weights", None), ("bias", 2)]),
            (L.sort_by_expert_words, SORT, (), [(k, v) for k, v in (("top_k", 0), ("experts", 0), ("places", None))]),
            (L.combine_experts_words, COMBINE, (), [("n", 12), ("bs", 4), ("out", None)])):
        keys = [k for k in case if k not in ("stream", "scale")]
        for k, v in bad:
            assert call(f, [v if x == k else case[x] for x in keys], *rest) == -1, k


def test_binding_refusals():
    """Wrong types and shapes raise before the library is called."""
    a, b = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((256, 256), dtype=torch.uint8)
    sa, sb, i = torch.zeros((4, 2)), torch.zeros((2, 2)), torch.zeros(2, dtype=torch.int64)
    out = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError):   # pageable host memory
        kvq.fp8_matmul(a, sa, b, sb, out=out)
    with pytest.raises(TypeError):
        kvq.fp8_matmul(a.float(), sa, b, sb, out=out)
    with pytest.raises(TypeError):
        kvq.fp8_matmul(a, sa, b, sb, out=out.float())
    for bad in (lambda: kvq.fp8_matmul(a, sa, b[:, :128], sb, out=out),
                lambda: kvq.fp8_matmul(a, sa, b[None], sb, out=out),
                lambda: kvq.fp8_gated_matmul(a, sa, b[:128], sb, out=a, out_scales=sa),
                lambda: kvq.fp8_expert_matmul(a, sa, b, sb, i, out=out),
                lambda: kvq.fp8_expert_matmul(a, sa, b[None], sb[None], None, out=out),
                lambda: kvq.fp8_expert_matmul(a, sa, b[None], sb[None], i[:1], out=out),
                lambda: kvq.fp8_expert_matmul(a, sa, b[None], sb[None], i, rows=i[None], out=out),
                lambda: kvq.route_experts(sa, 1, score="other"),
                lambda: kvq.route_experts(sa[0], 1),
                lambda: kvq.route_experts(sa, 0),
                lambda: kvq.route_experts(sa, 1, bias=torch.zeros(3)),
                lambda: kvq.sort_by_expert(i, 4),
                lambda: kvq.sort_by_expert(i[None], 0),
                lambda: kvq.combine_experts(out[0], i[None], sa),
                lambda: kvq.combine_experts(out, i, sa)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kvq.route_experts(i[None], 1)
    with pytest.raises(TypeError):
        kvq.combine_experts(sa, i[None], sa)


def words_of(monkeypatch, call):
    seen = []
    monkeypatch.setattr(kvq, "_tensors", lambda *_: 0)
    monkeypatch.setattr(kvq, "_call", lambda *x: seen.append(x[4]))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    call()
    return seen[-1]


def test_strides_reach_the_library(monkeypatch):
    """The strides that the tensors have, 0 for expanded scales; a single row's is made up."""
    st = torch.zeros(1, dtype=torch.int32)
    a, b = torch.zeros((4, 512), dtype=torch.uint8)[:, :256], torch.zeros((3, 130, 272), dtype=torch.uint8)[:, :128, :256]
    sa, sb = torch.zeros((1, 1)).expand(4, 1), torch.zeros((3, 2, 5))[:, :1, 1:3]
    out, i = torch.zeros((4, 140), dtype=torch.float16)[:, 4:132], torch.zeros(4, dtype=torch.int64)
    w = words_of(monkeypatch, lambda: kvq.fp8_expert_matmul(a, sa, b, sb, i, out=out, status=st))
    assert w[1] == 512 and w[3:6] == [0, 1, 4] and w[7:9] == [272, 130 * 272] and w[10:15] == [2, 10, 128, 256, 3]
    assert w[17] == 4 and w[19:21] == [140, 1]
    w = words_of(monkeypatch, lambda: kvq.fp8_matmul(a[:1], sa[:1], b[0, :1], sb[0], out=out[:1, :1], status=st))
    assert w[1] == 256 and w[3] == 1 and w[7] == 256 and w[19] == 1


def test_oracle_product_by_hand():
    a = e4m3_encode(np.array([[1.0] * 128 + [2.0] * 16]))
    b = e4m3_encode(np.array([[0.5] * 144, [-1.0] * 144]))
    y, mass = ref.matmul(a, np.array([[2.0, 3.0]]), b, np.array([[10.0, 100.0]]))
    assert np.array_equal(y, [[128 * .5 * 20 + 16 * 300, -128 * 20 - 32 * 300]]) and np.array_equal(mass, np.abs(y))
    y, _ = ref.matmul(a, np.array([[2.0]]), b, np.array([[10.0, 100.0]]))
    assert np.array_equal(y, [[128 * .5 * 20 + 16 * 200, -128 * 20 - 32 * 200]])


def test_oracle_routing_by_hand():
    x = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    chosen, w = ref.route(x, 2, "softmax", None, 1, 1, False, 1.0)
    assert chosen.tolist() == [[3, 2]] and np.allclose(w, [[0.4, 0.3]])
    chosen, w = ref.route(x, 2, "softmax", [0.5, 0, 0, 0], 1, 1, True, 3.0)
    assert chosen.tolist() == [[0, 3]] and np.allclose(w, [[0.6, 2.4]])
    # groups (0.1 + 0.2 and 0.3 + 0.4): only the second stays
    assert ref.route(x, 2, "softmax", None, 2, 1, False, 1.0)[0].tolist() == [[3, 2]]
    assert ref.route(x, 2, "softmax", [0.5, 0.5, 0, 0], 2, 1, False, 1.0)[0].tolist() == [[1, 0]]
    offsets, rows, places = ref.sort_by_expert(np.array([[2, 0], [2, 9]]), 3)
    assert offsets.tolist() == [0, 1, 1, 3] and rows.tolist() == [0, 0, 1, -1]
    assert places.tolist() == [[1, 0], [2, -1]]
