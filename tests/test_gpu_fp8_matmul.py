"""fp8_matmul and its kin against the 64-bit definition (tolerances: tests/_experts.py)."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._experts import (DEV, DTYPES, call_over_freed_blocks, check_gated, check_product, codes, f32, host,
                            i64, ref, u8, weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()
    # the fill that call_over_freed_blocks queues: loading its kernel waits for the device
    torch.empty(1, dtype=torch.uint8, device=DEV).fill_(0x55)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def dense(seed, m, n, k, per_token=False):
    rng = np.random.default_rng(seed)
    a, sa = codes(rng, (m, k))
    if per_token:
        sa = sa.max(1, keepdims=True)
    return (a, sa, *weights(rng, (n, k)))


def product(case, one_expert=False, gated=False, **kw):
    """One matrix, as such or as the only expert: the two choose their kernels by rules of their own."""
    a, sa, b, sb = u8(case[0]), f32(case[1]), u8(case[2]), f32(case[3])
    if one_expert:
        f = kvq.fp8_expert_gated_matmul if gated else kvq.fp8_expert_matmul
        return f(a, sa, b[None], sb[None], i64([0, len(case[0])]), **kw)
    return (kvq.fp8_gated_matmul if gated else kvq.fp8_matmul)(a, sa, b, sb, **kw)


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 128, 128), (2, 129, 128), (3, 8, 48), (16, 256, 256), (17, 100, 272), (5, 4096, 512),
    (31, 640, 1152), (33, 127, 1024), (48, 384, 2048), (64, 1000, 144), (65, 300, 384), (127, 255, 640),
    (128, 256, 128), (129, 257, 1040), (200, 1024, 896), (333, 777, 512), (300, 40, 2560), (8, 384, 8192),
    (1, 200, 16384), (321, 3900, 272), (1300, 1030, 144)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sizes(m, n, k, dtype):
    case = dense(m + n + k, m, n, k, per_token=(m + n) % 3 == 0)
    st = status()
    want = ref.matmul(*case)
    for one_expert in (False, True):
        got = product(case, one_expert, dtype=DTYPES[dtype], status=st)
        assert st.item() == 0 and got.dtype == DTYPES[dtype]
        check_product(got, *want, dtype)


@pytest.mark.parametrize("m,n,k", [
    (1, 128, 16), (1, 256, 128), (7, 384, 144), (16, 128, 1024), (17, 256, 400), (33, 640, 512), (64, 128, 2048),
    (65, 384, 256), (128, 256, 640), (130, 128, 1168), (300, 512, 384), (4, 128, 8192), (500, 2560, 272)])
def test_gated_sizes(m, n, k):
    case = dense(m + n + k, m, 2 * n, k, per_token=m % 2 == 0)
    st = status()
    want = ref.matmul(*case)
    for one_expert in (False, True):
        got = product(case, one_expert, gated=True, status=st)
        assert st.item() == 0
        check_gated(got, *want)


def split(rng, rows, experts, skew):
    """Offsets: some experts without rows, some with most."""
    p = rng.dirichlet(np.full(experts, skew))
    return np.concatenate([[0], np.cumsum(rng.multinomial(rows, p))])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens,rows,experts,n,k,skew", [
    (5, 1, 3, 128, 128, 1), (9, 40, 8, 128, 272, 0.3), (24, 144, 64, 256, 512, 1), (40, 300, 5, 384, 144, 0.5),
    (200, 900, 3, 128, 640, 2), (100, 700, 30, 256, 256, 0.2), (3, 513, 1024, 128, 128, 0.1), (50, 260, 2, 128, 1024, 5)])
def test_experts(tokens, rows, experts, n, k, skew, gated):
    rng = np.random.default_rng(rows + n)
    a, sa = codes(rng, (tokens, k))
    b, sb = weights(rng, (experts, 2 * n if gated else n, k))
    offsets, index = split(rng, rows, experts, skew), rng.integers(0, tokens, rows)
    y, mass = ref.by_expert(a, sa, b, sb, offsets, index, rows)
    args = u8(a), f32(sa), u8(b), f32(sb), i64(offsets)
    st = status()
    if gated:
        check_gated(kvq.fp8_expert_gated_matmul(*args, rows=i64(index), status=st), y, mass)
    else:
        check_product(kvq.fp8_expert_matmul(*args, rows=i64(index), status=st), y, mass, "bf16")
    assert st.item() == 0
    # rows of a in their order
    a, sa = codes(rng, (rows, k))
    y, mass = ref.by_expert(a, sa, b, sb, offsets, None, rows)
    if gated:
        check_gated(kvq.fp8_expert_gated_matmul(u8(a), f32(sa), *args[2:]), y, mass)
    else:
        check_product(kvq.fp8_expert_matmul(u8(a), f32(sa), *args[2:]), y, mass, "bf16")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [40, 600])
def test_rows_that_no_expert_has_stay(rows, gated):
    """Rows before the first and behind the last expert, and offsets outside, keep what they hold."""
    rng = np.random.default_rng(5)
    a, sa = codes(rng, (rows, 256))
    b, sb = weights(rng, (3, 256, 256))
    offsets = [-7, 5, 5, rows - 3] if rows == 40 else [11, 20, 300, rows - 11]
    low, high = max(offsets[0], 0), offsets[-1]
    y, mass = ref.by_expert(a, sa, b, sb, np.array(offsets), None, rows)
    n = 128 if gated else 256
    out = torch.full((rows, n), 0x55, dtype=torch.uint8, device=DEV) if gated else \
        torch.full((rows, n), 9.0, dtype=torch.float16, device=DEV)
    scales = torch.full((rows, 1), 7.0, device=DEV)
    args = u8(a), f32(sa), u8(b), f32(sb), i64(offsets)
    if gated:
        kvq.fp8_expert_gated_matmul(*args, out=out, out_scales=scales)
        check_gated((out[low:high], scales[low:high]), y[low:high], mass[low:high])
        assert torch.all(scales[:low] == 7) and torch.all(scales[high:] == 7)
    else:
        kvq.fp8_expert_matmul(*args, out=out)
        check_product(out[low:high], y[low:high], mass[low:high], "fp16")
    held = 0x55 if gated else 9
    assert torch.all(out[:low] == held) and torch.all(out[high:] == held)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,experts", [(12, 3), (600, 4), (40, 40)])
def test_decreasing_offsets_write_nothing(rows, experts, gated):
    a, sa, b, sb = dense(7, rows, 256, 2048)
    offsets = i64([0, rows] * (experts // 2) + [rows // 2] * (experts % 2) + [rows])
    if experts % 2 == 0:
        offsets[experts] = rows // 2
    b, sb = u8(b).expand(experts, -1, -1), f32(sb).expand(experts, -1, -1)
    out = torch.full((rows, 128 if gated else 256), 9, dtype=torch.uint8 if gated else torch.float16, device=DEV)
    scales, st = torch.full((rows, 1), 7.0, device=DEV), status()
    if gated:
        kvq.fp8_expert_gated_matmul(u8(a), f32(sa), b.contiguous(), sb.contiguous(), offsets, out=out,
                                    out_scales=scales, status=st)
    else:
        kvq.fp8_expert_matmul(u8(a), f32(sa), b.contiguous(), sb.contiguous(), offsets, out=out, status=st)
    assert torch.all(out == 9) and torch.all(scales == 7) and st.item() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [20, 500])
def test_rows_outside_count_as_zeros(rows, gated):
    """Whatever the row that stands in for them holds, NaN codes among it."""
    rng = np.random.default_rng(6)
    a, sa = codes(rng, (4, 256))
    a[0] = 0x7F
    b, sb = weights(rng, (2, 256, 256))
    index = rng.integers(1, 4, rows)
    index[::3] = -1
    index[1::5] = 4
    index[2::7] = 1 << 40
    offsets = np.array([0, rows // 3, rows])
    y, mass = ref.by_expert(a, sa, b, sb, offsets, index, rows)
    args = u8(a), f32(sa), u8(b), f32(sb), i64(offsets)
    if gated:
        got = kvq.fp8_expert_gated_matmul(*args, rows=i64(index))
        check_gated(got, y, mass)
    else:
        got = kvq.fp8_expert_matmul(*args, rows=i64(index))
        check_product(got, y, mass, "bf16")
        assert torch.all(got[::3] == 0)


@pytest.mark.parametrize("one_expert", [False, True])
@pytest.mark.parametrize("m", [7, 300])
def test_nan_and_range_stay_in_their_row_and_column(m, one_expert):
    case = [x.copy() for x in dense(3, m, 256, 384)]
    case[0][2, 5] = 0x7F
    case[2][9, 200] = 0xFF
    got = product(case, one_expert).float().cpu().numpy()
    bad = np.zeros(got.shape, bool)
    bad[2], bad[:, 9] = True, True
    assert np.array_equal(np.isnan(got), bad)
    case[0][2, 5] = case[2][9, 200] = 0
    y, mass = ref.matmul(*case)
    assert np.all(np.abs(got - y)[~bad] <= (2.0 ** -8 * np.abs(y) + 2.0 ** -14 * mass)[~bad])
    # gated: a NaN's code is 0x7F, and the scale goes by the others
    case[0][2, 5] = 0x7F
    out, scales = product(case, one_expert, gated=True)
    assert np.all(host(out)[2] == 0x7F) and np.all(host(out)[3:] != 0x7F)
    assert np.all(scales[2].cpu().numpy() == np.float32(1e-4) / np.float32(448))


@pytest.mark.parametrize("m", [9, 200])
def test_strides(m):
    """Rows, columns of scales and results with gaps; NaN lies in the gaps."""
    a, sa, b, sb = dense(4, m, 250, 400)
    wide = torch.full((m, 11), float("nan"), device=DEV)
    wide[:, 3:7] = f32(sa)
    blocks = torch.full((2, 9), float("nan"), device=DEV)
    blocks[:, :4] = f32(sb)
    out = torch.full((m, 301), 9.0, dtype=torch.bfloat16, device=DEV)
    got = kvq.fp8_matmul(u8(a, 416), wide[:, 3:7], u8(b, 448), blocks[:, :4], out=out[:, 1:251])
    check_product(got, *ref.matmul(a, sa, b, sb), "bf16")
    assert torch.all(out[:, 0] == 9) and torch.all(out[:, 251:] == 9)
    # experts that lie apart, and one scale for all rows
    rng = np.random.default_rng(1)
    b, sb = weights(rng, (3, 250, 400))
    far = torch.full((3, 260, 400), 0x7F, dtype=torch.uint8, device=DEV)
    far[:, :250] = u8(b)
    scales = torch.full((3, 5, 4), float("nan"), device=DEV)
    scales[:, :2] = f32(sb)
    one = f32(sa[:1, :1]).expand(m, 1)
    got = kvq.fp8_expert_matmul(u8(a), one, far[:, :250], scales[:, :2], i64([0, 4, 4, m]))
    check_product(got, *ref.by_expert(a, np.repeat(sa[:1, :1], m, 0), b, sb, [0, 4, 4, m], None, m), "bf16")
    # gated
    b, sb = weights(rng, (512, 400))
    out = torch.full((m, 272), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((m, 5), 7.0, device=DEV)
    got = kvq.fp8_gated_matmul(u8(a), f32(sa), u8(b, 416), f32(sb), out=out[:, :256], out_scales=s[:, 1:3])
    check_gated(got, *ref.matmul(a, sa, b, sb))
    assert torch.all(out[:, 256:] == 0x55) and torch.all(s[:, 0] == 7) and torch.all(s[:, 3:] == 7)


def far(t, stride):
    """The tensor with `stride` elements from one of its first dimension to the next."""
    at = torch.empty(t.shape[0] * stride, dtype=t.dtype, device=DEV).as_strided(t.shape, (stride, *t.stride()[1:]))
    return at.copy_(t)


@pytest.mark.parametrize("m", [40, 300])
def test_places_beyond_32_bits(m):
    """Rows of a and of the result, and experts, further apart than 32 bits reach."""
    rng = np.random.default_rng(m)
    a, sa = codes(rng, (m, 256))
    b, sb = weights(rng, (3, 256, 256))
    apart = 5_000_000_000 // m // 64 * 64
    index, offsets = rng.permutation(m), [0, m // 3, m // 2, m]
    args = far(u8(a), apart), far(f32(sa), apart // 32), far(u8(b), 2_500_000_000), f32(sb), i64(offsets)
    out = far(torch.zeros((m, 256), dtype=torch.bfloat16, device=DEV), apart // 2)
    y, mass = ref.by_expert(a, sa, b, sb, np.array(offsets), index, m)
    for rows in (i64(index), None):
        if rows is None:
            y, mass = ref.by_expert(a, sa, b, sb, np.array(offsets), None, m)
        check_product(kvq.fp8_expert_matmul(*args, rows=rows, out=out), y, mass, "bf16")
        z = far(torch.zeros((m, 128), dtype=torch.uint8, device=DEV), apart)
        check_gated(kvq.fp8_expert_gated_matmul(*args, rows=rows, out=z), y, mass)
    one = kvq.fp8_matmul(args[0], args[1], u8(b[1]), f32(sb[1]), out=out)
    check_product(one, *ref.matmul(a, sa, b[1], sb[1]), "bf16")


def test_no_rows():
    a, sa, b, sb = dense(4, 3, 128, 128)
    got = kvq.fp8_matmul(u8(a)[:0], f32(sa)[:0], u8(b), f32(sb))
    assert got.shape == (0, 128)
    got = kvq.fp8_expert_matmul(u8(a), f32(sa), u8(b)[None], f32(sb)[None], i64([0, 0]), rows=i64([]))
    assert got.shape == (0, 128)
    out = torch.full((3, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    kvq.fp8_expert_matmul(u8(a), f32(sa), u8(b)[None], f32(sb)[None], i64([3, 1]), out=out)
    assert torch.all(out == 9)


@pytest.mark.parametrize("m,one_expert", [(6, False), (400, False), (400, True)])
def test_same_bits_each_time_on_any_stream_and_in_a_graph(m, one_expert):
    a, sa, b, sb = dense(8, m, 1024, 2048)
    args = u8(a), f32(sa), u8(b), f32(sb)
    matmul, gated_matmul = kvq.fp8_matmul, kvq.fp8_gated_matmul
    if one_expert:
        args = u8(a), f32(sa), u8(b)[None], f32(sb)[None], i64([0, m])
        matmul, gated_matmul = kvq.fp8_expert_matmul, kvq.fp8_expert_gated_matmul
    st = status()
    want, z = matmul(*args), gated_matmul(*args)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    codes_, scales = torch.empty_like(z[0]), torch.empty_like(z[1])
    with torch.cuda.graph(graph):
        matmul(*args, out=out, status=st)
        gated_matmul(*args, out=codes_, out_scales=scales, status=st)
    for _ in range(3):
        out.zero_()
        scales.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(scales, z[1]) and np.array_equal(host(codes_), host(z[0]))
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for s, g in zip(streams, got):
            g.append(matmul(*args, status=st, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for g in got for x in g) and st.item() == 0


def test_only_scales_and_offsets_may_lie_in_host_memory():
    a, sa, b, sb = dense(8, 70, 256, 256)
    args = u8(a), f32(sa), u8(b), f32(sb)
    want = kvq.fp8_matmul(*args)
    assert torch.equal(kvq.fp8_matmul(args[0], args[1].cpu().pin_memory(), args[2], args[3].cpu().pin_memory()), want)
    out = torch.empty((70, 256), dtype=torch.bfloat16).pin_memory()
    for bad in (lambda: kvq.fp8_matmul(*args, out=out), lambda: kvq.fp8_matmul(args[0].cpu().pin_memory(), *args[1:]),
                lambda: kvq.fp8_matmul(args[0], args[1], args[2].cpu().pin_memory(), args[3]),
                lambda: kvq.fp8_gated_matmul(*args, out=out.view(torch.uint8)[:, :128].contiguous().pin_memory())):
        with pytest.raises(TypeError):
            bad()


def test_outputs_are_made_under_the_calls_stream():
    a, sa, b, sb = dense(8, 64, 1024, 512)
    args = u8(a), f32(sa), u8(b), f32(sb)
    want = kvq.fp8_matmul(*args)
    got = call_over_freed_blocks(lambda s: kvq.fp8_matmul(*args, stream=s), [want], (4,))
    assert torch.equal(got, want)
