"""The 8-bit products with several tiles for every block or pair of blocks: what runs on over a tile's
end, and matrices of more rows than a band of tiles has (tolerances: tests/_experts.py)."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._experts import DEV, check_gated, check_product, codes, f32, host, i64, ref, u8, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def by_expert(a, sa, b, sb, offsets, index):
    """The oracle's product, an expert's rows at once."""
    y, mass = (np.zeros((offsets[-1], b.shape[1])) for _ in range(2))
    for e in range(len(b)):
        at = np.arange(offsets[e], offsets[e + 1])
        row = at if index is None else index[at]
        at, row = at[(row >= 0) & (row < len(a))], row[(row >= 0) & (row < len(a))]
        y[at], mass[at] = ref.matmul(a[row], sa[row], b[e], sb[e])
    return y, mass


def run(offsets, n, k, gated, indexed, dtype, seed):
    """By expert, each row or through an index with rows outside; twice, with the same bits."""
    rng = np.random.default_rng(seed)
    rows = offsets[-1]
    a, sa = codes(rng, (rows // 3 if indexed else rows, k))
    b, sb = weights(rng, (len(offsets) - 1, 2 * n if gated else n, k))
    index = rng.integers(-1, len(a) + 1, rows) if indexed else None
    want = by_expert(a, sa, b, sb, offsets, index)
    args = u8(a), f32(sa), u8(b), f32(sb), i64(offsets)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    more = dict(rows=i64(index) if indexed else None, status=st)
    if gated:
        got = kvq.fp8_expert_gated_matmul(*args, **more)
        check_gated(got, *want)
        again = kvq.fp8_expert_gated_matmul(*args, **more)
        assert np.array_equal(host(got[0]), host(again[0])) and torch.equal(got[1], again[1])
    else:
        got = kvq.fp8_expert_matmul(*args, dtype=torch.float16 if dtype == "fp16" else torch.bfloat16, **more)
        check_product(got, *want, dtype)
        assert torch.equal(got, kvq.fp8_expert_matmul(*args, dtype=got.dtype, **more))
    assert st.item() == 0
    return args, got


KINDS = [("aligned", 3328), ("any", 3301), ("gated", 1664)]


@pytest.mark.parametrize("k", [128, 272, 512])
@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("kind,n", KINDS)
def test_many_rows_many_tiles(kind, n, indexed, k):
    """286 tiles of 256 rows by 13 blocks of columns, more than three for each of 76 pairs; 17 tiles
    of rows for one expert and 5 for another, last ones of 180 and 3 rows."""
    run([0, 4276, 4276, 4276 + 1027], n, k, kind == "gated", indexed, "fp16" if kind == "any" else "bf16", k + n)


@pytest.mark.parametrize("kind,n", KINDS)
def test_many_rows_of_one_matrix(kind, n):
    rng = np.random.default_rng(n)
    a, sa = codes(rng, (5003, 256))
    b, sb = weights(rng, (2 * n if kind == "gated" else n, 256))
    want = ref.matmul(a, sa, b, sb)
    args = u8(a), f32(sa), u8(b), f32(sb)
    if kind == "gated":
        check_gated(kvq.fp8_gated_matmul(*args), *want)
    else:
        check_product(kvq.fp8_matmul(*args), *want, "bf16")


@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,k", [(300, 1168), (600, 640), (1400, 400)])
def test_few_rows_many_tiles(rows, k, gated, indexed):
    """50 experts by 8 blocks of columns, in tiles of 16, 32 and 64 rows: two to four and more tiles
    for a block of the grid, each of several steps."""
    rng = np.random.default_rng(rows)
    share = rng.multinomial(rows, rng.dirichlet(np.full(50, 3.0)))
    run(np.concatenate([[0], np.cumsum(share)]), 1024, k, gated, indexed, "bf16", rows)
