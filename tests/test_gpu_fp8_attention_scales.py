"""fp8_paged_attention over pages whose value scales lie far apart, against the
64-bit oracle, with a bound that knows only what a row sees.

A probability p_j enters the second product times its page's value scale
2**e_j, as fp16 relative to a reference at least the row's largest visible
p_j 2**e_j over 2 and at most 2**6 of it, stored times 2**9: so with a relative
2^-11, or below fp16's normal numbers with an absolute 2^-25 / 2^8 = 2^-33 of
that largest product, times a code of at most 448, for each visible key. The
largest product is at most their sum, which is attention over values of 1.
Exponents up to 254 apart are added in binary32 before exp2: 2^-24 * 2^8 each,
2^-16 for the two sums and exp2 itself. Scores, sums and the output's rounding
as in test_gpu_fp8_attention.py; fp16 outputs lose 2^-25 below their normal
numbers, bf16 outputs (and binary32 sums) 2^-120."""
import numpy as np
import pytest
import torch

import __graft_entry__
from tests._fp8 import HALF_STEP, ref
from tests.test_gpu_fp8_attention import case, launch

pytestmark = pytest.mark.gpu

ONE = 0x38  # the code of 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def check(c):
    got = launch(c)
    args = c["scales"], c["table"], c["totals"], c["starts"], c["sm_scale"], c["causal"], c["window"]
    n = int(c["starts"][-1])
    want, lse, mass, spread = (x[:n] for x in ref.attention(c["q"], c["caches"], *args))
    ones = [c["caches"][0], np.full_like(c["caches"][1], ONE)]
    weight = ref.attention(c["q"], ones, *args)[0][:n]
    dx = 2.0 ** -19 * spread[..., None]
    bound = (2.0 ** -11 + 2 * dx + 2.0 ** -16) * mass + HALF_STEP[c["dtype"]] * np.abs(want) + \
        c["totals"].max() * 448 * 2.0 ** -33 * weight + \
        (2.0 ** -25 if c["dtype"] == "fp16" else 2.0 ** -120)
    out, glse = got[0][:n].cpu().double().numpy(), got[1][:n].cpu().double().numpy()
    assert np.array_equal(np.isnan(out), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.isfinite(out[fine]).all()
    over = (np.abs(out - want) / bound)[fine]
    assert over.max() <= 1, over.max()
    seen = np.isfinite(lse)
    assert np.array_equal(np.isfinite(glse), seen)
    assert np.all(np.abs(glse[seen] - lse[seen]) <=
                  dx[..., 0][seen] + 2.0 ** -18 + 2.0 ** -23 * np.abs(lse[seen]))


def quiet(c, pages, score_log2=-40.0):
    """Sets the queries near 1 and the keys of `pages` (of the cache) so that
    their scores lie `score_log2` log2 units below the others' middle."""
    c["q"] = (1.0 + c["q"] * 2.0 ** -6).astype(np.float32)
    c["q"] = torch.from_numpy(c["q"]).to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float16) \
        .float().numpy()
    k = score_log2 * np.log(2) / (c["q"].shape[2] * c["sm_scale"])
    c["caches"][0][pages] = ref.e4m3_encode(np.array([k]))[0]
    c["scales"][0][pages] = 127


NEWS = [[1, 1], [3, 2], [150, 40]]


@pytest.mark.parametrize("dim,page,dtype", [(64, 16, "bf16"), (128, 32, "fp16"), (128, 64, "bf16")])
@pytest.mark.parametrize("lift", [20, 24, 30, 40, 60])
@pytest.mark.parametrize("news", NEWS)
def test_a_loud_page_that_is_hardly_attended(news, lift, dim, page, dtype):
    """Its probabilities are 2^-40 of the others', its values 2^lift times
    theirs: from next to nothing of the output up to nearly all of it."""
    c = case(51, news, [290, 200], dim=dim, page=page, dtype=dtype)
    pages = [int(c["table"][0, 1]), int(c["table"][1, 0])]
    quiet(c, pages)
    c["scales"][1][:] -= 20                     # outputs within fp16
    c["scales"][1][pages] += lift - (20 if dtype == "fp16" and lift > 40 else 0)
    check(c)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("lift", [24, 30, 60, 120])
@pytest.mark.parametrize("news", NEWS)
def test_a_loud_page_that_some_rows_do_not_see(news, lift, dim, page):
    """Behind the window of the later rows, later than the earlier rows, or (with
    one token) out of sight of all: in tiles that are read in any case."""
    for window in (0, 100):
        c = case(52, news, [290, 200], dim=dim, page=page, window=window)
        for b, total in enumerate((290, 200)):
            first = total - news[b]                 # position of the first row
            behind = max(first - window, 0) if window else 0
            for p in (min(first + news[b] // 2 + page, total - 1), behind):
                c["scales"][1][c["table"][b, p // page]] += lift
        check(c)


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("news", NEWS)
def test_hidden_pages_of_the_largest_scale(news, page):
    """Pages that no row sees, next to some that it sees, hold the largest codes
    and the largest scale, or the NaN one."""
    for byte in (254, 255):
        c = case(53, news, [290, 200], dim=128, page=page, window=page + 3)
        for b, total in enumerate((290, 200)):
            low = max(total - news[b] - page - 2, 0)   # the first row's first key
            for column in range(low // page):
                c["scales"][1][c["table"][b, column]] = byte
                c["caches"][1][c["table"][b, column]] = 0x7E
        check(c)


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("down", [30, 70, 127])
def test_quiet_values_of_the_attended_page(news, down):
    """Nearly all weight on keys whose values are 2^-down of the others', which
    the output then hardly shows: the normaliser counts them in full."""
    c = case(54, news, [290, 200], dim=128, page=32)
    everything = np.arange(c["caches"][0].shape[0])
    few = [int(c["table"][0, 0]), int(c["table"][1, 0])]
    quiet(c, np.setdiff1d(everything, few), -20.0)
    c["scales"][1][few] = 127 - down
    check(c)


@pytest.mark.parametrize("key_step,value_step", [(3, -6), (-3, 6), (1, -2), (-1, 2)])
@pytest.mark.parametrize("news", [[1], [140]])
def test_scores_and_values_that_go_opposite_ways(news, key_step, value_step):
    """Along the sequence, a few units a page: one reference of a row rises in
    tile after tile while the other stays."""
    c = case(56, news, [640], dim=128, page=32, kv_heads=1)
    c["q"] = np.abs(c["q"])
    codes = c["caches"][0] != 0x7F
    c["caches"][0][codes] &= 0x7F
    for j in range(20):
        g = c["table"][0, j]
        c["scales"][0][g] = (118 if key_step > 0 else 124) + key_step * j // 8
        c["scales"][1][g] = 110 + value_step * (j - 10)
    check(c)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 2, 16], [150, 40, 33]])
@pytest.mark.parametrize("byte", [235, 246])
def test_large_scales(news, byte):
    """Values close to the largest of bf16, of one sign so that sums grow."""
    c = case(55, news, [290, 3, 9000], dim=128, page=64, q_size=2.0 ** -4)
    used = c["caches"][1] != 0x7F
    c["caches"][1][used] &= 0x7F
    c["scales"][1][:] = byte
    check(c)
    c["scales"][1][::2] = 60
    check(c)


@pytest.mark.parametrize("dim,page,window", [(64, 16, 0), (128, 16, 100), (128, 32, 0), (64, 64, 70)])
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("news", [[1, 1, 1], [3, 2, 16], [150, 40, 33]])
def test_scales_at_random(news, seed, dim, page, window):
    """Value scales from 2^-107 to 2^103, key scales that make rows flat or sharp."""
    c = case(57 + seed, news, [290, 200, 1500], dim=dim, page=page, window=window)
    rng = np.random.default_rng(seed)
    keys, values = c["scales"]
    keys += rng.integers(0, 6, keys.shape).astype(np.uint8)
    values[:] = rng.integers(20, 231, values.shape)
    check(c)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("news", NEWS)
def test_a_key_with_all_the_weight_gives_its_value(news, dim, page):
    """The key that raises a row's references is stored without rounding: with
    2^-40 of the weight elsewhere the output is that key's value, exactly."""
    c = case(60, news, [290, 200], dim=dim, page=page, dtype="fp16")
    quiet(c, np.arange(c["caches"][0].shape[0]), -40.3)
    values = []
    for b, total in enumerate((290, 200)):
        at = total - news[b]
        g, slot = c["table"][b, at // page], at % page
        c["caches"][0][g, :, slot] = 0
        two = np.exp2(c["scales"][1][g].astype(np.float64) - 127)
        values.append(ref.e4m3_decode(c["caches"][1][g, :, slot]) * two[:, None])
    out = launch(c)[0].cpu().double().numpy()
    for b in (0, 1):
        rows = out[c["starts"][b]:c["starts"][b + 1]]
        assert np.array_equal(rows, np.repeat(values[b], 2, 0)[None].repeat(news[b], 0))
