"""Cases for the tests of the paged E4M3 cache: numpy arrays that the oracle
takes, and the same on the GPU."""
import numpy as np
import torch

from tests._gpu import DEV, to_dev
from oracle import fp8_paged as ref

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def rows(rng, shape, dtype, spread=0.0):
    """Random values that the type holds exactly, as float32; `spread` (log2)
    varies the size of the rows."""
    x = rng.standard_normal(shape)
    if spread:
        x = x * np.exp2(rng.uniform(-spread, spread, shape[:-1]))[..., None]
    return torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).float().numpy()


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DTYPES[dtype]).to(DEV)


def make_table(rng, totals, page, spare=3, extra_columns=2, fill=-1):
    need = [-(-int(t) // page) for t in totals]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(totals), max(need + [0]) + extra_columns), fill, np.int64)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, pages


def random_cache(rng, pages, heads, page, dim, spread=1.0):
    """Codes of N(0, 1) values times a power of two per page and head."""
    x = rng.standard_normal((pages, heads, page, dim))
    e = np.round(rng.uniform(-spread, spread, (pages, heads))).astype(int)
    amax = np.abs(x).max((2, 3))
    ex = np.ceil(np.log2(amax / 448)).astype(int)
    codes = ref.e4m3_encode(x * np.exp2(-ex.astype(np.float64))[..., None, None])
    return codes, (ex + e + 127).astype(np.uint8)


def starts_of(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int64)


def cache_dev(codes, layout="hnd"):
    """A [pages, heads, slots, dim] view: contiguous, token-major ("nhd"), or
    with gaps between pages and slots ("gaps")."""
    t = torch.from_numpy(codes)
    if layout == "hnd":
        return t.to(DEV).view(torch.float8_e4m3fn)
    if layout == "nhd":
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    n, h, p, d = codes.shape
    big = torch.full((n, h, p + 1, d + 16), 0x7F, dtype=torch.uint8)
    big[:, :, :p, :d] = t
    return big.to(DEV)[:, :, :p, :d]


def host(t):
    t = t.view(torch.uint8) if t.dtype in (torch.float8_e4m3fn, torch.float8_e8m0fnu) else t
    return t.cpu().contiguous().numpy()


def call_over_freed_blocks(call, outputs, scratch=()):
    """What call(stream) makes on another stream, while work queued on the
    current stream still writes blocks of the same sizes that have been freed
    there. `outputs`: what the call returned when nothing was pending; `scratch`:
    bytes of other blocks that it makes."""
    freed = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in outputs]
    freed += [torch.empty(n, dtype=torch.uint8, device=DEV) for n in scratch]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # 0.1 s: a call takes a thousandth of it
    for t in freed:
        t.fill_(0x55)
    queued = torch.cuda.Event()
    queued.record()
    del freed, t
    got = call(stream)
    stream.synchronize()
    assert not queued.query()  # the writes come after the call's
    torch.cuda.synchronize()
    return got


__all__ = ["DEV", "DTYPES", "HALF_STEP", "cache_dev", "call_over_freed_blocks", "dev", "host", "make_table", "random_cache",
           "ref", "rows", "starts_of", "to_dev"]
