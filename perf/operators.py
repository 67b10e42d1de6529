"""Measured cases of the operators on a paged key-value cache held in 8 bits, and of the norm ahead of them.

Three operators, as a decoder layer with grouped heads uses them one after the other:

  norm       the residual's addition, RMSNorm with a weight, and an E4M3 output with one scale for each token or
             each 128 values (the input of an 8-bit projection)
  append     rotation of queries and keys by position, then keys and values into pages of E4M3 codes with one
             power-of-two scale (E8M0) for each page and head; a partly filled page whose scale has to grow is rescaled
  attention  softmax attention of new tokens over those pages: single tokens (decode), short runs, whole prompts

A page is the block of tokens that shares a scale. Sequences are ragged; their lengths come from the case alone,
their values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the residual stream of a small decode batch: latency
        dict(name="norm_decode", op="norm", tokens=8, hidden=4096, group=0, dtype="bf16", residual=True),
        # one prefill step of a large model, a scale for each 128 values, as block-scaled products take them
        dict(name="norm_prefill_groups", op="norm", tokens=8192, hidden=7168, group=128, dtype="bf16", residual=True),
        # an odd count of tokens, one scale for each token, no residual (a layer's first norm)
        dict(name="norm_odd", op="norm", tokens=5003, hidden=5120, group=0, dtype="fp16", residual=False),
        # one new token of each running request: latency
        dict(name="append_decode", op="append", seqs=64, new_min=1, new=1, ctx=8000, heads=32, kv_heads=8, dim=128,
             page=64, rotary=128, interleaved=True, dtype="bf16", lens=1),
        # a prefill step of ragged chunks that start inside pages
        dict(name="append_chunks", op="append", seqs=7, new_min=300, new=2048, ctx=5000, heads=32, kv_heads=8, dim=128,
             page=64, rotary=128, interleaved=False, dtype="bf16", lens=2),
        # whole prompts of a throughput run, small heads, small pages, half of each head rotated
        dict(name="append_prompts", op="append", seqs=24, new_min=700, new=4096, ctx=0, heads=32, kv_heads=8, dim=64,
             page=16, rotary=32, interleaved=False, dtype="fp16", lens=3),
        # a few short conversations, one token each: latency
        dict(name="attn_decode_small", op="attention", seqs=3, new_min=1, new=1, ctx_min=300, ctx=1200, heads=32,
             kv_heads=8, dim=128, page=64, causal=True, window=0, dtype="bf16", lens=4),
        # an ordinary decode batch with ragged contexts
        dict(name="attn_decode_batch", op="attention", seqs=64, new_min=1, new=1, ctx_min=500, ctx=16000, heads=32,
             kv_heads=8, dim=128, page=64, causal=True, window=0, dtype="bf16", lens=5),
        # few long documents, 16 query heads to a key head, two tokens at a time (a drafted one checked)
        dict(name="attn_verify_long", op="attention", seqs=4, new_min=2, new=2, ctx_min=60000, ctx=131000, heads=64,
             kv_heads=8, dim=128, page=128, causal=True, window=0, dtype="bf16", lens=6),
        # small heads and pages, a sliding window, several drafted tokens of one batch
        dict(name="attn_window", op="attention", seqs=33, new_min=1, new=4, ctx_min=100, ctx=20000, heads=16,
             kv_heads=4, dim=64, page=16, causal=True, window=4096, dtype="fp16", lens=7),
        # one whole prompt
        dict(name="attn_prompt", op="attention", seqs=1, new_min=8192, new=8192, ctx_min=0, ctx=0, heads=32,
             kv_heads=8, dim=128, page=64, causal=True, window=0, dtype="bf16", lens=8),
        # chunks of prompts behind contexts of several lengths, some single tokens among them
        dict(name="attn_chunks", op="attention", seqs=6, new_min=1, new=1024, ctx_min=0, ctx=12000, heads=32,
             kv_heads=8, dim=128, page=32, causal=True, window=0, dtype="bf16", lens=9),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "norm":
        group = rng.choice([0, 128])
        hidden = 128 * _log(rng, 4, 64) if group else 8 * _log(rng, 32, 1024)
        return dict(op=op, tokens=min(_log(rng, 1, 9000), 58_000_000 // hidden), hidden=hidden, group=group, dtype=dtype,
                    residual=rng.random() < 0.7)
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 5, 8, 16] if kv_heads < 8 else [1, 4, 8])
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, lens=rng.randrange(1 << 30))
    if op == "append":
        c["seqs"] = _log(rng, 1, 100)
        c["new"] = _log(rng, 1, max(2, 40_000 // c["seqs"]))
        c["new_min"] = max(1, min(c["new"], _log(rng, 1, c["new"])))
        c["ctx"] = _log(rng, 1, 6000) - 1
        c["rotary"] = rng.choice([dim, dim, dim // 2])
        c["interleaved"] = rng.random() < 0.5
        return c
    c["causal"] = rng.random() < 0.85
    c["window"] = rng.choice([0, 0, 0, _log(rng, 64, 8192)])
    if rng.random() < 0.6:  # decode, and short runs of drafted tokens
        c["seqs"] = _log(rng, 1, 100)
        c["new"] = rng.choice([1, 1, 1, 2, 4])
        c["new_min"] = 1
        c["ctx"] = _log(rng, 16, 600_000 // c["seqs"])
    else:
        c["seqs"] = _log(rng, 1, 6)
        c["new"] = _log(rng, 16, 1500)
        c["new_min"] = max(1, c["new"] // rng.choice([1, 3, 50]))
        c["ctx"] = _log(rng, 1, 9000) - 1
    c["ctx_min"] = min(c["ctx"], rng.choice([0, c["ctx"] // 4, c["ctx"]]))
    return c


def _lengths(case):
    """(new tokens, tokens that are in the cache before) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    news = [r.randint(case["new_min"], case["new"]) for _ in range(case["seqs"])]
    news[-1] = case["new"]
    low = case.get("ctx_min", 0)
    ctxs = [r.randint(low, case["ctx"]) for _ in range(case["seqs"])]
    ctxs[0] = case["ctx"]
    return news, ctxs


def _visible(case):
    """For attention: query-key pairs in all, and for each sequence the keys that some query sees."""
    news, ctxs = _lengths(case)
    pairs, keys = 0, []
    for n, c in zip(news, ctxs):
        total = n + c
        w = case["window"] or total
        at = np.arange(c, total, dtype=np.int64)
        high = at + 1 if case["causal"] else np.full_like(at, total)
        low = np.maximum(0, at + 1 - w)
        pairs += int((high - low).sum())
        keys.append(int(high.max() - low.min()))
    return pairs, keys


def work(case):
    """Each input read once, each output written once."""
    if case["op"] == "norm":
        n = case["tokens"] * case["hidden"]
        scales = case["tokens"] * (case["hidden"] // case["group"] if case["group"] else 1)
        return {"bytes": n * (7 if case["residual"] else 3) + 2 * case["hidden"] + 4 * scales, "flops": 6 * n}
    news, ctxs = _lengths(case)
    t, d = sum(news), case["dim"]
    if case["op"] == "append":
        pages = sum((c + n - 1) // case["page"] - c // case["page"] + 1 for n, c in zip(news, ctxs))
        row = case["heads"] * d * 4 + case["kv_heads"] * d * 2 * 3  # queries in and out; keys, values in and their codes out
        return {"bytes": t * (row + 4 * case["rotary"]) + pages * (2 * case["kv_heads"] + 8) + 16 * case["seqs"],
                "flops": t * (case["heads"] + case["kv_heads"]) * case["rotary"] * 3}
    pairs, keys = _visible(case)
    cache = sum(keys) * case["kv_heads"] * d * 2
    pages = sum(-(-k // case["page"]) for k in keys)
    return {"bytes": cache + pages * (2 * case["kv_heads"] + 8) + t * case["heads"] * (4 * d + 4) + 16 * case["seqs"],
            "flops": 4 * d * case["heads"] * pairs}


# ----------------------------------------------------------------- inputs ---

class State:
    pass


def _pages(g, pages, case, dev):
    """A cache of codes with their scales, as tokens appended before have left it: heads and pages of several sizes."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp2(torch.rand((pages, case["kv_heads"], 1, 1), generator=g, device=dev) * 2 - 1)
    amax = x.abs().amax((2, 3)).clamp_min_(1e-4)
    m, e = torch.frexp(amax * torch.tensor(1 / 448, dtype=torch.float32, device=dev))
    e = e - (m == 0.5).int()
    x *= torch.exp2(-e.float())[:, :, None, None]
    codes = x.clamp_(-448, 448).to(E4M3)
    return codes, (e + 127).to(torch.uint8).view(E8M0)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = State()
    s.case, s.dev = case, dev
    if case["op"] == "norm":
        t, h = case["tokens"], case["hidden"]
        s.x = torch.randn((t, h), generator=g, device=dev).to(dt)
        s.residual = (torch.randn((t, h), generator=g, device=dev) * 4).to(dt) if case["residual"] else None
        s.x[:, h // 3] *= 24  # a channel that stands out, as residual streams have
        s.weight = (torch.rand(h, generator=g, device=dev) + 0.5).to(dt)
        s.eps = 1e-6
        s.residual_out = torch.empty((t, h), dtype=dt, device=dev) if case["residual"] else None
        s.out = torch.empty((t, h), dtype=E4M3, device=dev)
        s.scales = torch.empty((t, h // case["group"] if case["group"] else 1), dtype=torch.float32, device=dev)
        return s
    news, ctxs = _lengths(case)
    t, hq, hk, d, p = sum(news), case["heads"], case["kv_heads"], case["dim"], case["page"]
    totals = [n + c for n, c in zip(news, ctxs)]
    need = [-(-x // p) for x in totals]
    width = max(need) + 2
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev)
    table = np.full((case["seqs"], width), -1, np.int64)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = np.arange(at, at + k)
        at += k
    table = torch.from_numpy(table).to(dev)
    s.block_table = torch.where(table >= 0, order[table.clamp_min(0)], table)
    s.query_start_loc = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int64, device=dev)
    s.context_lens = torch.tensor(ctxs, dtype=torch.int64, device=dev)
    s.seq_lens = torch.tensor(totals, dtype=torch.int64, device=dev)
    s.max_new, s.max_len = max(news), max(totals)
    # queries, keys and values as one projection leaves them: slices of [tokens, all heads * dim]
    qkv = torch.randn((t, (hq + 2 * hk) * d), generator=g, device=dev).to(dt)
    s.q = qkv[:, :hq * d].view(t, hq, d)
    s.k_cache, s.k_scales = _pages(g, pages, case, dev)
    s.v_cache, s.v_scales = _pages(g, pages, case, dev)
    if case["op"] == "append":
        s.k = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s.v = qkv[:, (hq + hk) * d:].view(t, hk, d)
        r = case["rotary"]
        freq = 10000.0 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
        angle = torch.arange(s.max_len, device=dev, dtype=torch.float64)[:, None] * freq
        s.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        s.q_out = torch.empty((t, hq, d), dtype=dt, device=dev)
        return s
    s.q = s.q.contiguous()
    s.sm_scale = 1 / math.sqrt(d)
    s.out = torch.empty_like(s.q)
    s.lse = torch.empty((t, hq), dtype=torch.float32, device=dev)
    s.status = torch.zeros(1, dtype=torch.int32, device=dev)
    s.workspace = torch.empty(64 << 20, dtype=torch.uint8, device=dev)  # one for all layers and steps of a program
    return s


# ------------------------------------------------------------ plain forms ---

def _plain_norm(s):
    h = s.x.float()
    if s.residual is not None:
        h = h + s.residual.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s.eps) * s.weight.float()
    t, n = y.shape
    grouped = y.view(t, -1, s.case["group"] or n)
    scales = grouped.abs().amax(2, keepdim=True).clamp_min(1e-4) / 448
    out = (grouped / scales).clamp(-448, 448).to(E4M3).view(t, n)
    return out, scales.squeeze(2), h.to(s.x.dtype) if s.residual is not None else None


def _rotated(x, cos, sin, case):
    r = case["rotary"]
    x = x.float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_store(x, cache, scales, page, slot, first_page, kept):
    """Values [tokens, heads, dim] into their pages. `first_page`, `kept`: each sequence's first page, and how many of its
    slots hold earlier tokens."""
    codes, bytes_ = cache.view(torch.uint8), scales.view(torch.uint8)
    pages, heads = bytes_.shape
    amax = torch.zeros((pages, heads), device=x.device).index_reduce_(0, page, x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax.clamp_min(1e-4) * torch.tensor(1 / 448, dtype=torch.float32, device=x.device))
    e = e - (m == 0.5).int()
    before = bytes_.int() - 127
    has = torch.zeros(pages, dtype=torch.bool, device=x.device)
    has[first_page] = kept > 0
    touched = torch.zeros(pages, dtype=torch.bool, device=x.device)
    touched[page] = True
    e = torch.where(has[:, None], torch.maximum(e, before), e)
    e = torch.where(touched[:, None], e, before)
    # the earlier tokens of a first page, on the new scale
    mine = codes[first_page]
    moved = mine.view(E4M3).float() * torch.exp2((before - e)[first_page].float())[:, :, None, None]
    early = torch.arange(mine.shape[2], device=x.device)[None, :] < kept[:, None]
    codes[first_page] = torch.where(early[:, None, :, None], moved.to(E4M3).view(torch.uint8), mine)
    new = (x * torch.exp2(-e[page].float())[:, :, None]).clamp(-448, 448).to(E4M3)
    codes[page, :, slot] = new.view(torch.uint8)
    bytes_.copy_((e + 127).to(torch.uint8))


def _plain_append(s):
    case = s.case
    t, p = s.q.shape[0], case["page"]
    token = torch.arange(t, device=s.dev)
    seq = torch.searchsorted(s.query_start_loc[1:], token, right=True)
    position = s.context_lens[seq] + token - s.query_start_loc[seq]
    page, slot = s.block_table[seq, position // p], position % p
    half = case["rotary"] // 2
    cos, sin = s.cos_sin[position, :half], s.cos_sin[position, half:2 * half]
    first, kept = s.block_table.gather(1, (s.context_lens // p)[:, None])[:, 0], s.context_lens % p
    _plain_store(_rotated(s.k, cos, sin, case), s.k_cache, s.k_scales, page, slot, first, kept)
    _plain_store(s.v.float(), s.v_cache, s.v_scales, page, slot, first, kept)
    s.q_out.copy_(_rotated(s.q, cos, sin, case))
    return s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.q_out


def _plain_values(cache, scales, table):
    """[seqs, heads, tokens, dim] of the pages that `table` names."""
    b, w = table.shape
    _, h, p, d = cache.shape
    x = cache.view(torch.uint8)[table].view(E4M3).float()
    x *= torch.exp2(scales.view(torch.uint8)[table].float() - 127)[..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, w * p, d)


def _plain_attention(s):
    case = s.case
    t, hq, d = s.q.shape
    hk, p = case["kv_heads"], case["page"]
    b, n = case["seqs"], s.max_new
    table = s.block_table[:, :-(-s.max_len // p)].clamp_min(0)
    k, v = _plain_values(s.k_cache, s.k_scales, table), _plain_values(s.v_cache, s.v_scales, table)
    token = torch.arange(t, device=s.dev)
    seq = torch.searchsorted(s.query_start_loc[1:], token, right=True)
    i = token - s.query_start_loc[seq]
    q = torch.zeros((b, n, hq, d), device=s.dev)
    q[seq, i] = s.q.float()
    q = q.view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(s.sm_scale).view(b, hk, hq // hk, n, -1)
    key = torch.arange(k.shape[2], device=s.dev)
    at = (s.context_lens[:, None] + torch.arange(n, device=s.dev))[:, :, None]
    hidden = key >= s.seq_lens[:, None, None]
    if case["causal"]:
        hidden = hidden | (key > at)
    if case["window"]:
        hidden = hidden | (key <= at - case["window"])
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(b, hk, -1, k.shape[2]), v).view(b, hk, hq // hk, n, d) / total.clamp_min(1e-38)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[seq, i]
    return out.to(s.q.dtype), lse.permute(0, 3, 1, 2).reshape(b, n, hq)[seq, i]


def run(s):
    op = s.case["op"]
    if own:
        import fp8_quantized_paged_store_gb300 as kvq
        if op == "norm":
            return kvq.add_rmsnorm_fp8(s.x, s.weight, s.eps, residual=s.residual, group=s.case["group"], out=s.out,
                                       scales=s.scales, residual_out=s.residual_out)
        if op == "append":
            kvq.rope_fp8_kv_append(s.k, s.v, s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.block_table, s.context_lens,
                                   s.query_start_loc, cos_sin=s.cos_sin, rotary_dim=s.case["rotary"],
                                   interleaved=s.case["interleaved"], q=s.q, q_out=s.q_out)
            return s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.q_out
        return kvq.fp8_paged_attention(s.q, s.k_cache, s.v_cache, s.k_scales, s.v_scales, s.block_table, s.seq_lens,
                                       s.query_start_loc, s.max_new, s.sm_scale, causal=s.case["causal"],
                                       window=s.case["window"], out=s.out, lse=s.lse, status=s.status,
                                       workspace=s.workspace)
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[op](s)


# ------------------------------------------------------ 64-bit definitions ---

def _to_e4m3(x):
    """Doubles rounded to the nearest E4M3 value, ties to even, saturating."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _decoded(scales):
    return torch.exp2(scales.view(torch.uint8).double() - 127)


def _exact_norm(s):
    h = s.x.double() + (s.residual.double() if s.residual is not None else 0)
    root = torch.sqrt(h.square().sum(1) / h.shape[1] + s.eps)
    y = h / root[:, None] * s.weight.double()
    g = s.case["group"] or y.shape[1]
    out, scales = torch.empty_like(y), []
    for at in range(0, y.shape[1], g):
        part = y[:, at:at + g]
        scale = part.abs().amax(1).clamp_min(1e-4) / 448
        out[:, at:at + g] = _to_e4m3(part / scale[:, None])
        scales.append(scale)
    return out, torch.stack(scales, 1), h if s.residual is not None else None


def _exact_turn(x, angles, case):
    half = case["rotary"] // 2
    c, sn = angles[:, None, :half], angles[:, None, half:]
    y = x.clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
    y[..., one] = x[..., one] * c - x[..., two] * sn
    y[..., two] = x[..., two] * c + x[..., one] * sn
    return y


def _exact_append(s):
    case, p = s.case, s.case["page"]
    news, ctxs = _lengths(case)
    caches = [s.k_cache.double(), s.v_cache.double()]
    scales = [_decoded(s.k_scales), _decoded(s.v_scales)]
    q_out = torch.empty(s.q.shape, dtype=torch.float64, device=s.dev)
    table, at = s.block_table.tolist(), 0
    for b, (n, c) in enumerate(zip(news, ctxs)):
        angles = s.cos_sin[c:c + n].double()
        q_out[at:at + n] = _exact_turn(s.q[at:at + n].double(), angles, case)
        rows = [_exact_turn(s.k[at:at + n].double(), angles, case), s.v[at:at + n].double()]
        at += n
        done = 0
        while done < n:
            column, old = divmod(c + done, p)
            take = min(p - old, n - done)
            page = table[b][column]
            for x, cache, scale in zip(rows, caches, scales):
                part = x[done:done + take].transpose(0, 1)  # heads, tokens, dim
                want = torch.exp2(torch.ceil(torch.log2(part.abs().amax((1, 2)).clamp_min(1e-4) / 448)))
                if old:
                    want = torch.maximum(want, scale[page])
                    cache[page, :, :old] = _to_e4m3(cache[page, :, :old] * (scale[page] / want)[:, None, None])
                scale[page] = want
                cache[page, :, old:old + take] = _to_e4m3(part / want[:, None, None])
            done += take
    return caches[0], caches[1], scales[0], scales[1], q_out


def _exact_attention(s):
    case, p = s.case, s.case["page"]
    news, ctxs = _lengths(case)
    hk, ratio = case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s.q.shape, dtype=torch.float64, device=s.dev)
    lse = torch.zeros(s.q.shape[:2], dtype=torch.float64, device=s.dev)
    start = 0
    for b, (n, c) in enumerate(zip(news, ctxs)):
        total = n + c
        pages = s.block_table[b, :-(-total // p)]
        for h in range(hk):
            k = (s.k_cache.view(torch.uint8)[pages, h].view(E4M3).double() * _decoded(s.k_scales)[pages, h, None, None]).flatten(0, 1)[:total]
            v = (s.v_cache.view(torch.uint8)[pages, h].view(E4M3).double() * _decoded(s.v_scales)[pages, h, None, None]).flatten(0, 1)[:total]
            for at in range(0, n, 2048):
                m = min(2048, n - at)
                rows = slice(start + at, start + at + m)
                heads = slice(h * ratio, (h + 1) * ratio)
                z = torch.einsum("mgd,kd->mgk", s.q[rows, heads].double(), k) * s.sm_scale
                where = torch.arange(c + at, c + at + m, device=s.dev)[:, None]
                key = torch.arange(total, device=s.dev)[None]
                seen = torch.ones((m, total), dtype=torch.bool, device=s.dev)
                if case["causal"]:
                    seen &= key <= where
                if case["window"]:
                    seen &= key > where - case["window"]
                z = torch.where(seen[:, None], z, -math.inf)
                l = torch.logsumexp(z, -1)
                lse[rows, heads] = l
                out[rows, heads] = torch.einsum("mgk,kd->mgd", torch.exp(z - l[..., None]), v)
        start += n
    return out, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "attention" and work(case)["flops"] > 6e12:
        return None
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](s)
