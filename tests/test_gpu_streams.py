"""Outputs, scratch and status words that the latent cache's read path makes
inside a call with stream=: none of them takes a block that work queued on the
current stream still writes, and a call without a status word ends behind its
kernels."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._fp8 import DEV, call_over_freed_blocks

pytestmark = pytest.mark.gpu

SLOTS = 4096


@pytest.fixture(scope="module")
def cache():
    __graft_entry__.build()
    g = torch.Generator(device=DEV).manual_seed(0)
    latent = torch.randn((SLOTS, 512), generator=g, device=DEV).bfloat16()
    cache = torch.zeros((SLOTS, 272), dtype=torch.uint8, device=DEV)
    kvq.mxfp4_mla_store(latent, torch.arange(SLOTS, device=DEV), cache)
    return cache


def queries(n, topk):
    g = torch.Generator(device=DEV).manual_seed(n)
    q = torch.randn((n, 16, 512), generator=g, device=DEV).bfloat16()
    idx = torch.from_numpy(np.random.default_rng(n).integers(0, SLOTS, (n, topk))).to(DEV)
    return q, idx


def test_gather(cache):
    idx = queries(3, 100)[1]
    want = kvq.mxfp4_mla_gather_dequant(cache, idx)
    got = call_over_freed_blocks(lambda s: kvq.mxfp4_mla_gather_dequant(cache, idx, stream=s), [want])
    assert torch.equal(got, want)


@pytest.mark.parametrize("workspace", [True, False])
def test_attention(cache, workspace):
    q, idx = queries(4, 2048)
    want, _ = kvq.mxfp4_mla_sparse_attention(q, cache, idx, 0.05, workspace=workspace)
    size = kvq.attention_workspace_size(4, 16, 2048) if workspace else 4
    assert size > 0
    got, _ = call_over_freed_blocks(
        lambda s: kvq.mxfp4_mla_sparse_attention(q, cache, idx, 0.05, workspace=workspace, stream=s),
        [want], (size, 4))
    assert torch.equal(got, want)


def test_ragged_attention(cache):
    q, idx = queries(3, 200)
    offsets = torch.tensor([0, 200, 250, 600], device=DEV)
    want, _ = kvq.mxfp4_mla_sparse_attention_ragged(q, cache, idx.view(-1), offsets, 0.05)
    got, _ = call_over_freed_blocks(
        lambda s: kvq.mxfp4_mla_sparse_attention_ragged(q, cache, idx.view(-1), offsets, 0.05,
                                                        stream=s), [want], (4,))
    assert torch.equal(got, want)


def test_calls_without_status_end_behind_their_kernels(cache):
    q, idx = queries(4, 2048)
    offsets = torch.tensor([0, 2048, 4000, 4100, 8192], device=DEV)
    torch.cuda.synchronize()
    for s in (torch.cuda.default_stream(), torch.cuda.Stream()):
        for stream in (s, s.cuda_stream):
            for call in (lambda: kvq.mxfp4_mla_sparse_attention(q, cache, idx, 0.05, stream=stream),
                         lambda: kvq.mxfp4_mla_sparse_attention_ragged(
                             q, cache, idx.view(-1), offsets, 0.05, stream=stream)):
                with torch.cuda.stream(s):
                    torch.cuda._sleep(50_000_000)
                call()
                assert s.query()
