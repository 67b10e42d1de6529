"""fp8_expert_layer called in ways that its own steps do not show."""
import numpy as np
import pytest
import torch

import __graft_entry__
import fp8_quantized_paged_store_gb300 as kvq
from tests._experts import DEV, codes, f32, u8, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build()


def layer(tokens, experts=8):
    rng = np.random.default_rng(tokens)
    gate_up, down = weights(rng, (experts, 512, 256)), weights(rng, (experts, 256, 256))
    logits = torch.from_numpy(rng.standard_normal((tokens, experts)).astype(np.float32))
    x, xs = codes(rng, (tokens, 256))
    return (u8(x), f32(xs)), logits, (u8(gate_up[0]), f32(gate_up[1] * 8), u8(down[0]), f32(down[1]), 3)


@pytest.mark.parametrize("tokens", [1, 40, 1000])
@pytest.mark.parametrize("given", [False, True])
def test_logits_in_host_memory(tokens, given):
    """The same bits as with logits on the device, whatever is done with page-locked memory
    behind the call; on the current stream and on a given one."""
    x, logits, rest = layer(tokens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = kvq.fp8_expert_layer(*x, logits.to(DEV), *rest, status=status)
    host = logits.pin_memory()
    torch.cuda.synchronize()
    got = kvq.fp8_expert_layer(*x, host, *rest, status=status, stream=torch.cuda.Stream() if given else None)
    for size in (tokens * 3, tokens * 3, tokens * 3, 9):
        torch.full((size,), -1, dtype=torch.int64).pin_memory()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and status.item() == 0


def test_no_tokens():
    x, logits, rest = layer(5)
    out = kvq.fp8_expert_layer(x[0][:0], x[1][:0], logits.to(DEV)[:0], *rest)
    assert out.shape == (0, 256)
    base = torch.zeros((0, 256), dtype=torch.float16, device=DEV)
    assert kvq.fp8_expert_layer(x[0][:0], x[1][:0], logits.to(DEV)[:0], *rest, base=base).dtype == torch.float16
