"""GPU: the router on rows whose element offsets pass 31 bits, both kernels: equal, bit for bit, to the dense rows."""
import pytest
import torch

import fine_grained_block_amd as fgb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(64, 6), (300, 9)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_offsets_past_31_bits(dev, E, k, dtype):
    T, ld = 66001, 32771
    assert T * ld > 1 << 31
    logits = torch.randn((T, E), generator=torch.Generator(device=dev).manual_seed(E), device=dev).to(dtype)
    buf = torch.full((T, ld), 9.0, dtype=dtype, device=dev)
    view = buf[:, ld - E:]
    view.copy_(logits)
    ids, w = fgb.moe_route(view, k)
    want_ids, want_w = fgb.moe_route(logits, k)
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
    top = torch.sort(logits.float(), dim=-1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(ids.long(), top)
