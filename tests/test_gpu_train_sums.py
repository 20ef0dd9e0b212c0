"""The balance loss's sums of probabilities, for every number of warps that a block has."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_router import balance64, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [40, 256, 264, 512, 520, 1000])
def test_sums_over_many_tokens(experts):
    """A warp adds up its tokens one by one, then come the block's warps (32, 16 above 256 experts, 8 above 512) and the
    blocks (one an SM): each addition rounds once."""
    tokens = 1 << 19
    l = logits_of(tokens, experts, 6, torch.bfloat16)
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda")
    b = fg.moe_balance_loss(l, offsets, 1.0)
    warps = 32 if experts <= 256 else 16 if experts <= 512 else 8
    blocks = torch.cuda.get_device_properties(0).multi_processor_count
    parts = [balance64(x, offsets, 1.0)[2] * x.shape[0] for x in l.split(1 << 16)]
    want = sum(parts) / tokens
    ref.within(b.probs, want, ((tokens // (blocks * warps) + 1 + warps + blocks) * 2.0 ** -24 + ref.REL) * want)
