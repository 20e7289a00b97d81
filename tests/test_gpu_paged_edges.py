"""The paged cache's operators at the ends of their ranges."""
import numpy as np
import pytest
import torch

import long_context_decode_nuq_b200 as K
import paged_testlib as R

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("exp", [-64, -39, -38, -37, -10, -9, -8, 0, 38, 64])
def test_append_values_far_past_the_largest_scale(dtype, exp):
    """The type's extremes and infinities of both signs, beside values of every size: a value past
    6 * 448 * 2^exp is stored as that, with its own sign."""
    big = float(torch.finfo(DT[dtype]).max)
    x = torch.randn((64, 1, 128), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    sizes = torch.exp2(torch.linspace(-100, 127, 64) if dtype == "bf16" else torch.linspace(-14, 14, 64))
    x[:, 0, :32] = (x[:, 0, :32].float() * sizes[:, None]).clamp(-big, big).to(DT[dtype])
    for j, (a, b) in enumerate([(big, -big), (float("inf"), -float("inf")), (-float("inf"), -big), (big, float("nan")), (-big / 2, 1.0)]):
        x[j::5, 0, 32 + 16 * j], x[j::5, 0, 37 + 16 * j] = a, b
    x[::7, 0, 112:] = -big
    want = torch.tensor(R.quantize(x.double().numpy(), exp) * 2.0 ** -exp).to(DT[dtype])
    c = K.PagedCache(K.make_paged_cfg(1, 1, 128, 16, 4, 4, DT[dtype], exp, exp))
    x, slots = x.cuda(), i32(range(64))
    K.kvq_paged_append(c, x, x, slots)
    kh, vh = torch.empty_like(x), torch.empty_like(x)
    # read with exponent 0, code * scale: exact in both types
    K.kvq_paged_dequantize(K.PagedCache(K.make_paged_cfg(1, 1, 128, 16, 4, 4, DT[dtype]), pool=c.pool), slots, kh, vh)
    assert torch.equal(kh.cpu(), want) and torch.equal(vh.cpu(), want)
    assert K.kvq_paged_get_status(c) == 0
