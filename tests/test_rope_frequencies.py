"""Rotary frequencies far past 1 radian per step: refused where their fraction of a turn is lost (no GPU), and
right up to there."""
import pytest
import torch

from long_context_exact_tma_b200 import api
from long_context_exact_tma_b200 import binding as B_

FAKE = 1 << 20  # 16-byte aligned, never dereferenced (validation fails first)


@pytest.mark.parametrize("value", [2.0 ** 40 * (1 + 2.0 ** -52), -(2.0 ** 41), 1e18, -1e300])
def test_frequencies_past_the_limit_are_refused(value):
    inv = torch.tensor([1.0, 0.5, value, 0.0], dtype=torch.float64)
    axis = torch.zeros(4, dtype=torch.int32)
    jobs = [(FAKE, 2 * FAKE, 2, (64, 32, 16), (64, 32, 16))]
    rc = B_.usp_rope_axes(jobs, 1, 2, 16, 8, B_.USP_BF16, FAKE, 64, 1, inv, axis, 0, 0, stream=0, check=False)
    assert rc == B_.USP_ERR_UNSUPPORTED and b"inv_freq[2]" in B_.lib().usp_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_frequencies(dtype, cuda):
    from test_gpu_rope import check
    R = 128
    sign = torch.where(torch.arange(R // 2) % 3 == 0, -1.0, 1.0).double()
    inv = sign * 2.0 ** torch.linspace(0, 40, R // 2, dtype=torch.float64)  # the last of them the limit itself
    axis = torch.zeros(R // 2, dtype=torch.int32)
    # steps whose products with the frequencies are exact in the 64-bit reference
    pos = torch.tensor([[[0, 1, -1, 2, -64, 1 << 40]]], device="cuda")
    x = torch.randn((1, pos.shape[2], 3, R), device="cuda").to(dtype)
    for inverse in (False, True):
        check(api.rope_axes(x, pos, inv, axis, inverse=inverse), x, pos, inv, axis, False, inverse)
