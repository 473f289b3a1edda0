"""The window and rotary calls of the api go through the binding's functions of the same names, those whose
refusals test_window_host.py checks: one order of arguments, not two."""
import pytest
import torch

from long_context_exact_tma_b200 import api
from long_context_exact_tma_b200 import binding as B_

pytestmark = pytest.mark.gpu


def test_the_api_calls_what_the_refusals_are_tested_on(cuda, monkeypatch):
    calls = []

    def counted(name, fn):
        return lambda *a, **kw: (calls.append(name), fn(*a, **kw))[1]

    names = ["usp_window_attn_fwd", "usp_window_attn_bwd", "usp_window_attn_decode", "usp_rope_axes"]
    for n in names:
        monkeypatch.setattr(B_, n, counted(n, getattr(B_, n)))
    q = torch.randn((1, 40, 2, 64), device="cuda").to(torch.bfloat16)
    out, lse = api.window_attn_fwd(q, q, q, 8, 1)
    api.window_attn_bwd(q, q, q, out, lse, q, 8, 1)
    api.window_attn_decode(q[:, -1:].contiguous(), q, q, torch.tensor([40], dtype=torch.int32, device="cuda"), 8, 1)
    api.rope_axes(q, torch.arange(40, device="cuda").view(1, 1, 40), torch.ones(4, dtype=torch.float64),
                  torch.zeros(4, dtype=torch.int32))
    assert calls == names
