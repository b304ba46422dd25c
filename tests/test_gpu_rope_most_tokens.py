"""hs_rope at the largest number of tokens that its argument holds."""
import math

import pytest
import torch

import dsa_sparse_mla_gb300 as hs

pytestmark = pytest.mark.gpu


def test_most_tokens():
    T, f = 2 ** 31 - 1, 0.3
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    x = torch.zeros((T, 1, 2), dtype=torch.bfloat16, device="cuda")
    x[..., 0] = 1.0
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    hs.hs_rope(x, pos, torch.tensor([f], dtype=torch.float64, device="cuda"))
    at = torch.tensor([0, 1, 7, 8, 12345, 2 ** 30 + 1, 2 ** 31 - 10, T - 8, T - 2, T - 1])
    got = x[at.cuda(), 0].double().cpu()
    want = torch.stack([torch.tensor([math.cos(float(p) * f), math.sin(float(p) * f)], dtype=torch.float64) for p in at])
    # bf16 rounding, fp32 arithmetic, and the angle: 2^31 of the frequency's 2^-53, in turns, on either side
    assert float((got - want).abs().max()) <= 2.0 ** -9 + 2.0 ** -20
