"""pipeline.DenseSession with stretched positions: YaRN's factor is a temperature of the whole logit, latent part included."""
import math

import numpy as np
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,factor", [("plain", 1.0), ("linear", 8.0), ("yarn", 1.0), ("yarn", 8.0), ("yarn", 40.0)])
def test_stretched_positions(kind, factor):
    H, T = 16, 150
    session = DenseSession(1, H, 8, 8, max_tokens=T, kind=kind, factor=factor)
    session.extend([T])
    g = torch.Generator().manual_seed(5)
    q, latent, rope = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((T, H, 576), (T, 512), (T, 64)))
    inv = hs.hs_rope_inv_freq(64, kind=kind, factor=factor)[0]
    # queries and keys turned without a factor, and rounded as they are stored
    want_q = q.clone()
    want_q[..., 512:] = torch.from_numpy(plain.rotate(q[..., 512:], session.positions, inv, False)[0]).bfloat16().cuda()
    key = torch.from_numpy(plain.rotate(rope[:, None], session.positions, inv, False)[0]).bfloat16()[:, 0]
    out, lse = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
    session.attend(0, q, latent, rope, out, lse)
    assert hs.hs_check_flag(session.err) == 0
    pool, j = session.pool[0].clone(), torch.arange(T, device="cuda")
    pool[session.table[0].long()[j // 64] * 64 + j % 64, 528:] = key.contiguous().view(torch.uint8).view(T, 128).cuda()
    temperature = (0.1 * math.log(factor) + 1.0) ** 2 if kind == "yarn" else 1.0
    ref, rlse, _, _ = plain.paged_attention(want_q, pool, session.table, session.req_start, session.seq_len, temperature / 24.0)
    # a rotary value may round to either neighbour where the 32-bit rotation is next to the middle: rare, and 2^-8 of a
    # value whose share of a logit is a 576th
    assert float((out.double() - ref).norm() / ref.norm()) <= 6e-3
    assert float((lse.double() - rlse).abs().max()) <= 1e-2
