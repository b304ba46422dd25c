"""hs_mla_expanded_fwd where both CTAs of a pair write what the first one's products read (P through shared memory, zeros behind a
request's last row), many times over: what is not ordered shows as bits that change, or as values of rows that nobody sees."""
import math

import pytest
import torch

import latent_ops as plain
from test_gpu_latent import HEADS, attend, batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Dn,Dv", HEADS)
@pytest.mark.parametrize("q_lens,kv_lens,H", [([256, 200, 140, 256] * 3, [256, 201, 300, 513] * 3, 24), ([250, 255] * 10, [1100, 700] * 10, 8)])
def test_both_halves_again_and_again(q_lens, kv_lens, H, Dn, Dv):
    """After every other request lies one without tokens whose rows hold NaN: the tiles that end before it reach into it."""
    q = [m for i, x in enumerate(q_lens) for m in ((x, 0) if i % 2 else (x,))]
    b = batch(q, [n for i, x in enumerate(kv_lens) for n in ((x, 130) if i % 2 else (x,))], H, Dn, Dv, seed=21)
    assert sum(q) > 128 * len(q)  # pairs
    start = b["kv_start"].tolist()
    for r in range(2, len(q), 3):
        b["kv"][start[r]:start[r + 1]], b["rope"][start[r]:start[r + 1]] = math.nan, math.nan
    ref, tol, rlse, ltol = plain.attention(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], Dn, b["scale"])
    want = attend(b, Dv)
    assert plain.holds(want[0], ref, tol) and plain.holds(want[1], rlse, ltol)
    for _ in range(100):
        assert all(torch.equal(x, y) for x, y in zip(want, attend(b, Dv)))


@pytest.mark.parametrize("Dn,Dv", HEADS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 200, 0], [0, 0, 5]), ([300, 1, 40], [0, 700, 0]), ([7], [1])])
def test_requests_without_rows(q_lens, kv_lens, causal, Dn, Dv):
    """At either end of the rows and between others: zeros, and a log-sum-exp of minus infinity."""
    check(batch(q_lens, kv_lens, 2, Dn, Dv, seed=22), Dn, Dv, causal)
