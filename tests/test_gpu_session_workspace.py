"""pipeline.DenseSession's workspace: sized by the rows that are cached, not by the tables' width, and grown as a session needs it."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu


def steps(session, H, lens):
    """Prompts and a few tokens more of every slot, each step held against 64-bit attention over the session's own rows."""
    g = torch.Generator().manual_seed(9)
    for new in lens:
        T = session.extend(new)
        q, latent, rope = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((T, H, 576), (T, 512), (T, 64)))
        out, lse = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
        session.attend(0, q, latent, rope, out, lse)
        assert hs.hs_check_flag(session.err) == 0
        ref, rlse, spread, delta = plain.paged_attention(q, session.pool[0], session.table, session.req_start, session.seq_len,
                                                         session.softmax_scale)
        tol, ltol = plain.attention_bound(ref, spread, delta, rlse)
        assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse.double() - rlse).abs() <= ltol).all())


def test_wide_tables_over_a_small_pool():
    """256 slots that may grow to a million tokens each, of which few are cached: room for every slot's longest would be 309 GB."""
    session = DenseSession(256, 64, 16, 16384)
    assert session.workspace.numel() < 1 << 28
    steps(session, 64, [[130, 0, 70] + [0] * 253, [1, 0, 1] + [0] * 253])
    assert session.workspace.numel() < 1 << 28


@pytest.mark.parametrize("max_tokens", [1, 4096])
def test_steps_beyond_what_it_was_made_for(max_tokens):
    """Prompts long enough for the variant that dequantises every row first; steps of more tokens than were announced."""
    session = DenseSession(2, 16, 40, 30, max_tokens=max_tokens)
    steps(session, 16, [[200, 150], [1, 1], [300, 120]])


def test_a_refused_step_leaves_the_session_as_it_was():
    session = DenseSession(2, 16, 4, 4, max_tokens=64)
    session.extend([100, 20])
    before = session.table.clone(), session.seq_len.clone(), session.refcount.clone(), session.kv_tokens
    with pytest.raises(RuntimeError):
        session.extend([100, 200])
    assert all(torch.equal(a, b) for a, b in zip(before, (session.table, session.seq_len, session.refcount)))
    assert session.kv_tokens == before[3] == 120
