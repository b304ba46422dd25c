"""pipeline.DenseSession: rotary positions, cache rows, dense attention, forks, frees and compaction as a serving loop uses
them. The same requests without any sharing give the rows and the 64-bit attention that the session is held against."""
import numpy as np
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu
H, L = 16, 2


class Source:
    """The layers' queries, latent rows and rotary keys of (branch, position): the same values wherever they are asked for."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g).bfloat16()
        self.q, self.latent, self.rope = r(L, 8, 700, H, 576), r(L, 8, 700, 512), r(L, 8, 700, 64)

    def take(self, layer, of):
        """``of``: (branch, position) of each token."""
        b, p = (torch.tensor(x) for x in zip(*of))
        return tuple(t[layer, b, p].cuda() for t in (self.q, self.latent, self.rope))


def step(session, source, new, of):
    T = session.extend(new)
    assert T == len(of)
    outs = []
    for layer in range(L):
        q, latent, rope = source.take(layer, of)
        raw_q, raw_rope = q.clone(), rope.clone()
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((T, H), device="cuda")
        session.attend(layer, q, latent, rope, out, lse)
        pos, inv = session.positions.cpu(), session.inv_freq.cpu()
        for got, x in ((q[..., 512:].cpu(), raw_q[..., 512:].cpu()), (rope[:, None].cpu(), raw_rope[:, None].cpu())):
            ref, size = plain.rotate(x, pos, inv, False, session.rope_scale)
            # rounded once to bf16; fp32 factors, products and their sum are off by 2^-20 of the pair's size
            assert (np.abs(got.double().numpy() - ref) <= np.abs(ref) * 2.0 ** -8 + size * 2.0 ** -20).all()
        outs.append((q, out, lse))
    return outs


def attention_holds(outs, session, rows):
    """``outs`` against float64 attention over ``rows`` (a session that shares nothing), whose slots hold the same tokens."""
    for layer, (q, out, lse) in enumerate(outs):
        ref, rlse, spread, delta = plain.paged_attention(q, rows.pool[layer], rows.table, rows.req_start, rows.seq_len,
                                                         rows.softmax_scale)
        tol, ltol = plain.attention_bound(ref, spread, delta, rlse)
        assert bool(((out.double() - ref).abs() <= tol).all())
        assert bool(((lse.double() - rlse).abs() <= ltol).all())
        assert float((out.double() - ref).norm() / ref.norm()) <= 5e-3
    assert hs.hs_check_flag(session.err) == 0


def same_rows(a, b):
    for r in range(a.B):
        n = int(a.seq_len[r])
        assert n == int(b.seq_len[r])
        j = torch.arange(n, device="cuda")
        at = lambda s: s.table[r].long()[j // 64] * 64 + j % 64
        for layer in range(L):
            assert torch.equal(a.pool[layer][at(a)], b.pool[layer][at(b)])


def test_branches_share_their_prompt():
    source = Source(1)
    shared, alone = (DenseSession(5, H, nblk, 12, L=L, max_tokens=800) for nblk in (40, 60))
    # slots 0 and 1 have prompts of 200 and 333 tokens; slots 2, 3 will branch from 0, slot 4 from 1
    prompt = {0: (0, 200), 1: (1, 333)}
    tokens = lambda slots: [(prompt[s][0], j) for s in slots for j in range(prompt[s][1])]
    outs = step(shared, source, [200, 333, 0, 0, 0], tokens([0, 1]))
    for s, of in ((2, 0), (3, 0), (4, 1)):
        prompt[s] = prompt[of]
    whole = step(alone, source, [200, 333, 200, 200, 333], tokens(range(5)))
    first = alone.req_start
    alone.req_start, table, lens = first[:3], alone.table, alone.seq_len  # the first two slots alone
    alone.table, alone.seq_len = table[:2], lens[:2]
    attention_holds(outs, shared, alone)
    alone.req_start, alone.table, alone.seq_len = first, table, lens
    attention_holds(whole, alone, alone)
    shared.fork([0, 0, 1], [2, 3, 4])
    assert int((shared.refcount > 1).sum()) == 200 // 64 + 333 // 64  # complete pages only
    same_rows(shared, alone)
    # every branch goes on with tokens of its own, one and four at a time
    at = [200, 333, 200, 200, 333]
    for m in (1, 1, 4, 60):
        of = [(3 + s, at[s] + i) for s in range(5) for i in range(m)]
        outs = step(shared, source, [m] * 5, of)
        step(alone, source, [m] * 5, of)
        attention_holds(outs, shared, alone)
        same_rows(shared, alone)
        at = [a + m for a in at]
    # two branches end; their pages are given back and the rest moves to the front
    for s in (shared, alone):
        s.free([0, 3])
    shared.compact()
    used = int(shared.counts[0])
    assert used == int((shared.refcount > 0).sum()) and bool((shared.refcount[:used] > 0).all())
    same_rows(shared, alone)
    of = [(3 + s, at[s]) for s in (1, 2, 4)]
    outs = step(shared, source, [0, 1, 1, 0, 1], of)
    step(alone, source, [0, 1, 1, 0, 1], of)
    attention_holds(outs, shared, alone)
    same_rows(shared, alone)


def test_a_cache_without_pages_refuses():
    session = DenseSession(2, H, 4, 4, L=1, max_tokens=64)
    session.extend([128, 100])
    with pytest.raises(RuntimeError):
        session.extend([1, 0])
    session.fork([1], [0])  # slot 1's tail needs a page of its own
    assert hs.hs_check_flag(session.err) == hs.FLAGS["NO_PAGES"]
