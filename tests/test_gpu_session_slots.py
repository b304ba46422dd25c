"""DenseSession.attend_heads where few of the session's slots have tokens: the expanded form is that of a session of those slots alone."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
import test_gpu_session_heads
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu


def steps(slots, at, H, Dn, Dv, w, graph=False):
    """A prompt for each of the slots ``at``, then more tokens for some of them: outputs, lse and units (the plan's first value) of every step."""
    s, g, got = DenseSession(slots, H, 200, 70, max_tokens=64), torch.Generator().manual_seed(60), []
    for new in ([700, 1, 300], [0, 1, 0], [0, 513, 2], [1, 2, 3], [150, 0, 0]):
        all_new = [0] * slots
        for r, m in zip(at, new):
            all_new[r] = m
        T = s.extend(all_new)
        x = [plain.rand(size, g).cuda() for size in ((T, H, Dn + 64), (T, 512), (T, 64))]
        out, lse = torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda")
        if graph:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                s.attend_heads(0, *x, w, out, lse, form="expanded")
            captured.replay()
        else:
            s.attend_heads(0, *x, w, out, lse, form="expanded")
        assert hs.hs_check_flag(s.err) == 0
        got.append((out, lse, s._kept["expanded"][:4].view(torch.int32).clone()))
    return got


@pytest.mark.parametrize("Dn,Dv", [(128, 128), (192, 256)])
def test_slots_without_tokens_change_nothing(Dn, Dv):
    w = plain.weights(3, Dn, Dv, torch.Generator().manual_seed(61)).cuda()
    want = steps(3, (0, 1, 2), 3, Dn, Dv, w)
    for slots, at in ((4, (0, 1, 2)), (64, (0, 17, 63)), (9, (3, 4, 8))):
        for graph in (False, True):
            for a, b in zip(want, steps(slots, at, 3, Dn, Dv, w, graph)):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_prompt_in_one_of_many_slots():
    """It is cut as in a session of its own (256 tokens to a block)."""
    H, T, units = 4, 2048, []
    w = plain.weights(H, 128, 128, torch.Generator().manual_seed(62)).cuda()
    for slots in (1, 64):
        g, s = torch.Generator().manual_seed(63), DenseSession(slots, H, 40, 40, max_tokens=T)
        s.extend([0] * (slots - 1) + [T])
        s.attend_heads(0, *(plain.rand(x, g).cuda() for x in ((T, H, 192), (T, 512), (T, 64))), w,
                       torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda"))
        assert hs.hs_check_flag(s.err) == 0
        units.append(int(s._kept["expanded"][:4].view(torch.int32)))
    assert units[0] == units[1]


@pytest.mark.parametrize("over,form", [(4000, "absorbed"), (100, "expanded")])
def test_prompts_among_single_tokens(over, form):
    """The form that pays for the whole step: rows that one token alone reads are not worth their expansion."""
    H, Dn, Dv, new = 2, 128, 128, [300, 0, 300, 1, 1, 1, 1, 0]
    w, g = plain.weights(H, Dn, Dv, torch.Generator().manual_seed(64)).cuda(), torch.Generator().manual_seed(65)
    s = DenseSession(8, H, 400, 64, max_tokens=600)
    for m in ([0] * 3 + [over] * 4 + [9], new):
        s._kept.clear()
        T = s.extend(m)
        q, latent, rope = (plain.rand(x, g).cuda() for x in ((T, H, Dn + 64), (T, 512), (T, 64)))
        turned, out, lse = q.clone(), torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda")
        hs.hs_rope(turned[..., Dn:], s.positions, s.inv_freq, scale=s.rope_scale)
        s.attend_heads(0, q, latent, rope, w, out, lse, form=None if m is new else "absorbed")
        assert hs.hs_check_flag(s.err) == 0
    assert ("kv" in s._kept) == (form == "expanded")
    ref, tol, rlse, ltol = test_gpu_session_heads.reference(s, 0, turned, w, Dn, (Dn + 64) ** -0.5)
    assert plain.holds(out, ref, tol) and plain.holds(lse, rlse, ltol)
