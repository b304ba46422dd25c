"""DenseSession.attend_heads and memory: the form where the expanded one's buffers cannot be had, and what a step gives back."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu
H, Dn, Dv, L = 2, 128, 128, 3


def session(new):
    s = DenseSession(2, H, 40, 20, L=L, max_tokens=64)
    return s, s.extend(new)


def inputs(T, seed):
    g = torch.Generator().manual_seed(seed)
    return [plain.rand(x, g).cuda() for x in ((T, H, Dn + 64), (T, 512), (T, 64))]


W = plain.weights(H, Dn, Dv, torch.Generator().manual_seed(70))


def test_without_room_a_step_is_absorbed(monkeypatch):
    new = [500, 300]
    want, T = session(new)
    s, _ = session(new)
    assert s._expanded_pays(T, Dn, Dv)
    asked, make = [], DenseSession._buffer

    def no_room(self, name, *shape, **kw):
        asked.append(name)
        if name == "kv":
            raise torch.OutOfMemoryError("no room")
        return make(self, name, *shape, **kw)

    for layer in range(L):
        outs = [torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        want.attend_heads(layer, *inputs(T, layer), W.cuda(), outs[0], form="absorbed")
        with monkeypatch.context() as m:
            m.setattr(DenseSession, "_buffer", no_room)
            if layer == 0:  # asked for, it says so, and nothing has happened
                x = inputs(T, layer)
                with pytest.raises(torch.OutOfMemoryError):
                    s.attend_heads(layer, *x, W.cuda(), outs[1], form="expanded")
                assert not s.pool.any() and bool((outs[1] == 7).all()) and all(torch.equal(a, b) for a, b in zip(x, inputs(T, layer)))
                asked.clear()
            s.attend_heads(layer, *inputs(T, layer), W.cuda(), outs[1])
        assert torch.equal(*outs) and hs.hs_check_flag(s.err) == 0
    assert asked.count("kv") == 1 and "rows" not in s._kept and torch.equal(want.pool, s.pool)
    T = s.extend([0, 400])  # the next step asks again
    s.attend_heads(0, *inputs(T, 9), W.cuda(), torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"))
    assert "kv" in s._kept


def test_keys_and_values_are_given_back():
    s, T = session([500, 300])
    s.attend_heads(0, *inputs(T, 0), W.cuda(), torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"))
    size = s._kept["kv"].untyped_storage().nbytes() + s._kept["rows"].untyped_storage().nbytes()
    assert size >= 2 * T * (H * (Dn + Dv) + 576)
    T = s.extend([1, 1])
    x, w, out = inputs(T, 1), W.cuda(), torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda")
    s._buffer("queries", T, H, 576), s._buffer("mixed", T, H, 512)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    s.attend_heads(0, *x, w, out)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before - size and hs.hs_check_flag(s.err) == 0


def test_an_extend_without_room_changes_nothing(monkeypatch):
    """Where the attention's workspace cannot be had, the step before stays the one that attend_heads runs."""
    s, T = session([500, 300])
    x, out = inputs(T, 2), [torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s.attend_heads(0, *x, W.cuda(), out[0])
    before = {k: v for k, v in vars(s).items() if isinstance(v, (int, bool, torch.Tensor))}
    held = {k: v.clone() for k, v in before.items() if isinstance(v, torch.Tensor)}

    def no_room(self, tokens, cached):
        raise torch.OutOfMemoryError("no room")

    with monkeypatch.context() as m:
        m.setattr(DenseSession, "_make_room", no_room)
        with pytest.raises(torch.OutOfMemoryError):
            s.extend([0, 900])
    assert all(getattr(s, k) is v if isinstance(v, torch.Tensor) else getattr(s, k) == v for k, v in before.items())
    assert all(torch.equal(getattr(s, k), v) for k, v in held.items())
    s.attend_heads(0, *inputs(T, 2), W.cuda(), out[1])
    assert torch.equal(*out) and hs.hs_check_flag(s.err) == 0
