"""pipeline.DenseSession.attend_heads: per-head queries to per-head outputs in both forms of latent attention, over several steps, held
against 64-bit attention over the session's own rows and the layer's weight."""
import math

import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
import plain_ops
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu


def reference(session, layer, q, w, Dn, scale):
    """float64 out, lse, and bounds. Each form rounds a logit's factors to bf16 twice on its way (the expanded one the latent and the
    key, the absorbed one the query in the latent space, its rows to fp16): off by 2^-7 + 2^-10 of its absolute terms; a value likewise;
    then a weight by 2^-8 and the result by 2^-8 (the absorbed form rounds the latent output and the result)."""
    T, H, _ = q.shape
    Dv = w.shape[1] - Dn
    out = torch.zeros((T, H, Dv), dtype=torch.float64, device="cuda")
    tol, lse = torch.zeros_like(out), torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    ltol = torch.zeros_like(lse)
    start, eps, W = session.req_start.tolist(), 2.0 ** -7 + 2.0 ** -10, w.double()
    for r, n in enumerate(session.seq_len.tolist()):
        m = start[r + 1] - start[r]
        if m == 0:
            continue
        j = torch.arange(n, device="cuda")
        lat, rope = plain_ops.read_rows(session.pool[layer][session.table[r].long()[j // 64] * 64 + j % 64])
        kv, size = torch.einsum("nc,hdc->hnd", lat, W), torch.einsum("nc,hdc->hnd", lat.abs(), W.abs())
        for i in range(m):
            t, see = start[r] + i, n - m + 1 + i
            qn, qr = q[t, :, :Dn].double(), q[t, :, Dn:].double()
            z = (torch.einsum("hd,hnd->hn", qn, kv[:, :see, :Dn]) + qr @ rope[:see].T) * scale
            terms = (torch.einsum("hd,hnd->hn", qn.abs(), size[:, :see, :Dn]) + qr.abs() @ rope[:see].abs().T) * scale
            delta = (terms * eps).amax(-1)
            p = torch.softmax(z, -1)
            out[t] = torch.einsum("hn,hnd->hd", p, kv[:, :see, Dn:])
            spread = torch.einsum("hn,hnd->hd", p, size[:, :see, Dn:])
            tol[t] = spread * (torch.expm1(2 * delta)[:, None] + eps + 2.0 ** -7) * (1 + 2.0 ** -6) + 1e-30
            lse[t] = torch.logsumexp(z, -1)
            ltol[t] = delta + 2.0 ** -14
    return out, tol, lse, ltol


@pytest.mark.parametrize("H,Dn,Dv", [(3, 128, 128), (2, 192, 256)])
def test_both_forms_over_several_steps(H, Dn, Dv):
    g = torch.Generator().manual_seed(7)
    L = 2
    ws = [plain.weights(H, Dn, Dv, g).cuda() for _ in range(L)]
    sessions = {f: DenseSession(4, H, 40, 10, L=L, max_tokens=64, kind="yarn", factor=4.0) for f in ("absorbed", "expanded", None)}
    scale = None
    for new in ([200, 0, 70, 1], [1, 1, 1, 1], [0, 130, 4, 300], [3, 0, 0, 0], [1, 1, 0, 1]):
        T = sum(new)
        for layer in range(L):
            q, latent, rope = (plain.rand(s, g).cuda() for s in ((T, H, Dn + 64), (T, 512), (T, 64)))
            got = {}
            for form, s in sessions.items():
                if layer == 0:
                    assert s.extend(new) == T
                qq, out, lse = q.clone(), torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda")
                s.attend_heads(layer, qq, latent.clone(), rope.clone(), ws[layer], out, lse, form=form)
                assert hs.hs_check_flag(s.err) == 0
                got[form] = (qq, out, lse)
            s = sessions["expanded"]
            scale = s.softmax_scale * 24 / math.sqrt(Dn + 64)
            ref, tol, rlse, ltol = reference(s, layer, got["expanded"][0], ws[layer], Dn, scale)
            for form, (_, out, lse) in got.items():
                assert plain.holds(out, ref, tol) and plain.holds(lse, rlse, ltol), form
                # the roundings' errors are spread: together they stay below the largest single ones by far
                assert float((out.double() - ref).norm() / ref.norm()) <= 2.0 ** -6, form
    assert torch.equal(sessions["absorbed"].pool, sessions["expanded"].pool)


def test_the_form_follows_the_tokens():
    s = DenseSession(2, 1, 64, 32, max_tokens=64)
    g = torch.Generator().manual_seed(8)
    w = plain.weights(1, 128, 128, g).cuda()
    for new, expanded in (([1, 1], False), ([600, 1], True), ([1, 0], False), ([0, 300], True)):
        T = s.extend(new)
        s._kept.pop("kv", None)
        s.attend_heads(0, *(plain.rand(x, g).cuda() for x in ((T, 1, 192), (T, 512), (T, 64))), w, torch.empty((T, 1, 128), dtype=torch.bfloat16, device="cuda"))
        assert ("kv" in s._kept) == expanded
    T = s.extend([0, 0])
    s.attend_heads(0, *(torch.empty(x, dtype=torch.bfloat16, device="cuda") for x in ((0, 1, 192), (0, 512), (0, 64))), w,
                   torch.empty((0, 1, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        s.attend_heads(0, torch.empty((0, 1, 192), device="cuda"), None, None, w, torch.empty((0, 1, 128), device="cuda"), form="both")


def test_a_step_in_a_graph():
    """Both forms captured and replayed on new queries: the same bits as the calls themselves."""
    g = torch.Generator().manual_seed(9)
    H, Dn, Dv = 4, 128, 128
    w = plain.weights(H, Dn, Dv, g).cuda()
    for form in ("absorbed", "expanded"):
        s = DenseSession(3, H, 32, 10, max_tokens=400)
        T = s.extend([150, 3, 200])
        q, latent, rope = (plain.rand(x, g).cuda() for x in ((T, H, Dn + 64), (T, 512), (T, 64)))
        held = [x.clone() for x in (q, latent, rope)]
        out, lse = torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
        s.attend_heads(0, *held, w, out, lse, form=form)
        first = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.attend_heads(0, *held, w, out, lse, form=form)
        for k in range(3):
            for h, x in zip(held, (q, latent, rope)):
                h.copy_(x)
            out.zero_()
            graph.replay()
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and hs.hs_check_flag(s.err) == 0


def test_heads_that_have_one_form_only():
    """Heads of 192 and 128 values run absorbed, however many tokens; asked for the other form, or with shapes that do not fit, a call
    changes nothing."""
    g = torch.Generator().manual_seed(10)
    H, Dn, Dv = 2, 192, 128
    s, w = DenseSession(1, H, 16, 16, max_tokens=400), plain.weights(H, Dn, Dv, g).cuda()
    T = s.extend([400])
    q, latent, rope = (plain.rand(x, g).cuda() for x in ((T, H, Dn + 64), (T, 512), (T, 64)))
    held = [x.clone() for x in (q, latent, rope)]
    out, lse = torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
    for bad in (dict(form="expanded"), dict(w=w[:, 64:].contiguous()), dict(q=q[1:]), dict(out=out[:, :1]), dict(latent=latent[:, :448]),
                dict(rope=rope.half()), dict(q=q.float()), dict(lse=lse[1:]),
                dict(q=torch.cat([q, q], 1), w=torch.cat([w, w]), out=torch.cat([out, out], 1))):
        args = dict(dict(q=q, latent=latent, rope=rope, w=w, out=out), **bad)
        with pytest.raises(ValueError):
            s.attend_heads(0, **args)
    assert not s.pool.any() and all(torch.equal(a, b) for a, b in zip(held, (q, latent, rope))) and bool((out == 7).all())
    s.attend_heads(0, q, latent, rope, w, out, lse)
    assert hs.hs_check_flag(s.err) == 0
    turned, scale = q.clone(), s.softmax_scale * 24 / math.sqrt(Dn + 64)
    hs.hs_rope(turned[..., Dn:], s.positions, s.inv_freq, scale=s.rope_scale)
    ref, tol, rlse, ltol = reference(s, 0, turned, w, Dn, scale)
    assert plain.holds(out, ref, tol) and plain.holds(lse, rlse, ltol)


def test_a_graph_keeps_its_buffers():
    """Captured, then called with larger heads, for which the buffers are made anew: the graph's replays still have theirs."""
    g = torch.Generator().manual_seed(11)
    H, T = 4, 300
    small, large = (plain.weights(H, Dn, Dv, g).cuda() for Dn, Dv in ((128, 128), (192, 256)))
    for form in ("absorbed", "expanded"):
        s = DenseSession(1, 2 * H, 16, 16, max_tokens=T)
        assert s.extend([T]) == T
        q, latent, rope = (plain.rand(x, g).cuda() for x in ((T, H, 192), (T, 512), (T, 64)))
        held, out = [x.clone() for x in (q, latent, rope)], torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda")
        s.attend_heads(0, *held, small, out, form=form)
        first, graph = out.clone(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.attend_heads(0, *held, small, out, form=form)
        kept = dict(s._kept)
        wide = [torch.cat([large] * 2), torch.empty((T, 2 * H, 256), dtype=torch.bfloat16, device="cuda")]
        s.attend_heads(0, plain.rand((T, 2 * H, 256), g).cuda(), latent.clone(), rope.clone(), *wide, form=form)
        names = ("queries", "mixed") if form == "absorbed" else ("kv", "expanded")
        assert all(s._kept[n] is not kept[n] and any(kept[n] is x for x in s._captured) for n in names)
        for h, x in zip(held, (q, latent, rope)):
            h.copy_(x)
        graph.replay()
        assert torch.equal(out, first) and hs.hs_check_flag(s.err) == 0
