"""DenseSession.attend_heads: a call that is refused has turned and written nothing, and whether it is refused does not depend on the
form; results in slices of wider rows."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu
T, H, Dn, Dv = 300, 3, 128, 128


def step(seed=31):
    g = torch.Generator().manual_seed(seed)
    return dict(zip(("q", "latent", "rope", "w"), (x.cuda() for x in (plain.rand((T, H, Dn + 64), g), plain.rand((T, 512), g), plain.rand((T, 64), g),
                                                                      plain.weights(H, Dn, Dv, g)))))


@pytest.mark.parametrize("form", ["absorbed", "expanded", None])
def test_refused_calls_change_nothing(form):
    s, a = DenseSession(2, H, 16, 8, max_tokens=T), step()
    with pytest.raises(ValueError):  # before any extend
        s.attend_heads(0, **a, out=torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"), form=form)
    s.extend([200, 100])
    held = {k: v.clone() for k, v in a.items()}
    out, lse = torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda")
    wide = torch.zeros((T, H, 2 * 192), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(layer=1), dict(w=a["w"].transpose(1, 2).contiguous().transpose(1, 2)), dict(latent=torch.cat([a["latent"]] * 2, 1)[:, :512]),
                dict(rope=torch.cat([a["rope"]] * 2, 1)[:, :64]), dict(q=wide[..., ::2]), dict(q=wide[..., 4:196]), dict(out=wide[..., 1:129]),
                dict(out=wide[..., :256:2]), dict(lse=lse.double()), dict(lse=torch.cat([lse, lse], 1)[:, :H]), dict(lse=lse.cpu()), dict(w=a["w"].cpu()),
                dict(q=torch.cat([a["q"], a["q"]], 2)[..., :160], w=torch.cat([a["w"], a["w"]], 1)[:, :224].contiguous())):
        with pytest.raises((ValueError, IndexError)):
            s.attend_heads(**{**dict(layer=0, **a, out=out, lse=lse, form=form), **bad})
    assert not s.pool.any() and all(torch.equal(a[k], held[k]) for k in a) and bool((out == 7).all()) and bool((lse == 7).all())
    s.attend_heads(0, **a, out=out, lse=lse, form=form)
    assert hs.hs_check_flag(s.err) == 0 and bool(out.isfinite().all()) and bool(s.pool.any())


@pytest.mark.parametrize("form", ["absorbed", "expanded", None])
def test_results_in_slices_of_wider_rows(form):
    got = []
    for shape, at in (((T, H, Dv), (0, 0)), ((T, H, Dv + 8), (0, 8)), ((T, H + 2, Dv), (1, 0))):
        s, a = DenseSession(2, H, 16, 8, max_tokens=T), step()
        s.extend([200, 100])
        mem = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        out = mem[:, at[0]:at[0] + H, at[1]:at[1] + Dv]
        s.attend_heads(0, **a, out=out, form=form)
        assert hs.hs_check_flag(s.err) == 0
        got.append(out.clone())
        out.fill_(7)
        assert bool((mem == 7).all())
    assert all(torch.equal(got[0], x) for x in got[1:])


def test_more_heads_than_the_session_was_made_for():
    """They run expanded, however few the tokens are, and not at all where that is not their form."""
    g = torch.Generator().manual_seed(32)
    for new in ([3, 1], [300, 0]):
        s, t = DenseSession(2, H - 1, 16, 8, max_tokens=T), sum(new)
        s.extend(new)
        for form in ("absorbed", None):
            for width in (128, 64):
                a = [plain.rand(x, g).cuda() for x in ((t, H, width + 64), (t, 512), (t, 64))]
                out = torch.full((t, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
                if form or width == 64:
                    with pytest.raises(ValueError):
                        s.attend_heads(0, *a, plain.weights(H, width, 128, g).cuda(), out, form=form)
                    assert bool((out == 7).all())
                else:
                    s.attend_heads(0, *a, plain.weights(H, width, 128, g).cuda(), out, form=form)
                    assert hs.hs_check_flag(s.err) == 0 and not bool((out == 7).all(-1).any())
