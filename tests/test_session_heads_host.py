"""What DenseSession.attend_heads asks of its arguments before anything is turned or written, without a GPU."""
import types

import pytest
import torch

from dsa_sparse_mla_gb300.pipeline import DenseSession, _check_heads

T, H, Dn, Dv = 5, 2, 128, 192
CPU = torch.device("cpu")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def odd(*shape):
    """A tensor that starts two bytes after a 16-byte boundary."""
    n = torch.Size(shape).numel()
    x = bf16(n + 16)
    at = next(k for k in range(9) if (x.data_ptr() + 2 * k) % 16 == 2)
    return x[at:at + n].view(shape)


def given(**changed):
    return {**dict(q=bf16(T, H, Dn + 64), latent=bf16(T, 512), rope=bf16(T, 64), w=bf16(H, Dn + Dv, 512), out=bf16(T, H, Dv),
                   lse=torch.zeros(T, H), tokens=T, device=CPU), **changed}


@pytest.mark.parametrize("changed", [dict(), dict(lse=None), dict(q=bf16(T, H, Dn + 72)[..., :Dn + 64]), dict(q=bf16(H, T, Dn + 64).transpose(0, 1)),
                                     dict(out=bf16(T, H, Dv + 8)[..., :Dv]), dict(out=bf16(T + 1, H + 1, Dv)[1:, 1:])], ids=str)
def test_what_is_taken(changed):
    assert _check_heads(**given(**changed)) == (T, H, Dn, Dv)


BAD = {
    "tokens": dict(tokens=T + 1), "rows of latent": dict(latent=bf16(T + 1, 512)), "rotary values": dict(rope=bf16(T, 32)),
    "heads of w": dict(w=bf16(H + 1, Dn + Dv, 512)), "width of w": dict(w=bf16(H, Dn + Dv + 64, 512)), "heads of out": dict(out=bf16(T, H + 1, Dv)),
    "shape of lse": dict(lse=torch.zeros(H, T)), "type of q": dict(q=torch.zeros(T, H, Dn + 64)), "type of w": dict(w=bf16(H, Dn + Dv, 512).half()),
    "type of lse": dict(lse=torch.zeros(T, H, dtype=torch.float64)), "key values": dict(q=bf16(T, H, 96 + 64), w=bf16(H, 96 + Dv, 512)),
    "values": dict(out=bf16(T, H, 96), w=bf16(H, Dn + 96, 512)), "many values": dict(out=bf16(T, H, 320), w=bf16(H, Dn + 320, 512)),
    "many heads": dict(q=bf16(T, 1025, Dn + 64), out=bf16(T, 1025, Dv), w=bf16(1, Dn + Dv, 512).expand(1025, -1, -1), lse=None),
    "device": dict(device=torch.device("cuda", 0)), "device of lse": dict(lse=torch.zeros((T, H), device="meta")),
    "w in parts": dict(w=bf16(H, 512, Dn + Dv).transpose(1, 2)), "latent in parts": dict(latent=bf16(T, 576)[:, :512]),
    "rope in parts": dict(rope=bf16(T, 576)[:, 512:]), "lse in parts": dict(lse=torch.zeros(H, T).T),
    "values of q apart": dict(q=bf16(T, Dn + 64, H).transpose(1, 2)), "values of out apart": dict(out=bf16(T, H, 2 * Dv)[..., ::2]),
    "step of q": dict(q=bf16(T, H, Dn + 68)[..., :Dn + 64]), "step of out": dict(out=bf16(T, H, Dv + 4)[..., :Dv]),
    "one q for all tokens": dict(q=bf16(1, H, Dn + 64).expand(T, -1, -1)), "one out for all heads": dict(out=bf16(T, 1, Dv).expand(-1, H, -1)),
    "start of q": dict(q=odd(T, H, Dn + 64)), "start of latent": dict(latent=odd(T, 512)), "start of rope": dict(rope=odd(T, 64)),
    "start of w": dict(w=odd(H, Dn + Dv, 512)), "start of out": dict(out=odd(T, H, Dv)),
}


@pytest.mark.parametrize("what", BAD)
def test_what_is_refused(what):
    with pytest.raises(ValueError):
        _check_heads(**given(**BAD[what]))


def pays(new, over, heads):
    step = types.SimpleNamespace(pairs=sum(m * (2 * n + m + 1) for m, n in zip(new, over)), read_tokens=sum(m + n for m, n in zip(new, over) if m))
    return DenseSession._expanded_pays(step, sum(new), *heads)


@pytest.mark.parametrize("heads", [(128, 128), (192, 256)])
def test_which_form_pays(heads):
    """Where the forms' times are far apart (measured, absorbed / expanded)."""
    assert pays([8192], [0], heads) and pays([128] * 8, [0] * 8, heads) and pays([512] * 16, [500] * 16, heads)  # 272 / 111 us, 8 x 128
    assert not pays([1] * 64, [2000] * 64, heads) and not pays([32] * 8, [8000] * 8, heads)
    assert not pays([8192] + [1] * 7, [0] + [60000] * 7, heads)  # 4,154 / 7,757
    assert not pays([700] * 3 + [1] * 5, [0] * 3 + [4000] * 5, heads)  # 352 / 447, 361 / 715
    assert pays([2048] + [1] * 63, [2000] + [100] * 63, heads) and pays([1024], [32000], heads)
    assert pays([192] * 8, [8000] * 8, heads) == (heads == (128, 128))  # 1,333 / 1,084, 1,347 / 1,834
