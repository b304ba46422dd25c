"""Steps of a DenseSession in graphs: replayed on other queries and rows than they were captured with, and after the session has gone on."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
from dsa_sparse_mla_gb300.pipeline import DenseSession

pytestmark = pytest.mark.gpu
H, NEW, MORE = 4, [150, 3, 200], [40, 0, 700]
T = sum(NEW)


def inputs(form, seed, tokens=T):
    g = torch.Generator().manual_seed(seed)
    D = 576 if form == "latent" else 192
    return [x.cuda() for x in (plain.rand((tokens, H, D), g), plain.rand((tokens, 512), g), plain.rand((tokens, 64), g))]


def call(s, form, w, x, out, lse):
    if form == "latent":
        s.attend(0, *x, out, lse)
    else:
        s.attend_heads(0, *x, w, out, lse, form=form)


def results(form, tokens=T):
    D = 512 if form == "latent" else 128
    return torch.full((tokens, H, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((tokens, H), 7.0, device="cuda")


@pytest.mark.parametrize("form", ["latent", "absorbed", "expanded"])
def test_replayed_on_other_inputs_and_after_more_tokens(form):
    w = plain.weights(H, 128, 128, torch.Generator().manual_seed(40)).cuda()

    def session():
        s = DenseSession(3, H, 40, 20, max_tokens=T)
        assert s.extend(NEW) == T
        return s

    want = []
    for seed in (41, 42, 43):
        s, r = session(), results(form)
        call(s, form, w, inputs(form, seed), *r)
        assert hs.hs_check_flag(s.err) == 0
        want.append(r)
    s, r, held = session(), results(form), inputs(form, 41)
    call(s, form, w, held, *r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, form, w, held, *r)
    names = ["positions", "token_req", "req_start", "seq_len", "workspace"] + ["read_start"] * (form == "expanded")
    assert all(any(getattr(s, n) is x for x in s._captured) for n in names)
    used = [getattr(s, n).data_ptr() for n in names]

    def replay(seed):
        for h, x in zip(held, inputs(form, seed)):
            h.copy_(x)
        for x in r:
            x.fill_(7)
        graph.replay()
        assert hs.hs_check_flag(s.err) == 0
        return all(torch.equal(a, b) for a, b in zip(r, want[seed - 41]))

    assert replay(42) and replay(43)
    # the session goes on: other tensors, a larger workspace; what was given back serves others
    tokens = s.extend(MORE)
    call(s, form, w, inputs(form, 50, tokens), *results(form, tokens))
    s._make_room(64 * T, 1 << 20)
    others = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (4, 4, 4, 4, T, T, T, T) for _ in range(20)]
    assert not any(x.data_ptr() in used for x in others) and all(getattr(s, n).data_ptr() != x for n, x in zip(names, used))
    for seed in (42, 41, 43):
        assert replay(seed)


def test_what_is_given_back_stays_with_the_graph():
    """Captured without a call before, in a session with idle slots; then an absorbed step gives the keys and values back, and what takes
    their place has no part in the replays."""
    w = plain.weights(H, 128, 128, torch.Generator().manual_seed(40)).cuda()

    def session():
        s = DenseSession(5, H, 40, 20, max_tokens=T)
        assert s.extend([0] + NEW + [0]) == T
        return s

    s, want = session(), results("expanded")
    call(s, "expanded", w, inputs("expanded", 44), *want)
    s, r, held = session(), results("expanded"), inputs("expanded", 44)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, "expanded", w, held, *r)
    size = s._kept["kv"].numel()
    tokens = s.extend([1] * 5)
    call(s, "absorbed", w, inputs("absorbed", 45, tokens), *results("absorbed", tokens))
    assert "kv" not in s._kept and "rows" not in s._kept
    others = [torch.full((size,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for h, x in zip(held, inputs("expanded", 44)):
        h.copy_(x)
    graph.replay()
    assert hs.hs_check_flag(s.err) == 0 and all(torch.equal(a, b) for a, b in zip(r, want)) and all(bool(x.isnan().all()) for x in others)
