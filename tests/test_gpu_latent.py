"""hs_kv_read, hs_mla_absorb, hs_mla_project, hs_mla_expand and hs_mla_expanded_fwd against 64-bit references."""
import math

import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
import plain_ops

pytestmark = pytest.mark.gpu


def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ the cache read back ----
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lens,first,wide", [([1], [0], 0), ([64, 0, 1, 63, 65], [0, 0, 3, 2, 64], 8), ([0, 0, 700], [1, 0, 5], 0),
                                             ([5] * 70, list(range(70)), 64)])
def test_read(dtype, lens, first, wide):
    b = plain_ops.make_batch([1] * len(lens), [f + n for f, n in zip(first, lens)], 1)
    n = sum(lens)
    out = torch.full((n + 3, 576 + wide), 7.0, dtype=dtype, device="cuda")
    e = err()
    hs.hs_kv_read(b["pool"], b["table"], plain.starts(lens).cuda(), out[:, :576], e, first=torch.tensor(first, dtype=torch.int32, device="cuda"))
    assert hs.hs_check_flag(e) == 0
    ref = []
    for r, (f, m) in enumerate(zip(first, lens)):
        j = torch.arange(f, f + m, device="cuda")
        ref.append(torch.cat(plain_ops.read_rows(b["pool"][b["table"][r].long()[j // 64] * 64 + j % 64]), 1))
    ref = torch.cat(ref)
    step = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}[dtype]
    low = 2.0 ** -25 if dtype is torch.float16 else 0.0  # half of fp16's smallest step
    assert bool(((out[:n, :576].double() - ref).abs() <= ref.abs() * (step + 2.0 ** -24) * (1 + 2.0 ** -8) + low).all())
    assert bool((out[n:] == 7).all()) and bool((out[:, 576:] == 7).all())


def test_read_without_first_and_its_flags():
    b = plain_ops.make_batch([1, 1], [100, 130], 1)
    out, e = torch.full((230, 576), 7.0, device="cuda"), err()
    start = plain.starts([100, 130]).cuda()
    hs.hs_kv_read(b["pool"], b["table"], start, out, e)
    assert hs.hs_check_flag(e) == 0 and bool(out.isfinite().all()) and not bool((out == 7).all(1).any())
    table = b["table"].clone()
    table[0, 1], table[1, 0] = -1, b["pool"].shape[0] // 64
    hs.hs_kv_read(b["pool"], table, start, out, e)
    assert hs.hs_check_flag(e) == hs.FLAGS["BAD_BLOCK"]
    assert not out[64:164].any() and bool(out[:64].any(1).all()) and bool(out[164:].any(1).all())
    e = err()
    far = torch.tensor([64 * table.shape[1] - 50, -1], dtype=torch.int32, device="cuda")
    hs.hs_kv_read(b["pool"], b["table"], start, out, e, first=far)
    assert hs.hs_check_flag(e) & hs.FLAGS["BAD_LENGTH"] and not out[50:101].any()
    for bad in ([0, 120, 100], [0, 100, 231], [3, 100, 230]):
        e = err()
        hs.hs_kv_read(b["pool"], b["table"], torch.tensor(bad, dtype=torch.int32, device="cuda"), out, e)
        assert hs.hs_check_flag(e) & hs.FLAGS["BAD_INDEX"]


# ------------------------------------------------------------------ products ---------------
SIZES = [(1, 1, 64, 64), (3, 2, 128, 128), (129, 3, 192, 256), (255, 1, 256, 64), (257, 5, 64, 192), (600, 2, 128, 256), (1030, 64, 128, 128)]


@pytest.mark.parametrize("T,H,Dn,Dv", SIZES)
def test_absorb(T, H, Dn, Dv):
    g = gen(T)
    q, w = plain.rand((T, H, Dn + 64), g).cuda(), plain.weights(H, Dn, Dv, g).cuda()
    out, e = torch.full((T + 2, H, 576), 7.0, dtype=torch.bfloat16, device="cuda"), err()
    hs.hs_mla_absorb(q[..., :Dn], w, out[:T, :, :512], e)
    assert hs.hs_check_flag(e) == 0
    ref, tol = plain.product(q[..., :Dn], w[:, :Dn], "thd,hdc->thc")
    assert plain.holds(out[:T, :, :512], ref, tol)
    assert bool((out[T:] == 7).all()) and bool((out[..., 512:] == 7).all())


@pytest.mark.parametrize("T,H,Dn,Dv", SIZES)
def test_project(T, H, Dn, Dv):
    g = gen(T + 1)
    x, w = plain.rand((T, H, 576), g).cuda(), plain.weights(H, Dn, Dv, g).cuda()
    out, e = torch.full((T + 2, H, Dv + 8), 7.0, dtype=torch.bfloat16, device="cuda"), err()
    hs.hs_mla_project(x[..., :512], w, out[:T, :, :Dv], e)
    assert hs.hs_check_flag(e) == 0
    ref, tol = plain.product(x[..., :512], w[:, Dn:], "thc,hdc->thd")
    assert plain.holds(out[:T, :, :Dv], ref, tol)
    assert bool((out[T:] == 7).all()) and bool((out[..., Dv:] == 7).all())


@pytest.mark.parametrize("T,H,Dn,Dv", SIZES)
def test_expand(T, H, Dn, Dv):
    g = gen(T + 2)
    c, w = plain.rand((T, 576), g).cuda(), plain.weights(H, Dn, Dv, g).cuda()
    wide = torch.full((T + 2, H * (Dn + Dv) + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    kv, e = wide[:T, :H * (Dn + Dv)].unflatten(1, (H, Dn + Dv)), err()
    hs.hs_mla_expand(c[:, :512], w, kv, e)
    assert hs.hs_check_flag(e) == 0
    ref, tol = plain.product(c[:, :512], w, "nc,hdc->nhd")
    assert plain.holds(kv, ref, tol)
    assert bool((wide[T:] == 7).all()) and bool((wide[:, H * (Dn + Dv):] == 7).all())


@pytest.mark.parametrize("T,H,Dn,Dv", SIZES)
def test_where_rows_start(T, H, Dn, Dv):
    """Results whose rows start on 32 bytes, on 16 bytes only, or on both in turn: within their bounds, the same bits, nothing beside them."""
    g = gen(T + 3)
    x, c, w = plain.rand((T, H, 512), g).cuda(), plain.rand((T, 512), g).cuda(), plain.weights(H, Dn, Dv, g).cuda()
    got = []
    for shift, pad in ((0, 0), (8, 0), (0, 8), (16, 16)):
        mem, e = torch.full((T * (H * (Dv + pad)) + shift + 8,), 7.0, dtype=torch.bfloat16, device="cuda"), err()
        out = mem[shift:][:T * H * (Dv + pad)].view(T, H, Dv + pad)
        hs.hs_mla_project(x, w, out[..., :Dv], e)
        width = H * (Dn + Dv)
        wide = torch.full((T * (width + pad) + shift + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        kv = wide[shift:][:T * (width + pad)].view(T, width + pad)
        hs.hs_mla_expand(c, w, kv[:, :width].unflatten(1, (H, Dn + Dv)), e)
        assert hs.hs_check_flag(e) == 0
        for m, o, n in ((mem, out, Dv), (wide, kv, width)):
            assert bool((o[..., n:] == 7).all()) and bool((m[:shift] == 7).all()) and bool((m[shift + o.numel():] == 7).all())
        got.append((out[..., :Dv].clone(), kv[:, :width].unflatten(1, (H, Dn + Dv)).clone()))
    assert plain.holds(got[0][0], *plain.product(x, w[:, Dn:], "thc,hdc->thd")) and plain.holds(got[0][1], *plain.product(c, w, "nc,hdc->nhd"))
    assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))


def test_heads_apart():
    """Heads first in memory ([H, T, D] storage), and results that equal those of the usual order bit for bit."""
    g = gen(5)
    T, H, Dn, Dv = 130, 4, 128, 128
    q, x, w = plain.rand((H, T, Dn), g).cuda(), plain.rand((H, T, 512), g).cuda(), plain.weights(H, Dn, Dv, g).cuda()
    a, b = (torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c, d = torch.empty((H, T, Dv), dtype=torch.bfloat16, device="cuda").transpose(0, 1), torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda")
    e = err()
    hs.hs_mla_absorb(q.transpose(0, 1), w, a, e)
    hs.hs_mla_absorb(q.transpose(0, 1).contiguous(), w, b, e)
    hs.hs_mla_project(x.transpose(0, 1), w, c, e)
    hs.hs_mla_project(x.transpose(0, 1).contiguous(), w, d, e)
    assert hs.hs_check_flag(e) == 0 and torch.equal(a, b) and torch.equal(c, d)


# ------------------------------------------------------------------ attention --------------
def batch(q_lens, kv_lens, H, Dn, Dv, seed=0, sigma=1.0, spare=0):
    g = gen(seed)
    T, N = sum(q_lens), sum(kv_lens) + spare
    q, kv, rows = plain.rand((T, H, Dn + 64), g, sigma), plain.rand((N, H, Dn + Dv), g), plain.rand((N, 576), g)
    if spare:
        kv[-spare:], rows[-spare:] = math.nan, math.nan
    return dict(q=q.cuda(), kv=kv.cuda(), rope=rows.cuda()[:, 512:], req_start=plain.starts(q_lens).cuda(), kv_start=plain.starts(kv_lens).cuda(),
                scale=(Dn + 64) ** -0.5)


def attend(b, Dv, causal=True, e=None, workspace=None):
    T, H, _ = b["q"].shape
    out = torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    e = err() if e is None else e
    if workspace is None:
        workspace = torch.full((hs.hs_mla_expanded_workspace_size(b["req_start"].numel() - 1, Dv),), 0xFF, dtype=torch.uint8, device="cuda")
    hs.hs_mla_expanded_fwd(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], b["scale"], out, e, workspace, lse=lse, causal=causal)
    assert hs.hs_check_flag(e) == 0
    return out, lse


def check(b, Dn, Dv, causal=True):
    out, lse = attend(b, Dv, causal)
    ref, tol, rlse, ltol = plain.attention(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], Dn, b["scale"], causal)
    assert plain.holds(lse, rlse, ltol)
    assert plain.holds(out, ref, tol)


HEADS = [(128, 128), (192, 256)]
BATCHES = [([1], [1], 1), ([1], [700], 3), ([5], [3], 2), ([130], [130], 2), ([257], [300], 1), ([0, 3, 0], [9, 128, 0], 2),
           ([1] * 9, [1, 2, 63, 64, 127, 128, 129, 255, 1000], 5), ([40, 1, 0, 300, 7], [40, 2000, 55, 129, 6], 4), ([600, 513], [600, 900], 2)]


@pytest.mark.parametrize("Dn,Dv", HEADS)
@pytest.mark.parametrize("q_lens,kv_lens,H", BATCHES)
def test_attention(q_lens, kv_lens, H, Dn, Dv):
    check(batch(q_lens, kv_lens, H, Dn, Dv, spare=200), Dn, Dv)


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_without_mask(Dn, Dv):
    check(batch([3, 200, 0, 1], [150, 260, 4, 129], 3, Dn, Dv, spare=5), Dn, Dv, causal=False)


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_splits_long_rows(Dn, Dv):
    check(batch([1, 2, 20], [9000, 5000, 7001], 1, Dn, Dv, spare=3), Dn, Dv)


@pytest.mark.parametrize("Dn,Dv,q_lens,kv_lens,H", [(128, 128, [600], [2500], 32), (192, 256, [600], [2500], 32), (128, 128, [60], [2300], 200),
                                                    (128, 128, [3, 520, 0, 1], [40, 4500, 9, 1], 37)])
def test_attention_of_more_blocks_than_workers(Dn, Dv, q_lens, kv_lens, H):
    """Blocks of several tiles for more than one turn of all workers, with some left over; the same bits each time."""
    b = batch(q_lens, kv_lens, H, Dn, Dv, seed=H)
    check(b, Dn, Dv)
    check(b, Dn, Dv, causal=False)
    first = attend(b, Dv)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(first, attend(b, Dv)))


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_scales_its_output(Dn, Dv):
    """Logits that grow along the rows move the reference (and scale the output) at most tiles; negative and zero scales."""
    b = batch([3, 140], [1500, 1000], 2, Dn, Dv, seed=3)
    ramp = torch.linspace(0, 3, 2500, device="cuda")[:, None, None]
    b["kv"][..., :Dn] = (b["q"][0, 0, :Dn].float() * ramp + b["kv"][..., :Dn].float()).bfloat16()
    for scale in (b["scale"], -b["scale"], 0.0):
        b["scale"] = scale
        check(b, Dn, Dv)


@pytest.mark.parametrize("Dn,Dv", HEADS)
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_attention_leaves_masked_rows_out(what, Dn, Dv):
    """Values, keys and rotary keys that are not finite, in rows that some tokens do not see."""
    for part in ("key", "value", "rope"):
        b = batch([150, 1, 30], [400, 300, 1800], 2, Dn, Dv, seed=4)
        rows = torch.tensor([399, 390, 2499, 2490, 2480], device="cuda")  # the last rows of the first and third request
        if part == "key":
            b["kv"][rows, :, 5] = what
        elif part == "value":
            b["kv"][rows, 1, Dn + 7] = what
        else:
            b["rope"][rows, 63] = what
        out, lse = attend(b, Dv)
        ref, tol, rlse, ltol = plain.attention(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], Dn, b["scale"])
        clear = rlse.isfinite() & ref.isfinite().all(-1)  # tokens and heads that see none of them
        assert int(clear.sum()) > 250
        assert bool(((out.double() - ref).abs() <= tol)[clear].all()) and bool(((lse.double() - rlse).abs() <= ltol)[clear].all())
        if what != -math.inf or part == "value":  # a key's -inf may leave its row out
            bad = ~ref.isfinite()
            assert bool(out[bad].isfinite().logical_not().all())


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_again_and_again(Dn, Dv):
    """Many units of few tokens and few tiles, and of few tokens and many, on every pair of CTAs: the same bits each time."""
    for q_lens, kv_lens, H in (([1, 2, 40] * 30, [1, 130, 300] * 30, 16), ([1] * 20, [4000] * 20, 16), ([300] * 4, [300, 900, 2000, 310], 40)):
        b = batch(q_lens, kv_lens, H, Dn, Dv, seed=5, spare=130)
        ref, tol, rlse, ltol = plain.attention(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], Dn, b["scale"])
        first = attend(b, Dv)
        assert plain.holds(first[0], ref, tol) and plain.holds(first[1], rlse, ltol)
        for _ in range(20):
            again = attend(b, Dv)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_of_few_and_many_tokens_together(Dn, Dv):
    """Both sides of the rule between CTAs by themselves and pairs (128 tokens per request on average), with blocks of few tokens in pairs
    and requests of several blocks in CTAs."""
    check(batch([1, 700], [300, 900], 2, Dn, Dv, seed=11, spare=9), Dn, Dv)
    check(batch([2, 400, 1, 0, 3], [300, 500, 1, 7, 4000], 2, Dn, Dv, seed=12, spare=9), Dn, Dv)
    check(batch([128, 128], [128, 129], 3, Dn, Dv, seed=13), Dn, Dv)
    check(batch([128, 129], [128, 129], 3, Dn, Dv, seed=13), Dn, Dv)


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_flags(Dn, Dv):
    """Offsets that are out of order: the flag, the tokens whose results stay those of the good call, those that see nothing, and those
    that are left alone. Requests of 3, 200 and 4 tokens over 50, 300 and 9 rows."""
    b = batch([3, 200, 4], [50, 300, 9], 2, Dn, Dv, seed=14)
    good, _ = attend(b, Dv)
    T, H, _ = b["q"].shape
    for key, bad, same, nothing, alone in (
            ("req_start", [0, 203, 3, 207], [], [], [(0, 207)]),                 # 203 and 204 tokens: more than there are
            ("req_start", [0, 207, 0, 207], [], [], [(0, 207)]),
            ("req_start", [0, 3, 203, 206], [(0, 203)], [], [(206, 207)]),       # the last token is nobody's
            ("req_start", [1, 3, 203, 207], [(3, 207)], [], [(0, 1)]),           # the first one is
            ("req_start", [0, -1, 203, 207], [(203, 207)], [], [(0, 203)]),
            ("req_start", [0, 300, 203, 207], [(203, 207)], [], [(0, 203)]),
            ("kv_start", [0, 50, 350, 400], [(0, 203)], [(203, 207)], []),       # past the 359 rows
            ("kv_start", [0, -5, 350, 359], [(203, 207)], [(0, 203)], [])):
        c = dict(b)
        c[key] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out, lse, e = torch.full((T, H, Dv), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 7.0, device="cuda"), err()
        ws = torch.empty(hs.hs_mla_expanded_workspace_size(3, Dv), dtype=torch.uint8, device="cuda")
        hs.hs_mla_expanded_fwd(c["q"], c["kv"], c["rope"], c["req_start"], c["kv_start"], c["scale"], out, e, ws, lse=lse)
        assert hs.hs_check_flag(e) == hs.FLAGS["BAD_INDEX" if key == "req_start" else "BAD_LENGTH"], bad
        for lo, hi in same:
            assert torch.equal(out[lo:hi], good[lo:hi]), bad
        for lo, hi in nothing:
            assert not out[lo:hi].any() and bool((lse[lo:hi] == -math.inf).all()), bad
        for lo, hi in alone:
            assert bool((out[lo:hi] == 7).all()) and bool((lse[lo:hi] == 7).all()), bad


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_calls_on_other_streams_and_in_graphs(Dn, Dv):
    """Two calls at once with workspaces of their own, and captured calls replayed on new data: the bits of the plain calls."""
    bs = [batch(q, k, 4, Dn, Dv, seed=s) for s, (q, k) in enumerate((([1] * 8, [900] * 8), ([300, 40], [700, 2000])))]
    want = [attend(b, Dv) for b in bs]
    ws = [torch.empty(hs.hs_mla_expanded_workspace_size(8, Dv), dtype=torch.uint8, device="cuda") for _ in bs]
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    e = err()
    streams = [torch.cuda.Stream() for _ in bs]

    def call(k, stream=None):
        b, (o, l) = bs[k], outs[k]
        hs.hs_mla_expanded_fwd(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], b["scale"], o, e, ws[k], lse=l, stream=stream)

    torch.cuda.synchronize()
    for _ in range(5):
        for k in (0, 1):
            call(k, streams[k])
    torch.cuda.synchronize()
    for (o, l), (a, b) in zip(outs, want):
        assert torch.equal(o, a) and torch.equal(l, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0), call(1), call(0)
    other = batch([1] * 8, [900] * 8, 4, Dn, Dv, seed=77)
    bs[0]["q"].copy_(other["q"]), bs[0]["kv"].copy_(other["kv"]), bs[0]["rope"].copy_(other["rope"])
    again = attend(bs[0], Dv)
    for _ in range(3):
        outs[0][0].zero_(), outs[1][0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], again[0]) and torch.equal(outs[0][1], again[1]) and torch.equal(outs[1][0], want[1][0])
    assert hs.hs_check_flag(e) == 0


def test_calls_one_after_another_wait_for_each_other():
    """Each call starts early and reads what the one before it wrote: rows -> keys and values -> attention -> products, many times over."""
    g = gen(20)
    H, Dn, Dv, n = 8, 128, 128, 640
    c, w, q = plain.rand((n, 576), g).cuda(), plain.weights(H, Dn, Dv, g).cuda(), plain.rand((40, H, Dn + 64), g).cuda()
    start, kv_start = plain.starts([40]).cuda(), plain.starts([n]).cuda()
    e, ws = err(), torch.empty(hs.hs_mla_expanded_workspace_size(1, Dv), dtype=torch.uint8, device="cuda")
    kv, out, lat = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((n, H, Dn + Dv), (40, H, Dv), (40, H, 512)))

    def step(k, sync):
        rows = c * (1.0 + 0.125 * k)
        for call in (lambda: hs.hs_mla_expand(rows[:, :512], w, kv, e), lambda: hs.hs_mla_expanded_fwd(q, kv, rows[:, 512:], start, kv_start, 0.05, out, e, ws),
                     lambda: hs.hs_mla_absorb(out, w, lat, e), lambda: hs.hs_mla_project(lat, w, out, e)):
            call()
            if sync:
                torch.cuda.synchronize()
        return kv.clone(), lat.clone(), out.clone()

    slow = [step(k, True) for k in range(6)]
    fast = [step(k, False) for k in range(6)]
    for a, b in zip(slow, fast):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert hs.hs_check_flag(e) == 0


@pytest.mark.parametrize("Dn,Dv", HEADS)
def test_attention_with_strides_and_without_lse(Dn, Dv):
    """Queries that are slices (also with the heads first in memory), rows of keys and values wider than their heads, no lse: the bits of
    the plain call."""
    b = batch([70, 1, 260], [200, 65, 400], 3, Dn, Dv, seed=15)
    want, _ = attend(b, Dv)
    T, H, D = b["q"].shape
    N = b["kv"].shape[0]
    wide = torch.full((T, H, D + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[..., :D] = b["q"]
    first = torch.empty((H, T, D), dtype=torch.bfloat16, device="cuda")
    first.copy_(b["q"].transpose(0, 1))
    rows = torch.full((N, H * (Dn + Dv) + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    rows[:, :H * (Dn + Dv)] = b["kv"].flatten(1)
    kv = rows[:, :H * (Dn + Dv)].unflatten(1, (H, Dn + Dv))
    e, ws = err(), torch.empty(hs.hs_mla_expanded_workspace_size(3, Dv), dtype=torch.uint8, device="cuda")
    for q in (wide[..., :D], first.transpose(0, 1)):
        out = torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda")
        hs.hs_mla_expanded_fwd(q, kv, b["rope"].contiguous(), b["req_start"], b["kv_start"], b["scale"], out, e, ws)
        assert hs.hs_check_flag(e) == 0 and torch.equal(out, want)
    with pytest.raises(hs.HSError):  # too little workspace
        hs.hs_mla_expanded_fwd(b["q"], b["kv"], b["rope"], b["req_start"], b["kv_start"], b["scale"], out, e, ws[:-1])
    with pytest.raises(hs.HSError):  # values of a head not one after the other
        hs.hs_mla_expanded_fwd(b["q"].transpose(1, 2).contiguous().transpose(1, 2), b["kv"], b["rope"], b["req_start"], b["kv_start"], b["scale"], out, e, ws)
    assert hs.hs_check_flag(e) == 0


def test_rows_past_four_gigabytes():
    """Keys and values whose bytes need more than 32 bits: the last rows of a large call equal those of a small one."""
    g = gen(16)
    N, H, Dn, Dv = 70000, 128, 128, 128
    latent = torch.empty((N, 576), dtype=torch.bfloat16, device="cuda").normal_()
    w = plain.weights(H, Dn, Dv, g).cuda()
    kv, small, e = torch.empty((N, H, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((600, H, 256), dtype=torch.bfloat16, device="cuda"), err()
    assert 2 * kv.numel() > 1 << 32
    hs.hs_mla_expand(latent[:, :512], w, kv, e)
    hs.hs_mla_expand(latent[-600:, :512], w, small, e)
    assert torch.equal(kv[-600:], small)
    q = plain.rand((210, H, 192), g).cuda()
    outs = []
    for m in (10, 200):  # few tokens and many
        ws = torch.empty(hs.hs_mla_expanded_workspace_size(2, Dv), dtype=torch.uint8, device="cuda")
        pair = []
        for rows, r, starts in ((kv, latent, [0, N - 600, N]), (small, latent[-600:], [0, 0, 600])):
            out = torch.empty((m, H, Dv), dtype=torch.bfloat16, device="cuda")
            hs.hs_mla_expanded_fwd(q[:m], rows, r[:, 512:], plain.starts([0, m]).cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"), 0.07, out, e, ws)
            pair.append(out)
        assert torch.equal(*pair)
    # outputs past 2^32 bytes, both products
    T = 33000
    x = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda").normal_()
    assert 2 * x.numel() > 1 << 32
    out, tail = torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"), torch.empty((300, H, Dv), dtype=torch.bfloat16, device="cuda")
    hs.hs_mla_project(x, w, out, e)
    hs.hs_mla_project(x[-300:], w, tail, e)
    assert torch.equal(out[-300:], tail)
    hs.hs_mla_absorb(out, w, x, e)
    back = torch.empty((300, H, 512), dtype=torch.bfloat16, device="cuda")
    hs.hs_mla_absorb(tail, w, back, e)
    assert torch.equal(x[-300:], back) and hs.hs_check_flag(e) == 0


def test_attention_of_many_requests():
    """More requests than the smaller plan takes, up to the most a call may have; most of them small."""
    g = gen(17)
    for B in (512, 513, 4096):
        q_lens = [(1, 0, 2, 1)[r % 4] for r in range(B)]
        kv_lens = [1 + 37 * r % 150 for r in range(B)]
        q_lens[-1], kv_lens[-1] = 5, 2000
        b = batch(q_lens, kv_lens, 1, 128, 128, seed=B)
        out, lse = attend(b, 128)
        some = sorted({0, 1, B // 2, B - 2, B - 1} | {int(x) for x in torch.randint(0, B, (40,), generator=g)})
        for r in some:
            q, k = sum(q_lens[:r]), sum(kv_lens[:r])
            one = dict(q=b["q"][q:q + q_lens[r]], kv=b["kv"][k:k + kv_lens[r]], rope=b["rope"][k:k + kv_lens[r]])
            if q_lens[r]:
                ref, tol, rlse, ltol = plain.attention(one["q"], one["kv"], one["rope"], plain.starts([q_lens[r]]), plain.starts([kv_lens[r]]), 128, b["scale"])
                assert plain.holds(out[q:q + q_lens[r]], ref, tol) and plain.holds(lse[q:q + q_lens[r]], rlse, ltol), r
