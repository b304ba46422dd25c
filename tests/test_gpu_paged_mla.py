"""hs_paged_mla_fwd against 64-bit attention, one request at a time. The unused rows of every pool are poisoned."""
import math

import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain

pytestmark = pytest.mark.gpu


def run(b, causal=True, lse=True, stream=None):
    T, H, _ = b["q"].shape
    B = b["table"].shape[0]
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((T, H), 7.0, device="cuda") if lse else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((hs.hs_paged_mla_workspace_size(T, B, H, b["kv_tokens"]),), 0xFF, dtype=torch.uint8, device="cuda")
    hs.hs_paged_mla_fwd(b["q"], b["pool"], b["table"], b["req_start"], b["seq_len"], b["kv_tokens"], b["scale"], out, err, ws,
                        lse=l, causal=causal, stream=stream)
    return out, l, hs.hs_check_flag(err, stream=stream)


def check(b, causal=True, flag=0):
    out, lse, got = run(b, causal)
    assert got == flag
    ref, rlse, spread, delta = plain.paged_attention(b["q"], b["pool"], b["table"], b["req_start"], b["seq_len"], b["scale"], causal)
    tol, ltol = plain.attention_bound(ref, spread, delta, rlse)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))
    empty = rlse == -math.inf
    assert torch.equal(empty, lse == -math.inf) and not out[empty].any()
    assert bool(((lse.double() - rlse).abs()[~empty] <= ltol[~empty]).all())
    norm = float(ref.norm())
    assert norm == 0 or float((out.double() - ref).norm()) / norm <= 5e-3   # what the roundings come to at random
    return out, lse


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 500])
@pytest.mark.parametrize("H", [1, 64])
def test_one_token(n, H):
    check(plain.make_batch([1], [n], H, seed=n))


@pytest.mark.parametrize("H", [2, 3, 16, 24, 100, 128])
def test_heads(H):
    check(plain.make_batch([5, 1, 9], [70, 200, 9], H, seed=H))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,kv", [([4, 4, 4], [300, 4, 129]), ([0, 3, 0, 1, 0], [50, 3, 0, 1, 10]), ([5, 2, 7], [2, 0, 3]), ([300], [300]), ([130, 1, 33], [1000, 700, 33])])
def test_ragged(q, kv, causal):
    check(plain.make_batch(q, kv, 16, seed=sum(kv)), causal)


def test_requests_alone_in_split_work():
    """One token over many tiles: every cluster takes a share and the parts are joined."""
    check(plain.make_batch([1], [30_001], 64, seed=1))
    check(plain.make_batch([1, 1, 1], [9000, 3, 20_000], 8, seed=2))


def test_chunk_of_many_blocks():
    check(plain.make_batch([150], [1500], 64, seed=3))


def test_many_requests():
    check(plain.make_batch([1 + (i % 3) for i in range(230)], [3 + (i * 37) % 200 for i in range(230)], 8, seed=4))


@pytest.mark.parametrize("sigma", [1e-30, 1e-5, 4.0, 3e4])
def test_query_magnitudes(sigma):
    b = plain.make_batch([3, 1], [200, 90], 16, seed=5, sigma_q=sigma)
    b["q"][1, 3] *= 2.0 ** 20 if sigma < 1 else 1.0
    if sigma > 100:
        b["scale"] /= sigma
    check(b)


@pytest.mark.parametrize("scale", [0.0, -1.0 / 24.0, 0.5])
def test_scales(scale):
    b = plain.make_batch([3, 2], [300, 65], 16, seed=6, sigma_q=0.5)
    b["scale"] = scale
    check(b)


def test_rising_logits_move_the_maximum():
    """Keys whose logits grow along the context: the reference maximum moves tile after tile."""
    b = plain.make_batch([2], [2000], 16, seed=7)
    rows = b["table"][0].long()[torch.arange(2000, device="cuda") // 64] * 64 + torch.arange(2000, device="cuda") % 64
    ramp = (torch.arange(2000, device="cuda") / 50.0)[:, None].expand(2000, 64)
    b["pool"][rows, 528:] = ramp.bfloat16().contiguous().view(torch.uint8)
    b["q"][..., 512:] = 1.0
    check(b)


def test_rows_that_a_token_does_not_see_never_reach_it():
    """A NaN code in the last row: only the last token of the chunk sees it."""
    b = plain.make_batch([4], [200], 16, seed=8)
    clean = run(b)[0]
    row = int(b["table"][0, 199 // 64]) * 64 + 199 % 64
    b["pool"][row, 17] = 0x7F
    out, lse, flag = run(b)
    assert torch.equal(out[:3], clean[:3]) and bool(out[3].isnan().all()) and bool(lse[3].isnan().all())
    # an infinite scale instead: flagged, and the other tokens keep their results
    b["pool"][row, 17] = 0x38
    b["pool"][row, 512:516] = torch.tensor([math.inf]).view(torch.uint8).cuda()
    out, lse, flag = run(b)
    assert torch.equal(out[:3], clean[:3]) and flag == hs.FLAGS["RANGE"]
    # an infinite or NaN rotary value
    for v in (math.inf, math.nan):
        b["pool"][row, 512:516] = torch.tensor([1.0]).view(torch.uint8).cuda()
        b["pool"][row, 528:530] = torch.tensor([v], dtype=torch.bfloat16).view(torch.uint8).cuda()
        assert torch.equal(run(b)[0][:3], clean[:3])


def test_not_a_number_in_a_query_stays_in_its_row():
    b = plain.make_batch([3], [100], 16, seed=9)
    clean = run(b)[0]
    b["q"][1, 5, 100] = math.nan
    out, _, flag = run(b)
    assert flag == hs.FLAGS["RANGE"] and bool(out[1, 5].isnan().all())
    out[1, 5] = clean[1, 5]
    assert torch.equal(out, clean)


def test_bad_blocks_and_lengths_are_told():
    b = plain.make_batch([2, 2], [200, 300], 16, seed=10)
    clean = run(b)[0]
    table = b["table"].clone()
    b["table"][0, 1] = -1
    out, _, flag = run(b)
    assert flag == hs.FLAGS["BAD_BLOCK"] and torch.equal(out[2:], clean[2:]) and bool(out.isfinite().all())
    b["table"][0, 1] = b["pool"].shape[0] // 64
    assert run(b)[2] == hs.FLAGS["BAD_BLOCK"]
    b["table"] = table
    b["seq_len"][0] = table.shape[1] * 64 + 1
    out, lse, flag = run(b)
    assert flag & hs.FLAGS["BAD_LENGTH"] and not out[:2].any() and torch.equal(out[2:], clean[2:])
    b["seq_len"][0] = 200
    b["req_start"][1] = 5
    assert run(b)[2] & hs.FLAGS["BAD_INDEX"]


def test_same_bits_each_time_streams_and_graph():
    b = plain.make_batch([1, 40, 4], [5000, 900, 64], 64, seed=11)
    want, wl, _ = run(b)
    for _ in range(3):
        out, l, _ = run(b)
        assert torch.equal(out, want) and torch.equal(l, wl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, l, _ = run(b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    T, H, _ = b["q"].shape
    ws = torch.empty(hs.hs_paged_mla_workspace_size(T, 3, H, b["kv_tokens"]), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_paged_mla_fwd(b["q"], b["pool"], b["table"], b["req_start"], b["seq_len"], b["kv_tokens"], b["scale"], out, err, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_agrees_with_sparse_attention_over_every_row():
    b = plain.make_batch([1, 1], [300, 2048], 64, seed=12)
    out, lse = check(b)
    idx = torch.arange(2048, dtype=torch.int32, device="cuda").repeat(2, 1)
    idx[0, 300:] = -1
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.hs_sparse_mla_fwd(b["q"], b["pool"], idx, b["scale"], o2, err, lse=l2, block_table=b["table"],
                         token_req=torch.arange(2, dtype=torch.int32, device="cuda"))
    assert hs.hs_check_flag(err) == 0
    assert float((out.double() - o2.double()).norm() / out.double().norm()) <= 5e-3 and float((lse - l2).abs().max()) <= 2e-3


def test_far_rows_pass_32_bits():
    """Pages at the end of a 4.4 GB pool."""
    b = plain.make_batch([2], [200], 16, seed=13)
    want = run(b)[0]
    nblk, have = 105_000, b["pool"].shape[0] // 64
    pool = torch.zeros((nblk * 64, 656), dtype=torch.uint8, device="cuda")
    pool[-have * 64:] = b["pool"]
    b["pool"] = pool
    b["table"] = torch.where(b["table"] >= 0, b["table"] + (nblk - have), -1)
    out, _, flag = run(b)
    assert flag == 0 and torch.equal(out, want)


# Batches by (token, head) rows per request on average, here with two requests: few (at most 128), some (at most 768), many (the
# cached rows are dequantised first). Tests that add requests run in another variant; see test_gpu_paged_rule.py.
SIZES = {"few": [2, 3], "some": [9, 12], "many": [60, 40]}


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("causal", [True, False])
def test_sizes(size, causal):
    for kv in ([700, 90], [64, 128], [129, 5000]):
        check(plain.make_batch(SIZES[size], kv, 16, seed=20 + sum(kv)), causal)


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_masked_values_never_reach_a_row(size):
    """What only a request's last token sees: a NaN code, an infinite scale, infinite and NaN rotary values."""
    m = SIZES[size]
    b = plain.make_batch(m, [200, 300], 16, seed=21)
    clean, last = run(b)[0], m[0] - 1
    row = int(b["table"][0, 199 // 64]) * 64 + 199 % 64
    keep = b["pool"][row].clone()
    for at, value, flag in ((slice(17, 18), torch.tensor([0x7F], dtype=torch.uint8), 0),
                            (slice(512, 516), torch.tensor([math.inf]).view(torch.uint8), hs.FLAGS["RANGE"]),
                            (slice(528, 530), torch.tensor([math.inf], dtype=torch.bfloat16).view(torch.uint8), 0),
                            (slice(528, 530), torch.tensor([math.nan], dtype=torch.bfloat16).view(torch.uint8), 0)):
        b["pool"][row] = keep
        b["pool"][row, at] = value.cuda()
        out, _, got = run(b)
        others = torch.arange(sum(m), device="cuda") != last
        assert got == flag and torch.equal(out[others], clean[others])
        if at.start == 17 or bool(torch.isnan(b["pool"][row, 528:530].view(torch.bfloat16)).any()):
            assert bool(out[last].isnan().all())


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_bad_pages_and_lengths(size):
    m = SIZES[size]
    b = plain.make_batch(m, [200, 300], 16, seed=22)
    clean, table = run(b)[0], b["table"].clone()
    for bad in (-1, b["pool"].shape[0] // 64, 2 ** 31 - 1):
        b["table"][0, 1] = bad
        out, lse, flag = run(b)
        assert flag == hs.FLAGS["BAD_BLOCK"] and torch.equal(out[m[0]:], clean[m[0]:])
        assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    b["table"] = table
    b["seq_len"][0] = -1
    out, lse, flag = run(b)
    assert flag & hs.FLAGS["BAD_LENGTH"] and not out[:m[0]].any() and bool((lse[:m[0]] == -math.inf).all())
    assert torch.equal(out[m[0]:], clean[m[0]:])


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_more_cached_rows_than_told(size):
    """kv_tokens bounds the sum of the lengths (the workspace is sized by it): a batch beyond it is flagged, nothing is computed."""
    b = plain.make_batch(SIZES[size], [200, 300], 16, seed=23)
    b["kv_tokens"] = 499
    out, lse, flag = run(b)
    assert flag == hs.FLAGS["BAD_LENGTH"] and bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_workspace_too_small(size):
    b = plain.make_batch(SIZES[size], [200, 300], 16, seed=24)
    T, H, _ = b["q"].shape
    out, err = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(hs.hs_paged_mla_workspace_size(T, 2, H, b["kv_tokens"]) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(hs.HSError, match="workspace"):
        hs.hs_paged_mla_fwd(b["q"], b["pool"], b["table"], b["req_start"], b["seq_len"], b["kv_tokens"], b["scale"], out, err, ws)


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("scale", [0.0, -1.0 / 24.0])
def test_sizes_scales_and_queries(size, scale):
    b = plain.make_batch(SIZES[size], [300, 65], 16, seed=25, sigma_q=0.5)
    b["scale"] = scale
    check(b)
    b = plain.make_batch(SIZES[size], [300, 65], 16, seed=26, sigma_q=3e4)
    b["scale"] = 1.0 / 24.0 / 3e4
    b["q"][1, 3] *= 2.0 ** -20
    check(b)
    clean = run(b)[0]
    b["q"][1, 5, 100] = math.inf
    out, _, flag = run(b)
    assert flag == hs.FLAGS["RANGE"]
    out[1, 5] = clean[1, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_same_bits_each_time(size):
    """One request over many tiles: every share of the work is a part, and the parts are joined in their order."""
    m = SIZES[size]
    b = plain.make_batch([m[0], 0, m[1]], [20_000, 0, 5000], 16, seed=27)
    want, lse, _ = run(b)
    for _ in range(3):
        out, l, flag = run(b)
        assert flag == 0 and torch.equal(out, want) and torch.equal(l, lse)
    assert torch.equal(run(b, lse=False)[0], want)
    check(b)


@pytest.mark.parametrize("H", [8, 64])
def test_many_short_requests_again_and_again(H):
    """Several blocks of one to four pages per SM, many times over: what is not ordered shows as bits that change."""
    b = plain.make_batch([1 + (i % 3) for i in range(230)], [3 + (i * 37) % 200 for i in range(230)], H, seed=4)
    want, lse = check(b)
    for _ in range(150):
        out, l, flag = run(b)
        assert flag == 0 and torch.equal(out, want) and torch.equal(l, lse)
