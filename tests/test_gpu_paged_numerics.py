"""hs_paged_mla_fwd where 16-bit operands run out of range: queries whose latent part is far below their rotary part, and caches
so long that many small weights count together. Every test runs in all three variants (by rows per request)."""
import math

import pytest
import torch

import plain_ops as plain
from test_gpu_paged_mla import check, run

pytestmark = pytest.mark.gpu

# New tokens of two requests with 16 heads: at most 128 rows per request on average, at most 768, more.
SIZES = {"few": [2, 3], "some": [9, 12], "many": [60, 40]}


def in_size(size, T, B, H):
    rows = T * H
    return {"few": rows <= 128 * B, "some": 128 * B < rows <= 768 * B, "many": rows > 768 * B}[size]


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("latent", [2.0 ** -20, 2.0 ** -60, 2.0 ** -100, 2.0 ** -107, 2.0 ** -112, 2.0 ** -130])
@pytest.mark.parametrize("scale", [1.0 / 24.0, 0.3])
def test_latent_part_far_below_the_rotary_part(size, latent, scale):
    """The power of two that brings a row's latent values into fp16's range scales its rotary values too: ordinary ones must
    neither overflow nor lose their way back. Ordinary rows stand beside the small ones."""
    b = plain.make_batch(SIZES[size], [300, 130], 16, seed=31, sigma_q=2.0)
    assert in_size(size, sum(SIZES[size]), 2, 16)
    b["q"][:, ::3, :512] = (b["q"][:, ::3, :512].double() * latent).bfloat16()
    assert bool(b["q"][:, ::3, :512].any())
    b["scale"] = scale
    check(b)


@pytest.mark.parametrize("size", list(SIZES))
def test_small_parts_under_a_large_scale(size):
    """Both parts tiny, the softmax scale as large: the logits are of order one and either part shows in them."""
    b = plain.make_batch(SIZES[size], [300, 130], 16, seed=32)
    b["q"][..., :512] = (b["q"][..., :512].double() * 2.0 ** -100).bfloat16()
    b["q"][..., 512:] = (b["q"][..., 512:].double() * 2.0 ** -97).bfloat16()
    b["scale"] = 2.0 ** 96
    check(b)


@pytest.mark.parametrize("size", list(SIZES))
def test_many_small_weights(size):
    """The first row has nearly all the weight and a latent part of zeros; each of the others has 2^-25.25 of it, together 0.65 %,
    and ones. Enough requests that a block's rows are not spread over all SMs. All pages after the first are one page."""
    H, n = 16, 1 << 18
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m, B = {"few": (4, sms), "some": (16, sms // 4), "many": (64, sms // 16)}[size]
    assert in_size(size, m * B, B, H)
    rows = torch.zeros((128, 656), dtype=torch.uint8)
    rows[1:, :512] = 0x38                                                                  # 1.0
    rows[:, 512:528] = torch.ones((128, 4)).view(torch.uint8)
    rows[0, 528:530] = torch.tensor([25.25], dtype=torch.bfloat16).view(torch.uint8)
    table = torch.ones((B, n // 64), dtype=torch.int32)
    table[:, 0] = 0
    q = torch.zeros((m * B, H, 576), dtype=torch.bfloat16)
    q[..., 512] = 1.0
    b = dict(q=q.cuda(), pool=rows.cuda(), table=table.cuda(), kv_tokens=B * n, scale=math.log(2.0),
             req_start=(torch.arange(B + 1, dtype=torch.int32) * m).cuda(), seq_len=torch.full((B,), n, dtype=torch.int32).cuda())
    out, lse, flag = run(b, causal=False)
    assert flag == 0
    tail = (n - 1) * 2.0 ** -25.25
    want = tail / (1.0 + tail)
    # a weight is off by half of fp16's smallest step, 2^-25, of a reference held 2^7 above one; sums over 2^12 pages
    # and the result's rounding: 2^-12 and 2^-8 of the value
    assert float((out.double() - want).abs().max()) <= want * (2.0 ** -8 + 2.0 ** -12) + n * 2.0 ** -32
    assert float((lse.double() - math.log(2.0 ** 25.25 + n - 1)).abs().max()) <= 2.0 ** -12 + 2.0 ** -20 * 17.5


@pytest.mark.parametrize("m", [1, 16])
def test_longest_length(m):
    """2^31 - 64 cached rows, the most that a table of 2^25 - 1 pages holds (here one page, over and over): tiles count up to the
    last row. All rows are alike, and their values powers of two, so that sums stay exact."""
    H, n = 16, 2 ** 31 - 64
    g = torch.Generator().manual_seed(33)
    row = torch.zeros(656, dtype=torch.uint8)
    value = torch.randint(-3, 4, (512,), generator=g)
    latent = torch.ldexp(torch.where(torch.rand(512, generator=g) < 0.5, -1.0, 1.0), value)
    row[:512] = latent.to(torch.float8_e4m3fn).view(torch.uint8)
    row[512:528] = torch.ones(4).view(torch.uint8)
    row[528:] = torch.full((64,), 0.5, dtype=torch.bfloat16).view(torch.uint8)
    b = dict(q=torch.randn((m, H, 576), generator=g).bfloat16().cuda(), pool=row.expand(64, 656).contiguous().cuda(),
             table=torch.zeros((1, n // 64), dtype=torch.int32, device="cuda"), kv_tokens=n, scale=1.0 / 24.0,
             req_start=torch.tensor([0, m], dtype=torch.int32, device="cuda"),
             seq_len=torch.tensor([n], dtype=torch.int32, device="cuda"))
    out, lse, flag = run(b, causal=False)
    assert flag == 0
    want = latent.double().cuda()
    assert bool(((out.double() - want).abs() <= want.abs() * 2.0 ** -8).all())
    logit = (b["q"].double() @ torch.cat([want, torch.full((64,), 0.5, device="cuda", dtype=torch.float64)])) / 24.0
    assert float((lse.double() - logit - math.log(n)).abs().max()) <= 2.0 ** -11
