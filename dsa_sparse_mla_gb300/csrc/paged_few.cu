// paged_few.cu — dense attention over paged FP8 latent rows for requests with few (token, head) rows (decode): the formulas of
// paged.cu on one SM per block of 64 rows.
//
//   S = Q K^T (M = 64 rows, N = 64 cached rows, 36 MMAs),  P = 2^(c S - m),
//   O^T += V^T P^T (M = 128 dims x 4, N = 64 rows, 16 MMAs)
//
// Why not 128 or 256 rows as in paged.cu: a request has only 64, and each SM pays for dequantising every cached row that it
// visits; with O transposed, O^T of 64 rows takes 256 of the tensor memory's columns, so S (two buffers of 64 columns) and
// half of Q (128 columns) fit beside it and nothing crosses SMs.
//
// Work. Persistent, one CTA per SM; units as in paged.cu (block of rows, 128 cached rows), shared out evenly, split blocks joined
// by paged_merge_kernel. Inside a unit the step is one page (64 cached rows).
//
// Shared memory: Q's other half (five blocks of [64 rows][64 dims], 128-byte swizzle), two pages dequantised (nine blocks
// each), one page as it lies in the pool.
//
// Roles (768 threads; warp w runs on sub-partition w % 4). Warp 16 brings a page by one bulk copy, with the next one asked into
// L2. Warps 1-3, 5-7, 12-15, 17-19 and 21-23 are the producers: each takes four rows into registers, so that the next
// page can land, and writes them as fp16 (code * group scale, rounded once), in two halves of the dims that QK starts on as
// soon as every producer has written one; PV gives them back in halves too. Warp 0 issues QK (Q's first 256 dims from
// tensor memory as a 128-row A of which 64 lanes are rows, the rest from shared memory), warp 4 PV. Warps 8-11 are the
// softmax, 16 rows each, two threads per row with 32 columns each (what a 64-row product leaves in tensor memory);
// they also load Q, rescale and write O^T. P goes into the page's rotary block, which QK has read by then.
//
// Lazy maximum and masks as in paged.cu: a row's reference moves only when a logit passes it by more than 2^8; one OR-barrier
// per page tells the softmax warps, which then rescale O^T's columns. A latent value that is NaN or cannot be fp16 is zeroed
// and its row's rotary values become NaN: rows that see it are NaN, P = 0 times it stays 0.
//
// Measured on a GB300 (events, inputs far larger than L2): 32 requests x 64 heads over 30-131 thousand rows 546 to 556 us,
// 3,330 GB/s of cache, 0.50 of a plain copy's rate; about 3,800 cycles per page. The chain fill -> QK -> softmax -> PV of a page's slot sets
// that pace (two slots); at 4,170 cycles it took 3,150 without the MMAs and 3,800 without the producers' arithmetic. On
// the way: eight producer warps 5,450 cycles; rows loaded straight into registers 4,600 (4,430 in one batch per
// page: the loads seem to wait for each other); four hand-overs per page 4,750. 8 requests over 200-2,000 rows 28 us: about 2 us until
// the shares are known, 5 for Q, 2 to 3 per page, 4 for the partial results (7 with 4-byte stores), the rest launches and the join.
#include "paged.cuh"

namespace hs {
namespace paged {
namespace few {

constexpr int kRows = 64, kPageKeys = HS_PAGE;
constexpr int kThreads = 768;
constexpr int kPvWarp = 4, kLoadWarp = 16, kSmWarp0 = 8, kProducers = 16;
constexpr int kBlk = kPageKeys * 128;          // [64][64 dims] of 16 bits
constexpr int kTile = 9 * kBlk;
constexpr int kOffQ = 0;                       // Q's dims 256 .. 575: five blocks
constexpr int kOffTile = 5 * kBlk;
constexpr int kOffScratch = kOffTile;          // int64 [B + 1] and int32 [B + 1] during the set-up
constexpr int kOffRaw = kOffTile + 2 * kTile;  // a page as it lies in the pool: four rows per producer
constexpr int kRawRows = 4 * HS_KV_ROW_BYTES;
constexpr int kOffRow = kOffRaw + kProducers * kRawRows;  // [64] each: factors, 1 / sums, Q's largest values and scales
constexpr int kOffBar = kOffRow + 4 * 256;
struct Bars {
  uint64_t full[2][2];   // producers have written a half of a page's dims -> QK
  uint64_t free[2][2];   // PV has read a half (the second: and P) -> producers, softmax
  uint64_t wide_done;    // a page's 128-row products of QK are complete (its issuer's own)
  uint64_t s_full[2];    // S complete -> softmax
  uint64_t s_empty[2];   // S read -> QK
  uint64_t p_full[2];    // P written, O^T rescaled -> PV
  uint64_t q_ready;      // a block's Q is in place -> QK
  uint64_t drain[2];
  uint64_t raw_full;     // a page's codes have landed -> producers
  uint64_t raw_free;     // they have read them
};
constexpr int32_t kEnd = -1;
struct Misc {
  uint32_t tmem;
  volatile uint32_t abort;
  int32_t left;          // rows in use of the page that has landed; kEnd after the last one
  Start start;
};
constexpr int kOffMisc = kOffBar + (int)sizeof(Bars);
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448 && 12 * (kMaxReq + 1) <= 2 * kTile && kOffBar % 8 == 0 && kOffMisc % 8 == 0, "shared memory");
// Tensor memory columns: O^T 0 .. 255, S buffers, Q's dims 0 .. 255 as pairs. Row r of Q and S is in lane
// 32 (r / 16) + r % 16, where a 64-row product has it; the other lanes belong to no row.
constexpr int kColS = 256, kColQ = 384;

// Index of warp w among the producers, or -1.
__host__ __device__ constexpr int producer_index(int w) {
  return w == 12 ? 15 : w % 4 == 0 || (w >= 8 && w < 12) ? -1 : (w < 8 ? w / 4 : w / 4 - 1) * 3 + w % 4 - 1;
}

// Pages [first, end) of a segment: the last tile of a block may need only its first page.
__device__ __forceinline__ int first_page(const Seg& s) { return 2 * s.ta; }
__device__ __forceinline__ int end_page(const Params& p, const Seg& s) {
  const int n = sees<kRows>(p, s.q, (int64_t)s.b * kRows + s.nrows - 1);
  const int pages = n > 0 ? (int)(((uint32_t)n + kPageKeys - 1) / kPageKeys) : 1;
  return 2 * s.tb < pages ? 2 * s.tb : pages;
}

// A CTA's pages in order.
struct Page {
  int32_t blk;  // block-table entry, -1 where there is none
  int left;     // cached rows from its first key on
  bool live;
};
struct Pages {
  Walk<kRows> walk;
  Seg s;
  int j, end;
  __device__ __forceinline__ Pages(const Params& p, const Start& st) : walk(p, st), j(0), end(0) {}
  __device__ __forceinline__ Page next(const Params& p) {
    Page g = {-1, 0, false};
    if (j == end) {
      if (!walk.next(p, s)) return g;
      j = first_page(s);
      end = end_page(p, s);
    }
    g.live = true;
    g.left = s.q.seq - j * kPageKeys;
    if (j < p.bt_stride) g.blk = ldg_nc_s32(p.bt + (int64_t)s.r * p.bt_stride + j);
    ++j;
    return g;
  }
};

// A producer lane's part of a page: of row 4 w + l / 8, of every group the codes 8 (l % 8) .. + 7 and 64 further (so that the
// eight lanes of a row store its eight 16-byte pieces of a block at once, in different banks), the four scales and 16
// bytes of the rotary values.
struct Raw {
  uint2 code[4][2];
  uint4 rope, scale;
};

// Whether one of 16 codes is NaN (0x7F, 0xFF).
__device__ __forceinline__ bool has_nan(const uint2& a, const uint2& b) {
  const uint32_t m = 0x7F7F7F7Fu, o = 0x01010101u;
  return ((((a.x & m) + o) | ((a.y & m) + o) | ((b.x & m) + o) | ((b.y & m) + o)) & 0x80808080u) != 0u;
}

// Stores what tmem_ld16x2_32 reads, 16 columns to a half: thread i < 16 lane (base + i), columns [c, c + 16), thread i >= 16
// lane (base + i - 16), columns [c + 16, c + 32).
__device__ __forceinline__ void tmem_st16x2_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], 16, {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A from tensor memory (two 16-bit values to a column, row = lane).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
               "l"(b), "r"(idesc), "r"(accumulate));
}

__global__ void __launch_bounds__(kThreads, 1) few_kernel(const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  Bars& br = *reinterpret_cast<Bars*>(smem + kOffBar);
  Misc& mc = *reinterpret_cast<Misc*>(smem + kOffMisc);
  float* alpha = reinterpret_cast<float*>(smem + kOffRow);
  float* inverse = alpha + 64;
  uint32_t* largest = reinterpret_cast<uint32_t*>(alpha + 128);
  float* scales = alpha + 192;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  let_next();
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      for (int g = 0; g < 2; ++g) mbar_init(&br.full[s][g], kProducers);
      for (int g = 0; g < 2; ++g) mbar_init(&br.free[s][g], 1);
      mbar_init(&br.s_full[s], 1);
      mbar_init(&br.s_empty[s], 4);
      mbar_init(&br.p_full[s], 4);
      mbar_init(&br.drain[s], 1);
    }
    mbar_init(&br.q_ready, 4);
    mbar_init(&br.wide_done, 1);
    mbar_init(&br.raw_full, 1);
    mbar_init(&br.raw_free, kProducers);
    mbar_fence_init();
    mc.abort = 0;
  }
  find_units<kRows>(p, reinterpret_cast<int64_t*>(smem + kOffScratch), &mc.start, c, kThreads);
  fence_proxy_async_smem();
  if (warp == 0) tmem_alloc(&mc.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mc.tmem;
  const Start& st = mc.start;
  const int pw = producer_index(warp);

  // 768 threads start with 80 registers each (61,440 in all); the softmax warps (128 threads) take 120, the others keep 72:
  // 61,440
  if (warp >= kSmWarp0 && warp < kSmWarp0 + 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ================================================================ softmax, output ===========
    const int quad = warp & 3, half = lane >> 4, row = 16 * quad + (lane & 15);  // half: columns 32 half .. + 31
    const uint32_t quarter = tmem + ((uint32_t)(32 * quad) << 16);
    const int64_t U = st.U, C = U < p.clusters ? U : p.clusters;
    Desc desc = {0, 0, 0, 0};
    int64_t cost = st.cost;  // of the blocks before this one
    Walk<kRows> walk(p, st);
    Seg s;
    int i = 0;
    bool ok = true;
#pragma unroll 1
    while (walk.next(p, s)) {  // to the end even after a failure: the four warps meet at barriers
      const int64_t row0 = (int64_t)s.q.start * p.H + (int64_t)s.b * kRows;
      if (s.ta == 0 && s.tb < s.tiles) {
        desc.row0 = (int32_t)row0;
        desc.nrows = s.nrows;
        desc.nparts = (int32_t)(unit_cta(cost + s.tiles + kBlockCost - 1, U, C) - c + 1);
      }
      if (s.tb == s.tiles) cost += s.tiles + kBlockCost;
      const bool idle = 16 * quad >= s.nrows, mine = row < s.nrows;
      // Q: the block before has been read (its last S is complete). Rows past the block's are read as its first row. A row
      // whose largest latent value is outside [2^-6, 2^15) is scaled by a power of two that puts it in [2^14, 2^15) and its
      // logits are scaled back: rare, so the values are converted as they are first, and again if need be.
      float coef = 1.f;
      if (!idle) {
        const uint8_t* q0 = p.q + row0 * (HS_D_QK * 2);
        auto row_at = [&](int r) { return q0 + (int64_t)(r < s.nrows ? r : 0) * (HS_D_QK * 2); };
        // everything this warp reads, asked for at once (nine lines a row)
#pragma unroll 1
        for (int k = lane; k < 16 * 9; k += 32) prefetch_l2(row_at(16 * quad + k / 9) + 128 * (k % 9));
        auto scaled = [&](uint32_t w, float f, bool half16) -> uint32_t {
          const uint32_t u = w ^ p.flip;
          const float a = __uint_as_float(u << 16) * f, b = __uint_as_float(u & 0xFFFF0000u) * f;
          if (half16) return pack_half2(a, b);
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
          return *reinterpret_cast<const uint32_t*>(&b2);
        };
        const uint8_t* own = row_at(row) + 64 * half;
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          // dims 64 h + 32 half .. + 31 of this thread's row to tensor memory
          const float own_scale = pass ? scales[row] : 1.f;
          uint32_t mx = 0u;
#pragma unroll 1
          for (int h = 0; h < 4; h += 2) {
            uint4 v[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) v[e][k] = ldg_nc_v4(own + 128 * (h + e) + 16 * k);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[4 * k] = v[e][k].x, w[4 * k + 1] = v[e][k].y, w[4 * k + 2] = v[e][k].z, w[4 * k + 3] = v[e][k].w;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                mx = __vmaxu2(mx, w[k] & 0x7FFF7FFFu);
                w[k] = scaled(w[k], own_scale, true);
              }
              tmem_st16x2_16(quarter + kColQ + 32 * (h + e), w);
            }
          }
          // the rest to shared memory, four rows of 64 dims per load
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            const int r = 16 * quad + 4 * h + (lane >> 3);
            const uint8_t* src = row_at(r) + 512 + 16 * (lane & 7);
            const float f = pass ? scales[r] : 1.f;
            uint4 v[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) v[k] = ldg_nc_v4(src + 128 * k);
            uint32_t m = 0u;
#pragma unroll
            for (int k = 0; k < 5; ++k) {
              if (k < 4)
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu)));
              *reinterpret_cast<uint4*>(smem + kOffQ + k * kBlk + sw128_offset(r, 16 * (lane & 7))) =
                  make_uint4(scaled(v[k].x, f, k < 4), scaled(v[k].y, f, k < 4), scaled(v[k].z, f, k < 4), scaled(v[k].w, f, k < 4));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((lane & 7) == 0) largest[r] = m;
          }
          if (pass) break;
          __syncwarp();
          mx = __vmaxu2(__vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 16)), largest[row]);
          const uint32_t amax = max(mx & 0xFFFFu, mx >> 16);
          int e = 0;
          if (amax >= 0x7F80u) {
            if (mine) flag_error(p.err, HS_FLAG_RANGE);
          } else if (amax >= 0x4700u || (amax >= 0x0080u && amax < 0x3C80u)) {
            e = 14 - ((int)(amax >> 7) - 127);
          } else if (amax > 0u && amax < 0x0080u) {
            e = 126;
          }
          e = e < -126 ? -126 : (e > 126 ? 126 : e);
          if (__any_sync(0xffffffffu, e > 0)) {  // rare: the rotary values go along
            uint32_t m = 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 v = ldg_nc_v4(own + 1024 + 16 * k);
              m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 16));
            e = query_exponent(e, max(m & 0xFFFFu, m >> 16));
          }
          // not 0, so that a masked column stays -inf (softmax scales next to 0, or rows that are tiny in both parts: their
          // logits stay below 2^-60 and do not show)
          coef = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 7.5e-37f);
          if (!__any_sync(0xffffffffu, e != 0)) break;
          if (half == 0) scales[row] = __uint_as_float((uint32_t)(e + 127) << 23);
          tmem_wait_st();
          __syncwarp();
        }
        tmem_wait_st();
        tc_fence_before();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&br.q_ready);

      const int nsee = mine ? sees<kRows>(p, s.q, (int64_t)s.b * kRows + row) : 0;
      const int first = first_page(s), end = end_page(p, s);
      const int32_t* bt = p.bt + (int64_t)s.r * p.bt_stride;
      int32_t next_k = ldg_nc_s32(bt + (first < p.bt_stride ? first : 0));
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = first; j < end; ++j, ++i) {
        const int b = i & 1;
        const uint32_t ph = (uint32_t)(i >> 1) & 1u;
        const int32_t k = next_k;  // this page's entry, read a page ahead
        next_k = ldg_nc_s32(bt + (j + 1 < p.bt_stride ? j + 1 : 0));
        // a warp that gives up still comes to the barriers, so that the others do not wait there
        bool here = ok && !mc.abort && warp_wait_all(&br.s_full[b], ph, p.err);
        if (!here) mc.abort = 1;
        tc_fence_after();
        uint32_t x[32];
        tmem_ld16x2_32(quarter + kColS + 64 * b, x);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.s_empty[b]);
        const bool there = j < p.bt_stride && k >= 0 && ((int64_t)k + 1) * HS_PAGE <= p.R;
        const int lim = there ? nsee - j * kPageKeys - 32 * half : 0;  // columns that this thread's row sees
        if (!__all_sync(0xffffffffu, lim >= 32)) {
#pragma unroll
          for (int z = 0; z < 32; ++z) x[z] = z < lim ? x[z] : 0xFF800000u;
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int z = 0; z < 32; z += 2) m0 = fmaxf(m0, __uint_as_float(x[z])), m1 = fmaxf(m1, __uint_as_float(x[z + 1]));
        float top = fmaxf(m0, m1);
        top = top == -INFINITY ? top : top * coef;
        if (named_bar_or(1, 128, top > ref + kThreshold)) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const bool up = top > ref + kThreshold;
          const float to = up ? top : ref;
          const float al = up ? fast_exp2(ref - to) : 1.f;
          l *= al;
          ref = to;
          if (j > first) {
            if (half == 0) alpha[row] = al;
            here = here && warp_wait_all(&br.free[b ^ 1][1], (uint32_t)((i - 1) >> 1) & 1u, p.err);  // PV so far is complete
            if (!here) mc.abort = 1;
            named_bar(2, 128);
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 8; ++h) {  // 32 of a group's 64 columns (rows of the block)
              if (32 * (h & 1) >= s.nrows) continue;
              uint32_t o[32];
              tmem_ld32(quarter + 32 * h, o);
              tmem_wait_ld();
#pragma unroll
              for (int z = 0; z < 32; z += 4) {
                const float4 a = *reinterpret_cast<const float4*>(alpha + 32 * (h & 1) + z);
                o[z] = __float_as_uint(__uint_as_float(o[z]) * a.x);
                o[z + 1] = __float_as_uint(__uint_as_float(o[z + 1]) * a.y);
                o[z + 2] = __float_as_uint(__uint_as_float(o[z + 2]) * a.z);
                o[z + 3] = __float_as_uint(__uint_as_float(o[z + 3]) * a.w);
              }
              tmem_st32(quarter + 32 * h, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        if (!idle) {
          const float me = ref == -INFINITY ? 0.f : ref - kLift;
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int z = 0; z < 16; ++z) {
            const float a = fast_exp2(fmaf(__uint_as_float(x[2 * z]), coef, -me));
            const float d = fast_exp2(fmaf(__uint_as_float(x[2 * z + 1]), coef, -me));
            s0 += a;
            s1 += d;
            x[z] = pack_half2(a, d);
          }
          l += s0 + s1;
          uint8_t* pb = smem + kOffTile + b * kTile + 8 * kBlk;
#pragma unroll
          for (int z = 0; z < 4; ++z)
            *reinterpret_cast<uint4*>(pb + sw128_offset(row, 64 * half + 16 * z)) =
                make_uint4(x[4 * z], x[4 * z + 1], x[4 * z + 2], x[4 * z + 3]);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.p_full[b]);
        ok = here;
      }
      // the block's result
      const float sum = l + __shfl_xor_sync(0xffffffffu, l, 16);
      const bool whole = s.ta == 0 && s.tb == s.tiles;
      const int64_t part = 2 * c + (s.ta == 0 ? 1 : 0);
      if (half == 0) {
        inverse[row] = sum == 0.f ? 0.f : 1.f / sum;
        if (mine) {
          const float z = sum == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref - kLift) + log2f(sum)) * kLn2;
          if (!whole)
            p.part_lse[part * kRows + row] = z;
          else if (p.lse)
            p.lse[row0 + row] = z;
        }
      }
      const bool done = ok && !mc.abort && warp_wait_all(&br.free[(i - 1) & 1][1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
      if (!done) mc.abort = 1;
      named_bar(2, 128);
      tc_fence_after();
      if (done) {
        // O^T: lane = dim 128 g + 32 quad + lane, column = row. 16 rows of 32 dims at a time, turned in Q's place (the block's
        // QK is done; rows of 36 floats: both sides hit all banks), so that stores are 16 bytes wide.
        // Unrolled by four: with a smaller loop here the whole kernel came out 8 % slower on long caches.
        float* turn = reinterpret_cast<float*>(smem + kOffQ) + quad * 16 * 36;
#pragma unroll 4
        for (int h = 0; h < 16; ++h) {
          const int r0 = 16 * (h & 3), n = s.nrows - r0, d = 128 * (h >> 2) + 32 * quad;
          if (n <= 0) continue;
          uint32_t o[16];
          tmem_ld16(quarter + 16 * h, o);
          tmem_wait_ld();
          __syncwarp();  // the rows before have been read
#pragma unroll
          for (int z = 0; z < 16; ++z) turn[36 * z + lane] = __uint_as_float(o[z]) * inverse[r0 + z];
          __syncwarp();
          if (whole) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = 8 * j + (lane >> 2);
              const float4 x = *reinterpret_cast<const float4*>(turn + 36 * r + 8 * (lane & 3));
              const float4 y = *reinterpret_cast<const float4*>(turn + 36 * r + 8 * (lane & 3) + 4);
              alignas(16) const __nv_bfloat162 b2[4] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w),
                                            __floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
              if (r < n)
                *reinterpret_cast<uint4*>(p.out + (row0 + r0 + r) * HS_D_LATENT + d + 8 * (lane & 3)) = *reinterpret_cast<const uint4*>(b2);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = 4 * j + (lane >> 3);
              if (r < n)
                *reinterpret_cast<float4*>(p.part_out + (part * kRows + r0 + r) * HS_D_LATENT + d + 4 * (lane & 7)) =
                    *reinterpret_cast<const float4*>(turn + 36 * r + 4 * (lane & 7));
            }
          }
        }
      }
      tc_fence_before();
      ok = ok && done;
      named_bar(2, 128);  // the rows' factors have been read
    }
    if (!ok) mc.abort = 1;
    if (warp == kSmWarp0 && lane == 0) p.desc[c] = desc;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (pw >= 0) {
      // ================================================================ producers =================
      const int rl = lane >> 3, c8 = lane & 7;
      const int row = 4 * pw + rl;
      const uint32_t at = sw128_offset(row, 16 * c8);
      const uint8_t* mine = smem + kOffRaw + row * HS_KV_ROW_BYTES;
      Raw raw;
      int left = kEnd;
      bool range_ok = true, ok = true;
      // this warp's rows of the next page into registers; the place is handed back at once
      auto take = [&](int i) {
        ok = ok && !mc.abort && warp_wait_all(&br.raw_full, (uint32_t)i & 1u, p.err);
        if (!ok) return;
        left = mc.left;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) raw.code[g][h] = *reinterpret_cast<const uint2*>(mine + 128 * g + 64 * h + 8 * c8);
        raw.scale = *reinterpret_cast<const uint4*>(mine + HS_D_LATENT);
        raw.rope = *reinterpret_cast<const uint4*>(mine + HS_D_LATENT + 16 + 16 * c8);
        fence_proxy_async_smem();  // these reads come before the next page's copy
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.raw_free);
      };
      take(0);
#pragma unroll 1
      for (int i = 0; ok && left != kEnd; ++i) {
        const int s = i & 1;
        uint8_t* tile = smem + kOffTile + s * kTile + at;
        bool bad = false;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if ((g & 1) == 0) {
            ok = ok && warp_wait_all(&br.free[s][g >> 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err);
            if (!ok) break;
          }
          float f = row < left ? __uint_as_float((&raw.scale.x)[g]) : 0.f;
          range_ok &= f == 0.f || (fabsf(f) >= kScaleMin && fabsf(f) <= kScaleMax);
          const bool wild = !(fabsf(f) <= kScaleMax);
          f = wild ? 0.f : f;
          const __half2 h2 = __floats2half2_rn(f, f);
          const float lo = f - __low2float(h2);
          const __half2 l2 = __floats2half2_rn(lo, lo);
          const uint32_t hu = *reinterpret_cast<const uint32_t*>(&h2), lu = *reinterpret_cast<const uint32_t*>(&l2);
          uint2 v = raw.code[g][0], w = raw.code[g][1];
          if (has_nan(v, w) || wild) {
            v = w = make_uint2(0, 0);
            bad = true;
          }
          *reinterpret_cast<uint4*>(tile + 2 * g * kBlk) = dequant8(v.x, v.y, hu, lu);
          *reinterpret_cast<uint4*>(tile + (2 * g + 1) * kBlk) = dequant8(w.x, w.y, hu, lu);
          if (g == 3) {
            if ((__ballot_sync(0xffffffffu, bad) >> (8 * rl)) & 0xFFu) raw.rope.x = 0x7FC07FC0u;  // two bf16 NaN
            *reinterpret_cast<uint4*>(tile + 8 * kBlk) = raw.rope;
          }
          if (g & 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&br.full[s][g >> 1]);
          }
        }
        take(i + 1);
      }
      if (!ok) mc.abort = 1;
      if (!range_ok) flag_error(p.err, HS_FLAG_RANGE);
    } else if (warp == kLoadWarp) {
      // ================================================================ codes =====================
      // One page at a time, the next as soon as the producers have taken it into registers. Table entries are read three pages
      // ahead, pages asked into L2 two ahead.
      if (lane == 0) {
        Pages pages(p, st);
        auto good = [&](const Page& g) { return g.blk >= 0 && ((int64_t)g.blk + 1) * HS_PAGE <= p.R; };
        constexpr uint32_t kPageBytes = HS_PAGE * HS_KV_ROW_BYTES;
        Page now = pages.next(p), then = pages.next(p), after = pages.next(p);
        bool ok = true;
        int i = 0;
#pragma unroll 1
        for (;; ++i) {
          ok = !mc.abort && mbar_wait(&br.raw_free, ((uint32_t)i & 1u) ^ 1u, p.err);
          if (!ok) break;
          const bool have = now.live && good(now) && now.left > 0;
          if (now.live && now.left > 0 && !have) flag_error(p.err, HS_FLAG_BAD_BLOCK);
          mc.left = !now.live ? kEnd : have ? now.left : 0;
          if (have) {  // also rows past the length: the page is there
            mbar_arrive_expect_tx(&br.raw_full, kPageBytes);
            bulk_g2s(smem + kOffRaw, p.kv + (int64_t)now.blk * kPageBytes, kPageBytes, &br.raw_full);
          } else {
            mbar_arrive(&br.raw_full);
          }
          if (!now.live) break;
          now = then;
          then = after;
          after = pages.next(p);
          if (then.live && good(then)) bulk_prefetch_l2(p.kv + (int64_t)then.blk * kPageBytes, kPageBytes);
        }
        if (!ok) {
          mc.abort = 1;
          if (i > 0) mbar_wait(&br.raw_full, (uint32_t)(i - 1) & 1u, p.err);  // no copy is under way at the end
        }
      }
    } else if (warp == 0) {
      // ================================================================ QK ========================
      if (lane == 0) {
        constexpr uint32_t wide = idesc_f16(128, kPageKeys, 0, 0), lat = idesc_f16(kRows, kPageKeys, 0, 0), rop = idesc_bf16(kRows, kPageKeys, 0, 0);
        const uint64_t qd = smem_desc(smem_u32(smem + kOffQ), 16, 1024, 2);
        Walk<kRows> walk(p, st);
        Seg s;
        int i = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; ok && walk.next(p, s); ++n) {
          ok = !mc.abort && mbar_wait(&br.q_ready, (uint32_t)n & 1u, p.err);
          tc_fence_after();
          const int end = end_page(p, s);
#pragma unroll 1
          for (int j = first_page(s); ok && j < end; ++j, ++i) {
            const int b = i & 1;
            const uint32_t ph = (uint32_t)(i >> 1) & 1u;
            ok = !mc.abort && mbar_wait(&br.s_empty[b], ph ^ 1u, p.err);
            const uint64_t kd = smem_desc(smem_u32(smem + kOffTile + b * kTile), 16, 1024, 2);
            const uint32_t d = tmem + kColS + 64 * b;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if ((g & 1) == 0) {
                ok = ok && mbar_wait(&br.full[b][g >> 1], ph, p.err);
                // products of different shapes on one accumulator are not kept in order by themselves
                if (g == 2) ok = ok && mbar_wait(&br.wide_done, (uint32_t)i & 1u, p.err);
                if (!ok) break;
                tc_fence_after();
              }
#pragma unroll
              for (int k = 0; k < (g < 3 ? 8 : 12); ++k) {  // 16 dims each
                const int blk = 2 * g + k / 4;
                const uint64_t b16 = kd + (uint64_t)((blk * kBlk + (k % 4) * 32) >> 4);
                if (g < 2)  // Q from tensor memory: 128 lanes, of which 64 are rows
                  mma_f16_ts(d, tmem + kColQ + 64 * g + 8 * k, b16, wide, (g | k) != 0 ? 1u : 0u);
                else
                  mma_bf16_ss(d, qd + (uint64_t)(((blk - 4) * kBlk + (k % 4) * 32) >> 4), b16, k < 8 ? lat : rop, 1u);
              }
              if (g == 1) mma_commit(&br.wide_done);
            }
            if (ok) mma_commit(&br.s_full[b]);
          }
        }
        if (!ok) mc.abort = 1;
        mma_commit(&br.drain[0]);
        mbar_wait(&br.drain[0], 0, p.err);
      }
    } else if (warp == kPvWarp) {
      // ================================================================ PV ========================
      if (lane == 0) {
        constexpr uint32_t id = idesc_f16(128, kRows, 1, 0);
        Walk<kRows> walk(p, st);
        Seg s;
        int i = 0;
        bool ok = true;
#pragma unroll 1
        while (ok && walk.next(p, s)) {
          const int first = first_page(s), end = end_page(p, s);
#pragma unroll 1
          for (int j = first; ok && j < end; ++j, ++i) {
            const int b = i & 1;
            ok = !mc.abort && mbar_wait(&br.p_full[b], (uint32_t)(i >> 1) & 1u, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = smem_u32(smem + kOffTile + b * kTile);
            const uint64_t vd = smem_desc(at, kBlk, 1024, 2), pd = smem_desc(at + 8 * kBlk, 16, 1024, 2);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_ss(tmem + 64 * g, vd + (uint64_t)((2 * g * kBlk + k * 2048) >> 4), pd + (uint64_t)((k * 32) >> 4), id,
                            j > first || k > 0 ? 1u : 0u);
              if (g & 1) mma_commit(&br.free[b][g >> 1]);
            }
          }
        }
        if (!ok) mc.abort = 1;
        mma_commit(&br.drain[1]);
        mbar_wait(&br.drain[1], 0, p.err);
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace few

uint64_t few_bytes(int sms) { return (uint64_t)2 * sms * few::kRows * (HS_D_LATENT + 1) * 4 + (uint64_t)sms * sizeof(Desc); }

cudaError_t launch_few(const Params& p0, int sms, cudaStream_t stream) {
  using namespace few;
  cudaError_t e = cudaFuncSetAttribute(few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  Params p = p0;
  p.clusters = sms < kMaxClusters ? sms : kMaxClusters;
  p.part_lse = p.part_out + (int64_t)2 * sms * kRows * HS_D_LATENT;
  p.desc = reinterpret_cast<Desc*>(p.part_lse + (int64_t)2 * sms * kRows);
  few_kernel<<<p.clusters, kThreads, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(paged_merge_kernel<kRows>, Merge<kRows>::grid(p.clusters), kMergeThreads, 0, stream, p);
}

}  // namespace paged
}  // namespace hs
