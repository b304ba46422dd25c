// paged_few.cu — dense attention over paged FP8 latent rows for requests with few (token, head) rows (decode): the formulas of
// paged.cu on one SM per block of 64 rows.
//
//   S = Q K^T (M = 64 rows, N = 64 cached rows, 36 MMAs of 45 cycles),  P = 2^(c S - m),
//   O^T += V^T P^T (M = 128 dims x 4, N = 64 rows, 16 MMAs): O^T takes 256 of the SM's tensor memory columns, two S buffers 128.
//
// Work. Persistent, one CTA per SM; units as in paged.cu (block of rows, 128 cached rows), shared out evenly, split blocks joined
// by paged_merge_kernel. Inside a unit the step is one page (64 rows).
//
// Roles (warp w runs on sub-partition w % 4, so the two issuing warps share theirs with one softmax warp only). Warp 0 issues QK,
// warp 4 PV. Warps 1-3, 5-7, 13, 14 are the producers: each turns 8 rows of a page from codes into fp16 (code * group scale,
// rounded once) in 128-byte-swizzled blocks [64 rows][64 dims], from registers that it loaded a page ahead. Two pages fit beside
// Q; a 128-dim group of a page is handed to QK when all producers have written it and comes back when PV has read it. Warps 8-11
// are the softmax, 16 rows each, two threads per row with 32 columns each (what a 64-row product leaves in tensor memory).
// P goes into the page's rotary block, which QK has read by then.
//
// Lazy maximum and masks as in paged.cu: a row's reference moves only when a logit passes it by more than 2^8; one OR-barrier
// per page tells the softmax warps, which then rescale O^T's columns. A latent value that is NaN or cannot be fp16 is zeroed
// and its row's rotary values become NaN: rows that see it are NaN, P = 0 times it stays 0.
#include "paged.cuh"

namespace hs {
namespace paged {
namespace few {

constexpr int kRows = 64, kPageKeys = HS_PAGE;
constexpr int kThreads = 768;
constexpr int kPvWarp = 4, kSmWarp0 = 8, kProducers = 16;
constexpr int kQuads = kPageKeys / (4 * kProducers);  // fours of rows per producer
constexpr int kBlk = kPageKeys * 128;          // [64][64 dims] of 16 bits
constexpr int kTile = 9 * kBlk;
constexpr int kOffQ = 0, kOffTile = kTile;
constexpr int kOffScratch = kOffTile;          // int64 [B + 1] and int32 [B + 1] during the set-up
constexpr int kOffRow = 3 * kTile;             // float [64] each: factors, 1 / sums, logit coefficients
constexpr int kOffBar = kOffRow + 3 * 256;
struct Bars {
  uint64_t full[2][4];   // producers have written a group of a page -> QK
  uint64_t free[2][4];   // PV has read it (group 3: and P) -> producers, softmax
  uint64_t s_full[2];    // S complete -> softmax
  uint64_t s_empty[2];   // S read -> QK
  uint64_t p_full[2];    // P written, O^T rescaled -> PV
  uint64_t q_ready;      // a block's Q is in place -> QK
  uint64_t drain[2];
};
struct Misc {
  uint32_t tmem;
  volatile uint32_t abort;
  Start start;
};
constexpr int kOffMisc = kOffBar + (int)sizeof(Bars);
constexpr int kSmem = kOffMisc + (int)sizeof(Misc);
static_assert(kSmem <= 232448 && 12 * (kMaxReq + 1) <= 2 * kTile && kOffBar % 8 == 0 && kOffMisc % 8 == 0, "shared memory");
constexpr int kColS = 256;                     // S buffers; O^T is columns 0 .. 255

// Index of warp w among the producers, or -1.
__host__ __device__ constexpr int producer_index(int w) {
  return w == 12 ? 15 : w % 4 == 0 || (w >= 8 && w < 12) ? -1 : (w < 8 ? w / 4 : w / 4 - 1) * 3 + w % 4 - 1;
}

// Pages [first, end) of a segment: the last tile of a block may need only its first page.
__device__ __forceinline__ int first_page(const Seg& s) { return 2 * s.ta; }
__device__ __forceinline__ int end_page(const Params& p, const Seg& s) {
  const int n = sees(p, s.q, (int64_t)s.b * kRows + s.nrows - 1);
  const int pages = n > 0 ? (n + kPageKeys - 1) / kPageKeys : 1;
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

// A producer lane's part of a page: of two rows (8 w + l / 8, and 4 further) 16 codes of every group, the four scales
// and 16 bytes of the rotary values.
struct Raw {
  uint4 code[4][kQuads], rope[kQuads], scale[kQuads];
};

// Whether one of 16 codes is NaN (0x7F, 0xFF).
__device__ __forceinline__ bool has_nan(const uint4& v) {
  const uint32_t m = 0x7F7F7F7Fu, o = 0x01010101u;
  return ((((v.x & m) + o) | ((v.y & m) + o) | ((v.z & m) + o) | ((v.w & m) + o)) & 0x80808080u) != 0u;
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
  float* coefs = alpha + 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      for (int g = 0; g < 4; ++g) {
        mbar_init(&br.full[s][g], kProducers);
        mbar_init(&br.free[s][g], 1);
      }
      mbar_init(&br.s_full[s], 1);
      mbar_init(&br.s_empty[s], 4);
      mbar_init(&br.p_full[s], 4);
      mbar_init(&br.drain[s], 1);
    }
    mbar_init(&br.q_ready, 4);
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
      // Q: four rows of 64 dims per load; the block before has been read (its last S is complete). Rows past the block's are
      // read as its first row.
      if (!idle) {
        const uint8_t* q0 = p.q + row0 * (HS_D_QK * 2) + 16 * (lane & 7);
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          const int r = 16 * quad + 4 * h + (lane >> 3);
          const uint8_t* src = q0 + (int64_t)(r < s.nrows ? r : 0) * (HS_D_QK * 2);
          uint4 v[9];
#pragma unroll
          for (int k = 0; k < 9; ++k) v[k] = ldg_nc_v4(src + 128 * k);
          uint32_t mx = 0u;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                       __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu)));
          uint32_t amax = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // A row whose largest latent value is outside [2^-6, 2^15) is scaled by a power of two that puts it in
          // [2^14, 2^15); its logits are scaled back.
          int e = 0;
          if (amax >= 0x7F80u) {
            if (r < s.nrows) flag_error(p.err, HS_FLAG_RANGE);
          } else if (amax >= 0x4700u || (amax >= 0x0080u && amax < 0x3C80u)) {
            e = 14 - ((int)(amax >> 7) - 127);
          } else if (amax > 0u && amax < 0x0080u) {
            e = 126;
          }
          e = e < -126 ? -126 : (e > 126 ? 126 : e);
          const float f = __uint_as_float((uint32_t)(e + 127) << 23);
          // not 0, so that a masked column stays -inf; logits below 2^-60 or so do not show anyway
          if ((lane & 7) == 0) coefs[r] = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 7.5e-37f);
#pragma unroll
          for (int k = 0; k < 9; ++k) {
            uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t u = w[z] ^ p.flip;
              const float a = __uint_as_float(u << 16) * f, b = __uint_as_float(u & 0xFFFF0000u) * f;
              if (k < 8) {
                w[z] = pack_half2(a, b);
              } else {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
                w[z] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
            *reinterpret_cast<uint4*>(smem + kOffQ + k * kBlk + sw128_offset(r, 16 * (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&br.q_ready);
      const float coef = idle ? 1.f : coefs[row];

      const int nsee = mine ? sees(p, s.q, (int64_t)s.b * kRows + row) : 0;
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
            here = here && warp_wait_all(&br.free[b ^ 1][3], (uint32_t)((i - 1) >> 1) & 1u, p.err);  // PV so far is complete
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
          const float me = ref == -INFINITY ? 0.f : ref;
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
          const float z = sum == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(sum)) * kLn2;
          if (!whole)
            p.part_lse[part * kRows + row] = z;
          else if (p.lse)
            p.lse[row0 + row] = z;
        }
      }
      const bool done = ok && !mc.abort && warp_wait_all(&br.free[(i - 1) & 1][3], (uint32_t)((i - 1) >> 1) & 1u, p.err);
      if (!done) mc.abort = 1;
      named_bar(2, 128);
      tc_fence_after();
      if (done) {
        // O^T: lane = dim 128 g + 32 quad + lane, column = row
#pragma unroll 1
        for (int h = 0; h < 8; ++h) {
          const int g = h >> 1, r0 = 32 * (h & 1), d = 128 * g + 32 * quad + lane;
          if (r0 >= s.nrows) continue;
          uint32_t o[32];
          tmem_ld32(quarter + 32 * h, o);
          tmem_wait_ld();
          const int n = s.nrows - r0;
#pragma unroll
          for (int z = 0; z < 32; z += 2) {
            const float2 f = *reinterpret_cast<const float2*>(inverse + r0 + z);
            const float a = __uint_as_float(o[z]) * f.x, e = __uint_as_float(o[z + 1]) * f.y;
            if (whole) {  // lanes swap, so that each stores two dims: the even one of row z, the odd one of row z + 1
              const float y = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : e, 1);
              const __nv_bfloat162 b2 = lane & 1 ? __floats2bfloat162_rn(y, e) : __floats2bfloat162_rn(a, y);
              const int r = z + (lane & 1);
              if (r < n) *reinterpret_cast<__nv_bfloat162*>(p.out + (row0 + r0 + r) * HS_D_LATENT + (d & ~1)) = b2;
            } else {
              float* to = p.part_out + (part * kRows + r0 + z) * HS_D_LATENT + d;
              if (z < n) to[0] = a;
              if (z + 1 < n) to[HS_D_LATENT] = e;
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
      const uint32_t odd = (uint32_t)((c8 >> 2) ^ (rl & 1));  // which half of its codes a lane stores first: spreads the banks
      Pages pages(p, st);
      Raw raw;
      auto rows_of = [&](const Page& g) -> const uint8_t* {
        const bool good = g.blk >= 0 && ((int64_t)g.blk + 1) * HS_PAGE <= p.R;
        if (g.live && !good && g.left > 0 && lane == 0) flag_error(p.err, HS_FLAG_BAD_BLOCK);
        return good ? p.kv + ((int64_t)g.blk * HS_PAGE + 4 * kQuads * pw + rl) * HS_KV_ROW_BYTES : nullptr;
      };
      auto load = [&](const uint8_t* from, int off) { return from ? ldg_nc_v4(from + off) : make_uint4(0, 0, 0, 0); };
      auto load_group = [&](const uint8_t* from, int g) {
#pragma unroll
        for (int h = 0; h < kQuads; ++h) raw.code[g][h] = load(from, h * 4 * HS_KV_ROW_BYTES + 128 * g + 16 * c8);
      };
      auto load_rest = [&](const uint8_t* from) {
#pragma unroll
        for (int h = 0; h < kQuads; ++h) {
          raw.scale[h] = load(from, h * 4 * HS_KV_ROW_BYTES + HS_D_LATENT);
          raw.rope[h] = load(from, h * 4 * HS_KV_ROW_BYTES + HS_D_LATENT + 16 + 16 * c8);
        }
      };
      Page now = pages.next(p);
      const uint8_t* from = rows_of(now);
      load_rest(from);
#pragma unroll
      for (int g = 0; g < 4; ++g) load_group(from, g);
      Page then = pages.next(p), after = pages.next(p);  // table entries are read two pages ahead, rows one
      bool range_ok = true, ok = true;
#pragma unroll 1
      for (int i = 0; ok && now.live; ++i) {
        const int s = i & 1;
        uint8_t* tile = smem + kOffTile + s * kTile;
        const uint8_t* ahead = rows_of(then);
        bool bad[kQuads] = {};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          ok = ok && !mc.abort && warp_wait_all(&br.free[s][g], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err);
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < kQuads; ++h) {
            const int row = 4 * kQuads * pw + 4 * h + rl;
            const uint32_t* sc = &raw.scale[h].x;
            const float f = row < now.left ? __uint_as_float(sc[g]) : 0.f;
            const bool fits = f == 0.f || (fabsf(f) >= kScaleMin && fabsf(f) <= kScaleMax);
            range_ok &= fits;
            const __half hi = __float2half_rn(f);
            const __half2 h2 = __half2half2(hi), l2 = __float2half2_rn(f - __half2float(hi));
            const uint32_t hu = *reinterpret_cast<const uint32_t*>(&h2), lu = *reinterpret_cast<const uint32_t*>(&l2);
            const uint4 v = raw.code[g][h];
            uint4 d0 = dequant8(odd ? v.z : v.x, odd ? v.w : v.y, hu, lu);
            uint4 d1 = dequant8(odd ? v.x : v.z, odd ? v.y : v.w, hu, lu);
            if (has_nan(v) || !(fabsf(f) <= kScaleMax)) {
              d0 = d1 = make_uint4(0, 0, 0, 0);
              bad[h] = true;
            }
            uint8_t* blk = tile + (2 * g + (c8 >> 2)) * kBlk;
            const uint32_t at = sw128_offset(row, 32 * (c8 & 3) + 16 * odd);
            *reinterpret_cast<uint4*>(blk + at) = d0;
            *reinterpret_cast<uint4*>(blk + (at ^ 16u)) = d1;
            if (g == 3) {
              uint4 r = raw.rope[h];
              if ((__ballot_sync(0xffffffffu, bad[h]) >> (8 * rl)) & 0xFFu) r.x = 0x7FC07FC0u;  // two bf16 NaN
              *reinterpret_cast<uint4*>(tile + 8 * kBlk + sw128_offset(row, 16 * c8)) = r;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&br.full[s][g]);
          load_group(ahead, g);
        }
        load_rest(ahead);
        now = then;
        then = after;
        after = pages.next(p);
      }
      if (!ok) mc.abort = 1;
      if (!range_ok) flag_error(p.err, HS_FLAG_RANGE);
    } else if (warp == 0) {
      // ================================================================ QK ========================
      if (lane == 0) {
        constexpr uint32_t lat = idesc_f16(kRows, kPageKeys, 0, 0), rop = idesc_bf16(kRows, kPageKeys, 0, 0);
        const uint64_t qd = smem_desc(smem_u32(smem + kOffQ), 16, 1024, 2);
        Walk<kRows> walk(p, st);
        Seg s;
        int i = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; ok && walk.next(p, s); ++n) {
          ok = !mc.abort && mbar_wait(&br.q_ready, (uint32_t)n & 1u, p.err);
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
              ok = ok && mbar_wait(&br.full[b][g], ph, p.err);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < (g < 3 ? 8 : 12); ++k) {  // 16 dims each
                const uint64_t at = (uint64_t)(((2 * g + k / 4) * kBlk + (k % 4) * 32) >> 4);
                mma_bf16_ss(d, qd + at, kd + at, k < 8 ? lat : rop, (g | k) != 0 ? 1u : 0u);
              }
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
              mma_commit(&br.free[b][g]);
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
  paged_merge_kernel<kRows><<<dim3((unsigned)p.clusters, kRows / kMergeRows), kMergeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace hs
