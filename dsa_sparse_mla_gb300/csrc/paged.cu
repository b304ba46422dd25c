// paged.cu — dense attention of each request's new tokens over its paged FP8 latent rows (MLA in MQA
// form), on tcgen05, two SMs per block of rows.
//
// [P1] "vLLM v0.32.0 GLM-5.3 サービング ...", sections 「再現方法と必要なフラグ」 and 「数字がうまくいく理由」:
// every cached row serves all heads; QK runs over 576 dims (512 latent + 64 RoPE), PV over the 512
// latent dims. A request's (token, head) pairs, 128 at a time, are the rows of one softmax attention:
//   S = Q K^T,  P = 2^(c S - m),  O = P V,  out = O / sum P,     V = the first 512 dims of K.
//
// Why two SMs. O of 128 rows and 512 fp32 dims fills an SM's tensor memory, so S has no place beside
// it; 64 rows per SM would halve the work per row loaded and pay the fixed cost of small MMAs. A cluster of
// two CTAs splits the two products instead: CTA A computes S and the softmax, CTA B keeps O and computes PV,
// each with M = 128 rows at the tensor core's full rate (36 MMAs of N = 128 per 128 keys in A, 32 in B).
// P (fp16) goes from A's registers straight into B's shared memory. Both CTAs dequantise the rows they
// need themselves (fp16, code * group scale rounded once).
//
// Work. Units are (block of 128 rows, 128 cached rows); every cluster takes an equal share of all units
// of the batch, found by prefix sums at the start (no plan on the host, which does not know the lengths). A block whose
// units span clusters leaves fp32 partial outputs and their log-sum-exps in the workspace;
// paged_merge_kernel joins them.
//
// Roles (512 threads; warp w runs on sub-partition w % 4 and reads tensor-memory lanes 32 (w % 4) .. + 31):
//   warps 1-3, 5-7, 13, 14   producers: read rows, dequantise, write 128-byte-swizzled [128 keys][64 dims]
//                            blocks into the ring (A: 5 blocks of 16 KB, nine per tile; B: 5 stages
//                            of two blocks, four per tile);
//   warp 0                   issues the MMAs (and in A loads Q by TMA);
//   warps 8-11               A: Q to fp16, softmax, thread = row; B: rescaling of O and the output, thread = row;
//   warp 4                   B: tells A when PV has read a P buffer.
// The issuing warp shares its sub-partition with one softmax warp only: producers there would starve it.
//
// Lazy maximum: a row's reference max moves only when a logit exceeds it by more than 2^8 (P stays below
// 2^8, well inside fp16); then A sends the row's factor with P and B rescales that row of O. Masked
// columns are selected away before the maximum and the exponential, so what they hold does not matter; V rows
// that fp16 cannot hold are zeroed in B, so that P = 0 times them is 0.
#include "paged.cuh"

namespace hs {
namespace paged {

constexpr int kThreads = 512;
constexpr int kRows = 128;                     // (token, head) rows per block
constexpr int kBlk = kKeys * 128;              // one swizzled [128][64 x 16-bit] block
constexpr int kSlots = 5;                      // A: blocks in the K ring;  B: stages in the V ring
constexpr int kSmWarp0 = 8;
constexpr int kProdWarps = 8;
__host__ __device__ constexpr int producer_index(int w) {
  return (w % 4 == 0 || (w >= 8 && w < 12) || w == 15) ? -1 : (w < 8 ? w - 1 - w / 4 : w - 7);
}
// shared memory, A: Q [9 blocks], K ring; B: P [2][2 blocks], V ring [5][2 blocks]
constexpr int kOffRingA = 9 * kBlk;
constexpr int kOffRingB = 4 * kBlk;
constexpr int kOffSmall = 14 * kBlk;           // 229,376
constexpr int kOffAlpha = kOffSmall;           // B: float [2][128]
constexpr int kOffSum = kOffAlpha + 1024;      // B: float [2][128]
constexpr int kOffMoved = kOffSum + 1024;      // B: u32 [2][4]
constexpr int kOffBar = kOffMoved + 32;
constexpr int kNumBars = 32;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;  // tmem base, abort, Start
constexpr int kSmem = kOffMisc + 64;
constexpr int kOffScratch = kOffRingA;         // int64 [B + 1] during the set-up
static_assert(kOffRingB + 10 * kBlk <= kOffSmall && kOffScratch + 8 * (kMaxReq + 1) <= kOffSmall, "layout");
static_assert(kSmem <= 232448, "shared memory");

// A latent group's pieces that a producer lane holds: 16 codes of each of its four rows, and their scales.
struct Chunk {
  uint4 v[4];
  float s[4];
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap map_q, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + kOffBar);
  uint64_t* full = bars;                  // [5] producers wrote a slot -> MMA
  uint64_t* empty = bars + kSlots;        // [5] MMA read it -> producers
  uint64_t* s_full = bars + 2 * kSlots;   // A [2] S complete -> softmax
  uint64_t* s_empty = s_full + 2;         // A [2] softmax read S -> MMA
  uint64_t* p_empty = s_full + 4;         // A [2] B has read P, its factors and sums -> softmax
  uint64_t* p_full = s_full + 6;          // B [2] P written (by A) -> MMA, correction
  uint64_t* corr = s_full + 8;            // B [2] O rescaled for this P -> MMA
  uint64_t* pv_done = s_full + 10;        // B [2] PV complete -> correction, relay
  uint64_t* q_full = s_full + 12;         // A
  uint64_t* q_ready = s_full + 13;        // A: Q is fp16
  uint64_t* q_free = s_full + 14;         // A: the block's QK MMAs have read Q
  uint64_t* o_free = s_full + 15;         // B: O read out -> MMA
  uint64_t* drain = s_full + 16;
  uint32_t* misc = (uint32_t*)(smem + kOffMisc);
  volatile uint32_t* abort_flag = misc + 1;
  Start* st = (Start*)(misc + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool isA = cluster_ctarank() == 0;
  const int c = blockIdx.x >> 1;
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in every CTA
    if (tid == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], kProdWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 4);
      mbar_init(&p_empty[s], 5);
      mbar_init(&p_full[s], 4);
      mbar_init(&corr[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_ready, 4);
    mbar_init(q_free, 1);
    mbar_init(o_free, 4);
    mbar_init(drain, 1);
    mbar_fence_init();
    misc[1] = 0;
  }
  if (warp == 0) tmem_alloc(&misc[0], 512);
  find_units<kRows>(p, (int64_t*)(smem + kOffScratch), st, c, kThreads);
  fence_proxy_async_all();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int64_t u0 = st->u0, u1 = st->u1, U = st->U;
  Walk<kRows> walk(p, *st);

  const int pw = producer_index(warp);
  if (pw >= 0) {
    // ================================================================ producers =================
    // Warp pw owns rows 16 pw .. + 15 of every tile (one page holds them all); in pass ps lane l works on row
    // 16 pw + 4 ps + l / 8 and on the 16 codes 16 (l % 8) of a latent group, which become 16-byte pieces
    // 2 (l % 4) and + 1 of a row of block (l % 8) / 4. Lanes with l % 8 >= 4 store their second piece first, so
    // that the eight lanes of a row hit eight bank groups. Two groups are in registers ahead of the one
    // written; pages are asked into L2 two tiles ahead.
    const int rl = lane >> 3, c8 = lane & 7;
    const bool swp = c8 >= 4;
    uint8_t* ring = smem + (isA ? kOffRingA : kOffRingB);
    Seg seg;
    int jt = 0;
    bool more = walk.next(p, seg);
    if (more) jt = seg.ta;
    struct Ent {
      int32_t blk;   // block-table entry (loaded, not yet checked)
      int32_t left;  // cached rows from this warp's first row on
      bool page;     // there is such a page
    };
    auto fetch = [&]() -> Ent {  // the next tile of this cluster
      Ent e;
      e.left = 0;
      int page = 0, r = 0;
      if (more) {
        page = 2 * jt + (pw >> 2);
        r = seg.r;
        e.left = seg.q.seq - jt * kKeys - pw * 16;
        if (++jt == seg.tb) {
          more = walk.next(p, seg);
          if (more) jt = seg.ta;
        }
      }
      e.page = page < p.bt_stride;
      e.blk = ldg_nc_s32(p.bt + (int64_t)r * p.bt_stride + (e.page ? page : 0));
      return e;
    };
    struct Src {
      const uint8_t* row;  // this lane's row of pass 0
      uint32_t ok;         // bit ps: the row of pass ps exists
    };
    auto resolve = [&](const Ent& e) -> Src {
      Src s;
      const bool good = e.page && e.blk >= 0 && ((int64_t)e.blk + 1) * HS_PAGE <= p.R;
      if (e.left > 0 && !good && lane == 0) flag_error(p.err, HS_FLAG_BAD_BLOCK);
      s.ok = 0u;
#pragma unroll
      for (int ps = 0; ps < 4; ++ps) s.ok |= (good && rl + 4 * ps < e.left) ? 1u << ps : 0u;
      s.row = p.kv + ((int64_t)e.blk * HS_PAGE + (pw & 3) * 16 + rl) * HS_KV_ROW_BYTES;
      if (isA && good && e.left > 0 && (pw & 3) == 0 && lane == 0)  // the page's rows in use
        bulk_prefetch_l2(p.kv + (int64_t)e.blk * kKeys / 2 * HS_KV_ROW_BYTES, (e.left < HS_PAGE ? e.left : HS_PAGE) * HS_KV_ROW_BYTES);
      return s;
    };
    auto at = [&](const Src& s, int ps) { return ((s.ok >> ps) & 1u) ? s.row + ps * 4 * HS_KV_ROW_BYTES : p.kv; };
    auto ld_group = [&](Chunk& ch, const Src& s, int g) {
#pragma unroll
      for (int ps = 0; ps < 4; ++ps) {
        const uint8_t* src = at(s, ps);
        ch.v[ps] = ldg_nc_v4(src + 128 * g + 16 * c8);
        ch.s[ps] = ldg_nc_f32(src + HS_D_LATENT + 4 * g);
      }
    };
    int slot = 0;
    uint32_t par = 1;  // parity to wait for: the first round finds the slots free
    bool go = true;
    auto take = [&]() {  // the next slot of the ring, once it is free
      const bool ok = go && !*abort_flag && mbar_wait(&empty[slot], par, p.err);
      go = __all_sync(0xffffffffu, ok);
      return ring + slot * (isA ? kBlk : 2 * kBlk);
    };
    auto publish = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[slot]);
      if (++slot == kSlots) {
        slot = 0;
        par ^= 1u;
      }
    };
    bool range_ok = true;
    auto st_group = [&](const Chunk& ch, const Src& s) {
      uint8_t *b0, *b1;  // blocks of dims 0-63 and 64-127 of the group
      const int s0 = slot;
      if (isA) {
        b0 = take();
        if (++slot == kSlots) {
          slot = 0;
          par ^= 1u;
        }
        b1 = take();
      } else {
        b0 = take();
        b1 = b0 + kBlk;
      }
      if (!go) return;
      uint8_t* blk = swp ? b1 : b0;
      const uint32_t o0 = 32 * (c8 & 3) + (swp ? 16 : 0);
#pragma unroll
      for (int ps = 0; ps < 4; ++ps) {
        const int row = 16 * pw + 4 * ps + rl;
        const bool live = (s.ok >> ps) & 1u;
        const float sc = live ? ch.s[ps] : 0.f;
        range_ok &= !live || (fabsf(sc) >= kScaleMin && fabsf(sc) <= kScaleMax);
        const __half shi = __float2half_rn(sc);
        const __half2 h2 = __half2half2(shi), l2 = __float2half2_rn(sc - __half2float(shi));
        const uint32_t hu = *reinterpret_cast<const uint32_t*>(&h2), lu = *reinterpret_cast<const uint32_t*>(&l2);
        const uint4 v = live ? ch.v[ps] : make_uint4(0, 0, 0, 0);
        uint4 d0 = dequant8(swp ? v.z : v.x, swp ? v.w : v.y, hu, lu);
        uint4 d1 = dequant8(swp ? v.x : v.z, swp ? v.y : v.w, hu, lu);
        if (!isA && unsound(d0, d1)) d0 = d1 = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(blk + sw128_offset(row, o0)) = d0;
        *reinterpret_cast<uint4*>(blk + sw128_offset(row, o0 ^ 16u)) = d1;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (isA && lane == 0) mbar_arrive(&full[s0]);
      publish();
    };
    const int64_t ntiles = u1 - u0;
    Src cur, nxt, after;
    {
      const Ent e0 = fetch(), e1 = fetch();
      cur = resolve(e0);
      nxt = resolve(e1);
    }
    Ent e2 = fetch();
    Chunk c0, c1;
    if (ntiles > 0) {
      ld_group(c0, cur, 0);
      ld_group(c1, cur, 1);
    }
#pragma unroll 1
    for (int64_t i = 0; i < ntiles && go; ++i) {
      after = resolve(e2);
      e2 = fetch();
      uint4 rope[4];
      st_group(c0, cur);
      ld_group(c0, cur, 2);
      st_group(c1, cur);
      ld_group(c1, cur, 3);
      if (isA) {
#pragma unroll
        for (int ps = 0; ps < 4; ++ps) rope[ps] = ldg_nc_v4(at(cur, ps) + HS_D_LATENT + 16 + 16 * c8);
      }
      st_group(c0, cur);
      ld_group(c0, nxt, 0);
      st_group(c1, cur);
      ld_group(c1, nxt, 1);
      if (isA) {
        uint8_t* blk = take();
        if (go) {
#pragma unroll
          for (int ps = 0; ps < 4; ++ps)
            *reinterpret_cast<uint4*>(blk + sw128_offset(16 * pw + 4 * ps + rl, 16 * c8)) =
                ((cur.ok >> ps) & 1u) ? rope[ps] : make_uint4(0, 0, 0, 0);
          publish();
        }
      }
      cur = nxt;
      nxt = after;
    }
    if (!go) *abort_flag = 1;
    if (isA && !range_ok) flag_error(p.err, HS_FLAG_RANGE);
  } else if (warp == 0 && isA) {
    // ================================================================ A: QK =====================
    if (lane == 0) {
      constexpr uint32_t lat = idesc_f16(kRows, kKeys, 0, 0), rop = idesc_bf16(kRows, kKeys, 0, 0);
      prefetch_tensormap(&map_q);
      const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t kd = smem_desc(smem_u32(smem + kOffRingA), 16, 1024, 2);
      Seg s;
      int slot = 0, n = 0, i = 0;
      uint32_t par = 0;
      bool ok = true;
#pragma unroll 1
      for (; ok && walk.next(p, s); ++n) {
        if (n > 0) {  // the previous block's MMAs must have read Q
          mma_commit(q_free);
          if (!mbar_wait(q_free, (uint32_t)(n - 1) & 1u, p.err)) {
            ok = false;
            break;
          }
        }
        mbar_arrive_expect_tx(q_full, 9 * kBlk);
        const int32_t y = (int32_t)((int64_t)s.q.start * p.H + (int64_t)s.b * kRows);
#pragma unroll 1
        for (int d = 0; d < 9; ++d) tma_load_2d(smem + d * kBlk, &map_q, q_full, 64 * d, y);
        if (!mbar_wait(q_ready, (uint32_t)n & 1u, p.err)) {
          ok = false;
          ++n;
          break;
        }
#pragma unroll 1
        for (int jt = s.ta; jt < s.tb && ok; ++jt, ++i) {
          const int sb = i & 1;
          if (*abort_flag || !mbar_wait(&s_empty[sb], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int d = 0; d < 9; ++d) {
            if (!mbar_wait(&full[slot], par, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss(tmem + kKeys * sb, qd + (uint64_t)((d * kBlk + kk * 32) >> 4), kd + (uint64_t)((slot * kBlk + kk * 32) >> 4),
                          d < 8 ? lat : rop, (d | kk) != 0 ? 1u : 0u);
            mma_commit(&empty[slot]);
            if (++slot == kSlots) {
              slot = 0;
              par ^= 1u;
            }
          }
          if (ok) mma_commit(&s_full[sb]);
        }
      }
      if (!ok) *abort_flag = 1;
      mma_commit(drain);
      mbar_wait(drain, 0, p.err);
      if (n > 0) mbar_wait(q_full, (uint32_t)(n - 1) & 1u, p.err);  // the last Q copy has landed
    }
  } else if (warp == 0) {
    // ================================================================ B: PV =====================
    if (lane == 0) {
      constexpr uint32_t id = idesc_f16(kRows, 128, 0, 1);
      const uint64_t pd = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t vd = smem_desc(smem_u32(smem + kOffRingB), kBlk, 1024, 2);
      Seg s;
      int slot = 0, n = 0, i = 0;
      uint32_t par = 0;
      bool ok = true;
#pragma unroll 1
      for (; ok && walk.next(p, s); ++n) {
        if (n > 0 && !mbar_wait(o_free, (uint32_t)(n - 1) & 1u, p.err)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int jt = s.ta; jt < s.tb && ok; ++jt, ++i) {
          const int pb = i & 1;
          const uint32_t ph = (uint32_t)(i >> 1) & 1u;
          if (*abort_flag || !mbar_wait_cluster(&p_full[pb], ph, p.err) || !mbar_wait(&corr[pb], ph, p.err)) {
            ok = false;
            break;
          }
          fence_proxy_async_all();
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            if (!mbar_wait(&full[slot], par, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_bf16_ss(tmem + 128 * mt, pd + (uint64_t)(((2 * pb + kk / 4) * kBlk + (kk % 4) * 32) >> 4),
                          vd + (uint64_t)((2 * slot * kBlk + kk * 2048) >> 4), id, (jt > s.ta || kk > 0) ? 1u : 0u);
            mma_commit(&empty[slot]);
            if (++slot == kSlots) {
              slot = 0;
              par ^= 1u;
            }
          }
          if (ok) mma_commit(&pv_done[pb]);
        }
      }
      if (!ok) *abort_flag = 1;
      mma_commit(drain);
      mbar_wait(drain, 0, p.err);
    }
  } else if (warp == 4 && !isA) {
    // ================================================================ B: P buffers back to A ====
    if (lane == 0) {
      const uint32_t back = remote_smem(p_empty, 0);
      const int64_t ntiles = u1 - u0;
#pragma unroll 1
      for (int64_t i = 0; i < ntiles; ++i) {
        if (*abort_flag || !mbar_wait(&pv_done[i & 1], (uint32_t)(i >> 1) & 1u, p.err)) {
          *abort_flag = 1;
          break;
        }
        remote_arrive(back + 8 * (uint32_t)(i & 1));
      }
    }
  } else if (warp >= kSmWarp0 && warp < kSmWarp0 + 4 && isA) {
    // ================================================================ A: softmax ================
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const uint32_t r_p = remote_smem(smem, 1), r_alpha = remote_smem(smem + kOffAlpha, 1), r_sum = remote_smem(smem + kOffSum, 1);
    const uint32_t r_moved = remote_smem(smem + kOffMoved, 1), r_full = remote_smem(p_full, 1);
    Seg s;
    int n = 0, i = 0;
    bool ok = true;
#pragma unroll 1
    for (; ok && walk.next(p, s); ++n) {
      const bool idle = 32 * quad >= s.nrows;  // no row of this warp exists
      const bool mine = row < s.nrows;
      // Q's latent dims bf16 -> fp16 in place, this thread's row (the swizzle spreads the rows over the banks). A row
      // whose largest value is outside [2^-6, 2^15) is rewritten from global memory times a power of two that
      // puts it in [2^14, 2^15); its logits are scaled back below.
      float coef = p.scale_log2;
      ok = warp_wait_all(q_full, (uint32_t)n & 1u, p.err);
      if (ok && !idle) {
        uint32_t mx = 0u;
#pragma unroll 1
        for (int d = 0; d < 8; ++d) {
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            uint4* a = reinterpret_cast<uint4*>(smem + d * kBlk + sw128_offset(row, 16 * h));
            uint4 v = *a;
            uint32_t* w = &v.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mx = __vmaxu2(mx, w[k] & 0x7FFF7FFFu);
              w[k] ^= p.flip;
              w[k] = pack_half2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
            }
            *a = v;
          }
        }
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
        if (!mine) e = 0;
        if (e != 0) {
          coef *= __uint_as_float((uint32_t)(127 - e) << 23);
          const float f = __uint_as_float((uint32_t)(e + 127) << 23);
          const uint8_t* src = p.q + ((int64_t)s.q.start * p.H + (int64_t)s.b * kRows + row) * (HS_D_QK * 2);
#pragma unroll 1
          for (int h = 0; h < 72; ++h) {
            uint4 v = ldg_nc_v4(src + 16 * h);
            uint32_t* w = &v.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              w[k] ^= p.flip;
              const float lo = __uint_as_float(w[k] << 16) * f, hi = __uint_as_float(w[k] & 0xFFFF0000u) * f;
              if (h < 64) {
                w[k] = pack_half2(lo, hi);
              } else {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(lo, hi);
                w[k] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
            *reinterpret_cast<uint4*>(smem + (h / 8) * kBlk + sw128_offset(row, 16 * (h % 8))) = v;
          }
        } else if (p.flip) {
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            uint4* a = reinterpret_cast<uint4*>(smem + 8 * kBlk + sw128_offset(row, 16 * h));
            uint4 v = *a;
            v.x ^= p.flip, v.y ^= p.flip, v.z ^= p.flip, v.w ^= p.flip;
            *a = v;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      if (!ok) break;

      const int64_t g = (int64_t)s.b * kRows + row;
      const int nsee = mine ? sees(p, s.q, g) : 0;
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
        const int sb = i & 1;
        const uint32_t ph = (uint32_t)(i >> 1) & 1u;
        // the tile's two pages, while S is on its way
        const int32_t* bt = p.bt + (int64_t)s.r * p.bt_stride;
        const bool in1 = 2 * jt + 1 < p.bt_stride;
        const int32_t k0 = ldg_nc_s32(bt + (2 * jt < p.bt_stride ? 2 * jt : 0)), k1 = ldg_nc_s32(bt + (in1 ? 2 * jt + 1 : 0));
        ok = !*abort_flag && warp_wait_all(&s_full[sb], ph, p.err);
        ok = ok && warp_wait_all(&p_empty[sb], ph ^ 1u, p.err);
        if (!ok) break;
        tc_fence_after();
        fence_acq_rel_cluster();
        if (!idle) {
          const bool v0 = k0 >= 0 && ((int64_t)k0 + 1) * HS_PAGE <= p.R;
          const bool v1 = in1 && k1 >= 0 && ((int64_t)k1 + 1) * HS_PAGE <= p.R;
          const int lim = nsee - jt * kKeys;  // columns of this tile that the row sees
          const uint32_t sc = tmem + lane_base + kKeys * sb;
          const bool all = __all_sync(0xffffffffu, lim >= kKeys && v0 && v1);
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t x[32];
            tmem_ld32(sc + 32 * h, x);
            tmem_wait_ld();
            if (all) {
#pragma unroll
              for (int k = 0; k < 32; ++k) mx = fmaxf(mx, __uint_as_float(x[k]));
            } else if (h < 2 ? v0 : v1) {
#pragma unroll
              for (int k = 0; k < 32; ++k) mx = fmaxf(mx, 32 * h + k < lim ? __uint_as_float(x[k]) : -INFINITY);
            }
          }
          mx = mx == -INFINITY ? mx : mx * coef;
          const bool up = mx > ref + kThreshold;
          const bool moved = __any_sync(0xffffffffu, up);
          if (moved) {
            const float to = up ? mx : ref;
            const float al = up ? fast_exp2(ref - to) : 1.f;
            l *= al;
            ref = to;
            remote_st_f32(r_alpha + 4 * (128 * sb + row), al);
          }
          if (lane == 0) remote_st_u32(r_moved + 4 * (4 * sb + quad), moved ? 1u : 0u);
          const float me = ref == -INFINITY ? 0.f : ref;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t x[32], pk[16];
            tmem_ld32(sc + 32 * h, x);
            tmem_wait_ld();
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a = fast_exp2(fmaf(__uint_as_float(x[2 * k]), coef, -me));
              float b = fast_exp2(fmaf(__uint_as_float(x[2 * k + 1]), coef, -me));
              if (!all) {
                const bool v = h < 2 ? v0 : v1;
                a = v && 32 * h + 2 * k < lim ? a : 0.f;
                b = v && 32 * h + 2 * k + 1 < lim ? b : 0.f;
              }
              sum += a + b;
              pk[k] = pack_half2(a, b);
            }
            l += sum;
            const uint32_t blk = r_p + (uint32_t)((2 * sb + h / 2) * kBlk);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              remote_st_v4(blk + sw128_offset(row, 64 * (h & 1) + 16 * k), pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
          }
          if (jt == s.tb - 1) remote_st_f32(r_sum + 4 * (128 * sb + row), l);
        }
        // S has been read; P, the factors and the sums are on their way to B
        tc_fence_before();
        fence_proxy_async_all();
        fence_acq_rel_cluster();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_empty[sb]);
          remote_arrive(r_full + 8 * (uint32_t)sb);
        }
      }
      if (ok && mine) {
        const float v = l == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(l)) * kLn2;
        if (s.ta == 0 && s.tb == s.tiles) {
          if (p.lse) p.lse[(int64_t)s.q.start * p.H + g] = v;
        } else {
          p.part_lse[(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + row] = v;
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= kSmWarp0 && warp < kSmWarp0 + 4) {
    // ================================================================ B: rescaling, output ======
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const uint32_t back = remote_smem(p_empty, 0);
    const float* alpha = (const float*)(smem + kOffAlpha);
    const float* sums = (const float*)(smem + kOffSum);
    const uint32_t* moved = (const uint32_t*)(smem + kOffMoved);
    const int64_t C = U < p.clusters ? U : p.clusters;
    Desc desc = {0, 0, 0, 0};
    int64_t u = u0;
    Seg s;
    int i = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p, s)) {
      const bool idle = 32 * quad >= s.nrows;
      const int64_t row0 = (int64_t)s.q.start * p.H + (int64_t)s.b * kRows;
      if (s.ta == 0 && s.tb < s.tiles) {
        desc.row0 = (int32_t)row0;
        desc.nrows = s.nrows;
        desc.nparts = (int32_t)(unit_cta(u + s.tiles - 1, U, C) - c + 1);
      }
      u += s.tb - s.ta;
      float sum = 0.f;
#pragma unroll 1
      for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
        const int pb = i & 1;
        const uint32_t ph = (uint32_t)(i >> 1) & 1u;
        ok = !*abort_flag && __all_sync(0xffffffffu, mbar_wait_cluster(&p_full[pb], ph, p.err));
        if (!ok) break;
        if (!idle) {
          if (jt == s.tb - 1) sum = sums[128 * pb + row];
          if (moved[4 * pb + quad] && jt > s.ta) {
            const float al = alpha[128 * pb + row];
            ok = warp_wait_all(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 16; ++h) {
              uint32_t x[32];
              tmem_ld32(tmem + lane_base + 32 * h, x);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * al);
              tmem_st32(tmem + lane_base + 32 * h, x);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&corr[pb]);
          remote_arrive(back + 8 * (uint32_t)pb);
        }
      }
      if (ok) ok = warp_wait_all(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const bool whole = s.ta == 0 && s.tb == s.tiles;
        __nv_bfloat16* o = p.out + (row0 + row) * HS_D_LATENT;
        float* po = p.part_out + ((int64_t)(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + row) * HS_D_LATENT;
#pragma unroll 1
        for (int h = 0; h < 16; ++h) {
          uint32_t x[32];
          tmem_ld32(tmem + lane_base + 32 * h, x);
          tmem_wait_ld();
          if (row < s.nrows) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(x[8 * k + 2 * z]) * inv,
                                                                  __uint_as_float(x[8 * k + 2 * z + 1]) * inv);
                  w[z] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(o + 32 * h + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float4*>(po + 32 * h + 4 * k) =
                    make_float4(__uint_as_float(x[4 * k]) * inv, __uint_as_float(x[4 * k + 1]) * inv,
                                __uint_as_float(x[4 * k + 2]) * inv, __uint_as_float(x[4 * k + 3]) * inv);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
    if (!ok) *abort_flag = 1;
    if (warp == kSmWarp0 && lane == 0) p.desc[c] = desc;
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still write to it
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace paged

uint64_t paged_mla_workspace_bytes(int sms) {
  using namespace paged;
  const uint64_t c = (uint64_t)(sms / 2);
  return 2 * c * kRows * (HS_D_LATENT + 1) * 4 + c * sizeof(Desc);
}

cudaError_t launch_paged_mla(const hs_paged_mla_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace paged;
  CUtensorMap mq;
  if (!encode_2d(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a->q, HS_D_QK, (uint64_t)a->T * a->H, HS_D_QK * 2, 64, kRows,
                 CU_TENSOR_MAP_SWIZZLE_128B)) {
    *why = "cuTensorMapEncodeTiled failed for q";
    return cudaErrorInvalidValue;
  }
  const int C = sms / 2;
  Params p;
  p.T = a->T;
  p.B = a->B;
  p.H = a->H;
  p.causal = a->causal;
  p.bt_stride = a->bt_stride;
  p.clusters = C;
  p.q = reinterpret_cast<const uint8_t*>(a->q);
  p.kv = a->kv_pool;
  p.R = a->R;
  p.bt = a->block_table;
  p.req_start = a->req_start;
  p.seq_len = a->seq_len;
  p.kv_tokens = a->kv_tokens;
  p.scale_log2 = fabsf(a->softmax_scale) * kLog2e;
  p.flip = a->softmax_scale < 0.f ? 0x80008000u : 0u;
  p.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.err = a->err_flag;
  p.part_out = reinterpret_cast<float*>(a->workspace);
  p.part_lse = p.part_out + (int64_t)2 * C * kRows * HS_D_LATENT;
  p.desc = reinterpret_cast<Desc*>(p.part_lse + (int64_t)2 * C * kRows);
  cudaError_t e = cudaFuncSetAttribute(paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  paged_kernel<<<2 * C, kThreads, kSmem, stream>>>(mq, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  paged_merge_kernel<kRows><<<dim3((unsigned)C, kRows / kMergeRows), kMergeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace hs
