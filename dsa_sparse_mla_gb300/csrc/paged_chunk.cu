// paged_chunk.cu — dense attention of chunks of new tokens over the paged FP8 latent rows: four SMs per
// block of 256 (token, head) rows.
//
// The products, masks and splits are paged.cu's (S = Q K^T, P = 2^(c S - m), O = P V, per block of rows, the
// block's rows sharing all cached rows they see). With many rows per request two things change:
//  - A row is dequantised once per call, not once per block: expand_kernel writes each request's rows as
//    [512 fp16][64 bf16] to the workspace (1,152 bytes; a NaN code becomes zeros and a NaN rotary value, so that
//    only rows that see it are NaN), and TMA feeds the tensor cores from there.
//  - The two products run as two-SM MMAs (cta_group::2, M = 256): CTAs 0 and 1 of a cluster compute S and the softmax of
//    128 rows each, CTAs 2 and 3 keep those rows' O. Each CTA loads half of every K or V tile, which halves
//    the reads from L2 (a tile of 128 rows costs each CTA 74 or 64 KB per 256 rows) and from shared memory.
// Q's latent dims sit in tensor memory (256 columns beside two S buffers of 128) as the A operand, so that a QK
// MMA reads only K from shared memory.
//
// Per tile of 128 cached rows and cluster: QK 36 MMAs of M 256, N 128, K 16 (64 cycles each), PV 16 of N 256 (128
// cycles each) on the other pair: 2,304 cycles.
//
// Roles (384 threads). Softmax CTA: warp 0 loads K by TMA, warps 1 and 3 of CTA 0 issue QK, each for every other
// tile (the tensor core queues too little to stay busy while one warp waits and commits), warp 2 of CTA 1 tells CTA 0
// that its half of K is there, warps 4-11 are the softmax: thread = row and 64 of the tile's columns; two threads
// of a row agree on the maximum through shared memory. P goes through shared memory to the CTA that keeps the same
// rows' O, 4 KB per warp as one bulk copy. Output CTA: warp 0 loads V, warp 1 issues PV (CTA 2), warp 2 of CTA 3
// tells CTA 2 of its half of V, warp 3 arms P's barrier and hands P buffers back, warps 4-11 rescale O and write the
// result: thread = row and 256 of O's columns.
#include <atomic>

#include "paged.cuh"

namespace hs {
namespace paged {
namespace chunk {

constexpr int kThreads = 384;
constexpr int kRows = 256;
constexpr int kHalf = 128;                     // rows of a CTA
constexpr int kKBlk = 64 * 128;                // [64 keys][64 dims]: half a K block
constexpr int kKStage = 3 * kKBlk;             // three dim blocks
constexpr int kStA = 5;
constexpr int kVBlk = kKeys * 128;             // [128 keys][64 dims]
constexpr int kVStage = 2 * kVBlk;             // 128 of the 256 dims of one MMA
constexpr int kStB = 5;
constexpr int kPBuf = 2 * kHalf * 128;         // P of a tile: 2 x [128 rows][64 keys]
// softmax CTA: Q's rotary dims, K ring, P staging [2];  output CTA: P [2], V ring
constexpr int kOffQ = 0;
constexpr int kOffK = kHalf * 128;
constexpr int kOffStage = kOffK + kStA * kKStage;
constexpr int kOffP = 0;
constexpr int kOffV = 2 * kPBuf;
constexpr int kOffAlpha = 14 * 16384;          // float [2][128]: staging, and at the same place of the output CTA
constexpr int kOffSum = kOffAlpha + 1024;      // float [2][128]
constexpr int kOffBar = kOffSum + 1024;
constexpr int kNumBars = 40;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;
constexpr int kSmem = kOffMisc + 64;
constexpr int kOffMax = kOffStage + 2 * kPBuf; // softmax CTA: float [2][2][128]
constexpr int kOffScratch = kOffK;             // int64 [B + 1] during the set-up
static_assert(kOffMax + 2048 <= kOffAlpha && kOffV + kStB * kVStage <= kOffAlpha, "layout");
static_assert(kOffScratch + 8 * (kMaxReq + 1) <= kOffAlpha && kSmem <= 232448, "shared memory");
static_assert(kOffK % 1024 == 0 && kOffStage % 1024 == 0 && kOffV % 1024 == 0, "swizzled blocks");

// ------------------------------------------------------------------ dequantisation ---------
// One warp per row: lane l turns codes 16 l .. + 15 into fp16, lanes 0-7 copy the rotary values. Rows past a
// request's length (its last tile) and rows of a bad page are zeros. HBM-bound: 656 bytes read, 1,152 written.
constexpr int kExpandThreads = 512;
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const Params p, uint16_t* out) {
  __shared__ int64_t pre[kMaxReq + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    int64_t run = 0, cached = 0;
    if (lane == 0) pre[0] = 0;
    for (int at = 0; at < p.B; at += 32) {
      Req q = {0, 0, 0, 0};
      if (at + lane < p.B) q = load_req<kRows>(p, at + lane);
      const int64_t x = warp_scan(copy_rows(q), lane);
      if (at + lane < p.B) pre[at + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
      cached += q.seq;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cached += __shfl_xor_sync(0xffffffffu, cached, o);
    if (cached > p.kv_tokens && lane == 0) pre[p.B] = -1;  // nothing is computed
  }
  __syncthreads();
  const int64_t total = pre[p.B];
  bool range_ok = true;
  // 16 consecutive rows per warp and turn (a quarter of a page)
  for (int64_t w = (int64_t)blockIdx.x * (kExpandThreads / 32) + warp; w * 16 < total; w += (int64_t)gridDim.x * (kExpandThreads / 32)) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= w * 16)
        lo = mid;
      else
        hi = mid;
    }
    const int j0 = (int)(w * 16 - pre[lo]);
    const int seq = load_req<kRows>(p, lo).seq;
    const int32_t blk = j0 / HS_PAGE < p.bt_stride ? p.bt[(int64_t)lo * p.bt_stride + j0 / HS_PAGE] : -1;
    const bool good = blk >= 0 && ((int64_t)blk + 1) * HS_PAGE <= p.R;
    if (!good && j0 < seq && lane == 0) flag_error(p.err, HS_FLAG_BAD_BLOCK);
    const int n = good ? min(16, seq - j0) : 0;  // rows that exist
    const uint8_t* src = p.kv + ((int64_t)(good ? blk : 0) * HS_PAGE + j0 % HS_PAGE) * HS_KV_ROW_BYTES;
    uint16_t* dst = out + w * 16 * HS_D_QK;
#pragma unroll 1
    for (int h = 0; h < 16; h += 4) {
      uint4 v[4], r[4];
      float s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = r[k] = make_uint4(0, 0, 0, 0);
        s[k] = 0.f;
        if (h + k < n) {
          const uint8_t* a = src + (h + k) * HS_KV_ROW_BYTES;
          v[k] = ldg_nc_v4(a + 16 * lane);
          s[k] = ldg_nc_f32(a + HS_D_LATENT + 4 * (lane >> 3));
          if (lane < 8) r[k] = ldg_nc_v4(a + HS_D_LATENT + 16 + 16 * lane);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        range_ok &= h + k >= n || (fabsf(s[k]) >= kScaleMin && fabsf(s[k]) <= kScaleMax);
        const __half shi = __float2half_rn(s[k]);
        const __half2 h2 = __half2half2(shi), l2 = __float2half2_rn(s[k] - __half2float(shi));
        const uint32_t hu = *reinterpret_cast<const uint32_t*>(&h2), lu = *reinterpret_cast<const uint32_t*>(&l2);
        uint4 d0 = dequant8(v[k].x, v[k].y, hu, lu), d1 = dequant8(v[k].z, v[k].w, hu, lu);
        const bool bad = unsound(d0, d1);
        if (bad) d0 = d1 = make_uint4(0, 0, 0, 0);
        if (__any_sync(0xffffffffu, bad) && lane == 0) r[k].x = 0x7FC07FC0u;  // two bf16 NaN
        uint4* d = reinterpret_cast<uint4*>(dst + (h + k) * HS_D_QK);
        d[2 * lane] = d0;
        d[2 * lane + 1] = d1;
        if (lane < 8) d[64 + lane] = r[k];
      }
    }
  }
  if (!range_ok) flag_error(p.err, HS_FLAG_RANGE);
}

// ------------------------------------------------------------------ attention --------------
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in every CTA
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  uint64_t* bars = (uint64_t*)(smem + kOffBar);
  uint64_t* full = bars;            // [5] this CTA's half of a stage has landed; in the issuing CTA the other's too
  uint64_t* empty = bars + 10;      // [5] the MMAs have read the stage (both CTAs)
  uint64_t* s_full = bars + 15;     // [2] S complete (both)
  uint64_t* s_empty = bars + 17;    // [2] CTA 0: both CTAs' softmax warps have read S
  uint64_t* p_empty = bars + 19;    // [2] softmax CTA: its P buffer and staging are free
  uint64_t* p_full = bars + 21;     // [2] output CTA: P and the factors have landed
  uint64_t* corr = bars + 23;       // [2] CTA 2: both CTAs have rescaled O for this P
  uint64_t* pv_done = bars + 25;    // [2] PV complete (both)
  uint64_t* q_ready = bars + 27;    // CTA 0: both CTAs' Q is in place
  uint64_t* q_free = bars + 28;     // the block's QK MMAs have read Q (both)
  uint64_t* o_free = bars + 29;     // CTA 2: both CTAs have read O out
  uint64_t* drain = bars + 30;
  uint64_t* drain2 = bars + 35;
  uint64_t* swap = bars + 31;       // [4] softmax CTA: the two warps of a lane quarter have written their values
  uint32_t* misc = (uint32_t*)(smem + kOffMisc);
  volatile uint32_t* abort_flag = misc + 1;
  Start* st = (Start*)(misc + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool isA = rank < 2, lead = (rank & 1) == 0;
  const uint16_t pair_mask = isA ? 0x3 : 0xC;
  const int c = blockIdx.x >> 2;

  if (tid == 0) {
    for (int s = 0; s < 5; ++s) {
      mbar_init(&full[s], lead ? 2 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 16);
      mbar_init(&p_empty[s], 1);
      mbar_init(&p_full[s], 1);
      mbar_init(&corr[s], 16);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_ready, 16);
    mbar_init(q_free, 2);
    mbar_init(o_free, 16);
    mbar_init(drain, 1);
    mbar_init(drain2, 1);
    for (int q = 0; q < 4; ++q) mbar_init(&swap[q], 2);
    mbar_fence_init();
    misc[1] = 0;
  }
  find_units<kRows>(p, (int64_t*)(smem + kOffScratch), st, c, kThreads);
  fence_proxy_async_all();
  __syncthreads();
  cluster_sync();  // every CTA's barriers exist
  if (warp == 0) tmem_alloc2(&misc[0], 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int64_t u0 = st->u0, ntiles = st->u1 - st->u0, U = st->U;
  Walk<kRows> walk(p, *st);
  Seg s;

  if (warp == 0) {
    // ================================================================ loads =====================
    if (lane == 0) {
      const CUtensorMap* map = isA ? &map_k : &map_v;
      prefetch_tensormap(map);
      const int half = (int)(rank & 1), slots = isA ? kStA : kStB;
      int slot = 0;
      uint32_t par = 1;
      int64_t issued = 0;
      bool ok = true;
#pragma unroll 1
      while (ok && walk.next(p, s)) {
#pragma unroll 1
        for (int jt = s.ta; jt < s.tb && ok; ++jt) {
          const int32_t y = (int32_t)(s.base + (int64_t)jt * kKeys);
#pragma unroll 1
          for (int k = 0; k < (isA ? 3 : 2); ++k) {
            if (*abort_flag || !mbar_wait(&empty[slot], par, p.err)) {
              ok = false;
              break;
            }
            if (isA) {  // dim blocks 3 k .. + 2, this CTA's 64 keys
              mbar_arrive_expect_tx(&full[slot], kKStage);
              uint8_t* d = smem + kOffK + slot * kKStage;
#pragma unroll
              for (int b = 0; b < 3; ++b) tma_load_2d(d + b * kKBlk, map, &full[slot], 64 * (3 * k + b), y + 64 * half);
            } else {    // dims 256 k + 128 half .. + 127, all keys
              mbar_arrive_expect_tx(&full[slot], kVStage);
              uint8_t* d = smem + kOffV + slot * kVStage;
#pragma unroll
              for (int b = 0; b < 2; ++b) tma_load_2d(d + b * kVBlk, map, &full[slot], 256 * k + 128 * half + 64 * b, y);
            }
            ++issued;
            if (++slot == slots) {
              slot = 0;
              par ^= 1u;
            }
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // every copy has landed before the CTA may leave
      for (int64_t j = issued > slots ? issued - slots : 0; j < issued; ++j) mbar_wait(&full[j % slots], (uint32_t)(j / slots) & 1u, p.err);
    }
  } else if (lead && (warp == 1 || (warp == 3 && isA))) {
    // ================================================================ MMAs ======================
    if (lane == 0) {
      int slot = 0, i = 0, n = 0;
      uint32_t par = 0;
      bool ok = true;
      const int slots = isA ? kStA : kStB;
      auto stage = [&]() -> bool {  // both halves of the next stage
        const bool r = mbar_wait(&full[slot], par, p.err);
        tc_fence_after();
        return r;
      };
      auto skip = [&](int k) {
        slot += k;
        if (slot >= slots) {
          slot -= slots;
          par ^= 1u;
        }
      };
      auto pass = [&]() {
        mma2_commit(&empty[slot], pair_mask);
        skip(1);
      };
      if (isA) {
        constexpr uint32_t lat = idesc_f16(kRows, kKeys, 0, 0), rop = idesc_bf16(kRows, kKeys, 0, 0);
        const uint64_t qd = smem_desc(smem_u32(smem + kOffQ), 16, 1024, 2);
        const uint64_t kd = smem_desc(smem_u32(smem + kOffK), 16, 1024, 2);
        const int mine = warp == 1 ? 0 : 1;  // the parity of the tiles that this warp issues
#pragma unroll 1
        for (; ok && walk.next(p, s); ++n) {
          if (!mbar_wait_cluster(q_ready, (uint32_t)n & 1u, p.err)) {
            ok = false;
            break;
          }
          fence_proxy_async_all();
#pragma unroll 1
          for (int jt = s.ta; jt < s.tb && ok; ++jt, ++i) {
            if ((i & 1) != mine) {
              skip(3);
              continue;
            }
            const uint32_t d = tmem + kKeys * mine;
            if (*abort_flag || !mbar_wait(&s_empty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              if (!stage()) {
                ok = false;
                break;
              }
              const uint64_t kb = kd + (uint64_t)((slot * kKStage) >> 4);
#pragma unroll
              for (int b = 0; b < 3; ++b)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t bd = kb + (uint64_t)((b * kKBlk + kk * 32) >> 4);
                  if (3 * k + b < 8)
                    mma2_f16_ts(d, tmem + 256 + 32 * (3 * k + b) + 8 * kk, bd, lat, (k | b | kk) != 0 ? 1u : 0u);
                  else
                    mma2_f16_ss(d, qd + (uint64_t)((kk * 32) >> 4), bd, rop, 1u);
                }
              pass();
            }
            if (ok) mma2_commit(&s_full[i & 1], pair_mask);
          }
          if (ok) mma2_commit(q_free, pair_mask);
        }
      } else {
        constexpr uint32_t id = idesc_f16(kRows, 256, 0, 1);
        const uint64_t pd = smem_desc(smem_u32(smem + kOffP), 16, 1024, 2);
        const uint64_t vd = smem_desc(smem_u32(smem + kOffV), kVBlk, 1024, 2);
#pragma unroll 1
        for (; ok && walk.next(p, s); ++n) {
          if (n > 0 && !mbar_wait(o_free, (uint32_t)(n - 1) & 1u, p.err)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int jt = s.ta; jt < s.tb && ok; ++jt, ++i) {
            if (*abort_flag || !mbar_wait(&corr[i & 1], (uint32_t)(i >> 1) & 1u, p.err)) {
              ok = false;
              break;
            }
            const uint64_t pb = pd + (uint64_t)(((i & 1) * kPBuf) >> 4);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (!stage()) {
                ok = false;
                break;
              }
              const uint64_t vb = vd + (uint64_t)((slot * kVStage) >> 4);
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma2_f16_ss(tmem + 256 * k, pb + (uint64_t)(((kk / 4) * (kPBuf / 2) + (kk % 4) * 32) >> 4),
                            vb + (uint64_t)((kk * 2048) >> 4), id, (jt > s.ta || kk > 0) ? 1u : 0u);
              pass();
            }
            if (ok) mma2_commit(&pv_done[i & 1], pair_mask);
          }
        }
      }
      if (!ok) *abort_flag = 1;
      uint64_t* done = warp == 1 ? drain : drain2;
      mma2_commit(done, (uint16_t)(1u << rank));
      mbar_wait(done, 0, p.err);
    }
  } else if (warp == 2 && !lead) {
    // ================================================================ the other half is there ===
    if (lane == 0) {
      const uint32_t to = remote_smem(full, rank - 1);
      const int slots = isA ? kStA : kStB;
      const int64_t stages = ntiles * (isA ? 3 : 2);
      int slot = 0;
      uint32_t par = 0;
#pragma unroll 1
      for (int64_t j = 0; j < stages; ++j) {
        if (*abort_flag || !mbar_wait(&full[slot], par, p.err)) {
          *abort_flag = 1;
          break;
        }
        remote_arrive_relaxed(to + 8 * (uint32_t)slot);
        if (++slot == slots) {
          slot = 0;
          par ^= 1u;
        }
      }
    }
  } else if (warp == 3 && !isA) {
    // ================================================================ P buffers =================
    // Arms a buffer's barrier with the bytes that its tile brings (4 KB of P and 128 bytes of factors per
    // 32 rows, at a block's last tile 128 bytes of sums), then hands it to the softmax CTA.
    if (lane == 0) {
      const uint32_t back = remote_smem(p_empty, rank - 2);
      int i = 0;
      bool ok = true;
#pragma unroll 1
      while (ok && walk.next(p, s)) {
        const int left = s.nrows - (int)(rank & 1) * kHalf;
        const uint32_t quads = left <= 0 ? 0 : left >= kHalf ? 4 : (uint32_t)(left + 31) / 32;
#pragma unroll 1
        for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
          if (i >= 2 && (*abort_flag || !mbar_wait(&pv_done[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err))) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&p_full[i & 1], quads * (8192u + 128u + (jt == s.tb - 1 ? 128u : 0u)));
          remote_arrive_relaxed(back + 8 * (uint32_t)(i & 1));
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else if (warp >= 4 && isA) {
    // ================================================================ softmax ===================
    const int quad = warp & 3, g = (warp - 4) >> 2, row = 32 * quad + lane;  // g: columns 64 g .. + 63
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const uint32_t to = rank + 2;
    const uint32_t r_p = remote_smem(smem + kOffP, to), r_alpha = remote_smem(smem + kOffAlpha, to), r_sum = remote_smem(smem + kOffSum, to);
    const uint32_t r_full = remote_smem(p_full, to), r_sempty = remote_smem(s_empty, 0), r_qready = remote_smem(q_ready, 0);
    float* smax = (float*)(smem + kOffMax);  // [2][2][128]
    float* salpha = (float*)(smem + kOffAlpha);
    float* ssum = (float*)(smem + kOffSum);
    int n = 0, i = 0, x = 0;  // x: exchanges through smax, alternating halves
    bool ok = true;
    // The row's two threads give each other a value. The wait is bounded like every other (ok turns false).
    auto other = [&](float v) -> float {
      float* at = smax + 256 * (x & 1);
      at[128 * g + row] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&swap[quad]);
      ok = warp_wait_all(&swap[quad], (uint32_t)x & 1u, p.err);
      ++x;
      return at[128 * (g ^ 1) + row];
    };
#pragma unroll 1
    for (; ok && walk.next(p, s); ++n) {
      const int64_t grow = (int64_t)s.b * kRows + (int64_t)rank * kHalf + row;  // of the request's rows
      const int have = s.nrows - (int)rank * kHalf;                            // rows of this CTA that exist
      const bool idle = 32 * quad >= have, mine = row < have;
      float coef = p.scale_log2;
      if (n > 0) ok = warp_wait_all(q_free, (uint32_t)(n - 1) & 1u, p.err);
      if (ok && !idle) {
        // This thread's half of Q's row: latent dims 256 g .. + 255 to fp16 in tensor memory, rotary dims 32 g .. + 31 to
        // shared memory. A row whose largest latent value is outside [2^-6, 2^15) is scaled by a power of two that puts it
        // in [2^14, 2^15); its logits are scaled back.
        const uint8_t* src = p.q + ((int64_t)s.q.start * p.H + (mine ? grow : (int64_t)s.b * kRows)) * (HS_D_QK * 2) + 512 * g;
        uint32_t mx = 0u;
#pragma unroll 4
        for (int h = 0; h < 32; ++h) {
          const uint4 v = ldg_nc_v4(src + 16 * h);
          mx = __vmaxu2(__vmaxu2(mx, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
          mx = __vmaxu2(__vmaxu2(mx, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
        }
        uint32_t amax = max(mx & 0xFFFFu, mx >> 16);
        amax = max(amax, __float_as_uint(other(__uint_as_float(amax))));
        int e = 0;
        if (amax >= 0x7F80u) {
          if (mine) flag_error(p.err, HS_FLAG_RANGE);
        } else if (amax >= 0x4700u || (amax >= 0x0080u && amax < 0x3C80u)) {
          e = 14 - ((int)(amax >> 7) - 127);
        } else if (amax > 0u && amax < 0x0080u) {
          e = 126;
        }
        e = e < -126 ? -126 : (e > 126 ? 126 : e);
        const float f = __uint_as_float((uint32_t)(e + 127) << 23);
        coef *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {  // 64 dims: 32 columns
          uint32_t w[32];
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const uint4 v = ldg_nc_v4(src + 128 * b + 16 * h);
            w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint32_t u = w[k] ^ p.flip;
            w[k] = pack_half2(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f);
          }
          tmem_st32(tmem + lane_base + 256 + 128 * g + 32 * b, w);
        }
        tmem_wait_st();
        const uint8_t* rsrc = src + 1024 - 512 * g + 64 * g;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint4 v = ldg_nc_v4(rsrc + 16 * h);
          uint32_t* w = &v.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t u = w[k] ^ p.flip;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xFFFF0000u) * f);
            w[k] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          *reinterpret_cast<uint4*>(smem + kOffQ + sw128_offset(row, 64 * g + 16 * h)) = v;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(r_qready);
      if (!ok) break;

      const int nsee = mine ? sees(p, s.q, grow) : 0;
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
        const int b = i & 1;
        const uint32_t ph = (uint32_t)(i >> 1) & 1u;
        // this warp's page of the tile, while S is on its way
        const int page = 2 * jt + g;
        const int32_t k = ldg_nc_s32(p.bt + (int64_t)s.r * p.bt_stride + (page < p.bt_stride ? page : 0));
        ok = !*abort_flag && warp_wait_all(&s_full[b], ph, p.err);
        if (!ok) break;
        tc_fence_after();
        if (idle) {
          __syncwarp();
          if (lane == 0) remote_arrive_relaxed(r_sempty + 8 * (uint32_t)b);
          continue;
        }
        uint32_t v[64];
        {
          const uint32_t at = tmem + lane_base + kKeys * b + 64 * g;
          uint32_t a0[32], a1[32];
          tmem_ld32(at, a0);
          tmem_ld32(at + 32, a1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = a0[j], v[32 + j] = a1[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) remote_arrive_relaxed(r_sempty + 8 * (uint32_t)b);
        const bool there = page < p.bt_stride && k >= 0 && ((int64_t)k + 1) * HS_PAGE <= p.R;
        const int lim = there ? nsee - jt * kKeys - 64 * g : 0;  // columns that this thread's row sees
        if (!__all_sync(0xffffffffu, lim >= 64)) {
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = j < lim ? v[j] : 0xFF800000u;  // -inf
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 64; j += 2) m0 = fmaxf(m0, __uint_as_float(v[j])), m1 = fmaxf(m1, __uint_as_float(v[j + 1]));
        float mx = fmaxf(m0, m1);
        mx = fmaxf(mx, other(mx));
        if (!ok) break;
        mx = mx == -INFINITY ? mx : mx * coef;
        const bool up = mx > ref + kThreshold;
        const float to_ref = up ? mx : ref;
        const float al = up ? fast_exp2(ref - to_ref) : 1.f;
        l *= al;
        ref = to_ref;
        const float me = ref == -INFINITY ? 0.f : ref;
        // masked columns are -inf: their P is 0 (where a row's own values are infinite or NaN, so is its result)
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float a = v[2 * j] == 0xFF800000u ? 0.f : fast_exp2(fmaf(__uint_as_float(v[2 * j]), coef, -me));
          const float c2 = v[2 * j + 1] == 0xFF800000u ? 0.f : fast_exp2(fmaf(__uint_as_float(v[2 * j + 1]), coef, -me));
          s0 += a;
          s1 += c2;
          v[j] = pack_half2(a, c2);
        }
        l += s0 + s1;
        const bool last = jt == s.tb - 1;
        float sum = 0.f;
        if (last) {
          sum = l + other(l);
          if (!ok) break;
          if (g == 0 && mine) {
            const float z = sum == 0.f ? -INFINITY : (me + log2f(sum)) * kLn2;
            if (s.ta == 0 && s.tb == s.tiles) {
              if (p.lse) p.lse[(int64_t)s.q.start * p.H + grow] = z;
            } else {
              p.part_lse[(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + rank * kHalf + row] = z;
            }
          }
        }
        ok = warp_wait_all(&p_empty[b], ph, p.err);
        if (!ok) break;
        uint8_t* blk = smem + kOffStage + b * kPBuf + g * (kPBuf / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(blk + sw128_offset(row, 16 * j)) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        if (g == 0) {
          salpha[128 * b + row] = al;
          if (last) ssum[128 * b + row] = sum;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = r_full + 8 * (uint32_t)b, off = (uint32_t)(b * kPBuf + g * (kPBuf / 2) + 32 * quad * 128);
          bulk_s2remote(r_p + off, smem + kOffStage + off, 4096, bar);
          if (g == 0) {
            const uint32_t o4 = 4 * (uint32_t)(128 * b + 32 * quad);
            bulk_s2remote(r_alpha + o4, smem + kOffAlpha + o4, 128, bar);
            if (last) bulk_s2remote(r_sum + o4, smem + kOffSum + o4, 128, bar);
          }
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 4) {
    // ================================================================ rescaling, output =========
    const int quad = warp & 3, g = (warp - 4) >> 2, row = 32 * quad + lane;  // g: O's columns 256 g .. + 255
    const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + 256 * g;
    const uint32_t half = rank & 1;
    const uint32_t r_corr = remote_smem(corr, 2), r_ofree = remote_smem(o_free, 2);
    const float* alpha = (const float*)(smem + kOffAlpha);
    const float* sums = (const float*)(smem + kOffSum);
    const int64_t C = U < p.clusters ? U : p.clusters;
    Desc desc = {0, 0, 0, 0};
    int64_t u = u0;
    int i = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p, s)) {
      const int have = s.nrows - (int)half * kHalf;
      const bool idle = 32 * quad >= have;
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
        const int b = i & 1;
        ok = !*abort_flag && warp_wait_all(&p_full[b], (uint32_t)(i >> 1) & 1u, p.err);
        if (!ok) break;
        if (!idle) {
          if (jt == s.tb - 1) sum = sums[128 * b + row];
          const float al = alpha[128 * b + row];
          if (__any_sync(0xffffffffu, al != 1.f) && jt > s.ta) {
            ok = warp_wait_all(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 8; ++h) {
              uint32_t v[32];
              tmem_ld32(at + 32 * h, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * al);
              tmem_st32(at + 32 * h, v);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        __syncwarp();
        if (lane == 0) remote_arrive_relaxed(r_corr + 8 * (uint32_t)b);
      }
      if (ok) ok = warp_wait_all(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const bool whole = s.ta == 0 && s.tb == s.tiles, mine = row < have;
        const int64_t r = (int64_t)half * kHalf + row;
        __nv_bfloat16* o = p.out + (row0 + r) * HS_D_LATENT + 256 * g;
        float* po = p.part_out + ((int64_t)(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + r) * HS_D_LATENT + 256 * g;
#pragma unroll 1
        for (int h = 0; h < 8; ++h) {
          uint32_t v[32];
          tmem_ld32(at + 32 * h, v);
          tmem_wait_ld();
          if (mine) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const __nv_bfloat162 b2 =
                      __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * z]) * inv, __uint_as_float(v[8 * k + 2 * z + 1]) * inv);
                  w[z] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(o + 32 * h + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float4*>(po + 32 * h + 4 * k) =
                    make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                                __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive_relaxed(r_ofree);
    }
    if (!ok) *abort_flag = 1;
    if (rank == 2 && warp == 4 && lane == 0) p.desc[c] = desc;
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may still write to it
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

}  // namespace chunk
}  // namespace paged

// Rows of the dequantised copy: every request's last tile is whole.
static int64_t chunk_rows(int B, int64_t kv_tokens) { return kv_tokens + (int64_t)B * paged::kKeys; }

uint64_t paged_chunk_workspace_bytes(int B, int64_t kv_tokens, int sms) {
  using namespace paged;
  const uint64_t c = (uint64_t)(sms / 4);
  return 2 * c * chunk::kRows * (HS_D_LATENT + 1) * 4 + c * sizeof(Desc) + 16 + (uint64_t)chunk_rows(B, kv_tokens) * HS_D_QK * 2;
}

cudaError_t launch_paged_chunk(const hs_paged_mla_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace paged;
  using namespace paged::chunk;
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int most = sms / 4;
  // Clusters that run at once: the SMs of a GPC need not be a multiple of four. Asked once per device.
  static std::atomic<int> asked[64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int C = dev < 64 ? asked[dev].load(std::memory_order_relaxed) : 0;
  if (C == 0) {
    C = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4 * most);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {4, 1, 1};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, chunk_kernel, &cfg) == cudaSuccess && n > 0 && n < C) C = n;
    if (dev < 64) asked[dev].store(C, std::memory_order_relaxed);
  }
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
  p.part_lse = p.part_out + (int64_t)2 * most * kRows * HS_D_LATENT;
  p.desc = reinterpret_cast<Desc*>(p.part_lse + (int64_t)2 * most * kRows);
  uint16_t* rows = reinterpret_cast<uint16_t*>(p.desc + most);
  p.rows16 = rows;
  const uint64_t n = (uint64_t)chunk_rows(a->B, a->kv_tokens);
  CUtensorMap mk, mv;
  if (!encode_2d(&mk, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows, HS_D_QK, n, HS_D_QK * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&mv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows, HS_D_QK, n, HS_D_QK * 2, 64, kKeys, CU_TENSOR_MAP_SWIZZLE_128B)) {
    *why = "cuTensorMapEncodeTiled failed for the dequantised rows";
    return cudaErrorInvalidValue;
  }
  expand_kernel<<<4 * sms, kExpandThreads, 0, stream>>>(p, rows);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  chunk_kernel<<<4 * C, kThreads, kSmem, stream>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  paged_merge_kernel<kRows><<<dim3((unsigned)C, kRows / kMergeRows), kMergeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace hs
