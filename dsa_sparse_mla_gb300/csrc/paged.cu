// paged.cu — dense attention of each request's new tokens over its paged FP8 latent rows (MLA in MQA
// form), on tcgen05.
//
// [P1] "vLLM v0.32.0 GLM-5.3 サービング ...", sections 「再現方法と必要なフラグ」 and 「数字がうまくいく理由」:
// every cached row serves all heads; QK runs over 576 dims (512 latent + 64 RoPE), PV over the 512
// latent dims. A request's (token, head) pairs are the rows of one softmax attention:
//   S = Q K^T,  P = 2^(c S - m),  O = P V,  out = O / sum P,     V = the first 512 dims of K.
//
// Why the two products run on different SMs. O of 128 rows and 512 fp32 dims fills an SM's tensor memory, so S has no
// place beside it; 64 rows per SM would halve the work per cached row and pay the fixed cost of small MMAs. Here
// one half of a cluster computes S and the softmax, the other keeps O and computes PV, each with 128 rows per SM
// at the tensor core's full rate: per tile of 128 cached rows 2,304 cycles of QK, 2,048 of PV.
//
// Products are two-SM MMAs (cta_group::2, M = 256): blocks of 256 rows, and each CTA of a pair brings half of every K or V
// tile, which halves what it reads from L2, dequantises, and feeds its tensor core from shared memory. A cluster is the
// softmax pair (ranks 0, 1) and the output pair (ranks 2, 3).
//
// Two variants, chosen by copies() below (requests with few rows go to paged_few.cu):
//   raw   eight (softmax CTA) or six (output CTA) producer warps dequantise the rows' codes, which TMA brings as they lie in
//         the pool, to fp16 (code * group scale rounded once) in 128-byte-swizzled blocks.
//   copy  expand_kernel first writes every row dequantised to the workspace ([512 fp16][64 bf16], 1,152 bytes), and TMA brings
//         the blocks from there.
// Q's latent dims sit in tensor memory as the A operand (256 columns beside two S buffers of 128), so that a QK MMA reads
// only K from shared memory.
//
// Work. Units are (block of rows, 128 cached rows); every cluster takes an equal share of all units of the batch, found by
// prefix sums at the start (no plan on the host, which does not know the lengths). A block whose units span
// clusters leaves fp32 partial outputs and their log-sum-exps in the workspace; paged_merge_kernel joins them.
//
// Roles. Softmax CTA: warp 1 loads K (raw: codes, scales, rotary blocks); warps 0 and 3 of the issuing CTA issue QK, each for
// every other tile (the tensor core queues too little to stay busy while one warp waits and commits); warp 2 of the other CTA
// tells that its half is there; warps 4-11 are the softmax: thread = row and 64 of the tile's columns, the two threads of a
// row agree on the maximum through shared memory. P goes through shared memory to the CTA that keeps the same rows' O,
// 4 KB per warp as one bulk copy. Output CTA: warp 1 loads V, warp 0 of the issuing CTA issues PV, warp 2 of the other as above,
// warp 3 arms P's barriers and hands P buffers back, one more warp (2 or 0) looks at each tile's factors and wakes warps
// 4-11, which rescale O and write the result: thread = row and 256 of O's columns. raw adds a warp that splits scales and the
// producers (warps 12-19).
//
// Measured on a GB300 (events, inputs far larger than L2). copy, 2,048 tokens x 64 heads over 32,768 rows: 6.1 to 6.4 ms,
// 1,420 to 1,490 TFLOP/s, 0.72 to 0.76 of a bf16 matrix product's burst rate and 0.80 to 0.84 of its sustained rate; about 3,170 cycles per tile, of which QK's MMAs take
// 2,304. raw, 64 requests x 4 tokens x 64 heads over 16-65 thousand rows: 1.15 ms, 1,155 TFLOP/s; about 3,600 cycles per
// tile, the sum of hand-offs (codes -> producers -> K -> S -> P): no single unit is busy all the time, and
// more or fewer producer warps, deeper code rings, whole pages as bulk copies and single or double P buffers change it by less
// than 3 %.
//
// Lazy maximum: a row's reference max moves only when a logit exceeds it by more than 2^8 (P, held 2^7 times as large, stays
// below 2^15, inside fp16); then its factor goes along with P and O's row is rescaled. Masked columns are selected away before the
// maximum and the exponential, so what they hold does not matter; V values that fp16 cannot hold are zeroed, so that P = 0
// times them is 0, while K keeps them (the copy: a NaN in the rotary part), so that rows that see them are NaN.
#include <atomic>

#include "paged.cuh"

namespace hs {
namespace paged {

constexpr int G = 2;                           // CTAs that share a product
constexpr int kHalf = 128;                     // rows of a CTA
constexpr int kPBuf = 2 * kHalf * 128;         // P of a tile: 2 x [128 rows][64 keys]
// Roles by warp (warp w runs on sub-partition w % 4).
constexpr int kIssue0 = 0, kIssue1 = 3, kLoadWarp = 1, kRelayWarp = 2, kBufWarp = 3, kSmWarp0 = 4;
constexpr int kScaleWarpB = 12;  // splits scales in the output CTA; in the softmax CTA warp 2 (issuing) or 0 does
// Producers, two groups of kProd warps: softmax CTA 12-15 and 16-19, output CTA 13-15 and 17-19. Index of warp w, or -1.
__host__ __device__ constexpr int producer_index(int w, bool isA) { return w < 12 ? -1 : isA ? w - 12 : w % 4 == 0 ? -1 : w - 13 - (w - 12) / 4; }
static_assert(producer_index(13, false) == 0 && producer_index(15, false) == 2 && producer_index(17, false) == 3 && producer_index(19, false) == 5, "roles");
constexpr int kVBlk = kKeys * 128;             // [128 keys][64 dims]
constexpr int kVStage = 2 * kVBlk;             // 128 dims
constexpr int kMaxSlots = 8;
// Shared memory. Softmax CTA: Q's rotary dims, P staging [2], exchange, then the K ring (and raw: codes, scales);
// output CTA: P [2], exchange unused, V ring (and codes, scales). Both: factors, sums, barriers.
constexpr int kOffQ = 0;
constexpr int kOffStage = kHalf * 128;
constexpr int kOffMax = kOffStage + 2 * kPBuf; // softmax CTA: float [2][2][128]
constexpr int kOffK = kOffMax + 2048;
constexpr int kOffP = 0;
constexpr int kOffV = 2 * kPBuf;
constexpr int kOffAlpha = 14 * 16384;          // float [2][128]: staging, and at the same place of the output CTA
constexpr int kOffSum = kOffAlpha + 1024;      // float [2][128]
constexpr int kOffBar = kOffSum + 1024;
constexpr int kNumBars = 58;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;
constexpr int kSmem = kOffMisc + 128;
constexpr int kOffScratch = kOffK;             // int64 [B + 1] and int32 [B + 1] during the set-up
static_assert(kOffScratch + 12 * (kMaxReq + 1) <= kOffAlpha && kSmem <= 232448, "shared memory");
static_assert(kOffK % 1024 == 0 && kOffStage % 1024 == 0 && kOffV % 1024 == 0, "swizzled blocks");

// What differs between the variants.
template <bool kRaw>
struct Shape {
  static constexpr int kThreads = kRaw ? 640 : 384;
  static constexpr int kRows = kHalf * G;          // rows of a block
  static constexpr int kMine = kKeys / G;          // keys of a K block in one CTA
  static constexpr int kKBlk = kMine * 128;        // [kMine keys][64 dims]
  // K stages of a tile in the ring: raw four latent groups of two blocks (the rotary block has two buffers of its own), TMA
  // three times three blocks
  static constexpr int kBlocks = kRaw ? 2 : 3;
  static constexpr int kStages = kRaw ? 4 : 3;
  static constexpr int kKStage = kBlocks * kKBlk;
  static constexpr int kStA = kRaw ? 4 : 5;
  static constexpr int kVStages = 4 / G;           // per tile; an MMA takes 128 G dims of one
  static constexpr int kStB = kRaw ? 2 : 5;
  // raw: rotary blocks [2], rings of undecoded latent groups ([keys][128 codes]), two tiles' scales ([keys][4]) and those
  // split into fp16 pairs ([4 groups][keys])
  static constexpr int kCodesA = kMine * 128, kCodesB = kKeys * 128;
  static constexpr int kSlotsA = 6, kSlotsB = 4;   // of the rings of codes
  static constexpr int kOffRotary = kOffK + kStA * kKStage;
  static constexpr int kOffCodesA = kOffRotary + 2 * kKBlk, kOffCodesB = kOffV + kStB * kVStage;
  static constexpr int kOffScaleA = kOffCodesA + kSlotsA * kCodesA, kOffScaleB = kOffCodesB + kSlotsB * kCodesB;
  static constexpr int kOffSplitA = kOffScaleA + 2 * kMine * 16, kOffSplitB = kOffScaleB + 2 * kKeys * 16;
  static_assert(!kRaw || (kOffSplitA + 8 * kMine * 8 <= kOffAlpha && kOffSplitB + 8 * kKeys * 8 <= kOffAlpha), "layout");
  static_assert(kOffK + kStA * kKStage <= kOffAlpha && kOffV + kStB * kVStage <= kOffAlpha, "layout");
};
constexpr int kRotaryBar = 6;  // raw: full and empty barriers 6 and 7 belong to the rotary buffers

// ------------------------------------------------------------------ dequantisation ---------
// One warp per row: lane l turns codes 16 l .. + 15 into fp16, lanes 0-7 copy the rotary values. Rows past a
// request's length (its last tile) and rows of a bad page are zeros. HBM-bound: 656 bytes read, 1,152 written; 64
// requests of 30,000 rows, 3.47 GB, take 577 us, 6,010 GB/s.
constexpr int kExpandThreads = 512;
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const Params p, uint16_t* out) {
  let_next();
  __shared__ int64_t pre[kMaxReq + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    int64_t run = 0, cached = 0;
    if (lane == 0) pre[0] = 0;
    for (int at = 0; at < p.B; at += 32) {
      Req q = {0, 0, 0, 0};
      if (at + lane < p.B) q = load_req<kHalf>(p, at + lane);
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
    const int seq = load_req<kHalf>(p, lo).seq;
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
        range_ok &= s[k] == 0.f || (fabsf(s[k]) >= kScaleMin && fabsf(s[k]) <= kScaleMax);
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
// A position in a ring of barriers: its slot, and the parity to wait for.
struct Ring {
  int slot;
  uint32_t par;
  __device__ __forceinline__ void next(int slots) {
    if (++slot >= slots) {
      slot -= slots;
      par ^= 1u;
    }
  }
};

// Barriers and small arrays of a CTA.
struct Bars {
  uint64_t full[kMaxSlots];       // this CTA's part of a stage is there; in the issuing CTA the other's too
  uint64_t empty[kMaxSlots];      // the MMAs have read the stage (both CTAs)
  uint64_t codes_full[6];         // raw: a latent group's codes have landed
  uint64_t scale_full[2];         // raw: a tile's scales have landed
  uint64_t codes_empty[6];        // raw: the producers have read them
  uint64_t split_full[2];         // raw: a tile's scales are split -> producers
  uint64_t split_empty[2];        // raw: both groups of producers are done with them
  uint64_t s_full[2];             // S complete (both)
  uint64_t s_empty[2];            // issuing softmax CTA: all softmax warps have read S
  uint64_t p_empty[2];            // softmax CTA: its P buffer and staging are free (a phase per tile of a block in which it has rows)
  uint64_t p_full[2];             // output CTA: P and the factors have landed
  uint64_t corr[2];               // issuing output CTA: O is rescaled for this P (both)
  uint64_t pv_done[2];            // PV complete (both)
  uint64_t q_ready;               // issuing softmax CTA: Q is in place (both)
  uint64_t q_free;                // the block's QK MMAs have read Q (both)
  uint64_t o_free;                // issuing output CTA: O is read out (both)
  uint64_t out_done[2];           // output CTA: a block's output has left the P buffer of its last tile
  uint64_t drain[2];
  uint64_t swap[4];               // softmax CTA: the two warps of a lane quarter have written their values
};
static_assert(sizeof(Bars) <= 8 * kNumBars, "barriers");
struct Misc {
  uint32_t tmem;
  volatile uint32_t abort;
  Start start;
  volatile int32_t seen[2];       // stages that each of the two issuing warps has found there
  int32_t left[2];                // raw: cached rows from the tile's first key on
  volatile int32_t todo;          // output CTA: what the output warps are woken for (kRescale, kLast, kStop)
  int32_t tile;                   // and for which tile
  volatile int32_t stop[2];       // raw: a group of producers' first warp gave up
};
static_assert(sizeof(Misc) <= 128, "misc");
constexpr int kRescale = 1, kLast = 2, kStop = 4;
// Named barriers. Warps that need not look at a tile (the output warps while no maximum moves) or that work in step (the
// producers) sleep in these while one warp polls: every arrival on any barrier of a CTA wakes its polling warps.
constexpr int kWake = 1, kWoken = 2, kGo = 3, kDone = 5;  // kGo, kDone: and the next one for the second group
__device__ __forceinline__ void named_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Asks for the queries of a block's rows in this CTA into L2, some tiles before they are read.
__device__ __forceinline__ void prefetch_q(const Params& p, const Seg& s, int half) {
  const int have = s.nrows - half * kHalf;
  if (have > 0)
    bulk_prefetch_l2(p.q + ((int64_t)s.q.start * p.H + (int64_t)s.b * (kHalf * G) + half * kHalf) * (HS_D_QK * 2),
                     (have < kHalf ? have : kHalf) * (HS_D_QK * 2));
}

// raw: one thread brings a tile's undecoded rows: the scales, in the softmax CTA the rotary block, and latent group by
// latent group the codes. A page that the table does not name, or that lies outside the pool, is read past the pool's
// end: zeros.
template <bool isA>
__device__ __forceinline__ void load_raw(const Params& p, uint8_t* smem, Bars& br, Misc& mc, const CUtensorMap* codes,
                                         const CUtensorMap* scales, const CUtensorMap* rotary, Walk<kHalf * G>& walk, int half) {
  using Sh = Shape<true>;
  constexpr int kSlots = isA ? Sh::kSlotsA : Sh::kSlotsB, kCodes = isA ? Sh::kCodesA : Sh::kCodesB;
  constexpr int kPages = isA ? 1 : 2, kGroups = isA ? 4 : 4 / G;
  uint8_t* cring = smem + (isA ? Sh::kOffCodesA : Sh::kOffCodesB);
  uint8_t* sring = smem + (isA ? Sh::kOffScaleA : Sh::kOffScaleB);
  prefetch_tensormap(codes);
  prefetch_tensormap(scales);
  Ring ring = {0, 1};
  int64_t issued = 0;
  int tile = 0, rotaries = 0;
  bool ok = true;
  Seg s;
  // block-table entries of the next tile, read one tile ahead
  int jn = 0;
  bool more = walk.next(p, s);
  if (more) jn = s.ta;
  int32_t blk[2] = {0, 0};
  int left = 0;  // cached rows from this CTA's first key of the tile on
  bool live = false;
  auto fetch = [&]() {
    live = more;
    if (!more) return;
    left = s.q.seq - jn * kKeys - (isA ? half * HS_PAGE : 0);
#pragma unroll
    for (int h = 0; h < kPages; ++h) {
      const int page = 2 * jn + (isA ? half : h);
      blk[h] = page < p.bt_stride ? ldg_nc_s32(p.bt + (int64_t)s.r * p.bt_stride + page) : -1;
    }
    if (++jn == s.tb) {
      more = walk.next(p, s);
      if (more) jn = s.ta;
      if (more && isA) prefetch_q(p, s, half);
    }
  };
  fetch();
#pragma unroll 1
  for (; ok && live; ++tile) {
    const int t = tile & 1;
    const uint32_t ph = (uint32_t)(tile >> 1) & 1u;
    int32_t y[2];
    const int now = left;
#pragma unroll
    for (int h = 0; h < kPages; ++h) {
      const bool good = blk[h] >= 0 && ((int64_t)blk[h] + 1) * HS_PAGE <= p.R;
      if (!good && now > h * HS_PAGE) flag_error(p.err, HS_FLAG_BAD_BLOCK);
      y[h] = good ? blk[h] * HS_PAGE : (int32_t)p.R;
    }
    fetch();
    // the scales of the tile before the last are split
    ok = !mc.abort && (tile < 2 || mbar_wait(&br.split_full[t], ph ^ 1u, p.err));
    if (!ok) break;
    mc.left[t] = now;
    mbar_arrive_expect_tx(&br.scale_full[t], kCodes / 8);
#pragma unroll
    for (int h = 0; h < kPages; ++h)
      tma_load_2d(sring + (t * kPages + h) * HS_PAGE * 16, scales, &br.scale_full[t], HS_D_LATENT, y[h]);
#pragma unroll 1
    for (int k = 0; k < kGroups; ++k) {
      if (mc.abort || !mbar_wait(&br.codes_empty[ring.slot], ring.par, p.err)) {
        ok = false;
        break;
      }
      uint64_t* bar = &br.codes_full[ring.slot];
      const int g = isA ? k : 2 * k + half;
      mbar_arrive_expect_tx(bar, kCodes);
#pragma unroll
      for (int h = 0; h < kPages; ++h) tma_load_2d(cring + ring.slot * kCodes + h * HS_PAGE * 128, codes, bar, 128 * g, y[h]);
      ++issued;
      ring.next(kSlots);
    }
    if (isA && ok) {
      ok = mbar_wait(&br.empty[kRotaryBar + t], ph ^ 1u, p.err);
      if (ok) {
        mbar_arrive_expect_tx(&br.full[kRotaryBar + t], Sh::kKBlk);
        tma_load_2d(smem + Sh::kOffRotary + t * Sh::kKBlk, rotary, &br.full[kRotaryBar + t], (HS_D_LATENT + 16) / 2, y[0]);
        ++rotaries;
      }
    }
  }
  if (!ok) mc.abort = 1;
  // every copy has landed before the CTA may leave: slots before the position were used in its round
  for (int q = 0; q < kSlots; ++q)
    if (q < issued) mbar_wait(&br.codes_full[q], q < ring.slot ? ring.par ^ 1u : ring.par, p.err);
  for (int u = tile > 2 ? tile - 2 : 0; u < tile; ++u) mbar_wait(&br.scale_full[u & 1], (uint32_t)(u >> 1) & 1u, p.err);
  // (full also counts the other CTA's word, which an abort may leave out: the wait's limit then gives the copy its time)
  for (int u = rotaries > 2 ? rotaries - 2 : 0; u < rotaries; ++u)
    mbar_wait(&br.full[kRotaryBar + (u & 1)], (uint32_t)(u >> 1) & 1u, p.err);
}

// raw: one warp splits every scale of a tile into two fp16 parts (see dequant8), each twice in a 32-bit word, for the
// producers; rows past the request's length get scale 0.
template <bool isA>
__device__ __forceinline__ void split_scales(const Params& p, uint8_t* smem, Bars& br, Misc& mc, int ntiles, int lane) {
  using Sh = Shape<true>;
  constexpr int kKeysHere = isA ? Sh::kMine : kKeys;
  const float4* in = reinterpret_cast<const float4*>(smem + (isA ? Sh::kOffScaleA : Sh::kOffScaleB));
  uint2* out = reinterpret_cast<uint2*>(smem + (isA ? Sh::kOffSplitA : Sh::kOffSplitB));
  bool range_ok = true;
#pragma unroll 1
  for (int i = 0; i < ntiles; ++i) {
    const int t = (int)(i & 1);
    const uint32_t ph = (uint32_t)(i >> 1) & 1u;
    const bool ok = !mc.abort && mbar_wait(&br.scale_full[t], ph, p.err) && mbar_wait(&br.split_empty[t], ph ^ 1u, p.err);
    if (!__all_sync(0xffffffffu, ok)) {
      mc.abort = 1;
      break;
    }
    const int left = mc.left[t];
#pragma unroll
    for (int j = 0; j < kKeysHere / 32; ++j) {
      const int row = lane + 32 * j;
      const float4 f = in[t * kKeysHere + row];
      const float sc[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float v = row < left ? sc[g] : 0.f;
        range_ok &= v == 0.f || (fabsf(v) >= kScaleMin && fabsf(v) <= kScaleMax);
        const __half hi = __float2half_rn(v);
        const __half2 h2 = __half2half2(hi), l2 = __float2half2_rn(v - __half2float(hi));
        out[(t * 4 + g) * kKeysHere + row] = make_uint2(*reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&l2));
      }
    }
    fence_proxy_async_smem();  // the scales' reads come before the next copy over them
    __syncwarp();
    if (lane == 0) mbar_arrive(&br.split_full[t]);
  }
  if (isA && !range_ok) flag_error(p.err, HS_FLAG_RANGE);
}

// raw: the producers turn a latent group's codes into fp16 blocks of the K or V ring. Two groups of warps take turns,
// so that one converts while the other waits and hands over (the rings' slots are even in number: a slot is always the
// same group's). Warp w of a group works on the quads of rows w, w + kProd, ...: lane l reads the codes 16 (l % 8) .. + 15 of row
// l / 8 of a quad as two 8-byte pieces, which become the 16-byte pieces 2 (l % 4) and + 1 of a row of block (l % 8) / 4.
// Which of the two a lane takes first alternates with l / 4 and with the row, so that the reads and the stores of a warp hit
// different banks. Bound by issue slots: about 40 instructions per 512 codes, most of them (cvt, half2 arithmetic) at half
// rate.
template <bool isA>
__device__ __forceinline__ void produce(uint8_t* smem, Bars& br, Misc& mc, int32_t* err, int ntiles, int half, int pw, int lane) {
  using Sh = Shape<true>;
  constexpr int kBlk = isA ? Sh::kKBlk : kVBlk, kStage = 2 * kBlk;
  constexpr int kSlots = isA ? Sh::kStA : Sh::kStB;
  constexpr int kCodes = isA ? Sh::kCodesA : Sh::kCodesB, kCodeSlots = isA ? Sh::kSlotsA : Sh::kSlotsB;
  constexpr int kKeysHere = isA ? Sh::kMine : kKeys;
  constexpr int kProd = isA ? 4 : 3, kBatch = isA ? 2 : 3;
  constexpr int kQuads = kKeysHere / 4, kPass = (kQuads + kProd - 1) / kProd;
  constexpr int kGroups = isA ? 4 : 4 / G;
  static_assert(kSlots % 2 == 0 && kCodeSlots % 2 == 0 && kGroups % 2 == 0, "a slot belongs to one group");
  const int e = pw / kProd, w = pw % kProd;
  const int rl = lane >> 3, c8 = lane & 7;
  const uint32_t odd = (uint32_t)((c8 >> 2) ^ (rl & 1));  // the piece taken first
  const uint8_t* codes = smem + (isA ? Sh::kOffCodesA : Sh::kOffCodesB) + rl * 128 + 16 * c8;
  const uint2* split = reinterpret_cast<const uint2*>(smem + (isA ? Sh::kOffSplitA : Sh::kOffSplitB)) + rl;
  uint8_t* out = smem + (isA ? kOffK : kOffV) + (c8 >> 2) * kBlk;
  const uint32_t o0 = 32 * (c8 & 3) + 16 * odd;
  Ring ring = {e, 1}, cr = {e, 0};
  const bool first = w == 0;
  bool go = true;
  // the group's first warp waits for what a stage needs
  auto take = [&](uint64_t* bar, uint32_t par) { go = go && __all_sync(0xffffffffu, !mc.abort && mbar_wait(bar, par, err)); };
#pragma unroll 1
  for (int i = 0; i < ntiles && go; ++i) {
    const int t = (int)(i & 1);
#pragma unroll 1
    for (int k = e; k < kGroups; k += 2) {
      if (first) {
        if (k == e) take(&br.split_full[t], (uint32_t)(i >> 1) & 1u);
        take(&br.codes_full[cr.slot], cr.par);
        take(&br.empty[ring.slot], ring.par);
        if (!go) mc.stop[e] = 1;
        __syncwarp();
      }
      named_bar(kGo + e, 32 * kProd);
      go = mc.stop[e] == 0;  // the same for every warp of the group
      if (!go) break;
      const int g = isA ? k : 2 * k + half;
      uint8_t* blk = out + ring.slot * kStage;
#pragma unroll
      for (int p0 = 0; p0 < kPass; p0 += kBatch) {  // a few quads at a time
        uint2 va[kBatch], vb[kBatch], sc[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int q = w + kProd * (p0 + j);
          if (q < kQuads) {
            const uint8_t* c = codes + cr.slot * kCodes + q * 512;
            va[j] = *reinterpret_cast<const uint2*>(c + 8 * odd);
            vb[j] = *reinterpret_cast<const uint2*>(c + 8 * (odd ^ 1u));
            sc[j] = split[(t * 4 + g) * kKeysHere + 4 * q];
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int q = w + kProd * (p0 + j);
          if (q < kQuads) {
            uint4 d0 = dequant8(va[j].x, va[j].y, sc[j].x, sc[j].y);
            uint4 d1 = dequant8(vb[j].x, vb[j].y, sc[j].x, sc[j].y);
            if (!isA && unsound(d0, d1)) d0 = d1 = make_uint4(0, 0, 0, 0);
            const uint32_t at = sw128_offset(4 * q + rl, o0);
            *reinterpret_cast<uint4*>(blk + at) = d0;
            *reinterpret_cast<uint4*>(blk + (at ^ 16u)) = d1;
          }
        }
      }
      fence_proxy_async_smem();
      if (first) {
        named_bar(kDone + e, 32 * kProd);
        if (lane == 0) {
          mbar_arrive(&br.full[ring.slot]);
          mbar_arrive(&br.codes_empty[cr.slot]);
          if (k + 2 >= kGroups) mbar_arrive(&br.split_empty[t]);
        }
      } else {
        named_arrive(kDone + e, 32 * kProd);
      }
      ring.next(kSlots);
      ring.next(kSlots);
      cr.next(kCodeSlots);
      cr.next(kCodeSlots);
    }
  }
  if (!go) mc.abort = 1;
}

template <bool kRaw>
__global__ void __cluster_dims__(2 * G, 1, 1) __launch_bounds__(Shape<kRaw>::kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_r, const Params p) {
  // map_k, map_v: K and V blocks of the copy, or raw: codes and scales; map_r: raw: rotary blocks
  using Sh = Shape<kRaw>;
  constexpr int kRows = Sh::kRows, kKBlk = Sh::kKBlk, kKStage = Sh::kKStage, kStA = Sh::kStA, kStB = Sh::kStB;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in every CTA
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  Bars& br = *reinterpret_cast<Bars*>(smem + kOffBar);
  Misc& mc = *reinterpret_cast<Misc*>(smem + kOffMisc);
  uint64_t *full = br.full, *empty = br.empty, *s_full = br.s_full, *s_empty = br.s_empty, *p_empty = br.p_empty, *p_full = br.p_full,
           *corr = br.corr, *pv_done = br.pv_done, *q_ready = &br.q_ready, *q_free = &br.q_free, *o_free = &br.o_free, *drain = br.drain,
           *swap = br.swap;
  volatile uint32_t* abort_flag = &mc.abort;
  Start* st = &mc.start;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  let_next();
  if (!kRaw) after_previous();
  const uint32_t rank = cluster_ctarank();
  const bool isA = rank < G, lead = rank % G == 0;
  const int half = (int)rank % G;  // which rows of a block, and which part of every K and V tile
  const uint16_t pair_mask = isA ? 0x3 : 0xC;
  const int c = blockIdx.x / (2 * G);

  if (tid == 0) {
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(&full[s], lead ? 2 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 6; ++s) {
      mbar_init(&br.codes_full[s], 1);
      mbar_init(&br.codes_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&br.scale_full[s], 1);
      mbar_init(&br.split_full[s], 1);
      mbar_init(&br.split_empty[s], 2);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 8 * G);
      mbar_init(&p_empty[s], 1);
      mbar_init(&p_full[s], 1);
      mbar_init(&corr[s], G);
      mbar_init(&pv_done[s], 1);
      mbar_init(&br.out_done[s], 8);
    }
    mbar_init(q_ready, 8 * G);
    mbar_init(q_free, 2);
    mbar_init(o_free, 8 * G);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    for (int q = 0; q < 4; ++q) mbar_init(&swap[q], 2);
    mbar_fence_init();
    mc.abort = 0;
    mc.stop[0] = mc.stop[1] = 0;
    mc.seen[0] = mc.seen[1] = 0;
  }
  find_units<kRows>(p, (int64_t*)(smem + kOffScratch), st, c, Sh::kThreads);
  fence_proxy_async_all();
  __syncthreads();
  cluster_sync();  // every CTA's barriers exist
  if (warp == 0) tc2::alloc(&mc.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mc.tmem;
  const int64_t U = st->U;
  const int ntiles = st->ntiles;
  // raw: 640 threads start with 96 registers each (61,440 in all); the softmax and output warps (256 threads) take 120, the
  // others (384) keep 80: 61,440
  const bool rows_warp = warp >= kSmWarp0 && warp < kSmWarp0 + 8;
  Walk<kRows> walk(p, *st);
  Seg s;

  if (rows_warp && isA) {
    if (kRaw) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ================================================================ softmax ===================
    const int quad = warp & 3, g = (warp - 4) >> 2, row = 32 * quad + lane;  // g: columns 64 g .. + 63
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const uint32_t to = rank + G;
    const uint32_t r_p = remote_smem(smem + kOffP, to), r_alpha = remote_smem(smem + kOffAlpha, to), r_sum = remote_smem(smem + kOffSum, to);
    const uint32_t r_full = remote_smem(p_full, to), r_sempty = remote_smem(s_empty, 0), r_qready = remote_smem(q_ready, 0);
    float* smax = (float*)(smem + kOffMax);  // [2][2][128]
    float* salpha = (float*)(smem + kOffAlpha);
    float* ssum = (float*)(smem + kOffSum);
    int n = 0, i = 0, x = 0;  // x: exchanges through smax, alternating halves
    uint32_t skipped = 0;     // bit b: whether the tiles in buffer b that had no phase of p_empty[b] are odd in number
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
      const int64_t grow = (int64_t)s.b * kRows + (int64_t)half * kHalf + row;  // of the request's rows
      const int have = s.nrows - half * kHalf;                            // rows of this CTA that exist
      const bool idle = 32 * quad >= have, mine = row < have;
      float coef = p.scale_log2;
      if (n > 0) ok = warp_wait_all(q_free, (uint32_t)(n - 1) & 1u, p.err);
      if (ok && !idle) {
        // Q's rows 32 quad .. + 31 of this CTA: latent dims 256 g .. + 255 to fp16 in tensor memory, rotary dims 32 g .. + 31 to
        // shared memory. 32 dims at a time: coalesced loads (lane l takes 16 bytes of rows l / 4 + 8 j), through 2 KB of the
        // rotary block's place (64-byte swizzle) to the thread that owns the row. Rows past the block's are read as its
        // first row.
        const uint8_t* base = p.q + ((int64_t)s.q.start * p.H + (int64_t)s.b * kRows) * (HS_D_QK * 2);
        const int64_t myrow = mine ? (int64_t)half * kHalf + row : 0;
        uint8_t* scratch = smem + kOffQ + 4096 * quad + 2048 * g;
        const uint8_t* src[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 32 * quad + 8 * j + (lane >> 2);
          src[j] = base + (r < have ? (int64_t)half * kHalf + r : 0) * (HS_D_QK * 2) + 512 * g + 16 * (lane & 3);
        }
        uint32_t mx = 0u;
#pragma unroll 1
        for (int c0 = 0; c0 < 8; c0 += 2) {
          uint4 x[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[u][j] = ldg_nc_v4(src[j] + 64 * (c0 + u));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            __syncwarp();  // the piece before has been read
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(scratch + sw64_offset(8 * j + (lane >> 2), 16 * (lane & 3))) = x[u][j];
            __syncwarp();
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint4 v = *reinterpret_cast<const uint4*>(scratch + sw64_offset(lane, 16 * h));
              w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              mx = __vmaxu2(mx, w[k] & 0x7FFF7FFFu);
              const uint32_t f = w[k] ^ p.flip;
              w[k] = pack_half2(__uint_as_float(f << 16), __uint_as_float(f & 0xFFFF0000u));
            }
            tmem_st16(tmem + lane_base + 256 + 128 * g + 16 * (c0 + u), w);
          }
        }
        // A row whose largest latent value is outside [2^-6, 2^15) is scaled by a power of two that puts it in
        // [2^14, 2^15); its logits are scaled back.
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
        const uint8_t* own = base + myrow * (HS_D_QK * 2);
        if (__any_sync(0xffffffffu, e > 0)) {  // rare: the rotary values go along
          uint32_t m = 0u;
#pragma unroll 1
          for (int h = 0; h < 8; ++h) {
            const uint4 v = ldg_nc_v4(own + 1024 + 16 * h);
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
          }
          e = query_exponent(e, max(m & 0xFFFFu, m >> 16));
        }
        const float f = __uint_as_float((uint32_t)(e + 127) << 23);
        // not 0, so that a masked column stays -inf (softmax scales next to 0, or rows that are tiny in both parts: their logits
        // stay below 2^-60 and do not show)
        coef = fmaxf(coef * __uint_as_float((uint32_t)(127 - e) << 23), 7.5e-37f);
        if (__any_sync(0xffffffffu, e != 0)) {  // rare: again, each thread its row
#pragma unroll 1
          for (int b = 0; b < 8; ++b) {
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint4 v = ldg_nc_v4(own + 512 * g + 64 * b + 16 * h);
              w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint32_t q = w[k] ^ p.flip;
              w[k] = pack_half2(__uint_as_float(q << 16) * f, __uint_as_float(q & 0xFFFF0000u) * f);
            }
            tmem_st16(tmem + lane_base + 256 + 128 * g + 16 * b, w);
          }
        }
        tmem_wait_st();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint4 v = ldg_nc_v4(own + 1024 + 64 * g + 16 * h);
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

      const int nsee = mine ? sees<kRows>(p, s.q, grow) : 0;
      float ref = -INFINITY, l = 0.f;
      const int32_t* bt = p.bt + (int64_t)s.r * p.bt_stride;
      int32_t next_k = ldg_nc_s32(bt + (2 * s.ta + g < p.bt_stride ? 2 * s.ta + g : 0));
#pragma unroll 1
      for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
        const int b = i & 1;
        const uint32_t ph = (uint32_t)(i >> 1) & 1u;
        const int page = 2 * jt + g;  // this warp's page of the tile, read a tile ahead
        const int32_t k = next_k;
        next_k = ldg_nc_s32(bt + (page + 2 < p.bt_stride ? page + 2 : 0));
        ok = !*abort_flag && warp_wait_all(&s_full[b], ph, p.err);
        if (!ok) break;
        tc_fence_after();
        if (idle) {
          __syncwarp();
          if (lane == 0) remote_arrive_relaxed(r_sempty + 8 * (uint32_t)b);
          // Where this CTA has rows, its other warps wait for p_empty's phase, and all of them before the next block's first S;
          // where it has none, there is no phase that a later wait could take for its own.
          if (have <= 0) skipped ^= 1u << b;
          continue;
        }
        const bool there = page < p.bt_stride && k >= 0 && ((int64_t)k + 1) * HS_PAGE <= p.R;
        const int lim = there ? nsee - jt * kKeys - 64 * g : 0;  // columns that this thread's row sees
        const bool all = __all_sync(0xffffffffu, lim >= 64);
        const uint32_t at = tmem + lane_base + kKeys * b + 64 * g;
        // 32 columns, masked ones -inf
        auto columns = [&](int h, uint32_t (&x)[32]) {
          tmem_ld32(at + 32 * h, x);
          tmem_wait_ld();
          if (!all) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 32 * h + j < lim ? x[j] : 0xFF800000u;
          }
        };
        auto taken = [&]() {  // S has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive_relaxed(r_sempty + 8 * (uint32_t)b);
        };
        auto top = [&](const uint32_t (&x)[32]) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 2) m0 = fmaxf(m0, __uint_as_float(x[j])), m1 = fmaxf(m1, __uint_as_float(x[j + 1]));
          return fmaxf(m0, m1);
        };
        uint32_t v0[32], v1[32];
        columns(0, v0);
        float mx = top(v0);
        columns(1, v1);
        taken();
        mx = fmaxf(mx, top(v1));
        mx = fmaxf(mx, other(mx));
        if (!ok) break;
        mx = mx == -INFINITY ? mx : mx * coef;
        const bool up = mx > ref + kThreshold;
        const float to_ref = up ? mx : ref;
        const float al = up ? fast_exp2(ref - to_ref) : 1.f;
        l *= al;
        ref = to_ref;
        const float me = ref == -INFINITY ? 0.f : ref - kLift;
        ok = warp_wait_all(&p_empty[b], ph ^ ((skipped >> b) & 1u), p.err);
        if (!ok) break;
        uint8_t* blk = smem + kOffStage + b * kPBuf + g * (kPBuf / 2);
        // P of 32 columns; masked columns are -inf and coef > 0: their P is 0
        auto weights = [&](int h, uint32_t (&x)[32]) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float a = fast_exp2(fmaf(__uint_as_float(x[2 * j]), coef, -me));
            const float c2 = fast_exp2(fmaf(__uint_as_float(x[2 * j + 1]), coef, -me));
            s0 += a;
            s1 += c2;
            x[j] = pack_half2(a, c2);
          }
          l += s0 + s1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(blk + sw128_offset(row, 64 * h + 16 * j)) =
                make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        };
        weights(0, v0);
        weights(1, v1);
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
              p.part_lse[(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + half * kHalf + row] = z;
            }
          }
        }
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
  } else if (rows_warp) {
    if (kRaw) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ================================================================ rescaling, output =========
    const int quad = warp & 3, g = (warp - 4) >> 2, row = 32 * quad + lane;  // g: O's columns 256 g .. + 255
    const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + 256 * g;
    const uint32_t r_ofree = remote_smem(o_free, G);
    const float* alpha = (const float*)(smem + kOffAlpha);
    const float* sums = (const float*)(smem + kOffSum);
    const int64_t C = U < p.clusters ? U : p.clusters;
    Desc desc = {0, 0, 0, 0};
    int64_t cost = st->cost;  // of the blocks before this one
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p, s)) {
      const int have = s.nrows - half * kHalf;
      const bool idle = 32 * quad >= have;
      const int64_t row0 = (int64_t)s.q.start * p.H + (int64_t)s.b * kRows;
      if (s.ta == 0 && s.tb < s.tiles) {
        desc.row0 = (int32_t)row0;
        desc.nrows = s.nrows;
        desc.nparts = (int32_t)(unit_cta(cost + s.tiles + kBlockCost - 1, U, C) - c + 1);
      }
      if (s.tb == s.tiles) cost += s.tiles + kBlockCost;
      float sum = 0.f;
      int todo, i;
#pragma unroll 1
      do {
        named_bar(kWake, 288);
        todo = mc.todo;
        i = mc.tile;
        if ((todo & kLast) && !idle) sum = sums[128 * (i & 1) + row];
        if ((todo & kRescale) && !idle) {
          const float al = alpha[128 * (i & 1) + row];
          tc_fence_after();
          if (__any_sync(0xffffffffu, al != 1.f)) {
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
          }
          tc_fence_before();
        }
        named_bar(kWoken, 288);
      } while (!(todo & (kLast | kStop)));
      ok = !(todo & kStop) && warp_wait_all(&pv_done[i & 1], (uint32_t)(i >> 1) & 1u, p.err);
      if (!ok) {
        *abort_flag = 1;
        if (todo & kStop) break;
        ok = true;  // the controlling warp sees the flag and stops everyone at the next tile
        continue;
      }
      tc_fence_after();
      if (!idle) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const bool whole = s.ta == 0 && s.tb == s.tiles;
        // 128 bytes of each of the warp's rows at a time, through 4 KB of the last tile's P buffer (PV has read it), so that a
        // store covers whole lines of four rows
        uint8_t* scratch = smem + kOffP + (i & 1) * kPBuf + 4096 * (4 * g + quad);
        const int pl = lane & 7, rl = lane >> 3;
        auto rows_out = [&](uint8_t* to, int64_t pitch) {  // scratch to rows 32 quad + 4 j + rl of this CTA
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r4 = 4 * j + rl;
            const uint4 v = *reinterpret_cast<const uint4*>(scratch + sw128_offset(r4, 16 * pl));
            if (32 * quad + r4 < have) *reinterpret_cast<uint4*>(to + (32 * quad + r4) * pitch + 16 * pl) = v;
          }
          __syncwarp();
        };
        const int64_t r = (int64_t)half * kHalf;
        uint8_t* o = reinterpret_cast<uint8_t*>(p.out + (row0 + r) * HS_D_LATENT + 256 * g);
        uint8_t* po = reinterpret_cast<uint8_t*>(p.part_out + ((int64_t)(2 * c + (s.ta == 0 ? 1 : 0)) * kRows + r) * HS_D_LATENT + 256 * g);
#pragma unroll 1
        for (int h = 0; h < 8; ++h) {  // 32 columns
          uint32_t v[32];
          tmem_ld32(at + 32 * h, v);
          tmem_wait_ld();
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
              *reinterpret_cast<uint4*>(scratch + sw128_offset(lane, 64 * (h & 1) + 16 * k)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (h & 1) rows_out(o + 64 * (h - 1), HS_D_LATENT * 2);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(scratch + sw128_offset(lane, 16 * k)) =
                  make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                              __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
            rows_out(po + 128 * h, HS_D_LATENT * 4);
          }
        }
      }
      fence_proxy_async_smem();  // the buffer's reads come before the next P's copy into it
      __syncwarp();
      if (lane == 0) mbar_arrive(&br.out_done[i & 1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive_relaxed(r_ofree);
    }
    if (!ok) *abort_flag = 1;
    if (rank == G && warp == 4 && lane == 0) p.desc[c] = desc;
  } else {
    if (kRaw) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kLoadWarp) {
      // ================================================================ loads =====================
      if (kRaw && lane == 0) {
        if (isA)
          load_raw<true>(p, smem, br, mc, &map_k, &map_v, &map_r, walk, half);
        else
          load_raw<false>(p, smem, br, mc, &map_k, &map_v, &map_r, walk, half);
      } else if (lane == 0) {
        const CUtensorMap* map = isA ? &map_k : &map_v;
        prefetch_tensormap(map);
        const int slots = isA ? kStA : kStB;
        Ring ring = {0, 1};
        int64_t issued = 0;
        bool ok = true;
#pragma unroll 1
        while (ok && walk.next(p, s)) {
          if (isA) prefetch_q(p, s, half);
#pragma unroll 1
          for (int jt = s.ta; jt < s.tb && ok; ++jt) {
            const int32_t y = (int32_t)(s.base + (int64_t)jt * kKeys);
#pragma unroll 1
            for (int k = 0; k < (isA ? Sh::kStages : Sh::kVStages); ++k) {
              uint64_t* bar = &full[ring.slot];
              if (*abort_flag || !mbar_wait(&empty[ring.slot], ring.par, p.err)) {
                ok = false;
                break;
              }
              if (isA) {  // dim blocks 3 k .. + 2, this CTA's keys
                uint8_t* d = smem + kOffK + ring.slot * kKStage;
                mbar_arrive_expect_tx(bar, kKStage);
#pragma unroll
                for (int b = 0; b < 3; ++b) tma_load_2d(d + b * kKBlk, map, bar, 64 * (3 * k + b), y + Sh::kMine * half);
              } else {    // dims 128 (G k + half) .. + 127, all keys
                uint8_t* d = smem + kOffV + ring.slot * kVStage;
                mbar_arrive_expect_tx(bar, kVStage);
                tma_load_2d(d, map, bar, 128 * (G * k + half), y);
                tma_load_2d(d + kVBlk, map, bar, 128 * (G * k + half) + 64, y);
              }
              ++issued;
              ring.next(slots);
            }
          }
        }
        if (!ok) *abort_flag = 1;
        // every copy has landed before the CTA may leave: slots before the position were used in its round
        for (int q = 0; q < slots; ++q)
          if (q < issued) mbar_wait(&full[q], q < ring.slot ? ring.par ^ 1u : ring.par, p.err);
      }
    } else if (lead && (warp == kIssue0 || (warp == kIssue1 && isA))) {
      // ================================================================ MMAs ======================
      // The raw variant's loops over stages and steps are not unrolled: its roles' code shares the instruction caches, and 28 MMAs
      // less of it make the whole kernel 19 % faster (64 requests x 4 tokens 1,350 -> 1,097 us). The copy variant, with fewer
      // roles, is 20 % slower without unrolling (chunk 5.95 -> 7.2 ms).
      if (lane == 0) {
        const int mine = warp == kIssue0 ? 0 : 1;  // QK: the parity of the tiles that this warp issues
        const int slots = isA ? kStA : kStB;
        int slot = 0, i = 0, n = 0;
        uint32_t par = 0;
        int32_t stages = 0;  // stages of the ring before this one
        bool ok = true;
        // The next stage is there (the other CTA's part too). A parity tells two phases apart, so a warp that did not see
        // the slot's last use (the other warp's tile) makes sure that the other warp has.
        auto stage = [&]() -> bool {
          bool r = true;
          const int32_t last = stages - slots;  // the slot's last use
          if (isA && last >= 0 && ((last / Sh::kStages) & 1) != mine) {
            const uint64_t t0 = globaltimer();
            for (uint32_t it = 0; mc.seen[mine ^ 1] <= last; ++it)
              if ((it & 63) == 63 && (*abort_flag || globaltimer() - t0 > kWaitLimitNs)) {
                flag_error(p.err, HS_FLAG_TIMEOUT);
                r = false;
                break;
              }
          }
          r = r && mbar_wait(&full[slot], par, p.err);
          if (isA) mc.seen[mine] = stages + 1;
          tc_fence_after();
          return r;
        };
        auto skip = [&](int k) {
          stages += k;
          for (slot += k; slot >= slots; slot -= slots) par ^= 1u;
        };
        auto pass = [&]() {
          tc2::commit(&empty[slot], pair_mask);
          skip(1);
        };
        if (isA) {
          constexpr uint32_t lat = idesc_f16(kRows, kKeys, 0, 0), rop = idesc_bf16(kRows, kKeys, 0, 0);
          const uint64_t qd = smem_desc(smem_u32(smem + kOffQ), 16, 1024, 2);
          const uint64_t kd = smem_desc(smem_u32(smem + kOffK), 16, 1024, 2);
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
                skip(Sh::kStages);
                continue;
              }
              const uint32_t d = tmem + kKeys * mine;
              if (*abort_flag || !mbar_wait(&s_empty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err)) {
                ok = false;
                break;
              }
#pragma unroll (kRaw ? 1 : Sh::kStages)
              for (int k = 0; k < Sh::kStages; ++k) {
                if (!stage()) {
                  ok = false;
                  break;
                }
                const uint64_t kb = kd + (uint64_t)((slot * kKStage) >> 4);
#pragma unroll
                for (int b = 0; b < Sh::kBlocks && Sh::kBlocks * k + b < 9; ++b)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t bd = kb + (uint64_t)((b * kKBlk + kk * 32) >> 4);
                    if (Sh::kBlocks * k + b < 8)
                      tc2::ts(d, tmem + 256 + 32 * (Sh::kBlocks * k + b) + 8 * kk, bd, lat, (k | b | kk) != 0 ? 1u : 0u);
                    else
                      tc2::ss(d, qd + (uint64_t)((kk * 32) >> 4), bd, rop, 1u);
                  }
                pass();
              }
              if (kRaw && ok) {
                const uint32_t rb = kRotaryBar + (uint32_t)mine;
                ok = mbar_wait(&full[rb], (uint32_t)(i >> 1) & 1u, p.err);
                tc_fence_after();
                if (!ok) break;
                const uint64_t rd = smem_desc(smem_u32(smem + Sh::kOffRotary + mine * kKBlk), 16, 1024, 2);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) tc2::ss(d, qd + (uint64_t)((kk * 32) >> 4), rd + (uint64_t)((kk * 32) >> 4), rop, 1u);
                tc2::commit(&empty[rb], pair_mask);
              }
              if (ok) tc2::commit(&s_full[i & 1], pair_mask);
            }
            if (ok) tc2::commit(q_free, pair_mask);
          }
        } else {
          constexpr uint32_t id = idesc_f16(kRows, 128 * G, 0, 1);
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
#pragma unroll (kRaw ? 1 : Sh::kVStages)
              for (int k = 0; k < Sh::kVStages; ++k) {
                if (!stage()) {
                  ok = false;
                  break;
                }
                const uint64_t vb = vd + (uint64_t)((slot * kVStage) >> 4);
#pragma unroll (kRaw ? 4 : kKeys / 16)
                for (int kk = 0; kk < kKeys / 16; ++kk)
                  tc2::ss(tmem + 128 * G * k, pb + (uint64_t)(((kk / 4) * (kPBuf / 2) + (kk % 4) * 32) >> 4),
                              vb + (uint64_t)((kk * 2048) >> 4), id, (jt > s.ta || kk > 0) ? 1u : 0u);
                pass();
              }
              if (ok) tc2::commit(&pv_done[i & 1], pair_mask);
            }
          }
        }
        if (!ok) *abort_flag = 1;
        uint64_t* done = &drain[mine];
        tc2::commit(done, (uint16_t)(1u << rank));
        mbar_wait(done, 0, p.err);
      }
    } else if (warp == kRelayWarp && !lead) {
      // ================================================================ the other half is there ===
      if (lane == 0) {
        const uint32_t to = remote_smem(full, rank - 1);
        const int slots = isA ? kStA : kStB;
        Ring ring = {0, 0};
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < ntiles && ok; ++i) {
#pragma unroll 1
          for (int k = 0; k < (isA ? Sh::kStages : Sh::kVStages) && ok; ++k) {
            ok = !*abort_flag && mbar_wait(&full[ring.slot], ring.par, p.err);
            if (ok) remote_arrive_cta(to + 8 * (uint32_t)ring.slot);
            ring.next(slots);
          }
          if (kRaw && isA && ok) {
            const uint32_t rb = kRotaryBar + (uint32_t)(i & 1);
            ok = mbar_wait(&full[rb], (uint32_t)(i >> 1) & 1u, p.err);
            if (ok) remote_arrive_cta(to + 8 * rb);
          }
        }
        if (!ok) *abort_flag = 1;
      }
    } else if (!isA && warp == (lead ? kRelayWarp : kIssue0)) {
      // ================================================================ output control ============
      // Waits for every tile's P; wakes the output warps where some row's maximum moved (once PV of the tile before has
      // completed) or the block ends, and lets PV go on.
      const uint32_t r_corr = remote_smem(corr, G);
      const float4* alpha = (const float4*)(smem + kOffAlpha);
      int i = 0;
      bool ok = true;
#pragma unroll 1
      while (ok && walk.next(p, s)) {
        const int have = s.nrows - half * kHalf;
#pragma unroll 1
        for (int jt = s.ta; jt < s.tb && ok; ++jt, ++i) {
          const int b = i & 1;
          ok = !*abort_flag && warp_wait_all(&p_full[b], (uint32_t)(i >> 1) & 1u, p.err);
          int todo = ok ? 0 : kStop;
          if (ok && jt > s.ta) {
            const float4 al = alpha[32 * b + lane];  // rows 4 lane .. + 3
            if (__any_sync(0xffffffffu, 32 * (lane >> 3) < have && (al.x != 1.f || al.y != 1.f || al.z != 1.f || al.w != 1.f))) {
              ok = warp_wait_all(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, p.err);
              todo = ok ? kRescale : kStop;
              tc_fence_after();
              tc_fence_before();
            }
          }
          if (jt == s.tb - 1 && ok) todo |= kLast;
          if (todo) {
            if (lane == 0) {
              mc.todo = todo;
              mc.tile = i;
            }
            __syncwarp();
            named_bar(kWake, 288);
            named_bar(kWoken, 288);
          }
          if (ok && lane == 0) remote_arrive_relaxed(r_corr + 8 * (uint32_t)b);
        }
      }
      if (!ok) *abort_flag = 1;
    } else if (warp == kBufWarp && !isA) {
      // ================================================================ P buffers =================
      // Arms a buffer's barrier with the bytes that its tile brings (4 KB of P and 128 bytes of factors per
      // 32 rows, at a block's last tile 128 bytes of sums), then hands it to the softmax CTA.
      if (lane == 0) {
        const uint32_t back = remote_smem(p_empty, rank - G);
        int i = 0;          // tiles
        uint32_t ends = 0;  // bit j: the tile j before this one ended a block
        // bit b: parity of the next block whose output passes through buffer b. A barrier per buffer: the next phase needs a tile
        // that is armed after this wait, so it cannot be over before the wait has seen the one before.
        uint32_t outs = 0;
        bool ok = true;
#pragma unroll 1
        while (ok && walk.next(p, s)) {
          const int left = s.nrows - half * kHalf;
          const uint32_t quads = left <= 0 ? 0 : left >= kHalf ? 4 : (uint32_t)(left + 31) / 32;
#pragma unroll 1
          for (int jt = s.ta; jt < s.tb; ++jt, ++i) {
            const int b = i & 1;
            if (i >= 2 && (*abort_flag || !mbar_wait(&pv_done[b], ((uint32_t)(i >> 1) & 1u) ^ 1u, p.err) ||
                           ((ends & 4u) && !mbar_wait(&br.out_done[b], (outs >> b) & 1u, p.err)))) {
              ok = false;
              break;
            }
            if (ends & 4u) outs ^= 1u << b;
            mbar_arrive_expect_tx(&p_full[b], quads * (8192u + 128u + (jt == s.tb - 1 ? 128u : 0u)));
            if (quads) remote_arrive_relaxed(back + 8 * (uint32_t)b);  // without rows nobody would see the phase
            ends = (ends | (jt == s.tb - 1 ? 1u : 0u)) << 1;
          }
        }
        if (!ok) *abort_flag = 1;
        // every P and factor that was sent has landed before the CTA may leave: an armed buffer is sent to once, and those before
        // the last two have been used (after an abort a part may never be sent: the wait's limit then gives the rest its time)
        for (int u = i > 2 ? i - 2 : 0; u < i; ++u) mbar_wait(&p_full[u & 1], (uint32_t)(u >> 1) & 1u, p.err);
      }
    } else if (kRaw && warp == (!isA ? kScaleWarpB : lead ? kRelayWarp : kIssue0)) {
      // ================================================================ scales ====================
      if (isA)
        split_scales<true>(p, smem, br, mc, ntiles, lane);
      else
        split_scales<false>(p, smem, br, mc, ntiles, lane);
    } else if (kRaw && producer_index(warp, isA) >= 0) {
      // ================================================================ producers =================
      if (isA)
        produce<true>(smem, br, mc, p.err, ntiles, half, producer_index(warp, isA), lane);
      else
        produce<false>(smem, br, mc, p.err, ntiles, half, producer_index(warp, isA), lane);
    }
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may still write to it
  if (warp == 0) {
    tc_fence_after();
    tc2::dealloc(tmem, 512);
  }
}

}  // namespace paged

namespace paged {
// Rows of the dequantised copy: every request's last tile is whole.
static int64_t copy_capacity(int B, int64_t kv_tokens) { return kv_tokens + (int64_t)B * kKeys; }
static uint64_t part_bytes(int sms) {
  const uint64_t c = (uint64_t)(sms / (2 * G)), n = 2 * c * (kHalf * G) * (HS_D_LATENT + 1) * 4 + c * sizeof(Desc), f = few_bytes(sms);
  return ((n > f ? n : f) + 15) / 16 * 16;
}

// Whether T tokens of B requests with H heads have rows enough for a dequantised copy to pay: when its cost, a pass over the cached
// rows, is shared by more than three blocks of a request. Measured (raw / copy, us, 30,000 cached rows per request): 64
// requests x 256 rows 893 / 1,346; x 512 1,806 / 2,097; 32 x 768 1,365 / 1,447; 32 x 1,024 1,816 / 1,813; 16 x 2,048 1,806 / 1,687. With
// 2,000 cached rows: 8 x 512 58 / 67; x 1,024 62 / 60-68; x 2,048 107 / 110; x 4,096 181 / 174.
static bool copies(int T, int B, int H) { return (int64_t)T * H > 768ll * B; }
// Whether they have few enough for paged_few.cu: two of its blocks of 64 per request on average. Measured (us, this file's raw
// variant / paged_few.cu): 64 requests x 64 rows over 30,000 cached rows 860 / 380; x 128 rows 871 / 710; x 144 (three
// blocks) 883 / 1,042; 8 x 128 over 1,000 42 / 34; 64 x 128 over 200 46 / 29.
static bool few_rows(int T, int B, int H) { return (int64_t)T * H <= 128ll * B; }

template <bool kRaw>
static cudaError_t launch(const Params& p0, const uint16_t* rows, uint64_t n, int sms, cudaStream_t stream, const char** why) {
  using Sh = Shape<kRaw>;
  auto kernel = paged_kernel<kRaw>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // Clusters that run at once: the SMs of a GPC need not be a multiple of a cluster. Asked once per device.
  static std::atomic<int> asked[64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int C = dev < 64 ? asked[dev].load(std::memory_order_relaxed) : 0;
  if (C == 0) {
    C = sms / (2 * G);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * G * C);
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {2 * G, 1, 1};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int most = 0;
    if (cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) == cudaSuccess && most > 0 && most < C) C = most;
    if (dev < 64) asked[dev].store(C, std::memory_order_relaxed);
  }
  Params p = p0;
  p.clusters = C;
  CUtensorMap mk = {}, mv = {}, mr = {};
  if (kRaw) {
    if (!encode_2d(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.kv, HS_KV_ROW_BYTES, (uint64_t)p.R, HS_KV_ROW_BYTES, 128, HS_PAGE,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&mv, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.kv, HS_KV_ROW_BYTES, (uint64_t)p.R, HS_KV_ROW_BYTES, 16, HS_PAGE,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&mr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.kv, HS_KV_ROW_BYTES / 2, (uint64_t)p.R, HS_KV_ROW_BYTES, 64, HS_PAGE,
                   CU_TENSOR_MAP_SWIZZLE_128B)) {
      *why = "cuTensorMapEncodeTiled failed for the pool";
      return cudaErrorInvalidValue;
    }
  } else {
    if (!encode_2d(&mk, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows, HS_D_QK, n, HS_D_QK * 2, 64, Sh::kMine, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&mv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows, HS_D_QK, n, HS_D_QK * 2, 64, kKeys, CU_TENSOR_MAP_SWIZZLE_128B)) {
      *why = "cuTensorMapEncodeTiled failed for the dequantised rows";
      return cudaErrorInvalidValue;
    }
    expand_kernel<<<4 * sms, kExpandThreads, 0, stream>>>(p, const_cast<uint16_t*>(rows));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (kRaw) {
    kernel<<<2 * G * C, Sh::kThreads, kSmem, stream>>>(mk, mv, mr, p);
    e = cudaGetLastError();
  } else {
    e = launch_next(kernel, dim3(2 * G * C), Sh::kThreads, kSmem, stream, mk, mv, mr, p);
  }
  if (e != cudaSuccess) return e;
  return launch_next(paged_merge_kernel<Sh::kRows>, Merge<Sh::kRows>::grid(C), kMergeThreads, 0, stream, p);
}
}  // namespace paged

uint64_t paged_mla_workspace_bytes(int T, int B, int H, int64_t kv_tokens, int sms) {
  using namespace paged;
  return part_bytes(sms) + (copies(T, B, H) ? (uint64_t)copy_capacity(B, kv_tokens) * HS_D_QK * 2 : 0);
}

cudaError_t launch_paged_mla(const hs_paged_mla_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace paged;
  const int most = sms / (2 * G);
  Params p;
  p.T = a->T;
  p.B = a->B;
  p.H = a->H;
  p.causal = a->causal;
  p.bt_stride = a->bt_stride;
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
  if (few_rows(a->T, a->B, a->H)) return launch_few(p, sms, stream);
  p.part_lse = p.part_out + (int64_t)2 * most * (kHalf * G) * HS_D_LATENT;
  p.desc = reinterpret_cast<Desc*>(p.part_lse + (int64_t)2 * most * (kHalf * G));
  const uint16_t* rows = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(a->workspace) + part_bytes(sms));
  const uint64_t n = (uint64_t)copy_capacity(a->B, a->kv_tokens);
  return copies(a->T, a->B, a->H) ? launch<false>(p, rows, n, sms, stream, why) : launch<true>(p, rows, n, sms, stream, why);
}

}  // namespace hs
