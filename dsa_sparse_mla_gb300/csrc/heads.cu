// heads.cu — the products between latent vectors and heads: hs_mla_expand (keys and values of every head from latent rows),
// hs_mla_absorb (queries into the latent space) and hs_mla_project (latent outputs to values).
//
// One weight W [H, Dn + Dv, 512] serves all three, as it is stored:
//   expand   kv[n, (h, d)]  = sum_c latent[n, c] W[h, d, c]         B = W, reduced over c: K-major
//   project  out[t, h, d]   = sum_c x[t, h, c]   W[h, Dn + d, c]    the same, a product per head
//   absorb   out[t, h, c]   = sum_d q[t, h, d]   W[h, d, c]         reduced over d: W is the MN-major operand
// so one kernel computes C[m, h, n] = sum_k A[m, h, k] B_h[n, k] and the calls differ in coordinates and in B's major-ness.
//
// A pair of CTAs computes tiles of 256 rows and kBN columns with two-SM MMAs: each CTA holds its 128 rows of A, half of the
// columns of B, and its rows of the accumulator (two tiles of them in tensor memory, so that one tile's epilogue runs under the next
// tile's products). All of a head's B (or 256 columns of the expanded width: 128 KB of shared memory per CTA at most) is there at
// once. Where every group of columns reads the same A (expand) it stays for up to four row tiles, and only A streams through the ring; absorb
// and project, whose A differs from head to head, load it again for each tile. B comes and goes in chunks of 64 reduced values, with
// barriers of their own, so that a change of B costs no more than a load's latency. Eight epilogue warps round to bf16 once. Rows beyond
// M are read as zeros and not stored.
//
// Stores. expand and project, which multiply 512 values for each one that they store, need a deep ring more than anything, since copies of
// A wait behind the stores (expand, lines through shared memory, 3, 4 and 5 slots: 394, 364, 351 us): a lane stores its row in sectors of
// 32 bytes straight from registers, and the ring has all of the room (six slots: 319; in pieces of 16 bytes, where a stride leaves
// nothing else, 423). absorb stores three bytes of four: whole 128-byte lines through shared memory (240 us, in sectors 251; 256 tokens
// 7.7 and 8.5).
//
// absorb and project are bound by HBM: 16,384 tokens x 64 heads (1.35 GB) 231 to 242 us, 5.6 to 5.8 TB/s; 4,099 x 128 (192, 256) 142 to
// 146, 5.8 TB/s. expand: 32,768 rows x 64 heads x 256 319 to 329 us in a few calls (1,670 to 1,720 TFLOP/s; one library product of the
// same sizes 324 to 333) and 365 to 385 in long runs (1,430 to 1,510), bound by power: with zeros for inputs it takes 287. What the issuing thread
// executes between two batches of MMAs is not hidden: a wait in its loop that expand never reaches, eight times unrolled, made it 359
// instead of 345 (without copies and stores 278 and 237; 229 are MMAs). Tried and not kept: B streaming with A, two issuing warps, two
// copying warps, TMA stores, 16 epilogue warps, clusters of four with A multicast to both pairs (36 of them fit, 144 SMs: 336 where
// pairs took 329).
#include "launch.cuh"
#include "pair.cuh"

namespace hs {
namespace heads {

constexpr int kBM = 256, kHalfM = 128, kBK = 64;
constexpr int kThreads = 384;                 // copies, MMAs, two idle, eight epilogue warps
constexpr int kSlot = kHalfM * kBK * 2;       // 16 KB of A
constexpr int kRoom = 14;                     // slots in all: B's chunks, then A's ring, then the epilogue's lines
constexpr int kMaxSlots = 11, kMaxChunks = 8;
constexpr int kEpiWarps = 8, kScratch = 4096; // 32 rows x 128 bytes per epilogue warp
constexpr int kOffEpi = kRoom * kSlot - kEpiWarps * kScratch, kOffBar = kRoom * kSlot, kSmem = kOffBar + 512;
static_assert(kSmem <= 232448, "shared memory");

struct Params {
  int64_t units;
  uint16_t* c;
  int64_t c_stride_m, c_stride_h;
  int32_t M, N;            // rows; columns per head
  int32_t m_tiles, m_unit; // row tiles; of a unit
  int32_t groups;          // heads, or parts of the expanded width
  int32_t n_tiles;         // column tiles of a group, one or two: their B stays together
  int32_t per_head;        // groups per head
  int32_t k_steps, slots;
  int32_t a_again;         // A is read by every group
  int32_t b_head, b_row;   // B's rows of head h start at h * b_head + b_row
  int32_t sectors;         // C's rows start on 32 bytes
  int32_t* err;
};

struct Bars {
  uint64_t a_full[kMaxSlots], a_empty[kMaxSlots], b_full[kMaxChunks], b_empty[kMaxChunks], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// A pair's items: every so many of the units, a unit being up to m_unit row tiles of one group. Units follow one another with the groups
// fastest, so that pairs running at the same time read the same rows of A and write whole rows of C.
struct Run {
  int64_t unit, step, units;
  int32_t g, m, end, groups, m_unit, m_tiles;
  __device__ __forceinline__ explicit Run(const Params& p) {
    step = gridDim.x >> 1, unit = blockIdx.x >> 1, units = p.units;
    groups = p.groups, m_unit = p.m_unit, m_tiles = p.m_tiles;
    start();
  }
  __device__ __forceinline__ void start() {
    const int32_t s = (int32_t)(unit / groups);
    g = (int32_t)(unit - (int64_t)s * groups);
    m = s * m_unit;
    end = min(m + m_unit, m_tiles);
  }
  __device__ __forceinline__ bool more() const { return unit < units; }
  __device__ __forceinline__ bool last() const { return m + 1 == end; }  // of its unit
  __device__ __forceinline__ void next() {
    if (++m == end) {
      unit += step;
      if (unit < units) start();
    }
  }
};

// 16 values, 32 bytes on a 32-byte boundary, in one store.
__device__ __forceinline__ void store_sector(uint16_t* to, const uint32_t* w) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int kBN, bool kMnMajor>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    heads_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Params p) {
  constexpr int kChunk = kBN / 2 * kBK * 2;  // of B per CTA
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in both CTAs
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  Bars& br = *reinterpret_cast<Bars*>(smem + kOffBar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  uint8_t* ring_a = smem + p.n_tiles * p.k_steps * kChunk;
  let_next();
  if (tid < kMaxSlots) {
    mbar_init(&br.a_full[tid], 2);
    mbar_init(&br.a_empty[tid], 1);
  } else if (tid >= 32 && tid < 32 + kMaxChunks) {
    mbar_init(&br.b_full[tid - 32], 2);
    mbar_init(&br.b_empty[tid - 32], 1);
  } else if (tid >= 64 && tid < 66) {
    mbar_init(&br.acc_full[tid - 64], 1);
    mbar_init(&br.acc_empty[tid - 64], 2 * kEpiWarps);
  } else if (tid == 66) {
    mbar_init(&br.drain, 1);
  } else if (tid == 96) {
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
  }
  mbar_fence_init();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  if (warp == 0) tc2::alloc(&br.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem;
  Run run(p);
  after_previous();

  if (warp == 0) {
    // ================================================================ copies ====================
    if (lane == 0) {
      const uint32_t a_full = remote_smem(br.a_full, 0), b_full = remote_smem(br.b_full, 0);
      const uint64_t keep = l2_policy_evict_last(), stream = l2_policy_evict_first();
      int slot = 0;
      uint32_t par = 1, groups = 0;
      bool ok = true;
#pragma unroll 1
      for (bool first = true; run.more() && ok; first = run.last(), run.next()) {
        const int h = run.g / p.per_head, n0 = run.g % p.per_head * p.n_tiles * kBN + (int)rank * (kBN / 2);
        const int rows = h * p.b_head + p.b_row, y = run.m * kBM + kHalfM * (int)rank;
#pragma unroll 1
        for (int c = 0; c < (first ? p.n_tiles : 1) * p.k_steps; ++c) {  // chunk c: column tile c / k_steps
          const int nt = c >= p.k_steps ? 1 : 0, k = c - nt * p.k_steps;
          // The first column tile's chunk of B is needed together with A's stage and counts on its barrier; the second one's on its own.
          uint32_t bar = b_full + 8 * (uint32_t)c;
          if (nt == 0) {
            ok = mbar_wait(&br.a_empty[slot], par, p.err);
            if (!ok) break;
            bar = a_full + 8 * (uint32_t)slot;
            pair::arrive_expect_tx(bar, first ? kSlot + kChunk : kSlot);
            pair::load_3d(ring_a + slot * kSlot, &map_a, bar, k * kBK, h, y, p.a_again ? keep : stream);
            if (++slot == p.slots) slot = 0, par ^= 1u;
          }
          if (first) {
            ok = mbar_wait(&br.b_empty[c], (groups & 1u) ^ 1u, p.err);
            if (!ok) break;
            uint8_t* d = smem + c * kChunk;
            if (nt == 1) pair::arrive_expect_tx(bar, kChunk);
            if (kMnMajor) {  // 64 reduced rows of this CTA's columns, 64 columns to a block
#pragma unroll 1
              for (int b = 0; b < kBN / 128; ++b) pair::load_2d(d + b * 8192, &map_b, bar, n0 + nt * kBN + 64 * b, rows + k * kBK, keep);
            } else {
              pair::load_2d(d, &map_b, bar, k * kBK, rows + n0 + nt * kBN, keep);
            }
          }
        }
        if (first) ++groups;
      }
      if (!ok) pair::let_copies_land();
    }
  } else if (warp == 1) {
    // ================================================================ MMAs ======================
    // Whether the next stage is there is asked before a stage's MMAs, whose issue hides the answer's latency. The loop has to be small:
    // only absorb has a second column tile, whose B it waits for.
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = idesc_bf16(kBM, kBN, 0, kMnMajor ? 1 : 0);
      const uint64_t ad = smem_desc(smem_u32(ring_a), 16, 1024, 2);
      const uint64_t bd = smem_desc(smem_u32(smem), kMnMajor ? 8192 : 16, 1024, 2);
      int slot0 = 0;
      uint32_t par0 = 0, it = 0, groups = 0;
      bool ok = true, there = false;  // there: the next stage of A has been seen
#pragma unroll 1
      for (bool first = true; run.more() && ok; first = run.last(), run.next()) {
        const bool last = run.last();
        int slot = slot0;
        uint32_t par = par0;
#pragma unroll 1
        for (int nt = 0, c = 0; nt < p.n_tiles && ok; ++nt, ++it) {
          const uint32_t b = it & 1u, d = tmem + b * 256u;
          slot = slot0, par = par0;
          ok = mbar_wait(&br.acc_empty[b], ((it >> 1) & 1u) ^ 1u, p.err);
          if (!ok) break;
#pragma unroll(kMnMajor ? 1 : 8)
          for (int k = 0; k < (kMnMajor ? p.k_steps : HS_D_LATENT / kBK); ++k, ++c) {
            if (nt == 0 && !there) ok = mbar_wait(&br.a_full[slot], par, p.err);
            if (kMnMajor && nt == 1 && first && ok) ok = mbar_wait(&br.b_full[c], groups & 1u, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = ad + (uint64_t)((slot * kSlot) >> 4), w = bd + (uint64_t)((c * kChunk) >> 4);
            uint64_t* empty = &br.a_empty[slot];
            if (++slot == p.slots) slot = 0, par ^= 1u;
            there = pair::test_wait(&br.a_full[slot], par);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              tc2::ss(d, a + 2 * kk, w + (kMnMajor ? 128 : 2) * kk, id, (k | kk) != 0 ? 1u : 0u);
            if (nt + 1 == p.n_tiles) tc2::commit(empty, 0x3);
            if (last) tc2::commit(&br.b_empty[c], 0x3);
          }
          if (ok) tc2::commit(&br.acc_full[b], 0x3);
        }
        slot0 = slot, par0 = par;
        if (first) ++groups;
      }
      tc2::commit(&br.drain, 0x1);
      mbar_wait(&br.drain, 0, p.err);
    }
  } else if (warp >= 4) {
    // ================================================================ epilogue ==================
    // Warp (quad, g): rows 32 quad .. + 31 of this CTA, columns g kBN / 2 .. of the tile, 64 at a time.
    const int quad = warp & 3, g = (warp - 4) >> 2;
    const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(g * (kBN / 2));
    const uint32_t acc_empty = remote_smem(br.acc_empty, 0);
    uint8_t* s = smem + kOffEpi + (warp - 4) * kScratch;
    const int pl = lane & 7, rl = lane >> 3;
    uint32_t it = 0;
    bool ok = true;
#pragma unroll 1
    for (; run.more() && ok; run.next()) {
      const int h = run.g / p.per_head, n0 = run.g % p.per_head * p.n_tiles * kBN + g * (kBN / 2);
      const int row = run.m * kBM + kHalfM * (int)rank + 32 * quad, left = p.M - row;
      uint16_t* const c0 = p.c + (int64_t)(row + (kMnMajor ? rl : lane)) * p.c_stride_m + (int64_t)h * p.c_stride_h + n0 + (kMnMajor ? 8 * pl : 0);
#pragma unroll 1
      for (int nt = 0; nt < p.n_tiles; ++nt, ++it) {
        const uint32_t b = it & 1u;
        ok = warp_wait_all(&br.acc_full[b], (it >> 1) & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kBN / 128; ++c) {
          uint32_t v[2][32];
          tmem_ld32(at + b * 256u + 64 * c, v[0]);
          tmem_ld32(at + b * 256u + 64 * c + 32, v[1]);
          tmem_wait_ld();
          if (c == kBN / 128 - 1) {  // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive_relaxed(acc_empty + 8 * b);
          }
          const int col = nt * kBN + 64 * c;
          if (left <= 0 || n0 + col >= p.N) continue;
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[i >> 4][2 * (i & 15)]), __uint_as_float(v[i >> 4][2 * (i & 15) + 1]));
            w[i] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          uint16_t* to = c0 + col;
          if constexpr (kMnMajor) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(s + sw128_offset(lane, 16 * j)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j, to += 4 * p.c_stride_m) {
              const uint4 x = *reinterpret_cast<const uint4*>(s + sw128_offset(4 * j + rl, 16 * pl));
              if (4 * j + rl < left) __stcs(reinterpret_cast<uint4*>(to), x);
            }
            __syncwarp();
          } else if (lane < left) {
            if (p.sectors) {
#pragma unroll
              for (int j = 0; j < 4; ++j) store_sector(to + 16 * j, w + 8 * j);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) __stcs(reinterpret_cast<uint4*>(to + 8 * j), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
            }
          }
        }
      }
    }
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still signal or read it
  if (warp == 0) {
    tc_fence_after();
    tc2::dealloc(tmem, 512);
  }
}

template <int kBN, bool kMnMajor>
static cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, Params p, int sms, cudaStream_t stream) {
  auto kernel = heads_kernel<kBN, kMnMajor>;
  const cudaError_t e = pair::allow_smem(kernel, kSmem);
  if (e != cudaSuccess) return e;
  p.m_tiles = (int)(((int64_t)p.M + kBM - 1) / kBM);
  // Units of several row tiles reload B less often, but are fewer: at least four for each pair (1,501 rows x 28 groups 17.5 us with units of
  // four row tiles, 15.0 with one).
  while (p.m_unit > 1 && (int64_t)p.m_tiles * p.groups < (int64_t)p.m_unit * 4 * (sms / 2)) p.m_unit /= 2;
  p.units = ((int64_t)p.m_tiles + p.m_unit - 1) / p.m_unit * p.groups;
  const int slots = ((kMnMajor ? kOffEpi : kOffBar) - p.n_tiles * p.k_steps * (kBN / 2 * kBK * 2)) / kSlot;  // 6 at least; absorb 4
  p.sectors = (reinterpret_cast<uintptr_t>(p.c) | (uintptr_t)(p.c_stride_m * 2) | (uintptr_t)(p.c_stride_h * 2)) % 32 == 0;
  p.slots = slots < kMaxSlots ? slots : kMaxSlots;
  const int64_t pairs = p.units < sms / 2 ? p.units : sms / 2;
  return launch_next(kernel, dim3((unsigned)(2 * pairs)), kThreads, kSmem, stream, ma, mb, p);
}

static cudaError_t maps_failed(const char** why) {
  *why = "cuTensorMapEncodeTiled failed";
  return cudaErrorInvalidValue;
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapSwizzle kSw128 = CU_TENSOR_MAP_SWIZZLE_128B;

}  // namespace heads

cudaError_t launch_mla_expand(const hs_mla_expand_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace heads;
  const int width = a->H * a->width;
  CUtensorMap ma, mb;
  if (!pair::encode_heads(&ma, a->latent, HS_D_LATENT, 1, a->N, HS_D_LATENT, a->latent_stride, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)width, HS_D_LATENT * 2, kBK, 128, kSw128))
    return maps_failed(why);
  Params p = {};
  p.c = a->kv, p.c_stride_m = a->kv_stride, p.c_stride_h = width;
  p.M = a->N, p.N = width, p.n_tiles = 1, p.per_head = p.groups = (width + 255) / 256, p.k_steps = HS_D_LATENT / kBK;
  p.a_again = 1, p.m_unit = 4, p.err = a->err_flag;
  return launch<256, false>(ma, mb, p, sms, stream);
}

cudaError_t launch_mla_absorb(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace heads;
  CUtensorMap ma, mb;
  if (!pair::encode_heads(&ma, a->x, a->Dn, a->H, a->T, a->x_stride_h, a->x_stride_t, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)a->H * (a->Dn + a->Dv), HS_D_LATENT * 2, 64, kBK, kSw128))
    return maps_failed(why);
  Params p = {};
  p.c = a->out, p.c_stride_m = a->out_stride_t, p.c_stride_h = a->out_stride_h;
  p.M = a->T, p.N = HS_D_LATENT, p.n_tiles = 2, p.per_head = 1, p.groups = a->H, p.k_steps = a->Dn / kBK;
  p.b_head = a->Dn + a->Dv, p.m_unit = 1, p.err = a->err_flag;
  return launch<256, true>(ma, mb, p, sms, stream);
}

cudaError_t launch_mla_project(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace heads;
  const int bn = a->Dv > 128 ? 256 : 128;
  CUtensorMap ma, mb;
  if (!pair::encode_heads(&ma, a->x, HS_D_LATENT, a->H, a->T, a->x_stride_h, a->x_stride_t, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)a->H * (a->Dn + a->Dv), HS_D_LATENT * 2, kBK, bn / 2, kSw128))
    return maps_failed(why);
  Params p = {};
  p.c = a->out, p.c_stride_m = a->out_stride_t, p.c_stride_h = a->out_stride_h;
  p.M = a->T, p.N = a->Dv, p.n_tiles = 1, p.per_head = 1, p.groups = a->H, p.k_steps = HS_D_LATENT / kBK;
  p.b_head = a->Dn + a->Dv, p.b_row = a->Dn, p.m_unit = 1, p.err = a->err_flag;
  return bn == 256 ? launch<256, false>(ma, mb, p, sms, stream) : launch<128, false>(ma, mb, p, sms, stream);
}

}  // namespace hs
