// heads.cu — the products between latent vectors and heads: hs_mla_expand (keys and values of every head from latent rows),
// hs_mla_absorb (queries into the latent space) and hs_mla_project (latent outputs to values).
//
// One weight W [H, Dn + Dv, 512] serves all three, as it is stored:
//   expand   kv[n, (h, d)]  = sum_c latent[n, c] W[h, d, c]         B = W, reduced over c: K-major
//   project  out[t, h, d]   = sum_c x[t, h, c]   W[h, Dn + d, c]    the same, a product per head
//   absorb   out[t, h, c]   = sum_d q[t, h, d]   W[h, d, c]         reduced over d: W is the MN-major operand
// so one kernel computes C[m, h, n] = sum_k A[m, h, k] B_h[n, k] and the calls differ in coordinates and in B's major-ness.
//
// A pair of CTAs computes a tile of 256 rows and kBN columns with two-SM MMAs: each CTA holds its 128 rows of A, half of the
// B tile, and its rows of the accumulator (two of them in tensor memory, so that one tile's epilogue runs under the next
// tile's products). TMA feeds a ring of stages of 64 reduced values; eight epilogue warps round to bf16 once and store whole
// 128-byte lines by TMA, which also leaves out what is past the tensor's ends. Reduced values beyond K or rows beyond M are read
// as zeros. Tiles go to the pairs in order, heads (or columns) fastest, so that pairs running at the same time read and
// write whole rows of A and C.
#include <atomic>

#include "pair.cuh"

namespace hs {
namespace heads {

constexpr int kBM = 256, kHalfM = 128, kBK = 64;
constexpr int kThreads = 384;                 // producer, MMAs, two idle, eight epilogue warps
constexpr int kABytes = kHalfM * kBK * 2;     // 16 KB
constexpr int kEpiWarps = 8, kScratch = 4096; // 32 rows x 128 bytes, two per epilogue warp

template <int kBN>
struct Shape {
  static constexpr int kBBytes = kBN / 2 * kBK * 2, kStage = kABytes + kBBytes;
  static constexpr int kStages = kBN == 256 ? 5 : 6;
  static constexpr int kOffEpi = kStages * kStage, kOffBar = kOffEpi + kEpiWarps * 2 * kScratch;
  static constexpr int kSmem = kOffBar + 256;
  static_assert(kSmem <= 232448 && kStage % 1024 == 0, "shared memory");
};

struct Params {
  int64_t tiles;
  int32_t M, N;            // rows; columns per head
  int32_t n_tiles, heads;  // column tiles per head
  int32_t k_steps;
  int32_t b_head, b_row;   // B's rows of head h start at h * b_head + b_row
  int32_t* err;
};

struct Bars {
  uint64_t full[6], empty[6], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
};

template <int kBN, bool kMnMajor>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    heads_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_c, const Params p) {
  using Sh = Shape<kBN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in both CTAs
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  Bars& br = *reinterpret_cast<Bars*>(smem + Sh::kOffBar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < 6; ++s) {
      mbar_init(&br.full[s], 2);
      mbar_init(&br.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&br.acc_full[b], 1);
      mbar_init(&br.acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&br.drain, 1);
    mbar_fence_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    prefetch_tensormap(&map_c);
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  if (warp == 0) tc2::alloc(&br.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem;

  auto place = [&](int64_t tile, int& m0, int& h, int& n0) {
    const int per_row = p.n_tiles * p.heads;
    m0 = (int)(tile / per_row) * kBM;
    const int rest = (int)(tile % per_row);
    h = rest / p.n_tiles;
    n0 = rest % p.n_tiles * kBN;
  };

  if (warp == 0) {
    // ================================================================ copies ====================
    if (lane == 0) {
      const uint32_t full = remote_smem(br.full, 0);
      int slot = 0;
      uint32_t par = 1;
      bool ok = true;
#pragma unroll 1
      for (int64_t tile = first; tile < p.tiles && ok; tile += step) {
        int m0, h, n0;
        place(tile, m0, h, n0);
#pragma unroll 1
        for (int k = 0; k < p.k_steps; ++k) {
          if (!mbar_wait(&br.empty[slot], par, p.err)) {
            ok = false;
            break;
          }
          const uint32_t bar = full + 8 * (uint32_t)slot;
          uint8_t* a = smem + slot * Sh::kStage;
          pair::arrive_expect_tx(bar, Sh::kStage);
          pair::load_3d(a, &map_a, bar, k * kBK, h, m0 + kHalfM * (int)rank);
          if (kMnMajor) {  // 64 reduced rows of this CTA's columns, 64 columns to a block
#pragma unroll
            for (int b = 0; b < kBN / 128; ++b)
              pair::load_2d(a + kABytes + b * 8192, &map_b, bar, n0 + (int)rank * (kBN / 2) + 64 * b, h * p.b_head + p.b_row + k * kBK);
          } else {
            pair::load_2d(a + kABytes, &map_b, bar, k * kBK, h * p.b_head + p.b_row + n0 + (int)rank * (kBN / 2));
          }
          if (++slot == Sh::kStages) slot = 0, par ^= 1u;
        }
      }
      if (!ok) pair::let_copies_land();
    }
  } else if (warp == 1) {
    // ================================================================ MMAs ======================
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = idesc_bf16(kBM, kBN, 0, kMnMajor ? 1 : 0);
      const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t bd = smem_desc(smem_u32(smem + kABytes), kMnMajor ? 8192 : 16, 1024, 2);
      int slot = 0;
      uint32_t par = 0;
      uint32_t it = 0;
      bool ok = true;
#pragma unroll 1
      for (int64_t tile = first; tile < p.tiles && ok; tile += step, ++it) {
        const uint32_t b = it & 1u, d = tmem + b * 256u;
        if (!mbar_wait(&br.acc_empty[b], ((it >> 1) & 1u) ^ 1u, p.err)) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < p.k_steps; ++k) {
          if (!mbar_wait(&br.full[slot], par, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)((slot * Sh::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            tc2::ss(d, ad + off + (uint64_t)((kk * 32) >> 4), bd + off + (uint64_t)((kk * (kMnMajor ? 2048 : 32)) >> 4), id,
                    (k | kk) != 0 ? 1u : 0u);
          tc2::commit(&br.empty[slot], 0x3);
          if (++slot == Sh::kStages) slot = 0, par ^= 1u;
        }
        if (ok) tc2::commit(&br.acc_full[b], 0x3);
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
    uint8_t* scratch = smem + Sh::kOffEpi + (warp - 4) * 2 * kScratch;
    uint32_t it = 0, n = 0;
#pragma unroll 1
    for (int64_t tile = first; tile < p.tiles; tile += step, ++it) {
      const uint32_t b = it & 1u;
      if (!warp_wait_all(&br.acc_full[b], (it >> 1) & 1u, p.err)) break;
      tc_fence_after();
      int m0, h, n0;
      place(tile, m0, h, n0);
      m0 += kHalfM * (int)rank + 32 * quad;
#pragma unroll
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
        const int col = n0 + g * (kBN / 2) + 64 * c;
        if (m0 >= p.M || col >= p.N) continue;
        uint8_t* s = scratch + (n++ & 1u) * kScratch;
        if (lane == 0) pair::store_wait_read<1>();  // the store before the last one has read its scratch
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 8 * j + 2 * z;
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[e >> 5][e & 31]), __uint_as_float(v[e >> 5][(e & 31) + 1]));
            w[z] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          *reinterpret_cast<uint4*>(s + sw128_offset(lane, 16 * j)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          pair::store_3d(&map_c, s, col, h, m0);
          pair::store_commit();
        }
      }
    }
    if (lane == 0) pair::store_wait_all();
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still signal or read it
  if (warp == 0) {
    tc_fence_after();
    tc2::dealloc(tmem, 512);
  }
}

template <int kBN, bool kMnMajor>
static cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const Params& p, int sms, cudaStream_t stream) {
  auto kernel = heads_kernel<kBN, kMnMajor>;
  constexpr int smem = Shape<kBN>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = p.tiles < sms / 2 ? p.tiles : sms / 2;
  kernel<<<(int)(2 * pairs), kThreads, smem, stream>>>(ma, mb, mc, p);
  return cudaGetLastError();
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
  CUtensorMap ma, mb, mc;
  if (!pair::encode_heads(&ma, a->latent, HS_D_LATENT, 1, a->N, HS_D_LATENT, a->latent_stride, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)width, HS_D_LATENT * 2, kBK, 128, kSw128) ||
      !pair::encode_heads(&mc, a->kv, width, 1, a->N, width, a->kv_stride, 32))
    return maps_failed(why);
  Params p = {};
  p.M = a->N, p.N = width, p.heads = 1, p.n_tiles = (width + 255) / 256, p.k_steps = HS_D_LATENT / kBK, p.err = a->err_flag;
  p.tiles = ((int64_t)a->N + kBM - 1) / kBM * p.n_tiles;
  return launch<256, false>(ma, mb, mc, p, sms, stream);
}

cudaError_t launch_mla_absorb(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace heads;
  CUtensorMap ma, mb, mc;
  if (!pair::encode_heads(&ma, a->x, a->Dn, a->H, a->T, a->x_stride_h, a->x_stride_t, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)a->H * (a->Dn + a->Dv), HS_D_LATENT * 2, 64, kBK, kSw128) ||
      !pair::encode_heads(&mc, a->out, HS_D_LATENT, a->H, a->T, a->out_stride_h, a->out_stride_t, 32))
    return maps_failed(why);
  Params p = {};
  p.M = a->T, p.N = HS_D_LATENT, p.heads = a->H, p.n_tiles = HS_D_LATENT / 256, p.k_steps = a->Dn / kBK, p.err = a->err_flag;
  p.b_head = a->Dn + a->Dv;
  p.tiles = ((int64_t)a->T + kBM - 1) / kBM * p.n_tiles * p.heads;
  return launch<256, true>(ma, mb, mc, p, sms, stream);
}

cudaError_t launch_mla_project(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace heads;
  const int bn = a->Dv > 128 ? 256 : 128;
  CUtensorMap ma, mb, mc;
  if (!pair::encode_heads(&ma, a->x, HS_D_LATENT, a->H, a->T, a->x_stride_h, a->x_stride_t, kHalfM) ||
      !encode_2d(&mb, kBf16, a->w, HS_D_LATENT, (uint64_t)a->H * (a->Dn + a->Dv), HS_D_LATENT * 2, kBK, bn / 2, kSw128) ||
      !pair::encode_heads(&mc, a->out, a->Dv, a->H, a->T, a->out_stride_h, a->out_stride_t, 32))
    return maps_failed(why);
  Params p = {};
  p.M = a->T, p.N = a->Dv, p.heads = a->H, p.n_tiles = 1, p.k_steps = HS_D_LATENT / kBK, p.err = a->err_flag;
  p.b_head = a->Dn + a->Dv, p.b_row = a->Dn;
  p.tiles = ((int64_t)a->T + kBM - 1) / kBM * p.heads;
  return bn == 256 ? launch<256, false>(ma, mb, mc, p, sms, stream) : launch<128, false>(ma, mb, mc, p, sms, stream);
}

}  // namespace hs
