// rope.cu — rotary positions of queries and keys, any even part of a head, one launch for both.
//
// Token t at position p turns pair i of each head by the angle p * inv_freq[i]:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos)
// where (a, b) are values (2i, 2i + 1) of the rotary part (interleaved) or (i, i + rot / 2) (halves).
// [P1] "vLLM v0.32.0 GLM-5.3 サービング ...", section 「数字がうまくいく理由」: a cached row carries 64
// bf16 RoPE values beside its latent codes; hs_kv_append stores them and the MLA reads them as given.
//
// The angle of a far position. p * inv_freq in fp32 is off by up to p * inv_freq * 2^-24, 0.06 rad
// at a million. Here a pair's frequency is a 64-bit fixed-point fraction of a turn, f = inv_freq /
// (2 pi) * 2^64 (one fp64 multiplication per pair and CTA), and the product p * f mod 2^64 drops whole
// turns exactly, in integers. What is left, read as a signed fraction, is rounded to fp32 once (2^-24
// of half a turn) and goes to sincospif. No table of positions is read or kept.
//
// Bound by HBM: every value is read and written once. A CTA computes the cosines and sines of its
// tokens into shared memory (one thread per (token, pair)), then its threads take units of 8 pairs
// (16-bit types) or 4 pairs (fp32), two 16-byte loads and two 16-byte stores each, over tokens, heads
// and pair groups. Where a base address or a stride is no multiple of 16 bytes, or rot / 2 no multiple
// of the unit's pairs, a unit is one pair (element loads).
//
// A CTA has at most eight tokens (fewer when there are few, so that all SMs have work), each thread two units in flight
// before the first is stored, and a unit's token and head follow from the thread's last one by additions. Measured on a GB300:
// 16,384 tokens x 64 heads x 64 values, heads 192 and 576 wide, 53 us, 5,130 GB/s (a contiguous copy of the same bytes takes
// 43 us, a strided copy in PyTorch 141 us); with divisions per unit and one unit in flight it took 76 us.
#include "common.cuh"

namespace hs {
namespace rope {

constexpr int kThreads = 256;

struct Tensor {
  const uint8_t* x;
  uint8_t* out;
  int64_t xt, xh, ot, oh;  // strides in bytes: token, head
};

struct Params {
  int32_t T, H, H2, half, inverse, per_cta;
  int32_t step_t, step_h, step_g;  // kThreads units as tokens, heads and pair groups
  float scale;
  const int32_t* pos;
  const double* inv_freq;
  Tensor a, b;
};

template <typename E>
__device__ __forceinline__ float to_f(E v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// Two pieces of a unit: V pairs' values. Interleaved: 2 V consecutive values; halves: V values of the
// first half and the V matching ones of the second.
template <typename E, int V>
union Unit {
  E v[2 * V];
  uint4 w[sizeof(E) * V >= 16 ? 2 : 1];
};

// A unit's place in the CTA's work: token, head (of both tensors) and pair group, stepped by kThreads
// units without divisions.
struct Place {
  int t, h, g;
  __device__ __forceinline__ void step(const Params& p, int groups, int heads) {
    g += p.step_g;
    const bool a = g >= groups;
    g -= a ? groups : 0;
    h += p.step_h + (a ? 1 : 0);
    const bool b = h >= heads;
    h -= b ? heads : 0;
    t += p.step_t + (b ? 1 : 0);
  }
};

template <typename E, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const Params p) {
  extern __shared__ float2 cs[];  // [per_cta][half]: scale * (cos, sin)
  const int t0 = blockIdx.x * p.per_cta;
  const int nt = min(p.per_cta, p.T - t0);
  const int groups = p.half / V;  // units of a head
  const int heads = p.H + p.H2;
  constexpr bool kVec = V > 1;
  constexpr int kAhead = kVec ? 2 : 8;  // units in flight per thread
  Unit<E, V> u[kAhead];
  E* dst[kAhead];
  int at[kAhead];  // the unit's cosines; -1: no unit

  Place w;
  {
    const int th = threadIdx.x / groups;
    w.g = threadIdx.x - th * groups;
    w.t = th / heads;
    w.h = th - w.t * heads;
  }
  auto load = [&]() {  // this thread's next units
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at[k] = -1;
      if (w.t < nt) {
        const bool first = w.h < p.H;
        const int64_t tt = t0 + w.t, hh = first ? w.h : w.h - p.H;
        const int off = kInterleaved ? 2 * V * w.g : V * w.g;
        const E* s0 = reinterpret_cast<const E*>((first ? p.a.x : p.b.x) + tt * (first ? p.a.xt : p.b.xt) + hh * (first ? p.a.xh : p.b.xh)) + off;
        dst[k] = reinterpret_cast<E*>((first ? p.a.out : p.b.out) + tt * (first ? p.a.ot : p.b.ot) + hh * (first ? p.a.oh : p.b.oh)) + off;
        at[k] = w.t * p.half + V * w.g;
        const E* s1 = kInterleaved ? s0 + V : s0 + p.half;
        if constexpr (kVec) {
          u[k].w[0] = *reinterpret_cast<const uint4*>(s0);
          u[k].w[1] = *reinterpret_cast<const uint4*>(s1);
        } else {
          u[k].v[0] = *s0;
          u[k].v[1] = *s1;
        }
      }
      w.step(p, groups, heads);
    }
  };

  load();  // the first units' values are on their way while the angles are computed
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int t = i / p.half, k = i - t * p.half;
    double f = p.inv_freq[k] * 0.15915494309189533577;  // turns per position
    f -= floor(f);
    const uint64_t step = (uint64_t)(f * 18446744073709551616.0);
    const int64_t turn = (int64_t)((uint64_t)(int64_t)p.pos[t0 + t] * step);  // whole turns drop out
    float s, c;
    sincospif((float)turn * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    cs[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
  }
  __syncthreads();
  while (at[0] >= 0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (at[k] < 0) break;
      const float2* c = cs + at[k];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int ia = kInterleaved ? 2 * j : j, ib = kInterleaved ? 2 * j + 1 : V + j;
        const float a = to_f(u[k].v[ia]), b = to_f(u[k].v[ib]);
        const float2 e = c[j];
        u[k].v[ia] = from_f<E>(a * e.x - b * e.y);
        u[k].v[ib] = from_f<E>(a * e.y + b * e.x);
      }
      E* d1 = kInterleaved ? dst[k] + V : dst[k] + p.half;
      if constexpr (kVec) {
        *reinterpret_cast<uint4*>(dst[k]) = u[k].w[0];
        *reinterpret_cast<uint4*>(d1) = u[k].w[1];
      } else {
        dst[k][0] = u[k].v[0];
        d1[0] = u[k].v[1];
      }
    }
    load();
  }
}

template <typename E, int V>
cudaError_t launch(const Params& p, bool interleaved, unsigned grid, size_t smem, cudaStream_t stream) {
  if (interleaved)
    rope_kernel<E, V, true><<<grid, kThreads, smem, stream>>>(p);
  else
    rope_kernel<E, V, false><<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rope

cudaError_t launch_rope(const hs_rope_args* a, int sms, cudaStream_t stream) {
  using namespace rope;
  const int64_t e = a->dtype == HS_FP32 ? 4 : 2;
  Params p;
  p.T = a->T;
  p.H = a->H;
  p.H2 = a->y ? a->H2 : 0;
  p.half = a->rot / 2;
  p.inverse = a->inverse;
  p.scale = a->scale;
  p.pos = a->positions;
  p.inv_freq = a->inv_freq;
  p.a = {(const uint8_t*)a->x, (uint8_t*)a->out, a->x_stride_t * e, a->x_stride_h * e, a->out_stride_t * e, a->out_stride_h * e};
  p.b = p.a;
  if (a->y)
    p.b = {(const uint8_t*)a->y, (uint8_t*)a->y_out, a->y_stride_t * e, a->y_stride_h * e, a->y_out_stride_t * e,
           a->y_out_stride_h * e};
  uint64_t bits = 0;  // every address and stride; a multiple of 16 bytes only if all are
  for (const Tensor* t : {&p.a, &p.b})
    bits |= (uint64_t)(uintptr_t)t->x | (uint64_t)(uintptr_t)t->out | (uint64_t)t->xt | (uint64_t)t->xh | (uint64_t)t->ot |
            (uint64_t)t->oh;
  const int V = e == 4 ? 4 : 8;
  const bool vec = (bits & 15) == 0 && p.half % V == 0;
  const int groups = p.half / (vec ? V : 1), heads = p.H + p.H2;
  p.step_g = kThreads % groups;
  p.step_h = kThreads / groups % heads;
  p.step_t = kThreads / groups / heads;
  // Tokens per CTA: up to eight, while a thread gets no more than eight units and every SM still gets eight CTAs
  const int64_t units = (int64_t)heads * groups;
  int per = 1;
  while (per < 8 && 2 * per * units <= 8 * kThreads && (int64_t)a->T >= 16LL * per * sms) per *= 2;
  p.per_cta = per;
  const unsigned grid = ((unsigned)a->T + per - 1) / per;
  const size_t smem = (size_t)per * p.half * sizeof(float2);
  const bool il = a->interleaved != 0;
  switch (a->dtype) {
    case HS_FP32: return vec ? launch<float, 4>(p, il, grid, smem, stream) : launch<float, 1>(p, il, grid, smem, stream);
    case HS_FP16: return vec ? launch<__half, 8>(p, il, grid, smem, stream) : launch<__half, 1>(p, il, grid, smem, stream);
    default:
      return vec ? launch<__nv_bfloat16, 8>(p, il, grid, smem, stream) : launch<__nv_bfloat16, 1>(p, il, grid, smem, stream);
  }
}

}  // namespace hs
