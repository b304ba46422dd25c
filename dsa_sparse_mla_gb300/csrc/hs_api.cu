// hs_api.cu — the C ABI declared in include/hs.h: host-side argument checks, then launches.
// Nothing here allocates device memory, synchronises the stream (hs_check_flag aside) or keeps
// state between calls except the calling thread's last error text.
#include <atomic>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <unistd.h>

#include "common.cuh"

namespace hs {
cudaError_t launch_indexer(const hs_indexer_args* a, int num_sms, bool keep_scores, cudaStream_t stream,
                           const char** why);
cudaError_t launch_topk(const float* scores, int64_t ld, const int32_t* kvlen, int32_t T, int32_t k, int32_t* idx,
                        int32_t* err, bool discard, cudaStream_t stream);
cudaError_t launch_mla(const hs_mla_args* a, int sms, cudaStream_t stream, const char** why);
uint64_t mla_workspace_bytes(int32_t H, int sms);
cudaError_t launch_resolve(const hs_resolve_args* a, cudaStream_t stream);
cudaError_t launch_append(const hs_kv_append_args* a, int sms, cudaStream_t stream);
cudaError_t launch_offload(const hs_kv_offload_args* a, int sms, cudaStream_t stream);
cudaError_t launch_touch_host(int32_t B, const uint8_t* const* host_rows, const int32_t* seq_len,
                              const int32_t* resident_start, int64_t page, int32_t* err, cudaStream_t stream);
cudaError_t launch_rope(const hs_rope_args* a, int sms, cudaStream_t stream);
cudaError_t launch_paged_mla(const hs_paged_mla_args* a, int sms, cudaStream_t stream, const char** why);
uint64_t paged_mla_workspace_bytes(int T, int B, int H, int64_t kv_tokens, int sms);
cudaError_t launch_copy_pages(const hs_kv_copy_args* a, int sms, cudaStream_t stream);
cudaError_t launch_fork(const hs_kv_fork_args* a, cudaStream_t stream);
cudaError_t launch_free(const hs_kv_free_args* a, cudaStream_t stream);
cudaError_t launch_compact(const hs_kv_compact_args* a, int sms, cudaStream_t stream);
uint64_t compact_workspace_bytes(int64_t nblk);
cudaError_t launch_kv_read(const hs_kv_read_args* a, cudaStream_t stream);
cudaError_t launch_mla_absorb(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why);
cudaError_t launch_mla_project(const hs_mla_heads_args* a, int sms, cudaStream_t stream, const char** why);
cudaError_t launch_mla_expand(const hs_mla_expand_args* a, int sms, cudaStream_t stream, const char** why);
cudaError_t launch_mla_expanded(const hs_mla_expanded_args* a, int sms, cudaStream_t stream, const char** why);
uint64_t mla_expanded_workspace_bytes(int B, int Dv, int sms);
}  // namespace hs

namespace {

thread_local char g_last_error[512] = "";

hs_status fail(hs_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return s;
}

hs_status ok() {
  g_last_error[0] = '\0';
  return HS_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// The kernels use sm_103a instructions (tcgen05, TMA); other devices are refused up front.
hs_status check_device(int* num_sms) {
  static std::atomic<int> known[64];  // per device: its SMs, once it was found to be the right kind
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64) sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(HS_ERR_CUDA, "device query failed: %s", cudaGetErrorString(e));
    if (major != 10 || minor != 3)
      return fail(HS_ERR_UNSUPPORTED, "device %d has compute capability %d.%d; this library needs 10.3 (sm_103a)", dev,
                  major, minor);
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  if (num_sms) *num_sms = sms;
  return HS_OK;
}

hs_status launched(cudaError_t e, const char* what, const char* why) {
  if (e != cudaSuccess) {
    if (e == cudaErrorInvalidValue && why) return fail(HS_ERR_INVALID, "%s: %s", what, why);
    return fail(HS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  }
  return ok();
}

}  // namespace

namespace hs {
// Sets the calling thread's hs_last_error() text; returns s (for calls defined in other files).
hs_status set_last_error(hs_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return s;
}
}  // namespace hs

#define REQUIRE(cond, ...) \
  do {                     \
    if (!(cond)) return fail(HS_ERR_INVALID, __VA_ARGS__); \
  } while (0)

extern "C" {

int hs_abi_version(void) { return HS_ABI_VERSION; }

const char* hs_status_str(hs_status s) {
  switch (s) {
    case HS_OK: return "HS_OK";
    case HS_ERR_INVALID: return "HS_ERR_INVALID";
    case HS_ERR_UNSUPPORTED: return "HS_ERR_UNSUPPORTED";
    case HS_ERR_CUDA: return "HS_ERR_CUDA";
    case HS_ERR_DEVICE_FLAG: return "HS_ERR_DEVICE_FLAG";
    case HS_ERR_TIMEOUT: return "HS_ERR_TIMEOUT";
  }
  return "HS_(unknown status)";
}

const char* hs_last_error(void) { return g_last_error; }

hs_status hs_check_flag(const int32_t* err_flag, int32_t* flag_out, hs_stream_t stream) {
  REQUIRE(err_flag, "err_flag is NULL");
  int32_t h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, err_flag, sizeof h, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "reading err_flag: %s", cudaGetErrorString(e));
  if (flag_out) *flag_out = h;
  if (h == 0) return ok();
  if (h & HS_FLAG_TIMEOUT) return fail(HS_ERR_TIMEOUT, "device flag 0x%x (bounded wait ran out)", h);
  return fail(HS_ERR_DEVICE_FLAG, "device flag 0x%x", h);
}

hs_status hs_indexer_scores(const hs_indexer_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->B >= 1, "need T >= 0 and B >= 1 (T=%d, B=%d)", a->T, a->B);
  REQUIRE(a->Hi == 8 || a->Hi == 16 || a->Hi == 32 || a->Hi == 64, "Hi must be 8, 16, 32 or 64 (got %d)", a->Hi);
  REQUIRE(a->Di == 64 || a->Di == 128, "Di must be 64 or 128 (got %d)", a->Di);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->q && a->q_scale && a->weights && a->k_cache && a->k_scale && a->block_table && a->token_req &&
              a->token_kvlen && a->scores,
          "a required pointer is NULL");
  REQUIRE(aligned16(a->q) && aligned16(a->k_cache), "q and k_cache must be 16-byte aligned");
  REQUIRE(a->nblk >= 1 && a->nblk * 64 <= INT32_MAX, "nblk out of range (%lld)", (long long)a->nblk);
  REQUIRE(a->bt_stride >= 1 && a->ld >= 1, "bt_stride and ld must be >= 1");
  REQUIRE((int64_t)a->T * a->Hi <= INT32_MAX, "T * Hi too large");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  const char* why = nullptr;
  return launched(hs::launch_indexer(a, sms, false, (cudaStream_t)stream, &why), "hs_indexer_scores", why);
}

hs_status hs_topk(const float* scores, int64_t ld, const int32_t* token_kvlen, int32_t T, int32_t k, int32_t* idx,
                  int32_t* err_flag, hs_stream_t stream) {
  REQUIRE(T >= 0, "T must be >= 0");
  REQUIRE(k >= 1 && k <= 65536, "k must be in [1, 65536] (got %d)", k);
  REQUIRE(ld >= 1, "ld must be >= 1");
  REQUIRE(err_flag, "err_flag is NULL");
  if (T == 0) return ok();
  REQUIRE(scores && token_kvlen && idx, "a required pointer is NULL");
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  return launched(hs::launch_topk(scores, ld, token_kvlen, T, k, idx, err_flag, false, (cudaStream_t)stream), "hs_topk",
                  nullptr);
}

hs_status hs_indexer_topk(const hs_indexer_args* a, int32_t k, int32_t* idx, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->B >= 1, "need T >= 0 and B >= 1 (T=%d, B=%d)", a->T, a->B);
  REQUIRE(a->Hi == 8 || a->Hi == 16 || a->Hi == 32 || a->Hi == 64, "Hi must be 8, 16, 32 or 64 (got %d)", a->Hi);
  REQUIRE(a->Di == 64 || a->Di == 128, "Di must be 64 or 128 (got %d)", a->Di);
  REQUIRE(k >= 1 && k <= 65536, "k must be in [1, 65536] (got %d)", k);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->q && a->q_scale && a->weights && a->k_cache && a->k_scale && a->block_table && a->token_req &&
              a->token_kvlen && a->scores && idx,
          "a required pointer is NULL");
  REQUIRE(aligned16(a->q) && aligned16(a->k_cache), "q and k_cache must be 16-byte aligned");
  REQUIRE(a->nblk >= 1 && a->nblk * 64 <= INT32_MAX, "nblk out of range (%lld)", (long long)a->nblk);
  REQUIRE(a->bt_stride >= 1 && a->ld >= 1, "bt_stride and ld must be >= 1");
  REQUIRE((int64_t)a->T * a->Hi <= INT32_MAX, "T * Hi too large");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  const char* why = nullptr;
  st = launched(hs::launch_indexer(a, sms, true, (cudaStream_t)stream, &why), "hs_indexer_topk (indexer)", why);
  if (st != HS_OK) return st;
  return launched(hs::launch_topk(a->scores, a->ld, a->token_kvlen, a->T, k, idx, a->err_flag, true,
                                  (cudaStream_t)stream),
                  "hs_indexer_topk (top-k)", nullptr);
}

hs_status hs_sparse_mla_fwd(const hs_mla_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0, "T must be >= 0");
  REQUIRE(a->H >= 1 && a->H <= 64, "H must be in [1, 64] (got %d)", a->H);
  REQUIRE(a->k >= 1, "k must be >= 1");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->q && a->kv_pool && a->idx && a->out, "a required pointer is NULL");
  REQUIRE(aligned16(a->q) && aligned16(a->kv_pool), "q and kv_pool must be 16-byte aligned");
  REQUIRE(a->R >= 1 && a->R <= INT32_MAX, "R must be in [1, 2^31 - 1]");
  REQUIRE(!a->block_table || (a->token_req && a->bt_stride >= 1), "block_table needs token_req and bt_stride >= 1");
  REQUIRE(!a->idx_row || a->idx_rows >= 1, "idx_row needs idx_rows >= 1");
  REQUIRE(!a->token_kvlen || a->block_table, "token_kvlen needs block_table (it limits logical token indices)");
  REQUIRE((int64_t)a->T * a->H <= INT32_MAX && (int64_t)a->T * a->k <= ((int64_t)1 << 40), "T * H or T * k too large");
  REQUIRE(a->softmax_scale == a->softmax_scale, "softmax_scale is NaN");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  if (a->workspace) {
    REQUIRE(aligned16(a->workspace), "workspace must be 16-byte aligned");
    const uint64_t need = hs::mla_workspace_bytes(a->H, sms);
    REQUIRE(a->workspace_bytes >= need, "workspace holds %llu bytes; H = %d needs %llu on this device",
            (unsigned long long)a->workspace_bytes, a->H, (unsigned long long)need);
  }
  const char* why = nullptr;
  return launched(hs::launch_mla(a, sms, (cudaStream_t)stream, &why), "hs_sparse_mla_fwd", why);
}

hs_status hs_sparse_mla_workspace_size(int32_t H, uint64_t* bytes) {
  REQUIRE(bytes, "bytes is NULL");
  REQUIRE(H >= 1 && H <= 64, "H must be in [1, 64] (got %d)", H);
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  *bytes = hs::mla_workspace_bytes(H, sms);
  return ok();
}

hs_status hs_hisparse_resolve(const hs_resolve_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->B >= 0, "B must be >= 0");
  REQUIRE(a->k >= 1 && a->k <= a->S, "need 1 <= k <= S (k=%d, S=%d)", a->k, a->S);
  REQUIRE(a->S <= 8192, "S must be <= 8192 (got %d)", a->S);
  REQUIRE(a->step >= 0, "step must be >= 0");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->B == 0) return ok();
  REQUIRE(a->idx && a->seq_len && a->resident_start && a->block_table && a->host_rows && a->kv_pool && a->slot_row &&
              a->slot_token && a->slot_stamp && a->tok2slot && a->out_rows && a->counters,
          "a required pointer is NULL");
  REQUIRE(aligned16(a->kv_pool), "kv_pool must be 16-byte aligned");
  REQUIRE(a->R >= 1 && a->ld_t2s >= 1 && a->bt_stride >= 1, "R, ld_t2s and bt_stride must be >= 1");
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  return launched(hs::launch_resolve(a, (cudaStream_t)stream), "hs_hisparse_resolve", nullptr);
}

hs_status hs_kv_append(const hs_kv_append_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0, "T must be >= 0");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->B >= 1, "B must be >= 1");
  REQUIRE(a->latent || a->index_key, "nothing to append: latent and index_key are both NULL");
  REQUIRE(a->token_req && a->token_pos && a->block_table && a->bt_stride >= 1,
          "token_req, token_pos and block_table are required (bt_stride >= 1)");
  if (a->latent) {
    REQUIRE(a->rope && a->kv_pool && a->R >= 1, "latent needs rope, kv_pool and R >= 1");
    REQUIRE(aligned16(a->latent) && aligned16(a->rope) && aligned16(a->kv_pool),
            "latent, rope and kv_pool must be 16-byte aligned");
  }
  if (a->index_key) {
    REQUIRE(a->Di == 64 || a->Di == 128, "Di must be 64 or 128 (got %d)", a->Di);
    REQUIRE(a->k_cache && a->k_scale && a->nblk >= 1, "index_key needs k_cache, k_scale and nblk >= 1");
    REQUIRE(aligned16(a->index_key) && aligned16(a->k_cache), "index_key and k_cache must be 16-byte aligned");
  }
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  return launched(hs::launch_append(a, sms, (cudaStream_t)stream), "hs_kv_append", nullptr);
}

hs_status hs_kv_offload(const hs_kv_offload_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->n >= 0, "n must be >= 0");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->n == 0) return ok();
  REQUIRE(a->L >= 1 && a->B >= 1, "L and B must be >= 1");
  REQUIRE(a->pools && a->host_rows && a->layer && a->req && a->page && a->block_table && a->seq_len,
          "a required pointer is NULL");
  REQUIRE(a->bt_stride >= 1 && a->R >= 64, "bt_stride must be >= 1 and R >= 64");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  return launched(hs::launch_offload(a, sms, (cudaStream_t)stream), "hs_kv_offload", nullptr);
}

hs_status hs_hisparse_touch_host(int32_t B, const uint8_t* const* host_rows, const int32_t* seq_len,
                                 const int32_t* resident_start, int32_t* err_flag, hs_stream_t stream) {
  REQUIRE(B >= 0, "B must be >= 0");
  REQUIRE(err_flag, "err_flag is NULL");
  if (B == 0) return ok();
  REQUIRE(host_rows && seq_len && resident_start, "a required pointer is NULL");
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  const long page = sysconf(_SC_PAGESIZE);
  return launched(hs::launch_touch_host(B, host_rows, seq_len, resident_start, page > 0 ? page : 4096, err_flag,
                                        (cudaStream_t)stream),
                  "hs_hisparse_touch_host", nullptr);
}

hs_status hs_rope(const hs_rope_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->H >= 1, "need T >= 0 and H >= 1 (T=%d, H=%d)", a->T, a->H);
  REQUIRE(a->rot >= 2 && a->rot <= 512 && a->rot % 2 == 0, "rot must be even, in [2, 512] (got %d)", a->rot);
  REQUIRE(a->dtype == HS_BF16 || a->dtype == HS_FP16 || a->dtype == HS_FP32, "dtype must be HS_BF16, HS_FP16 or HS_FP32 (got %d)",
          a->dtype);
  REQUIRE(isfinite(a->scale), "scale is not finite");
  if (a->T == 0) return ok();
  REQUIRE(a->positions && a->inv_freq && a->x && a->out, "a required pointer is NULL");
  REQUIRE(a->x_stride_t >= 0 && a->x_stride_h >= 0 && a->out_stride_t >= 0 && a->out_stride_h >= 0, "strides must be >= 0");
  const uintptr_t mask = a->dtype == HS_FP32 ? 3 : 1;
  REQUIRE((((uintptr_t)a->x | (uintptr_t)a->out | (uintptr_t)a->y | (uintptr_t)a->y_out) & mask) == 0,
          "x, out, y and y_out must be aligned to their type");
  int64_t heads = a->H;
  if (a->y) {
    REQUIRE(a->y_out && a->H2 >= 1, "y needs y_out and H2 >= 1");
    REQUIRE(a->y_stride_t >= 0 && a->y_stride_h >= 0 && a->y_out_stride_t >= 0 && a->y_out_stride_h >= 0, "strides must be >= 0");
    heads += a->H2;
  }
  REQUIRE(heads * a->rot <= (1 << 26), "too many values per token");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  return launched(hs::launch_rope(a, sms, (cudaStream_t)stream), "hs_rope", nullptr);
}

hs_status hs_rope_inv_freq(int32_t rot, double base, int32_t kind, double factor, int32_t original, double beta_fast,
                           double beta_slow, double* inv_freq, float* scale) {
  REQUIRE(rot >= 2 && rot <= 512 && rot % 2 == 0, "rot must be even, in [2, 512] (got %d)", rot);
  REQUIRE(base > 1.0 && isfinite(base), "base must be finite and > 1");
  REQUIRE(kind == HS_ROPE_PLAIN || kind == HS_ROPE_LINEAR || kind == HS_ROPE_YARN, "unknown kind %d", kind);
  REQUIRE(kind == HS_ROPE_PLAIN || (factor >= 1.0 && isfinite(factor)), "factor must be finite and >= 1");
  REQUIRE(kind != HS_ROPE_YARN || (original >= 1 && beta_fast > beta_slow && beta_slow > 0.0 && isfinite(beta_fast)),
          "need original >= 1 and beta_fast > beta_slow > 0");
  REQUIRE(inv_freq && scale, "a required pointer is NULL");
  double lo = 0.0, hi = 0.0;
  if (kind == HS_ROPE_YARN) {
    // the (real-valued) index of the pair that turns beta times within `original` positions
    const double per = rot / (2.0 * log(base)), turn = 6.283185307179586476925;
    lo = fmax(floor(per * log(original / (beta_fast * turn))), 0.0);
    hi = fmin(ceil(per * log(original / (beta_slow * turn))), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot);
    double slow = kind == HS_ROPE_LINEAR ? 1.0 : 0.0;  // share of the stretched angle
    if (kind == HS_ROPE_YARN) slow = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
    inv_freq[i] = slow == 0.0 ? f : f / factor * slow + f * (1.0 - slow);
  }
  *scale = kind == HS_ROPE_YARN && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return ok();
}

hs_status hs_paged_mla_workspace_size(int32_t T, int32_t B, int32_t H, int64_t kv_tokens, uint64_t* bytes) {
  REQUIRE(bytes, "bytes is NULL");
  REQUIRE(T >= 0 && B >= 1 && B <= 4096, "need T >= 0 and B in [1, 4096] (T=%d, B=%d)", T, B);
  REQUIRE(H >= 1 && H <= 128, "H must be in [1, 128] (got %d)", H);
  REQUIRE(kv_tokens >= 0 && kv_tokens <= INT32_MAX, "kv_tokens must be in [0, 2^31 - 1]");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  *bytes = hs::paged_mla_workspace_bytes(T, B, H, kv_tokens, sms);
  return ok();
}

hs_status hs_paged_mla_fwd(const hs_paged_mla_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->B >= 1 && a->B <= 4096, "need T >= 0 and B in [1, 4096] (T=%d, B=%d)", a->T, a->B);
  REQUIRE(a->H >= 1 && a->H <= 128, "H must be in [1, 128] (got %d)", a->H);
  REQUIRE(a->kv_tokens >= 0 && a->kv_tokens <= INT32_MAX, "kv_tokens must be in [0, 2^31 - 1]");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->q && a->kv_pool && a->block_table && a->req_start && a->seq_len && a->out && a->workspace, "a required pointer is NULL");
  REQUIRE(aligned16(a->q) && aligned16(a->kv_pool) && aligned16(a->out) && aligned16(a->workspace),
          "q, kv_pool, out and workspace must be 16-byte aligned");
  REQUIRE(a->R >= 1 && a->R <= INT32_MAX, "R must be in [1, 2^31 - 1]");
  REQUIRE(a->bt_stride >= 1 && (int64_t)a->bt_stride * 64 <= INT32_MAX, "bt_stride out of range (%d)", a->bt_stride);
  REQUIRE((int64_t)a->T * a->H <= INT32_MAX - 128, "T * H too large");
  REQUIRE(isfinite(a->softmax_scale), "softmax_scale is not finite");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  const uint64_t need = hs::paged_mla_workspace_bytes(a->T, a->B, a->H, a->kv_tokens, sms);
  REQUIRE(a->workspace_bytes >= need, "workspace holds %llu bytes; these sizes need %llu on this device",
          (unsigned long long)a->workspace_bytes, (unsigned long long)need);
  const char* why = nullptr;
  return launched(hs::launch_paged_mla(a, sms, (cudaStream_t)stream, &why), "hs_paged_mla_fwd", why);
}

// The layers of a page operation: L latent pools, Li indexer caches.
#define REQUIRE_LAYERS(a)                                                                                          \
  REQUIRE((a)->L >= 0 && (a)->Li >= 0 && (a)->L + (a)->Li <= 4096, "need L, Li >= 0 and L + Li <= 4096");           \
  REQUIRE((a)->L == 0 || (a)->pools, "pools is NULL");                                                             \
  REQUIRE((a)->Li == 0 || ((a)->k_caches && (a)->k_scales), "k_caches or k_scales is NULL");                       \
  REQUIRE((a)->Li == 0 || (a)->Di == 64 || (a)->Di == 128, "Di must be 64 or 128 (got %d)", (a)->Di);              \
  REQUIRE((a)->nblk >= 1 && (a)->nblk * 64 <= INT32_MAX, "nblk out of range (%lld)", (long long)(a)->nblk)

hs_status hs_kv_copy_pages(const hs_kv_copy_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->n >= 0, "n must be >= 0");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->n == 0) return ok();
  REQUIRE(a->src && a->dst, "a required pointer is NULL");
  REQUIRE_LAYERS(a);
  if (a->L + a->Li == 0) return ok();
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  return launched(hs::launch_copy_pages(a, sms, (cudaStream_t)stream), "hs_kv_copy_pages", nullptr);
}

hs_status hs_kv_fork(const hs_kv_fork_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->n >= 0 && a->n <= 8192, "n must be in [0, 8192] (got %d)", a->n);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->n == 0) return ok();
  REQUIRE(a->parent && a->child && a->block_table && a->seq_len && a->refcount && a->src && a->dst, "a required pointer is NULL");
  REQUIRE(a->B >= 1 && a->bt_stride >= 1, "B and bt_stride must be >= 1");
  REQUIRE_LAYERS(a);
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  return launched(hs::launch_fork(a, (cudaStream_t)stream), "hs_kv_fork", nullptr);
}

hs_status hs_kv_free(const hs_kv_free_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->n >= 0, "n must be >= 0");
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->n == 0) return ok();
  REQUIRE(a->req && a->block_table && a->seq_len && a->refcount, "a required pointer is NULL");
  REQUIRE(a->B >= 1 && a->bt_stride >= 1 && a->nblk >= 1, "B, bt_stride and nblk must be >= 1");
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  return launched(hs::launch_free(a, (cudaStream_t)stream), "hs_kv_free", nullptr);
}

hs_status hs_kv_compact_workspace_size(int64_t nblk, uint64_t* bytes) {
  REQUIRE(bytes, "bytes is NULL");
  REQUIRE(nblk >= 1 && nblk * 64 <= INT32_MAX, "nblk out of range (%lld)", (long long)nblk);
  *bytes = hs::compact_workspace_bytes(nblk);
  return ok();
}

hs_status hs_kv_compact(const hs_kv_compact_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->B >= 0 && a->bt_stride >= 1, "need B >= 0 and bt_stride >= 1");
  REQUIRE(a->err_flag, "err_flag is NULL");
  REQUIRE_LAYERS(a);
  REQUIRE(a->refcount && a->refcount_out && a->src && a->dst && a->counts && a->workspace, "a required pointer is NULL");
  REQUIRE(a->B == 0 || (a->block_table && a->table_out), "block_table or table_out is NULL");
  REQUIRE(((uintptr_t)a->workspace & 3) == 0 && a->workspace_bytes >= hs::compact_workspace_bytes(a->nblk),
          "workspace must be 4-byte aligned and hold hs_kv_compact_workspace_size() bytes");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  return launched(hs::launch_compact(a, sms, (cudaStream_t)stream), "hs_kv_compact", nullptr);
}

hs_status hs_kv_read(const hs_kv_read_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->B >= 1 && a->n >= 0, "need B >= 1 and n >= 0 (B=%d, n=%lld)", a->B, (long long)a->n);
  REQUIRE(a->dtype == HS_BF16 || a->dtype == HS_FP16 || a->dtype == HS_FP32, "dtype must be HS_BF16, HS_FP16 or HS_FP32 (got %d)",
          a->dtype);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->n == 0) return ok();
  REQUIRE(a->kv_pool && a->block_table && a->out_start && a->out, "a required pointer is NULL");
  REQUIRE(a->R >= 1 && a->bt_stride >= 1, "R and bt_stride must be >= 1");
  REQUIRE(a->n <= INT32_MAX, "n must be at most 2^31 - 1");
  REQUIRE(aligned16(a->kv_pool) && aligned16(a->out), "kv_pool and out must be 16-byte aligned");
  REQUIRE(a->out_stride >= HS_D_QK && a->out_stride % (a->dtype == HS_FP32 ? 4 : 8) == 0,
          "out_stride must be >= 576 and a multiple of 16 bytes (got %lld)", (long long)a->out_stride);
  hs_status st = check_device(nullptr);
  if (st != HS_OK) return st;
  return launched(hs::launch_kv_read(a, (cudaStream_t)stream), "hs_kv_read", nullptr);
}

// Strides that TMA can step by: positive multiples of 16 bytes, below 2^40 bytes.
static bool tma_stride(int64_t values) { return values > 0 && values % 8 == 0 && values < ((int64_t)1 << 38); }
static bool head_dim(int32_t d) { return d == 64 || d == 128 || d == 192 || d == 256; }

static hs_status check_heads(const hs_mla_heads_args* a) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->H >= 1 && a->H <= 1024, "need T >= 0 and H in [1, 1024] (T=%d, H=%d)", a->T, a->H);
  REQUIRE(head_dim(a->Dn) && head_dim(a->Dv), "Dn and Dv must be 64, 128, 192 or 256 (got %d, %d)", a->Dn, a->Dv);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return HS_OK;
  REQUIRE(a->x && a->w && a->out, "a required pointer is NULL");
  REQUIRE(aligned16(a->x) && aligned16(a->w) && aligned16(a->out), "x, w and out must be 16-byte aligned");
  REQUIRE(tma_stride(a->x_stride_t) && tma_stride(a->x_stride_h) && tma_stride(a->out_stride_t) && tma_stride(a->out_stride_h),
          "strides must be positive multiples of 8");
  return HS_OK;
}

hs_status hs_mla_absorb(const hs_mla_heads_args* a, hs_stream_t stream) {
  hs_status st = check_heads(a);
  if (st != HS_OK) return st;
  if (a->T == 0) return ok();
  int sms = 0;
  st = check_device(&sms);
  if (st != HS_OK) return st;
  const char* why = nullptr;
  return launched(hs::launch_mla_absorb(a, sms, (cudaStream_t)stream, &why), "hs_mla_absorb", why);
}

hs_status hs_mla_project(const hs_mla_heads_args* a, hs_stream_t stream) {
  hs_status st = check_heads(a);
  if (st != HS_OK) return st;
  if (a->T == 0) return ok();
  int sms = 0;
  st = check_device(&sms);
  if (st != HS_OK) return st;
  const char* why = nullptr;
  return launched(hs::launch_mla_project(a, sms, (cudaStream_t)stream, &why), "hs_mla_project", why);
}

hs_status hs_mla_expand(const hs_mla_expand_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->N >= 0 && a->H >= 1 && a->H <= 1024, "need N >= 0 and H in [1, 1024] (N=%d, H=%d)", a->N, a->H);
  REQUIRE(a->width >= 64 && a->width <= 512 && a->width % 64 == 0, "width must be a multiple of 64 in [64, 512] (got %d)", a->width);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->N == 0) return ok();
  REQUIRE(a->latent && a->w && a->kv, "a required pointer is NULL");
  REQUIRE(aligned16(a->latent) && aligned16(a->w) && aligned16(a->kv), "latent, w and kv must be 16-byte aligned");
  REQUIRE(tma_stride(a->latent_stride) && tma_stride(a->kv_stride), "strides must be positive multiples of 8");
  REQUIRE(a->latent_stride >= HS_D_LATENT && a->kv_stride >= (int64_t)a->H * a->width,
          "latent_stride must be >= 512 and kv_stride >= H * width");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  const char* why = nullptr;
  return launched(hs::launch_mla_expand(a, sms, (cudaStream_t)stream, &why), "hs_mla_expand", why);
}

hs_status hs_mla_expanded_workspace_size(int32_t B, int32_t Dv, uint64_t* bytes) {
  REQUIRE(bytes, "bytes is NULL");
  REQUIRE(B >= 1 && B <= 4096, "B must be in [1, 4096] (got %d)", B);
  REQUIRE(Dv == 128 || Dv == 256, "Dv must be 128 or 256 (got %d)", Dv);
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  *bytes = hs::mla_expanded_workspace_bytes(B, Dv, sms);
  return ok();
}

hs_status hs_mla_expanded_fwd(const hs_mla_expanded_args* a, hs_stream_t stream) {
  REQUIRE(a, "args is NULL");
  REQUIRE(a->T >= 0 && a->B >= 1 && a->B <= 4096, "need T >= 0 and B in [1, 4096] (T=%d, B=%d)", a->T, a->B);
  REQUIRE(a->H >= 1 && a->H <= 1024, "H must be in [1, 1024] (got %d)", a->H);
  REQUIRE((a->Dn == 128 && a->Dv == 128) || (a->Dn == 192 && a->Dv == 256), "Dn and Dv must be 128 and 128, or 192 and 256 (got %d, %d)",
          a->Dn, a->Dv);
  REQUIRE(a->err_flag, "err_flag is NULL");
  if (a->T == 0) return ok();
  REQUIRE(a->q && a->kv && a->rope && a->req_start && a->kv_start && a->out && a->workspace, "a required pointer is NULL");
  REQUIRE(aligned16(a->q) && aligned16(a->kv) && aligned16(a->rope) && aligned16(a->out) && aligned16(a->workspace),
          "q, kv, rope, out and workspace must be 16-byte aligned");
  REQUIRE(a->N >= 1 && a->N <= INT32_MAX - 512, "N must be in [1, 2^31 - 513] (got %lld)", (long long)a->N);
  REQUIRE(tma_stride(a->q_stride_t) && tma_stride(a->q_stride_h) && tma_stride(a->kv_stride) && tma_stride(a->rope_stride),
          "strides must be positive multiples of 8");
  REQUIRE(a->kv_stride >= (int64_t)a->H * (a->Dn + a->Dv) && a->rope_stride >= HS_D_ROPE, "kv_stride or rope_stride is too small");
  REQUIRE((int64_t)a->T * a->H <= INT32_MAX - 1024 * 512, "T * H too large");
  REQUIRE(isfinite(a->softmax_scale), "softmax_scale is not finite");
  int sms = 0;
  hs_status st = check_device(&sms);
  if (st != HS_OK) return st;
  const uint64_t need = hs::mla_expanded_workspace_bytes(a->B, a->Dv, sms);
  REQUIRE(a->workspace_bytes >= need, "workspace holds %llu bytes; these sizes need %llu on this device",
          (unsigned long long)a->workspace_bytes, (unsigned long long)need);
  const char* why = nullptr;
  return launched(hs::launch_mla_expanded(a, sms, (cudaStream_t)stream, &why), "hs_mla_expanded_fwd", why);
}

}  // extern "C"
