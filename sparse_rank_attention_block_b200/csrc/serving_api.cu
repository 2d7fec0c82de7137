// Host side of the serving operators' C entry points (include/sda.h): argument
// checks, workspace layout, launches. No device memory is allocated here.

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "../../include/sda.h"
#include "kernels.h"
#include "serving.h"

namespace {

using sda::Cache;
using sda::CacheLayout;
using sda::Prompt;

int32_t fail(int32_t code, const char* msg) { return sda::set_error(code, msg); }
template <class... A>
int32_t fail(int32_t code, const char* fmt, A... a) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a...);
  return sda::set_error(code, buf);
}

#define SDA_TRY(x)                 \
  do {                             \
    const int32_t rc_ = (x);       \
    if (rc_ != SDA_OK) return rc_; \
  } while (0)

constexpr int kMaxSequences = 65535;

int32_t check_heads(int32_t H, int32_t H_kv, int32_t d) {
  if (H < 1 || H_kv < 1 || H % H_kv != 0) return fail(SDA_ERR_SHAPE, "H_kv (%d) must divide H (%d), both >= 1", H_kv, H);
  if (H > 1024) return fail(SDA_ERR_UNSUPPORTED, "H = %d exceeds 1024", H);
  if (d != 64 && d != 128) return fail(SDA_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d);
  return SDA_OK;
}

// Distance between rows: 0 stands for dense. The largest byte offset must fit the 40 bits of a tensor map's stride.
int32_t check_ld(const char* name, int64_t ld, int32_t heads, int32_t d, long long* out) {
  const int64_t dense = static_cast<int64_t>(heads) * d;
  if (ld == 0) ld = dense;
  if (ld < dense) return fail(SDA_ERR_SHAPE, "%s (%lld) is below heads * d (%lld)", name, (long long)ld, (long long)dense);
  if (ld % 8 != 0) return fail(SDA_ERR_ALIGN, "%s (%lld) must be a multiple of 8", name, (long long)ld);
  if (ld >= (int64_t(1) << 32)) return fail(SDA_ERR_UNSUPPORTED, "%s (%lld) is too large", name, (long long)ld);
  *out = ld;
  return SDA_OK;
}

int32_t check_scale(double scale, int32_t d, float* scale_log2) {
  if (!(scale >= 0.0) || !std::isfinite(scale)) return fail(SDA_ERR_SHAPE, "scale must be finite and >= 0");
  const double s = scale == 0.0 ? 1.0 / std::sqrt(static_cast<double>(d)) : scale;
  *scale_log2 = static_cast<float>(s * 1.4426950408889634);
  if (!(*scale_log2 > 0.f) || !std::isfinite(*scale_log2)) return fail(SDA_ERR_SHAPE, "scale is out of fp32's range");
  return SDA_OK;
}

int32_t check_ptr(const void* p, const char* name) {
  if (p == nullptr) return fail(SDA_ERR_NULLPTR, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return fail(SDA_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return SDA_OK;
}

int32_t check_ws(size_t need, void* ws, size_t ws_bytes) {
  if (ws == nullptr) return fail(SDA_ERR_NULLPTR, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(SDA_ERR_ALIGN, "workspace is not 256-byte aligned");
  if (ws_bytes < need) return fail(SDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  return SDA_OK;
}

int32_t launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(SDA_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
  return SDA_OK;
}

int32_t make_prompt(const sda_prompt_params* p, Prompt* P) {
  if (p == nullptr) return fail(SDA_ERR_NULLPTR, "params is NULL");
  if (p->n_seq < 1 || p->n_seq > kMaxSequences) return fail(SDA_ERR_SHAPE, "n_seq must be 1..%d (got %d)", kMaxSequences, p->n_seq);
  if (p->rows_q < 1 || p->rows_k < 1) return fail(SDA_ERR_SHAPE, "rows_q and rows_k must be >= 1");
  SDA_TRY(check_heads(p->H, p->H_kv, p->d));
  if (p->causal != 0 && p->causal != 1) return fail(SDA_ERR_SHAPE, "causal must be 0 or 1");
  std::memset(P, 0, sizeof(*P));
  SDA_TRY(check_ld("ld_q", p->ld_q, p->H, p->d, &P->ld_q));
  SDA_TRY(check_ld("ld_k", p->ld_k, p->H_kv, p->d, &P->ld_k));
  SDA_TRY(check_ld("ld_v", p->ld_v, p->H_kv, p->d, &P->ld_v));
  SDA_TRY(check_ld("ld_o", p->ld_o, p->H, p->d, &P->ld_o));
  SDA_TRY(check_scale(p->scale, p->d, &P->scale_log2));
  if (static_cast<int64_t>(p->rows_q / 128 + p->n_seq) * p->H >= (int64_t(1) << 31) || p->rows_q > (1 << 30) ||
      p->rows_k > (1 << 30))
    return fail(SDA_ERR_UNSUPPORTED, "too many rows for one launch");
  P->n_seq = p->n_seq;
  P->rows_q = p->rows_q;
  P->rows_k = p->rows_k;
  P->H = p->H;
  P->H_kv = p->H_kv;
  P->d = p->d;
  P->causal = p->causal;
  return SDA_OK;
}

int32_t make_cache(const sda_cache_params* p, Cache* C) {
  if (p == nullptr) return fail(SDA_ERR_NULLPTR, "params is NULL");
  if (p->B < 1 || p->B > kMaxSequences) return fail(SDA_ERR_SHAPE, "B must be 1..%d (got %d)", kMaxSequences, p->B);
  SDA_TRY(check_heads(p->H, p->H_kv, p->d));
  if (p->block != 16 && p->block != 32 && p->block != 64 && p->block != 128)
    return fail(SDA_ERR_UNSUPPORTED, "block must be 16, 32, 64 or 128 (got %d)", p->block);
  if (p->n_blocks < 1 || p->max_blocks < 1) return fail(SDA_ERR_SHAPE, "n_blocks and max_blocks must be >= 1");
  if (p->rows < 0 || p->max_new < 0) return fail(SDA_ERR_SHAPE, "rows and max_new must be >= 0");
  if (p->weights != 0 && p->weights != 1) return fail(SDA_ERR_SHAPE, "weights must be 0 or 1");
  if (p->keep < 0 || p->recent < 0 || p->recent > p->keep)
    return fail(SDA_ERR_SHAPE, "0 <= recent (%d) <= keep (%d) must hold", p->recent, p->keep);
  std::memset(C, 0, sizeof(*C));
  SDA_TRY(check_ld("ld_q", p->ld_q, p->H, p->d, &C->ld_q));
  SDA_TRY(check_ld("ld_k", p->ld_k, p->H_kv, p->d, &C->ld_k));
  SDA_TRY(check_ld("ld_v", p->ld_v, p->H_kv, p->d, &C->ld_v));
  SDA_TRY(check_ld("ld_o", p->ld_o, p->H, p->d, &C->ld_o));
  SDA_TRY(check_scale(p->scale, p->d, &C->scale_log2));
  const int64_t tokens = static_cast<int64_t>(p->max_blocks) * p->block;
  if (static_cast<int64_t>(p->n_blocks) * p->H_kv * p->block >= (int64_t(1) << 31) || tokens > (1 << 24) ||
      static_cast<int64_t>(p->B) * p->max_blocks >= (int64_t(1) << 31) || p->keep > (1 << 24) || p->max_new > (1 << 20))
    return fail(SDA_ERR_UNSUPPORTED, "the cache is too large (n_blocks * H_kv * block rows, tokens of a sequence, keep or max_new)");
  C->B = p->B;
  C->H = p->H;
  C->H_kv = p->H_kv;
  C->g = p->H / p->H_kv;
  C->d = p->d;
  C->block = p->block;
  C->n_blocks = p->n_blocks;
  C->max_blocks = p->max_blocks;
  C->rows = p->rows;
  C->max_new = p->max_new;
  C->weights = p->weights;
  C->keep = p->keep;
  C->recent = p->recent;
  C->dst_blocks = (p->keep + p->block - 1) / p->block;
  return SDA_OK;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + off);
}

int32_t check_pool(const int32_t* lens, const int32_t* table, const uint8_t* k_codes, const uint8_t* v_codes,
                   const float* k_scale, const float* v_scale) {
  SDA_TRY(check_ptr(lens, "lens"));
  SDA_TRY(check_ptr(table, "block_table"));
  SDA_TRY(check_ptr(k_codes, "k_codes"));
  SDA_TRY(check_ptr(v_codes, "v_codes"));
  SDA_TRY(check_ptr(k_scale, "k_scale"));
  return check_ptr(v_scale, "v_scale");
}

// Eviction's scratch behind the status word: the row of the pool that each target comes from.
size_t evict_rows_bytes(const Cache& C) { return static_cast<size_t>(C.B) * C.H_kv * C.keep * 4; }

int32_t need_rows(const Cache& C) {
  if (C.rows < 1 || C.max_new < 1) return fail(SDA_ERR_SHAPE, "rows and max_new must be >= 1 for this call");
  return SDA_OK;
}

std::atomic<uint64_t> g_wait_limit_ns{2000000000ull};  // 2 s: far beyond any legitimate wait

}  // namespace

namespace sda {
uint64_t serving_wait_limit() { return g_wait_limit_ns.load(); }
void set_serving_wait_limit(uint64_t limit_ns) { g_wait_limit_ns.store(limit_ns); }
}  // namespace sda

extern "C" {

size_t sda_prompt_workspace_size(const sda_prompt_params* p) {
  Prompt P;
  if (make_prompt(p, &P) != SDA_OK) return 0;
  return 256;  // the status word
}

int32_t sda_prompt_attn_fwd(const sda_prompt_params* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                            const int32_t* seq_q, const int32_t* seq_k, uint16_t* o, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  Prompt P;
  SDA_TRY(make_prompt(p, &P));
  SDA_TRY(check_ws(256, ws, ws_bytes));
  SDA_TRY(check_ptr(q, "q"));
  SDA_TRY(check_ptr(k, "k"));
  SDA_TRY(check_ptr(v, "v"));
  SDA_TRY(check_ptr(seq_q, "seq_q"));
  SDA_TRY(check_ptr(seq_k, "seq_k"));
  SDA_TRY(check_ptr(o, "o"));
  if (lse != nullptr) SDA_TRY(check_ptr(lse, "lse"));
  SDA_TRY(sda::require_device());
  return launched(sda::launch_prompt_attn(P, q, k, v, seq_q, seq_k, o, lse, at<unsigned>(ws, 0),
                                          static_cast<cudaStream_t>(stream)),
                  "prompt attention");
}

size_t sda_cache_workspace_size(const sda_cache_params* p) {
  Cache C;
  if (make_cache(p, &C) != SDA_OK) return 0;
  const size_t attn = C.max_new > 0 ? sda::make_cache_layout(C).total : 256, evict = 256 + evict_rows_bytes(C);
  return attn > evict ? attn : evict;
}

int32_t sda_cache_append(const sda_cache_params* p, const uint16_t* k, const uint16_t* v, const int32_t* seq,
                         const int32_t* lens, const int32_t* block_table, uint8_t* k_codes, uint8_t* v_codes,
                         float* k_scale, float* v_scale, float* w, void* ws, size_t ws_bytes, void* stream) {
  Cache C;
  SDA_TRY(make_cache(p, &C));
  SDA_TRY(need_rows(C));
  SDA_TRY(check_ws(256, ws, ws_bytes));
  SDA_TRY(check_ptr(k, "k"));
  SDA_TRY(check_ptr(v, "v"));
  SDA_TRY(check_ptr(seq, "seq"));
  SDA_TRY(check_pool(lens, block_table, k_codes, v_codes, k_scale, v_scale));
  if (w != nullptr) SDA_TRY(check_ptr(w, "w"));
  SDA_TRY(sda::require_device());
  return launched(sda::launch_cache_append(C, k, v, seq, lens, block_table, k_codes, v_codes, k_scale, v_scale, w,
                                           at<unsigned>(ws, 0), static_cast<cudaStream_t>(stream)),
                  "cache append");
}

int32_t sda_cache_attn_fwd(const sda_cache_params* p, const uint16_t* q, const int32_t* seq, const int32_t* lens,
                           const int32_t* block_table, const uint8_t* k_codes, const uint8_t* v_codes,
                           const float* k_scale, const float* v_scale, const float* w_in, float* w_out,
                           uint16_t* o, void* ws, size_t ws_bytes, void* stream) {
  Cache C;
  SDA_TRY(make_cache(p, &C));
  SDA_TRY(need_rows(C));
  const CacheLayout y = sda::make_cache_layout(C);
  if (y.join_ctas >= (1ll << 31) || y.line_places >= (1ll << 31) - (1 << 20))
    return fail(SDA_ERR_UNSUPPORTED, "too much work for one launch (B * H * max_new rows over max_blocks * block tokens)");
  SDA_TRY(check_ws(y.total, ws, ws_bytes));
  SDA_TRY(check_ptr(q, "q"));
  SDA_TRY(check_ptr(seq, "seq"));
  SDA_TRY(check_pool(lens, block_table, k_codes, v_codes, k_scale, v_scale));
  SDA_TRY(check_ptr(o, "o"));
  if (w_out != nullptr) {
    if (C.weights == 0) return fail(SDA_ERR_SHAPE, "w_out is given, but weights is 0 in the parameters");
    SDA_TRY(check_ptr(w_out, "w_out"));
  }
  if (w_in != nullptr) {
    if (w_out == nullptr) return fail(SDA_ERR_NULLPTR, "w_in is given without w_out");
    SDA_TRY(check_ptr(w_in, "w_in"));
  }
  SDA_TRY(sda::require_device());
  return launched(sda::launch_cache_attn(C, y, ws, q, seq, lens, block_table, k_codes, v_codes, k_scale, v_scale, w_in,
                                         w_out, o, static_cast<cudaStream_t>(stream)),
                  "cache attention");
}

int32_t sda_cache_evict(const sda_cache_params* p, const int32_t* lens, const int32_t* block_table, uint8_t* k_codes,
                        uint8_t* v_codes, float* k_scale, float* v_scale, float* w, const int32_t* dst_table,
                        int32_t* kept, int32_t* dst_lens, void* ws, size_t ws_bytes, void* stream) {
  Cache C;
  SDA_TRY(make_cache(p, &C));
  if (C.keep < 1) return fail(SDA_ERR_SHAPE, "keep must be >= 1 for this call");
  SDA_TRY(check_ws(256 + evict_rows_bytes(C), ws, ws_bytes));
  SDA_TRY(check_pool(lens, block_table, k_codes, v_codes, k_scale, v_scale));
  SDA_TRY(check_ptr(w, "w"));
  SDA_TRY(check_ptr(dst_table, "dst_table"));
  SDA_TRY(check_ptr(kept, "kept"));
  SDA_TRY(check_ptr(dst_lens, "dst_lens"));
  SDA_TRY(sda::require_device());
  return launched(sda::launch_cache_evict(C, lens, block_table, k_codes, v_codes, k_scale, v_scale, w, dst_table, kept,
                                          dst_lens, at<int32_t>(ws, 256), at<unsigned>(ws, 0), static_cast<cudaStream_t>(stream)),
                  "cache eviction");
}

}  // extern "C"
