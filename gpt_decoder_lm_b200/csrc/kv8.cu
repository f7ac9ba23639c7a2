// C entry points of the 8-bit key / value cache (include/gpt.h, gpt_kv8_*):
// argument checks, then the launches of k_kv8.cu and k_kv8_attn.cu.
#include "kv8.cuh"

gpt_status gpt::kv8_cache_args(const gpt_kv8_cache* c, gpt::Kv8Args* a) {
  if (!c || !c->d_k || !c->d_v || !c->d_k_scale || !c->d_v_scale || !c->d_table || !c->d_len) return GPT_ERR_INVALID_ARG;
  if (c->n_seq < 1 || c->n_head_kv < 1 || c->n_blocks < 1 || c->max_blocks < 1) return GPT_ERR_INVALID_ARG;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return GPT_ERR_UNSUPPORTED;
  if (c->block_tokens != 16 && c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128)
    return GPT_ERR_UNSUPPORTED;
  // grid limits, and slots counted in 32 bits
  if (c->n_seq > 65535 || c->n_head_kv > 32767 || (int64_t)c->max_blocks * c->block_tokens > (1 << 30))
    return GPT_ERR_UNSUPPORTED;
  auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  if (!aligned16(c->d_k) || !aligned16(c->d_v)) return GPT_ERR_INVALID_ARG;
  *a = gpt::Kv8Args{};
  a->S = c->n_seq;
  a->H = c->n_head_kv;
  a->P = c->block_tokens;
  a->lgP = __builtin_ctz((unsigned)c->block_tokens);
  a->n_blocks = c->n_blocks;
  a->max_blocks = c->max_blocks;
  a->k = static_cast<uint8_t*>(c->d_k);
  a->v = static_cast<uint8_t*>(c->d_v);
  a->ks = c->d_k_scale;
  a->vs = c->d_v_scale;
  a->w = c->d_weight;
  a->table = c->d_table;
  a->len = c->d_len;
  a->flags = c->d_flags;
  return GPT_OK;
}

namespace {

using namespace gpt;

// The step's rows.
gpt_status row_args(const int32_t* d_start, int32_t n_rows, int32_t max_new, Kv8Args* a) {
  if (n_rows < 1 || max_new < 1 || (!d_start && (max_new != 1 || n_rows > a->S))) return GPT_ERR_INVALID_ARG;
  a->start = d_start;
  a->n_rows = n_rows;
  a->max_new = max_new < n_rows ? max_new : n_rows;  // a bound: no sequence has more rows than there are
  if (a->max_new > (1 << 30)) return GPT_ERR_UNSUPPORTED;
  return GPT_OK;
}

// Rows of `heads` heads with pitch ld, of bf16 or fp32 elements aligned as such.
bool rows_ok(const void* p, int64_t ld, int64_t heads, int32_t hd, int32_t bf16_rows) {
  return p && ld >= heads * hd && (reinterpret_cast<uintptr_t>(p) & (bf16_rows ? 1 : 3)) == 0;
}

// Runs a launch on the current device.  A launch error of this call shows as a new last error; one that the
// caller's earlier work left behind is neither reported nor cleared.
template <typename F>
gpt_status launch(void* stream, F f) {
  Ctx c;
  c.stream = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GPT_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) c.num_sms = sms;
  const bool clean_before = cudaPeekAtLastError() == cudaSuccess;
  const bool ok = f(c);
  if (clean_before && cudaPeekAtLastError() != cudaSuccess) {
    cudaGetLastError();
    return GPT_ERR_CUDA;
  }
  return ok ? GPT_OK : GPT_ERR_CUDA;
}

int capacity(const Kv8Args& a) { return a.max_blocks << a.lgP; }

}  // namespace

extern "C" gpt_status gpt_kv8_append(const gpt_kv8_cache* cache, const int32_t* d_start, int32_t n_rows, int32_t max_new,
                                     int32_t rows_bf16, const void* d_k, int64_t k_ld, const void* d_v, int64_t v_ld,
                                     void* cuda_stream) {
  Kv8Args a;
  gpt_status st = kv8_cache_args(cache, &a);
  if (st == GPT_OK) st = row_args(d_start, n_rows, max_new, &a);
  if (st != GPT_OK) return st;
  if (!rows_ok(d_k, k_ld, a.H, cache->head_dim, rows_bf16) || !rows_ok(d_v, v_ld, a.H, cache->head_dim, rows_bf16))
    return GPT_ERR_INVALID_ARG;
  return launch(cuda_stream, [&](Ctx& c) {
    kv8_append(c, a, cache->head_dim, rows_bf16 != 0, d_k, k_ld, d_v, v_ld);
    return true;
  });
}

extern "C" gpt_status gpt_kv8_attention(const gpt_kv8_cache* cache, const int32_t* d_start, int32_t n_rows,
                                        int32_t max_new, int32_t n_head, int32_t rows_bf16, const void* d_q,
                                        int64_t q_ld, float scale, int32_t max_len, void* d_out, int64_t out_ld,
                                        float* d_lse, void* cuda_stream) {
  Kv8Args a;
  gpt_status st = kv8_cache_args(cache, &a);
  if (st == GPT_OK) st = row_args(d_start, n_rows, max_new, &a);
  if (st != GPT_OK) return st;
  if (n_head < 1 || n_head % a.H || max_len < 0 || !(scale == scale) || !rows_ok(d_q, q_ld, n_head, cache->head_dim, rows_bf16) ||
      !rows_ok(d_out, out_ld, n_head, cache->head_dim, rows_bf16))
    return GPT_ERR_INVALID_ARG;
  const int G = n_head / a.H, cap = capacity(a);
  if ((int64_t)a.max_new * G > (1 << 30)) return GPT_ERR_UNSUPPORTED;
  return launch(cuda_stream, [&](Ctx& c) {
    return kv8_attention(c, a, cache->head_dim, G, rows_bf16 != 0, d_q, q_ld, scale,
                         max_len == 0 || max_len > cap ? cap : max_len, d_out, out_ld, d_lse);
  });
}

extern "C" gpt_status gpt_kv8_accumulate(const gpt_kv8_cache* cache, const int32_t* d_start, int32_t n_rows,
                                         int32_t max_new, int32_t n_head, int32_t rows_bf16, const void* d_q,
                                         int64_t q_ld, float scale, int32_t max_len, const float* d_lse,
                                         void* cuda_stream) {
  Kv8Args a;
  gpt_status st = kv8_cache_args(cache, &a);
  if (st == GPT_OK) st = row_args(d_start, n_rows, max_new, &a);
  if (st != GPT_OK) return st;
  if (!a.w || !d_lse || n_head < 1 || n_head % a.H || max_len < 0 || !(scale == scale) ||
      !rows_ok(d_q, q_ld, n_head, cache->head_dim, rows_bf16))
    return GPT_ERR_INVALID_ARG;
  const int G = n_head / a.H, cap = capacity(a);
  if ((int64_t)a.max_new * G > (1 << 30)) return GPT_ERR_UNSUPPORTED;
  return launch(cuda_stream, [&](Ctx& c) {
    return kv8_accumulate(c, a, cache->head_dim, G, rows_bf16 != 0, d_q, q_ld, scale,
                          max_len == 0 || max_len > cap ? cap : max_len, d_lse);
  });
}

extern "C" gpt_status gpt_kv8_evict(const gpt_kv8_cache* cache, const int32_t* d_table_out, int32_t max_blocks_out,
                                    int32_t budget, int32_t recent, int32_t* d_kept, void* cuda_stream) {
  Kv8Args a;
  gpt_status st = kv8_cache_args(cache, &a);
  if (st != GPT_OK) return st;
  if (!a.w || !d_table_out || d_table_out == cache->d_table || !d_kept || budget < 1 || recent < 0 || recent > budget ||
      max_blocks_out < 1 || (int64_t)max_blocks_out * a.P < budget)
    return GPT_ERR_INVALID_ARG;
  // slots counted in 32 bits, and a grid of at most a block for each destination block and head
  if (budget > (1 << 30) || (int64_t)((budget + a.P - 1) / a.P) * a.H * a.S > 0x7fffffff) return GPT_ERR_UNSUPPORTED;
  return launch(cuda_stream, [&](Ctx& c) {
    return kv8_evict(c, a, cache->head_dim, d_table_out, max_blocks_out, budget, recent, d_kept);
  });
}

extern "C" gpt_status gpt_kv8_advance(const gpt_kv8_cache* cache, const int32_t* d_start, int32_t n_rows,
                                      int32_t max_new, int32_t max_len, void* cuda_stream) {
  Kv8Args a;
  gpt_status st = kv8_cache_args(cache, &a);
  if (st == GPT_OK && max_new > 0) st = row_args(d_start, n_rows, max_new, &a);  // max_new 0: no new tokens
  if (st != GPT_OK) return st;
  const int cap = capacity(a);
  if (max_len < 0 || max_new < 0) return GPT_ERR_INVALID_ARG;
  return launch(cuda_stream, [&](Ctx& c) {
    kv8_advance(c, a, max_len == 0 || max_len > cap ? cap : max_len);
    return true;
  });
}
