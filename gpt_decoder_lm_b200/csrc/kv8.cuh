// The 8-bit key / value cache: what its kernels and its C entry points share.
#pragma once

#include "../../include/gpt.h"
#include "kernels.cuh"

namespace gpt {

// A block's exponent range: with e in it 2^e, 2^-e and code * 2^e are all
// normal fp32 numbers for every e4m3 code above the smallest.
constexpr int KV8_E_MIN = -110, KV8_E_MAX = 120;

// Device flag bits (gpt.h's GPT_FLAG_BLOCK_RANGE, GPT_FLAG_CACHE_FULL, GPT_FLAG_ROW_RANGE)
enum : uint32_t { FLAG_BLOCK = 1u << 4, FLAG_FULL = 1u << 5, FLAG_ROWS = 1u << 6 };

struct Kv8Args {
  int S, H, P, lgP;        // sequences, key / value heads, tokens a block (a power of two) and its logarithm
  int n_blocks, max_blocks;
  uint8_t* k;              // codes [n_blocks, H, P, hd]
  uint8_t* v;
  float* ks;               // scales [n_blocks, H]
  float* vs;
  float* w;                // accumulated weights [n_blocks, H, P] or null
  const int32_t* table;    // [S, max_blocks]
  int32_t* len;            // [S]
  uint32_t* flags;         // or null
  // the step's new tokens: rows start[s] .. start[s + 1] - 1 (start null: row s)
  const int32_t* start;
  int n_rows, max_new;
  // ... or, of a padded batch (every > 0): sequence s has the first count[s % n_count] of rows (s % n_count) every ..
  int every;
  const int32_t* count;
  int n_count;
};

#ifdef __CUDACC__
__device__ __forceinline__ void kv8_flag(const Kv8Args& a, uint32_t bit) {
  if (a.flags) atomicOr(a.flags, bit);
}

// First row and number of new tokens of sequence s; offsets that descend, leave
// [0, n_rows] or give a sequence more than max_new count as no tokens.
__device__ __forceinline__ int kv8_rows(const Kv8Args& a, int s, int* r0) {
  if (a.every) {
    int i = s;
    while (i >= a.n_count) i -= a.n_count;  // (a division would cost the other callers registers)
    *r0 = i * a.every;
    return min(max(a.count[i], 0), a.max_new);
  }
  if (!a.start) {
    *r0 = s;
    return s < a.n_rows ? 1 : 0;
  }
  const int b = a.start[s], e = a.start[s + 1];
  *r0 = b;
  if (b < 0 || e < b || e > a.n_rows || e - b > a.max_new) {
    kv8_flag(a, FLAG_ROWS);
    return 0;
  }
  return e - b;
}

// Tokens that sequence s holds, within its table's capacity.
__device__ __forceinline__ int kv8_len(const Kv8Args& a, int s) {
  const int n = a.len[s], cap = a.max_blocks << a.lgP;
  return n < 0 ? 0 : n > cap ? cap : n;
}

// Block id bi of sequence s, or -1 (flagged) where the table holds none of the pool's.
__device__ __forceinline__ int kv8_block(const Kv8Args& a, int s, int bi) {
  const int b = a.table[(size_t)s * a.max_blocks + bi];
  if ((unsigned)b < (unsigned)a.n_blocks) return b;
  kv8_flag(a, FLAG_BLOCK);
  return -1;
}

// The smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8 is e4m3's largest
// value), from the bits of amax >= 0: a mantissa above 1.75 needs one more.
__device__ __forceinline__ int kv8_exponent(uint32_t amax_bits) {
  if (amax_bits < 0x00800000u) return KV8_E_MIN;
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, KV8_E_MIN), KV8_E_MAX);
}
__device__ __forceinline__ float kv8_pow2(int e) { return __int_as_float((e + 127) << 23); }
// exponent of a stored scale (a power of two)
__device__ __forceinline__ int kv8_scale_exponent(float s) {
  return min(max((int)((__float_as_uint(s) >> 23) & 255u) - 127, KV8_E_MIN), KV8_E_MAX);
}

// Two values to two e4m3 codes (round to nearest even); lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes (the low 16 bits of x) to two fp16 values, exactly; a NaN code gives NaN.
__device__ __forceinline__ uint32_t f16x2_e4m3(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
  return r;
}
#endif

// Checks a cache (host) and fills the kernels' arguments but for the rows.
gpt_status kv8_cache_args(const gpt_kv8_cache* c, Kv8Args* a);

// dtype of q, k, v rows and outputs: bf16 or fp32
void kv8_append(Ctx& c, const Kv8Args& a, int hd, bool bf16_rows, const void* k, long k_ld, const void* v, long v_ld);
// max_len: host bound on the slots that any row sees (the split over the
// sequence goes by it).  False: the launch failed.
bool kv8_attention(Ctx& c, const Kv8Args& a, int hd, int G, bool bf16_rows, const void* q, long q_ld, float scale,
                   int max_len, void* o, long o_ld, float* lse);
bool kv8_accumulate(Ctx& c, const Kv8Args& a, int hd, int G, bool bf16_rows, const void* q, long q_ld, float scale,
                    int max_len, const float* lse);
bool kv8_evict(Ctx& c, const Kv8Args& a, int hd, const int32_t* table_out, int max_blocks_out, int budget, int recent,
               int32_t* kept);
void kv8_advance(Ctx& c, const Kv8Args& a, int max_len);

}  // namespace gpt
