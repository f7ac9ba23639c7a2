// Filling the 8-bit key / value cache: append, the eviction's selection and
// move, and the lengths' advance.
//
// A block of P tokens of one head has one scale 2^e; a stored code c (e4m3)
// stands for c * 2^e.  With a power of two a code moves to a larger exponent
// without a second rounding (except among e4m3's subnormals), so a block that
// is filled token by token holds what a block that is filled at once holds.
#include "kv8.cuh"

namespace gpt {
namespace {

// ---------------------------------------------------------------- append

// Eight elements of a row as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p, bool vec) {
    if (vec) {
      a = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
      a = make_uint4(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16, u[4] | (uint32_t)u[5] << 16,
                     u[6] | (uint32_t)u[7] << 16);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool vec) {
    if (vec) {
      a = reinterpret_cast<const float4*>(p)[0];
      b = reinterpret_cast<const float4*>(p)[1];
    } else {
      a = make_float4(p[0], p[1], p[2], p[3]);
      b = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// the largest of the block's threads' values (bits of non-negative floats)
__device__ uint32_t block_max_bits(uint32_t v) {
  __shared__ uint32_t red[8];
  v = __reduce_max_sync(0xffffffffu, v);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  for (unsigned i = 0; i < blockDim.x / 32; i++) v = max(v, red[i]);
  return v;
}

constexpr int AU = 8;  // units of 8 elements that a thread holds: 256 threads cover 128 tokens x 128

// One thread block: the new tokens that fall into one cache block, of one
// head, of K or of V (grid: touched block, 2 H, sequence).  HBM-bound: the
// rows are read once, held as they came, and quantised after the block's
// maximum is known.
template <typename T>
__global__ void __launch_bounds__(256) k_kv8_append(Kv8Args a, int hd, const T* __restrict__ xk, long k_ld,
                                                    const T* __restrict__ xv, long v_ld, int vec) {
  const int s = blockIdx.z, h = blockIdx.y >> 1, is_v = blockIdx.y & 1;
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s);
  const int bi = (len >> a.lgP) + blockIdx.x, slot0 = bi << a.lgP;
  const int lo = max(len, slot0), hi = min(len + n, slot0 + a.P);
  if (n > 0 && blockIdx.x == 0 && threadIdx.x == 0 && len + n > a.max_blocks << a.lgP) kv8_flag(a, FLAG_FULL);
  if (lo >= hi || bi >= a.max_blocks) return;
  const int b = kv8_block(a, s, bi);
  if (b < 0) return;
  const size_t bh = (size_t)b * a.H + h;
  const long ld = is_v ? v_ld : k_ld;
  const T* x = (is_v ? xv : xk) + (long)(r0 + lo - len) * ld + (long)h * hd;
  uint8_t* codes = (is_v ? a.v : a.k) + bh * a.P * hd;
  float* scale = (is_v ? a.vs : a.ks) + bh;
  const int upr = hd / 8, units = (hi - lo) * upr;  // units a row, in all

  Raw8<T> raw[AU];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < AU; u++) {
    const int i = u * blockDim.x + threadIdx.x;
    if (i < units) raw[u].load(x + (long)(i / upr) * ld + (i % upr) * 8, vec);
  }
#pragma unroll
  for (int u = 0; u < AU; u++)
    if (u * blockDim.x + threadIdx.x < units) {
      float f[8];
      raw[u].get(f);
#pragma unroll
      for (int j = 0; j < 8; j++) {  // the scale goes by the finite values
        const uint32_t m = __float_as_uint(f[j]) & 0x7fffffffu;
        top = max(top, m < 0x7f800000u ? m : 0u);
      }
    }
  top = block_max_bits(top);
  int e = kv8_exponent(top);
  if (lo > slot0) {  // the block's earlier tokens stay: its exponent only grows
    const int e_old = kv8_scale_exponent(*scale);
    e = max(e, e_old);
    if (e > e_old) {
      const float f = kv8_pow2(max(e_old - e, -126));
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int i = threadIdx.x; i < (lo - slot0) * hd / 4; i += blockDim.x) {
        const uint32_t c = w[i];
        const uint32_t p = f16x2_e4m3(c), q = f16x2_e4m3(c >> 16);
        const float2 x0 = __half22float2(*reinterpret_cast<const __half2*>(&p));
        const float2 x1 = __half22float2(*reinterpret_cast<const __half2*>(&q));
        w[i] = e4m3x2(x0.x * f, x0.y * f) | e4m3x2(x1.x * f, x1.y * f) << 16;
      }
    }
    __syncthreads();  // every thread has read the old scale
  }
  if (threadIdx.x == 0) *scale = kv8_pow2(e);
  const float f = kv8_pow2(-e);
  uint2* out = reinterpret_cast<uint2*>(codes + (size_t)(lo - slot0) * hd);
#pragma unroll
  for (int u = 0; u < AU; u++) {
    const int i = u * blockDim.x + threadIdx.x;
    if (i < units) {
      float g[8];
      raw[u].get(g);
#pragma unroll
      for (int j = 0; j < 8; j++)  // e4m3 has no infinity: what is not finite is stored as NaN
        g[j] = (__float_as_uint(g[j]) & 0x7f800000u) == 0x7f800000u ? __int_as_float(0x7fc00000) : g[j] * f;
      out[i] = make_uint2(e4m3x2(g[0], g[1]) | e4m3x2(g[2], g[3]) << 16, e4m3x2(g[4], g[5]) | e4m3x2(g[6], g[7]) << 16);
    }
  }
  if (a.w && !is_v)
    for (int j = lo - slot0 + threadIdx.x; j < hi - slot0; j += blockDim.x) a.w[bh * a.P + j] = 0.f;
}

// ---------------------------------------------------------------- eviction

constexpr int ET = 1024;        // threads of the selection
constexpr int EW = ET / 32;
constexpr int EBINS = 2048;     // 11-bit digits: 11 + 11 + 10
constexpr int EKEYS = 40960;    // keys that fit in shared memory (160 KB)

// order of the accumulated weights as unsigned integers; NaN is below every number
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t slot_key(const Kv8Args& a, int s, int h, int j) {
  const int b = kv8_block(a, s, j >> a.lgP);
  return b < 0 ? 0u : weight_key(a.w[((size_t)b * a.H + h) * a.P + (j & (a.P - 1))]);
}

// The slots that head h of sequence s keeps, in order: the last `recent` and,
// of the others, the `budget - recent` heaviest (ties: the lowest slots).  The
// threshold key is found digit by digit, from the top; the kept slots are then
// written in order from counts of each warp's range.
template <bool SMEM>
__global__ void __launch_bounds__(ET) k_kv8_select(Kv8Args a, int budget, int recent, int32_t* __restrict__ kept) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[EBINS];
  __shared__ uint32_t wsum[EW], wtie[EW];
  __shared__ uint32_t pick[2];
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int len = kv8_len(a, s);
  int32_t* out = kept + ((size_t)s * a.H + h) * budget;
  if (len <= budget) {
    for (int j = tid; j < budget; j += ET) out[j] = j < len ? j : -1;
    return;
  }
  const int n = len - recent;           // candidates
  uint32_t need = budget - recent;      // of them to keep
  for (int j = tid; j < recent; j += ET) out[budget - recent + j] = n + j;
  if (need == 0) return;
  if (SMEM) {
    for (int j = tid; j < n; j += ET) keys[j] = slot_key(a, s, h, j);
    __syncthreads();
  }
  auto key = [&](int j) -> uint32_t { return SMEM ? keys[j] : slot_key(a, s, h, j); };

  uint32_t prefix = 0, mask = 0;
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < EBINS; i += ET) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += ET) {
      const uint32_t k = key(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
    }
    __syncthreads();
    // counts from the top: thread t holds bins 2047 - 2t and 2046 - 2t
    const uint32_t c0 = hist[EBINS - 1 - 2 * tid], c1 = hist[EBINS - 2 - 2 * tid];
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    uint32_t base = 0;
    for (int i = 0; i < w; i++) base += wsum[i];
    incl += base;
    const uint32_t before = incl - c0 - c1;  // keys above this thread's bins
    if (before < need && need <= incl) {
      const bool first = need <= before + c0;
      pick[0] = first ? EBINS - 1 - 2 * tid : EBINS - 2 - 2 * tid;
      pick[1] = need - before - (first ? 0 : c0);
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    mask |= digit << shift;
    need = pick[1];
    __syncthreads();
  }
  // every key above the threshold, and the first `need` equal to it
  const uint32_t thr = prefix;
  const int per = (n + EW * 32 - 1) / (EW * 32) * 32;  // a warp's contiguous range
  const int j0 = min(n, w * per), j1 = min(n, j0 + per);
  uint32_t above = 0, tie = 0;
  for (int i = j0; i < j1; i += 32) {
    const int j = i + lane;
    const uint32_t k = j < j1 ? key(j) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, j < j1 && k > thr));
    tie += __popc(__ballot_sync(0xffffffffu, j < j1 && k == thr));
  }
  if (lane == 0) wsum[w] = above, wtie[w] = tie;
  __syncthreads();
  above = tie = 0;
  for (int i = 0; i < w; i++) above += wsum[i], tie += wtie[i];
  const uint32_t lt = (1u << lane) - 1u;
  for (int i = j0; i < j1; i += 32) {
    const int j = i + lane;
    const uint32_t k = j < j1 ? key(j) : 0u;
    const uint32_t ba = __ballot_sync(0xffffffffu, j < j1 && k > thr);
    const uint32_t bt = __ballot_sync(0xffffffffu, j < j1 && k == thr);
    const uint32_t ta = above + __popc(ba & lt), tt = tie + __popc(bt & lt);
    if (j < j1 && (k > thr || (k == thr && tt < need))) out[ta + min(tt, need)] = j;
    above += __popc(ba);
    tie += __popc(bt);
  }
}

constexpr int MT = 128;  // threads of the move
constexpr int MU = 8;    // 16-byte chunks a thread holds: 128 tokens x 128 codes

// One thread block: one destination block of one head, of K or of V.  The kept
// tokens' codes are read from their blocks, the destination's exponent is found
// anew from their values, and the codes are written at it.
__global__ void __launch_bounds__(MT) k_kv8_move(Kv8Args a, int hd, const int32_t* __restrict__ table_out,
                                                 int max_blocks_out, int budget, const int32_t* __restrict__ kept) {
  const int s = blockIdx.z, h = blockIdx.y >> 1, is_v = blockIdx.y & 1, bi = blockIdx.x;
  const int m = min(kv8_len(a, s), budget), n = min(a.P, m - (bi << a.lgP));
  if (n <= 0) return;
  const int bo = table_out[(size_t)s * max_blocks_out + bi];
  if ((unsigned)bo >= (unsigned)a.n_blocks) {
    if (threadIdx.x == 0) kv8_flag(a, FLAG_BLOCK);
    return;
  }
  __shared__ size_t src[128];   // (block, head) index * P + slot of each token; ~0: none
  __shared__ float sscale[128];
  const uint8_t* codes = is_v ? a.v : a.k;
  const float* scale = is_v ? a.vs : a.ks;
  const int32_t* list = kept + ((size_t)s * a.H + h) * budget + ((size_t)bi << a.lgP);
  const size_t obh = (size_t)bo * a.H + h;
  for (int j = threadIdx.x; j < n; j += MT) {
    const int slot = list[j], b = kv8_block(a, s, slot >> a.lgP);
    const size_t at = ((size_t)b * a.H + h) * a.P + (slot & (a.P - 1));
    src[j] = b < 0 ? ~(size_t)0 : at;
    sscale[j] = b < 0 ? 1.f : scale[(size_t)b * a.H + h];
    if (!is_v) a.w[obh * a.P + j] = b < 0 ? 0.f : a.w[at];
  }
  __syncthreads();
  const int cpr = hd / 16, chunks = n * cpr;
  uint4 c[MU];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int i = u * MT + threadIdx.x;
    c[u] = make_uint4(0, 0, 0, 0);
    if (i < chunks && src[i / cpr] != ~(size_t)0)
      c[u] = *reinterpret_cast<const uint4*>(codes + src[i / cpr] * hd + (i % cpr) * 16);
  }
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int i = u * MT + threadIdx.x;
    if (i < chunks) {
      // e4m3 magnitudes are ordered as integers; NaN (0x7f) does not count
      const uint32_t x[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      uint32_t big = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t mag = x[j] & 0x7f7f7f7fu;
        const uint32_t nan = ((mag + 0x01010101u) & 0x80808080u) >> 7;  // 1 in each NaN's byte
        big = __vmaxu4(big, mag & ~(nan * 0xffu));
      }
      big = __vmaxu4(big, big >> 16);
      big = __vmaxu4(big, big >> 8) & 0x7fu;
      const uint32_t hv = f16x2_e4m3(big);
      const float val = __half2float(__ushort_as_half((uint16_t)hv)) * sscale[i / cpr];
      top = max(top, __float_as_uint(val) & 0x7fffffffu);
    }
  }
  top = block_max_bits(top);
  const int e = kv8_exponent(top);
  const float f = kv8_pow2(-e);
  if (threadIdx.x == 0) (is_v ? a.vs : a.ks)[obh] = kv8_pow2(e);
  uint8_t* out = (is_v ? a.v : a.k) + obh * a.P * hd;
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int i = u * MT + threadIdx.x;
    if (i < chunks) {
      const float g = sscale[i / cpr] * f;
      if (g != 1.f) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&c[u]);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t p = f16x2_e4m3(x[j]), q = f16x2_e4m3(x[j] >> 16);
          const float2 x0 = __half22float2(*reinterpret_cast<const __half2*>(&p));
          const float2 x1 = __half22float2(*reinterpret_cast<const __half2*>(&q));
          x[j] = e4m3x2(x0.x * g, x0.y * g) | e4m3x2(x1.x * g, x1.y * g) << 16;
        }
      }
      reinterpret_cast<uint4*>(out)[i] = c[u];
    }
  }
}

__global__ void k_kv8_advance(Kv8Args a, int max_len) {
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= a.S) return;
  int r0;
  const int n = kv8_rows(a, s, &r0);
  a.len[s] = min(kv8_len(a, s) + n, max_len);
}

}  // namespace

void kv8_append(Ctx& c, const Kv8Args& a, int hd, bool bf16_rows, const void* k, long k_ld, const void* v, long v_ld) {
  LaunchScope s(c, "kv8_append");
  const int touched = min((a.max_new + a.P - 2) / a.P + 1, a.max_blocks);
  const int units = min(a.max_new, a.P) * hd / 8;
  const int threads = min(256, max(32, (units / 4 + 31) / 32 * 32));  // about 4 units each
  const int elem = bf16_rows ? 2 : 4;
  const int vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                  k_ld * elem % 16 == 0 && v_ld * elem % 16 == 0;
  const dim3 grid(touched, 2 * a.H, a.S);
  if (bf16_rows)
    k_kv8_append<bf16><<<grid, threads, 0, c.stream>>>(a, hd, (const bf16*)k, k_ld, (const bf16*)v, v_ld, vec);
  else
    k_kv8_append<float><<<grid, threads, 0, c.stream>>>(a, hd, (const float*)k, k_ld, (const float*)v, v_ld, vec);
}

bool kv8_evict(Ctx& c, const Kv8Args& a, int hd, const int32_t* table_out, int max_blocks_out, int budget, int recent,
               int32_t* kept) {
  {
    LaunchScope s(c, "kv8_select");
    const long cap = (long)a.max_blocks << a.lgP;
    if (cap <= EKEYS) {
      if (cudaFuncSetAttribute(k_kv8_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, EKEYS * 4) != cudaSuccess)
        return false;
      k_kv8_select<true><<<dim3(a.H, a.S), ET, (size_t)cap * 4, c.stream>>>(a, budget, recent, kept);
    } else {
      k_kv8_select<false><<<dim3(a.H, a.S), ET, 0, c.stream>>>(a, budget, recent, kept);
    }
  }
  LaunchScope s(c, "kv8_move");
  k_kv8_move<<<dim3((budget + a.P - 1) / a.P, 2 * a.H, a.S), MT, 0, c.stream>>>(a, hd, table_out, max_blocks_out, budget,
                                                                               kept);
  return true;
}

void kv8_advance(Ctx& c, const Kv8Args& a, int max_len) {
  LaunchScope s(c, "kv8_advance");
  k_kv8_advance<<<(a.S + 127) / 128, 128, 0, c.stream>>>(a, max_len);
}

}  // namespace gpt
