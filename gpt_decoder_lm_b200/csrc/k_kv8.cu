// Filling the 8-bit key / value cache: append, the eviction's selection and
// move, and the lengths' advance.
//
// A block of P tokens of one head has one scale 2^e; a stored code c (e4m3)
// stands for c * 2^e.  With a power of two a code moves to a larger exponent
// without a second rounding (except among e4m3's subnormals), so a block that
// is filled token by token holds what a block that is filled at once holds.
#include <cooperative_groups.h>

#include <cuda_fp16.h>

#include "kv8.cuh"

namespace cg = cooperative_groups;

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
  // bits of the largest magnitude, as fp32; infinities and NaN are above the others
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
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
  __device__ __forceinline__ uint32_t top() const {
    float x[8];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
  }
};

// the largest of the block's threads' values (bits of non-negative floats)
__device__ uint32_t block_max_bits(uint32_t v) {
  __shared__ uint32_t red[16];
  v = __reduce_max_sync(0xffffffffu, v);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  for (unsigned i = 0; i < blockDim.x / 32; i++) v = max(v, red[i]);
  return v;
}

constexpr int AU = 4;  // units of 8 elements that a thread holds: 512 threads cover 128 tokens x 128

// One thread block: the new tokens that fall into one cache block, of one
// head, of K or of V (grid: touched block, 2 H, sequence).  HBM-bound: the
// rows are read once, held as they came, and quantised after the block's
// maximum is known.  B200: 6800 bf16 tokens of 25 heads of 64 in 15.5 us, 65% of
// the copy bandwidth (reads and writes do not overlap within a block), fp32 in 21.9
// us, 77%; one token for each of 12 sequences 2.7 us, a launch.
template <typename T, int HD>
__global__ void __launch_bounds__(512) k_kv8_append(Kv8Args a, const T* __restrict__ xk, long k_ld,
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
  const T* x = (is_v ? xv : xk) + (long)(r0 + lo - len) * ld + (long)h * HD;
  uint8_t* codes = (is_v ? a.v : a.k) + ((bh << a.lgP) * HD);
  float* scale = (is_v ? a.vs : a.ks) + bh;
  constexpr int UPR = HD / 8;              // units a row
  const int units = (hi - lo) * UPR, step = blockDim.x / UPR;
  x += (long)(threadIdx.x / UPR) * ld + (threadIdx.x % UPR) * 8;

  Raw8<T> raw[AU];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < AU; u++) {
    const int i = u * blockDim.x + threadIdx.x;
    if (i < units) raw[u].load(x + (long)(u * step) * ld, vec);
  }
#pragma unroll
  for (int u = 0; u < AU; u++)
    if (u * blockDim.x + threadIdx.x < units) {
      uint32_t m = raw[u].top();
      if (m >= 0x7f800000u) {  // the scale goes by the finite values
        m = 0;
        float f[8];
        raw[u].get(f);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const uint32_t x = __float_as_uint(f[j]) & 0x7fffffffu;
          m = max(m, x < 0x7f800000u ? x : 0u);
        }
      }
      top = max(top, m);
    }
  top = block_max_bits(top);
  int e = kv8_exponent(top);
  if (lo > slot0) {  // the block's earlier tokens stay: its exponent only grows
    const int e_old = kv8_scale_exponent(*scale);
    e = max(e, e_old);
    if (e > e_old) {
      const float f = kv8_pow2(max(e_old - e, -126));
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int i = threadIdx.x; i < (lo - slot0) * HD / 4; i += blockDim.x) {
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
  uint2* out = reinterpret_cast<uint2*>(codes + (size_t)(lo - slot0) * HD);
#pragma unroll
  for (int u = 0; u < AU; u++) {
    const int i = u * blockDim.x + threadIdx.x;
    if (i < units) {
      float g[8];
      raw[u].get(g);
      if (raw[u].top() >= 0x7f800000u) {  // e4m3 has no infinity: what is not finite is stored as NaN
#pragma unroll
        for (int j = 0; j < 8; j++)
          if ((__float_as_uint(g[j]) & 0x7f800000u) == 0x7f800000u) g[j] = __int_as_float(0x7fc00000);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) g[j] *= f;
      out[i] = make_uint2(e4m3x2(g[0], g[1]) | e4m3x2(g[2], g[3]) << 16, e4m3x2(g[4], g[5]) | e4m3x2(g[6], g[7]) << 16);
    }
  }
  if (a.w && !is_v)
    for (int j = lo - slot0 + threadIdx.x; j < hi - slot0; j += blockDim.x) a.w[bh * a.P + j] = 0.f;
}

// ---------------------------------------------------------------- eviction

constexpr int EBINS = 2048;     // 11-bit digits: 11 + 11 + 10
constexpr int EKEYS = 40960;    // keys that a block holds in shared memory (160 KB)

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
// written in order from counts of each warp's range.  A cluster of blocks takes
// a head, each an equal part of its slots.  Bound by barriers (B200: 768 heads of
// up to 1023 slots 13 us; 48 heads of up to 40000 slots, eight blocks each, 24 us,
// before the cluster 49 us).
template <int ET, bool SMEM>
__global__ void __launch_bounds__(ET, ET == 256 ? 6 : 3) k_kv8_select(Kv8Args a, int budget, int recent, int32_t* __restrict__ kept) {
  constexpr int EW = ET / 32;
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[EBINS];
  __shared__ __align__(16) uint32_t sums[EBINS];  // of a cluster
  __shared__ uint32_t wsum[EW], wtie[EW];
  __shared__ uint32_t pick[2];
  cg::cluster_group cl = cg::this_cluster();
  const int nb = gridDim.x, rank = blockIdx.x;
  const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int len = kv8_len(a, s);
  int32_t* out = kept + ((size_t)s * a.H + h) * budget;
  if (len <= budget) {
    for (int j = rank * ET + tid; j < budget; j += nb * ET) out[j] = j < len ? j : -1;
    return;
  }
  const int n = len - recent;           // candidates
  uint32_t need = budget - recent;      // of them to keep
  for (int j = rank * ET + tid; j < recent; j += nb * ET) out[budget - recent + j] = n + j;
  if (need == 0) return;
  const int part = (n + nb - 1) / nb, p0 = min(n, rank * part), p1 = min(n, p0 + part);  // this block's slots
  if (SMEM) {
    constexpr int U = 8;  // loads in flight
    for (int j = p0 + tid; j < p1; j += U * ET) {
      int b[U];
      float x[U];
#pragma unroll
      for (int u = 0; u < U; u++)
        b[u] = j + u * ET < p1 ? a.table[(size_t)s * a.max_blocks + ((j + u * ET) >> a.lgP)] : -1;
#pragma unroll
      for (int u = 0; u < U; u++) {
        const bool on = (unsigned)b[u] < (unsigned)a.n_blocks;
        x[u] = on ? a.w[((size_t)b[u] * a.H + h) * a.P + ((j + u * ET) & (a.P - 1))] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; u++)
        if (j + u * ET < p1) {
          const bool on = (unsigned)b[u] < (unsigned)a.n_blocks;
          if (!on) kv8_flag(a, FLAG_BLOCK);
          keys[j + u * ET - p0] = on ? weight_key(x[u]) : 0u;
        }
    }
  }
  auto key = [&](int j) -> uint32_t { return SMEM ? keys[j - p0] : slot_key(a, s, h, j); };

  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < EBINS / 4; i += ET) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int j = p0 + tid; j < p1; j += ET) {
      const uint32_t k = key(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
    }
    const uint32_t* all = hist;
    if (nb > 1) {  // a block adds its share of the bins and gives the sums to all
      cl.sync();
      const int share = EBINS / 4 / nb, at = rank * share + tid;
      if (tid < share) {
        uint4 c = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (i < nb) {
            const uint4 x = reinterpret_cast<const uint4*>(cl.map_shared_rank(hist, i))[at];
            c.x += x.x, c.y += x.y, c.z += x.z, c.w += x.w;
          }
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (i < nb) reinterpret_cast<uint4*>(cl.map_shared_rank(sums, i))[at] = c;
      }
      cl.sync();
      all = sums;
    } else {
      __syncthreads();
    }
    constexpr int BPT = EBINS / ET;  // counts from the top: thread t holds bins 2047 - BPT t and BPT - 1 below it
    uint32_t c[BPT];
#pragma unroll
    for (int i = 0; i < BPT; i += 4) {
      const uint4 x = reinterpret_cast<const uint4*>(all)[(EBINS - BPT * tid - i) / 4 - 1];
      c[i] = x.w, c[i + 1] = x.z, c[i + 2] = x.y, c[i + 3] = x.x;
    }
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < BPT; i++) own += c[i];
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    for (int i = 0; i < w; i++) incl += wsum[i];
    uint32_t before = incl - own;  // keys above this thread's bins
    if (before < need && need <= incl) {
#pragma unroll
      for (int i = 0; i < BPT; i++) {
        if (before < need && need <= before + c[i]) {
          pick[0] = EBINS - 1 - BPT * tid - i;
          pick[1] = need - before;
        }
        before += c[i];
      }
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    mask |= digit << shift;
    need = pick[1];
  }
  // every key above the threshold, and the first `need` equal to it
  const uint32_t thr = prefix;
  const int per = (part + ET - 1) / ET * 32;  // a warp's contiguous range
  const int j0 = min(p1, p0 + w * per), j1 = min(p1, j0 + per);
  uint32_t above = 0, tie = 0;
  for (int i = j0; i < j1; i += 32) {
    const int j = i + lane;
    const uint32_t k = j < j1 ? key(j) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, j < j1 && k > thr));
    tie += __popc(__ballot_sync(0xffffffffu, j < j1 && k == thr));
  }
  __syncthreads();  // wsum has been read
  if (lane == 0) wsum[w] = above, wtie[w] = tie;
  if (nb > 1) cl.sync(); else __syncthreads();
  above = tie = 0;
  for (int i = 0; i < w; i++) above += wsum[i], tie += wtie[i];
  if (nb > 1) {
    uint32_t ra = 0, rt = 0;  // of the blocks before
    for (int i = lane; i < rank * EW; i += 32) {
      ra += *cl.map_shared_rank(&wsum[i % EW], i / EW);
      rt += *cl.map_shared_rank(&wtie[i % EW], i / EW);
    }
    above += __reduce_add_sync(0xffffffffu, ra);
    tie += __reduce_add_sync(0xffffffffu, rt);
    cl.sync();  // no block leaves while another reads its shared memory
  }
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

constexpr int MT = 256;  // threads of the move

// The largest magnitude code of 16 codes, NaN (0x7f) apart.
__device__ __forceinline__ uint32_t chunk_max(const uint4& v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  // e4m3 magnitudes are ordered as integers; as 16-bit pairs the upper byte decides
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const uint32_t mag = x[j] & 0x7f7f7f7fu;
    hi = __vmaxu2(hi, mag);
    lo = __vmaxu2(lo, mag & 0x007f007fu);
  }
  lo = __vmaxu2(lo, hi >> 8 & 0x007f007fu);
  lo = max(lo & 0x7fu, lo >> 16);
  if (lo == 0x7fu) {
    lo = 0;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int b = 0; b < 32; b += 8) {
        const uint32_t m = x[j] >> b & 0x7fu;
        lo = max(lo, m == 0x7fu ? 0u : m);
      }
  }
  return lo;
}

// 16 codes times 2^k.  fp16 holds every product that does not become 0 in e4m3, which rounds it once.  A code that is
// not 0 is 2^-9 or more and its product at most 448, so that k is below 18 where there is one; zeros alone may come
// with any k (their new block goes by other values, or has none), and stay zeros with any finite factor.
__device__ __forceinline__ uint4 chunk_scale(const uint4& v, int k) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
  const __half2 f = __float2half2_rn(kv8_pow2(min(max(k, -24), 15)));
  const __half2 f2 = __float2half2_rn(kv8_pow2(min(max(k - 15, 0), 15)));
  auto two = [&](uint32_t c) -> uint32_t {
    const uint32_t u = f16x2_e4m3(c);
    __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&u), f);
    if (k > 15) h = __hmul2(h, f2);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
    return r;
  };
#pragma unroll
  for (int j = 0; j < 4; j++) x[j] = two(x[j]) | two(x[j] >> 16) << 16;
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// WPU warps: one destination block of one head, K and V.  The kept tokens'
// codes are read from their blocks, the destination's exponents are found anew
// from their values, and the codes are written at them.  Bound by the chain of
// loads (kept slot, block id, scale and codes): every thread follows it for its
// own MU chunks of K and of V.  B200: 393,600 tokens of 128 in 42 us (75% of the
// copy bandwidth), 393,200 of 64 in blocks of 16 in 23 us (66%).
template <int WPU, int MU>
__global__ void __launch_bounds__(MT) k_kv8_move(Kv8Args a, int hd, const int32_t* __restrict__ table_out,
                                                 int max_blocks_out, int budget, const int32_t* __restrict__ kept) {
  constexpr int UT = WPU * 32;  // threads of a destination block
  __shared__ uint32_t red[2][MT / 32];
  const int nblk = (budget + a.P - 1) >> a.lgP;
  const long unit = (long)blockIdx.x * (MT / UT) + threadIdx.x / UT;
  const int t = threadIdx.x % UT, w = threadIdx.x >> 5;
  const int bi = (int)(unit % nblk), h = (int)(unit / nblk % a.H), s = (int)(unit / nblk / a.H);
  int n = s < a.S ? min(a.P, min(kv8_len(a, s), budget) - (bi << a.lgP)) : 0;  // tokens
  int bo = -1;
  if (n > 0) {
    bo = table_out[(size_t)s * max_blocks_out + bi];
    if ((unsigned)bo >= (unsigned)a.n_blocks) {
      if (t == 0) kv8_flag(a, FLAG_BLOCK);
      n = 0;
    }
  }
  const int32_t* list = kept + ((size_t)s * a.H + h) * budget + ((size_t)bi << a.lgP);
  const size_t obh = (size_t)max(bo, 0) * a.H + h;
  const int lc = hd == 32 ? 1 : hd == 64 ? 2 : 3, chunks = n << lc;  // log2 of the chunks a token

  uint4 ck[MU], cv[MU];
  float sk[MU], sv[MU], wt[MU];
  int slot[MU], b[MU];
  uint32_t topk = 0, topv = 0;
#pragma unroll
  for (int u = 0; u < MU; u++) slot[u] = u * UT + t < chunks ? list[(u * UT + t) >> lc] : 0;
#pragma unroll
  for (int u = 0; u < MU; u++)
    b[u] = u * UT + t < chunks ? a.table[(size_t)s * a.max_blocks + (slot[u] >> a.lgP)] : -1;
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int ch = (u * UT + t) & ((1 << lc) - 1);
    const bool on = (unsigned)b[u] < (unsigned)a.n_blocks;
    const size_t bh = (size_t)(on ? b[u] : 0) * a.H + h, at = (bh << a.lgP) + (slot[u] & (a.P - 1));
    ck[u] = on ? *reinterpret_cast<const uint4*>(a.k + at * hd + ch * 16) : make_uint4(0, 0, 0, 0);
    cv[u] = on ? *reinterpret_cast<const uint4*>(a.v + at * hd + ch * 16) : make_uint4(0, 0, 0, 0);
    sk[u] = on ? a.ks[bh] : 1.f;
    sv[u] = on ? a.vs[bh] : 1.f;
    wt[u] = on && ch == 0 ? a.w[at] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int i = u * UT + t;
    if (i < chunks && (i & ((1 << lc) - 1)) == 0) {
      a.w[(obh << a.lgP) + (i >> lc)] = wt[u];
      if ((unsigned)b[u] >= (unsigned)a.n_blocks) kv8_flag(a, FLAG_BLOCK);
    }
  }
  auto value = [](uint32_t code, float scale) -> uint32_t {
    return __float_as_uint(__half2float(__ushort_as_half((uint16_t)f16x2_e4m3(code))) * scale) & 0x7fffffffu;
  };
#pragma unroll
  for (int u = 0; u < MU; u++)
    if (u * UT + t < chunks) {
      topk = max(topk, value(chunk_max(ck[u]), sk[u]));
      topv = max(topv, value(chunk_max(cv[u]), sv[u]));
    }
  topk = __reduce_max_sync(0xffffffffu, topk);
  topv = __reduce_max_sync(0xffffffffu, topv);
  if (WPU > 1) {
    if ((threadIdx.x & 31) == 0) red[0][w] = topk, red[1][w] = topv;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPU; i++) {
      topk = max(topk, red[0][w / WPU * WPU + i]);
      topv = max(topv, red[1][w / WPU * WPU + i]);
    }
  }
  const int ek = kv8_exponent(topk), ev = kv8_exponent(topv);
  if (t == 0 && n > 0) {
    a.ks[obh] = kv8_pow2(ek);
    a.vs[obh] = kv8_pow2(ev);
  }
  uint4* ok = reinterpret_cast<uint4*>(a.k + (obh << a.lgP) * hd);
  uint4* ov = reinterpret_cast<uint4*>(a.v + (obh << a.lgP) * hd);
#pragma unroll
  for (int u = 0; u < MU; u++) {
    const int i = u * UT + t;
    if (i < chunks) {
      const int gk = kv8_scale_exponent(sk[u]) - ek, gv = kv8_scale_exponent(sv[u]) - ev;
      ok[i] = gk ? chunk_scale(ck[u], gk) : ck[u];
      ov[i] = gv ? chunk_scale(cv[u], gv) : cv[u];
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
  const int threads = min(512, max(32, (units / AU + 31) / 32 * 32));
  const int elem = bf16_rows ? 2 : 4;
  const int vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                  k_ld * elem % 16 == 0 && v_ld * elem % 16 == 0;
  const dim3 grid(touched, 2 * a.H, a.S);
  auto run = [&](auto kernel, auto* pk, auto* pv) { kernel<<<grid, threads, 0, c.stream>>>(a, pk, k_ld, pv, v_ld, vec); };
  if (bf16_rows) {
    auto kern = hd == 32 ? k_kv8_append<bf16, 32> : hd == 64 ? k_kv8_append<bf16, 64> : k_kv8_append<bf16, 128>;
    run(kern, (const bf16*)k, (const bf16*)v);
  } else {
    auto kern = hd == 32 ? k_kv8_append<float, 32> : hd == 64 ? k_kv8_append<float, 64> : k_kv8_append<float, 128>;
    run(kern, (const float*)k, (const float*)v);
  }
}

bool kv8_evict(Ctx& c, const Kv8Args& a, int hd, const int32_t* table_out, int max_blocks_out, int budget, int recent,
               int32_t* kept) {
  {
    LaunchScope s(c, "kv8_select");
    // few long sequences: a cluster a head, each block with a few thousand slots or more
    const long cap = (long)a.max_blocks << a.lgP;
    int nb = 1;
    while (nb < 8 && cap / nb > 2048 && (long)a.S * a.H * nb < 4L * c.num_sms) nb *= 2;
    const long part = (cap + nb - 1) / nb;
    const bool fits = part <= EKEYS;
    const int threads = nb > 1 ? 512 : 256;
    auto k = nb > 1 ? (fits ? k_kv8_select<512, true> : k_kv8_select<512, false>)
                    : (fits ? k_kv8_select<256, true> : k_kv8_select<256, false>);
    if (fits && !(nb > 1 ? allow_smem<k_kv8_select<512, true>>(EKEYS * 4) : allow_smem<k_kv8_select<256, true>>(EKEYS * 4)))
      return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nb, a.H, a.S);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = fits ? (size_t)part * 4 : 0;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nb;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k, a, budget, recent, kept) != cudaSuccess) return false;
  }
  LaunchScope s(c, "kv8_move");
  const int chunks = a.P * hd / 16, wpu = chunks <= 64 ? 1 : min(chunks / 64, 8);  // 1, 2, 4 or 8
  const long units = (long)((budget + a.P - 1) / a.P) * a.H * a.S, grid = (units * wpu + MT / 32 - 1) / (MT / 32);
  auto k = wpu == 1 ? k_kv8_move<1, 2> : wpu == 2 ? k_kv8_move<2, 2> : wpu == 4 ? k_kv8_move<4, 2>
           : chunks <= 512 ? k_kv8_move<8, 2> : k_kv8_move<8, 4>;
  k<<<(unsigned)grid, MT, 0, c.stream>>>(a, hd, table_out, max_blocks_out, budget, kept);
  return true;
}

void kv8_advance(Ctx& c, const Kv8Args& a, int max_len) {
  LaunchScope s(c, "kv8_advance");
  k_kv8_advance<<<(a.S + 127) / 128, 128, 0, c.stream>>>(a, max_len);
}

}  // namespace gpt
