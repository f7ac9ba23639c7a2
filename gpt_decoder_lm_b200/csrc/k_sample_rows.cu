// Draws from rows of logits, each row with its own temperature, top-k, top-p
// and min-p: one cluster of thread blocks per row, each with a contiguous part
// of the row in shared memory, so that a logit is read from HBM once.
//
// A draw is a decision: a token changes as soon as a probability moves across
// a border, so probabilities are held much closer than fp32.  With
//   y = (z_max - z) log2(e) / temperature  (fp64),   w = 2^-y
// w is a fixed-point number with 44 fractional bits (relative to the largest
// token's 1), good to about 2^-34 of itself: 2^-y is a table's 2^(-j / 1024),
// j the top ten bits of y's fraction, times a cubic in the rest, which is below
// 2^-10.  Sums of such integers are exact and have no order: masses, running
// sums and their comparisons come out the same however a row is divided.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace cg = cooperative_groups;

namespace gpt {
namespace {

constexpr int NT = 512;            // threads of a block
constexpr int NWP = NT / 32;
constexpr int QW = 44;             // fractional bits of a token's weight
constexpr int SMEM_ROW = 200 << 10; // bytes of a row that a block holds

typedef unsigned long long u64;

// 2^(-j / 1024) with 48 fractional bits, by the exponential's series
struct Pow2Table {
  u64 v[1024];
  constexpr Pow2Table() : v() {
    for (int j = 0; j < 1024; j++) {
      const double x = -0.69314718055994530942 * j / 1024;
      double t = 1.0, s = 1.0;
      for (int n = 1; n < 24; n++) {
        t *= x / n;
        s += t;
      }
      v[j] = (u64)(s * 281474976710656.0 + 0.5);
    }
  }
};
__device__ const Pow2Table g_pow2;

// order-preserving image of a logit; NaN below every number
__device__ __forceinline__ uint32_t logit_key(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t KEY_NONE = 0x007fffffu;  // the key of -infinity: it and NaN are never drawn

struct RowArgs {
  const void* logits;
  long ld;
  int V;
  const float* temperature;  // null: 1
  const int32_t* top_k;      // null: off
  const float* top_p;        // null: off
  const float* min_p;        // null: off
  const float* uniform;
  int32_t* out;
  float* logp;               // or null
  int seg;                   // logits a block (a multiple of 32 * NWP)
};

// Weight of a token with distance y (log2) from the largest, 44 fractional bits.
__device__ __forceinline__ u64 weight_of(double y, const u64* tab) {
  if (!(y < 48.0)) return 0;
  const u64 b = (u64)__double_as_longlong(y + 4096.0);  // y in [0, 48) as mantissa bits: 40 of them fractional
  const uint32_t whole = (uint32_t)(b >> 40) & 0xfffu, j = (uint32_t)(b >> 30) & 1023u;
  const float r = (float)((uint32_t)b & 0x3fffffffu) * 0x1p-40f;  // below 2^-10
  // 1 - 2^-r = r ln 2 - (r ln 2)^2 / 2 + (r ln 2)^3 / 6 - ..., next term below 2^-44
  const float q = r * fmaf(r, fmaf(r, 0.0555041087f, -0.240226507f), 0.693147181f);
  const uint32_t q42 = (uint32_t)(q * 0x1p42f);
  const u64 t = tab[j];
  const u64 w48 = t - (((t >> 17) * q42) >> 25);
  const uint32_t sh = 48 - QW + whole;
  return (w48 + (1ull << (sh - 1))) >> sh;
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the block's threads and the cluster's blocks.  Slots alternate, so
// that one barrier an exchange is enough.
struct Exchange {
  u64 warp[2][NWP];
  u64 block[2];
};
template <typename CL>
__device__ u64 cluster_sum(u64 v, Exchange& x, int& turn, CL& cl, int nb) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  turn ^= 1;
  v = warp_sum_u64(v);
  if (lane == 0) x.warp[turn][w] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < NWP; i++) v += x.warp[turn][i];
  if (nb == 1) return v;
  if (threadIdx.x == 0) x.block[turn] = v;
  cl.sync();
  v = 0;
  for (int i = 0; i < nb; i++) v += *cl.map_shared_rank(&x.block[turn], i);
  return v;
}

template <typename T, bool SMEM>
__global__ void __launch_bounds__(NT) k_sample_rows(RowArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ u64 tab[1024];
  __shared__ Exchange x;
  __shared__ u64 best[2];  // the block's (key, ~index) maximum, by turns
  __shared__ u64 wmass[NWP];
  cg::cluster_group cl = cg::this_cluster();
  const int nb = gridDim.x, rank = blockIdx.x, row = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int i0 = min(a.V, rank * a.seg), n = min(a.V, i0 + a.seg) - i0;  // this block's part
  const T* g = reinterpret_cast<const T*>(a.logits) + (long)row * a.ld + i0;
  T* sm = reinterpret_cast<T*>(smem);
  int turn = 0;

  for (int i = tid; i < 1024; i += NT) tab[i] = g_pow2.v[i];
  u64 top = 0;
  for (int i = tid; i < n; i += NT) {
    const T v = g[i];
    if (SMEM) sm[i] = v;
    const u64 k = (u64)logit_key(to_f<T>(v)) << 32 | (uint32_t)~(i0 + i);  // ties: the lowest index
    top = max(top, k);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) wmass[w] = top;
  __syncthreads();
  top = wmass[0];
  for (int i = 1; i < NWP; i++) top = max(top, wmass[i]);
  if (nb > 1) {
    if (tid == 0) best[0] = top;
    cl.sync();
    for (int i = 0; i < nb; i++) top = max(top, *cl.map_shared_rank(&best[0], i));
  }
  auto at = [&](int i) -> float { return to_f<T>(SMEM ? sm[i] : g[i]); };

  const float temp = a.temperature ? a.temperature[row] : 1.f;
  const uint32_t top_key = (uint32_t)(top >> 32);
  const int top_idx = (int)~(uint32_t)top;
  if (top_key <= KEY_NONE || !(temp > 0.f)) {
    // nothing to draw from, or greedy
    if (rank == 0 && tid == 0) {
      a.out[row] = top_key <= KEY_NONE ? -1 : top_idx;
      if (a.logp) a.logp[row] = top_key <= KEY_NONE ? -INFINITY : 0.f;
    }
    if (nb > 1) cl.sync();  // no block leaves while another reads its shared memory
    return;
  }
  const float zf = __uint_as_float((top_key & 0x80000000u) ? (top_key & 0x7fffffffu) : ~top_key);
  const double zmax = (double)zf, c = 1.4426950408889634074 / (double)temp;
  auto dist = [&](float z) -> double { return z == zf ? 0.0 : (zmax - (double)z) * c; };

  // ---- the lowest key that is kept
  uint32_t thr = KEY_NONE + 1;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < a.V) {
    // the largest key that at least k tokens reach, bit by bit
    uint32_t cur = 0;
    for (int bit = 31; bit >= 0; bit--) {
      const uint32_t cand = cur | 1u << bit;
      uint32_t cnt = 0;
      for (int i = tid; i < n; i += NT) cnt += logit_key(at(i)) >= cand;
      if (cluster_sum(cnt, x, turn, cl, nb) >= (u64)k) cur = cand;
    }
    thr = max(thr, cur);
  }
  auto weight = [&](float z) -> u64 { return logit_key(z) >= thr ? weight_of(dist(z), tab) : 0ull; };
  const float tp = a.top_p ? a.top_p[row] : 1.f;
  if (tp < 1.f) {
    u64 m = 0;
    for (int i = tid; i < n; i += NT) m += weight(at(i));
    m = cluster_sum(m, x, turn, cl, nb);
    const double target = fmax((double)tp, 0.0) * (double)m;
    // the largest key whose tokens and those above it hold the target (and something)
    uint32_t cur = 0;
    for (int bit = 31; bit >= 0; bit--) {
      const uint32_t cand = cur | 1u << bit;
      u64 s = 0;
      for (int i = tid; i < n; i += NT) {
        const float z = at(i);
        if (logit_key(z) >= cand) s += weight(z);
      }
      s = cluster_sum(s, x, turn, cl, nb);
      if (s > 0 && (double)s >= target) cur = cand;
    }
    thr = max(thr, cur);
  }
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const u64 least = mp > 0.f ? (u64)ceil(fmin((double)mp, 1.0) * (double)(1ull << QW)) : 0ull;
  auto kept = [&](float z) -> u64 {
    const u64 v = weight(z);
    return v >= least ? v : 0ull;
  };

  // ---- the draw: the first token whose running kept mass exceeds u times the whole
  const int per = a.seg / NWP, j0 = min(n, w * per), j1 = min(n, j0 + per);
  u64 m = 0;
  for (int i = j0 + lane; i < j1; i += 32) m += kept(at(i));
  m = warp_sum_u64(m);
  __syncthreads();
  if (lane == 0) wmass[w] = m;
  const u64 mass = cluster_sum(lane == 0 ? m : 0ull, x, turn, cl, nb);
  u64 before = 0;
  for (int i = 0; i < rank; i++) before += *cl.map_shared_rank(&x.block[turn], i);
  for (int i = 0; i < w; i++) before += wmass[i];
  const float u = a.uniform[row];
  u64 target = u > 0.f ? (u64)((double)u * (double)mass) : 0ull;
  target = min(target, mass - 1);
  if (before <= target && target < before + m) {
    for (int i = j0; i < j1; i += 32) {
      const u64 v = i + lane < j1 ? kept(at(i + lane)) : 0ull;
      u64 run = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + run > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          a.out[row] = i0 + i + lane;
          if (a.logp)
            a.logp[row] = (float)(-0.69314718055994530942 * dist(at(i + lane)) -
                                  log((double)mass / (double)(1ull << QW)));
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
  }
  if (nb > 1) cl.sync();
}

template <typename T>
bool launch(Ctx& c, RowArgs a, int rows) {
  // a cluster a row: more blocks while the rows leave SMs idle, or while a block's part does not fit
  int nb = 1;
  auto bytes = [&](int b) {
    const long part = (a.V + b - 1) / b;
    return (part + 32 * NWP - 1) / (32 * NWP) * (32 * NWP) * (long)sizeof(T);
  };
  while (nb < 8 && ((long)rows * nb * 2 <= c.num_sms || bytes(nb) > SMEM_ROW)) nb *= 2;
  a.seg = (int)(bytes(nb) / (long)sizeof(T));
  const bool fits = bytes(nb) <= SMEM_ROW;
  auto k = fits ? k_sample_rows<T, true> : k_sample_rows<T, false>;
  const size_t smem = fits ? (size_t)bytes(nb) : 0;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ROW) != cudaSuccess) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nb, rows);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nb;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a) == cudaSuccess;
}

}  // namespace

bool sample_rows_each(Ctx& c, const void* logits, bool bf16_logits, int rows, int V, long ld, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, const float* uniform, int32_t* out,
                      float* logp) {
  LaunchScope s(c, "sample_rows");
  const RowArgs a{logits, ld, V, temperature, top_k, top_p, min_p, uniform, out, logp, 0};
  return bf16_logits ? launch<bf16>(c, a, rows) : launch<float>(c, a, rows);
}

}  // namespace gpt
