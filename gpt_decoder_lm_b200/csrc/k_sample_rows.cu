// Draws from rows of logits, each row with its own temperature, top-k, top-p
// and min-p: one cluster of thread blocks per row, each with a contiguous part
// of the row in shared memory, so that a logit is read from HBM once.
//
// A draw is a decision: a token changes as soon as a probability moves across
// a border, so probabilities are held much closer than fp32.  With
//   y = (z_max - z) log2(e) / temperature,   w = 2^-y   (fp64, good to 2^-38)
// a token's weight w is rounded to a whole number of 2^-44 (the largest token
// has 1).  Sums of such integers are exact and have no order: masses, running
// sums and their comparisons come out the same however a row is divided.
//
// A threshold (the k-th largest logit, the nucleus' border) is found from a
// histogram over y, 32 bins an octave, in fp32: counts say exactly which bin
// holds the k-th largest; masses, held to 2^-14, leave a bin or two for the
// nucleus.  Only the tokens of those bins, a few hundred, are then listed and
// searched bit by bit, with exact counts or masses.  Rows whose tokens crowd
// into a bin are searched in place.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace cg = cooperative_groups;

namespace gpt {
namespace {

constexpr int NT = 512;            // threads of a block
constexpr int NWP = NT / 32;
constexpr int QW = 44;             // fractional bits of a token's weight
constexpr int SMEM_ROW = 200 << 10; // bytes of a row that a block holds
constexpr int NBIN = 1536;         // 48 octaves: a token below 2^-48 of the largest has no weight
constexpr int CW = 80;             // tokens that a warp lists
constexpr int GATHER = 4 * NT;     // listed tokens of a whole row: 4 a thread
constexpr int SMEM_HEAD = (GATHER + NWP * CW) * 4;  // histogram (later the row's list), the warps' lists
// Two blocks of 50,257 bf16 logits fit on an SM with these.
static_assert(NBIN <= GATHER && NBIN == 3 * NT, "a thread has three bins");

typedef unsigned long long u64;

// order-preserving image of a logit that is not NaN, and back
__device__ __forceinline__ uint32_t logit_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

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
  int seg;                   // logits a block
};

// The row's scale: distances from its largest logit, in log2 of probability.
struct Scale {
  float zf, cf;   // the largest logit; log2(e) / temperature
  double zd, cd;
  __device__ __forceinline__ double dist(float z) const { return z == zf ? 0.0 : (zd - (double)z) * cd; }
  // rint(32 y) in fp32; both roundings keep the order of logits.  NBIN or more: no weight.  *fr: 32 y - bin
  __device__ __forceinline__ int bin(float z, float* fr = nullptr) const {
    const float d = fmaxf(zf - z, 0.f);  // 0 for inf - inf
    const float t = fmaf(d, cf, 12582912.f);
    if (fr) *fr = fmaf(d, cf, -(t - 12582912.f));
    return __float_as_int(t) - 0x4b400000;
  }
  // The weight, 44 fractional bits, of a token in a bin below NBIN.  2^-y = 2^-n (1 + f P(f)), |f| <= 1/2, with P the
  // polynomial that meets (2^-f - 1) / f at the eight Chebyshev nodes (relative error 2^-38.7; f = 0 gives 1).
  __device__ __forceinline__ u64 weight(float z) const {
    const double d = z == zf ? 0.0 : zd - (double)z;
    const double t = fma(d, cd, 6755399441055744.0);
    const double f = fma(d, cd, -(t - 6755399441055744.0));
    double p = 1.325080551750225e-06;
    p = fma(p, f, -1.5303700711365693e-05);
    p = fma(p, f, 0.00015403475186530786);
    p = fma(p, f, -0.0013333478473685416);
    p = fma(p, f, 0.00961812913523614);
    p = fma(p, f, -0.055504109063258665);
    p = fma(p, f, 0.24022650695888503);
    p = fma(p, f, -0.6931471805568324);
    p = fma(p, f, 1.0);
    const double scale = __hiloint2double((1023 + QW - __double2loint(t)) << 20, 0);
    // adding 2^52 leaves the product, rounded, in the mantissa
    return (u64)__double_as_longlong(fma(p, scale, 4503599627370496.0)) & 0xfffffffffffffull;
  }
};

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Reductions over the block's threads and the cluster's blocks.  Slots
// alternate, so that one barrier an exchange is enough.
struct Exchange {
  u64 warp[2][NWP];
  u64 block[2];
};
struct Group {
  cg::cluster_group cl;
  Exchange& x;
  int nb, turn;
  __device__ __forceinline__ void sync() {
    if (nb > 1) cl.sync(); else __syncthreads();
  }
  // over the first `blocks` blocks (1: this one alone)
  template <bool MAX>
  __device__ u64 reduce(u64 v, int blocks) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    turn ^= 1;
    if (MAX) {
      v = __reduce_max_sync(0xffffffffu, (uint32_t)v);
    } else {
      v = warp_sum_u64(v);
    }
    if (lane == 0) x.warp[turn][w] = v;
    __syncthreads();
    v = x.warp[turn][0];
#pragma unroll
    for (int i = 1; i < NWP; i++) v = MAX ? max(v, x.warp[turn][i]) : v + x.warp[turn][i];
    if (blocks == 1) return v;
    if (threadIdx.x == 0) x.block[turn] = v;
    cl.sync();
    v = *cl.map_shared_rank(&x.block[turn], 0);
    for (int i = 1; i < blocks; i++) {
      const u64 o = *cl.map_shared_rank(&x.block[turn], i);
      v = MAX ? max(v, o) : v + o;
    }
    return v;
  }
  __device__ u64 sum(u64 v) { return reduce<false>(v, nb); }
  __device__ uint32_t top(uint32_t v) { return (uint32_t)reduce<true>(v, nb); }
};

// A block's part of a row.  Position p holds logit p - mis: with mis the offset
// of the first logit from a 16-byte boundary, vectors of positions are aligned
// in memory and in shared memory; positions outside the part read as -infinity,
// and so does NaN.
template <typename T, bool SMEM>
struct Part {
  static constexpr int VEC = 16 / sizeof(T);
  const T* g;
  T* sm;
  int mis, n;

  static __device__ __forceinline__ float clean(float f) { return f != f ? -INFINITY : f; }
  __device__ __forceinline__ float at(int p) const {
    if (SMEM) return to_f<T>(sm[p]);
    return p >= mis && p < mis + n ? clean(to_f<T>(g[p - mis])) : -INFINITY;
  }
  static __device__ __forceinline__ void split(const uint4& v, float (&z)[VEC]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (sizeof(T) == 2) {
        z[(2 * i) % VEC] = __uint_as_float(w[i] << 16);
        z[(2 * i + 1) % VEC] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        z[i] = __uint_as_float(w[i]);
      }
    }
  }
  // f(logit, position) over positions [j0, j1), multiples of VEC; every lane of a warp runs every step
  template <typename F>
  __device__ __forceinline__ void each(int j0, int j1, F f) const {
    for (int base = j0; base < j1; base += 32 * VEC) {
      const int p = base + (threadIdx.x & 31) * VEC;
      float z[VEC];
      if (SMEM) {
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        split(p < j1 ? *reinterpret_cast<const uint4*>(sm + p) : make_uint4(none, none, none, none), z);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j++) z[j] = p < j1 ? at(p + j) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < VEC; j++) f(z[j], p + j);
    }
  }
  // Brings the part into shared memory; the thread's largest logit.
  __device__ __forceinline__ float load(int positions) const {
    float top = -INFINITY;
    if (!SMEM) {
      for (int p = mis + threadIdx.x; p < mis + n; p += NT) top = fmaxf(top, at(p));
      return top;
    }
    constexpr int U = 4;  // vectors in flight
    for (int v0 = threadIdx.x * VEC; v0 < positions; v0 += U * NT * VEC) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int p = v0 + u * NT * VEC;
        if (p >= mis && p + VEC <= mis + n) raw[u] = *reinterpret_cast<const uint4*>(g + (p - mis));
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int p = v0 + u * NT * VEC;
        if (p >= positions) continue;
        bool whole = p >= mis && p + VEC <= mis + n;
        if (whole) {
          float z[VEC];
          split(raw[u], z);
#pragma unroll
          for (int j = 0; j < VEC; j++) {
            top = fmaxf(top, z[j]);  // ignores NaN
            whole &= z[j] == z[j];
          }
        }
        if (whole) {
          *reinterpret_cast<uint4*>(sm + p) = raw[u];
        } else {  // the ends, and vectors with a NaN
          for (int j = 0; j < VEC; j++) {
            const int q = p + j;
            const float z = q >= mis && q < mis + n ? clean(to_f<T>(g[q - mis])) : -INFINITY;
            top = fmaxf(top, z);
            sm[q] = from_f<T>(z);
          }
        }
      }
    }
    return top;
  }
};

struct Shared {
  Exchange x;
  u64 wmass[NWP];       // kept mass of each warp's positions
  u64 mass[2];          // the block's: all that the nucleus is taken of, that of the bins above the listed ones
  uint32_t cnt[NWP];    // tokens that each warp has listed (or would have)
  int offs[8 * NWP + 1];
  double wsum[NWP];
  int pick[2];
  double before;
};

template <typename T, bool SMEM>
__global__ void __launch_bounds__(NT, 2) k_sample_rows(RowArgs a) {
  constexpr int VEC = Part<T, SMEM>::VEC;
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ Shared sh;
  uint32_t* hist = dyn;               // [NBIN]; later the row's listed keys [GATHER]
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint32_t* list = dyn + GATHER + w * CW;
  const int nb = gridDim.x, rank = blockIdx.x, row = blockIdx.y;
  Group grp{cg::this_cluster(), sh.x, nb, 0};
  const int i0 = min(a.V, rank * a.seg);
  Part<T, SMEM> part;
  part.g = reinterpret_cast<const T*>(a.logits) + (long)row * a.ld + i0;
  part.sm = reinterpret_cast<T*>(dyn + GATHER + NWP * CW);
  part.mis = (int)((reinterpret_cast<uintptr_t>(part.g) & 15) / sizeof(T));
  part.n = min(a.V, i0 + a.seg) - i0;
  const int positions = (part.mis + part.n + VEC - 1) / VEC * VEC;
  const int per = (positions / VEC + NWP - 1) / NWP * VEC;  // positions a warp
  const int j0 = min(positions, w * per), j1 = min(positions, j0 + per);

  for (int i = tid; i < NBIN; i += NT) hist[i] = 0;
  const uint32_t top = grp.top(logit_key(part.load(positions)));

  const float temp = a.temperature ? a.temperature[row] : 1.f;
  Scale sc;
  sc.zf = key_logit(top);
  if (sc.zf == -INFINITY || !(temp > 0.f)) {
    // nothing to draw from, or greedy: the lowest index of the largest logit
    uint32_t best = 0;
    if (sc.zf != -INFINITY) {
      part.each(j0, j1, [&](float z, int p) { best = max(best, z == sc.zf ? ~(uint32_t)(i0 + p - part.mis) : 0u); });
      best = grp.top(best);
    }
    if (rank == 0 && tid == 0) {
      a.out[row] = sc.zf == -INFINITY ? -1 : (int)~best;
      if (a.logp) a.logp[row] = sc.zf == -INFINITY ? -INFINITY : 0.f;
    }
    if (nb > 1) grp.sync();  // no block leaves while another reads its shared memory
    return;
  }
  sc.zd = (double)sc.zf;
  sc.cd = 1.4426950408889634074 / (double)temp;
  sc.cf = fminf((float)sc.cd * 32.f, 3.0e38f);

  float thr = -INFINITY;  // the lowest logit that is kept (-infinity itself has no weight)

  // ---- the histogram of the kept tokens' counts or masses, over the whole row; each thread's running sums of its three bins
  double run[4];
  auto histogram = [&](bool masses) {
    part.each(j0, j1, [&](float z, int) {
      float fr;
      const int b = sc.bin(z, &fr);
      if (b < NBIN && z >= thr) {
        uint32_t inc = 1;
        if (masses) {  // 2^-(fr / 32), 15 fractional bits
          const float r = fmaf(fr, fmaf(fr, 2.3460e-4f, -2.16608e-2f), 1.f);
          inc = __float_as_uint(fmaf(r, 32768.f, 8388608.f)) - 0x4b000000u;
        }
        atomicAdd(&hist[b], inc);
      }
    });
    if (tid < 2) sh.pick[tid] = NBIN;
    grp.sync();
    double c[3] = {0.0, 0.0, 0.0};
    for (int i = 0; i < nb; i++) {
      const uint32_t* h = nb > 1 ? grp.cl.map_shared_rank(hist, i) : hist;
#pragma unroll
      for (int j = 0; j < 3; j++) c[j] += (double)h[3 * tid + j];
    }
    if (masses) {
#pragma unroll
      for (int j = 0; j < 3; j++) c[j] *= (double)exp2f((float)(3 * tid + j) * -0.03125f);
    }
    double incl = c[0] + c[1] + c[2];
    const double own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.wsum[w] = incl;
    __syncthreads();
    double base = 0.0;
    for (int i = 0; i < w; i++) base += sh.wsum[i];
    run[0] = base + (incl - own);
#pragma unroll
    for (int j = 0; j < 3; j++) run[j + 1] = run[j] + c[j];
  };
  // the first bin at which the running sum reaches v (NBIN: none); two threads' sums may differ in their last bits
  auto locate = [&](int slot, double v) {
#pragma unroll
    for (int j = 2; j >= 0; j--)
      if (run[j + 1] >= v && run[j] * (1.0 - 0x1p-40) < v) atomicMin(&sh.pick[slot], 3 * tid + j);
  };
  // lists a token (every lane of the warp calls it)
  uint32_t listed = 0;
  auto append = [&](bool on, float z) {
    const uint32_t m = __ballot_sync(0xffffffffu, on);
    if (m) {
      const uint32_t at = listed + __popc(m & ((1u << lane) - 1u));
      if (on && at < CW) list[at] = logit_key(z);
      listed += __popc(m);
    }
  };
  // Brings the blocks' lists together.  False: too many tokens.
  int n_list = 0;
  auto gather = [&]() -> bool {
    if (lane == 0) sh.cnt[w] = listed;
    grp.sync();  // the lists, their counts and sh.mass; the histogram has been read by all
    if (w == 0) {
      int c[4], s = 0;
      bool fit = true;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int i = 4 * lane + j;
        c[j] = i < nb * NWP ? (int)*grp.cl.map_shared_rank(&sh.cnt[i % NWP], i / NWP) : 0;
        fit &= c[j] <= CW;
        s += c[j];
      }
      int incl = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int at = incl - s;
      for (int j = 0; j < 4; j++) {
        sh.offs[4 * lane + j] = at;
        at += c[j];
      }
      fit = __all_sync(0xffffffffu, fit);
      if (lane == 31) sh.offs[8 * NWP] = fit && incl <= GATHER ? incl : -1;
    }
    __syncthreads();
    n_list = sh.offs[8 * NWP];
    if (n_list < 0) return false;
    for (int i = w; i < nb * NWP; i += NWP) {
      const int o = sh.offs[i], c = (i + 1 < 8 * NWP ? sh.offs[i + 1] : n_list) - o;
      const uint32_t* src = dyn + GATHER + (i % NWP) * CW;
      if (nb > 1) src = grp.cl.map_shared_rank(src, i / NWP);
      for (int k = lane; k < c; k += 32) hist[o + k] = src[k];
    }
    __syncthreads();
    return true;
  };
  // The largest key at which base + what the candidate tokens at or above it hold reaches `need`, bit by bit;
  // hold: each one's count or weight.  The candidates are the listed tokens, or those of bins b0 .. b1.
  auto search = [&](bool in_list, int b0, int b1, u64 base, double need, bool masses) -> float {
    uint32_t e[GATHER / NT];
    u64 hold[GATHER / NT];
    uint32_t lo = 0xffffffffu, hi = 0;
    auto candidate = [&](float z) -> bool {
      const int b = sc.bin(z);
      return b >= b0 && b <= b1 && z >= thr;
    };
    if (in_list) {
#pragma unroll
      for (int j = 0; j < GATHER / NT; j++) {
        const bool on = j * NT + tid < n_list;
        e[j] = on ? hist[j * NT + tid] : 0u;
        hold[j] = on ? (masses ? sc.weight(key_logit(e[j])) : 1ull) : 0ull;
        if (on) lo = min(lo, e[j]), hi = max(hi, e[j]);
      }
    } else {
      part.each(j0, j1, [&](float z, int) {
        if (candidate(z)) lo = min(lo, logit_key(z)), hi = max(hi, logit_key(z));
      });
    }
    const int blocks = in_list ? 1 : nb;
    hi = (uint32_t)grp.reduce<true>(hi, blocks);
    lo = ~(uint32_t)grp.reduce<true>(~lo, blocks);
    int bit = hi == lo ? -1 : 31 - __clz(hi ^ lo);
    uint32_t cur = bit < 0 ? hi : hi & ~((2u << bit) - 1u);
    for (; bit >= 0; bit--) {
      const uint32_t cand = cur | 1u << bit;
      u64 s = 0;
      if (in_list) {
#pragma unroll
        for (int j = 0; j < GATHER / NT; j++) s += e[j] >= cand ? hold[j] : 0ull;
      } else {
        part.each(j0, j1, [&](float z, int) {
          if (candidate(z) && logit_key(z) >= cand) s += masses ? sc.weight(z) : 1ull;
        });
      }
      s = grp.reduce<false>(s, blocks);
      if ((double)(base + s) >= need) cur = cand;
    }
    return key_logit(cur);
  };

  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < a.V) {
    histogram(false);
    locate(0, (double)k);
    __syncthreads();
    const int b = sh.pick[0];
    if (b < NBIN) {  // else every token that has a weight is kept
      if (b / 3 == tid) sh.before = run[b % 3];
      part.each(j0, j1, [&](float z, int) { append(sc.bin(z) == b, z); });
      const bool ok = gather();
      thr = search(ok, b, b, (u64)sh.before, (double)k, false);
    }
    grp.sync();  // the histogram's next use
    for (int i = tid; i < NBIN; i += NT) hist[i] = 0;
    __syncthreads();
    listed = 0;
  }

  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const u64 least = mp > 0.f ? (u64)ceil(fmin((double)mp, 1.0) * (double)(1ull << QW)) : 0ull;
  // bins behind this one hold nothing that min-p keeps
  const int far = mp > 0.f ? (int)fminf(ceilf(-log2f(fminf(mp, 1.f)) * 32.f) + 2.f, (float)(NBIN - 1)) : NBIN - 1;
  auto kept = [&](float z) -> u64 {
    if (!(z >= thr) || sc.bin(z) > far) return 0ull;
    const u64 v = sc.weight(z);
    return v >= least ? v : 0ull;
  };

  u64 mine = 0;  // kept mass of the warp's positions
  const float tp = a.top_p ? a.top_p[row] : 1.f;
  bool known = false;
  if (tp <= 0.f) {
    thr = sc.zf;
  } else if (tp < 1.f) {
    histogram(true);
    if (tid == NT - 1) sh.before = run[3];
    __syncthreads();
    const double want = (double)tp * sh.before;
    locate(0, want * (1.0 - 0x1p-13));
    locate(1, want * (1.0 + 0x1p-13));
    __syncthreads();
    const int b0 = sh.pick[0], b1 = min(sh.pick[1], NBIN - 1);
    u64 all = 0, above = 0;
    part.each(j0, j1, [&](float z, int) {
      const int b = sc.bin(z);
      const bool on = b < NBIN && z >= thr;
      if (__any_sync(0xffffffffu, on)) {
        const u64 v = on ? sc.weight(z) : 0ull;
        all += v;
        if (b < b0) {
          above += v;
          mine += v >= least ? v : 0ull;
        }
        append(on && b >= b0 && b <= b1, z);
      }
    });
    all = grp.reduce<false>(all, 1);
    above = grp.reduce<false>(above, 1);
    if (tid == 0) sh.mass[0] = all, sh.mass[1] = above;
    const bool ok = gather();
    if (nb > 1) {
      all = above = 0;
      for (int i = 0; i < nb; i++) {
        const u64* m = grp.cl.map_shared_rank(sh.mass, i);
        all += m[0];
        above += m[1];
      }
    }
    thr = search(ok, b0, b1, above, (double)tp * (double)all, true);
    if (ok) {  // the warp's own listed tokens join those of the bins above
      for (uint32_t i = lane; i < listed; i += 32) mine += kept(key_logit(list[i]));
      known = true;
    } else {
      mine = 0;
    }
  }
  if (!known)
    part.each(j0, j1, [&](float z, int) {
      const bool on = z >= thr && sc.bin(z) <= far;
      if (__any_sync(0xffffffffu, on)) {
        const u64 v = on ? sc.weight(z) : 0ull;
        mine += v >= least ? v : 0ull;
      }
    });

  // ---- the draw: the first token whose running kept mass exceeds u times the whole
  mine = warp_sum_u64(mine);
  if (lane == 0) sh.wmass[w] = mine;
  const u64 mass = grp.sum(lane == 0 ? mine : 0ull);
  u64 before = 0;
  if (nb > 1)
    for (int i = 0; i < rank; i++) before += *grp.cl.map_shared_rank(&sh.x.block[grp.turn], i);
  const float u = a.uniform[row];
  u64 target = u > 0.f ? (u64)((double)u * (double)mass) : 0ull;
  target = min(target, mass - 1);
  int cw = -1;  // the warp whose positions hold the token
  for (int i = 0; i < NWP && cw < 0; i++) {
    const u64 m = sh.wmass[i];
    if (before > target) break;
    if (target - before < m) cw = i; else before += m;
  }
  if (cw >= 0) {
    // its positions are divided again among the warps
    const int c0 = cw * per, c1 = min(positions, c0 + per);
    const int sub = (per + NT - 1) / NT * 32;
    const int s0 = min(c1, c0 + w * sub), s1 = min(c1, s0 + sub);
    u64 m = 0;
    for (int p = s0 + lane; p < s1; p += 32) m += kept(part.at(p));
    m = warp_sum_u64(m);
    __syncthreads();  // sh.wmass has been read
    if (lane == 0) sh.wmass[w] = m;
    __syncthreads();
    for (int i = 0; i < w; i++) before += sh.wmass[i];
    if (before <= target && target - before < m) {
      for (int p = s0; p < s1; p += 32) {
        const u64 v = p + lane < s1 ? kept(part.at(p + lane)) : 0ull;
        u64 sum = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + sum > target);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            a.out[row] = i0 + p + lane - part.mis;
            if (a.logp)
              a.logp[row] = (float)(-0.69314718055994530942 * sc.dist(part.at(p + lane)) -
                                    log((double)mass / (double)(1ull << QW)));
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
  }
  if (nb > 1) grp.sync();
}

template <typename T>
bool launch(Ctx& c, RowArgs a, int rows) {
  // a cluster a row: more blocks while the rows leave SMs idle, or while a block's part does not fit
  int nb = 1;
  constexpr int VEC = 16 / sizeof(T);
  auto part = [&](int b) { return ((a.V + b - 1) / b + VEC - 1) / VEC * VEC; };
  auto bytes = [&](int b) { return (part(b) + VEC) * (long)sizeof(T); };  // room for the first logit's offset
  while (nb < 8 && ((long)rows * nb * 2 <= c.num_sms || bytes(nb) > SMEM_ROW)) nb *= 2;
  a.seg = part(nb);
  const bool fits = bytes(nb) <= SMEM_ROW;
  auto k = fits ? k_sample_rows<T, true> : k_sample_rows<T, false>;
  const size_t smem = SMEM_HEAD + (fits ? (size_t)bytes(nb) : 0);
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_HEAD + SMEM_ROW) != cudaSuccess) return false;
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
