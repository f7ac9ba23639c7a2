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
// nucleus.  Only the tokens of those bins, a few hundred, are then listed, and
// searched by their keys' digits with exact counts or masses.  Rows whose
// tokens crowd into a bin are searched in place.
//
// Measured on a B200, 50,257 logits: one row 4 us greedy, 7 us with min-p, 14
// to 17 us with top-k or top-p (latency: four or five cluster barriers and the
// passes between them); 256 bf16 rows 9 us greedy (43% of the copy bandwidth),
// 38 us unfiltered (the weights' fp64 arithmetic: 13 operations a token), 57 us
// nucleus (beside that, one shared-memory addition a token: about five cycles
// a warp).
#include <cfloat>

#include <cooperative_groups.h>

#include "kernels.cuh"

namespace cg = cooperative_groups;

namespace gpt {
namespace {

constexpr int NT = 512;            // threads of a block
constexpr int NWP = NT / 32;
constexpr int QW = 44;             // fractional bits of a token's weight
constexpr int SMEM_ROW = 176 << 10; // bytes of a row that a block holds
constexpr int NBIN = 1536;         // 48 octaves: a token below 2^-48 of the largest has no weight
constexpr int GATHER = 2 * NT;     // listed tokens of a whole row: 2 a thread
static_assert(NBIN == 3 * NT, "a thread has three bins");

// Shared memory in front of the row: the block's histogram, later that of the listed tokens' keys; a cluster's
// histogram of the row; the block's list.  With one block a row the list takes the histogram's place (two such blocks
// with 50,257 bf16 logits each fit on an SM).
constexpr int HIST_BYTES = NBIN * 4 + 16, ENTRY = 12;
constexpr int HEAD_ONE = GATHER * ENTRY, HEAD_MANY = HIST_BYTES + NBIN * 4 + GATHER * ENTRY;
static_assert(GATHER * ENTRY >= HIST_BYTES && NBIN >= 3 * NT, "the lists take the histogram's place");

typedef unsigned long long u64;

// order-preserving image of a logit that is not NaN, and back; bf16 has 16 bits of them
template <typename T>
__device__ __forceinline__ uint32_t logit_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 + 0 = +0
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return sizeof(T) == 2 ? k >> 16 : k;
}
template <typename T>
__device__ __forceinline__ float key_logit(uint32_t k) {
  if (sizeof(T) == 2) return __uint_as_float(((k & 0x8000u) ? (k & 0x7fffu) : ~k & 0xffffu) << 16);
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
  float zf, cf;   // the largest logit; 32 log2(e) / temperature, divided by `half`
  float half;     // 1, or 1/2 where a distance that counts may pass fp32's range
  double cd;      // log2(e) / temperature
  __device__ __forceinline__ void set(float top, float temperature) {
    zf = top;
    cd = 1.4426950408889634074 / (double)fmaxf(temperature, 0x1p-122f);  // cf in fp32's range
    half = 48.0 / cd < 1.7e38 ? 1.f : 0.5f;  // (cd may be 0)
    cf = (float)(cd * 32.0 / half);
  }
  __device__ __forceinline__ double dist(float z) const { return ((double)zf - (double)z) * cd; }
  // rint(32 y) in fp32, of a logit not below floor(48); both roundings keep the order of logits.  *fr: 32 y - bin.
  // half * (zf - z), in one rounding: with temperatures of 1e37 and more (infinity included) logits as far apart as
  // fp32 allows have weights, and their distance itself would be infinite, its bin outside the histogram.
  __device__ __forceinline__ int bin(float z, float* fr = nullptr) const {
    const float d = fmaf(-half, z, half * zf);
    const float t = fmaf(d, cf, 12582912.f);
    if (fr) *fr = fmaf(d, cf, 12582912.f - t);
    return __float_as_int(t) - 0x4b400000;
  }
  // The weight, 44 fractional bits, of a token not below floor().  2^-y = 2^-n (1 + f P(f)), |f| <= 1/2, with P the
  // polynomial that meets (2^-f - 1) / f at the eight Chebyshev nodes (relative error 2^-38.7; f = 0 gives 1).
  __device__ __forceinline__ u64 weight(float z) const {
    const double d = (double)zf - (double)z;
    const double t = fma(d, cd, 6755399441055744.0);
    const double f = fma(d, cd, 6755399441055744.0 - t);
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
  // the least finite logit whose y is at most `octaves`
  __device__ __forceinline__ float floor(double octaves) const {
    return __double2float_ru(fmax((double)zf - octaves / cd, -(double)FLT_MAX));  // cd may be 0
  }
};

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Reductions over the block's threads and the cluster's blocks.  Slots
// alternate, so that one barrier an exchange is enough.  A block writes its
// value into every block's memory before the barrier: behind it all reads are
// local, and no block waits for another before it leaves.
struct Exchange {
  u64 warp[2][NWP];
  u64 block[2][8];
};
struct Group {
  cg::cluster_group cl;
  Exchange& x;
  int nb, rank, turn, block_turn;
  __device__ __forceinline__ void sync() {
    if (nb > 1) cl.sync(); else __syncthreads();
  }
  // over this block alone, or the cluster
  template <bool MAX>
  __device__ u64 reduce(u64 v, bool alone) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    auto warp = [&](u64 y) -> u64 { return MAX ? (u64)__reduce_max_sync(0xffffffffu, (uint32_t)y) : warp_sum_u64(y); };
    turn ^= 1;
    v = warp(v);
    if (lane == 0) x.warp[turn][w] = v;
    __syncthreads();
    v = warp(lane < NWP ? x.warp[turn][lane] : 0ull);
    if (alone || nb == 1) return v;
    block_turn ^= 1;
    if (threadIdx.x < nb) *cl.map_shared_rank(&x.block[block_turn][rank], threadIdx.x) = v;
    cl.sync();
    return warp(lane < nb ? x.block[block_turn][lane] : 0ull);
  }
  __device__ u64 sum(u64 v) { return reduce<false>(v, false); }
  __device__ uint32_t top(uint32_t v) { return (uint32_t)reduce<true>(v, false); }
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
  bool inf;  // the row has a +infinity: its equals read as 0, every other logit as -infinity

  static __device__ __forceinline__ float clean(float f) { return f != f ? -INFINITY : f; }
  __device__ __forceinline__ float at(int p) const {
    if (SMEM) return to_f<T>(sm[p]);
    const float z = p >= mis && p < mis + n ? clean(to_f<T>(g[p - mis])) : -INFINITY;
    return !inf ? z : z == INFINITY ? 0.f : -INFINITY;
  }
  __device__ __forceinline__ void only_infinities(int positions) {
    inf = true;
    if (SMEM)
      for (int p = threadIdx.x; p < positions; p += NT) sm[p] = from_f<T>(to_f<T>(sm[p]) == INFINITY ? 0.f : -INFINITY);
    __syncthreads();
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
  // f(VEC logits, the largest of them, first position) over positions [j0, j1), multiples of VEC; every lane of a warp
  // runs every step
  template <typename F>
  __device__ __forceinline__ void each(int j0, int j1, F f) const {
#pragma unroll 1
    for (int base = j0; base < j1; base += 32 * VEC) {
      const int p = base + (threadIdx.x & 31) * VEC;
      float z[VEC], m = -INFINITY;
      if (SMEM) {
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        const uint4 raw = p < j1 ? *reinterpret_cast<const uint4*>(sm + p) : make_uint4(none, none, none, none);
        split(raw, z);
        m = largest(raw);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          z[j] = p < j1 ? at(p + j) : -INFINITY;
          m = fmaxf(m, z[j]);
        }
      }
      f(z, m, p);
    }
  }
  // the largest of a vector's logits; NaN where there is one
  static __device__ __forceinline__ float largest(const uint4& v) {
    uint32_t m;
    if (sizeof(T) == 2) {
      asm("{ .reg .b32 a, b; max.NaN.bf16x2 a, %1, %2; max.NaN.bf16x2 b, %3, %4; max.NaN.bf16x2 %0, a, b; }"
          : "=r"(m) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
      const float lo = __uint_as_float(m << 16), hi = __uint_as_float(m & 0xffff0000u);
      return lo != lo ? lo : hi != hi ? hi : fmaxf(lo, hi);
    }
    asm("{ .reg .f32 a, b; max.NaN.f32 a, %1, %2; max.NaN.f32 b, %3, %4; max.NaN.f32 a, a, b; mov.b32 %0, a; }"
        : "=r"(m) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)), "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w)));
    return __uint_as_float(m);
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
          const float m = largest(raw[u]);
          whole = m == m;
          if (whole) top = fmaxf(top, m);
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
  u64 sums[2][NWP];     // each warp's share of: all that is counted, what lies above the listed tokens
  u64 row[3][8];        // each block's: the same two, and the tokens that it has listed (or would have)
  int n_list;           // tokens that the block lists
  uint32_t late[3 * NWP];  // the kept listed tokens' share of wmass, 15 bits at a time
  double wsum[NWP];
  int pick[2];
  int found;            // a digit of the border's key
  u64 above;
};

template <typename T, bool SMEM>
__global__ void __launch_bounds__(NT, 2) k_sample_rows(RowArgs a) {
  constexpr int VEC = Part<T, SMEM>::VEC;
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int nb = gridDim.x, rank = blockIdx.x, row = blockIdx.y;
  Group grp{cg::this_cluster(), sh.x, nb, rank, 0, 0};
  if (nb > 1) grp.cl.barrier_arrive();  // another block's memory may be written once all have started
  const int i0 = min(a.V, rank * a.seg);
  Part<T, SMEM> part;
  part.g = reinterpret_cast<const T*>(a.logits) + (long)row * a.ld + i0;
  uint32_t* hist = dyn;
  float* row_hist = reinterpret_cast<float*>(dyn + HIST_BYTES / 4);  // of a cluster
  // listed tokens: their weights, with the warp in the top bits, and their keys
  u64* list_w = reinterpret_cast<u64*>(dyn + (nb > 1 ? (HIST_BYTES + NBIN * 4) / 4 : 0));
  uint32_t* list_k = reinterpret_cast<uint32_t*>(list_w + GATHER);
  part.sm = reinterpret_cast<T*>(dyn + (nb > 1 ? HEAD_MANY : HEAD_ONE) / 4);
  part.inf = false;
  part.mis = (int)((reinterpret_cast<uintptr_t>(part.g) & 15) / sizeof(T));
  part.n = min(a.V, i0 + a.seg) - i0;
  const int positions = (part.mis + part.n + VEC - 1) / VEC * VEC;
  const int per = (positions / VEC + NWP - 1) / NWP * VEC;  // positions a warp
  const int j0 = min(positions, w * per), j1 = min(positions, j0 + per);

  const float temp = a.temperature ? a.temperature[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float tp = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.uniform[row];
  const float mine_top = part.load(positions);
  if (nb > 1) grp.cl.barrier_wait();
  float top = key_logit<T>(grp.top(logit_key<T>(mine_top)));
  if (top == -INFINITY || !(temp > 0.f)) {
    // nothing to draw from, or greedy: the lowest index of the largest logit
    uint32_t best = 0;
    if (top != -INFINITY) {
      part.each(j0, j1, [&](const float (&z)[VEC], float, int p) {
#pragma unroll
        for (int j = 0; j < VEC; j++) best = max(best, z[j] == top ? ~(uint32_t)(i0 + p + j - part.mis) : 0u);
      });
      best = grp.top(best);
    }
    if (rank == 0 && tid == 0) {
      a.out[row] = top == -INFINITY ? -1 : (int)~best;
      if (a.logp) a.logp[row] = top == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  if (top == INFINITY) {
    part.only_infinities(positions);
    top = 0.f;
  }
  Scale sc;
  sc.set(top, temp);

  // the lowest logit that is kept: a token below 2^-48 of the largest has no weight
  float lo = sc.floor(48.0);
  const u64 least = mp > 0.f ? (u64)ceil(fmin((double)mp, 1.0) * (double)(1ull << QW)) : 0ull;
  u64 mine = 0;  // kept mass of the warp's positions
  bool known = false;

  // ---- top-k (counts), then the nucleus (masses)
#pragma unroll 1
  for (int stage = 0; stage < 2; stage++) {
    const bool masses = stage == 1;
    if (masses ? !(tp < 1.f) : !(k > 0 && k < a.V)) continue;
    if (masses && tp <= 0.f) {
      lo = top;
      continue;
    }
    for (int i = tid; i < HIST_BYTES / 4; i += NT) hist[i] = 0;
    if (tid < 2) sh.pick[tid] = NBIN;
    if (tid == 0) sh.n_list = 0;
    __syncthreads();
    // a token adds 2^-(fr / 32), or 1, with 15 fractional bits to its bin
    const float c1 = masses ? -2.16608e-2f * 32768.f : 0.f, c2 = masses ? 2.3460e-4f * 32768.f : 0.f;
    part.each(j0, j1, [&](const float (&z)[VEC], float m, int) {
      if (!__any_sync(0xffffffffu, m >= lo)) return;
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        float fr;
        const int b = sc.bin(z[j], &fr);
        const float r = fmaf(fr, fmaf(fr, c2, c1), 8388608.f + 32768.f);
        if (z[j] >= lo) atomicAdd(&hist[b], __float_as_uint(r) - 0x4b000000u);
      }
    });
    grp.sync();
    // the whole row's; each thread's running sums of its three bins
    double run[4];
    {
      if (nb > 1) {
        // a block adds its share of the bins and gives the sums to all
        const int share = NBIN / 4 / nb, at = rank * share + tid;
        if (tid < share) {
          uint4 c[8];
#pragma unroll
          for (int i = 0; i < 8; i++)
            c[i] = i < nb ? reinterpret_cast<const uint4*>(grp.cl.map_shared_rank(hist, i))[at] : make_uint4(0, 0, 0, 0);
          u64 t[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 8; i++) t[0] += c[i].x, t[1] += c[i].y, t[2] += c[i].z, t[3] += c[i].w;
          const float4 f = make_float4((float)t[0], (float)t[1], (float)t[2], (float)t[3]);
#pragma unroll
          for (int i = 0; i < 8; i++)
            if (i < nb) reinterpret_cast<float4*>(grp.cl.map_shared_rank(row_hist, i))[at] = f;
        }
        grp.cl.sync();
      }
      double c[3];
#pragma unroll
      for (int j = 0; j < 3; j++) {
        const int b = 3 * tid + j;
        c[j] = (nb > 1 ? (double)row_hist[b] : (double)hist[b]) * (masses ? (double)exp2f((float)b * -0.03125f) : 0x1p-15);
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
      double sums = lane < NWP ? sh.wsum[lane] : 0.0;
#pragma unroll
      for (int o = 1; o < NWP; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += y;
      }
      const double total = __shfl_sync(0xffffffffu, sums, NWP - 1);
      const double base = w ? __shfl_sync(0xffffffffu, sums, max(w - 1, 0)) : 0.0;
      run[0] = base + (incl - own);
#pragma unroll
      for (int j = 0; j < 3; j++) run[j + 1] = run[j] + c[j];
      // The first bin at which the running sum reaches what is wanted, with slack for the masses' roundings: the border
      // lies in bins pick[0] .. pick[1].  (Two threads' sums may differ in their last bits.)
      const double want = masses ? (double)tp * total : (double)k, slack = masses ? 0x1p-13 : 0.0;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const double v = i ? want * (1.0 + slack) : want * (1.0 - slack);
#pragma unroll
        for (int j = 0; j < 3; j++)
          if (run[j + 1] >= v && run[j] * (1.0 - 0x1p-40) < v) atomicMin(&sh.pick[i], 3 * tid + j);
      }
      __syncthreads();
    }
    const int b0 = sh.pick[0], b1 = min(sh.pick[1], NBIN - 1);
    if (b0 == NBIN) {  // top-k: fewer tokens have a weight
      grp.sync();      // the histogram's next use
      continue;
    }
    // Those bins' logits, and a little more: z_above > z >= z_list.  The rest of the search goes by these two alone.
    const float z_above = sc.floor(((double)b0 - 0.51) / 32.0), z_list = fmaxf(lo, sc.floor(((double)b1 + 0.51) / 32.0));
    // ---- exact counts or masses: of all, and of the tokens above; the tokens between are listed
    u64 all = 0, above = 0;
    part.each(j0, j1, [&](const float (&z)[VEC], float m, int) {
      if (!__any_sync(0xffffffffu, m >= (masses ? lo : z_list))) return;
      uint32_t pend = 0;
      u64 v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        v[j] = 1;
        if (masses) {
          v[j] = sc.weight(z[j]);
          all += z[j] >= lo ? v[j] : 0ull;
        }
        if (z[j] >= z_above) above += v[j];
        else if (z[j] >= z_list) pend |= 1u << j;
      }
      if (pend) {
        int at = atomicAdd(&sh.n_list, __popc(pend));
#pragma unroll
        for (int j = 0; j < VEC; j++)
          if (pend >> j & 1u) {
            if (at < GATHER) {
              list_k[at] = logit_key<T>(z[j]);
              list_w[at] = v[j] | (u64)w << 60;
            }
            at++;
          }
      }
    });
    mine = above;
    all = warp_sum_u64(all);
    above = warp_sum_u64(above);
    if (lane == 0) sh.sums[0][w] = all, sh.sums[1][w] = above;
    __syncthreads();
    if (w == 0) {
      all = warp_sum_u64(lane < NWP ? sh.sums[0][lane] : 0ull);
      above = warp_sum_u64(lane < NWP ? sh.sums[1][lane] : 0ull);
      if (lane < nb) {
        u64* to = nb > 1 ? grp.cl.map_shared_rank(&sh.row[0][rank], lane) : &sh.row[0][0];
        to[0] = all;
        to[8] = above;
        to[16] = sh.n_list;
      }
    }
    grp.sync();  // the lists, their lengths and sums; the histogram has been read by all
    // ---- the row's listed tokens, two a thread, and the row's sums
    bool in_list;  // else too many: they are searched in place
    int n_list;
    uint32_t e[GATHER / NT];
    u64 hold[GATHER / NT];
    bool own[GATHER / NT];
    {
      const int c = lane < nb ? (int)sh.row[2][lane] : 0;
      all = warp_sum_u64(lane < nb ? sh.row[0][lane] : 0ull);
      above = warp_sum_u64(lane < nb ? sh.row[1][lane] : 0ull);
      n_list = __reduce_add_sync(0xffffffffu, c);
      in_list = n_list <= GATHER;
#pragma unroll
      for (int j = 0; j < GATHER / NT; j++) {
        int at = j * NT + tid, b = 0;
        e[j] = 0;
        hold[j] = 0;
        for (int i = 0; i < nb - 1; i++) {
          const int ci = __shfl_sync(0xffffffffu, c, i);
          if (b == i && at >= ci) at -= ci, b++;
        }
        own[j] = b == rank;
        if (in_list && j * NT + tid < n_list) {
          e[j] = nb > 1 ? *grp.cl.map_shared_rank(list_k + at, b) : list_k[at];
          hold[j] = nb > 1 ? *grp.cl.map_shared_rank(list_w + at, b) : list_w[at];
        }
      }
    }
    // ---- The largest key at which `above` and what the tokens between hold at or above the key reach the need: nine
    // bits at a time, by a histogram of the tokens that share the bits found so far.  Its 44-bit sums are kept as three
    // of 15 bits.
    const u64 need = masses ? (u64)ceil((double)tp * (double)all) : (u64)k;
    uint32_t kmin = 0xffffffffu, kmax = 0;
    if (in_list) {
#pragma unroll
      for (int j = 0; j < GATHER / NT; j++)
        if (hold[j]) kmin = min(kmin, e[j]), kmax = max(kmax, e[j]);
    } else {
      part.each(j0, j1, [&](const float (&z)[VEC], float, int) {
#pragma unroll
        for (int j = 0; j < VEC; j++)
          if (z[j] >= z_list && z[j] < z_above) kmin = min(kmin, logit_key<T>(z[j])), kmax = max(kmax, logit_key<T>(z[j]));
      });
    }
    kmax = (uint32_t)grp.reduce<true>(kmax, in_list);
    kmin = ~(uint32_t)grp.reduce<true>(~kmin, in_list);
    int bits = kmax == kmin ? 0 : 32 - __clz(kmax ^ kmin);  // still to be found
    uint32_t cur = bits == 32 ? 0u : kmax >> bits << bits;
#pragma unroll 1
    while (bits > 0) {
      const int sh_bits = max(bits - 9, 0);
      const uint32_t fixed = bits == 32 ? 0u : ~0u << bits;
      for (int i = tid; i < 3 * NT; i += NT) hist[i] = 0;
      __syncthreads();
      auto count = [&](uint32_t key, u64 v) {
        if (((key ^ cur) & fixed) == 0) {
          uint32_t* h = hist + (key >> sh_bits & 511u);
          atomicAdd(h, (uint32_t)v & 0x7fffu);
          if (v >> 15) {
            atomicAdd(h + NT, (uint32_t)(v >> 15) & 0x7fffu);
            atomicAdd(h + 2 * NT, (uint32_t)(v >> 30) & 0x7fffu);
          }
        }
      };
      if (in_list) {
#pragma unroll
        for (int j = 0; j < GATHER / NT; j++)
          if (hold[j]) count(e[j], hold[j] & ((1ull << 60) - 1));
        __syncthreads();
      } else {
        part.each(j0, j1, [&](const float (&z)[VEC], float m, int) {
          if (!__any_sync(0xffffffffu, m >= z_list)) return;
#pragma unroll
          for (int j = 0; j < VEC; j++)
            if (z[j] >= z_list && z[j] < z_above) count(logit_key<T>(z[j]), masses ? sc.weight(z[j]) : 1ull);
        });
        grp.sync();
      }
      u64 c = 0;  // thread t: digit 511 - t
      for (int i = 0; i < (in_list ? 1 : nb); i++) {
        const uint32_t* h = in_list || nb == 1 ? hist : grp.cl.map_shared_rank(hist, i);
        const int d = NT - 1 - tid;
        c += (u64)h[d] + ((u64)h[d + NT] << 15) + ((u64)h[d + 2 * NT] << 30);
      }
      u64 incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sh.wmass[w] = incl;
      if (tid == 0) sh.found = 0, sh.above = above;
      __syncthreads();
      u64 base = lane < w ? sh.wmass[lane & (NWP - 1)] : 0ull;
      base = above + warp_sum_u64(base);
      if (base + incl >= need && base + incl - c < need) {
        sh.found = NT - 1 - tid;
        sh.above = base + incl - c;
      }
      if (in_list) __syncthreads(); else grp.sync();
      cur |= (uint32_t)sh.found << sh_bits;
      above = sh.above;
      bits = sh_bits;
    }
    lo = fmaxf(lo, key_logit<T>(cur));
    known = masses && in_list && least == 0;
    if (known) {  // the listed tokens that are kept join those above, in their warps' sums
      if (tid < 3 * NWP) sh.late[tid] = 0;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < GATHER / NT; j++)
        if (hold[j] && own[j] && e[j] >= cur) {
          uint32_t* h = sh.late + (int)(hold[j] >> 60);
          atomicAdd(h, (uint32_t)hold[j] & 0x7fffu);
          atomicAdd(h + NWP, (uint32_t)(hold[j] >> 15) & 0x7fffu);
          atomicAdd(h + 2 * NWP, (uint32_t)(hold[j] >> 30) & 0x7fffu);
        }
      __syncthreads();
      if (lane == 0) mine += (u64)sh.late[w] + ((u64)sh.late[w + NWP] << 15) + ((u64)sh.late[w + 2 * NWP] << 30);
    } else {
      mine = 0;
    }
    if (!masses) grp.sync();  // the lists and the histogram are used again
  }

  if (mp > 0.f) lo = fmaxf(lo, sc.floor(-(double)log2f(fminf(mp, 1.f)) + 0.001));  // about where weights meet `least`
  auto kept = [&](float z) -> u64 {
    const u64 v = z >= lo ? sc.weight(z) : 0ull;
    return v >= least ? v : 0ull;
  };
  if (!known)
    part.each(j0, j1, [&](const float (&z)[VEC], float m, int) {
      if (__any_sync(0xffffffffu, m >= lo)) {
#pragma unroll
        for (int j = 0; j < VEC; j++) mine += kept(z[j]);
      }
    });

  // ---- the draw: the first token whose running kept mass exceeds u times the whole
  mine = warp_sum_u64(mine);
  if (lane == 0) sh.wmass[w] = mine;
  const u64 mass = grp.sum(lane == 0 ? mine : 0ull);
  u64 before = 0;
  if (nb > 1)
    for (int i = 0; i < rank; i++) before += sh.x.block[grp.block_turn][i];
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
  const size_t smem = (nb > 1 ? HEAD_MANY : HEAD_ONE) + (fits ? (size_t)bytes(nb) : 0);
  constexpr int most = HEAD_MANY + SMEM_ROW;
  if (!(fits ? allow_smem<k_sample_rows<T, true>>(most) : allow_smem<k_sample_rows<T, false>>(most))) return false;
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
