// Attention over the 8-bit key / value cache, and the accumulation of its
// weights (which eviction goes by).
//
//   o_r = sum_j softmax_j(scale q_r k_j) v_j   over the slots j that row r sees
//
// Row r = (new token i, query head) of a sequence with len tokens before this
// step sees slots 0 .. len + i.  With G query heads to a key / value head, the
// n G rows that share one are taken 8 NT at a time, as the columns of
//   S^T = K Q^T   and   O^T = V^T P^T
// by the 16 x 8 x 16 warp MMA: the cache is on its 16-row side, so that one row
// of queries (decoding) wastes seven of eight columns and not fifteen of
// sixteen rows, and a code that has been converted serves NT products.  Codes
// become fp16 by one exact conversion for two of them; the MMA takes the
// multiply-adds, so that the kernel is bound by reading the cache, or by the
// conversions, whatever the number of rows.
//
// The order of a dot product's terms and of a sum's is free, which the operand
// layouts use: lane (g, t) of the QK product takes a contiguous quarter of two
// keys' rows, and lane (g, t) of the PV product a contiguous eighth of the rows
// of four tokens; neither needs a transposition in memory.  P^T, the second
// product's other operand, is S^T's registers with each 8 x 8 part transposed
// (movmatrix).
#include <cfloat>

#include <cooperative_groups.h>

#include "kv8.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace gpt {
namespace {

constexpr int TT = 32;      // tokens a tile: two 16-token groups, each within one block of the cache
constexpr float LAZY = 8.f; // running maxima may be stale by this much (log2): weights stay below 2^8

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the parts of (lo, hi) that pack_f16 rounded off, times `up`, as fp16
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t p, float up = 1.f) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
  return pack_f16((lo - f.x) * up, (hi - f.y) * up);
}

// Weights in fp16.  They come times 2^7: the largest is 2^15, and what falls below fp16's grid is under 2^-32 of the
// largest weight.  With fp32 rows the second term comes times 2^11 more, against V times 2^-11 (exact: codes are
// multiples of 2^-9, fp16's grid is 2^-24), and leaves under 2^-43: a long tail of small weights, the same for all,
// keeps its sum.  (With neither factor 40,000 slots 12 nats below one lost 1.6e-4 of the output.)
constexpr float P_LOG2 = 7.f, REST = 2048.f;
__device__ __forceinline__ uint32_t pack_p_rest(float lo, float hi, uint32_t p) { return pack_rest(lo, hi, p, REST); }
__device__ __forceinline__ uint32_t v_rest(uint32_t v) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(1.f / REST));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The MMA cuts its sums off, which over hundreds of steps shows in fp32 (a long
// context's outputs were off by 1e-5 of the largest).  For fp32 rows' scores it
// adds up one step at a time, and the steps are added here, rounded to nearest.
struct Exact {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add_to(float (&d)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; i++) d[i] += x[i];
  }
};
// Their outputs add up in the tensor cores over CHAIN slots; then they are added, rounded, to sums set aside, so that
// there are few roundings of either kind over a long context.
constexpr int CHAIN = 256;
// The warp MMA's sums set aside, four to an index, in the thread's local memory: they are touched once in a chain, and
// registers and shared memory decide how many warps run.  (In shared memory, 16 KB more a block of 128 dimensions, two
// blocks an SM in place of three: 6 sequences of 30,000 slots, 32 on 8 heads of 128, 117 us; so 82 us.)
template <int N>
struct Aside {
  float4 mem[N > 0 ? N : 1];
  float4* x;
  bool any = false;
  __device__ __forceinline__ Aside() {
    x = mem;
    if (N > 0) asm volatile("" : "+l"(x));  // (an address that the compiler does not see through: not registers)
  }
  __device__ __forceinline__ void take(int i, float (&o)[4]) {
    float4 y = any ? x[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    y.x += o[0], y.y += o[1], y.z += o[2], y.w += o[3];
    x[i] = y;
    o[0] = o[1] = o[2] = o[3] = 0.f;
  }
  __device__ __forceinline__ void give(int i, float (&o)[4]) const {
    const float4 y = x[i];
    o[0] += y.x, o[1] += y.y, o[2] += y.z, o[3] += y.w;
  }
  __device__ __forceinline__ void scale(int i, float f0, float f1, float f2, float f3) {
    float4 y = x[i];
    y.x *= f0, y.y *= f1, y.z *= f2, y.w *= f3;
    x[i] = y;
  }
};
// The sums of weights carry what an addition rounds off (Kahan): equal weights would round the same way each time.
__device__ __forceinline__ void add_kept(float& sum, float& off, float x) {
  const float y = x - off, t = sum + y;
  off = (t - sum) - y;
  sum = t;
}

// A V block's factor of the weights (2^P_LOG2 among it), from its log2.  Past 2^120 (a block far above the one whose
// values set the running maximum of scores + log2(V scale): all its weights have underflowed) it stays finite, so that
// they remain 0.
__device__ __forceinline__ float v_factor(float log2) { return sfu_exp2(fminf(log2 + P_LOG2, 120.f)); }

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The power of two that brings a row's largest magnitude to 2^14 .. 2^15 (tiny rows: 2^100, so that it can be undone);
// 0 where it is 0 or infinite.  At fp32's largest values it is 2^-113.
__device__ __forceinline__ int row_exponent(float top) {
  return top > 0.f && top < INFINITY ? min(14 - ((int)(__float_as_uint(top) >> 23) - 127), 100) : 0;
}

// Rows of q as the B operand of the QK product, 8 NT of them.  bf16 rows are
// exact in fp16 once a power of two has brought the row's largest magnitude to
// 2^14 .. 2^15 (what falls below fp16's range then is under 2^-38 of it); fp32
// rows take two fp16 terms, 22 bits, which leaves less than the fp32 sum of the
// products does.
template <typename T, int HD, int NT>
struct QFrag {
  static constexpr int KS = HD / 16;
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  uint32_t b[TERMS][NT][KS][2];
  float f[NT][2];  // of rows 8 nt + 2 t + e: what a score has to be multiplied by to be scale * q k * log2(e)

  // first dimension of the four codes that lane t feeds to step ks
  static __device__ __forceinline__ int dim0(int t, int ks) {
    if (HD == 32) return t * 8 + 4 * ks;
    return (ks / 4) * 64 + t * 16 + (ks % 4) * 4;
  }

  // row r: token r / G, head r % G; q: the sequence's first row, at the group's first head
  __device__ void load(const T* __restrict__ q, long q_ld, int G, int row0, int R, float scale) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool vec = ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)(q_ld * (long)sizeof(T))) & (4 * sizeof(T) - 1)) == 0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const int r = row0 + 8 * nt + g;
      const bool on = r < R;
      const T* p = q + (on ? (long)(r / G) * q_ld + (r % G) * HD : 0);
      float x[KS][4];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        T y[4] = {from_f<T>(0.f), from_f<T>(0.f), from_f<T>(0.f), from_f<T>(0.f)};
        if (on) {
          const T* e = p + dim0(t, ks);
          if (vec) {
            if (sizeof(T) == 2)
              *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(e);
            else
              *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(e);
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++) y[j] = e[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          x[ks][j] = to_f<T>(y[j]);
          top = fmaxf(top, fabsf(x[ks][j]));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = row_exponent(top);
      const float up = kv8_pow2(e), down = kv8_pow2(-e) * scale * 1.4426950408889634f;
      f[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      f[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float lo = x[ks][2 * j] * up, hi = x[ks][2 * j + 1] * up;
          const uint32_t v = pack_f16(lo, hi);
          b[0][nt][ks][j] = v;
          if (TERMS == 2) b[TERMS - 1][nt][ks][j] = pack_rest(lo, hi, v);
        }
    }
  }

  // d = k q^T for 16 keys; w0, w1: the lane's quarters of its two keys' codes
  __device__ __forceinline__ void qk(float (&d)[NT][4], const uint32_t (&w0)[KS], const uint32_t (&w1)[KS]) const {
#pragma unroll
    for (int nt = 0; nt < NT; nt++) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
      const uint32_t a0 = f16x2_e4m3(w0[ks]), a1 = f16x2_e4m3(w1[ks]);
      const uint32_t a2 = f16x2_e4m3(w0[ks] >> 16), a3 = f16x2_e4m3(w1[ks] >> 16);
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        if (TERMS == 1) {
          mma(d[nt], a0, a1, a2, a3, b[0][nt][ks][0], b[0][nt][ks][1]);
        } else {
          Exact e;
#pragma unroll
          for (int m = TERMS - 1; m >= 0; m--) mma(e.x, a0, a1, a2, a3, b[m][nt][ks][0], b[m][nt][ks][1]);
          e.add_to(d[nt]);
        }
      }
    }
  }
};

// A tile's K and V as they lie in shared memory: 128-byte lines of 128 / HD
// tokens, their 16-byte chunks exchanged within the line so that the QK loads
// (two tokens 4 apart in a quarter warp) and the PV loads (four successive
// tokens) each touch all banks once.
template <int HD>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  constexpr int RPL = 128 / HD;
  const int line = row / RPL, c = (row % RPL) * (HD / 16) + chunk;
  const int x = HD == 128 ? ((row & 3) << 1) ^ (((row >> 2) & 1) << 2)
              : HD == 64  ? ((line & 1) << 1) | (((line >> 1) & 1) << 2)
                          : (line & 1) << 2;
  return line * 128 + ((c ^ x) << 4);
}

// The token, within its 16, of the QK product's row g + 8 half.  Lane t of the
// PV product then owns tokens t, t + 4, t + 8, t + 12 (k = 2 t, 2 t + 1, 2 t + 8,
// 2 t + 9 of its 16).
__device__ __forceinline__ int key_token(int g, int half) { return (g >> 1) + 4 * ((g & 1) + 2 * half); }

template <int HD>
struct alignas(16) Stage {
  uint8_t k[TT * HD];
  uint8_t v[TT * HD];
  float ks[2], vs[2];  // the groups' scales
  int ok;              // bit i: group i's block is one of the pool's
  int pad[3];
};

struct AttnArgs {
  const void* q;
  long q_ld;
  float scale;
  int G, n_split;
  void* o;
  long o_ld;
  float* lse;
};

constexpr int MAX_SPLIT = 16;  // blocks of a cluster

// What a block has of its rows when it is done with its part of the slots.
template <int ROWS>
struct RowStats {
  float m[ROWS], mv[ROWS], l[ROWS];  // maxima and sum, as above
  float fac[MAX_SPLIT][ROWS];        // for the join: each part's factor, then the row's
  float inv[ROWS], back[ROWS];
};

// Joins the cluster's blocks, part = [ROWS][PITCH] unnormalised outputs at each block's own maxima: block `split`
// finishes its share of the rows' values.
template <typename T, int HD, int ROWS, int PITCH, int THREADS>
__device__ __forceinline__ void join_blocks(RowStats<ROWS>& st, const float* part, int n_split, int split, int rows,
                                            const AttnArgs& at, int r0, int row0, int h, int heads) {
  cg::cluster_group cl = cg::this_cluster();
  const int G = at.G;
  if (n_split > 1) cl.sync(); else __syncthreads();
  for (int r = threadIdx.x; r < rows; r += THREADS) {
    float km[MAX_SPLIT], kv[MAX_SPLIT], kl[MAX_SPLIT], mm = -INFINITY, mmv = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < MAX_SPLIT; k++)
      if (k < n_split) {
        const RowStats<ROWS>* o = n_split > 1 ? cl.map_shared_rank(&st, k) : &st;
        km[k] = o->m[r];
        kv[k] = o->mv[r];
        kl[k] = o->l[r];
      }
#pragma unroll
    for (int k = 0; k < MAX_SPLIT; k++)
      if (k < n_split) mm = fmaxf(mm, km[k]), mmv = fmaxf(mmv, kv[k]);
#pragma unroll
    for (int k = 0; k < MAX_SPLIT; k++)
      if (k < n_split) {
        ll += km[k] == -INFINITY ? kl[k] : kl[k] * sfu_exp2(km[k] - mm);
        st.fac[k][r] = kv[k] == -INFINITY ? 1.f : sfu_exp2(kv[k] - mmv);
      }
    // a row that sees nothing: zeros, and the log of an empty sum
    st.inv[r] = ll == 0.f ? 0.f : 1.f / ll;
    st.back[r] = ll == 0.f ? 0.f : exp2f(mmv - mm - P_LOG2);
    if (split == 0 && at.lse) {
      const int rr = row0 + r;
      at.lse[(long)(r0 + rr / G) * heads + h * G + rr % G] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  T* out = reinterpret_cast<T*>(at.o);
  const bool vec = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(at.o_ld * (long)sizeof(T))) & (4 * sizeof(T) - 1)) == 0;
  constexpr int U = ROWS * HD / 4 >= 4 * THREADS ? 4 : 1;  // values in flight a thread, of each block
  const int used = rows * (HD / 4), share = (used + n_split - 1) / n_split, end = min(used, (split + 1) * share);
  for (int i0 = split * share + threadIdx.x; i0 < end; i0 += U * THREADS) {
    float4 y[U];
#pragma unroll
    for (int u = 0; u < U; u++) y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < n_split; k++) {
      const float* from = n_split > 1 ? cl.map_shared_rank(part, k) : part;
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int i = min(i0 + u * THREADS, end - 1), r = i / (HD / 4);
        const float4 x = *reinterpret_cast<const float4*>(from + r * PITCH + i % (HD / 4) * 4);
        const float f = st.fac[k][r];
        y[u].x = fmaf(f, x.x, y[u].x), y[u].y = fmaf(f, x.y, y[u].y), y[u].z = fmaf(f, x.z, y[u].z), y[u].w = fmaf(f, x.w, y[u].w);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int i = i0 + u * THREADS;
      if (i >= end) break;
      const int r = i / (HD / 4), rr = row0 + r;
      const float f = st.inv[r], b = st.back[r];
      T v[4] = {from_f<T>(y[u].x * f * b), from_f<T>(y[u].y * f * b), from_f<T>(y[u].z * f * b), from_f<T>(y[u].w * f * b)};
      T* p = out + (long)(r0 + rr / G) * at.o_ld + (long)(h * G + rr % G) * HD + i % (HD / 4) * 4;
      if (vec) {
        if (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(v);
        else
          *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) p[j] = v[j];
      }
    }
  }
  if (n_split > 1) cl.sync();  // no block leaves while another reads its shared memory
}

// One thread block (NW warps): 8 NT rows of one key / value head of one
// sequence, over one of the cluster's equal parts of the slots.  Each warp takes
// every NW-th tile of 32 tokens through its own ring of NS stages (cp.async, no
// block-wide barrier in the loop) with its own running maxima and sums; the
// warps, then the cluster's blocks through distributed shared memory, are joined
// at the end in a fixed order.
//
// B200: 6 sequences of 20000 to 40000 slots, 32 on 8 heads of 128: 66 us, 86%
// of the copy bandwidth (fp32 rows, twice the MMA: 94 us).  64 sequences of up to
// 1023 slots, 12 heads of 64: 19.5 us (8.6 us at the copy bandwidth; fp32 25 us).
// A warp's tile of 32 slots takes some 540 cycles of its scheduler (64 conversions
// at 2, 16 MMA at 12.5, the rest softmax), which for all tiles over all schedulers
// is 6.7 us; about 3 us pass before the first tile (start, length, table, codes)
// and 2 in the join; the rest is uneven work: one block a (sequence, head) whatever
// its length, 768 on 740 places, so that an SM takes what its five happen to hold.
template <typename T, int HD, int NT, int NW, int NS, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB) k_kv8_attn(Kv8Args a, AttnArgs at) {
  constexpr int ROWS = 8 * NT, TERMS = sizeof(T) == 4 ? 2 : 1;
  constexpr int BPL = HD / 8;         // dimensions a lane loads of a V row
  constexpr int MT = HD / 16;         // 16-dimension tiles of the output
  constexpr int OP = HD + 4;          // pitch of a row of partial outputs
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float st_m[NW][ROWS], st_mv[NW][ROWS], st_l[NW][ROWS];
  __shared__ RowStats<ROWS> stats;

  const int n_split = at.n_split, split = blockIdx.x % n_split, rt = blockIdx.x / n_split;
  const int h = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  // The length, the first tile's block ids (the first part's tiles start at 0 whatever the length) and the rows are
  // asked for together, not one after the other.
  const int32_t* ids = a.table + (size_t)s * a.max_blocks;
  const int len_raw = a.len[s];
  int pre0 = -1, pre1 = -1;
  if (split == 0) {
    if ((w * TT) >> a.lgP < a.max_blocks) pre0 = ids[(w * TT) >> a.lgP];
    if ((w * TT + 16) >> a.lgP < a.max_blocks) pre1 = ids[(w * TT + 16) >> a.lgP];
  }
  int r0;
  const int n = kv8_rows(a, s, &r0), G = at.G;
  const int R = n * G, row0 = rt * ROWS;
  if (row0 >= R) return;  // the same for every block of the cluster
  QFrag<T, HD, NT> q;
  q.load(reinterpret_cast<const T*>(at.q) + (long)r0 * at.q_ld + h * G * HD, at.q_ld, G, row0, R, at.scale);
  const int cap = a.max_blocks << a.lgP, len = min(max(len_raw, 0), cap);
  const int see_lo = min(len + row0 / G + 1, cap), see_hi = min(len + min(R - 1, row0 + ROWS - 1) / G + 1, cap);

  float o[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int nt = 0; nt < NT; nt++) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
  // of rows 8 nt + 2 t + e: running maximum of the scores (log2), that of scores + log2(V scale), the sum of
  // 2^(score - m), and the slots that the row sees
  float m[NT][2], mv[NT][2], l[NT][2], l_off[NT][2];
  int see[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      m[nt][e] = mv[nt][e] = -INFINITY;
      l[nt][e] = l_off[nt][e] = 0.f;
      see[nt][e] = min(len + min(row0 + 8 * nt + 2 * t + e, R - 1) / G + 1, cap);
    }

  const int tiles = (see_hi + TT - 1) / TT;
  const int per = (tiles + n_split - 1) / n_split;
  const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);
  Stage<HD>* ring = reinterpret_cast<Stage<HD>*>(smem) + w * NS;

  // fp32 rows: the lane's outputs of the chains before
  Aside<TERMS == 2 ? MT * NT : 0> aside;
  int chained = 0;

  // block ids of the next tile to be requested, looked up one tile ahead and first touched when they are needed
  int b0 = -1, b1 = -1;
  auto look = [&](int tile) {
    b0 = b1 = -1;
    if (tile < t1) {
      b0 = ids[(tile * TT) >> a.lgP];
      if (tile * TT + 16 < see_hi) b1 = ids[(tile * TT + 16) >> a.lgP];
    }
  };
  // A group's 16 rows are contiguous in its block: chunk u of a tile lies 512 u bytes on, in memory and (but for
  // the lane's constant) in the stage.
  constexpr int CPR = HD / 16;
  const uint32_t to_even = tile_at<HD>(lane / CPR, lane % CPR);
  const uint32_t to_odd = HD == 128 ? tile_at<HD>(32 / CPR + lane / CPR, lane % CPR) - 512 : to_even;
  auto request = [&](int tile, int slot) {
    if (tile < t1) {
      Stage<HD>& st = ring[slot];
      const int base = tile * TT;
      const bool bad0 = (unsigned)b0 >= (unsigned)a.n_blocks, bad1 = (unsigned)b1 >= (unsigned)a.n_blocks;
      if (bad0 || bad1) {
        if (lane == 0 && (bad0 || base + 16 < see_hi)) kv8_flag(a, FLAG_BLOCK);
        if (bad0) b0 = -1;
        if (bad1) b1 = -1;
      }
      const size_t p0 = ((size_t)max(b0, 0) * a.H + h), p1 = ((size_t)max(b1, 0) * a.H + h);
      const size_t s0 = ((p0 << a.lgP) + (base & (a.P - 1))) * HD + lane * 16;
      const size_t s1 = ((p1 << a.lgP) + ((base + 16) & (a.P - 1))) * HD + lane * 16;
      const uint32_t sk = (uint32_t)__cvta_generic_to_shared(st.k), sv = (uint32_t)__cvta_generic_to_shared(st.v);
      if (base + TT <= see_hi && b0 >= 0 && b1 >= 0) {
#pragma unroll
        for (int u = 0; u < CPR; u++) {
          const size_t src = u < CPR / 2 ? s0 + u * 512 : s1 + (u - CPR / 2) * 512;
          const uint32_t dst = u * 512 + (u & 1 ? to_odd : to_even);
          cp16(sk + dst, a.k + src, true);
          cp16(sv + dst, a.v + src, true);
        }
      } else {  // slots that no row sees, and groups without a block, are filled with zeros
#pragma unroll
        for (int u = 0; u < CPR; u++) {
          const bool on = base + (u * 32 + lane) / CPR < see_hi && (u < CPR / 2 ? b0 : b1) >= 0;
          const size_t src = on ? (u < CPR / 2 ? s0 + u * 512 : s1 + (u - CPR / 2) * 512) : 0;
          const uint32_t dst = u * 512 + (u & 1 ? to_odd : to_even);
          cp16(sk + dst, a.k + src, on);
          cp16(sv + dst, a.v + src, on);
        }
      }
      if (lane < 4) {
        const size_t p = (lane & 1) ? p1 : p0;
        cp4((uint32_t)__cvta_generic_to_shared(lane < 2 ? &st.ks[lane & 1] : &st.vs[lane & 1]),
            (lane < 2 ? a.ks : a.vs) + p, ((lane & 1) ? b1 : b0) >= 0);
      }
      if (lane == 0) st.ok = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
    }
    cp_commit();
  };

  int next = t0 + w;
  if (split == 0) {
    if (next < t1) b0 = pre0;
    if (next < t1 && next * TT + 16 < see_hi) b1 = pre1;
  } else {
    look(next);
  }
#pragma unroll
  for (int i = 0; i < NS - 1; i++) {
    request(next, i);
    next += NW;
    look(next);
  }
  int slot = 0;
  for (int tile = t0 + w; tile < t1; tile += NW) {
    cp_wait<NS - 2>();
    __syncwarp();  // the lanes' copies are visible to each other, and all are done with the stage requested into next
    request(next, slot == 0 ? NS - 1 : slot - 1);
    next += NW;
    look(next);
    const Stage<HD>& st = ring[slot];
    slot = slot == NS - 1 ? 0 : slot + 1;

    // ---- scores of 2 x 16 keys: [group][rows][key half, row parity]
    float sc[2][NT][4];
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      uint32_t kw[2][HD / 16];
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int row = gr * 16 + key_token(g, half);
        if (HD == 32) {
          const uint2 x = *reinterpret_cast<const uint2*>(st.k + tile_at<HD>(row, t >> 1) + (t & 1) * 8);
          kw[half][0] = x.x, kw[half][1] = x.y;
        } else {
#pragma unroll
          for (int c = 0; c < HD / 64; c++) {
            const uint4 x = *reinterpret_cast<const uint4*>(st.k + tile_at<HD>(row, c * 4 + t));
            kw[half][(4 * c) % CPR] = x.x, kw[half][(4 * c + 1) % CPR] = x.y;
            kw[half][(4 * c + 2) % CPR] = x.z, kw[half][(4 * c + 3) % CPR] = x.w;
          }
        }
      }
      q.qk(sc[gr], kw[0], kw[1]);
    }
    const int ok = st.ok;
    const bool full = tile * TT + TT <= see_lo && ok == 3;
    const float k0 = st.ks[0], k1 = st.ks[1];
    // log2 of the V scales (powers of two); a group without tokens has none
    const float v0 = ok & 1 ? (float)((int)(__float_as_uint(st.vs[0]) >> 23) - 127) : -INFINITY;
    const float v1 = ok & 2 ? (float)((int)(__float_as_uint(st.vs[1]) >> 23) - 127) : -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++)
#pragma unroll
        for (int gr = 0; gr < 2; gr++) {
          const float f = q.f[nt][e] * (gr ? k1 : k0);
          sc[gr][nt][e] *= f;
          sc[gr][nt][2 + e] *= f;
        }
    if (!full) {
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
          for (int gr = 0; gr < 2; gr++)
#pragma unroll
            for (int half = 0; half < 2; half++)
              if (tile * TT + gr * 16 + key_token(g, half) >= see[nt][e] || !(ok >> gr & 1)) sc[gr][nt][2 * half + e] = -INFINITY;
    }
    bool grow = false;
    float top[NT][2], topv[NT][2];  // largest score, and score + log2 V scale
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const float big[2] = {fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e])};
        top[nt][e] = fmaxf(big[0], big[1]);
        topv[nt][e] = fmaxf(big[0] + v0, big[1] + v1);
        grow |= top[nt][e] > m[nt][e] + LAZY || topv[nt][e] > mv[nt][e] + LAZY;
      }
    if (__any_sync(0xffffffffu, grow)) {  // the lanes' maxima are brought together only where one of them says so
      float fo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], d));
            topv[nt][e] = fmaxf(topv[nt][e], __shfl_xor_sync(0xffffffffu, topv[nt][e], d));
          }
          const float m1 = fmaxf(m[nt][e], top[nt][e]), mv1 = fmaxf(mv[nt][e], topv[nt][e]);
          const float fl = m1 == -INFINITY ? 1.f : sfu_exp2(m[nt][e] - m1);
          fo[nt][e] = mv1 == -INFINITY ? 1.f : sfu_exp2(mv[nt][e] - mv1);
          m[nt][e] = m1, mv[nt][e] = mv1;
          l[nt][e] *= fl;
          l_off[nt][e] *= fl;
#pragma unroll
          for (int i = 0; i < MT; i++) o[i][nt][e] *= fo[nt][e], o[i][nt][2 + e] *= fo[nt][e];
        }
      if (TERMS == 2 && aside.any) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int i = 0; i < MT; i++) aside.scale(i * NT + nt, fo[nt][0], fo[nt][1], fo[nt][0], fo[nt][1]);
      }
    }
    // ---- weights: 2^(score - m) for the sum, times 2^(log2 V scale + m - mv + P_LOG2) for the product with V's codes
    uint32_t p[2][NT][2], plo[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      float c[2][2];  // [group][row]
      float mm[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        mm[e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        const float d = mm[e] - (mv[nt][e] == -INFINITY ? 0.f : mv[nt][e]);
        c[0][e] = v_factor(v0 + d);
        c[1][e] = v0 == v1 ? c[0][e] : v_factor(v1 + d);
      }
      float lt[2] = {0.f, 0.f};  // the tile's sums
#pragma unroll
      for (int gr = 0; gr < 2; gr++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const float x = sfu_exp2(sc[gr][nt][2 * half] - mm[0]), y = sfu_exp2(sc[gr][nt][2 * half + 1] - mm[1]);
          lt[0] += x;
          lt[1] += y;
          const uint32_t v = pack_f16(x * c[gr][0], y * c[gr][1]);
          p[gr][nt][half] = transpose8(v);
          if (TERMS == 2) plo[gr][nt][half] = transpose8(pack_p_rest(x * c[gr][0], y * c[gr][1], v));
        }
      add_kept(l[nt][0], l_off[nt][0], lt[0]);
      add_kept(l[nt][1], l_off[nt][1], lt[1]);
    }
    // ---- o += v^T p^T
    bool poison = false;
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      uint32_t vw[4][HD / 32];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int row = gr * 16 + t + 4 * i;
        if (HD == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(st.v + tile_at<HD>(row, g));
          vw[i][0] = x.x, vw[i][1 % (HD / 32)] = x.y, vw[i][2 % (HD / 32)] = x.z, vw[i][3 % (HD / 32)] = x.w;
        } else if (HD == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(st.v + tile_at<HD>(row, g >> 1) + (g & 1) * 8);
          vw[i][0] = x.x, vw[i][1 % (HD / 32)] = x.y;
        } else {
          vw[i][0] = *reinterpret_cast<const uint32_t*>(st.v + tile_at<HD>(row, g >> 2) + (g & 3) * 4);
        }
      }
      if (!full && see_lo != see_hi) {
        // a NaN that some of the rows do not see must not reach them as 0 * NaN: it is taken out here, and put
        // into the rows that see it below
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int c = 0; c < HD / 32; c++) {
            const uint32_t nan = (((vw[i][c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            poison |= nan != 0;
            vw[i][c] &= ~(nan * 0xffu);
          }
      }
#pragma unroll
      for (int c = 0; c < HD / 32; c++) {
        // bytes j and j + 1 (x), j + 2 and j + 3 (y) of the tokens' pairs
        const uint32_t x01 = __byte_perm(vw[0][c], vw[1][c], 0x5140), y01 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
        const uint32_t x23 = __byte_perm(vw[2][c], vw[3][c], 0x5140), y23 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
        const uint32_t aa[2][4] = {
            {f16x2_e4m3(x01), f16x2_e4m3(x01 >> 16), f16x2_e4m3(x23), f16x2_e4m3(x23 >> 16)},
            {f16x2_e4m3(y01), f16x2_e4m3(y01 >> 16), f16x2_e4m3(y23), f16x2_e4m3(y23 >> 16)}};
#pragma unroll
        for (int i = 0; i < 2; i++) {
          if (TERMS == 2) {  // the weights' second fp16 term
            const uint32_t r0 = v_rest(aa[i][0]), r1 = v_rest(aa[i][1]), r2 = v_rest(aa[i][2]), r3 = v_rest(aa[i][3]);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) mma(o[2 * c + i][nt], r0, r1, r2, r3, plo[gr][nt][0], plo[gr][nt][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
            mma(o[2 * c + i][nt], aa[i][0], aa[i][1], aa[i][2], aa[i][3], p[gr][nt][0], p[gr][nt][1]);
        }
      }
    }
    if (__any_sync(0xffffffffu, poison)) {
      for (int row = 0; row < TT; row++) {
        const int j = tile * TT + row;
#pragma unroll
        for (int x = 0; x < BPL; x++) {
          const int d = g * BPL + x;
          if ((st.v[tile_at<HD>(row, d / 16) + d % 16] & 0x7f) == 0x7f)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (j < see[nt][e]) o[x / 2][nt][2 * (x & 1) + e] = __int_as_float(0x7fc00000);
        }
      }
    }
    if (TERMS == 2 && ++chained == CHAIN / TT) {
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++) aside.take(i * NT + nt, o[i][nt]);
      chained = 0;
      aside.any = true;
    }
  }
  if (TERMS == 2 && aside.any) {
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int nt = 0; nt < NT; nt++) aside.give(i * NT + nt, o[i][nt]);
  }

  // ---- join the warps: each row's maxima and sum, then the outputs at the common maximum
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      float x = l[nt][e] - l_off[nt][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const int r = 8 * nt + 2 * t + e;
      if (g == 0) st_m[w][r] = m[nt][e], st_mv[w][r] = mv[nt][e], st_l[w][r] = x;
    }
  cp_wait<0>();
  __syncthreads();  // every warp is done with its stages
  float* part = reinterpret_cast<float*>(smem);  // [NW][ROWS][OP]
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int e = 0; e < 2; e++)
#pragma unroll
      for (int i = 0; i < MT; i += 2)
        if (8 * nt + 2 * t + e < R - row0) *reinterpret_cast<float4*>(part + (w * ROWS + 8 * nt + 2 * t + e) * OP + g * BPL + 2 * i) =
            make_float4(o[i][nt][e], o[i][nt][2 + e], o[i + 1][nt][e], o[i + 1][nt][2 + e]);
  if (threadIdx.x < ROWS) {
    const int r = threadIdx.x;
    float mm = -INFINITY, mmv = -INFINITY, ll = 0.f;
    for (int i = 0; i < NW; i++) mm = fmaxf(mm, st_m[i][r]), mmv = fmaxf(mmv, st_mv[i][r]);
    for (int i = 0; i < NW; i++) {
      ll += st_m[i][r] == -INFINITY ? st_l[i][r] : st_l[i][r] * sfu_exp2(st_m[i][r] - mm);
      st_mv[i][r] = st_mv[i][r] == -INFINITY ? 0.f : sfu_exp2(st_mv[i][r] - mmv);  // the warp's factor
    }
    stats.m[r] = mm, stats.mv[r] = mmv, stats.l[r] = ll;
  }
  __syncthreads();
  float* sum = part + NW * ROWS * OP;  // [ROWS][HD]
  const int used = min(ROWS, R - row0) * HD;
  for (int i = threadIdx.x; i < used; i += NW * 32) {
    const int r = i / HD, d = i % HD;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < NW; k++) x = fmaf(st_mv[k][r], part[(k * ROWS + r) * OP + d], x);
    sum[i] = x;
  }
  join_blocks<T, HD, ROWS, HD, NW * 32>(stats, sum, n_split, split, min(ROWS, R - row0), at, r0, row0, h, a.H * G);
}

// ---------------------------------------------------------------- many rows

// A prompt's next part: 64 rows of one key / value head and sequence, 16 a warp,
// over one of the cluster's equal parts of the slots.  With that many rows the
// conversions are what costs, so a tile of codes becomes fp16 in shared memory
// once for all warps, and the warps multiply from there (rows on the 16-row side
// of the MMA, as S = Q K^T, O = P V).  The next tile's codes are on their way
// meanwhile; two tiles alternate, so that one barrier a tile is enough.  The
// statistics are those of k_kv8_attn.
//
// For 17 to 48 rows (fp32: 64) of 64 or fewer dimensions.  B200, 20 to 40 rows over
// up to 1501 slots, 4 sequences of 25 heads of 64: 19 us (fp32 27 us), 500 blocks
// on 444 places; barriers and the first loads (2.8 and 1.7 cycles an issued
// instruction) bound it, not the MMA: a prologue and a join are a third of a
// block's time, and with half of the rows in use the pipe is 8% busy.
constexpr int MR = 64, MW = 4, MT = 64;  // rows and warps of a block, slots of a tile

template <int HD>
__device__ __forceinline__ uint32_t half_at(int row, int chunk) {  // byte offset of 16 bytes of a tile of fp16 rows
  const int x = HD == 32 ? (row >> 1) & 3 : row & 7;
  return (uint32_t)(row * HD * 2 + ((chunk ^ x) << 4));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

template <int HD>
struct alignas(16) HalfTile {
  uint8_t k[MT * HD * 2];
  uint8_t v[MT * HD * 2];
};

template <typename T, int HD, int MINB>
__global__ void __launch_bounds__(MW * 32, MINB) k_kv8_attn_many(Kv8Args a, AttnArgs at) {
  constexpr int KS = HD / 16, NG = MT / 16, TERMS = sizeof(T) == 4 ? 2 : 1;
  constexpr int CPR = HD / 16, CPT = MT * CPR / (MW * 32);  // 16-code chunks a row; of K, and of V, a thread
  constexpr int OP = HD + 4;
  static_assert(CPT >= 1, "a thread has a chunk");
  extern __shared__ __align__(16) uint8_t smem[];
  HalfTile<HD>* tile_mem = reinterpret_cast<HalfTile<HD>*>(smem);
  __shared__ float g_ks[2][NG], g_v[2][NG];  // the groups' K scales and log2 V scales (-infinity: no block)
  __shared__ RowStats<MR> stats;

  const int n_split = at.n_split, split = blockIdx.x % n_split, rt = blockIdx.x / n_split;
  const int h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s), G = at.G;
  const int R = n * G, row0 = rt * MR;
  if (row0 >= R) return;  // the same for every block of the cluster
  const int cap = a.max_blocks << a.lgP;
  const int see_lo = min(len + row0 / G + 1, cap), see_hi = min(len + min(R - 1, row0 + MR - 1) / G + 1, cap);
  const int wrow = row0 + 16 * w;  // the warp's rows
  const int w_lo = min(len + min(R - 1, wrow) / G + 1, cap), w_hi = min(len + min(R - 1, wrow + 15) / G + 1, cap);

  const int tiles = (see_hi + MT - 1) / MT;
  const int per = (tiles + n_split - 1) / n_split;
  const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);

  // ---- a thread's chunks of a tile: codes in flight, their blocks looked up a tile earlier
  int blk[CPT];
  uint4 ck[CPT], cv[CPT];
  float gks = 0.f, gvs = 0.f;  // 0: no block
  int gblk = -1;
  const int32_t* ids = a.table + (size_t)s * a.max_blocks;
  const int trow = tid / CPR;  // the thread's first row of a tile; its others are MW * 32 / CPR apart
  auto look = [&](int tile) {
#pragma unroll
    for (int u = 0; u < CPT; u++) {
      const int j = tile * MT + trow + u * (MW * 32 / CPR);
      blk[u] = -1;
      if (tile < t1 && j < see_hi) blk[u] = ids[j >> a.lgP];  // first touched when the tile is fetched
    }
    gblk = -1;
    if (tid < NG && tile < t1 && tile * MT + tid * 16 < see_hi) gblk = ids[(tile * MT + tid * 16) >> a.lgP];
  };
  auto fetch = [&](int tile) {
#pragma unroll
    for (int u = 0; u < CPT; u++) {
      ck[u] = cv[u] = make_uint4(0, 0, 0, 0);
      if ((unsigned)blk[u] < (unsigned)a.n_blocks) {
        const int j = tile * MT + trow + u * (MW * 32 / CPR);
        const size_t src = ((((size_t)blk[u] * a.H + h) << a.lgP) + (j & (a.P - 1))) * HD + (tid % CPR) * 16;
        ck[u] = *reinterpret_cast<const uint4*>(a.k + src);
        cv[u] = *reinterpret_cast<const uint4*>(a.v + src);
      }
    }
    if (tid < NG && tile < t1) {
      const bool on = (unsigned)gblk < (unsigned)a.n_blocks;
      if (!on && tile * MT + tid * 16 < see_hi) kv8_flag(a, FLAG_BLOCK);
      const size_t bh = (size_t)(on ? gblk : 0) * a.H + h;
      gks = gvs = 0.f;
      if (on) gks = a.ks[bh], gvs = a.vs[bh];
    }
  };
  // Writes the fetched tile as fp16.  A NaN that some of the rows do not see must not reach them as 0 * NaN: in a tile
  // that not every row sees whole it is taken out of V.  True where that happened.
  auto convert = [&](int tile, int buf) -> bool {
    bool nan = false;
    const bool partial = tile * MT + MT > see_lo && see_lo != see_hi;
    HalfTile<HD>& m = tile_mem[buf];
#pragma unroll
    for (int u = 0; u < CPT; u++) {
      const int i = u * MW * 32 + tid, row = i / CPR, ch = 2 * (i % CPR);
      uint32_t x[4] = {ck[u].x, ck[u].y, ck[u].z, ck[u].w}, y[4] = {cv[u].x, cv[u].y, cv[u].z, cv[u].w};
      if (partial) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t bad = (((y[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
          nan |= bad != 0;
          y[j] &= ~(bad * 0xffu);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; j++) {
        *reinterpret_cast<uint4*>(m.k + half_at<HD>(row, ch + j)) =
            make_uint4(f16x2_e4m3(x[2 * j]), f16x2_e4m3(x[2 * j] >> 16), f16x2_e4m3(x[2 * j + 1]), f16x2_e4m3(x[2 * j + 1] >> 16));
        *reinterpret_cast<uint4*>(m.v + half_at<HD>(row, ch + j)) =
            make_uint4(f16x2_e4m3(y[2 * j]), f16x2_e4m3(y[2 * j] >> 16), f16x2_e4m3(y[2 * j + 1]), f16x2_e4m3(y[2 * j + 1] >> 16));
      }
    }
    if (tid < NG) {
      g_ks[buf][tid] = gks;
      g_v[buf][tid] = gvs > 0.f ? (float)((int)(__float_as_uint(gvs) >> 23) - 127) : -INFINITY;
    }
    return nan;
  };

  // ---- the warp's rows, asked for before the first tile whose block ids are still on their way
  look(t0);
  T qraw[2][KS][4];
#pragma unroll
  for (int half = 0; half < 2; half++) {
    const int r = wrow + g + 8 * half;
    const T* p = reinterpret_cast<const T*>(at.q) + (r < R ? (long)(r0 + r / G) * at.q_ld + (h * G + r % G) * HD : 0);
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        qraw[half][ks][j] = from_f<T>(0.f);
        if (r < R) qraw[half][ks][j] = p[ks * 16 + 2 * t + (j & 1) + (j >> 1) * 8];
      }
  }
  fetch(t0);
  look(t0 + 1);

  // ---- the A operand: fp16 after a power of two, as in QFrag
  uint32_t q[TERMS][KS][4];
  float qf[2];
  int see[2];
#pragma unroll
  for (int half = 0; half < 2; half++) {
    const int r = wrow + g + 8 * half;
    see[half] = min(len + min(r, R - 1) / G + 1, cap);
    float x[KS][4], top = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        x[ks][j] = to_f<T>(qraw[half][ks][j]);
        top = fmaxf(top, fabsf(x[ks][j]));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = row_exponent(top);
    const float up = kv8_pow2(e);
    qf[half] = kv8_pow2(-e) * at.scale * 1.4426950408889634f;
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const float lo = x[ks][2 * j] * up, hi = x[ks][2 * j + 1] * up;
        const uint32_t v = pack_f16(lo, hi);
        q[0][ks][2 * j + half] = v;
        if (TERMS == 2) q[TERMS - 1][ks][2 * j + half] = pack_rest(lo, hi, v);
      }
  }
  // the lane's offsets into a tile for ldmatrix; eight or sixteen rows on, they are the same but for the rows' bytes
  uint32_t k_off[KS / 2], v_off[HD / 16];
#pragma unroll
  for (int ks = 0; ks < KS; ks += 2) k_off[ks / 2] = half_at<HD>(lane & 7, 2 * ks + (lane >> 3));
#pragma unroll
  for (int i = 0; i < HD / 8; i += 2) v_off[i / 2] = half_at<HD>(lane & 15, i + (lane >> 4));
  float o[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, l_off[2] = {0.f, 0.f};
  Aside<TERMS == 2 ? HD / 8 : 0> aside;  // fp32 rows: the thread's outputs of the chains before
  int chained = 0;

  for (int tile = t0; tile < t1; tile++) {
    const int buf = (tile - t0) & 1;
    const bool poison = __syncthreads_or(convert(tile, buf));
    fetch(tile + 1);
    look(tile + 2);
    if (wrow >= R || tile * MT >= w_hi) continue;  // nothing that the warp's rows see
    const uint32_t kb = (uint32_t)__cvta_generic_to_shared(tile_mem[buf].k), vb = (uint32_t)__cvta_generic_to_shared(tile_mem[buf].v);

    // ---- scores: [8 tokens][row half, token parity]
    float sc[MT / 8][4];
#pragma unroll
    for (int j = 0; j < MT / 8; j++) {
      sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t b[4];
        ldsm4(b, kb + k_off[ks / 2] + j * 16 * HD);
        if (TERMS == 1) {
          mma(sc[j], q[0][ks][0], q[0][ks][1], q[0][ks][2], q[0][ks][3], b[0], b[1]);
          mma(sc[j], q[0][ks + 1][0], q[0][ks + 1][1], q[0][ks + 1][2], q[0][ks + 1][3], b[2], b[3]);
        } else {
          Exact e0, e1;
#pragma unroll
          for (int x = TERMS - 1; x >= 0; x--) {
            mma(e0.x, q[x][ks][0], q[x][ks][1], q[x][ks][2], q[x][ks][3], b[0], b[1]);
            mma(e1.x, q[x][ks + 1][0], q[x][ks + 1][1], q[x][ks + 1][2], q[x][ks + 1][3], b[2], b[3]);
          }
          e0.add_to(sc[j]);
          e1.add_to(sc[j]);
        }
      }
    }
    float vl[NG], top[2] = {-INFINITY, -INFINITY}, topv[2] = {-INFINITY, -INFINITY};
    bool all = tile * MT + MT <= w_lo;
#pragma unroll
    for (int gr = 0; gr < NG; gr++) {
      vl[gr] = g_v[buf][gr];
      all &= vl[gr] != -INFINITY;
      const float ks = g_ks[buf][gr];
#pragma unroll
      for (int x = 0; x < 2; x++)
#pragma unroll
        for (int y = 0; y < 4; y++) sc[2 * gr + x][y] *= qf[y >> 1] * ks;
    }
    if (!all) {
#pragma unroll
      for (int j = 0; j < MT / 8; j++)
#pragma unroll
        for (int y = 0; y < 4; y++)
          if (tile * MT + 8 * j + 2 * t + (y & 1) >= see[y >> 1] || vl[j / 2] == -INFINITY) sc[j][y] = -INFINITY;
    }
    bool grow = false;
#pragma unroll
    for (int half = 0; half < 2; half++) {
#pragma unroll
      for (int gr = 0; gr < NG; gr++) {
        const float x = fmaxf(fmaxf(sc[2 * gr][2 * half], sc[2 * gr][2 * half + 1]),
                              fmaxf(sc[2 * gr + 1][2 * half], sc[2 * gr + 1][2 * half + 1]));
        top[half] = fmaxf(top[half], x);
        topv[half] = fmaxf(topv[half], x + vl[gr]);
      }
      grow |= top[half] > m[half] + LAZY || topv[half] > mv[half] + LAZY;
    }
    if (__any_sync(0xffffffffu, grow)) {  // the lanes' maxima are brought together only where one of them says so
      float fo[2];
#pragma unroll
      for (int half = 0; half < 2; half++) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], d));
          topv[half] = fmaxf(topv[half], __shfl_xor_sync(0xffffffffu, topv[half], d));
        }
        const float m1 = fmaxf(m[half], top[half]), mv1 = fmaxf(mv[half], topv[half]);
        const float fl = m1 == -INFINITY ? 1.f : sfu_exp2(m[half] - m1);
        fo[half] = mv1 == -INFINITY ? 1.f : sfu_exp2(mv[half] - mv1);
        m[half] = m1, mv[half] = mv1;
        l[half] *= fl;
        l_off[half] *= fl;
#pragma unroll
        for (int i = 0; i < HD / 8; i++) o[i][2 * half] *= fo[half], o[i][2 * half + 1] *= fo[half];
      }
      if (TERMS == 2 && aside.any) {
#pragma unroll
        for (int i = 0; i < HD / 8; i++) aside.scale(i, fo[0], fo[0], fo[1], fo[1]);
      }
    }
    float mm[2], dv[2], lt[2] = {0.f, 0.f};  // (lt: the tile's sums)
#pragma unroll
    for (int half = 0; half < 2; half++) {
      mm[half] = m[half] == -INFINITY ? 0.f : m[half];
      dv[half] = mm[half] - (mv[half] == -INFINITY ? 0.f : mv[half]);
    }
#pragma unroll
    for (int kk = 0; kk < NG; kk++) {
      const float c0 = v_factor(vl[kk] + dv[0]), c1 = v_factor(vl[kk] + dv[1]);
      uint32_t p[4], plo[4];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const float e0 = sfu_exp2(sc[2 * kk + x][0] - mm[0]), e1 = sfu_exp2(sc[2 * kk + x][1] - mm[0]);
        const float e2 = sfu_exp2(sc[2 * kk + x][2] - mm[1]), e3 = sfu_exp2(sc[2 * kk + x][3] - mm[1]);
        lt[0] += e0 + e1;
        lt[1] += e2 + e3;
        p[2 * x] = pack_f16(e0 * c0, e1 * c0);
        p[2 * x + 1] = pack_f16(e2 * c1, e3 * c1);
        if (TERMS == 2) {
          plo[2 * x] = pack_p_rest(e0 * c0, e1 * c0, p[2 * x]);
          plo[2 * x + 1] = pack_p_rest(e2 * c1, e3 * c1, p[2 * x + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < HD / 8; i += 2) {
        uint32_t b[4];
        ldsm4t(b, vb + v_off[i / 2] + kk * 32 * HD);
        if (TERMS == 2) {
          mma(o[i], plo[0], plo[1], plo[2], plo[3], v_rest(b[0]), v_rest(b[1]));
          mma(o[i + 1], plo[0], plo[1], plo[2], plo[3], v_rest(b[2]), v_rest(b[3]));
        }
        mma(o[i], p[0], p[1], p[2], p[3], b[0], b[1]);
        mma(o[i + 1], p[0], p[1], p[2], p[3], b[2], b[3]);
      }
    }
    add_kept(l[0], l_off[0], lt[0]);
    add_kept(l[1], l_off[1], lt[1]);
    if (poison) {  // the NaN that were taken out go into the rows that see them
      for (int row = 0; row < MT; row++) {
        const int j = tile * MT + row;
        if (j >= see_hi) break;
        const int b = ids[j >> a.lgP];
        if ((unsigned)b >= (unsigned)a.n_blocks) continue;
        const uint8_t* c = a.v + ((((size_t)b * a.H + h) << a.lgP) + (j & (a.P - 1))) * HD;
#pragma unroll
        for (int i = 0; i < HD / 8; i++)
#pragma unroll
          for (int y = 0; y < 4; y++)
            if ((c[8 * i + 2 * t + (y & 1)] & 0x7f) == 0x7f && j < see[y >> 1]) o[i][y] = __int_as_float(0x7fc00000);
      }
    }
    if (TERMS == 2 && ++chained == CHAIN / MT) {
#pragma unroll
      for (int i = 0; i < HD / 8; i++) aside.take(i, o[i]);
      chained = 0;
      aside.any = true;
    }
  }
  if (TERMS == 2 && aside.any) {
#pragma unroll
    for (int i = 0; i < HD / 8; i++) aside.give(i, o[i]);
  }

#pragma unroll
  for (int half = 0; half < 2; half++) {
    l[half] -= l_off[half];
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
  }
  __syncthreads();  // every warp is done with the tiles
  float* part = reinterpret_cast<float*>(smem);  // [MR][OP]
#pragma unroll
  for (int half = 0; half < 2; half++) {
    const int r = 16 * w + g + 8 * half;
#pragma unroll
    for (int i = 0; i < HD / 8; i++)
      *reinterpret_cast<float2*>(part + r * OP + 8 * i + 2 * t) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
    if (t == 0) stats.m[r] = m[half], stats.mv[r] = mv[half], stats.l[r] = l[half];
  }
  join_blocks<T, HD, MR, OP, MW * 32>(stats, part, n_split, split, min(MR, R - row0), at, r0, row0, h, a.H * G);
}

// ---------------------------------------------------------------- many rows: tcgen05
//
// 128 rows of one key / value head and sequence over one of the cluster's equal
// parts of the slots, 64 slots a tile.  Two or four warps turn codes into fp16 tiles
// (128-byte swizzle, as a TMA load would leave them) through a ring of stages;
// one thread issues S = Q K^T into one of two TMEM buffers and, a tile later,
// O += P V with P read from TMEM; four warps, a row a thread, do the softmax:
// scores are scaled by the row's and the group's factors, P goes back to TMEM as
// fp16 over its scores, and O is rescaled in TMEM only where a running maximum
// has to grow.  Statistics and joins are those of k_kv8_attn.
//
// fp32 rows: Q and P are two fp16 terms each (a stage has V twice, for P's second
// term times 2^-11), and the products of four tiles at a time are added to sums
// of their own (FLUSH): 6e-7 of the outputs' norm over 20,000 and 100,000 slots,
// where sums left in the tensor core drift off by 2.7e-6.
//
// B200: 2 sequences of 900 to 1000 new rows over 3000 to 4000 slots, 16 heads of
// 64: 102 us, 302 TFLOP/s of the visible products (the warp MMA's blocks of 64
// rows: 203 us; fp32 rows 157 us).  Two resident blocks keep the SFU and the schedulers of the
// softmax warps busy: a tile is 8192 exponentials at 16 a cycle and SM, and about
// five other instructions each.  63 to 200 new rows over up to 1501 slots, 4
// sequences of 25 heads: 28 us (33 us), two fifths of it before the first tile
// and in the join (fp32 39 us).  fp32, 3 sequences of 71 new rows over 4300 slots,
// 8 heads of 128: 66 us (with two converting warps 81 us, the warp MMA's blocks
// 100 us).
constexpr int CR = 128, CT = 64;             // rows of a block, slots of a tile
constexpr int C_SOFT = 4;                    // softmax warps; one more issues, others convert

template <typename T, int HD>
struct TcShape {
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;                  // fp16 terms of Q and P
  static constexpr int MINB = TERMS == 2 && HD == 128 ? 1 : 2;          // blocks an SM
  // fp32 rows: the products add up over FLUSH tiles only; then they are added, rounded to nearest, to the sums so far,
  // which have their own columns (the tensor core cuts its sums off: over hundreds of tiles that shows in fp32)
  static constexpr int FLUSH = TERMS == 2 ? CHAIN / CT : 1 << 30, SUMS = 128 + (HD == 128 ? 128 : 64);
  static constexpr int COLS = TERMS == 2 && HD == 128 ? 512 : 256;      // TMEM columns
  static constexpr int MAKE = MINB == 1 ? 4 : 2;                        // converting warps (two blocks of an SM: two each)
  static constexpr int THREADS = (C_SOFT + 1 + MAKE) * 32;
  static constexpr int NB = HD == 128 ? 2 : 1, WD = HD < 64 ? HD : 64;  // blocks of 64 dimensions, dimensions a block
  static constexpr int NS = HD == 128 || TERMS == 2 ? 2 : 3;            // stages
  static constexpr int QB = CR * 128, TB = CT * 128;                    // bytes of a block's Q, and of K or V
  // the first stage: K blocks, V blocks, fp32 rows: V blocks for the weights' second term
  static constexpr int KV = TERMS * NB * QB, STAGE = (1 + TERMS) * NB * TB;
  static constexpr int END = KV + NS * STAGE, PITCH = HD + 4;           // (later: outputs [CR][PITCH])
  static_assert(CR * PITCH * 4 <= END, "the outputs take the tiles' place");
};
struct TcShared {
  RowStats<CR> stats;
  uint64_t q_full, kv_full[3], kv_empty[3], s_full[2], p_full[2], pv_done[2];
  float ks[3][4], vl[3][4];  // a stage's groups: K scale, log2 of the V scale (-infinity: no block)
  int nan[3][4];             // a NaN has been taken out of the stage's V
  uint32_t tmem, no_flags;
  int abort;
};

template <typename T, int HD>
__global__ void __launch_bounds__((TcShape<T, HD>::THREADS), (TcShape<T, HD>::MINB)) k_kv8_attn_tc(Kv8Args a, AttnArgs at) {
  using S = TcShape<T, HD>;
  using namespace sm100;
  constexpr int CPR = HD / 16, CPT = (CT * CPR + S::MAKE * 32 - 1) / (S::MAKE * 32);  // 16-code chunks a row; of K, and of V, a thread
  extern __shared__ uint8_t raw_smem[];
  // swizzled tiles need 1024-byte alignment
  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  TcShared& sh = *reinterpret_cast<TcShared*>(smem + S::END);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_split = at.n_split, split = blockIdx.x % n_split, rt = blockIdx.x / n_split;
  const int h = blockIdx.y, s = blockIdx.z;
  const int32_t* ids = a.table + (size_t)s * a.max_blocks;
  const int len_raw = a.len[s];
  int r0;
  const int n = kv8_rows(a, s, &r0), G = at.G;
  const int R = n * G, row0 = rt * CR;
  if (row0 >= R) return;  // the same for every block of the cluster
  const int cap = a.max_blocks << a.lgP, len = min(max(len_raw, 0), cap);
  const int see_lo = min(len + row0 / G + 1, cap), see_hi = min(len + min(R - 1, row0 + CR - 1) / G + 1, cap);
  const int tiles = (see_hi + CT - 1) / CT, per = (tiles + n_split - 1) / n_split;
  const int t0 = min(tiles, split * per), nt = min(tiles, t0 + per) - t0;
  uint32_t* gflags = a.flags ? a.flags : &sh.no_flags;
  volatile int* abort_flag = &sh.abort;
  const uint32_t q_full = smem_u32(&sh.q_full), kv_full0 = smem_u32(sh.kv_full), kv_empty0 = smem_u32(sh.kv_empty);
  const uint32_t s_full0 = smem_u32(sh.s_full), p_full0 = smem_u32(sh.p_full), pv_done0 = smem_u32(sh.pv_done);

  if (tid == 0) {
    mbar_init(q_full, C_SOFT);
    for (int i = 0; i < 3; i++) {
      mbar_init(kv_full0 + 8 * i, S::MAKE);
      mbar_init(kv_empty0 + 8 * i, 1);
    }
    for (int u = 0; u < 2; u++) {
      mbar_init(s_full0 + 8 * u, 1);
      mbar_init(p_full0 + 8 * u, C_SOFT);
      mbar_init(pv_done0 + 8 * u, 1);
    }
    sh.abort = 0;
    sh.no_flags = 0;
    fence_barrier_init();
  }
  if (warp == C_SOFT) {
    tmem_alloc(smem_u32(&sh.tmem), S::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp > C_SOFT) {
    // ================= codes to fp16 tiles
    const int me = tid - (C_SOFT + 1) * 32, w = warp - C_SOFT - 1;
    const int trow = me / CPR, part = me % CPR;
    constexpr int STEP = S::MAKE * 32 / CPR;  // rows between a thread's chunks
    // the next tile's codes in flight, and the block ids of the tile behind it
    int blk[CPT], gblk = -1;
    uint4 ck[CPT], cv[CPT];
    float gks = 0.f, gvs = 0.f;  // 0: no block
    auto look = [&](int j) {
#pragma unroll
      for (int u = 0; u < CPT; u++) {
        const int row = trow + u * STEP, slot = (t0 + j) * CT + row;
        blk[u] = -1;
        if (j < nt && row < CT && slot < see_hi) blk[u] = ids[slot >> a.lgP];  // first touched when the tile is fetched
      }
      gblk = -1;
      if (me < 4 && j < nt && (t0 + j) * CT + me * 16 < see_hi) gblk = ids[((t0 + j) * CT + me * 16) >> a.lgP];
    };
    auto fetch = [&](int j, uint4 (&k)[CPT], uint4 (&v)[CPT], float& ks, float& vs) {
#pragma unroll
      for (int u = 0; u < CPT; u++) {
        k[u] = v[u] = make_uint4(0, 0, 0, 0);
        if ((unsigned)blk[u] < (unsigned)a.n_blocks) {
          const int slot = (t0 + j) * CT + trow + u * STEP;
          const size_t src = ((((size_t)blk[u] * a.H + h) << a.lgP) + (slot & (a.P - 1))) * HD + part * 16;
          k[u] = *reinterpret_cast<const uint4*>(a.k + src);
          v[u] = *reinterpret_cast<const uint4*>(a.v + src);
        }
      }
      if (me < 4 && j < nt) {
        const bool on = (unsigned)gblk < (unsigned)a.n_blocks;
        if (!on && (t0 + j) * CT + me * 16 < see_hi) kv8_flag(a, FLAG_BLOCK);
        const size_t bh = (size_t)(on ? gblk : 0) * a.H + h;
        ks = vs = 0.f;
        if (on) ks = a.ks[bh], vs = a.vs[bh];
      }
    };
    auto make = [&](int j, const uint4 (&ckj)[CPT], const uint4 (&cvj)[CPT], float ks, float vs) -> bool {
      const int st = j % S::NS;
      if (!mbar_wait(kv_empty0 + 8 * st, ((j / S::NS) & 1) ^ 1, abort_flag, gflags)) return false;
      uint8_t* tk = smem + S::KV + st * S::STAGE;
      uint8_t* tv = tk + S::NB * S::TB;
      const int tile = t0 + j;
      // a NaN that some of the rows do not see must not reach them as 0 * NaN: in a tile that not every row sees whole
      // it is taken out of V, and put into the rows that see it at the end
      const bool partial = tile * CT + CT > see_lo && see_lo != see_hi;
      bool nan = false;
#pragma unroll
      for (int u = 0; u < CPT; u++) {
        const int row = trow + u * STEP;
        if (row >= CT) break;
        uint32_t x[4] = {ckj[u].x, ckj[u].y, ckj[u].z, ckj[u].w}, y[4] = {cvj[u].x, cvj[u].y, cvj[u].z, cvj[u].w};
        if (partial) {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint32_t bad = (((y[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
            nan |= bad != 0;
            y[i] &= ~(bad * 0xffu);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const uint32_t off = (part / 4) * S::TB + half_at<64>(row, part % 4 * 2 + i);
          *reinterpret_cast<uint4*>(tk + off) =
              make_uint4(f16x2_e4m3(x[2 * i]), f16x2_e4m3(x[2 * i] >> 16), f16x2_e4m3(x[2 * i + 1]), f16x2_e4m3(x[2 * i + 1] >> 16));
          const uint4 v =
              make_uint4(f16x2_e4m3(y[2 * i]), f16x2_e4m3(y[2 * i] >> 16), f16x2_e4m3(y[2 * i + 1]), f16x2_e4m3(y[2 * i + 1] >> 16));
          *reinterpret_cast<uint4*>(tv + off) = v;
          if (S::TERMS == 2)
            *reinterpret_cast<uint4*>(tv + S::NB * S::TB + off) = make_uint4(v_rest(v.x), v_rest(v.y), v_rest(v.z), v_rest(v.w));
        }
      }
      if (me < 4) {
        sh.ks[st][me] = ks;
        sh.vl[st][me] = vs > 0.f ? (float)((int)(__float_as_uint(vs) >> 23) - 127) : -INFINITY;
      }
      nan = __any_sync(0xffffffffu, nan);
      if (lane == 0) sh.nan[st][w] = nan;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(kv_full0 + 8 * st);
      return true;
    };
    look(0);
    fetch(0, ck, cv, gks, gvs);
    look(1);
    for (int j = 0; j < nt; j++) {
      if (!make(j, ck, cv, gks, gvs)) break;
      fetch(j + 1, ck, cv, gks, gvs);
      look(j + 2);
    }
  } else if (warp == C_SOFT) {
    // ================= the products
    if (lane == 0 && nt > 0) {
      // D fp32, A and B fp16; 128 rows; S: 64 slots, O: a block's dimensions, V with the dimensions outermost
      constexpr uint32_t id_s = (1u << 4) | ((CT >> 3) << 17) | ((CR >> 4) << 24);
      constexpr uint32_t id_o = (1u << 4) | (1u << 16) | ((S::WD >> 3) << 17) | ((CR >> 4) << 24);
      bool ok = mbar_wait(q_full, 0, abort_flag, gflags);
      auto issue_pv = [&](int i) -> bool {
        const int u = i & 1;
        if (!mbar_wait(p_full0 + 8 * u, (i >> 1) & 1, abort_flag, gflags)) return false;
        tc_fence_after();
        const uint32_t v = sb + S::KV + (i % S::NS) * S::STAGE + S::NB * S::TB;
#pragma unroll
        for (int nb = 0; nb < S::NB; nb++)
#pragma unroll
          for (int x = S::TERMS - 1; x >= 0; x--)
#pragma unroll
            for (int kk = 0; kk < CT / 16; kk++)
              mma_bf16_ts(tmem + 128 + 64 * nb, tmem + 64 * u + 32 * x + 8 * kk, desc_sw128(v + (x * S::NB + nb) * S::TB + kk * 2048, S::TB, 1024),
                          id_o, ((S::TERMS == 2 ? i % S::FLUSH : i) > 0 || kk > 0 || x < S::TERMS - 1) ? 1u : 0u);
        mma_commit(pv_done0 + 8 * u);
        mma_commit(kv_empty0 + 8 * (i % S::NS));
        return true;
      };
      for (int j = 0; j < nt && ok; j++) {
        const int st = j % S::NS;
        if (!(ok = mbar_wait(kv_full0 + 8 * st, (j / S::NS) & 1, abort_flag, gflags))) break;
        tc_fence_after();
        // S[j & 1] is free: its previous tile's P (j - 2) was waited for below
        const uint32_t k = sb + S::KV + st * S::STAGE;
#pragma unroll
        for (int x = S::TERMS - 1; x >= 0; x--)
#pragma unroll
          for (int nb = 0; nb < S::NB; nb++)
#pragma unroll
            for (int kk = 0; kk < S::WD / 16; kk++)
              mma_bf16_ss(tmem + 64 * (j & 1), desc_sw128(sb + (x * S::NB + nb) * S::QB + kk * 32, 16, 1024),
                          desc_sw128(k + nb * S::TB + kk * 32, 16, 1024), id_s, x < S::TERMS - 1 || nb > 0 || kk > 0);
        mma_commit(s_full0 + 8 * (j & 1));
        if (j >= 1 && !(ok = issue_pv(j - 1))) break;
      }
      if (ok) issue_pv(nt - 1);
    }
    __syncwarp();
  } else {
    // ================= a row a thread
    const int r = tid, rr = row0 + r;
    const bool on = rr < R;
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    float qf = 0.f;
    if (nt > 0) {
      // fp16 after a power of two, as in QFrag
      const T* p = reinterpret_cast<const T*>(at.q) + (on ? (long)(r0 + rr / G) * at.q_ld + (long)(h * G + rr % G) * HD : 0);
      const bool vec = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
      constexpr int EV = 16 / sizeof(T);  // elements of a 16-byte load
      alignas(16) T x[HD];
#pragma unroll
      for (int i = 0; i < HD; i += EV) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on && vec) v = *reinterpret_cast<const uint4*>(p + i);
        *reinterpret_cast<uint4*>(x + i) = v;
        if (on && !vec) {
#pragma unroll
          for (int e = 0; e < EV; e++) x[i + e] = p[i + e];
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < HD; i++) top = fmaxf(top, fabsf(to_f<T>(x[i])));
      const int e = row_exponent(top);
      // the scores' factor has no sign (a maximum may be taken before it): the scale's goes with the row
      const float up = copysignf(kv8_pow2(e), at.scale);
      qf = kv8_pow2(-e) * fabsf(at.scale) * 1.4426950408889634f;
#pragma unroll
      for (int i = 0; i < HD; i += 8) {
        uint32_t f[4], lo[4];
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const float x0 = to_f<T>(x[i + 2 * w]) * up, x1 = to_f<T>(x[i + 2 * w + 1]) * up;
          f[w] = pack_f16(x0, x1);
          if (S::TERMS == 2) lo[w] = pack_rest(x0, x1, f[w]);
        }
        uint8_t* to = smem + (i / 64) * S::QB + half_at<64>(r, i % 64 / 8);
        *reinterpret_cast<uint4*>(to) = make_uint4(f[0], f[1], f[2], f[3]);
        if (S::TERMS == 2) *reinterpret_cast<uint4*>(to + S::NB * S::QB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int see = min(len + min(rr, R - 1) / G + 1, cap);
    float m = -INFINITY, mv = -INFINITY, l = 0.f, l_off = 0.f;
    uint32_t nan_dims[HD / 32];
#pragma unroll
    for (int i = 0; i < HD / 32; i++) nan_dims[i] = 0;
    bool ok = true;
    for (int j = 0; j < nt; j++) {
      const int u = j & 1, st = j % S::NS, base = (t0 + j) * CT;
      if (!(ok = mbar_wait(kv_full0 + 8 * st, (j / S::NS) & 1, abort_flag, gflags))) break;  // the stage's scales
      if (!(ok = mbar_wait(s_full0 + 8 * u, (j >> 1) & 1, abort_flag, gflags))) break;
      tc_fence_after();
      uint32_t v[2][32];
      tmem_ld_32x32b_x32(trow + 64 * u, v[0]);
      tmem_ld_32x32b_x32(trow + 64 * u + 32, v[1]);
      float vl[4], f[4];
      bool all = base + CT <= see;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        vl[g] = sh.vl[st][g];
        // above 0: the scores that the row does not see are -infinity before the factor, and stay so
        f[g] = vl[g] == -INFINITY ? 1.f : fmaxf(qf * sh.ks[st][g], FLT_MIN);
        all &= vl[g] != -INFINITY;
      }
      tmem_ld_wait();
      if (!all) {
#pragma unroll
        for (int i = 0; i < CT; i++)
          if (base + i >= see || vl[i / 16] == -INFINITY) v[i / 32][i % 32] = 0xff800000u;
      }
      float top = -INFINITY, topv = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          x0 = fmaxf(x0, __uint_as_float(v[g / 2][g % 2 * 16 + i]));
          x1 = fmaxf(x1, __uint_as_float(v[g / 2][g % 2 * 16 + i + 1]));
        }
        const float x = fmaxf(x0, x1) * f[g];
        top = fmaxf(top, x);
        topv = fmaxf(topv, x + vl[g]);
      }
      const bool need = top > m + LAZY || topv > mv + LAZY;
      if (__any_sync(0xffffffffu, need)) {
        const float m1 = need ? fmaxf(m, top) : m, mv1 = need ? fmaxf(mv, topv) : mv;
        const float fl = m1 == -INFINITY ? 1.f : sfu_exp2(m - m1), fo = mv1 == -INFINITY ? 1.f : sfu_exp2(mv - mv1);
        m = m1, mv = mv1;
        l *= fl;
        l_off *= fl;
        if (j > 0) {
          // O holds the products of the tiles before.  S of this tile was issued after P V of tile j - 2, so that of
          // tile j - 1 is the only one that may be in flight.
          if (!(ok = mbar_wait(pv_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, abort_flag, gflags))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(trow + 128 + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
            tmem_st_32x32b_x16(trow + 128 + c, o);
          }
          if (S::TERMS == 2 && j > S::FLUSH) {  // the sums of earlier tiles
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(trow + S::SUMS + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
              tmem_st_32x32b_x16(trow + S::SUMS + c, o);
            }
          }
          tmem_st_wait();
        }
      }
      if (S::TERMS == 2 && j > 0 && j % S::FLUSH == 0) {
        if (!(ok = mbar_wait(pv_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, abort_flag, gflags))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HD; c += 16) {
          uint32_t o[16], q[16];
          tmem_ld_32x32b_x16(trow + 128 + c, o);
          if (j > S::FLUSH) tmem_ld_32x32b_x16(trow + S::SUMS + c, q);
          tmem_ld_wait();
          if (j > S::FLUSH) {
#pragma unroll
            for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(q[i]));
          }
          tmem_st_32x32b_x16(trow + S::SUMS + c, o);
        }
        tmem_st_wait();
      }
      float lt = 0.f;  // the tile's sum
      const float mm = m == -INFINITY ? 0.f : m, dv = mm - (mv == -INFINITY ? 0.f : mv);
#pragma unroll
      for (int half = 0; half < 2; half++) {
        uint32_t pk[16], pl[16];
#pragma unroll
        for (int g = 0; g < 2; g++) {
          const float c = v_factor(vl[2 * half + g] + dv);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float e0 = sfu_exp2(fmaf(__uint_as_float(v[half][16 * g + i]), f[2 * half + g], -mm));
            const float e1 = sfu_exp2(fmaf(__uint_as_float(v[half][16 * g + i + 1]), f[2 * half + g], -mm));
            lt += e0 + e1;
            pk[8 * g + i / 2] = pack_f16(e0 * c, e1 * c);
            if (S::TERMS == 2) pl[8 * g + i / 2] = pack_p_rest(e0 * c, e1 * c, pk[8 * g + i / 2]);
          }
        }
        // over the scores, which have been read: the A operand of P V (fp32 rows: its second terms behind it)
        tmem_st_32x32b_x16(trow + 64 * u + 16 * half, pk);
        if (S::TERMS == 2) tmem_st_32x32b_x16(trow + 64 * u + 32 + 16 * half, pl);
      }
      add_kept(l, l_off, lt);
      tmem_st_wait();
      bool nan = false;
#pragma unroll
      for (int i = 0; i < S::MAKE; i++) nan |= sh.nan[st][i] != 0;
      if (nan) {
        for (int i = 0; i < CT && base + i < see; i++) {
          const int b = ids[(base + i) >> a.lgP];
          if ((unsigned)b >= (unsigned)a.n_blocks) continue;
          const uint8_t* c = a.v + ((((size_t)b * a.H + h) << a.lgP) + ((base + i) & (a.P - 1))) * HD;
#pragma unroll
          for (int d = 0; d < HD; d++)
            if ((c[d] & 0x7f) == 0x7f) nan_dims[d / 32] |= 1u << d % 32;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full0 + 8 * u);
    }
    // the last two products may both be in flight
    if (ok && nt > 1) ok = mbar_wait(pv_done0 + 8 * (nt & 1), ((nt - 2) >> 1) & 1, abort_flag, gflags);
    if (ok && nt > 0) ok = mbar_wait(pv_done0 + 8 * ((nt - 1) & 1), ((nt - 1) >> 1) & 1, abort_flag, gflags);
    tc_fence_after();
    __syncwarp();
    float* part = reinterpret_cast<float*>(smem) + r * S::PITCH;
#pragma unroll
    for (int c = 0; c < HD; c += 16) {
      uint32_t o[16];
#pragma unroll
      for (int i = 0; i < 16; i++) o[i] = 0;
      if (nt > 0) {  // (the same for all threads)
        tmem_ld_32x32b_x16(trow + 128 + c, o);
        tmem_ld_wait();
        if (S::TERMS == 2 && nt > S::FLUSH) {
          uint32_t q[16];
          tmem_ld_32x32b_x16(trow + S::SUMS + c, q);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(q[i]));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; i++)
        if (nan_dims[(c + i) / 32] >> (c + i) % 32 & 1u) o[i] = 0x7fc00000u;
      // every row's products are done (each thread has waited for the last), so that the tiles' place is free
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(part + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
    sh.stats.m[r] = m, sh.stats.mv[r] = mv, sh.stats.l[r] = l - l_off;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C_SOFT) tmem_dealloc(tmem, S::COLS);
  join_blocks<T, HD, CR, S::PITCH, (TcShape<T, HD>::THREADS)>(sh.stats, reinterpret_cast<float*>(smem), n_split, split, min(CR, R - row0), at,
                                                 r0, row0, h, a.H * G);
}

// ---------------------------------------------------------------- accumulation of the weights

// weight[slot] += sum over the rows of exp(score - lse): the QK product again,
// now with the rows' final statistics, so that a slot's sum is formed by one
// warp in a fixed order.  Here (many rows) a warp holds the codes of 32 slots as
// the product's 16-row operand, converted once, and all rows pass by: 64 at a
// time as fp16 in shared memory, made once for the block's four warps while the
// tile before is used.  k_kv8_accumulate_few has the rows in registers.
//
// B200, 63 to 200 rows over up to 1501 slots, 4 sequences of 25 heads of 64: 17.6 us
// (fp32 29 us) on a floor of 1.3; 130 rows over 3000 slots, 6 sequences of 8 heads
// of 128: 59 us (fp32 110 us) on 3.5.  Bound by the warp MMA and what feeds it: the
// pipe is 20 to 28% busy, every block scales and converts all rows of q again, and
// the rows are not divided over blocks (500 rows on one head of 128 dimensions,
// 3000 slots: 24 blocks, 21 us, fp32 46 us).
constexpr int AR = 64, AT = 128;  // rows a tile, slots a block

// Where dimension d of a row lies so that the 16 x 8 x 16 MMA, which takes a row's halves in order, meets the
// dimensions that a lane's codes have (QFrag::dim0)
template <int HD>
__device__ __forceinline__ constexpr int half_place(int d) {
  const int t = HD == 32 ? d / 8 : d % 64 / 16, ks = HD == 32 ? d % 8 / 4 : d / 64 * 4 + d % 16 / 4, j = d % 4;
  return ks * 16 + 2 * t + (j & 1) + (j >> 1) * 8;
}

template <typename T, int HD, int MINB>
__global__ void __launch_bounds__(128, MINB) k_kv8_accumulate_many(Kv8Args a, AttnArgs at) {
  constexpr int KS = HD / 16, TERMS = sizeof(T) == 4 ? 2 : 1, DPT = HD / 2;  // dimensions of a row that a thread brings
  constexpr int TILE = AR * HD * 2;
  extern __shared__ __align__(16) uint8_t smem[];  // [2][TERMS][AR][HD] fp16
  __shared__ float r_f[2][AR], r_ls[2][AR];
  __shared__ int r_see[2][AR];
  const int h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s), G = at.G, R = n * G;
  const int cap = a.max_blocks << a.lgP, see_hi = min(len + n, cap);
  if (n == 0) return;
  const T* qs = reinterpret_cast<const T*>(at.q) + (long)r0 * at.q_ld + (long)h * G * HD;
  const bool vec = ((reinterpret_cast<uintptr_t>(qs) | (uintptr_t)(at.q_ld * (long)sizeof(T))) & 15) == 0;
  // the lane's offsets into a tile for ldmatrix; eight rows on, they are the same but for the rows' bytes
  uint32_t q_off[KS / 2];
#pragma unroll
  for (int ks = 0; ks < KS; ks += 2) q_off[ks / 2] = half_at<HD>(lane & 7, 2 * ks + (lane >> 3));

  // ---- half a row a thread: asked for, then written as fp16 after a power of two, as in QFrag
  alignas(16) T raw[DPT];
  float lse_raw = 0.f;
  const int my = tid >> 1, d0 = (tid & 1) * DPT;
  auto ask = [&](int row0) {
    const int r = row0 + my;
    const T* p = qs + (r < R ? (long)(r / G) * at.q_ld + (r % G) * HD + d0 : 0);
    constexpr int VEC = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < DPT; i += VEC) {
      if (vec) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < R) x = *reinterpret_cast<const uint4*>(p + i);
        *reinterpret_cast<uint4*>(raw + i) = x;
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          raw[i + j] = from_f<T>(0.f);
          if (r < R) raw[i + j] = p[i + j];
        }
      }
    }
    if (!(tid & 1) && r < R) lse_raw = at.lse[(long)(r0 + r / G) * (a.H * G) + h * G + r % G];
  };
  auto put = [&](int row0, int buf) {
    const int r = row0 + my;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < DPT; i++) top = fmaxf(top, fabsf(to_f<T>(raw[i])));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const int e = row_exponent(top);
    const float up = kv8_pow2(e);
    uint8_t* to = smem + buf * TERMS * TILE;
#pragma unroll
    for (int i = 0; i < DPT; i += 2) {
      const float lo = to_f<T>(raw[i]) * up, hi = to_f<T>(raw[i + 1]) * up;
      const uint32_t v = pack_f16(lo, hi);
      // (half a row of dimensions is half of the places of each step: d0 moves t by two)
      const int place = half_place<HD>(i) + (HD == 128 ? (tid & 1) * 64 : (tid & 1) * 4);
      const uint32_t off = half_at<HD>(my, place >> 3) + (place & 7) * 2;
      *reinterpret_cast<uint32_t*>(to + off) = v;
      if (TERMS == 2) *reinterpret_cast<uint32_t*>(to + TILE + off) = pack_rest(lo, hi, v);
    }
    if (!(tid & 1)) {
      const bool on = r < R && lse_raw != -INFINITY;  // else: no row, or one without weights
      r_f[buf][my] = kv8_pow2(-e) * at.scale * 1.4426950408889634f;
      r_ls[buf][my] = on ? lse_raw * 1.4426950408889634f : 0.f;
      r_see[buf][my] = on ? min(len + r / G + 1, cap) : 0;
    }
  };

  // the grid covers the caller's bound on the lengths; a longer sequence takes its blocks further
  for (long first = (long)blockIdx.x * AT; first < see_hi; first += (long)gridDim.x * AT) {
    const int base = (int)first + w * 32;  // the warp's slots
    // rows before this one see nothing of the block's slots
    const int start = (int)(max(0L, first - len) * G / AR) * AR;
    ask(start);
    uint32_t ka[2][KS][4];
    int blk[2];
    float ks[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int j0 = base + x * 16;
      blk[x] = j0 < see_hi ? kv8_block(a, s, j0 >> a.lgP) : -1;
      const size_t bh = (size_t)max(blk[x], 0) * a.H + h;
      ks[x] = blk[x] >= 0 ? a.ks[bh] : 0.f;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int j = j0 + g + 8 * half;
        const uint8_t* p = a.k + ((bh << a.lgP) + (j & (a.P - 1))) * HD;
        const bool on = blk[x] >= 0 && j < see_hi;
        uint32_t kw[KS];
        if (HD == 32) {
          const uint2 c = on ? *reinterpret_cast<const uint2*>(p + t * 8) : make_uint2(0, 0);
          kw[0] = c.x, kw[1] = c.y;
        } else {
#pragma unroll
          for (int i = 0; i < HD / 64; i++) {
            const uint4 c = on ? *reinterpret_cast<const uint4*>(p + i * 64 + t * 16) : make_uint4(0, 0, 0, 0);
            kw[(4 * i) % KS] = c.x, kw[(4 * i + 1) % KS] = c.y, kw[(4 * i + 2) % KS] = c.z, kw[(4 * i + 3) % KS] = c.w;
          }
        }
#pragma unroll
        for (int k = 0; k < KS; k++) {
          ka[x][k][half] = f16x2_e4m3(kw[k]);
          ka[x][k][2 + half] = f16x2_e4m3(kw[k] >> 16);
        }
      }
    }
    float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    int buf = 0;
    __syncthreads();  // every warp is done with the tiles of the slots before
    for (int row0 = start; row0 < R; row0 += AR, buf ^= 1) {
      put(row0, buf);
      __syncthreads();
      if (row0 + AR < R) ask(row0 + AR);
      const int last = min(R - 1, row0 + AR - 1);
      if (base >= min(len + last / G + 1, cap)) continue;  // no row of these sees the warp's slots
      const bool full = row0 + AR <= R && base + 32 <= min(len + row0 / G + 1, cap);
      const uint32_t qb = (uint32_t)__cvta_generic_to_shared(smem) + buf * TERMS * TILE;
#pragma unroll
      for (int nt = 0; nt < AR / 8; nt++) {
        float d[2][4];
#pragma unroll
        for (int x = 0; x < 2; x++) d[x][0] = d[x][1] = d[x][2] = d[x][3] = 0.f;
#pragma unroll
        for (int term = 0; term < TERMS; term++)
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t b[4];
            ldsm4(b, qb + term * TILE + q_off[k / 2] + nt * 16 * HD);
#pragma unroll
            for (int x = 0; x < 2; x++) {
              if (TERMS == 1) {
                mma(d[x], ka[x][k][0], ka[x][k][1], ka[x][k][2], ka[x][k][3], b[0], b[1]);
                mma(d[x], ka[x][k + 1][0], ka[x][k + 1][1], ka[x][k + 1][2], ka[x][k + 1][3], b[2], b[3]);
              } else {
                Exact e0, e1;
                mma(e0.x, ka[x][k][0], ka[x][k][1], ka[x][k][2], ka[x][k][3], b[0], b[1]);
                mma(e1.x, ka[x][k + 1][0], ka[x][k + 1][1], ka[x][k + 1][2], ka[x][k + 1][3], b[2], b[3]);
                e0.add_to(d[x]);
                e1.add_to(d[x]);
              }
            }
          }
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int r = 8 * nt + 2 * t + e;
          const float f = r_f[buf][r], ls = r_ls[buf][r];
          const int see = r_see[buf][r];
#pragma unroll
          for (int x = 0; x < 2; x++) {
            const float fk = f * ks[x];
#pragma unroll
            for (int half = 0; half < 2; half++) {
              const float p = sfu_exp2(fmaf(d[x][2 * half + e], fk, -ls));
              sum[x][half] += (full ? see > 0 : base + x * 16 + g + 8 * half < see) ? p : 0.f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
#pragma unroll
      for (int half = 0; half < 2; half++) {
        sum[x][half] += __shfl_xor_sync(0xffffffffu, sum[x][half], 1);
        sum[x][half] += __shfl_xor_sync(0xffffffffu, sum[x][half], 2);
      }
      // one of the four lanes that hold a sum adds it (atomically: two sequences may share a block)
      const int j = base + x * 16 + g + 8 * (t & 1);
      if (t < 2 && j < see_hi && blk[x] >= 0)
        atomicAdd(a.w + ((((size_t)blk[x] * a.H + h) << a.lgP) + (j & (a.P - 1))), t ? sum[x][1] : sum[x][0]);
    }
  }
}

// At most 8 NT rows (a decoding step): their operand is made once, and each warp
// of a (sequence, head) takes every so-manieth tile of 32 tokens, with the next
// tile's codes on their way and the block ids of the one behind it looked up.
// B200: long contexts (as k_kv8_attn's) 38.5 us, 79% of the copy bandwidth (fp32
// rows 43 us); the batch 13 us (4.8 us at the copy bandwidth; fp32 15 us): 4 us
// before the first tile, then uneven work as k_kv8_attn's.
template <typename T, int HD, int NT, int MINB>
__global__ void __launch_bounds__(128, MINB) k_kv8_accumulate_few(Kv8Args a, AttnArgs at) {
  constexpr int KS = HD / 16;
  const int h = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warps = gridDim.x * 4, first = blockIdx.x * 4 + (threadIdx.x >> 5);
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s), G = at.G, R = n * G;
  const int cap = a.max_blocks << a.lgP, see_hi = min(len + n, cap);
  if (n == 0) return;

  auto look = [&](int tile, int (&b)[2]) {
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      const int j = tile * TT + gr * 16;
      b[gr] = -1;
      if (j < see_hi) b[gr] = a.table[(size_t)s * a.max_blocks + (j >> a.lgP)];  // first touched when it is fetched
    }
  };
  auto fetch = [&](int tile, const int (&b)[2], uint32_t (&kw)[2][2][KS], float (&ks)[2]) {
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      const bool there = (unsigned)b[gr] < (unsigned)a.n_blocks;
      const size_t bh = (size_t)(there ? b[gr] : 0) * a.H + h;
      ks[gr] = there ? a.ks[bh] : 0.f;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int j = tile * TT + gr * 16 + key_token(g, half);
        const uint8_t* p = a.k + ((bh << a.lgP) + (j & (a.P - 1))) * HD;
        const bool on = there && j < see_hi;
        if (HD == 32) {
          const uint2 c = on ? *reinterpret_cast<const uint2*>(p + t * 8) : make_uint2(0, 0);
          kw[gr][half][0] = c.x, kw[gr][half][1] = c.y;
        } else {
#pragma unroll
          for (int i = 0; i < HD / 64; i++) {
            const uint4 c = on ? *reinterpret_cast<const uint4*>(p + i * 64 + t * 16) : make_uint4(0, 0, 0, 0);
            kw[gr][half][(4 * i) % KS] = c.x, kw[gr][half][(4 * i + 1) % KS] = c.y;
            kw[gr][half][(4 * i + 2) % KS] = c.z, kw[gr][half][(4 * i + 3) % KS] = c.w;
          }
        }
      }
    }
  };
  uint32_t kw[2][2][KS];
  float ks[2];
  int blk[2], ahead[2];
  look(first, blk);
  look(first + warps, ahead);
  fetch(first, blk, kw, ks);
  QFrag<T, HD, NT> q;
  q.load(reinterpret_cast<const T*>(at.q) + (long)r0 * at.q_ld + h * G * HD, at.q_ld, G, 0, R, at.scale);
  float ls[NT][2];
  int see[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int r = 8 * nt + 2 * t + e, i = min(r, R - 1) / G;
      see[nt][e] = r < R ? min(len + i + 1, cap) : 0;  // rows past the last see nothing
      const float x = r < R ? at.lse[(long)(r0 + i) * (a.H * G) + h * G + r % G] : 0.f;
      if (x == -INFINITY) see[nt][e] = 0;  // a row without weights
      ls[nt][e] = x * 1.4426950408889634f;
    }

  for (int tile = first; tile * TT < see_hi; tile += warps) {
    uint32_t kn[2][2][KS];
    float kns[2];
    const int now[2] = {blk[0], blk[1]};
    fetch(tile + warps, ahead, kn, kns);
    blk[0] = ahead[0], blk[1] = ahead[1];
    look(tile + 2 * warps, ahead);
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      float d[NT][4], sum[2] = {0.f, 0.f};
      q.qk(d, kw[gr][0], kw[gr][1]);
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const int j = tile * TT + gr * 16 + key_token(g, half);
#pragma unroll
          for (int e = 0; e < 2; e++)
            sum[half] += j < see[nt][e] ? sfu_exp2(d[nt][2 * half + e] * (q.f[nt][e] * ks[gr]) - ls[nt][e]) : 0.f;
        }
#pragma unroll
      for (int half = 0; half < 2; half++) {
        sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
        sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
      }
      const bool there = (unsigned)now[gr] < (unsigned)a.n_blocks;
      if (!there && lane == 0 && tile * TT + gr * 16 < see_hi) kv8_flag(a, FLAG_BLOCK);
      // one of the four lanes that hold a sum adds it (atomically: two sequences may share a block)
      const int j = tile * TT + gr * 16 + key_token(g, t & 1);
      if (t < 2 && j < see_hi && there)
        atomicAdd(a.w + ((((size_t)now[gr] * a.H + h) << a.lgP) + (j & (a.P - 1))), t ? sum[1] : sum[0]);
    }
#pragma unroll
    for (int gr = 0; gr < 2; gr++) {
      ks[gr] = kns[gr];
#pragma unroll
      for (int half = 0; half < 2; half++)
#pragma unroll
        for (int i = 0; i < KS; i++) kw[gr][half][i] = kn[gr][half][i];
    }
  }
}

// The widest cluster to be asked for.  More than 8 blocks, only for few clusters: see launch_split.
int widest(double blocks) { return blocks <= 18.0 ? MAX_SPLIT : 8; }

// few blocks: the slots of each are split over a cluster, each with `least` tiles or more
int split_of(const Ctx& c, long blocks, long resident, long tiles, long least) {
  const long want = (resident * c.num_sms + blocks - 1) / blocks, most = (tiles + least - 1) / least;
  const long split = want < most ? want : most;
  return (int)(split < 1 ? 1 : split > widest(blocks) ? widest(blocks) : split);
}

// How many clusters of `split` blocks the current device runs at once: asked of the driver once for each.
template <auto Kernel>
int active_clusters(int split, cudaLaunchConfig_t cfg) {
  static std::atomic<int> known[8][MAX_SPLIT + 1];  // number + 1
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 8 && (n = known[dev][split].load(std::memory_order_relaxed)) > 0) return n - 1;
  cfg.gridDim.x = split;
  if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) return 0;
  if (dev < 8) known[dev][split].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <auto Kernel>
bool launch_split(Ctx& c, const Kv8Args& a, AttnArgs at, int split, long row_tiles, int threads, size_t smem) {
  if (!allow_smem<Kernel>((int)smem, split > 8)) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, a.H, a.S);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // A cluster takes its SMs from one GPC, so that wide ones leave SMs over and may not all run at once: 8 heads of 128,
  // 30000 slots, took 24.4 us in clusters of 10 and 41.5 us, in two waves, in clusters of 12.
  for (; split > 8 && active_clusters<Kernel>(split, cfg) < a.S * a.H * row_tiles; split--) attr[0].val.clusterDim.x = split - 1;
  at.n_split = split;
  cfg.gridDim.x = (unsigned)(split * row_tiles);
  return cudaLaunchKernelEx(&cfg, Kernel, a, at) == cudaSuccess;
}

template <typename T, int HD, int NT, int NS, int MINB, int NW = 4>
bool launch_attn(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  constexpr int ROWS = 8 * NT;
  constexpr size_t ring = sizeof(Stage<HD>) * NW * NS, join = (size_t)(NW * ROWS * (HD + 4) + ROWS * HD) * 4;
  const long row_tiles = ((long)a.max_new * at.G + ROWS - 1) / ROWS;
  const int split = split_of(c, (long)a.S * a.H * row_tiles, MINB, (max_len + TT - 1) / TT, NW);
  return launch_split<k_kv8_attn<T, HD, NT, NW, NS, MINB>>(c, a, at, split, row_tiles, NW * 32, ring > join ? ring : join);
}

template <typename T, int HD, int MINB>
bool launch_attn_many(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  constexpr size_t tiles = sizeof(HalfTile<HD>) * 2, join = (size_t)MR * (HD + 4) * 4;
  const long row_tiles = ((long)a.max_new * at.G + MR - 1) / MR;
  const int split = split_of(c, (long)a.S * a.H * row_tiles, MINB, (max_len + MT - 1) / MT, 2);
  return launch_split<k_kv8_attn_many<T, HD, MINB>>(c, a, at, split, row_tiles, MW * 32, tiles > join ? tiles : join);
}

template <typename T, int HD>
bool launch_attn_tc(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  const long row_tiles = ((long)a.max_new * at.G + CR - 1) / CR;
  // Blocks that have rows, about half a tile a sequence above the rows' own; two are resident an SM.  A block costs its
  // tiles and about six more; blocks that do not fit at once cost a part of a wave beside their share.
  const double tiles = (max_len + CT - 1) / CT, places = (double)TcShape<T, HD>::MINB * c.num_sms;
  const double blocks = a.H * fmin((double)a.S * row_tiles, (double)a.n_rows * at.G / CR + 0.5 * a.S);
  int split = 1;
  double best = 0.0;
  for (int i = 1; i <= widest((double)a.S * a.H * row_tiles) && (i == 1 || 2 * i <= tiles); i++) {
    const double waves = blocks * i / places, cost = (waves <= 1.0 ? 1.0 : waves + 0.4) * (tiles / i + 6.0);
    if (i == 1 || cost < best) best = cost, split = i;
  }
  return launch_split<k_kv8_attn_tc<T, HD>>(c, a, at, split, row_tiles, (TcShape<T, HD>::THREADS), 1024 + TcShape<T, HD>::END + sizeof(TcShared));
}

template <typename T, int HD>
bool launch_attn_rows(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  const long rows = (long)a.max_new * at.G;
  // Stages a warp and blocks an SM, by trial: with 64 dimensions and 8 rows two stages and five blocks took 21.3 us for
  // 64 sequences of 12 heads, three and four 24.5 us.
  constexpr int NS = HD == 32 ? 4 : 2;
  // heads and sequences that even clusters of 8 leave SMs without a block: eight warps a block
  const long pairs = (long)a.S * a.H;
  if (rows <= 8 && pairs * 8 <= c.num_sms) return launch_attn<T, HD, 1, NS, 1, 8>(c, a, at, max_len);
  if (rows <= 8) return launch_attn<T, HD, 1, NS, HD == 128 ? 3 : HD == 64 && sizeof(T) == 2 ? 5 : 4>(c, a, at, max_len);
  if (rows <= 16) return launch_attn<T, HD, 2, NS, HD == 128 ? 2 : sizeof(T) == 2 ? 4 : 3>(c, a, at, max_len);
  // By trial (warp MMA's blocks of 64 rows against tcgen05): 20 to 48 rows of 64 or fewer dimensions mostly take less with
  // the former (bf16, 4 sequences of 25 heads of 64, 32 rows 24 us against 29; 2 of 8 heads of 32 12.6 against 18.3; but 30 of
  // 8 heads of 64 34 against 32), fp32 rows to 64, one block, where there are few blocks (one sequence of 12 heads 28 us
  // against 30, 2 of 8 heads of 32 15.5 against 23.1; 30 of 8 heads 55 against 46).  Above, and of 128 dimensions, tcgen05
  // takes less (100 rows of 30 sequences of 8 heads of 64: bf16 36 us against 63, fp32 52 against 98).
  if constexpr (HD == 128) {
    return launch_attn_tc<T, HD>(c, a, at, max_len);
  } else {
    if (rows > (sizeof(T) == 4 ? 64 : 48)) return launch_attn_tc<T, HD>(c, a, at, max_len);
    return launch_attn_many<T, HD, sizeof(T) == 4 ? 2 : 3>(c, a, at, max_len);
  }
}

template <typename T, int HD>
bool launch_accumulate_many(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  constexpr int TERMS = sizeof(T) == 4 ? 2 : 1, SMEM = 2 * TERMS * AR * HD * 2, MINB = HD == 128 ? 2 : sizeof(T) == 4 ? 3 : 4;
  constexpr auto kernel = k_kv8_accumulate_many<T, HD, MINB>;
  if (!allow_smem<kernel>(SMEM)) return false;
  kernel<<<dim3((max_len + AT - 1) / AT, a.H, a.S), 128, SMEM, c.stream>>>(a, at);
  return true;
}
template <typename T, int HD, int NT>
bool launch_accumulate_few(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  constexpr int MINB = HD == 128 ? (NT == 1 ? 4 : 3) : NT == 1 ? 6 : 4;
  // a warp for every two tiles, but no more blocks than the GPU holds at once
  const long tiles = (max_len + TT - 1) / TT, most = (tiles + 7) / 8, pairs = (long)a.H * a.S;
  long split = (long)MINB * c.num_sms / pairs;
  split = split > most ? most : split < 1 ? 1 : split;
  k_kv8_accumulate_few<T, HD, NT, MINB><<<dim3((unsigned)split, a.H, a.S), 128, 0, c.stream>>>(a, at);
  return true;
}
template <typename T, int HD>
bool launch_accumulate_rows(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  const long rows = (long)a.max_new * at.G;
  if (rows <= 8) return launch_accumulate_few<T, HD, 1>(c, a, at, max_len);
  if (rows <= 16) return launch_accumulate_few<T, HD, 2>(c, a, at, max_len);
  return launch_accumulate_many<T, HD>(c, a, at, max_len);
}

}  // namespace

bool kv8_attention(Ctx& c, const Kv8Args& a, int hd, int G, bool bf16_rows, const void* q, long q_ld, float scale,
                   int max_len, void* o, long o_ld, float* lse) {
  LaunchScope s(c, "kv8_attention");
  AttnArgs at{q, q_ld, scale, G, 0, o, o_ld, lse};
  if (bf16_rows) {
    if (hd == 32) return launch_attn_rows<bf16, 32>(c, a, at, max_len);
    if (hd == 64) return launch_attn_rows<bf16, 64>(c, a, at, max_len);
    return launch_attn_rows<bf16, 128>(c, a, at, max_len);
  }
  if (hd == 32) return launch_attn_rows<float, 32>(c, a, at, max_len);
  if (hd == 64) return launch_attn_rows<float, 64>(c, a, at, max_len);
  return launch_attn_rows<float, 128>(c, a, at, max_len);
}

bool kv8_accumulate(Ctx& c, const Kv8Args& a, int hd, int G, bool bf16_rows, const void* q, long q_ld, float scale,
                    int max_len, const float* lse) {
  LaunchScope s(c, "kv8_accumulate");
  AttnArgs at{q, q_ld, scale, G, 0, nullptr, 0, const_cast<float*>(lse)};
  if (bf16_rows) {
    if (hd == 32) return launch_accumulate_rows<bf16, 32>(c, a, at, max_len);
    if (hd == 64) return launch_accumulate_rows<bf16, 64>(c, a, at, max_len);
    return launch_accumulate_rows<bf16, 128>(c, a, at, max_len);
  }
  if (hd == 32) return launch_accumulate_rows<float, 32>(c, a, at, max_len);
  if (hd == 64) return launch_accumulate_rows<float, 64>(c, a, at, max_len);
  return launch_accumulate_rows<float, 128>(c, a, at, max_len);
}

}  // namespace gpt
