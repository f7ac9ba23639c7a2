// Attention over the 8-bit key / value cache, and the accumulation of its
// weights (which eviction goes by).
//
//   o_r = sum_j softmax_j(scale q_r k_j) v_j   over the slots j that row r sees
//
// Row r = (new token i, query head) of a sequence with len tokens before this
// step sees slots 0 .. len + i.  With G query heads to a key / value head, the
// n G rows that share one are taken 16 at a time as the 16 rows of the
// 16 x 8 x 16 warp MMA: each cached byte is read once for all of them.  Codes
// become fp16 by one exact conversion for two of them; the MMA takes the
// multiply-adds, so that at one row (most of the MMA empty) as at sixteen the
// kernel is bound by reading the cache.
//
// The order of a dot product's terms and of a sum's is free, which the operand
// layouts use: lane (g, t) of the QK product takes a contiguous quarter of key
// g's row, and lane (g, t) of the PV product a contiguous eighth of the rows of
// four tokens; neither needs a transposition.
#include <cooperative_groups.h>

#include "kv8.cuh"

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
// the parts of (lo, hi) that pack_f16 rounded off, as fp16
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t p) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
  return pack_f16(lo - f.x, hi - f.y);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows of q as the A operand of the QK product.  bf16 rows are exact in fp16
// once a power of two has brought the row's largest magnitude to 2^14 .. 2^15
// (what falls below fp16's range then is under 2^-38 of it); fp32 rows take two
// fp16 terms, 22 bits, which leaves less than the fp32 sum of the products does.
template <typename T, int HD, bool R8>
struct QFrag {
  static constexpr int KS = HD / 16;
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  uint32_t a[TERMS][KS][R8 ? 2 : 4];
  float f0, f1;  // of rows g and g + 8: what a score has to be multiplied by to be scale * q k * log2(e)

  // first dimension of the four codes that lane t feeds to step ks
  static __device__ __forceinline__ int dim0(int t, int ks) {
    if (HD == 32) return t * 8 + 4 * ks;
    return (ks / 4) * 64 + t * 16 + (ks % 4) * 4;
  }

  __device__ void load(const T* __restrict__ q, long q_ld, int hd_row, int G, int row0, int R, float scale) {
    // row r: token r / G, head r % G; hd_row: first element of the group's heads in a row of q
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int half = 0; half < (R8 ? 1 : 2); half++) {
      const int r = row0 + g + 8 * half;
      const bool on = r < R;
      const T* p = q + (on ? (long)(r / G) * q_ld + hd_row + (r % G) * HD : 0);
      float x[KS][4];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          x[ks][j] = on ? to_f<T>(p[dim0(t, ks) + j]) : 0.f;
          top = fmaxf(top, fabsf(x[ks][j]));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = top > 0.f && top < INFINITY ? 14 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
      e = min(max(e, -100), 100);
      const float f = kv8_pow2(e);
      (half ? f1 : f0) = kv8_pow2(-e) * scale * 1.4426950408889634f;
#pragma unroll
      for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float lo = x[ks][2 * j] * f, hi = x[ks][2 * j + 1] * f;
          const uint32_t v = pack_f16(lo, hi);
          a[0][ks][R8 ? j : 2 * j + half] = v;
          if (TERMS == 2) a[TERMS - 1][ks][R8 ? j : 2 * j + half] = pack_rest(lo, hi, v);
        }
    }
    if (R8) f1 = 0.f;
  }

  // d += q k^T for eight keys; w: the lane's quarter of its key's codes
  __device__ __forceinline__ void qk(float (&d)[4], const uint32_t (&w)[KS]) const {
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
      const uint32_t b0 = f16x2_e4m3(w[ks]), b1 = f16x2_e4m3(w[ks] >> 16);
#pragma unroll
      for (int m = 0; m < TERMS; m++) {
        if (R8)
          mma(d, a[m][ks][0], 0u, a[m][ks][1], 0u, b0, b1);
        else
          mma(d, a[m][ks][0], a[m][ks][1], a[m][ks][R8 ? 0 : 2], a[m][ks][R8 ? 0 : 3], b0, b1);
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

// The token, within its 16, of column 2 t + e of the group's n-tile nt: lane t
// then owns tokens t, t + 4, t + 8, t + 12, in the order that the PV product's
// operands need them.
__device__ __forceinline__ int col_token(int t, int nt, int e) { return t + 4 * (e + 2 * nt); }
// ... and the token of key column g of n-tile nt
__device__ __forceinline__ int key_token(int g, int nt) { return (g >> 1) + 4 * ((g & 1) + 2 * nt); }

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

// One thread block (NW warps): 16 rows (8 with R8) of one key / value head of
// one sequence, over one of the cluster's equal parts of the slots.  Each warp
// takes every NW-th tile of 32 tokens through its own ring of NS stages
// (cp.async, no block-wide barrier in the loop) with its own running maxima and
// sums; the warps, then the cluster's blocks through distributed shared memory,
// are joined at the end in a fixed order.
template <typename T, int HD, bool R8, int NW, int NS>
__global__ void __launch_bounds__(NW * 32) k_kv8_attn(Kv8Args a, AttnArgs at) {
  constexpr int ROWS = R8 ? 8 : 16;
  constexpr int NH = R8 ? 1 : 2;      // row halves a lane holds
  constexpr int BPL = HD / 8;         // dimensions a lane loads of a V row
  constexpr int OP = HD + 4;          // pitch of a row of partial outputs
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float st_m[NW][ROWS], st_mv[NW][ROWS], st_l[NW][ROWS];
  __shared__ float cl_m[ROWS], cl_mv[ROWS], cl_l[ROWS];

  const int n_split = at.n_split, split = blockIdx.x % n_split, rt = blockIdx.x / n_split;
  const int h = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s), G = at.G;
  const int R = n * G, row0 = rt * ROWS;
  if (row0 >= R) return;  // the same for every block of the cluster
  const int cap = a.max_blocks << a.lgP;
  const int i_lo = row0 / G, i_hi = min(R - 1, row0 + ROWS - 1) / G;
  const int see_lo = min(len + i_lo + 1, cap), see_hi = min(len + i_hi + 1, cap);
  // visible slots of rows g and g + 8
  const int see[2] = {min(len + min(row0 + g, R - 1) / G + 1, cap), min(len + min(row0 + g + 8, R - 1) / G + 1, cap)};

  QFrag<T, HD, R8> q;
  q.load(reinterpret_cast<const T*>(at.q) + (long)r0 * at.q_ld, at.q_ld, h * G * HD, G, row0, R, at.scale);

  float o[BPL][4];
#pragma unroll
  for (int j = 0; j < BPL; j++)
#pragma unroll
    for (int i = 0; i < 4; i++) o[j][i] = 0.f;
  // per row: running maximum of the scores (log2), that of scores + log2(V scale), and the sum of 2^(score - m)
  float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const int tiles = (see_hi + TT - 1) / TT;
  const int per = (tiles + n_split - 1) / n_split;
  const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);
  Stage<HD>* ring = reinterpret_cast<Stage<HD>*>(smem) + w * NS;

  // block ids of the next tile to be requested, looked up one tile ahead
  int b0 = -1, b1 = -1;
  auto look = [&](int tile) {
    b0 = b1 = -1;
    if (tile < t1) {
      b0 = kv8_block(a, s, (tile * TT) >> a.lgP);
      const int j1 = (tile * TT + 16) >> a.lgP;
      b1 = tile * TT + 16 < see_hi ? (j1 == (tile * TT) >> a.lgP ? b0 : kv8_block(a, s, j1)) : -1;
    }
  };
  auto request = [&](int tile, int slot) {
    if (tile < t1) {
      Stage<HD>& st = ring[slot];
      const int base = tile * TT;
      const size_t p0 = ((size_t)max(b0, 0) * a.H + h), p1 = ((size_t)max(b1, 0) * a.H + h);
      const uint32_t sk = (uint32_t)__cvta_generic_to_shared(st.k), sv = (uint32_t)__cvta_generic_to_shared(st.v);
      constexpr int CPR = HD / 16;
#pragma unroll
      for (int u = 0; u < CPR; u++) {
        const int idx = u * 32 + lane, row = idx / CPR, ch = idx % CPR;
        const int j = base + row;
        const bool second = row >= 16;
        const bool on = j < see_hi && (second ? b1 : b0) >= 0;
        const size_t src = on ? ((second ? p1 : p0) * a.P + (j & (a.P - 1))) * HD + ch * 16 : 0;
        const uint32_t dst = tile_at<HD>(row, ch);
        cp16(sk + dst, a.k + src, on);
        cp16(sv + dst, a.v + src, on);
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
  look(next);
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

    // ---- scores of 4 x 8 keys
    float sc[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; nt++) {
      const int row = (nt >> 1) * 16 + key_token(g, nt & 1);
      uint32_t kw[HD / 16];
      if (HD == 32) {
        const uint2 x = *reinterpret_cast<const uint2*>(st.k + tile_at<HD>(row, t >> 1) + (t & 1) * 8);
        kw[0] = x.x, kw[1] = x.y;
      } else {
#pragma unroll
        for (int c = 0; c < HD / 64; c++) {
          const uint4 x = *reinterpret_cast<const uint4*>(st.k + tile_at<HD>(row, c * 4 + t));
          kw[(4 * c) % (HD / 16)] = x.x, kw[(4 * c + 1) % (HD / 16)] = x.y;
          kw[(4 * c + 2) % (HD / 16)] = x.z, kw[(4 * c + 3) % (HD / 16)] = x.w;
        }
      }
      sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      q.qk(sc[nt], kw);
    }
    const int ok = st.ok;
    const bool full = tile * TT + TT <= see_lo && ok == 3;
    const float k0 = st.ks[0], k1 = st.ks[1];
    // log2 of the V scales; a group without tokens has none
    const float v0 = ok & 1 ? __log2f(st.vs[0]) : -INFINITY, v1 = ok & 2 ? __log2f(st.vs[1]) : -INFINITY;
    float top[2] = {-INFINITY, -INFINITY}, topv[2];  // largest score, and score + log2 V scale
#pragma unroll
    for (int hf = 0; hf < NH; hf++) {
      float top0 = -INFINITY;  // of the first group
      const float f = hf ? q.f1 : q.f0;
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float& x = sc[nt][2 * hf + e];
          x *= f * (nt < 2 ? k0 : k1);
          if (!full) {
            const int j = tile * TT + (nt >> 1) * 16 + col_token(t, nt & 1, e);
            if (j >= see[hf] || !(ok >> (nt >> 1) & 1)) x = -INFINITY;
          }
          if (nt < 2) top0 = fmaxf(top0, x); else top[hf] = fmaxf(top[hf], x);
        }
      topv[hf] = fmaxf(top0 + v0, top[hf] + v1);
      top[hf] = fmaxf(top[hf], top0);
      top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 1));
      top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xffffffffu, top[hf], 2));
      if (v0 == v1) {
        topv[hf] = top[hf] + v0;
      } else {
        topv[hf] = fmaxf(topv[hf], __shfl_xor_sync(0xffffffffu, topv[hf], 1));
        topv[hf] = fmaxf(topv[hf], __shfl_xor_sync(0xffffffffu, topv[hf], 2));
      }
    }
    bool grow = false;
#pragma unroll
    for (int hf = 0; hf < NH; hf++) grow |= top[hf] > m[hf] + LAZY || topv[hf] > mv[hf] + LAZY;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int hf = 0; hf < NH; hf++) {
        const float m1 = fmaxf(m[hf], top[hf]), mv1 = fmaxf(mv[hf], topv[hf]);
        const float fl = m1 == -INFINITY ? 1.f : sfu_exp2(m[hf] - m1), fo = mv1 == -INFINITY ? 1.f : sfu_exp2(mv[hf] - mv1);
        m[hf] = m1, mv[hf] = mv1;
        l[hf] *= fl;
#pragma unroll
        for (int j = 0; j < BPL; j++) o[j][2 * hf] *= fo, o[j][2 * hf + 1] *= fo;
      }
    }
    // ---- weights: 2^(score - m) for the sum, times 2^(log2 V scale + m - mv) for the product with V's codes
    uint32_t p[2][4], plo[2][4];
#pragma unroll
    for (int hf = 0; hf < NH; hf++) {
      const float mm = m[hf] == -INFINITY ? 0.f : m[hf], mmv = mv[hf] == -INFINITY ? 0.f : mv[hf];
      const float c0 = sfu_exp2(v0 + mm - mmv), c1 = sfu_exp2(v1 + mm - mmv);
#pragma unroll
      for (int nt = 0; nt < 4; nt++) {
        const float x = sfu_exp2(sc[nt][2 * hf] - mm), y = sfu_exp2(sc[nt][2 * hf + 1] - mm);
        l[hf] += x + y;
        const float c = nt < 2 ? c0 : c1;
        const uint32_t v = pack_f16(x * c, y * c);
        p[nt >> 1][2 * (nt & 1) + hf] = v;
        if (sizeof(T) == 4) plo[nt >> 1][2 * (nt & 1) + hf] = pack_rest(x * c, y * c, v);
      }
    }
    if (R8) {
#pragma unroll
      for (int gr = 0; gr < 2; gr++) p[gr][1] = p[gr][3] = plo[gr][1] = plo[gr][3] = 0u;
    }
    // ---- o += p v
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
        const uint32_t x01 = __byte_perm(vw[0][c], vw[1][c], 0x5140), y01 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
        const uint32_t x23 = __byte_perm(vw[2][c], vw[3][c], 0x5140), y23 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
        const uint32_t bb[4][2] = {{f16x2_e4m3(x01), f16x2_e4m3(x23)},
                                   {f16x2_e4m3(x01 >> 16), f16x2_e4m3(x23 >> 16)},
                                   {f16x2_e4m3(y01), f16x2_e4m3(y23)},
                                   {f16x2_e4m3(y01 >> 16), f16x2_e4m3(y23 >> 16)}};
#pragma unroll
        for (int j = 0; j < 4; j++) {
          mma(o[4 * c + j], p[gr][0], p[gr][1], p[gr][2], p[gr][3], bb[j][0], bb[j][1]);
          if (sizeof(T) == 4)  // fp32 outputs: the weights' second fp16 term
            mma(o[4 * c + j], plo[gr][0], plo[gr][1], plo[gr][2], plo[gr][3], bb[j][0], bb[j][1]);
        }
      }
    }
    if (__any_sync(0xffffffffu, poison)) {
      for (int row = 0; row < TT; row++) {
        const int j = tile * TT + row;
        for (int x = 0; x < 2 * BPL; x++) {
          const int d = 2 * t * BPL + x;
          if ((st.v[tile_at<HD>(row, d / 16) + d % 16] & 0x7f) != 0x7f) continue;
#pragma unroll
          for (int hf = 0; hf < NH; hf++)
            if (j < see[hf]) {
#pragma unroll
              for (int y = 0; y < 2 * BPL; y++)  // indexes of o are known when compiling
                if (y == x) o[y % BPL][2 * hf + y / BPL] = __int_as_float(0x7fc00000);
            }
        }
      }
    }
  }

  // ---- join the warps: each row's maxima and sum, then the outputs at the common maximum
#pragma unroll
  for (int hf = 0; hf < NH; hf++) {
    l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
    l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
    if (t == 0) st_m[w][g + 8 * hf] = m[hf], st_mv[w][g + 8 * hf] = mv[hf], st_l[w][g + 8 * hf] = l[hf];
  }
  cp_wait<0>();
  __syncthreads();  // every warp is done with its stages
  float* part = reinterpret_cast<float*>(smem);  // [NW][ROWS][OP]
#pragma unroll
  for (int hf = 0; hf < NH; hf++)
#pragma unroll
    for (int e = 0; e < 2; e++)
#pragma unroll
      for (int j = 0; j < BPL; j += 4)
        *reinterpret_cast<float4*>(part + ((size_t)w * ROWS + g + 8 * hf) * OP + (2 * t + e) * BPL + j) =
            make_float4(o[j][2 * hf + e], o[j + 1][2 * hf + e], o[j + 2][2 * hf + e], o[j + 3][2 * hf + e]);
  if (threadIdx.x < ROWS) {
    const int r = threadIdx.x;
    float mm = -INFINITY, mmv = -INFINITY, ll = 0.f;
    for (int i = 0; i < NW; i++) mm = fmaxf(mm, st_m[i][r]), mmv = fmaxf(mmv, st_mv[i][r]);
    for (int i = 0; i < NW; i++) {
      ll += st_m[i][r] == -INFINITY ? st_l[i][r] : st_l[i][r] * sfu_exp2(st_m[i][r] - mm);
      st_mv[i][r] = st_mv[i][r] == -INFINITY ? 0.f : sfu_exp2(st_mv[i][r] - mmv);  // the warp's factor
    }
    cl_m[r] = mm, cl_mv[r] = mmv, cl_l[r] = ll;
  }
  __syncthreads();
  float* sum = part + (size_t)NW * ROWS * OP;  // [ROWS][HD]
  for (int i = threadIdx.x; i < ROWS * HD; i += NW * 32) {
    const int r = i / HD, d = i % HD;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < NW; k++) x = fmaf(st_mv[k][r], part[((size_t)k * ROWS + r) * OP + d], x);
    sum[i] = x;
  }
  // ---- join the cluster's blocks: block `split` finishes its share of the rows' values
  cg::cluster_group cl = cg::this_cluster();
  if (n_split > 1) cl.sync(); else __syncthreads();
  T* out = reinterpret_cast<T*>(at.o);
  const int share = (ROWS * HD + n_split - 1) / n_split;
  for (int i = split * share + threadIdx.x; i < min(ROWS * HD, (split + 1) * share); i += NW * 32) {
    const int r = i / HD, d = i % HD, rr = row0 + r;
    if (rr >= R) break;
    float mm = -INFINITY, mmv = -INFINITY, ll = 0.f, x = 0.f;
    for (int k = 0; k < n_split; k++) {
      mm = fmaxf(mm, *(n_split > 1 ? cl.map_shared_rank(&cl_m[r], k) : &cl_m[r]));
      mmv = fmaxf(mmv, *(n_split > 1 ? cl.map_shared_rank(&cl_mv[r], k) : &cl_mv[r]));
    }
    for (int k = 0; k < n_split; k++) {
      const float km = *(n_split > 1 ? cl.map_shared_rank(&cl_m[r], k) : &cl_m[r]);
      const float kv = *(n_split > 1 ? cl.map_shared_rank(&cl_mv[r], k) : &cl_mv[r]);
      const float kl = *(n_split > 1 ? cl.map_shared_rank(&cl_l[r], k) : &cl_l[r]);
      const float kx = *(n_split > 1 ? cl.map_shared_rank(&sum[i], k) : &sum[i]);
      ll += km == -INFINITY ? kl : kl * sfu_exp2(km - mm);
      x += kv == -INFINITY ? kx : kx * sfu_exp2(kv - mmv);
    }
    // a row that sees nothing: zeros, and the log of an empty sum
    const float y = ll == 0.f ? 0.f : x / ll * exp2f(mmv - mm);
    const long row = r0 + rr / G;
    const int head = h * G + rr % G;
    out[row * at.o_ld + (long)head * HD + d] = from_f<T>(y);
    if (d == 0 && at.lse)
      at.lse[row * (long)(a.H * G) + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
  }
  if (n_split > 1) cl.sync();  // no block leaves while another reads its shared memory
}

// ---------------------------------------------------------------- accumulation of the weights

// weight[slot] += sum over the rows of exp(score - lse): the QK product again,
// now with the rows' final statistics, so that a slot's sum is formed by one
// lane in a fixed order.  HBM-bound on K; a warp holds the codes of TW tiles in
// registers and takes all rows past them.
template <typename T, int HD, int TW>
__global__ void __launch_bounds__(256) k_kv8_accumulate(Kv8Args a, AttnArgs at) {
  const int h = blockIdx.y, s = blockIdx.z;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int r0;
  const int n = kv8_rows(a, s, &r0), len = kv8_len(a, s), G = at.G, R = n * G;
  const int cap = a.max_blocks << a.lgP, see_hi = min(len + n, cap);
  if (n == 0) return;
  // the grid covers the caller's bound on the lengths; a longer sequence takes its blocks further
  for (long at_slot = (long)(blockIdx.x * (blockDim.x >> 5) + w) * TW * TT; at_slot < see_hi;
       at_slot += (long)gridDim.x * (blockDim.x >> 5) * TW * TT) {
    const int base = (int)at_slot;
    uint32_t kw[TW][4][HD / 16];
    size_t bh[TW][2];   // (block, head) of each group
    float ks[TW][2];
    bool ok[TW][2];
#pragma unroll
    for (int x = 0; x < TW; x++)
#pragma unroll
      for (int gr = 0; gr < 2; gr++) {
        const int j0 = base + x * TT + gr * 16;
        const int b = j0 < see_hi ? kv8_block(a, s, j0 >> a.lgP) : -1;
        ok[x][gr] = b >= 0;
        bh[x][gr] = (size_t)max(b, 0) * a.H + h;
      }
#pragma unroll
    for (int x = 0; x < TW; x++)
#pragma unroll
      for (int gr = 0; gr < 2; gr++) {
        const int j0 = base + x * TT + gr * 16;
        ks[x][gr] = ok[x][gr] ? a.ks[bh[x][gr]] : 0.f;
#pragma unroll
        for (int nt = 0; nt < 2; nt++) {
          const int j = j0 + key_token(g, nt);
          const uint8_t* p = a.k + (bh[x][gr] * a.P + (j & (a.P - 1))) * HD;
          const bool on = ok[x][gr] && j < see_hi;
          if (HD == 32) {
            const uint2 c = on ? *reinterpret_cast<const uint2*>(p + t * 8) : make_uint2(0, 0);
            kw[x][2 * gr + nt][0] = c.x, kw[x][2 * gr + nt][1] = c.y;
          } else {
#pragma unroll
            for (int i = 0; i < HD / 64; i++) {
              const uint4 c = on ? *reinterpret_cast<const uint4*>(p + i * 64 + t * 16) : make_uint4(0, 0, 0, 0);
              kw[x][2 * gr + nt][(4 * i) % (HD / 16)] = c.x, kw[x][2 * gr + nt][(4 * i + 1) % (HD / 16)] = c.y;
              kw[x][2 * gr + nt][(4 * i + 2) % (HD / 16)] = c.z, kw[x][2 * gr + nt][(4 * i + 3) % (HD / 16)] = c.w;
            }
          }
        }
      }
    float sum[TW][4][2];
#pragma unroll
    for (int x = 0; x < TW; x++)
#pragma unroll
      for (int nt = 0; nt < 4; nt++) sum[x][nt][0] = sum[x][nt][1] = 0.f;
    for (int row0 = 0; row0 < R; row0 += 16) {
      if (base >= len + min(R - 1, row0 + 15) / G + 1) continue;  // no row of these sees the warp's slots
      QFrag<T, HD, false> q;
      q.load(reinterpret_cast<const T*>(at.q) + (long)r0 * at.q_ld, at.q_ld, h * G * HD, G, row0, R, at.scale);
      float ls[2];
      int see[2];
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        const int r = row0 + g + 8 * hf, i = min(r, R - 1) / G;
        see[hf] = r < R ? min(len + i + 1, cap) : 0;  // rows past the last see nothing
        const float x = r < R ? at.lse[(long)(r0 + i) * (a.H * G) + h * G + r % G] : 0.f;
        if (x == -INFINITY) see[hf] = 0;  // a row without weights
        ls[hf] = x * 1.4426950408889634f;
      }
#pragma unroll
      for (int x = 0; x < TW; x++)
#pragma unroll
        for (int nt = 0; nt < 4; nt++) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          q.qk(d, kw[x][nt]);
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int j = base + x * TT + (nt >> 1) * 16 + col_token(t, nt & 1, e);
            const float k = ks[x][nt >> 1];
            const float p0 = j < see[0] ? sfu_exp2(d[e] * (q.f0 * k) - ls[0]) : 0.f;
            const float p1 = j < see[1] ? sfu_exp2(d[2 + e] * (q.f1 * k) - ls[1]) : 0.f;
            sum[x][nt][e] += p0 + p1;
          }
        }
    }
#pragma unroll
    for (int x = 0; x < TW; x++)
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float v = sum[x][nt][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          const int j = base + x * TT + (nt >> 1) * 16 + col_token(t, nt & 1, e);
          // one lane of the eight that hold the sum adds it (atomically: two sequences may share a block)
          if (g == 2 * nt + e && j < see_hi && ok[x][nt >> 1])
            atomicAdd(a.w + bh[x][nt >> 1] * a.P + (j & (a.P - 1)), v);
        }
  }
}

template <typename T, int HD, bool R8>
bool launch_attn(Ctx& c, const Kv8Args& a, AttnArgs at, long row_tiles, int max_len) {
  constexpr int NW = 8, NS = HD == 128 ? 3 : 4, ROWS = R8 ? 8 : 16;
  constexpr size_t ring = sizeof(Stage<HD>) * NW * NS, join = (size_t)NW * ROWS * (HD + 4) * 4 + ROWS * HD * 4;
  const size_t smem = ring > join ? ring : join;
  auto k = k_kv8_attn<T, HD, R8, NW, NS>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  // few blocks: the slots of each are split over a cluster of up to 8, each with a tile or more for every warp
  const long blocks = (long)a.S * a.H * row_tiles;
  const long tiles = (max_len + TT - 1) / TT;
  const long want = (2 * c.num_sms + blocks - 1) / blocks, most = (tiles + NW - 1) / NW;
  int split = (int)(want < most ? want : most);
  split = split < 1 ? 1 : split > 8 ? 8 : split;
  cudaLaunchConfig_t cfg = {};
  at.n_split = split;
  cfg.gridDim = dim3((unsigned)(split * row_tiles), a.H, a.S);
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a, at) == cudaSuccess;
}

template <typename T, int HD>
bool launch_attn_rows(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  const long rows = (long)a.max_new * at.G;
  if (rows <= 8) return launch_attn<T, HD, true>(c, a, at, 1, max_len);
  return launch_attn<T, HD, false>(c, a, at, (rows + 15) / 16, max_len);
}

template <typename T, int HD>
void launch_accumulate(Ctx& c, const Kv8Args& a, const AttnArgs& at, int max_len) {
  constexpr int TW = HD == 128 ? 1 : 2;
  const int per = 8 * TW * TT;
  k_kv8_accumulate<T, HD, TW><<<dim3((max_len + per - 1) / per, a.H, a.S), 256, 0, c.stream>>>(a, at);
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

void kv8_accumulate(Ctx& c, const Kv8Args& a, int hd, int G, bool bf16_rows, const void* q, long q_ld, float scale,
                    int max_len, const float* lse) {
  LaunchScope s(c, "kv8_accumulate");
  AttnArgs at{q, q_ld, scale, G, 0, nullptr, 0, const_cast<float*>(lse)};
  if (bf16_rows) {
    if (hd == 32) return launch_accumulate<bf16, 32>(c, a, at, max_len);
    if (hd == 64) return launch_accumulate<bf16, 64>(c, a, at, max_len);
    return launch_accumulate<bf16, 128>(c, a, at, max_len);
  }
  if (hd == 32) return launch_accumulate<float, 32>(c, a, at, max_len);
  if (hd == 64) return launch_accumulate<float, 64>(c, a, at, max_len);
  return launch_accumulate<float, 128>(c, a, at, max_len);
}

}  // namespace gpt
