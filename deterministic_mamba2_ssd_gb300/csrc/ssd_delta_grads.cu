// ssd_delta_grads.cu -- gradients of a chunk of the gated delta rule from what
// the two chains left: S0 (S16) and e (E16) of the forward; dS of the state
// leaving the chunk, F = dS k and dO (D16, F16, X16) of the backward.  With
// dR = beta F, U = beta e and D_ts = exp(G_t - G_s):
//
//   M1 = -(dR U^T) o D (s < t),  M2 = scale (dO U^T) o D (s <= t)    (64 x 64)
//   Y1 = scale exp(G) dO S0,  Y2 = -exp(G) dR S0,  Z = exp(G_C - G) U dS
//   dq = Y1 + M2 K,  dk = Y2 + M1 K + Z + M1^T K + M2^T Q
//   dbeta_t = F_t . e_t
//   dg_t = sum_{t' >= t} (q.Y1 + k.Y2)_t' + sum_{s < t} (k.Z)_s + exp(G_C) <S0, dS>
//          + sum_{t' >= t > s} W_t's,   W = M1 o K K^T + M2 o Q K^T
//
// (dg_t gathers what passes from before token t to it or past it: W's last sum
// is that of rows minus columns from t on, with the same W in both, so what
// does not pass cancels to the last bit's size.)
//
// The heads of a group accumulate dq and dk in registers, in ascending order:
// no slots, one order.  Their operands share one power of two for the whole
// group: the strips' scales relative to the largest are applied to the left
// operands (exact, and rarely needed).  M1 and M2 go through fp16 once more.
//
// CTA (chunk slot, group), 8 warps: warp (w % 4, w / 4) has 16 tokens and half
// of the columns of each product.  What bounds the kernel is the record, 1.75
// KB a token and head at headdim = dstate = 128, and the instructions around
// the products; the next head's rows are on their way while this head is worked
// on, and its states while the 64 x 64 products run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr int kWork = 256, kCopy = 128;      // threads with the products, threads that copy
constexpr int kThreads = kWork + kCopy;
constexpr int kPMax = 128;
constexpr int kRow = 2 * kPMax;              // bytes of a token's row of a [token][p] tile in shared memory
constexpr int kRows = kChunk * kRow;

template <int N>
struct Smem {
  uint8_t k[kChunk * N * 2], q[kChunk * N * 2];
  uint8_t X[2][kRows], F[2][kRows], E[2][kRows];    // [token][p]; of this head and the next
  uint8_t S[kPMax * N * 2], D[kPMax * N * 2];       // [p][n]
  uint8_t m1[kChunk * 128], m2[kChunk * 128];       // [t][s]
  float vec[2][kVec];                               // of this head and the next
  float rel[2][kPMax / 16];                         // the strips' scales relative to the group's
  uint32_t even[2];                                 // all of them 1
  float inner[2][kCopy / 32];                       // <S0, dS>, each copying warp's part
  float fe[2][kChunk];                              // [head parity]: F.e of each token
  float state[2][2][kChunk], down[2][2][kChunk];    // [head parity][column half]: q.Y1 + k.Y2, k.Z
  float wrow[2][2][kChunk], wcol[2][4][kChunk];     // row sums of W by column half, column sums by token strip
};

__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(~0u, v, 1);
  return v + __shfl_xor_sync(~0u, v, 2);
}
__device__ __forceinline__ uint32_t twice(float f) { return pack(f, f); }
__device__ __forceinline__ void scale_a(uint32_t (&a)[4], uint32_t f0, uint32_t f1) {   // rows g by f0, rows g + 8 by f1
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = i & 1 ? f1 : f0;
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a[i]), *reinterpret_cast<const __half2 *>(&f));
    a[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
}

// d and (kTwo) e += the left operands a and b times 16 rows [k][n] at `row`; at[i]: this lane's place in them for the
// i-th 16 columns of its warp.
template <int kPairs, bool kTwo>
__device__ __forceinline__ void step_t(float (&d)[2 * kPairs][4], float (&e)[2 * kPairs][4], const uint32_t (&a)[4],
                                       const uint32_t (&b)[4], uint32_t row, const uint32_t (&at)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    uint32_t r[4];
    ldsm4t(r, row + at[i]);
    mma(d[2 * i], a, r[0], r[1]);
    mma(d[2 * i + 1], a, r[2], r[3]);
    if (kTwo) {
      mma(e[2 * i], b, r[0], r[1]);
      mma(e[2 * i + 1], b, r[2], r[3]);
    }
  }
}
// Columns 16 j.. of a row at `row` (tiles are aligned to 128 bytes: the swizzle is an exclusive or of the address).
__device__ __forceinline__ uint32_t block(uint32_t row, int j) { return (row ^ ((j & 3) << 5)) + ((j >> 2) << 7); }

template <int N>
__global__ void __launch_bounds__(kThreads, 1) grads_tile_kernel(Shape s, Args a, Tiles t, BwdTiles o, int out4) {
  constexpr int NB = 2 * N;          // bytes of a row of k, q, S, D
  constexpr int kPairs = N / 32;     // pairs of column tiles of a warp (half of the columns)
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<N> &sm = *reinterpret_cast<Smem<N> *>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wm = warp & 3, wn = warp >> 2;
  const int64_t slot = blockIdx.x;
  const int grp = blockIdx.y, g = lane >> 2, c2 = 2 * (lane & 3);
  const int P = s.P, strips = P / 16;
  int64_t seq, b, e;
  if (!chunk_of_slot(s, a.cu, slot, seq, b, e)) return;
  const int n = int(e - b);
  const uint32_t ks = smem_at(sm.k), qs = smem_at(sm.q), Ss = smem_at(sm.S), Ds = smem_at(sm.D), m1s = smem_at(sm.m1),
                 m2s = smem_at(sm.m2);
  // the group's common power of two: the largest of the heads' and strips' up * ub
  float ref = 0.f;
  for (int x = lane; x < s.hpg * strips; x += 32) {
    const int64_t at = (slot * s.H + grp * s.hpg) * strips + x;
    ref = fmaxf(ref, t.up[at] * o.ub[at]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(~0u, ref, d));
  const float iref = pow2_inv(ref);

  if (tid >= kWork) {
    const int ct = tid - kWork;
    auto copy = [&](uint32_t to, const __half *from, int n16) {
#pragma unroll 8
      for (int x = ct; x < n16; x += kCopy) cp16(to + 16 * x, from + 8 * x);
    };
    const int per = P / 8, dr = kCopy / per, dj = kCopy % per;   // 16-byte pieces of a [token][p] row
    auto fetch_rows = [&](int i) {   // the [token][p] tiles, vectors and scales of head i of the group
      const int64_t ht = slot * s.H + grp * s.hpg + i, at0 = ht * kChunk * P;
      const int y = i & 1;
      const uint32_t Xs = smem_at(sm.X[y]), Fs = smem_at(sm.F[y]), Es = smem_at(sm.E[y]);
      int r = ct / per, j = ct % per;
#pragma unroll 4
      for (int x = ct; x < kChunk * per; x += kCopy) {
        const uint32_t at = swz(r, j, kRow);
        cp16(Xs + at, o.X16 + at0 + 8 * x);
        cp16(Fs + at, o.F16 + at0 + 8 * x);
        cp16(Es + at, t.E16 + at0 + 8 * x);
        r += dr;
        j += dj;
        if (j >= per) j -= per, ++r;
      }
      if (warp == 8) {   // which has read the vectors of two heads before
        for (int x = lane; x < kVec / 4; x += 32) cp16(smem_at(sm.vec[y]) + 16 * x, t.vec + ht * kVec + 4 * x);
        const float f = lane < strips ? t.up[ht * strips + lane] * o.ub[ht * strips + lane] * iref : 1.f;
        const bool all = __all_sync(~0u, f == 1.f);
        if (lane < kPMax / 16) sm.rel[y][lane] = f;
        if (lane == 0) sm.even[y] = all;
      }
      cp_commit();
    };
    auto product = [&](int i) {   // the same element of both states at the same place
      float sum = 0.f;
#pragma unroll 1
      for (int j = 0; j < strips; ++j) {
        float acc = 0.f;
#pragma unroll
        for (int y = 0; y < 2 * N; y += kCopy) {
          const int at = 16 * (2 * N * j + y + ct);
          const uint4 u = *reinterpret_cast<const uint4 *>(sm.S + at), v = *reinterpret_cast<const uint4 *>(sm.D + at);
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float2 fu = unpack(uu[z]), fv = unpack(vv[z]);
            acc = fmaf(fu.x, fv.x, fmaf(fu.y, fv.y, acc));
          }
        }
        sum = fmaf(acc, sm.rel[i & 1][j], sum);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      if (lane == 0) sm.inner[i & 1][ct >> 5] = sum;
    };
    // dg and dbeta of head i, by one warp, two tokens a lane
    auto finish = [&](int i) {
      const int x = i & 1, h = grp * s.hpg + i;
      const float *vec = sm.vec[x];
      float from[2], cut[2], dn[2];
      const float inner = (sm.inner[x][0] + sm.inner[x][1] + sm.inner[x][2] + sm.inner[x][3]) * vec[kVecEg + kChunk - 1];
  #pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 2 * lane + y;
        from[y] = sm.state[x][0][r] + sm.state[x][1][r];
        dn[y] = sm.down[x][0][r] + sm.down[x][1][r];
        cut[y] = (sm.wrow[x][0][r] + sm.wrow[x][1][r]) -
                 ((sm.wcol[x][0][r] + sm.wcol[x][1][r]) + (sm.wcol[x][2][r] + sm.wcol[x][3][r]));
      }
      float a1 = from[0] + from[1], a2 = cut[0] + cut[1], a3 = dn[0] + dn[1];
  #pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float u1 = __shfl_down_sync(~0u, a1, d), u2 = __shfl_down_sync(~0u, a2, d), u3 = __shfl_up_sync(~0u, a3, d);
        if (lane + d < 32) a1 += u1, a2 += u2;
        if (lane >= d) a3 += u3;
      }
      const float b3 = __shfl_up_sync(~0u, a3, 1), n1 = __shfl_down_sync(~0u, a1, 1), n2 = __shfl_down_sync(~0u, a2, 1);
      const float before = lane == 0 ? 0.f : b3;
      float dg[2];
      dg[1] = (lane == 31 ? 0.f : n1 + n2) + from[1] + cut[1] + before + dn[0] + inner;
      // nothing comes from before the first token but the state
      dg[0] = a1 + (lane == 0 ? 0.f : a2) + before + inner;
  #pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 2 * lane + y;
        if (r < n) {
          static_cast<__nv_bfloat16 *>(a.dg)[(b + r) * s.H + h] = __float2bfloat16_rn(ref * dg[y]);
          static_cast<__nv_bfloat16 *>(a.dbeta)[(b + r) * s.H + h] = __float2bfloat16_rn(ref * sm.fe[x][r]);
        }
      }
    };
    const int64_t at = (slot * s.G + grp) * kChunk * N;
    copy(ks, t.K16 + at, kChunk * N / 8);
    copy(qs, t.Q16 + at, kChunk * N / 8);
    cp_commit();
    fetch_rows(0);
    cp_wait<1>();
    __syncthreads();   // k and q
    for (int i = 0; i < s.hpg; ++i) {
      cp_wait<0>();
      __syncthreads();   // rows of head i
      const int64_t st = (slot * s.H + grp * s.hpg + i) * P * N;
      copy(Ds, o.D16 + st, P * N / 8);
      copy(Ss, t.S16 + st, P * N / 8);
      cp_commit();
      if (i > 0 && warp == 8) finish(i - 1);
      if (i + 1 < s.hpg) {
        fetch_rows(i + 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      __syncthreads();   // states of head i
      product(i);
    }
    __syncthreads();
    if (warp == 8) finish(s.hpg - 1);
    return;
  }

  const int rows[2] = {16 * wm + g, 16 * wm + g + 8}, n0 = wn * (N / 2);
  // where this lane's rows of operands begin in their tiles
  const uint32_t left = ((lane & 7) + (lane & 8)), half = lane >> 4, low = lane & 7;
  const uint32_t arow = (16 * wm + left) * kRow + ((half ^ low) << 4);            // left operand, X, F, E
  const uint32_t brow = (32 * wn + low + 8 * half) * kRow + ((((lane >> 3) & 1) ^ low) << 4);   // right operand, E as [n][k]
  uint32_t at[kPairs];                                                            // right operand, [k][n], this warp's columns
#pragma unroll
  for (int i = 0; i < kPairs; ++i) at[i] = block(left * NB + ((half ^ low) << 4), wn * kPairs + i);
  uint32_t kk2[4][2], qk2[4][2];   // this thread's part of K K^T and Q K^T, fp16
  {
    __syncthreads();
    float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < N; k0 += 16) {
      uint32_t ak[4], aq[4];
      ldsm4(ak, a_addr(ks, 16 * wm, k0, NB, lane));
      ldsm4(aq, a_addr(qs, 16 * wm, k0, NB, lane));
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (2 * wn + i <= wm) {
          uint32_t bb[4];
          ldsm4(bb, b_addr(ks, 32 * wn + 16 * i, k0, NB, lane));
          mma(kk[2 * i], ak, bb[0], bb[1]);
          mma(kk[2 * i + 1], ak, bb[2], bb[3]);
          mma(qk[2 * i], aq, bb[0], bb[1]);
          mma(qk[2 * i + 1], aq, bb[2], bb[3]);
        }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        kk2[y][r] = pack(kk[y][2 * r], kk[y][2 * r + 1]);
        qk2[y][r] = pack(qk[y][2 * r], qk[y][2 * r + 1]);
      }
  }
  // this thread's pair of k or q: rows[r], columns n0 + 8 y + c2
  auto pair_of = [&](const uint8_t *tile, int r, int y) {
    return unpack(*reinterpret_cast<const uint32_t *>(tile + swz(rows[r], (n0 >> 3) + y, NB) + 2 * c2));
  };
  // adds a head's product to the group's and gives its rows' products with k or q
  auto fold = [&](float (&sum)[2 * kPairs][4], const float (&y)[2 * kPairs][4], const uint8_t *tile, float (&dot)[2]) {
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 f = pair_of(tile, r, i);
        dot[r] = fmaf(f.x, y[i][2 * r], fmaf(f.y, y[i][2 * r + 1], dot[r]));
        sum[i][2 * r] += y[i][2 * r];
        sum[i][2 * r + 1] += y[i][2 * r + 1];
      }
  };
  float dq[2 * kPairs][4] = {}, dk[2 * kPairs][4] = {};
  for (int i = 0; i < s.hpg; ++i) {
    const int x = i & 1;
    const float *vec = sm.vec[x];
    const uint32_t Xs = smem_at(sm.X[x]), Fs = smem_at(sm.F[x]), Es = smem_at(sm.E[x]);
    __syncthreads();   // this head's rows are here
    const float ka = vec[kVecKa];
    const bool even = sm.even[x];
    {
      // blocks above the diagonal go along: a branch would cost more than they do
      float n1[4][4] = {}, n2[4][4] = {};
#pragma unroll 2
      for (int j = 0; j < strips; ++j) {
        uint32_t aX[4], aF[4], bb[2][4];
        ldsm4(aX, block(Xs + arow, j));
        ldsm4(aF, block(Fs + arow, j));
        ldsm4(bb[0], block(Es + brow, j));
        ldsm4(bb[1], block(Es + brow, j) + 16 * kRow);
        if (!even) {
          const uint32_t f = twice(sm.rel[x][j]);
          scale_a(aX, f, f);
          scale_a(aF, f, f);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mma(n1[2 * y], aF, bb[y][0], bb[y][1]);
          mma(n1[2 * y + 1], aF, bb[y][2], bb[y][3]);
          mma(n2[2 * y], aX, bb[y][0], bb[y][1]);
          mma(n2[2 * y + 1], aX, bb[y][2], bb[y][3]);
        }
      }
      const float Gr[2] = {vec[kVecG + rows[0]], vec[kVecG + rows[1]]};
      const float Lr[2] = {vec[kVecGl + rows[0]], vec[kVecGl + rows[1]]};
      const float w1[2] = {-ka * vec[kVecBeta + rows[0]], -ka * vec[kVecBeta + rows[1]]};
      const float w2 = ka * a.scale;
      float wrow[2] = {0.f, 0.f}, wcol[8];
      float2 Gc[4], Lc[4], be[4];   // all of them first: the stores below would hold back the loads after them
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int c = 32 * wn + 8 * y + c2;
        Gc[y] = *reinterpret_cast<const float2 *>(&vec[kVecG + c]);
        Lc[y] = *reinterpret_cast<const float2 *>(&vec[kVecGl + c]);
        be[y] = *reinterpret_cast<const float2 *>(&vec[kVecBeta + c]);
      }
      uint32_t m1[4][2], m2[4][2];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int c = 32 * wn + 8 * y + c2;
        wcol[2 * y] = wcol[2 * y + 1] = 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float d0 = __expf(acs_diff(Gr[r], Lr[r], Gc[y].x, Lc[y].x)) * be[y].x;
          const float d1 = __expf(acs_diff(Gr[r], Lr[r], Gc[y].y, Lc[y].y)) * be[y].y;
          const float x0 = c < rows[r] ? n1[y][2 * r] * d0 * w1[r] : 0.f;
          const float x1 = c + 1 < rows[r] ? n1[y][2 * r + 1] * d1 * w1[r] : 0.f;
          const float z0 = c <= rows[r] ? n2[y][2 * r] * d0 * w2 : 0.f;
          const float z1 = c + 1 <= rows[r] ? n2[y][2 * r + 1] * d1 * w2 : 0.f;
          m1[y][r] = pack(x0, x1);
          m2[y][r] = pack(z0, z1);
          const float2 kf = unpack(kk2[y][r]), qf = unpack(qk2[y][r]);
          // (the diagonal is not W's: nothing passes from a token to itself)
          const float v0 = fmaf(x0, kf.x, c < rows[r] ? z0 * qf.x : 0.f);
          const float v1 = fmaf(x1, kf.y, c + 1 < rows[r] ? z1 * qf.y : 0.f);
          wrow[r] += v0 + v1;
          wcol[2 * y] += v0;
          wcol[2 * y + 1] += v1;
        }
      }
      if (wn == wm >> 1 && (lane & 3) == (g >> 1)) {   // this thread has the diagonal's elements g and g + 8
        const int y = 2 * (wm & 1);
        const float(&lo)[4] = y ? n1[2] : n1[0];
        const float(&hi)[4] = y ? n1[3] : n1[1];
        sm.fe[x][rows[0]] = g & 1 ? lo[1] : lo[0];
        sm.fe[x][rows[1]] = g & 1 ? hi[3] : hi[2];
      }
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t to = swz(rows[r], 4 * wn + y, 128) + 2 * c2;
          *reinterpret_cast<uint32_t *>(sm.m1 + to) = m1[y][r];
          *reinterpret_cast<uint32_t *>(sm.m2 + to) = m2[y][r];
        }
      // over this strip's 16 tokens: eight columns by eight lanes, halving what each still carries
#pragma unroll
      for (int d = 4, lanes = 16; d > 0; d >>= 1, lanes >>= 1) {
        const bool up = lane & lanes;
#pragma unroll
        for (int z = 0; z < d; ++z) {
          const float give = up ? wcol[z] : wcol[z + d], keep = up ? wcol[z + d] : wcol[z];
          wcol[z] = keep + __shfl_xor_sync(~0u, give, lanes);
        }
      }
      // left with column 8 y + c2 + z, 2 y + z = g
      sm.wcol[x][wm][32 * wn + 8 * (g >> 1) + c2 + (g & 1)] = wcol[0] * ka;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        wrow[r] = quad_sum(wrow[r]);
        if (c2 == 0) sm.wrow[x][wn][rows[r]] = wrow[r] * ka;
      }
    }
    __syncthreads();   // M1 and M2 are here, and the states
    uint32_t fx[2], ff[2], fu[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float eg = vec[kVecEg + rows[r]], be = vec[kVecBeta + rows[r]];
      fx[r] = twice(a.scale * eg);
      ff[r] = twice(-eg * be);
      fu[r] = twice(vec[kVecTail + rows[r]] * be);
    }
    float state[2] = {0.f, 0.f}, down[2] = {0.f, 0.f};
    {
      float y1[2 * kPairs][4] = {}, y2[2 * kPairs][4] = {};
      uint32_t nX[4], nF[4];   // the left operands a step ahead
      ldsm4(nX, Xs + arow);
      ldsm4(nF, Fs + arow);
#pragma unroll 2
      for (int j = 0; j < strips; ++j) {
        uint32_t aX[4], aF[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          aX[z] = nX[z];
          aF[z] = nF[z];
        }
        if (j + 1 < strips) {
          ldsm4(nX, block(Xs + arow, j + 1));
          ldsm4(nF, block(Fs + arow, j + 1));
        }
        if (!even) {
          const uint32_t f = twice(sm.rel[x][j]);
          scale_a(aX, f, f);
          scale_a(aF, f, f);
        }
        scale_a(aX, fx[0], fx[1]);
        scale_a(aF, ff[0], ff[1]);
        step_t<kPairs, true>(y1, y2, aX, aF, Ss + j * 16 * NB, at);
      }
      fold(dq, y1, sm.q, state);
      fold(dk, y2, sm.k, state);
    }
    {
      float z[2 * kPairs][4] = {};
      uint32_t nE[4];
      ldsm4(nE, Es + arow);
#pragma unroll 2
      for (int j = 0; j < strips; ++j) {
        uint32_t aE[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) aE[y] = nE[y];
        if (j + 1 < strips) ldsm4(nE, block(Es + arow, j + 1));
        if (!even) {
          const uint32_t f = twice(sm.rel[x][j]);
          scale_a(aE, f, f);
        }
        scale_a(aE, fu[0], fu[1]);
        step_t<kPairs, false>(z, z, aE, aE, Ds + j * 16 * NB, at);
      }
      fold(dk, z, sm.k, down);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      state[r] = quad_sum(state[r]);
      down[r] = quad_sum(down[r]);
      if (c2 == 0) {
        sm.state[x][wn][rows[r]] = state[r] * ka;
        sm.down[x][wn][rows[r]] = down[r] * ka;
      }
    }
    // dq += M2 K, dk += M1 K + M1^T K + M2^T Q
#pragma unroll 1
    for (int j = 0; j <= wm; ++j) {
      uint32_t a2[4], a1[4];
      ldsm4(a2, a_addr(m2s, 16 * wm, 16 * j, 128, lane));
      ldsm4(a1, a_addr(m1s, 16 * wm, 16 * j, 128, lane));
      step_t<kPairs, true>(dq, dk, a2, a1, ks + j * 16 * NB, at);
    }
#pragma unroll 1
    for (int j = wm; j < 4; ++j) {
      uint32_t a1[4], a2[4];
      ldsm4t(a1, at_addr(m1s, 16 * wm, 16 * j, 128, lane));
      ldsm4t(a2, at_addr(m2s, 16 * wm, 16 * j, 128, lane));
      step_t<kPairs, false>(dk, dk, a1, a1, ks + j * 16 * NB, at);
      step_t<kPairs, false>(dk, dk, a2, a2, qs + j * 16 * NB, at);
    }
  }
  __syncthreads();   // what the copying warp still has to finish
  __nv_bfloat16 *oq = static_cast<__nv_bfloat16 *>(a.dq), *ok = static_cast<__nv_bfloat16 *>(a.dk);
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (rows[r] < n) {
      const int64_t to = ((b + rows[r]) * s.G + grp) * N + n0 + c2;
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y) {
        const uint32_t vq = pack_bf16(dq[y][2 * r] * ref, dq[y][2 * r + 1] * ref);
        const uint32_t vk = pack_bf16(dk[y][2 * r] * ref, dk[y][2 * r + 1] * ref);
        if (out4) {
          *reinterpret_cast<uint32_t *>(oq + to + 8 * y) = vq;
          *reinterpret_cast<uint32_t *>(ok + to + 8 * y) = vk;
        } else {
          oq[to + 8 * y] = __ushort_as_bfloat16(static_cast<unsigned short>(vq & 0xffffu));
          oq[to + 8 * y + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(vq >> 16));
          ok[to + 8 * y] = __ushort_as_bfloat16(static_cast<unsigned short>(vk & 0xffffu));
          ok[to + 8 * y + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(vk >> 16));
        }
      }
    }
}

template <int N>
cudaError_t launch(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  const int smem = int(sizeof(Smem<N>));
  const cudaError_t e = cudaFuncSetAttribute(grads_tile_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const bool out4 = ((reinterpret_cast<uintptr_t>(a.dq) | reinterpret_cast<uintptr_t>(a.dk)) & 3) == 0;
  grads_tile_kernel<N><<<dim3(unsigned(s.slots), unsigned(s.G)), kThreads, smem, st>>>(
      s, a, t, o, out4);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grads(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  if (s.slots == 0 || s.total == 0) return cudaSuccess;
  return s.N == 64 ? launch<64>(s, a, t, o, st) : launch<128>(s, a, t, o, st);
}

}  // namespace delta
}  // namespace ssd
