// ssd_delta_grads.cu -- gradients of a chunk of the gated delta rule from what
// the two chains left: S0 (S16) and e (E16) of the forward, dS of the state
// leaving the chunk (D16) and dR = beta F (R16) of the backward.
//
//   N1 = dR E^T, N2 = scale dO E^T                              (64 x 64)
//   M1 = -N1 o D beta (s < t), M2 = N2 o D beta (s <= t),  D_ts = exp(G_t - G_s)
//   Z  = E dS;  state_s = exp(G_C - G_s) beta_s Z_s             (64 x dstate)
//   dq = scale exp(G) dO S0 + M2 K
//   up = M1 K - exp(G) dR S0
//   down = M1^T K + M2^T Q + state,   dk = up + down
//   dG_t = q_t.dq_t + k_t.(up_t - down_t);  dG_C += exp(G_C) <S0, dS> + sum_s k_s.state_s
//   dg = suffix sums of dG
//   dbeta_s = sum_t (N2 o D o QK - N1 o D o KK)_ts + exp(G_C - G_s) k_s . Z_s
//
// CTA (chunk slot, group), 8 warps: warp (w % 4, w / 4) has 16 tokens and half
// of the columns of each product.  The heads of a group are taken in ascending
// order and dq, dk summed in registers, so the group's sum has one order and
// no slots.  Left operands stay in registers (each row scaled by a power of
// two), right operands come from shared memory; the tiles of the next head
// arrive while this one is worked on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr int kThreads = 256;
constexpr int kPMax = 128;
constexpr int kRow = 2 * kPMax;   // bytes of a token's row of dO, R16 or E16 in shared memory

template <int N>
struct Smem {
  uint8_t k[kChunk * N * 2], q[kChunk * N * 2];
  uint8_t dO[kChunk * kRow], R[kChunk * kRow], E[kChunk * kRow];   // [token][p]
  uint8_t S[kPMax * N * 2], D[kPMax * N * 2];                      // [p][n]
  uint8_t m1[kChunk * 128], m2[kChunk * 128];                      // [t][s]
  float4 kk[4][kThreads], qk[4][kThreads];                         // each thread's own part of K K^T and Q K^T
  float vec[2][kVec], up[2][kPMax], ub[2][kPMax];                  // of this head and the next
  float row[2][2][kChunk];    // [head parity][column half]: q.dq + k.(up - down)
  float kz[2][2][kChunk];     // k_s . exp(G_C - G_s) Z_s
  float col[2][4][kChunk];    // [head parity][token strip]: column sums of N2 o D o QK - N1 o D o KK
  float inner[2][8];          // <S0, dS> of each warp's part
  int some[2][8];             // whether S0 has an element that is not zero
  float top[2][8];            // largest |M1|, |M2| of each warp
};

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
  return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(~0u, v, 1);
  return v + __shfl_xor_sync(~0u, v, 2);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
  return v;
}

// 16 rows (m0..) of a [token][p] tile as A operands: element times w[p] and a
// power of two for its row, which comes back in `sc`.
template <bool kBf16>
__device__ __forceinline__ void rows_as_a(uint32_t (&a)[kPMax / 16][4], float (&sc)[2], uint32_t tile, int m0, int P,
                                          const float *w0, const float *w1, int lane) {
  float m[2] = {0.f, 0.f};
  const int c = 2 * (lane & 3);
  auto value = [&](int j, int i) {
    const float2 f = kBf16 ? unpack_bf16(a[j][i]) : unpack(a[j][i]);
    const int p = 16 * j + 8 * (i >> 1) + c;
    float2 w = *reinterpret_cast<const float2 *>(w0 + p);
    if (w1 != nullptr) {
      const float2 x = *reinterpret_cast<const float2 *>(w1 + p);
      w.x *= x.x;
      w.y *= x.y;
    }
    return make_float2(f.x * w.x, f.y * w.y);
  };
#pragma unroll
  for (int j = 0; j < kPMax / 16; ++j)
    if (16 * j < P) {
      ldsm4(a[j], a_addr(tile, m0, 16 * j, kRow, lane));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = value(j, i);
        m[i & 1] = fmaxf(m[i & 1], fmaxf(fabsf(v.x), fabsf(v.y)));
      }
    }
  float inv[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    sc[r] = pow2_above(quad_max(m[r]));
    inv[r] = pow2_inv(sc[r]);
  }
#pragma unroll
  for (int j = 0; j < kPMax / 16; ++j)
    if (16 * j < P) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = value(j, i);
        a[j][i] = pack(v.x * inv[i & 1], v.y * inv[i & 1]);
      }
    }
}

// d (tile pairs n0, n0 + 16, ... of kPairs) += A B over one 16-step; B from rows [k][n].
template <int kPairs>
__device__ __forceinline__ void step_t(float (&d)[2 * kPairs][4], const uint32_t (&a)[4], uint32_t tile, int n0, int k0,
                                       int bytes, int lane) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    uint32_t b[4];
    ldsm4t(b, bt_addr(tile, n0 + 16 * i, k0, bytes, lane));
    mma(d[2 * i], a, b[0], b[1]);
    mma(d[2 * i + 1], a, b[2], b[3]);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) grads_tile_kernel(Shape s, Args a, Tiles t, BwdTiles o, int gvec) {
  constexpr int NB = 2 * N;          // bytes of a row of k, q, S, D
  constexpr int kPairs = N / 32;     // pairs of column tiles of a warp (half of the columns)
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<N> &sm = *reinterpret_cast<Smem<N> *>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wm = warp & 3, wn = warp >> 2;
  const int64_t slot = blockIdx.x;
  const int grp = blockIdx.y, g = lane >> 2, c2 = 2 * (lane & 3);
  const int P = s.P;
  int64_t seq, b, e;
  if (!chunk_of_slot(s, a.cu, slot, seq, b, e)) return;
  const int n = int(e - b);
  const uint32_t ks = smem_at(sm.k), qs = smem_at(sm.q), dOs = smem_at(sm.dO), Rs = smem_at(sm.R), Es = smem_at(sm.E),
                 Ss = smem_at(sm.S), Ds = smem_at(sm.D), m1s = smem_at(sm.m1), m2s = smem_at(sm.m2);
  const __nv_bfloat16 *go = static_cast<const __nv_bfloat16 *>(a.dout);

  auto fetch_rows = [&](int i) {   // dO, R16, E16 and the vectors of head i of the group
    const int h = grp * s.hpg + i;
    const int64_t ht = slot * s.H + h;
    const uint8_t *R = reinterpret_cast<const uint8_t *>(o.R16 + ht * kChunk * P);
    const uint8_t *E = reinterpret_cast<const uint8_t *>(t.E16 + ht * kChunk * P);
    const int per = P / 8;   // 16-byte pieces of a row
    for (int x = tid; x < kChunk * per; x += kThreads) {
      const int r = x / per, j = x % per;
      const uint32_t at = swz(r, j, kRow);
      cp16(Rs + at, R + int64_t(x) * 16);
      cp16(Es + at, E + int64_t(x) * 16);
      const __nv_bfloat16 *src = go + ((b + r) * s.H + h) * P + 8 * j;
      if (r >= n) {
        *reinterpret_cast<uint4 *>(sm.dO + at) = make_uint4(0, 0, 0, 0);
      } else if (gvec & 1) {
        cp16(dOs + at, src);
      } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) reinterpret_cast<__nv_bfloat16 *>(sm.dO + at)[y] = src[y];
      }
    }
    const uint32_t v = smem_at(sm.vec[i & 1]), u = smem_at(sm.up[i & 1]), w = smem_at(sm.ub[i & 1]);
    for (int x = tid; x < kVec / 4; x += kThreads) cp16(v + 16 * x, t.vec + ht * kVec + 4 * x);
    for (int x = tid; x < P / 4; x += kThreads) {
      cp16(u + 16 * x, t.up + ht * P + 4 * x);
      cp16(w + 16 * x, o.ub + ht * P + 4 * x);
    }
    cp_commit();
  };
  auto fetch_state = [&](uint32_t to, const __half *from, int i) {
    const uint8_t *src = reinterpret_cast<const uint8_t *>(from + (slot * s.H + grp * s.hpg + i) * P * N);
    for (int x = tid; x < P * N / 8; x += kThreads) cp16(to + 16 * x, src + 16 * x);
    cp_commit();
  };
  // the last step of a head, by one warp: the sums over the token strips and column halves, and dg's suffix sums
  auto finish = [&](int i) {
    const int x = i & 1, h = grp * s.hpg + i;
    const float *vec = sm.vec[x];
    float inner = 0.f, tail = 0.f;
    int some = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      inner += sm.inner[x][w];
      some |= sm.some[x][w];
    }
    float dG[2], db[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int r = 2 * lane + y;
      const float kz = sm.kz[x][0][r] + sm.kz[x][1][r];
      dG[y] = sm.row[x][0][r] + sm.row[x][1][r];
      db[y] = ((sm.col[x][0][r] + sm.col[x][1][r]) + (sm.col[x][2][r] + sm.col[x][3][r])) + kz;
      tail = fmaf(vec[kVecBeta + r], kz, tail);
    }
    tail = warp_sum(tail);
    if (lane == 31) dG[1] += fmaf(vec[kVecEg + kChunk - 1], inner, tail);
    float suf = dG[0] + dG[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float up = __shfl_down_sync(~0u, suf, d);
      if (lane + d < 32) suf += up;
    }
    const float after = __shfl_down_sync(~0u, suf, 1);
    const float later = lane == 31 ? 0.f : after;
    dG[1] += later;
    dG[0] += dG[1];
    // the first decay multiplies S0 alone: where that is zero the terms above cancel but for their rounding
    if (lane == 0 && !some) dG[0] = 0.f;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int r = 2 * lane + y;
      if (r < n) {
        static_cast<__nv_bfloat16 *>(a.dg)[(b + r) * s.H + h] = __float2bfloat16_rn(dG[y]);
        static_cast<__nv_bfloat16 *>(a.dbeta)[(b + r) * s.H + h] = __float2bfloat16_rn(db[y]);
      }
    }
  };

  {
    const uint8_t *K = reinterpret_cast<const uint8_t *>(t.K16 + (slot * s.G + grp) * kChunk * N);
    const uint8_t *Q = reinterpret_cast<const uint8_t *>(t.Q16 + (slot * s.G + grp) * kChunk * N);
    for (int x = tid; x < kChunk * N / 8; x += kThreads) {
      cp16(ks + 16 * x, K + 16 * x);
      cp16(qs + 16 * x, Q + 16 * x);
    }
    cp_commit();
    fetch_rows(0);
    cp_wait<1>();
    __syncthreads();
    float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll
    for (int k0 = 0; k0 < N; k0 += 16) {
      uint32_t ak[4], aq[4];
      ldsm4(ak, a_addr(ks, 16 * wm, k0, NB, lane));
      ldsm4(aq, a_addr(qs, 16 * wm, k0, NB, lane));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t bb[4];
        ldsm4(bb, b_addr(ks, 32 * wn + 16 * i, k0, NB, lane));
        mma(kk[2 * i], ak, bb[0], bb[1]);
        mma(kk[2 * i + 1], ak, bb[2], bb[3]);
        mma(qk[2 * i], aq, bb[0], bb[1]);
        mma(qk[2 * i + 1], aq, bb[2], bb[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sm.kk[i][tid] = make_float4(kk[i][0], kk[i][1], kk[i][2], kk[i][3]);
      sm.qk[i][tid] = make_float4(qk[i][0], qk[i][1], qk[i][2], qk[i][3]);
    }
  }
  const int rows[2] = {16 * wm + g, 16 * wm + g + 8};
  float dq[2 * kPairs][4] = {}, dk[2 * kPairs][4] = {};
  // k, q of this thread's accumulator element pair: rows[r], columns n0 + 8 i + c2
  const int n0 = wn * (N / 2);
  auto pair_of = [&](const uint8_t *tile, int r, int i) {
    return unpack(*reinterpret_cast<const uint32_t *>(tile + swz(rows[r], (n0 >> 3) + i, NB) + 2 * c2));
  };

  for (int i = 0; i < s.hpg; ++i) {
    const int x = i & 1;
    const float *vec = sm.vec[x], *up = sm.up[x], *ub = sm.ub[x];
    cp_wait<0>();
    __syncthreads();   // this head's rows are here, the head before is done with the state tiles
    fetch_state(Ds, o.D16, i);
    fetch_state(Ss, t.S16, i);
    if (i > 0 && warp == 0) finish(i - 1);
    const float ka = vec[kVecKa], qa = vec[kVecQa];
    uint32_t aO[kPMax / 16][4], aR[kPMax / 16][4];
    float sO[2], sR[2];
    rows_as_a<true>(aO, sO, dOs, 16 * wm, P, up, nullptr, lane);
    rows_as_a<false>(aR, sR, Rs, 16 * wm, P, up, ub, lane);
    float f1, f2;   // powers of two that the fp16 M1, M2 stand for
    {
      float n1[4][4] = {}, n2[4][4] = {};
#pragma unroll
      for (int j = 0; j < kPMax / 16; ++j)
        if (16 * j < P) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t bb[4];
            ldsm4(bb, b_addr(Es, 32 * wn + 16 * y, 16 * j, kRow, lane));
            mma(n1[2 * y], aR[j], bb[0], bb[1]);
            mma(n1[2 * y + 1], aR[j], bb[2], bb[3]);
            mma(n2[2 * y], aO[j], bb[0], bb[1]);
            mma(n2[2 * y + 1], aO[j], bb[2], bb[3]);
          }
        }
      float top1 = 0.f, top2 = 0.f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4 kk = sm.kk[y][tid], qk = sm.qk[y][tid];
        const float kkv[4] = {kk.x, kk.y, kk.z, kk.w}, qkv[4] = {qk.x, qk.y, qk.z, qk.w};
        float part[2] = {0.f, 0.f};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int r = rows[z >> 1], c = 32 * wn + 8 * y + c2 + (z & 1);
          const float d = c <= r ? __expf(acs_diff(vec[kVecG + r], vec[kVecGl + r], vec[kVecG + c], vec[kVecGl + c])) : 0.f;
          const float be = vec[kVecBeta + c];
          const float w1 = c < r ? n1[y][z] * sR[z >> 1] * d : 0.f, w2 = a.scale * n2[y][z] * sO[z >> 1] * d;
          const float w2l = c <= r ? w2 : 0.f;
          part[z & 1] += w2l * (qkv[z] * (qa * ka)) - w1 * (kkv[z] * (ka * ka));
          n1[y][z] = -w1 * be;
          n2[y][z] = w2l * be;
          top1 = fmaxf(top1, fabsf(n1[y][z]));
          top2 = fmaxf(top2, fabsf(n2[y][z]));
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {   // over this strip's 16 tokens
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) part[z] += __shfl_xor_sync(~0u, part[z], d);
          if (g == 0) sm.col[x][wm][32 * wn + 8 * y + c2 + z] = part[z];
        }
      }
      top1 = warp_max(top1);
      top2 = warp_max(top2);
      if (lane == 0) {
        sm.top[0][warp] = top1;
        sm.top[1][warp] = top2;
      }
      __syncthreads();
      top1 = top2 = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        top1 = fmaxf(top1, sm.top[0][w]);
        top2 = fmaxf(top2, sm.top[1][w]);
      }
      f1 = pow2_above(top1);
      f2 = pow2_above(top2);
      const float i1 = pow2_inv(f1), i2 = pow2_inv(f2);
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t at = swz(rows[r], 4 * wn + y, 128) + 2 * c2;
          *reinterpret_cast<uint32_t *>(sm.m1 + at) = pack(n1[y][2 * r] * i1, n1[y][2 * r + 1] * i1);
          *reinterpret_cast<uint32_t *>(sm.m2 + at) = pack(n2[y][2 * r] * i2, n2[y][2 * r + 1] * i2);
        }
    }
    cp_wait<1>();      // dS
    __syncthreads();   // M1 and M2 are here
    float rowsum[2] = {0.f, 0.f};
    {
      // down: Z, then M1^T K and M2^T Q on the same accumulators
      float z[2 * kPairs][4] = {}, sE[2];
      uint32_t aE[kPMax / 16][4];
      rows_as_a<false>(aE, sE, Es, 16 * wm, P, up, ub, lane);
#pragma unroll
      for (int j = 0; j < kPMax / 16; ++j)
        if (16 * j < P) step_t<kPairs>(z, aE[j], Ds, n0, 16 * j, NB, lane);
      const float u1 = f1 * ka, u2 = f2 * qa;
      float w[2], kz[2] = {0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 2; ++r) w[r] = sE[r] * vec[kVecTail + rows[r]];
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 k = pair_of(sm.k, r, y);
          const float z0 = z[y][2 * r] * w[r], z1 = z[y][2 * r + 1] * w[r];
          kz[r] = fmaf(k.x, z0, fmaf(k.y, z1, kz[r]));
          const float be = vec[kVecBeta + rows[r]] * pow2_inv(u1);
          z[y][2 * r] = z0 * be;
          z[y][2 * r + 1] = z1 * be;
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        kz[r] = quad_sum(kz[r]) * ka;
        if (c2 == 0) sm.kz[x][wn][rows[r]] = kz[r];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)   // tokens t >= s only
        if (j >= wm) {
          uint32_t am[4];
          ldsm4t(am, at_addr(m1s, 16 * wm, 16 * j, 128, lane));
          step_t<kPairs>(z, am, ks, n0, 16 * j, NB, lane);
        }
      const float ratio = u1 * pow2_inv(u2);
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[y][r] *= ratio;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= wm) {
          uint32_t am[4];
          ldsm4t(am, at_addr(m2s, 16 * wm, 16 * j, 128, lane));
          step_t<kPairs>(z, am, qs, n0, 16 * j, NB, lane);
        }
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 k = pair_of(sm.k, r, y);
          const float d0 = z[y][2 * r] * u2, d1 = z[y][2 * r + 1] * u2;
          rowsum[r] -= ka * fmaf(k.x, d0, k.y * d1);
          dk[y][2 * r] += d0;
          dk[y][2 * r + 1] += d1;
        }
    }
    cp_wait<0>();      // S0
    __syncthreads();   // dO, R16 and E16 have been read
    if (i + 1 < s.hpg) fetch_rows(i + 1);
    {
      // <S0, dS>: the same element of both tiles at the same place
      float inner = 0.f;
      int some = 0;
      for (int y = tid; y < P * N / 8; y += kThreads) {
        const uint4 u = *reinterpret_cast<const uint4 *>(sm.S + 16 * y), v = *reinterpret_cast<const uint4 *>(sm.D + 16 * y);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
        const int p = y / (N / 8);
        float acc = 0.f;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float2 fu = unpack(uu[z]), fv = unpack(vv[z]);
          acc = fmaf(fu.x, fv.x, fmaf(fu.y, fv.y, acc));
          some |= (uu[z] & 0x7fff7fffu) != 0;
        }
        inner = fmaf(acc, up[p] * ub[p], inner);
      }
      inner = warp_sum(inner);
      some = __any_sync(~0u, some);
      if (lane == 0) {
        sm.inner[x][warp] = inner;
        sm.some[x][warp] = some;
      }
    }
    {
      float y1[2 * kPairs][4] = {};
#pragma unroll
      for (int j = 0; j < kPMax / 16; ++j)
        if (16 * j < P) step_t<kPairs>(y1, aO[j], Ss, n0, 16 * j, NB, lane);
      const float u2 = f2 * ka;
      float w[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) w[r] = a.scale * sO[r] * vec[kVecEg + rows[r]] * pow2_inv(u2);
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 4; ++r) y1[y][r] *= w[r >> 1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= wm) {
          uint32_t am[4];
          ldsm4(am, a_addr(m2s, 16 * wm, 16 * j, 128, lane));
          step_t<kPairs>(y1, am, ks, n0, 16 * j, NB, lane);
        }
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 q = pair_of(sm.q, r, y);
          const float d0 = y1[y][2 * r] * u2, d1 = y1[y][2 * r + 1] * u2;
          rowsum[r] += qa * fmaf(q.x, d0, q.y * d1);
          dq[y][2 * r] += d0;
          dq[y][2 * r + 1] += d1;
        }
    }
    {
      float y2[2 * kPairs][4] = {};
#pragma unroll
      for (int j = 0; j < kPMax / 16; ++j)
        if (16 * j < P) step_t<kPairs>(y2, aR[j], Ss, n0, 16 * j, NB, lane);
      const float u1 = f1 * ka;
      float w[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) w[r] = -sR[r] * vec[kVecEg + rows[r]] * pow2_inv(u1);
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 4; ++r) y2[y][r] *= w[r >> 1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= wm) {
          uint32_t am[4];
          ldsm4(am, a_addr(m1s, 16 * wm, 16 * j, 128, lane));
          step_t<kPairs>(y2, am, ks, n0, 16 * j, NB, lane);
        }
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 k = pair_of(sm.k, r, y);
          const float d0 = y2[y][2 * r] * u1, d1 = y2[y][2 * r + 1] * u1;
          rowsum[r] += ka * fmaf(k.x, d0, k.y * d1);
          dk[y][2 * r] += d0;
          dk[y][2 * r + 1] += d1;
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      rowsum[r] = quad_sum(rowsum[r]);
      if (c2 == 0) sm.row[x][wn][rows[r]] = rowsum[r];
    }
  }
  __syncthreads();
  if (warp == 0) finish(s.hpg - 1);
  __nv_bfloat16 *oq = static_cast<__nv_bfloat16 *>(a.dq), *ok = static_cast<__nv_bfloat16 *>(a.dk);
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (rows[r] < n) {
      const int64_t at = ((b + rows[r]) * s.G + grp) * N + n0 + c2;
#pragma unroll
      for (int y = 0; y < 2 * kPairs; ++y) {
        const uint32_t vq = pack_bf16(dq[y][2 * r], dq[y][2 * r + 1]), vk = pack_bf16(dk[y][2 * r], dk[y][2 * r + 1]);
        if (gvec & 2) {
          *reinterpret_cast<uint32_t *>(oq + at + 8 * y) = vq;
          *reinterpret_cast<uint32_t *>(ok + at + 8 * y) = vk;
        } else {
          oq[at + 8 * y] = __ushort_as_bfloat16(static_cast<unsigned short>(vq & 0xffffu));
          oq[at + 8 * y + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(vq >> 16));
          ok[at + 8 * y] = __ushort_as_bfloat16(static_cast<unsigned short>(vk & 0xffffu));
          ok[at + 8 * y + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(vk >> 16));
        }
      }
    }
}

template <int N>
cudaError_t launch(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  const int smem = int(sizeof(Smem<N>));
  const cudaError_t e = cudaFuncSetAttribute(grads_tile_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const bool rows16 = (reinterpret_cast<uintptr_t>(a.dout) & 15) == 0;
  const bool out4 = ((reinterpret_cast<uintptr_t>(a.dq) | reinterpret_cast<uintptr_t>(a.dk)) & 3) == 0;
  grads_tile_kernel<N><<<dim3(unsigned(s.slots), unsigned(s.G)), kThreads, smem, st>>>(
      s, a, t, o, (rows16 ? 1 : 0) | (out4 ? 2 : 0));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grads(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  if (s.slots == 0 || s.total == 0) return cudaSuccess;
  return s.N == 64 ? launch<64>(s, a, t, o, st) : launch<128>(s, a, t, o, st);
}

}  // namespace delta
}  // namespace ssd
