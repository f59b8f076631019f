// ssd_delta_prep.cu -- the parts of the gated delta rule that chunks can do side
// by side, before the chains go from chunk to chunk: prep_kernel before the
// forward's, prep_bwd_kernel before the backward's.  What they make is listed in
// ssd_delta_tiles.cuh.
//
// With L_ts = exp(G_t - G_s) (k_t . k_s), s < t, the chunk's equation for e is
//     (I + L beta) E = V - exp(G) K S0^T,
// and with Y = (I + L beta)^-1 L (beta: the diagonal matrix) its inverse is
// I - Y beta, without a division by beta, as (I + beta L)^-T is I - (beta Y)^T.
// So E = V' - W S0^T with V' = (I - Y beta) V, W = (I - Y beta) exp(G) K, both
// free of the state: the chain's step is one product with S, not two in a row.
// The backward likewise: F = A + B dS^T.
//
// CTA (chunk slot, group), 4 warps: k and q of the chunk once, K K^T and Q K^T on
// the tensor cores (fp16 operands are exact here: bf16 input scaled by a power of
// two), then the heads of the group, two at a time.  Y is found in fp32 by forward
// substitution, one thread a column, 16 rows at a time:
//     Y[t][j] = L[t][j] - sum_{j<s<t} L[t][s] beta_s Y[s][j],
// the 16 rows as packed pairs of fp32, earlier rows of the column read back from
// shared memory.  (With the whole column in registers the unrolled code, 2000
// products, did not fit the instruction cache: 220 us instead of 170 for 256
// chunks of 32 heads.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr int kThreads = 128;
constexpr int kPad = kChunk + 4;   // floats of a row of L and Y in shared memory
constexpr int kPMax = 128;

template <int N>
struct Smem {
  __half k[kChunk * N];
  union {
    __half q[kChunk * N];
    struct {   // of two heads, once the products of k and q are taken
      union {
        float L[2][kChunk][kPad];          // [s][t]
        __half v[2][kChunk * kPMax];       // v rows [t][p], once Y is found
      };
      float Y[2][kChunk][kPad];            // [t][s]
    };
  };
  float top[4][kThreads / 32];    // largest |k|, |q|, |v| of two heads, of each warp's part
  float G[2][kChunk], Gl[2][kChunk], beta[2][kChunk], eg[2][kChunk];
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4 *>(p);
  const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
  return make_uint4(u[0] | uint32_t(u[1]) << 16, u[2] | uint32_t(u[3]) << 16, u[4] | uint32_t(u[5]) << 16,
                    u[6] | uint32_t(u[7]) << 16);
}
__device__ __forceinline__ float top_of(const uint4 &u, float m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16(w[j]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return m;
}
__device__ __forceinline__ uint4 to_f16(const uint4 &u, float f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = unpack_bf16(w[j]);
    o[j] = pack(v.x * f, v.y * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  return m;
}
// Power of two that brings a tile's largest value `m` into [8, 16).
__device__ __forceinline__ float tile_scale(float m) { return pow2_above(m * 0.0625f); }

// This thread's part (16-byte pieces) of 64 rows of `cols` bf16, rows past the end zero; its largest magnitude.
template <int kPieces>
__device__ __forceinline__ float rows_in(const __nv_bfloat16 *src, int64_t stride, int n, int cols, bool vec,
                                         uint4 (&raw)[kPieces]) {
  const int per = cols / 8;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int x = threadIdx.x + i * kThreads, r = x / per;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r < n) raw[i] = load16(src + int64_t(r) * stride + 8 * (x % per), vec);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) m = top_of(raw[i], m);
  return warp_max(m);
}
// They times `f` as fp16 in panels, to shared memory and, where gtile is given, global memory.
template <int kPieces>
__device__ __forceinline__ void rows_out(const uint4 (&raw)[kPieces], float f, int cols, __half *tile, __half *gtile) {
  const int per = cols / 8;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int x = threadIdx.x + i * kThreads, r = x / per;
    if (r < kChunk) {
      const uint4 v = to_f16(raw[i], f);
      const uint32_t at = pan(r, x % per, kChunk);
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(tile) + at) = v;
      if (gtile != nullptr) *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(gtile) + at) = v;
    }
  }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b),
                     z = *reinterpret_cast<unsigned long long *>(&c);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(z) : "l"(x), "l"(y));
  return *reinterpret_cast<float2 *>(&z);
}

// Column j of Y; a warp has 32 neighbouring columns, the first of them j0 (rows up to j0 are zero).
__device__ __forceinline__ void solve(const float (*L)[kPad], const float *beta, float (*Y)[kPad], int j, int j0) {
#pragma unroll 1
  for (int r0 = j0; r0 < kChunk; r0 += 16) {
    float2 acc[8];
    const bool below = r0 + 16 > j;   // this strip of rows has a part of L's column j
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 v = below ? *reinterpret_cast<const float4 *>(&L[j][r0 + 2 * i]) : make_float4(0.f, 0.f, 0.f, 0.f);
      acc[i] = make_float2(v.x, v.y);
      acc[i + 1] = make_float2(v.z, v.w);
    }
#pragma unroll 4
    for (int s = j0; s < r0; ++s) {
      const float z = -beta[s] * Y[s][j];
      const float2 zz = make_float2(z, z);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(&L[s][r0 + 2 * i]);
        acc[i] = fma2(make_float2(v.x, v.y), zz, acc[i]);
        acc[i + 1] = fma2(make_float2(v.z, v.w), zz, acc[i + 1]);
      }
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float y = t & 1 ? acc[t >> 1].y : acc[t >> 1].x;
      Y[r0 + t][j] = y;
      const float z = -beta[r0 + t] * y;
      const float2 zz = make_float2(z, z);
#pragma unroll
      for (int i = (t + 1) / 4 * 2; i < 8; i += 2) {   // L is zero on and above the diagonal of this block
        const float4 v = *reinterpret_cast<const float4 *>(&L[r0 + t][r0 + 2 * i]);
        acc[i] = fma2(make_float2(v.x, v.y), zz, acc[i]);
        acc[i + 1] = fma2(make_float2(v.z, v.w), zz, acc[i + 1]);
      }
    }
  }
}

// The running sums of g as hi + lo (G, Gl), two tokens a lane.
__device__ __forceinline__ void running_sums(const float (&v)[2], float *G, float *Gl, int lane) {
  auto add = [](float &hi, float &lo, float yh, float yl) {   // (hi, lo) += (yh, yl)
    const float sum = __fadd_rn(hi, yh), bb = __fsub_rn(sum, hi);
    const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, bb)), __fsub_rn(yh, bb));
    lo = __fadd_rn(__fadd_rn(lo, yl), err);
    hi = sum;
  };
  float hi = v[0], lo = 0.f;
  add(hi, lo, v[1], 0.f);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float ph = __shfl_up_sync(~0u, hi, d), pl = __shfl_up_sync(~0u, lo, d);
    if (lane >= d) add(hi, lo, ph, pl);
  }
  G[2 * lane + 1] = hi;
  Gl[2 * lane + 1] = lo;
  float eh = __shfl_up_sync(~0u, hi, 1), el = __shfl_up_sync(~0u, lo, 1);
  if (lane == 0) eh = el = 0.f;
  add(eh, el, v[0], 0.f);
  G[2 * lane] = eh;
  Gl[2 * lane] = el;
}

// 16 rows of a product with column tiles 2 kPairs from n0: d -= A B, B from rows [k][n] of a panel tile.
template <int kTerms, int kPairs>
__device__ __forceinline__ void step(float (&d)[2 * kPairs][4], const uint32_t (&a)[kTerms][4], uint32_t tile, int n0,
                                     int k0, int lane) {
  auto at = [&](int r, int j) { return tile + pan(r, j, kChunk); };
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    uint32_t b[4];
    ldsm4t(b, bt_addr(at, n0 + 16 * i, k0, lane));
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      mma(d[2 * i], a[t], b[0], b[1]);
      mma(d[2 * i + 1], a[t], b[2], b[3]);
    }
  }
}

template <int N, int kTerms>
__global__ void __launch_bounds__(kThreads, 2) prep_kernel(Shape s, Args a, Tiles o, int vec) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<N> &sm = *reinterpret_cast<Smem<N> *>(raw);
  constexpr int kPieces = kChunk * N / 8 / kThreads;
  const int64_t slot = blockIdx.x;
  const int grp = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c2 = 2 * (lane & 3);
  // the warps' shares of a chunk are unequal: they change places from CTA to CTA, so that no SM partition has them all
  const int role = (warp + blockIdx.x) & 3;
  if (slot == 0 && grp == 0 && tid == 0) *o.status = 0;
  int64_t seq, b, e;
  if (!chunk_of_slot(s, a.cu, slot, seq, b, e)) return;
  const int n = int(e - b), P = s.P;
  const int64_t tile = (slot * s.G + grp) * kChunk * N;
  float ka;
  {
    uint4 rk[kPieces], rq[kPieces];
    const float mk = rows_in<kPieces>(static_cast<const __nv_bfloat16 *>(a.k) + b * s.ks + int64_t(grp) * N, s.ks, n, N,
                                      vec & 2, rk);
    const float mq = rows_in<kPieces>(static_cast<const __nv_bfloat16 *>(a.q) + b * s.qs + int64_t(grp) * N, s.qs, n, N,
                                      vec & 1, rq);
    if (lane == 0) {
      sm.top[0][warp] = mk;
      sm.top[1][warp] = mq;
    }
    __syncthreads();
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, fmaxf(sm.top[0][i], sm.top[1][i]));
    // one scale for both, so that their products with one matrix can be added up
    ka = tile_scale(top);
    rows_out<kPieces>(rk, pow2_inv(ka), N, sm.k, o.K16 + tile);
    rows_out<kPieces>(rq, pow2_inv(ka), N, sm.q, o.Q16 + tile);
  }
  __syncthreads();
  // rows 16 role.. of K K^T and Q K^T, columns up to the diagonal block
  float kk[8][4] = {}, qk[8][4] = {};
  const uint32_t ks = smem_at(sm.k), qs = smem_at(sm.q);
  auto kat = [&](int r, int j) { return ks + pan(r, j, kChunk); };
  auto qat = [&](int r, int j) { return qs + pan(r, j, kChunk); };
#pragma unroll
  for (int k0 = 0; k0 < N; k0 += 16) {
    uint32_t ak[4], aq[4];
    ldsm4(ak, a_addr(kat, 16 * role, k0, lane));
    ldsm4(aq, a_addr(qat, 16 * role, k0, lane));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= role) {
        uint32_t bb[4];
        ldsm4(bb, b_addr(kat, 16 * j, k0, lane));
        mma(kk[2 * j], ak, bb[0], bb[1]);
        mma(kk[2 * j + 1], ak, bb[2], bb[3]);
        mma(qk[2 * j], aq, bb[0], bb[1]);
        mma(qk[2 * j + 1], aq, bb[2], bb[3]);
      }
  }
  const int rows[2] = {16 * role + g, 16 * role + g + 8};
  const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + b * s.vs;
  for (int h0 = 0; h0 < s.hpg; h0 += 2) {
    const int nh = min(2, s.hpg - h0);
    __syncthreads();   // the products of k and q are taken, the heads before are done with Y, v and the vectors
    if (warp < nh) {
      const int h = grp * s.hpg + h0 + warp;
      float x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        // a decay to nothing stays a finite number: exp(-1e4) is zero all the same
        x[i] = t < n ? fmaxf(a.g[(b + t) * s.H + h], -1e4f) : 0.f;
        sm.beta[warp][t] = t < n ? a.beta[(b + t) * s.H + h] : 0.f;
      }
      running_sums(x, sm.G[warp], sm.Gl[warp], lane);
    }
    // v of both heads, on its way while Y is found
    uint4 rv[2][kChunk * kPMax / 8 / kThreads];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (w < nh) {
        const float m = rows_in<kChunk * kPMax / 8 / kThreads>(v + int64_t(grp * s.hpg + h0 + w) * P, s.vs, n, P, vec & 4,
                                                               rv[w]);
        if (lane == 0) sm.top[2 + w][warp] = m;
      }
    __syncthreads();
    for (int w = 0; w < nh; ++w) {
      const int64_t at = slot * s.H + grp * s.hpg + h0 + w;
      const float *G = sm.G[w], *Gl = sm.Gl[w];
      uint8_t *Pt = reinterpret_cast<uint8_t *>(o.P16 + at * kTri);
      const float Gr[2] = {G[rows[0]], G[rows[1]]}, Glr[2] = {Gl[rows[0]], Gl[rows[1]]};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = 8 * j + c2;
        if (j <= 2 * role + 1) {
          const float g0 = G[c], g1 = G[c + 1], l0 = Gl[c], l1 = Gl[c + 1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = rows[i];
            const float d0 = c <= t ? __expf(acs_diff(Gr[i], Glr[i], g0, l0)) : 0.f;
            const float d1 = c + 1 <= t ? __expf(acs_diff(Gr[i], Glr[i], g1, l1)) : 0.f;
            sm.L[w][c][t] = c < t ? d0 * kk[j][2 * i] * (ka * ka) : 0.f;
            sm.L[w][c + 1][t] = c + 1 < t ? d1 * kk[j][2 * i + 1] * (ka * ka) : 0.f;
            *reinterpret_cast<uint32_t *>(Pt + swz(t, j, 128) + 2 * c2) = pack(d0 * qk[j][2 * i], d1 * qk[j][2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) *reinterpret_cast<uint32_t *>(Pt + swz(rows[i], j, 128) + 2 * c2) = 0u;
        }
      }
      if (tid < kChunk) {
        float *vc = o.vec + at * kVec;
        const float eg = expf(G[tid] + Gl[tid]);
        sm.eg[w][tid] = eg;
        vc[kVecEg + tid] = eg;
        vc[kVecTail + tid] = expf(acs_diff(G[kChunk - 1], Gl[kChunk - 1], G[tid], Gl[tid]));
        vc[kVecBeta + tid] = sm.beta[w][tid];
        vc[kVecG + tid] = G[tid];
        vc[kVecGl + tid] = Gl[tid];
      }
    }
    __syncthreads();
    if ((role >> 1) < nh) solve(sm.L[role >> 1], sm.beta[role >> 1], sm.Y[role >> 1], 32 * (role & 1) + lane, 32 * (role & 1));
    __syncthreads();
    float sv[2] = {1.f, 1.f};
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (w < nh) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, sm.top[2 + w][i]);
        sv[w] = tile_scale(m);
        rows_out<kChunk * kPMax / 8 / kThreads>(rv[w], pow2_inv(sv[w]), P, sm.v[w], nullptr);
        if (tid == 0) {
          float *vc = o.vec + (slot * s.H + grp * s.hpg + h0 + w) * kVec;
          vc[kVecKa] = ka;
          vc[kVecSv] = sv[w];
        }
      }
    __syncthreads();
    for (int w = 0; w < nh; ++w) {
      const int64_t at = slot * s.H + grp * s.hpg + h0 + w;
      const float *beta = sm.beta[w], *eg = sm.eg[w];
      // W = exp(G) K - (Y beta exp(G)) K, V' = V - (Y beta) V, 16 rows a warp
      const uint32_t vs = smem_at(sm.v[w]);
      auto y_of = [&](int r, int c) {   // Y[rows[r]][c], c + 1
        const bool on = c < 32 || rows[r] >= 32;   // columns from 32 have no rows above 32
        return on ? *reinterpret_cast<const float2 *>(&sm.Y[w][rows[r]][c]) : make_float2(0.f, 0.f);
      };
      if (o.Y16 != nullptr) {
        uint8_t *Yt = reinterpret_cast<uint8_t *>(o.Y16 + at * kTri);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 y = j <= 2 * role + 1 ? y_of(r, 8 * j + c2) : make_float2(0.f, 0.f);
            *reinterpret_cast<uint32_t *>(Yt + swz(rows[r], j, 128) + 2 * c2) =
                pack(beta[rows[r]] * y.x, beta[rows[r]] * y.y);
          }
      }
      // the left operand of step j: -16 Y beta (times exp(G) for W); 16 keeps a second term a normal fp16
      auto left = [&](int j, bool decay, uint32_t (&A)[kTerms][4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 16 * j + 8 * (i >> 1) + c2;
          const float2 y = y_of(i & 1, c);
          float f0 = -16.f * beta[c], f1 = -16.f * beta[c + 1];
          if (decay) f0 *= eg[c], f1 *= eg[c + 1];
          uint32_t p[kTerms];
          split<kTerms>(y.x * f0, y.y * f1, p);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) A[t][i] = p[t];
        }
      };
      uint8_t *Wt = reinterpret_cast<uint8_t *>(o.W16 + at * kTerms * kChunk * N);
      const float er[2] = {eg[rows[0]], eg[rows[1]]};
#pragma unroll 1
      for (int n0 = 0; n0 < N; n0 += 64) {
        float d[8][4] = {};
#pragma unroll 1
        for (int j = 0; j <= role; ++j) {
          uint32_t A[kTerms][4];
          left(j, true, A);
          step<kTerms, 4>(d, A, ks, n0, 16 * j, lane);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t to = pan(rows[r], (n0 >> 3) + i, kChunk) + 2 * c2;
            const float2 k = unpack(*reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(sm.k) + to));
            uint32_t p[kTerms];
            split<kTerms>(fmaf(er[r], k.x, d[i][2 * r] * 0.0625f), fmaf(er[r], k.y, d[i][2 * r + 1] * 0.0625f), p);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) *reinterpret_cast<uint32_t *>(Wt + t * kChunk * N * 2 + to) = p[t];
          }
      }
      __half *Vt = o.V16 + at * kTerms * kChunk * P;
#pragma unroll 1
      for (int n0 = 0; n0 < P; n0 += 64) {
        float d[8][4] = {};
#pragma unroll 1
        for (int j = 0; j <= role; ++j) {
          uint32_t A[kTerms][4];
          left(j, false, A);
          step<kTerms, 4>(d, A, vs, n0, 16 * j, lane);   // columns past P are another head's or old: not stored
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n0 + 8 * i < P) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t from = pan(rows[r], (n0 >> 3) + i, kChunk) + 2 * c2;
              const float2 x = unpack(*reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(sm.v[w]) + from));
              uint32_t p[kTerms];
              split<kTerms>(fmaf(0.0625f, d[i][2 * r], x.x), fmaf(0.0625f, d[i][2 * r + 1], x.y), p);
#pragma unroll
              for (int t = 0; t < kTerms; ++t)
                *reinterpret_cast<uint32_t *>(Vt + (t * kChunk + rows[r]) * P + n0 + 8 * i + c2) = p[t];
            }
          }
      }
    }
  }
}

// ---- before the backward's chain ---------------------------------------------

template <int N>
struct BwdSmem {
  __half k[kChunk * N], x[kChunk * kPMax], u[kChunk * kPMax];   // k; dO [t][p]; scale 2^a P^T dO
  __half P[kTri], Y[kTri];
  float vec[kVec];
  float top[2][kThreads / 32];
};

// CTA (chunk slot, head): B = tail K - (beta Y)^T tail K and A = (I - (beta Y)^T) scale 2^a P^T dO, with the copies of dO
// that the chain and the gradient kernel read.
template <int N>
__global__ void __launch_bounds__(kThreads) prep_bwd_kernel(Shape s, Args a, Tiles t, BwdTiles o, int vec) {
  extern __shared__ __align__(1024) uint8_t raw[];
  BwdSmem<N> &sm = *reinterpret_cast<BwdSmem<N> *>(raw);
  const int64_t slot = blockIdx.x;
  const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c2 = 2 * (lane & 3);
  const int role = (warp + blockIdx.x) & 3, P = s.P;
  if (slot == 0 && h == 0 && tid == 0) *o.status = 0;
  int64_t seq, b, e;
  if (!chunk_of_slot(s, a.cu, slot, seq, b, e)) return;
  const int n = int(e - b);
  const int64_t at = slot * s.H + h;
  const uint32_t ks = smem_at(sm.k), xs = smem_at(sm.x), us = smem_at(sm.u), Ps = smem_at(sm.P), Ys = smem_at(sm.Y);
  {
    const __half *K = t.K16 + (slot * s.G + h / s.hpg) * kChunk * N;
    for (int i = tid; i < kChunk * N / 8; i += kThreads) cp16(ks + 16 * i, K + 8 * i);
    for (int i = tid; i < kTri / 8; i += kThreads) {
      cp16(Ps + 16 * i, t.P16 + at * kTri + 8 * i);
      cp16(Ys + 16 * i, t.Y16 + at * kTri + 8 * i);
    }
    for (int i = tid; i < kVec / 4; i += kThreads) cp16(smem_at(sm.vec) + 16 * i, t.vec + at * kVec + 4 * i);
    cp_commit();
  }
  constexpr int kPieces = kChunk * kPMax / 8 / kThreads;
  uint4 rx[kPieces];
  const float m = rows_in<kPieces>(static_cast<const __nv_bfloat16 *>(a.dout) + (b * s.H + h) * P, int64_t(s.H) * P, n, P,
                                   vec & 1, rx);
  if (lane == 0) sm.top[0][warp] = m;
  cp_wait<0>();
  __syncthreads();
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, sm.top[0][i]);
  const float sx = tile_scale(top), ix = pow2_inv(sx);
  rows_out<kPieces>(rx, ix, P, sm.x, o.X16 + at * kChunk * padded(P));
  {
    const int per = P / 8;
    uint8_t *to = reinterpret_cast<uint8_t *>(o.X2 + at * kChunk * padded(P));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = tid + i * kThreads, r = x / per;
      if (r < kChunk) *reinterpret_cast<uint4 *>(to + pan(r, x % per, kChunk)) = to_f16(rx[i], ix * sm.vec[kVecEg + r]);
    }
  }
  __syncthreads();
  auto pat = [&](int r, int j) { return Ps + swz(r, j, 128); };
  auto yat = [&](int r, int j) { return Ys + swz(r, j, 128); };
  const int rows[2] = {16 * role + g, 16 * role + g + 8};
  // U = P^T dO in units of 2^x (16 bits of P16 are bounded by 2^15, so by a further 2^-10), 16 rows (s) a warp
  constexpr float kU = 1.f / 1024.f;
  float u[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) u[i][r] = 0.f;
#pragma unroll 1
  for (int j = role; j < 4; ++j) {
    uint32_t A[1][4];
    ldsm4t(A[0], at_addr(pat, 16 * role, 16 * j, lane));
    float(&lo)[8][4] = *reinterpret_cast<float(*)[8][4]>(&u[0]);
    float(&hi)[8][4] = *reinterpret_cast<float(*)[8][4]>(&u[8]);
    step<1, 4>(lo, A, xs, 0, 16 * j, lane);
    if (P > 64) step<1, 4>(hi, A, xs, 64, 16 * j, lane);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (8 * i < P) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(sm.u) + pan(rows[r], i, kChunk) + 2 * c2) =
            pack(u[i][2 * r] * kU, u[i][2 * r + 1] * kU);
    }
  __syncthreads();
  // A = U - (beta Y)^T U: the right operand is U's fp16, the first term its fp32
  {
    float d[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) d[i][r] = 0.f;
#pragma unroll 1
    for (int j = role; j < 4; ++j) {
      uint32_t A[1][4];
      ldsm4t(A[0], at_addr(yat, 16 * role, 16 * j, lane));
      float(&lo)[8][4] = *reinterpret_cast<float(*)[8][4]>(&d[0]);
      float(&hi)[8][4] = *reinterpret_cast<float(*)[8][4]>(&d[8]);
      step<1, 4>(lo, A, us, 0, 16 * j, lane);
      if (P > 64) step<1, 4>(hi, A, us, 64, 16 * j, lane);
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (8 * i < P) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          d[i][r] = fmaf(u[i][r], kU, -d[i][r]);
          mx = fmaxf(mx, fabsf(d[i][r]));
        }
      }
    mx = warp_max(mx);
    if (lane == 0) sm.top[1][warp] = mx;
    __syncthreads();
    mx = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, sm.top[1][i]);
    const float sf = tile_scale(mx), jf = pow2_inv(sf);
    __half *to = o.A16 + at * kChunk * P;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (8 * i < P) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<uint32_t *>(to + rows[r] * P + 8 * i + c2) = pack(d[i][2 * r] * jf, d[i][2 * r + 1] * jf);
      }
    if (tid == 0) {
      // A16's unit takes in all of scale 2^a (of P16's k) 2^a (of its q)
      const float ka = sm.vec[kVecKa];
      o.side[at * kSide] = sf * sx * (1.f / kU) * a.scale * ka * ka;
      o.side[at * kSide + 1] = sx;
    }
  }
  // B = tail K - (beta Y)^T tail K
  uint8_t *Bt = reinterpret_cast<uint8_t *>(o.B16 + at * kChunk * N);
  const float *tail = sm.vec + kVecTail;
#pragma unroll 1
  for (int n0 = 0; n0 < N; n0 += 64) {
    float d[8][4] = {};
#pragma unroll 1
    for (int j = role; j < 4; ++j) {
      uint32_t A[1][4];
      ldsm4t(A[0], at_addr(yat, 16 * role, 16 * j, lane));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 16 * j + 8 * (i >> 1) + c2;
        const float2 y = unpack(A[0][i]);
        A[0][i] = pack(-y.x * tail[c], -y.y * tail[c + 1]);
      }
      step<1, 4>(d, A, ks, n0, 16 * j, lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t to = pan(rows[r], (n0 >> 3) + i, kChunk) + 2 * c2;
        const float2 k = unpack(*reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(sm.k) + to));
        *reinterpret_cast<uint32_t *>(Bt + to) =
            pack(fmaf(tail[rows[r]], k.x, d[i][2 * r]), fmaf(tail[rows[r]], k.y, d[i][2 * r + 1]));
      }
  }
}

bool vec16(const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

template <int N, int kTerms>
cudaError_t launch(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  const int smem = int(sizeof(Smem<N>));
  const cudaError_t e = cudaFuncSetAttribute(prep_kernel<N, kTerms>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int vec = (vec16(a.q, s.qs) ? 1 : 0) | (vec16(a.k, s.ks) ? 2 : 0) | (vec16(a.v, s.vs) ? 4 : 0);
  prep_kernel<N, kTerms><<<dim3(unsigned(s.slots), unsigned(s.G)), kThreads, smem, st>>>(s, a, t, vec);
  return cudaGetLastError();
}

template <int N>
cudaError_t launch_b(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  const int smem = int(sizeof(BwdSmem<N>));
  const cudaError_t e = cudaFuncSetAttribute(prep_bwd_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prep_bwd_kernel<N><<<dim3(unsigned(s.slots), unsigned(s.H)), kThreads, smem, st>>>(s, a, t, o, vec16(a.dout, 8));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  if (s.slots == 0 || s.total == 0) return cudaMemsetAsync(t.status, 0, sizeof(int), st);
  if (s.N == 64) return t.planes == 2 ? launch<64, 2>(s, a, t, st) : launch<64, 1>(s, a, t, st);
  return t.planes == 2 ? launch<128, 2>(s, a, t, st) : launch<128, 1>(s, a, t, st);
}

cudaError_t launch_prep_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &o, cudaStream_t st) {
  if (s.slots == 0 || s.total == 0) return cudaMemsetAsync(o.status, 0, sizeof(int), st);
  return s.N == 64 ? launch_b<64>(s, a, t, o, st) : launch_b<128>(s, a, t, o, st);
}

}  // namespace delta
}  // namespace ssd
