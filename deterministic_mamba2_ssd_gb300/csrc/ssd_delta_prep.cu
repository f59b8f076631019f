// ssd_delta_prep.cu -- the part of the gated delta rule that chunks can do
// side by side: for every chunk and head, with L_ts = exp(G_t - G_s) (k_t . k_s)
// for s < t, the matrix Y = (I + L diag(beta))^-1 L, the decayed scores
// q_t . k_s, and the vectors of decays and scales (see ssd_delta_tiles.cuh).
// Y serves both directions without a division by beta:
//     (I + L diag(beta))^-1 R = R - Y (beta R),
//     (I + diag(beta) L)^-T U = U - Y^T (beta U).
//
// CTA (chunk slot, group): k and q of the chunk once, K K^T and Q K^T on the
// tensor cores (fp16 operands are exact here: bf16 rows scaled by a power of
// two), then the heads of the group, two at a time.  Y is found in fp32 by
// forward substitution, one thread a column, 16 rows at a time:
//     Y[t][j] = L[t][j] - sum_{j<s<t} L[t][s] beta_s Y[s][j],
// the 16 rows as packed pairs of fp32, earlier rows of the column read back
// from shared memory.  (With the whole column in registers the unrolled code,
// 2000 products, did not fit the instruction cache: 220 us instead of 80 for
// 256 chunks of 32 heads.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = float(1.4426950408889634 - double(kLog2e));
constexpr int kPad = kChunk + 4;   // floats of a row of A and X in shared memory

template <int N>
struct Smem {
  union {
    struct {
      __half k[kChunk * N], q[kChunk * N];
    };
    struct {   // of two heads, once the products of k and q are taken
      float L[2][kChunk][kPad];   // [s][t]
      float Y[2][kChunk][kPad];   // [t][s]
    };
  };
  float top[2][kThreads / 32];    // largest |k|, |q| of each warp's part
  float G[2][kChunk], Gl[2][kChunk], beta[2][kChunk];
};

// This thread's part of the chunk's rows of q or k (16-byte pieces; rows past the end zero) and its largest magnitude.
template <int N>
__device__ __forceinline__ float rows_in(const __nv_bfloat16 *src, int64_t stride, int n, bool vec,
                                         uint4 (&raw)[kChunk * N / 8 / kThreads]) {
  constexpr int L = N / 8;   // lanes of a row
  const int l = threadIdx.x % L;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kChunk * L / kThreads; ++i) {
    const int r = threadIdx.x / L + i * (kThreads / L);
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r >= n) continue;
    const __nv_bfloat16 *p = src + int64_t(r) * stride + 8 * l;
    if (vec) {
      raw[i] = *reinterpret_cast<const uint4 *>(p);
    } else {
      const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
      raw[i] = make_uint4(u[0] | uint32_t(u[1]) << 16, u[2] | uint32_t(u[3]) << 16, u[4] | uint32_t(u[5]) << 16,
                          u[6] | uint32_t(u[7]) << 16);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunk * L / kThreads; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16(w[j]);
      m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  return m;
}

// The rows times `inv` as fp16, to shared memory's tile and to global memory.
template <int N>
__device__ __forceinline__ void rows_out(const uint4 (&raw)[kChunk * N / 8 / kThreads], float inv, __half *tile,
                                         __half *gtile) {
  constexpr int L = N / 8;
  const int l = threadIdx.x % L;
#pragma unroll
  for (int i = 0; i < kChunk * L / kThreads; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_bf16(w[j]);
      u[j] = pack(f.x * inv, f.y * inv);
    }
    const uint32_t at = swz(threadIdx.x / L + i * (kThreads / L), l, 2 * N);
    const uint4 v = make_uint4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(tile) + at) = v;
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(gtile) + at) = v;
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

template <int N>
__global__ void __launch_bounds__(kThreads) prep_kernel(Shape s, Args a, Tiles o, int two_planes, int vec) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem<N> &sm = *reinterpret_cast<Smem<N> *>(raw);
  const int64_t slot = blockIdx.x;
  const int grp = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t seq, b, e;
  if (!chunk_of_slot(s, a.cu, slot, seq, b, e)) return;
  const int n = int(e - b);
  const int64_t tile = (slot * s.G + grp) * kChunk * N;
  uint4 rk[kChunk * N / 8 / kThreads], rq[kChunk * N / 8 / kThreads];
  const float mk = rows_in<N>(static_cast<const __nv_bfloat16 *>(a.k) + b * s.ks + int64_t(grp) * N, s.ks, n, vec & 2, rk);
  const float mq = rows_in<N>(static_cast<const __nv_bfloat16 *>(a.q) + b * s.qs + int64_t(grp) * N, s.qs, n, vec & 1, rq);
  if (lane == 0) {
    sm.top[0][warp] = mk;
    sm.top[1][warp] = mq;
  }
  __syncthreads();
  float top[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    top[0] = fmaxf(top[0], sm.top[0][i]);
    top[1] = fmaxf(top[1], sm.top[1][i]);
  }
  // one scale for both, so that their products with one matrix can be added up
  const float ka = pow2_above(fmaxf(top[0], top[1]) * 0.0625f);
  rows_out<N>(rk, pow2_inv(ka), sm.k, o.K16 + tile);
  rows_out<N>(rq, pow2_inv(ka), sm.q, o.Q16 + tile);
  __syncthreads();
  // rows 16 warp.. of K K^T and Q K^T, columns up to the diagonal block
  float kk[8][4] = {}, qk[8][4] = {};
  const uint32_t ks = smem_at(sm.k), qs = smem_at(sm.q);
#pragma unroll
  for (int k0 = 0; k0 < N; k0 += 16) {
    uint32_t ak[4], aq[4];
    ldsm4(ak, a_addr(ks, 16 * warp, k0, 2 * N, lane));
    ldsm4(aq, a_addr(qs, 16 * warp, k0, 2 * N, lane));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= warp) {
        uint32_t bb[4];
        ldsm4(bb, b_addr(ks, 16 * j, k0, 2 * N, lane));
        mma(kk[2 * j], ak, bb[0], bb[1]);
        mma(kk[2 * j + 1], ak, bb[2], bb[3]);
        mma(qk[2 * j], aq, bb[0], bb[1]);
        mma(qk[2 * j + 1], aq, bb[2], bb[3]);
      }
  }
  const int rows[2] = {16 * warp + (lane >> 2), 16 * warp + (lane >> 2) + 8};
  for (int h0 = 0; h0 < s.hpg; h0 += 2) {
    const int nh = min(2, s.hpg - h0);
    __syncthreads();   // the products of k and q are taken, the heads before are done with L, Y and the vectors
    // running sums of g as hi + lo by a scan over 32 lanes x 2 tokens, warp w < 2 for head w
    if (warp < nh) {
      const int h = grp * s.hpg + h0 + warp;
      float v[2], vl[2];   // g log2(e), and what its rounding left over
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        // a decay to nothing stays a finite number: exp(-1e4) is zero all the same
        const float g = t < n ? fmaxf(a.g[(b + t) * s.H + h], -1e4f) : 0.f;
        v[i] = __fmul_rn(g, kLog2e);
        vl[i] = fmaf(g, kLog2eLow, fmaf(g, kLog2e, -v[i]));
        sm.beta[warp][t] = t < n ? a.beta[(b + t) * s.H + h] : 0.f;
      }
      auto add = [](float &hi, float &lo, float yh, float yl) {   // (hi, lo) += (yh, yl)
        const float sum = __fadd_rn(hi, yh), bb = __fsub_rn(sum, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, bb)), __fsub_rn(yh, bb));
        lo = __fadd_rn(__fadd_rn(lo, yl), err);
        hi = sum;
      };
      float hi = v[0], lo = vl[0];
      add(hi, lo, v[1], vl[1]);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float ph = __shfl_up_sync(~0u, hi, d), pl = __shfl_up_sync(~0u, lo, d);
        if (lane >= d) add(hi, lo, ph, pl);
      }
      sm.G[warp][2 * lane + 1] = hi;
      sm.Gl[warp][2 * lane + 1] = lo;
      float eh = __shfl_up_sync(~0u, hi, 1), el = __shfl_up_sync(~0u, lo, 1);
      if (lane == 0) eh = el = 0.f;
      add(eh, el, v[0], vl[0]);
      sm.G[warp][2 * lane] = eh;
      sm.Gl[warp][2 * lane] = el;
    }
    __syncthreads();
    for (int w = 0; w < nh; ++w) {
      const int64_t at = slot * s.H + grp * s.hpg + h0 + w;
      const float *G = sm.G[w], *Gl = sm.Gl[w];
      uint8_t *P = reinterpret_cast<uint8_t *>(o.P16 + at * kTri);
      const float Gr[2] = {G[rows[0]], G[rows[1]]}, Glr[2] = {Gl[rows[0]], Gl[rows[1]]};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j <= 2 * (warp | 1) + 1) {   // of the blocks above the diagonal, two are read
          const int c = 8 * j + 2 * (lane & 3);
          const float g0 = G[c], g1 = G[c + 1], l0 = Gl[c], l1 = Gl[c + 1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = rows[i];
            const float d0 = c <= t ? exp2f(acs_diff(Gr[i], Glr[i], g0, l0)) : 0.f;
            const float d1 = c + 1 <= t ? exp2f(acs_diff(Gr[i], Glr[i], g1, l1)) : 0.f;
            sm.L[w][c][t] = c < t ? d0 * kk[j][2 * i] * (ka * ka) : 0.f;
            sm.L[w][c + 1][t] = c + 1 < t ? d1 * kk[j][2 * i + 1] * (ka * ka) : 0.f;
            *reinterpret_cast<uint32_t *>(P + swz(t, j, 128) + 4 * (lane & 3)) =
                pack(d0 * qk[j][2 * i], d1 * qk[j][2 * i + 1]);
          }
        }
      if (tid < kChunk) {
        float *v = o.vec + at * kVec;
        v[kVecEg + tid] = exp2f(G[tid] + Gl[tid]);
        v[kVecTail + tid] = exp2f(acs_diff(G[kChunk - 1], Gl[kChunk - 1], G[tid], Gl[tid]));
        v[kVecBeta + tid] = sm.beta[w][tid];
        v[kVecG + tid] = G[tid];
        v[kVecGl + tid] = Gl[tid];
        if (tid == 0) v[kVecKa] = ka;
      }
    }
    __syncthreads();
    if ((warp >> 1) < nh) solve(sm.L[warp >> 1], sm.beta[warp >> 1], sm.Y[warp >> 1], tid & 63, 32 * (warp & 1));
    __syncthreads();
    // rows of Y to fp16, eight lanes a row
    for (int w = 0; w < nh; ++w) {
      const int64_t at = slot * s.H + grp * s.hpg + h0 + w;
      uint8_t *Y = reinterpret_cast<uint8_t *>(o.Y16 + at * 2 * kTri);
#pragma unroll 2
      for (int r = tid / 8; r < kChunk; r += kThreads / 8) {
        const int l = tid % 8;
        // columns from 32 have no rows above 32
        const bool on = l < 4 || r >= 32;
        const float4 u0 = on ? *reinterpret_cast<const float4 *>(&sm.Y[w][r][8 * l]) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 u1 = on ? *reinterpret_cast<const float4 *>(&sm.Y[w][r][8 * l + 4]) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        const float sc = pow2_above(m), inv = pow2_inv(sc);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[2];
          split<2>(v[2 * i] * inv, v[2 * i + 1] * inv, p);
          hi[i] = p[0];
          lo[i] = p[1];
        }
        *reinterpret_cast<uint4 *>(Y + swz(r, l, 128)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (two_planes)
          *reinterpret_cast<uint4 *>(Y + 2 * kTri + swz(r, l, 128)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (l == 0) o.vec[at * kVec + kVecTau + r] = sc;
      }
    }
  }
}

template <int N>
cudaError_t launch(const Shape &s, const Args &a, const Tiles &t, bool two_planes, int vec, cudaStream_t st) {
  const int smem = int(sizeof(Smem<N>));
  cudaError_t e = cudaFuncSetAttribute(prep_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prep_kernel<N><<<dim3(unsigned(s.slots), unsigned(s.G)), kThreads, smem, st>>>(s, a, t, two_planes, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep(const Shape &s, const Args &a, const Tiles &t, bool two_planes, cudaStream_t st) {
  if (s.slots == 0 || s.total == 0) return cudaSuccess;
  const int vec = ((reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && s.qs % 8 == 0 ? 1 : 0) |
                  ((reinterpret_cast<uintptr_t>(a.k) & 15) == 0 && s.ks % 8 == 0 ? 2 : 0);
  return s.N == 64 ? launch<64>(s, a, t, two_planes, vec, st) : launch<128>(s, a, t, two_planes, vec, st);
}

}  // namespace delta
}  // namespace ssd
