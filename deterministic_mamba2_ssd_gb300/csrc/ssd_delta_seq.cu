// ssd_delta_seq.cu -- gated delta rule on CUDA cores, whole sequences with few
// rows of state: the recurrent forward, and the recurrent backward of the
// state.  fp32 arithmetic throughout, any headdim, dstate up to 256.
//
// Rows of the state never mix: row p of S sees only v[p].  So a row is the unit
// of work: a warp keeps it in registers over the whole sequence.  Tokens go by
// four.  With S before the four, E_ts the decay from after s to after t and
// u = beta e,
//     e_t = v_t - E_t S k_t - sum_{s<t} E_ts (k_s . k_t) u_s,
// so the four sums over the lanes are one another's neighbours in the pipeline,
// not one after the other; the products k_s . k_t are the same for all rows.
// Backward, with F = dS k and w = beta F, likewise from the last of the four:
//     F_t = E_t dS k_t + sum_{r>=t} E_rt (scale do_r) (q_r . k_t) - sum_{r>t} E_rt w_r (k_r . k_t).
//
// What bounds a sequence is the latency of that chain, not a rate; all else is
// kept off it.  Four warps have a row each, four bring the next eight tokens
// into shared memory and multiply their keys, four write what the last eight
// gave.
// 517 tokens of 12 heads of 40 x 72 in fp32: 75 us forward, 2200 cycles for
// eight tokens, of which the chain itself is 1800 (its sums over the lanes 900);
// token by token on eight lanes a row it is 148.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta.h"

namespace ssd {
namespace delta {
namespace {

constexpr int kBlock = 8;       // tokens in shared memory at a time
constexpr int kWork = 128;      // threads with rows
constexpr int kIn = 128;        // threads that bring tokens
constexpr int kOut = 128;       // threads that write results
constexpr int kThreads = kWork + kIn + kOut;
constexpr int kLanes = 32;      // of a row
constexpr int kRows = kWork / kLanes;

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}
__device__ __forceinline__ void in_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kIn) : "memory"); }

// The state row of this lane: columns (kLanes j + lane) * 4 + i, zero past N.
template <int NJ>
__device__ __forceinline__ void load_row(float (&s)[4 * NJ], const float *row, int N, int lane) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int c = (kLanes * j + lane) * 4;
    if ((N & 3) == 0) {
      const float4 v = row != nullptr && c < N ? *reinterpret_cast<const float4 *>(row + c) : make_float4(0, 0, 0, 0);
      s[4 * j] = v.x;
      s[4 * j + 1] = v.y;
      s[4 * j + 2] = v.z;
      s[4 * j + 3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[4 * j + i] = row != nullptr && c + i < N ? row[c + i] : 0.f;
    }
  }
}
template <int NJ>
__device__ __forceinline__ void store_row(const float (&s)[4 * NJ], float *row, int N, int lane) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int c = (kLanes * j + lane) * 4;
    if ((N & 3) == 0) {
      if (c < N) *reinterpret_cast<float4 *>(row + c) = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < N) row[c + i] = s[4 * j + i];
    }
  }
}

// Eight tokens in shared memory, and what they give.
template <int NJ>
struct Tile {
  static constexpr int kWide = 4 * kLanes * NJ;
  float q[kBlock][kWide], k[kBlock][kWide];
  float x[kBlock][kRows];           // v (forward) or scale dout (backward)
  float g[kBlock], b[kBlock];       // exp(g), beta
  // of each run of four tokens: E_t, E_ts k_s.k_t (forward s < t; backward s > t), E_rt q_r.k_t (backward, r >= t)
  float run[kBlock], kk[kBlock][4], qk[kBlock][4];
  float y[kBlock][kRows][kLanes];   // each lane's part of o (forward)
  float z[kBlock][kRows], w[kBlock][kRows];   // e (forward); F and beta F (backward)
};

// What a thread has on its way to shared memory.
template <class T, int NJ, bool kBwd>
struct Stage {
  using Tl = Tile<NJ>;
  static constexpr int kHalf = kIn / 2, kVec = kBlock * Tl::kWide / kHalf;   // elements of q (first half of the threads) or k
  float v[kVec], x, g, b;

  __device__ __forceinline__ void load(const Shape &s, const Args &a, int64_t t0, int n, int h, int p0) {
    const int ht = threadIdx.x - kWork, u = ht % kHalf, at = ht - (kIn - kBlock);
    const bool is_k = ht >= kHalf;
    const int64_t stride = is_k ? s.ks : s.qs;
    const T *src = static_cast<const T *>(is_k ? a.k : a.q) + t0 * stride + int64_t(h / s.hpg) * s.N;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int e = u + i * kHalf, t = e / Tl::kWide, c = e % Tl::kWide;
      v[i] = t < n && c < s.N ? ld(src + t * stride + c) : 0.f;
    }
    x = 0.f;
    if (ht < kBlock * kRows) {   // (at most 128)
      const int t = ht / kRows, p = p0 + ht % kRows;
      if (t < n && p < s.P)
        x = kBwd ? a.scale * ld(static_cast<const T *>(a.dout) + ((t0 + t) * s.H + h) * s.P + p)
                 : ld(static_cast<const T *>(a.v) + (t0 + t) * s.vs + int64_t(h) * s.P + p);
    }
    if (at >= 0) {   // a token past the end leaves the state as it is
      g = at < n ? expf(a.g[(t0 + at) * s.H + h]) : 1.f;
      b = at < n ? a.beta[(t0 + at) * s.H + h] : 0.f;
    }
  }
  __device__ __forceinline__ void put(Tl &sm) const {
    const int ht = threadIdx.x - kWork, u = ht % kHalf, at = ht - (kIn - kBlock);
    float *to = ht >= kHalf ? &sm.k[0][0] : &sm.q[0][0];
#pragma unroll
    for (int i = 0; i < kVec; ++i) to[u + i * kHalf] = v[i];
    if (ht < kBlock * kRows) (&sm.x[0][0])[ht] = x;
    if (at >= 0) {
      sm.g[at] = g;
      sm.b[at] = b;
    }
  }
};

// Products of keys (and queries) of each run of four, eight lanes a product.
template <int NJ, bool kBwd>
__device__ __forceinline__ void runs(Tile<NJ> &sm) {
  using Tl = Tile<NJ>;
  const int ht = threadIdx.x - kWork, lane8 = ht & 7, group = ht >> 3;
  constexpr int kPairs = kBwd ? 16 : 6, kDots = kBlock / 4 * kPairs;   // of a run: 6 k.k, and 10 q.k
#pragma unroll
  for (int i = group; i < kDots; i += kIn / 8) {
    const int o = i / kPairs * 4, at = i % kPairs;
    // the pair (lo <= hi) of place `at`: k.k (0,1) (0,2) (0,3) (1,2) (1,3) (2,3), then q.k the same and the four (t, t)
    const int w = at < 6 ? at : at < 12 ? at - 6 : 0;
    const int lo = at < 12 ? (0x211000 >> (4 * w)) & 3 : at - 12, hi = at < 12 ? (0x332321 >> (4 * w)) & 3 : at - 12;
    const float *x = at < 6 ? sm.k[o + hi] : sm.q[o + hi], *y = sm.k[o + lo];
    const float g1 = lo < 1 && hi >= 1 ? sm.g[o + 1] : 1.f, g2 = lo < 2 && hi >= 2 ? sm.g[o + 2] : 1.f,
                g3 = lo < 3 && hi >= 3 ? sm.g[o + 3] : 1.f;
    float part[4] = {};
#pragma unroll
    for (int c = 0; c < Tl::kWide; c += 32) {
      const float4 f = *reinterpret_cast<const float4 *>(&x[c + 4 * lane8]), d = *reinterpret_cast<const float4 *>(&y[c + 4 * lane8]);
      part[0] = fmaf(f.x, d.x, part[0]);
      part[1] = fmaf(f.y, d.y, part[1]);
      part[2] = fmaf(f.z, d.z, part[2]);
      part[3] = fmaf(f.w, d.w, part[3]);
    }
    float sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffu << (threadIdx.x & 24), sum, d);
    sum *= g1 * g2 * g3;
    if (lane8 == 0) {
      if (!kBwd) sm.kk[o + hi][lo] = sum;
      else if (at < 6) sm.kk[o + lo][hi] = sum;
      else sm.qk[o + lo][hi] = sum;
    }
  }
  if (ht >= kIn - kBlock) {
    const int t = ht - (kIn - kBlock), o = t & ~3, i = t & 3;
    const float4 g = *reinterpret_cast<const float4 *>(&sm.g[o]);
    if (kBwd) sm.run[t] = (i < 1 ? g.y : 1.f) * (i < 2 ? g.z : 1.f) * (i < 3 ? g.w : 1.f);
    else sm.run[t] = g.x * (i >= 1 ? g.y : 1.f) * (i >= 2 ? g.z : 1.f) * (i >= 3 ? g.w : 1.f);
  }
}

// CTA (kRows rows of the state, head, sequence).
template <class T, int NJ>
__global__ void __launch_bounds__(kThreads, NJ == 1 ? 2 : 1) seq_fwd_kernel(Shape s, Args a, float *__restrict__ states, float *__restrict__ es) {
  using Tl = Tile<NJ>;
  __shared__ Tl tile[2];
  const int p0 = blockIdx.x * kRows, h = blockIdx.y;
  const int lane = threadIdx.x % kLanes, r = threadIdx.x / kLanes, p = p0 + r;
  const bool live = p < s.P;
  T *o = static_cast<T *>(a.o);
  for (int64_t seq = blockIdx.z; seq < s.nseq; seq += gridDim.z) {
    int64_t t0, te;
    seq_range(s, a.cu, seq, t0, te);
    const int64_t nb = (te - t0 + kBlock - 1) / kBlock;
    auto tokens = [&](int64_t blk) { return int(min(int64_t(kBlock), te - t0 - blk * kBlock)); };
    if (threadIdx.x >= kWork + kIn) {
      auto leave = [&](int64_t blk) {   // o and e of a block
        constexpr int kShare = kOut / (kBlock * kRows), kParts = kLanes / kShare;   // threads of an element
        const Tl &sm = tile[blk & 1];
        const int ot = threadIdx.x - kWork - kIn, x = ot / kShare, part = ot % kShare, t = x / kRows, rr = x % kRows;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; i += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(&sm.y[t][rr][kParts * part + i]);
          sum += (u.x + u.y) + (u.z + u.w);
        }
        sum = row_sum<kShare>(sum);
        if (part == 0 && t < tokens(blk) && p0 + rr < s.P) {
          const int64_t y = ((t0 + blk * kBlock + t) * s.H + h) * s.P + p0 + rr;
          o[y] = from_f32<T>(a.scale * sum);
          if (es != nullptr) es[y] = sm.z[t][rr];
        }
      };
      __syncthreads();
      for (int64_t blk = 0; blk < nb; ++blk) {
        if (blk > 0) leave(blk - 1);
        __syncthreads();
      }
      if (nb > 0) leave(nb - 1);
    } else if (threadIdx.x >= kWork) {
      Stage<T, NJ, false> st;
      auto load = [&](int64_t blk) {
        if (blk < nb) st.load(s, a, t0 + blk * kBlock, tokens(blk), h, p0);
      };
      auto put = [&](int64_t blk) {
        if (blk < nb) {
          st.put(tile[blk & 1]);
          in_sync();
          load(blk + 1);
          runs<NJ, false>(tile[blk & 1]);
        }
      };
      load(0);
      put(0);
      __syncthreads();
      for (int64_t blk = 0; blk < nb; ++blk) {
        put(blk + 1);
        __syncthreads();
      }
    } else {
      const int64_t row = ((seq * s.H + h) * s.P + p) * s.N, slot0 = first_slot(s, a.cu, seq, t0);
      float S[4 * NJ];
      load_row<NJ>(S, live && a.init != nullptr ? a.init + row : nullptr, s.N, lane);
      __syncthreads();
      for (int64_t blk = 0; blk < nb; ++blk) {
        Tl &sm = tile[blk & 1];
        if (states != nullptr && blk % (kChunk / kBlock) == 0) {
          const int64_t slot = slot0 + blk / (kChunk / kBlock);
          if (live && slot < s.slots) store_row<NJ>(S, states + ((slot * s.H + h) * s.P + p) * s.N, s.N, lane);
        }
#pragma unroll 1
        for (int c = 0; c < kBlock; c += 4) {   // tokens past the end change nothing
          float dot[4] = {}, u[4], x[4], run[4], b[4], dec[4];
          float4 kk[4];
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[c + t][(kLanes * j + lane) * 4]);
              dot[t] = fmaf(S[4 * j], kv.x, fmaf(S[4 * j + 1], kv.y, fmaf(S[4 * j + 2], kv.z, fmaf(S[4 * j + 3], kv.w, dot[t]))));
            }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            x[t] = sm.x[c + t][r];
            run[t] = sm.run[c + t];
            b[t] = sm.b[c + t];
            dec[t] = sm.g[c + t];
            kk[t] = *reinterpret_cast<const float4 *>(sm.kk[c + t]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) dot[t] = row_sum<kLanes>(dot[t]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float cc[4] = {kk[t].x, kk[t].y, kk[t].z, kk[t].w};
            float e = fmaf(-run[t], dot[t], x[t]);
#pragma unroll
            for (int z = 0; z < t; ++z) e = fmaf(-cc[z], u[z], e);
            u[t] = b[t] * e;
            x[t] = e;
          }
          float out[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float part[4] = {};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[c + t][(kLanes * j + lane) * 4]);
              const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[c + t][(kLanes * j + lane) * 4]);
              const float kx[4] = {kv.x, kv.y, kv.z, kv.w}, qx[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                S[4 * j + z] = fmaf(u[t], kx[z], dec[t] * S[4 * j + z]);
                part[z] = fmaf(S[4 * j + z], qx[z], part[z]);
              }
            }
            out[t] = (part[0] + part[1]) + (part[2] + part[3]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {   // the lanes' parts are added up by others
            sm.y[c + t][r][lane] = out[t];
            if (lane == 0) sm.z[c + t][r] = x[t];
          }
        }
        __syncthreads();
      }
      if (live && a.fin != nullptr) store_row<NJ>(S, a.fin + row, s.N, lane);
    }
    __syncthreads();   // before the next sequence's first block
  }
}

// The reverse recurrence of dS, tokens from the last to the first: writes the
// gradient of the state leaving each chunk, F, dv and the gradient of the
// initial state.
template <class T, int NJ>
__global__ void __launch_bounds__(kThreads, NJ == 1 ? 2 : 1) seq_bwd_kernel(Shape s, Args a, float *__restrict__ dstates, float *__restrict__ F) {
  using Tl = Tile<NJ>;
  __shared__ Tl tile[2];
  const int p0 = blockIdx.x * kRows, h = blockIdx.y;
  const int lane = threadIdx.x % kLanes, r = threadIdx.x / kLanes, p = p0 + r;
  const bool live = p < s.P;
  T *dv = static_cast<T *>(a.dv);
  for (int64_t seq = blockIdx.z; seq < s.nseq; seq += gridDim.z) {
    int64_t t0, te;
    seq_range(s, a.cu, seq, t0, te);
    const int64_t nb = (te - t0 + kBlock - 1) / kBlock;
    auto tokens = [&](int64_t blk) { return int(min(int64_t(kBlock), te - t0 - blk * kBlock)); };
    // step i of the sweep takes block nb - 1 - i
    if (threadIdx.x >= kWork + kIn) {
      auto leave = [&](int64_t i) {
        const Tl &sm = tile[i & 1];
        const int ot = threadIdx.x - kWork - kIn, t = ot / kRows, rr = ot % kRows;
        const int64_t blk = nb - 1 - i;
        if (t < tokens(blk) && p0 + rr < s.P) {
          const int64_t y = ((t0 + blk * kBlock + t) * s.H + h) * s.P + p0 + rr;
          F[y] = sm.z[t][rr];
          dv[y] = from_f32<T>(sm.w[t][rr]);
        }
      };
      __syncthreads();
      for (int64_t i = 0; i < nb; ++i) {
        if (i > 0) leave(i - 1);
        __syncthreads();
      }
      if (nb > 0) leave(nb - 1);
    } else if (threadIdx.x >= kWork) {
      Stage<T, NJ, true> st;
      auto load = [&](int64_t i) {
        if (i < nb) st.load(s, a, t0 + (nb - 1 - i) * kBlock, tokens(nb - 1 - i), h, p0);
      };
      auto put = [&](int64_t i) {
        if (i < nb) {
          st.put(tile[i & 1]);
          in_sync();
          load(i + 1);
          runs<NJ, true>(tile[i & 1]);
        }
      };
      load(0);
      put(0);
      __syncthreads();
      for (int64_t i = 0; i < nb; ++i) {
        put(i + 1);
        __syncthreads();
      }
    } else {
      const int64_t row = ((seq * s.H + h) * s.P + p) * s.N, slot0 = first_slot(s, a.cu, seq, t0);
      float S[4 * NJ];
      load_row<NJ>(S, live && a.dfinal != nullptr ? a.dfinal + row : nullptr, s.N, lane);
      __syncthreads();
      for (int64_t i = 0; i < nb; ++i) {
        Tl &sm = tile[i & 1];
        const int64_t blk = nb - 1 - i;
        if (live && (i == 0 || (blk + 1) % (kChunk / kBlock) == 0)) {
          const int64_t slot = slot0 + blk / (kChunk / kBlock);
          if (slot < s.slots) store_row<NJ>(S, dstates + ((slot * s.H + h) * s.P + p) * s.N, s.N, lane);
        }
#pragma unroll 1
        for (int c = kBlock - 4; c >= 0; c -= 4) {
          float dot[4] = {}, d[4], w[4], run[4], b[4], dec[4];
          float4 kk[4], qk[4];
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[c + t][(kLanes * j + lane) * 4]);
              dot[t] = fmaf(S[4 * j], kv.x, fmaf(S[4 * j + 1], kv.y, fmaf(S[4 * j + 2], kv.z, fmaf(S[4 * j + 3], kv.w, dot[t]))));
            }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            d[t] = sm.x[c + t][r];
            run[t] = sm.run[c + t];
            b[t] = sm.b[c + t];
            dec[t] = sm.g[c + t];
            kk[t] = *reinterpret_cast<const float4 *>(sm.kk[c + t]);
            qk[t] = *reinterpret_cast<const float4 *>(sm.qk[c + t]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) dot[t] = row_sum<kLanes>(dot[t]);
          float f[4];
#pragma unroll
          for (int t = 3; t >= 0; --t) {
            const float cc[4] = {kk[t].x, kk[t].y, kk[t].z, kk[t].w}, ee[4] = {qk[t].x, qk[t].y, qk[t].z, qk[t].w};
            f[t] = run[t] * dot[t];
#pragma unroll
            for (int z = 3; z >= t; --z) f[t] = fmaf(d[z], ee[z], f[t]);
#pragma unroll
            for (int z = 3; z > t; --z) f[t] = fmaf(-w[z], cc[z], f[t]);
            w[t] = b[t] * f[t];
          }
#pragma unroll
          for (int t = 3; t >= 0; --t)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[c + t][(kLanes * j + lane) * 4]);
              const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[c + t][(kLanes * j + lane) * 4]);
              const float kx[4] = {kv.x, kv.y, kv.z, kv.w}, qx[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) S[4 * j + z] = dec[t] * fmaf(-w[t], kx[z], fmaf(d[t], qx[z], S[4 * j + z]));
            }
          if (lane == 0)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              sm.z[c + t][r] = f[t];
              sm.w[c + t][r] = w[t];
            }
        }
        __syncthreads();
      }
      if (live && a.dinit != nullptr) store_row<NJ>(S, a.dinit + row, s.N, lane);
    }
    __syncthreads();
  }
}

dim3 grid_of(const Shape &s) {
  return dim3(unsigned((s.P + kRows - 1) / kRows), unsigned(s.H), unsigned(s.nseq < 65535 ? s.nseq : 65535));
}

template <class T>
cudaError_t fwd(const Shape &s, const Args &a, float *states, float *es, cudaStream_t st) {
  if (s.N <= 128) seq_fwd_kernel<T, 1><<<grid_of(s), kThreads, 0, st>>>(s, a, states, es);
  else seq_fwd_kernel<T, 2><<<grid_of(s), kThreads, 0, st>>>(s, a, states, es);
  return cudaGetLastError();
}
template <class T>
cudaError_t bwd(const Shape &s, const Args &a, float *dstates, float *F, cudaStream_t st) {
  if (s.N <= 128) seq_bwd_kernel<T, 1><<<grid_of(s), kThreads, 0, st>>>(s, a, dstates, F);
  else seq_bwd_kernel<T, 2><<<grid_of(s), kThreads, 0, st>>>(s, a, dstates, F);
  return cudaGetLastError();
}

}  // namespace

cudaError_t seq_fwd(const Shape &s, bool bf16, const Args &a, float *states, float *es, cudaStream_t st) {
  return bf16 ? fwd<__nv_bfloat16>(s, a, states, es, st) : fwd<float>(s, a, states, es, st);
}
cudaError_t seq_bwd(const Shape &s, bool bf16, const Args &a, float *dstates, float *F, cudaStream_t st) {
  return bf16 ? bwd<__nv_bfloat16>(s, a, dstates, F, st) : bwd<float>(s, a, dstates, F, st);
}

}  // namespace delta
}  // namespace ssd
