// ssd_qk.cu -- norm of queries and keys for each head, with the position
// rotation in the same pass, and its backward.
//
// Per head row x of length D (D = headdim), r = 1 / sqrt(m + eps) with m the
// mean (rms) or the sum (l2) of the squares, h = r x, y = w o h, and the first
// R elements of y turned in pairs by the angle of the token's position:
//     z_a = y_a cos - y_b sin,   z_b = y_a sin + y_b cos,
// (a, b) = (i, i + R/2), or (2i, 2i + 1) when interleaved.  Backward: dy is
// dz turned by the opposite angle, dw = sum over rows of dy o h, and
//     dx = r (u - h (u . h) / c),  u = w o dy,  c = D (rms) or 1 (l2).
//
// Bandwidth-bound: every row is read once and written once.  A thread holds
// the two ends of its pairs, so the rotation needs no exchange between
// threads; only the sum of squares (and u . h) is shared, by shuffles inside
// the lanes of one row.  Three forms of the same kernel:
//   - wide: pairs in runs of 8 consecutive elements (16-byte loads for bf16),
//     D / 16 lanes a row; D 32, 64, 128 or 256, R a multiple of 16, rows on
//     16-byte boundaries;
//   - pairs: runs of 2, half a warp or a warp a row; D even, R a multiple of 4,
//     rows on boundaries of two elements;
//   - narrow: one pair at a time, a warp a row; any D up to 512.
// A CTA takes a tile of consecutive tokens and a range of the heads of q or of
// k, so that a token's cos and sin are read once for all of them; the heads
// are cut into as many ranges as it takes to fill the GPU when tokens are few.
// Loads of kHeads heads are in flight at once in each of 3 (backward: 2) CTAs
// an SM.
//
// Bounded by bandwidth: 32768 tokens of 48 heads of 128 in bf16, forward 143 us
// (83% of the measured copy rate), backward with weights 227 (78%).  Pairs in
// place of narrow, 9345 tokens of 16 heads of 158: 36 and 56 us, 80 and 115.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mamba2_ssd.h"
#include "ssd_common.cuh"

namespace {

using ssd::ld;

constexpr int kThreads = 256;
constexpr int kHeads = 2;       // heads of a token that one group of lanes takes together
constexpr int kParts = 304;     // at most so many CTAs (and partial sums) of the weight gradients of q, and of k
constexpr int kFill = 608;      // CTAs that fill the GPU (four on each of 152 SMs)

struct Side {                   // q or k
  const void *x, *dz;
  void *out;                    // z (forward) or dx (backward)
  const float *w;
  float *part;                  // (kParts, D) partial weight gradients, or null
  int64_t stride;               // elements between tokens of x
  int heads;
};
struct Params {
  Side side[2];
  const float *cos, *sin;       // (positions, R / 2)
  const int32_t *pos;           // (tokens)
  int64_t tokens, npos;
  int D, R, interleaved, rms;
  float eps;
  int ranges0;                  // ranges that the heads of side 0 are cut into (gridDim.y counts both sides')
};

// A run of V elements as loaded, opened to fp32 when it is worked on.
template <int V, class T>
struct Run {
  uint32_t w[V == 1 ? 1 : V * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T *p, bool on) {
    if constexpr (V == 1) {
      w[0] = on ? __float_as_uint(ld(p)) : 0u;
    } else if constexpr (V == 2 && sizeof(T) == 2) {
      w[0] = on ? *reinterpret_cast<const uint32_t *>(p) : 0u;
    } else if constexpr (V == 2) {
      const uint2 u = on ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
      w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < int(V * sizeof(T) / 16); ++i) {
        const uint4 u = on ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void open(float (&o)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (V == 1 || sizeof(T) == 4) o[i] = __uint_as_float(w[i]);
      else o[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};
template <int V, class T>
__device__ __forceinline__ void store_run(T *p, const float (&v)[V]) {
  if constexpr (V == 1) {
    ssd::st(p, v[0]);
  } else if constexpr (V == 2 && sizeof(T) == 2) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Where unit u of a row lies: runs of V elements at `a` and `b`, turned
// against each other (rot: element i of the run at a with element i of the
// run at b), turned inside each run (interleaved), or left alone.
// na, nb: whether the runs are inside the row.
struct Place {
  int a, b, angle;
  bool rot, na, nb;
};
template <int V>
__device__ __forceinline__ Place place(const Params &q, int u) {
  Place p;
  const int R = q.R;
  if (q.interleaved || u * 2 * V >= R) {   // two neighbouring runs
    p.a = 2 * V * u;
    p.b = p.a + V;
    p.rot = u * 2 * V < R;
    p.angle = V * u;
  } else {                                 // the same run of each half
    p.a = V * u;
    p.b = p.a + R / 2;
    p.rot = true;
    p.angle = p.a;
  }
  p.na = p.a < q.D;
  p.nb = p.b < q.D;
  return p;
}

// Turns the runs (xa, xb) by the angles (c, s), sign +1 or -1.
template <int V>
__device__ __forceinline__ void turn(bool inter, float (&xa)[V], float (&xb)[V], const float (&c)[V], const float (&s)[V],
                                     float sign) {
  if (V > 1 && inter) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {   // angles 0..V/2-1 in run a, V/2..V-1 in run b
      const float a0 = xa[2 * i], a1 = xa[2 * i + 1], b0 = xb[2 * i], b1 = xb[2 * i + 1];
      const float sa = sign * s[i], sb = sign * s[V / 2 + i];
      xa[2 * i] = a0 * c[i] - a1 * sa;
      xa[2 * i + 1] = a0 * sa + a1 * c[i];
      xb[2 * i] = b0 * c[V / 2 + i] - b1 * sb;
      xb[2 * i + 1] = b0 * sb + b1 * c[V / 2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = xa[i], b = xb[i], sn = sign * s[i];
      xa[i] = a * c[i] - b * sn;
      xb[i] = a * sn + b * c[i];
    }
  }
}

// L lanes a row, each with PT units of two runs of V elements.
template <class T, int V, int L, int PT, bool kBwd, bool kHasW>
__global__ void __launch_bounds__(kThreads, V == 1 ? 1 : (kBwd ? 2 : 3)) qk_kernel(Params q) {
  constexpr int kGroups = kThreads / L;        // tokens of a CTA at a time
  constexpr int HB = V == 1 ? 1 : kHeads;
  const int which = int(blockIdx.y) >= q.ranges0;
  const Side sd = q.side[which];
  const int range = which ? blockIdx.y - q.ranges0 : blockIdx.y, ranges = which ? gridDim.y - q.ranges0 : q.ranges0;
  const int block = blockIdx.x * ranges + range;   // of this side
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  const int sets = (sd.heads + HB - 1) / HB;
  const int set0 = int(int64_t(sets) * range / ranges), set1 = int(int64_t(sets) * (range + 1) / ranges);
  const float over = q.rms ? 1.f / float(q.D) : 1.f;
  const T *x = static_cast<const T *>(sd.x);
  const T *dz = static_cast<const T *>(sd.dz);
  T *out = static_cast<T *>(sd.out);
  const bool inter = q.interleaved != 0;

  float wa[PT][V], wb[PT][V], ga[PT][V], gb[PT][V];
  if (kHasW) {
#pragma unroll
    for (int u = 0; u < PT; ++u) {
      const Place p = place<V>(q, lane + u * L);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        wa[u][i] = p.na ? sd.w[p.a + i] : 0.f;
        wb[u][i] = p.nb ? sd.w[p.b + i] : 0.f;
        ga[u][i] = gb[u][i] = 0.f;
      }
    }
  }
  // every lane of a warp takes part in the shuffles, so the loops are uniform over the CTA
  for (int64_t t0 = int64_t(blockIdx.x) * kGroups; t0 < q.tokens; t0 += int64_t(gridDim.x) * kGroups) {
    const bool live = t0 + grp < q.tokens;
    const int64_t tok = live ? t0 + grp : 0;
    float c[PT][V], s[PT][V];
    bool bad = false;
    if (q.R > 0) {
      const int64_t at = live ? q.pos[tok] : 0;
      bad = at < 0 || at >= q.npos;   // no such angle: the rows of this token come out as NaN
#pragma unroll
      for (int u = 0; u < PT; ++u) {
        const Place p = place<V>(q, lane + u * L);
        const bool on = p.rot && !bad;
        Run<V, float> rc, rs;
        rc.load(q.cos + at * (q.R / 2) + p.angle, on);
        rs.load(q.sin + at * (q.R / 2) + p.angle, on);
        rc.open(c[u]);
        rs.open(s[u]);
      }
    }
#pragma unroll 1
    for (int h0 = set0 * HB; h0 < set1 * HB; h0 += HB) {
      Run<V, T> xa[HB][PT], xb[HB][PT], da[kBwd ? HB : 1][PT], db[kBwd ? HB : 1][PT];
#pragma unroll
      for (int h = 0; h < HB; ++h)
#pragma unroll
        for (int u = 0; u < PT; ++u) {
          const Place p = place<V>(q, lane + u * L);
          const bool on = live && h0 + h < sd.heads;
          const T *row = x + tok * sd.stride + int64_t(h0 + h) * q.D;
          xa[h][u].load(row + p.a, on && p.na);
          xb[h][u].load(row + p.b, on && p.nb);
          if (kBwd) {
            const T *drow = dz + (tok * sd.heads + h0 + h) * q.D;
            da[h][u].load(drow + p.a, on && p.na);
            db[h][u].load(drow + p.b, on && p.nb);
          }
        }
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        float va[PT][V], vb[PT][V], ss = 0.f;
#pragma unroll
        for (int u = 0; u < PT; ++u) {
          xa[h][u].open(va[u]);
          xb[h][u].open(vb[u]);
#pragma unroll
          for (int i = 0; i < V; ++i) ss = fmaf(va[u][i], va[u][i], fmaf(vb[u][i], vb[u][i], ss));
        }
        ss = lanes_sum<L>(ss);
        // rows outside the problem stay zero even where eps is
        float r = live && h0 + h < sd.heads ? rsqrtf(fmaf(ss, over, q.eps)) : 0.f;
        if (bad) r = __int_as_float(0x7fc00000);
        if (!kBwd) {
#pragma unroll
          for (int u = 0; u < PT; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              va[u][i] *= kHasW ? r * wa[u][i] : r;
              vb[u][i] *= kHasW ? r * wb[u][i] : r;
            }
            if (place<V>(q, lane + u * L).rot) turn<V>(inter, va[u], vb[u], c[u], s[u], 1.f);
          }
        } else {
          float ua[PT][V], ub[PT][V], dot = 0.f;
#pragma unroll
          for (int u = 0; u < PT; ++u) {
            da[h][u].open(ua[u]);
            db[h][u].open(ub[u]);
            if (place<V>(q, lane + u * L).rot) turn<V>(inter, ua[u], ub[u], c[u], s[u], -1.f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              va[u][i] *= r;   // the normed row
              vb[u][i] *= r;
              if (kHasW) {
                ga[u][i] = fmaf(ua[u][i], va[u][i], ga[u][i]);
                gb[u][i] = fmaf(ub[u][i], vb[u][i], gb[u][i]);
                ua[u][i] *= wa[u][i];
                ub[u][i] *= wb[u][i];
              }
              dot = fmaf(ua[u][i], va[u][i], fmaf(ub[u][i], vb[u][i], dot));
            }
          }
          dot = lanes_sum<L>(dot) * over;
#pragma unroll
          for (int u = 0; u < PT; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              va[u][i] = r * fmaf(-va[u][i], dot, ua[u][i]);
              vb[u][i] = r * fmaf(-vb[u][i], dot, ub[u][i]);
            }
        }
        if (live && h0 + h < sd.heads) {
          T *row = out + (tok * sd.heads + h0 + h) * q.D;
#pragma unroll
          for (int u = 0; u < PT; ++u) {
            const Place p = place<V>(q, lane + u * L);
            if (p.na) store_run<V>(row + p.a, va[u]);
            if (p.nb) store_run<V>(row + p.b, vb[u]);
          }
        }
      }
    }
  }
  if constexpr (kBwd && kHasW) {
    // the CTA's groups added in ascending order, then one partial row a CTA
    __shared__ float red[kGroups][2 * V * L * PT];
#pragma unroll
    for (int u = 0; u < PT; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        red[grp][((u * L) + lane) * 2 * V + i] = ga[u][i];
        red[grp][((u * L) + lane) * 2 * V + V + i] = gb[u][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * V * L * PT; c += kThreads) {
      float acc = 0.f;
      for (int g = 0; g < kGroups; ++g) acc += red[g][c];
      const Place p = place<V>(q, c / (2 * V));
      const int i = c % (2 * V);
      const int col = i < V ? p.a + i : p.b + i - V;
      if (col < q.D) sd.part[int64_t(block) * q.D + col] = acc;
    }
  }
}

// dw[c] = sum of the CTA partials in ascending order, one warp a column: lane
// l adds partials l, l + 32, ..., the lanes are added by a fixed tree.
__global__ void weight_fold_kernel(const float *__restrict__ part0, const float *__restrict__ part1, int parts0,
                                   int parts1, int D, float *__restrict__ dw0, float *__restrict__ dw1) {
  const int c = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  const float *part = blockIdx.y ? part1 : part0;
  const int n = blockIdx.y ? parts1 : parts0;
  float *dw = blockIdx.y ? dw1 : dw0;
  if (c >= D || dw == nullptr) return;
  float acc = 0.f;
  for (int i = lane; i < n; i += 32) acc += part[int64_t(i) * D + c];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(~0u, acc, d);
  if (lane == 0) dw[c] = acc;
}

template <class T, int V, int L, int PT, bool kBwd>
void launch(const Params &q, dim3 blocks, bool has_w, cudaStream_t st) {
  if (has_w) qk_kernel<T, V, L, PT, kBwd, true><<<blocks, kThreads, 0, st>>>(q);
  else qk_kernel<T, V, L, PT, kBwd, false><<<blocks, kThreads, 0, st>>>(q);
}

// Elements of a run, and lanes of a row.
enum Form { kNarrow = 1, kPairs = 2, kWide = 8 };
int lanes_of(Form form, int D) { return form == kWide ? D / 16 : form == kPairs && D <= 64 ? 16 : 32; }

template <class T, bool kBwd>
void launch_form(const Params &q, Form form, dim3 blocks, bool has_w, cudaStream_t st) {
  if (form == kPairs) {
    if (q.D <= 64) return launch<T, 2, 16, 1, kBwd>(q, blocks, has_w, st);
    if (q.D <= 128) return launch<T, 2, 32, 1, kBwd>(q, blocks, has_w, st);
    if (q.D <= 256) return launch<T, 2, 32, 2, kBwd>(q, blocks, has_w, st);
    return launch<T, 2, 32, 4, kBwd>(q, blocks, has_w, st);
  }
  if (form == kWide) {
    switch (q.D) {
      case 32: return launch<T, 8, 2, 1, kBwd>(q, blocks, has_w, st);
      case 64: return launch<T, 8, 4, 1, kBwd>(q, blocks, has_w, st);
      case 128: return launch<T, 8, 8, 1, kBwd>(q, blocks, has_w, st);
      default: return launch<T, 8, 16, 1, kBwd>(q, blocks, has_w, st);
    }
  }
  if (q.D <= 64) return launch<T, 1, 32, 1, kBwd>(q, blocks, has_w, st);
  if (q.D <= 128) return launch<T, 1, 32, 2, kBwd>(q, blocks, has_w, st);
  if (q.D <= 256) return launch<T, 1, 32, 4, kBwd>(q, blocks, has_w, st);
  return launch<T, 1, 32, 8, kBwd>(q, blocks, has_w, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool dims_ok(const ssd_qk_dims *d) {
  if (d == nullptr || d->tokens < 0 || d->qheads < 1 || d->kheads < 1 || d->headdim < 1 || d->headdim > 512)
    return false;
  if (d->tokens > (int64_t(1) << 40) || d->qheads > 32768 || d->kheads > 32768) return false;
  if (d->rotary < 0 || d->rotary > d->headdim || d->rotary % 2 != 0) return false;
  if (d->rotary > 0 && (d->positions < 1 || d->positions > (int64_t(1) << 31))) return false;
  if (d->dtype != SSD_F32 && d->dtype != SSD_BF16) return false;
  if (d->norm != SSD_NORM_RMS && d->norm != SSD_NORM_L2) return false;
  if ((d->interleaved & ~1) != 0) return false;
  if (!(d->eps >= 0.f) || isinf(d->eps)) return false;
  if (d->q_stride != 0 && d->q_stride < int64_t(d->qheads) * d->headdim) return false;
  if (d->k_stride != 0 && d->k_stride < int64_t(d->kheads) * d->headdim) return false;
  return d->q_stride < (int64_t(1) << 40) && d->k_stride < (int64_t(1) << 40);
}

int64_t stride_of(int64_t given, int64_t heads, int64_t D) { return given != 0 ? given : heads * D; }

ssd_status run(const ssd_qk_dims *d, bool bwd, const void *q, const void *k, const void *dq_in, const void *dk_in,
               const float *wq, const float *wk, const float *cos, const float *sin, const int32_t *pos, void *oq,
               void *ok, float *dwq, float *dwk, void *ws, size_t ws_bytes, void *stream) {
  if (!dims_ok(d)) return SSD_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return SSD_ERR_INVALID_ARG;
  const bool has_w = wq != nullptr;
  if (bwd && has_w != (dwq != nullptr && dwk != nullptr)) return SSD_ERR_INVALID_ARG;
  if (bwd && !has_w && (dwq != nullptr || dwk != nullptr)) return SSD_ERR_INVALID_ARG;
  const size_t el = d->dtype == SSD_BF16 ? 2 : 4;
  const void *maybe[] = {wq, wk, cos, sin, pos, dwq, dwk};
  for (const void *p : maybe)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return SSD_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int D = d->headdim;
  if (d->tokens == 0) {
    if (bwd && has_w && (cudaMemsetAsync(dwq, 0, size_t(D) * 4, st) != cudaSuccess ||
                         cudaMemsetAsync(dwk, 0, size_t(D) * 4, st) != cudaSuccess))
      return SSD_ERR_CUDA;
    return SSD_OK;
  }
  const void *need[] = {q, k, oq, ok};
  for (const void *p : need)
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (el - 1))) return SSD_ERR_INVALID_ARG;
  if (bwd && (dq_in == nullptr || dk_in == nullptr || (reinterpret_cast<uintptr_t>(dq_in) & (el - 1)) ||
              (reinterpret_cast<uintptr_t>(dk_in) & (el - 1))))
    return SSD_ERR_INVALID_ARG;
  if (d->rotary > 0 && (cos == nullptr || sin == nullptr || pos == nullptr)) return SSD_ERR_INVALID_ARG;
  if (bwd && has_w) {
    if (ws_bytes < mamba2_ssd_qk_bwd_workspace_size(d)) return SSD_ERR_WORKSPACE;
    if (ws == nullptr || !aligned16(ws)) return SSD_ERR_INVALID_ARG;
  }
  Params p{};
  const int64_t qs = stride_of(d->q_stride, d->qheads, D), ks = stride_of(d->k_stride, d->kheads, D);
  p.side[0] = Side{q, dq_in, oq, wq, nullptr, qs, d->qheads};
  p.side[1] = Side{k, dk_in, ok, wk, nullptr, ks, d->kheads};
  p.cos = cos;
  p.sin = sin;
  p.pos = pos;
  p.tokens = d->tokens;
  p.npos = d->positions;
  p.D = D;
  p.R = d->rotary;
  p.interleaved = d->interleaved;
  p.rms = d->norm == SSD_NORM_RMS;
  p.eps = d->eps;
  const bool wide = (D == 32 || D == 64 || D == 128 || D == 256) && d->rotary % 16 == 0 && aligned16(q) &&
                    aligned16(k) && aligned16(oq) && aligned16(ok) && aligned16(dq_in) && aligned16(dk_in) &&
                    aligned16(cos) && aligned16(sin) && size_t(qs) * el % 16 == 0 && size_t(ks) * el % 16 == 0;
  const size_t two = 2 * el;
  const bool pairs = D % 2 == 0 && d->rotary % 4 == 0 && qs % 2 == 0 && ks % 2 == 0 && aligned_to(q, two) &&
                     aligned_to(k, two) && aligned_to(oq, two) && aligned_to(ok, two) && aligned_to(dq_in, two) &&
                     aligned_to(dk_in, two) && aligned_to(cos, 8) && aligned_to(sin, 8);
  const Form form = wide ? kWide : pairs ? kPairs : kNarrow;
  const int groups = kThreads / lanes_of(form, D);
  const int64_t tiles = (d->tokens + groups - 1) / groups;
  auto ranges = [&](int heads) {   // enough that tiles * ranges fill the GPU, half for each side
    const int64_t sets = form == kNarrow ? heads : (heads + kHeads - 1) / kHeads;
    const int64_t want = (kFill / 2 + tiles - 1) / tiles;
    return int(want < sets ? want : sets);
  };
  p.ranges0 = ranges(d->qheads);
  const int ranges1 = ranges(d->kheads);
  int64_t columns = tiles < (int64_t(1) << 30) ? tiles : int64_t(1) << 30;
  if (bwd && has_w) {   // as many partial rows as there is room for, whatever the device
    const int most = p.ranges0 > ranges1 ? p.ranges0 : ranges1;
    if (columns > kParts / most) columns = kParts / most;
  }
  if (bwd && has_w) {
    p.side[0].part = static_cast<float *>(ws);
    p.side[1].part = static_cast<float *>(ws) + int64_t(kParts) * D;
  }
  const dim3 blocks(unsigned(columns), unsigned(p.ranges0 + ranges1));
  if (d->dtype == SSD_BF16) {
    if (bwd) launch_form<__nv_bfloat16, true>(p, form, blocks, has_w, st);
    else launch_form<__nv_bfloat16, false>(p, form, blocks, has_w, st);
  } else {
    if (bwd) launch_form<float, true>(p, form, blocks, has_w, st);
    else launch_form<float, false>(p, form, blocks, has_w, st);
  }
  if (bwd && has_w)
    weight_fold_kernel<<<dim3(unsigned((D + 7) / 8), 2), 256, 0, st>>>(p.side[0].part, p.side[1].part,
                                                                       int(columns) * p.ranges0, int(columns) * ranges1, D, dwq,
                                                                       dwk);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace

extern "C" {

ssd_status mamba2_ssd_qk_fwd(const ssd_qk_dims *dims, const void *q, const void *k, const float *wq, const float *wk,
                             const float *cos, const float *sin, const int32_t *positions, void *yq, void *yk,
                             void *stream) {
  return run(dims, false, q, k, nullptr, nullptr, wq, wk, cos, sin, positions, yq, yk, nullptr, nullptr, nullptr, 0,
             stream);
}

size_t mamba2_ssd_qk_bwd_workspace_size(const ssd_qk_dims *dims) {
  if (!dims_ok(dims)) return 0;
  return size_t(2) * kParts * size_t(dims->headdim) * sizeof(float);
}

ssd_status mamba2_ssd_qk_bwd(const ssd_qk_dims *dims, const void *q, const void *k, const void *dyq, const void *dyk,
                             const float *wq, const float *wk, const float *cos, const float *sin,
                             const int32_t *positions, void *dq, void *dk, float *dwq, float *dwk, void *workspace,
                             size_t workspace_bytes, void *stream) {
  return run(dims, true, q, k, dyq, dyk, wq, wk, cos, sin, positions, dq, dk, dwq, dwk, workspace, workspace_bytes,
             stream);
}

}  // extern "C"
