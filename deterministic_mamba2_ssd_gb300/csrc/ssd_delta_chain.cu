// ssd_delta_chain.cu -- the gated delta rule from chunk to chunk: the forward
// recurrence of S with the outputs, and the reverse recurrence of dS.
//
// Rows of S (one for each element of v) never mix.  A strip of 16 rows, the
// height of a warp-level product, goes through the whole sequence with four
// warps; its S stays in their registers as fp32 accumulators, dstate / 4
// columns a warp.  Every product of a chunk has the strip's rows on its left
// and tiles of the chunk (K, Q, Y, P; see ssd_delta_tiles.cuh) on its right:
//
//   forward    X = S K16^T                    (p x t)   R = V - exp(G) 2^a X
//              E = R - (beta R) Y16^T 2^tau   (p x t)   U = beta 2^a E
//              O = (exp(G) S Q16^T + U P16^T) scale 2^a
//              S = exp(G_C) S + (U exp(G_C - G)) K16
//   backward   dU = (exp(G_C - G) dS K16^T + scale 2^a dO P16) 2^a
//              F = dU - (beta 2^tau dU) Y16,            dv = beta F
//              dS = exp(G_C) dS + scale 2^a (exp(G) dO) Q16 - (exp(G) 2^a dv) K16
//
// Each warp has 16 of the chunk's tokens as columns of X, R, E, O (dU, F) and
// a quarter of dstate as columns of S, so the left operands S, R and U pass
// through shared memory (16 rows, 2 to 4 KB) with one barrier each: three
// barriers a chunk.  What bounds the kernel is the latency of that chain, not
// a rate: few heads leave few strips, and every strip is sequential.  Hence
// the smallest left operand, S in registers, and all work that the next chunk
// does not wait for (outputs, records) behind the chain's own steps.  One warp
// a strip, with everything in registers and no barrier, took 3.2 us a chunk
// (2000 instructions of one warp).
//
// Operands are fp16 with power-of-two scales: the K, Q and Y tiles carry
// theirs (exact for bf16 k and q), the strip's S, V, dO and all between share
// one running scale, moved only when the largest value leaves [2^-2, 2^6].
// One fp16 term is 11 bits (2^-12): enough for what leaves as bf16.  Where the
// fp32 state itself is asked for, S, R, U and Y are carried as two terms (22
// bits); k and q are exact either way, and the sums are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr float kLow = 0.25f, kHigh = 64.f;   // window of a strip's largest value
constexpr int kStages = 3;    // chunks of tiles in shared memory: one worked on, two on their way
constexpr int kRing = 4;      // chunks of v (dO) rows: the next chunk's largest value is looked at a chunk ahead
constexpr int kBlock = kChunk * 32;   // bytes of a strip's rows: 64 tokens x 16

template <int N, int kTerms>
struct Layout {
  static constexpr int kK = 0, kQ = kChunk * N * 2, kY = 2 * kQ, kP = kY + 8192 * kTerms, kVecAt = kP + 8192,
                       kStage = kVecAt + (kVecChain * 4 + 127) / 128 * 128;
  // a strip's own space: ring of v or dO, then the left operands
  static constexpr int kS = kRing * kBlock, kR = kS + kTerms * 32 * N, kU = kR + kTerms * 2048, kW = kU + 2048,
                       kMax = kW + kTerms * 2048, kStrip = kMax + 128;
  __host__ __device__ static constexpr int bytes(int strips) { return kStages * kStage + strips * kStrip; }
};

struct Chunk {
  int64_t slot, b;   // chunk slot, first token
  int n;             // tokens
};

// Byte offset of 16-byte half `j` of token t in a strip's 64 x 16 block.
__device__ __forceinline__ uint32_t row_at(int t, int j) { return t * 32 + ((j ^ ((t >> 2) & 1)) << 4); }
// This lane's row of a transposing load or store of 16 tokens (4 matrices) of a block: accumulator layout, tokens as columns.
__device__ __forceinline__ uint32_t block_addr(uint32_t block, int t0, int lane) {
  return block + row_at(t0 + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
}

__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void strip_sync(int strip) { asm volatile("bar.sync %0, 128;" ::"r"(strip + 1) : "memory"); }

// 16 x 16 values (two accumulator tiles) rounded, as the four matrices of a store.
template <int kTerms>
__device__ __forceinline__ void to_a(const float (&x)[4], const float (&y)[4], uint32_t (&a)[kTerms][4]) {
  uint32_t p[kTerms];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    split<kTerms>(x[2 * i], x[2 * i + 1], p);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) a[t][i] = p[t];
    split<kTerms>(y[2 * i], y[2 * i + 1], p);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) a[t][2 + i] = p[t];
  }
}

// The chunk's tiles, copied by all threads of the CTA.
template <int N, int kTerms, int kThreads>
__device__ __forceinline__ void fetch_tiles(const Shape &s, const Tiles &t, int64_t slot, int h, uint32_t stage) {
  using L = Layout<N, kTerms>;
  const int tid = threadIdx.x;
  const int64_t kt = (slot * s.G + h / s.hpg) * kChunk * N, ht = slot * s.H + h;
  const uint8_t *K = reinterpret_cast<const uint8_t *>(t.K16 + kt) + 16 * tid;
  const uint8_t *Q = reinterpret_cast<const uint8_t *>(t.Q16 + kt) + 16 * tid;
  const uint8_t *Y = reinterpret_cast<const uint8_t *>(t.Y16 + ht * 2 * kTri) + 16 * tid;
  const uint8_t *P = reinterpret_cast<const uint8_t *>(t.P16 + ht * kTri) + 16 * tid;
  stage += 16 * tid;
#pragma unroll
  for (int i = 0; i < kChunk * N / 8; i += kThreads) {
    cp16(stage + L::kK + 16 * i, K + 16 * i);
    cp16(stage + L::kQ + 16 * i, Q + 16 * i);
  }
#pragma unroll
  for (int i = 0; i < 512 * kTerms; i += kThreads) cp16(stage + L::kY + 16 * i, Y + 16 * i);
#pragma unroll
  for (int i = 0; i < 512; i += kThreads) cp16(stage + L::kP + 16 * i, P + 16 * i);
  if (tid < kVecChain / 4) cp16(stage + L::kVecAt, reinterpret_cast<const uint8_t *>(t.vec + ht * kVec) + 16 * tid);
}

// The strip's 16 columns of the chunk's v or dO, one 16-byte piece a thread; tokens past the end are zero.
__device__ __forceinline__ void fetch_rows(const Chunk &c, const __nv_bfloat16 *x, int64_t stride, int col, bool vec,
                                           uint32_t block, uint8_t *gblock) {
  const int i = threadIdx.x & 127, r = i >> 1, j = i & 1;
  const uint32_t at = row_at(r, j);
  const __nv_bfloat16 *src = x + (c.b + r) * stride + col + 8 * j;
  if (vec) {
    const int n = r < c.n ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(block + at), "l"(n ? src : x), "r"(n) : "memory");
  } else {
    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(gblock + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) dst[e] = r < c.n ? src[e] : __float2bfloat16_rn(0.f);
  }
}

__device__ __forceinline__ void put_out(__nv_bfloat16 *p, bool vec, uint4 v) {
  if (vec) {
    *reinterpret_cast<uint4 *>(p) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[2 * i] = __ushort_as_bfloat16(static_cast<unsigned short>(w[i] & 0xffffu));
      p[2 * i + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(w[i] >> 16));
    }
  }
}

// This warp's 16 tokens x 16 rows through its part of `block` to [token][row]: the lane's token and half, and their 8 values.
__device__ __forceinline__ uint4 turned(uint8_t *gblock, uint32_t block, const uint32_t (&w)[4], int t0, int lane) {
  __syncwarp();
  stsm4t(block_addr(block, t0, lane), w);
  __syncwarp();
  return *reinterpret_cast<const uint4 *>(gblock + row_at(t0 + (lane >> 1), lane & 1));
}

// Largest magnitude of a warp's bf16 pairs, as the bits of a float.
__device__ __forceinline__ uint32_t top_of(const uint32_t (&w)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fff0000u, (w[i] << 16) & 0x7fff0000u));
  return __reduce_max_sync(~0u, m);
}
template <int kTiles>
__device__ __forceinline__ uint32_t top_of(const float (&S)[kTiles][4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) m = fmaxf(m, fmaxf(fmaxf(fabsf(S[i][0]), fabsf(S[i][1])), fmaxf(fabsf(S[i][2]), fabsf(S[i][3]))));
  return __reduce_max_sync(~0u, __float_as_uint(m));
}

// Factor that brings a strip's largest value `need` back into the window (1 while it is inside, zero or not finite).
// A power of 2^8, so that strips of like size share one scale and the gradient kernel has nothing to adjust.
__device__ __forceinline__ float rescale(float need, float dn) {
  if (!(need > kHigh || (need < kLow && need > 0.f)) || isinf(need)) return 1.f;
  const int e = int(__float_as_uint(need) >> 23) - 127 + 2;   // need = 2^-2 2^e (1 to 2)
  const int k = e >= 0 ? e / 8 : (e - 7) / 8;
  const float f = __uint_as_float(uint32_t(127 - 8 * max(-12, min(12, k))) << 23);
  const float lim = 1.0e33f;   // keeps both scales finite
  return dn * f > lim || dn * f < 1.f / lim ? 1.f : f;
}
__device__ __forceinline__ float strip_top(const float *mx) {
  const float4 v = *reinterpret_cast<const float4 *>(mx);
  return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
}

template <int kTiles>
__device__ __forceinline__ void load_state(float (&S)[kTiles][4], const float *p, bool on, int N, int lane) {
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 v = on ? *reinterpret_cast<const float2 *>(p + int64_t((lane >> 2) + 8 * r) * N + 8 * i + 2 * (lane & 3))
                          : make_float2(0.f, 0.f);
      S[i][2 * r] = v.x;
      S[i][2 * r + 1] = v.y;
    }
}
template <int kTiles>
__device__ __forceinline__ void store_state(const float (&S)[kTiles][4], float *p, float up, int N, int lane) {
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float2 *>(p + int64_t((lane >> 2) + 8 * r) * N + 8 * i + 2 * (lane & 3)) =
          make_float2(S[i][2 * r] * up, S[i][2 * r + 1] * up);
}

__device__ __forceinline__ float2 vec2(const float *v, int i, int lane) {
  return *reinterpret_cast<const float2 *>(v + 8 * i + 2 * (lane & 3));
}

// d (two token tiles) += left operand (16 x 16 at column k0 of `a`, rows of `ab` bytes) times 16 rows [n][k] of `tile`.
template <int kTerms>
__device__ __forceinline__ void mul_n(float (&d)[2][4], const uint32_t (&a)[kTerms][4], uint32_t tile, int n0, int k0,
                                      int bytes, int lane) {
  uint32_t b[4];
  ldsm4(b, b_addr(tile, n0, k0, bytes, lane));
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    mma(d[0], a[t], b[0], b[1]);
    mma(d[1], a[t], b[2], b[3]);
  }
}
// The same, kTiles column tiles from n0, with `tile` as rows [k][n].
template <int kTerms, int kTiles>
__device__ __forceinline__ void mul_t(float (&d)[kTiles][4], const uint32_t (&a)[kTerms][4], uint32_t tile, int n0, int k0,
                                      int bytes, int lane) {
#pragma unroll
  for (int i = 0; i < kTiles / 2; ++i) {
    uint32_t b[4];
    ldsm4t(b, bt_addr(tile, n0 + 16 * i, k0, bytes, lane));
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      mma(d[2 * i], a[t], b[0], b[1]);
      mma(d[2 * i + 1], a[t], b[2], b[3]);
    }
  }
}

// The state's fp16 terms to the strip's space; called by each warp for its columns.
template <int kTerms, int kTiles>
__device__ __forceinline__ void put_state(const float (&S)[kTiles][4], uint32_t at, int plane, int n0, int bytes, int lane) {
#pragma unroll
  for (int i = 0; i < kTiles / 2; ++i) {
    uint32_t a[kTerms][4];
    to_a<kTerms>(S[2 * i], S[2 * i + 1], a);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) stsm4(a_addr(at + t * plane, 0, n0 + 16 * i, bytes, lane), a[t]);
  }
}

// CTA (kStrips strips of 16 rows, head, sequence), four warps a strip.
template <int N, int kTerms, int kStrips, bool kSave>
__global__ void __launch_bounds__(128 * kStrips) chain_fwd_kernel(Shape s, Args a, Tiles t, int vvec, int ovec) {
  using L = Layout<N, kTerms>;
  constexpr int kTiles = N / 32, NB = 2 * N, kPlane = 32 * N;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 7, w = (threadIdx.x >> 5) & 3;
  const int h = blockIdx.y, p0 = (blockIdx.x * kStrips + strip) * 16, n0 = w * (N / 4), t0w = 16 * w;
  const bool live = p0 < s.P;
  const int64_t seq = blockIdx.z;
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0), nc = (te - t0 + kChunk - 1) / kChunk;
  const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v);
  __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o);
  const uint32_t base = smem_at(smem), own = base + kStages * L::kStage + strip * L::kStrip;
  uint8_t *gown = smem + kStages * L::kStage + strip * L::kStrip;
  float *mx = reinterpret_cast<float *>(gown + L::kMax);
  auto chunk = [&](int64_t c) {
    return Chunk{min(slot0 + c, s.slots - 1), t0 + c * kChunk, int(min(int64_t(kChunk), te - t0 - c * kChunk))};
  };
  auto fetch_v = [&](int64_t c) {
    if (c < nc && live) {
      const int at = int(c % kRing) * kBlock;
      fetch_rows(chunk(c), v, s.vs, h * s.P + p0, vvec, own + at, gown + at);
    }
  };
  auto fetch = [&](int64_t c) {   // the tiles of chunk c and the rows of the one after
    if (c < nc) fetch_tiles<N, kTerms, 128 * kStrips>(s, t, chunk(c).slot, h, base + int(c % kStages) * L::kStage);
    fetch_v(c + 1);
    cp_commit();
  };
  float S[kTiles][4], up = 1.f, dn = 1.f;
  const int64_t row = ((seq * s.H + h) * s.P + p0) * N + n0;
  load_state<kTiles>(S, a.init + row, live && a.init != nullptr, N, lane);
  fetch_v(0);
  cp_commit();
  fetch(0);
  fetch(1);
  // v of chunk c, this warp's tokens, as packed pairs
  auto load_v = [&](uint32_t (&x)[4], int64_t c) { ldsm4t(x, block_addr(own + int(c % kRing) * kBlock, t0w, lane)); };
  auto move = [&](float f) {
    if (f != 1.f) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][r] *= f;
      dn *= f;
      up *= pow2_inv(f);
    }
  };
  if (nc > 0) {
    cp_wait<2>();
    __syncthreads();
    if (live) {
      uint32_t x[4];
      load_v(x, 0);
      const float m = fmaxf(__uint_as_float(top_of(x)), __uint_as_float(top_of<kTiles>(S)));
      if (lane == 0) mx[4 + w] = m;
      strip_sync(strip);
      move(rescale(strip_top(mx + 4), 1.f));
    }
  }
  for (int64_t c = 0; c < nc; ++c) {
    if (live) put_state<kTerms, kTiles>(S, own + L::kS, kPlane, n0, NB, lane);
    cp_wait<1>();
    __syncthreads();   // tiles of c, rows of c + 1, S of every warp; everyone is done with chunk c - 1
    fetch(c + 2);
    if (!live) continue;
    const Chunk ck = chunk(c);
    const int64_t ht = ck.slot * s.H + h;
    const int stage = int(c % kStages) * L::kStage, ring = int(c % kRing) * kBlock;
    const uint32_t ks = base + stage + L::kK, qs = base + stage + L::kQ, ys = base + stage + L::kY, ps = base + stage + L::kP;
    const float *vec = reinterpret_cast<const float *>(smem + stage + L::kVecAt);
    const float ka = vec[kVecKa], last = vec[kVecEg + kChunk - 1];
    const float2 eg[2] = {vec2(vec + kVecEg + t0w, 0, lane), vec2(vec + kVecEg + t0w, 1, lane)};
    uint32_t vw[4];
    load_v(vw, c);
    float R[2][4] = {}, O[2][4] = {};
#pragma unroll
    for (int j = 0; j < N / 16; ++j) {
      uint32_t sa[kTerms][4], one[1][4];
#pragma unroll
      for (int i = 0; i < kTerms; ++i) ldsm4(sa[i], a_addr(own + L::kS + i * kPlane, 0, 16 * j, NB, lane));
#pragma unroll
      for (int i = 0; i < 4; ++i) one[0][i] = sa[0][i];
      mul_n<kTerms>(R, sa, ks, t0w, 16 * j, NB, lane);
      mul_n<1>(O, one, qs, t0w, 16 * j, NB, lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v0 = unpack_bf16(vw[2 * i]), v1 = unpack_bf16(vw[2 * i + 1]);
      const float c0 = eg[i].x * ka, c1 = eg[i].y * ka;
      R[i][0] = fmaf(-c0, R[i][0], v0.x * dn);
      R[i][1] = fmaf(-c1, R[i][1], v0.y * dn);
      R[i][2] = fmaf(-c0, R[i][2], v1.x * dn);
      R[i][3] = fmaf(-c1, R[i][3], v1.y * dn);
    }
    float2 be[2];
    {
      float B[2][4];
      uint32_t ra[kTerms][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        be[i] = vec2(vec + kVecBeta + t0w, i, lane);
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          B[i][r] = R[i][r] * be[i].x;
          B[i][r + 1] = R[i][r + 1] * be[i].y;
        }
      }
      to_a<kTerms>(B[0], B[1], ra);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) stsm4(a_addr(own + L::kR + 2048 * i, 0, t0w, 128, lane), ra[i]);
    }
    strip_sync(strip);
    float E[2][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        uint32_t ra[kTerms][4];
#pragma unroll
        for (int i = 0; i < kTerms; ++i) ldsm4(ra[i], a_addr(own + L::kR + 2048 * i, 0, 16 * j, 128, lane));
        mul_n<kTerms>(E, ra, ys, t0w, 16 * j, 128, lane);
        if constexpr (kTerms == 2) {
          uint32_t one[1][4] = {{ra[0][0], ra[0][1], ra[0][2], ra[0][3]}};
          mul_n<1>(E, one, ys + 8192, t0w, 16 * j, 128, lane);
        }
      }
    float W[2][4];
    uint32_t ew[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 tau = vec2(vec + kVecTau + t0w, i, lane), tl = vec2(vec + kVecTail + t0w, i, lane);
      const float c0 = be[i].x * ka, c1 = be[i].y * ka;
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const float e0 = fmaf(-tau.x, E[i][r], R[i][r]), e1 = fmaf(-tau.y, E[i][r + 1], R[i][r + 1]);
        if (kSave) ew[2 * i + r / 2] = pack(e0, e1);
        E[i][r] = e0 * c0;
        E[i][r + 1] = e1 * c1;
        W[i][r] = E[i][r] * tl.x;
        W[i][r + 1] = E[i][r + 1] * tl.y;
      }
    }
    {
      uint32_t ua[1][4], wa[kTerms][4];
      to_a<kTerms>(W[0], W[1], wa);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) stsm4(a_addr(own + L::kW + 2048 * i, 0, t0w, 128, lane), wa[i]);
      to_a<1>(E[0], E[1], ua);
      stsm4(a_addr(own + L::kU, 0, t0w, 128, lane), ua[0]);
    }
    {
      // the next chunk's scale: its rows, and this chunk's state (which one chunk cannot carry out of fp16's range)
      uint32_t x[4] = {0, 0, 0, 0};
      if (c + 1 < nc) load_v(x, c + 1);
      const float m = fmaxf(__uint_as_float(top_of(x)) * dn, __uint_as_float(top_of<kTiles>(S)));
      if (lane == 0) mx[4 * (c & 1) + w] = m;
    }
    if (kSave) {
      // the state entering the chunk as it stands in shared memory: 16 rows, contiguous in the record
      uint8_t *to = reinterpret_cast<uint8_t *>(t.S16 + (ht * s.P + p0) * N);
#pragma unroll
      for (int i = 0; i < 2 * N; i += 128) {
        const int at = 16 * (i + (threadIdx.x & 127));
        *reinterpret_cast<uint4 *>(to + at) = *reinterpret_cast<const uint4 *>(gown + L::kS + at);
      }
      if ((threadIdx.x & 127) == 0) t.up[(ht * s.P + p0) >> 4] = up;
    }
    strip_sync(strip);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] *= last;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t wa[kTerms][4];
#pragma unroll
      for (int i = 0; i < kTerms; ++i) ldsm4(wa[i], a_addr(own + L::kW + 2048 * i, 0, 16 * j, 128, lane));
      mul_t<kTerms, kTiles>(S, wa, ks, n0, 16 * j, NB, lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        O[i][r] *= eg[i].x;
        O[i][r + 1] *= eg[i].y;
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        uint32_t ua[1][4];
        ldsm4(ua[0], a_addr(own + L::kU, 0, 16 * j, 128, lane));
        mul_n<1>(O, ua, ps, t0w, 16 * j, 128, lane);
      }
    // outputs and record through this warp's tokens of the v block, which it alone has read
    const int tok = t0w + (lane >> 1);
    const float co = a.scale * ka * up;
    uint32_t ow[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ow[2 * i] = pack_bf16(O[i][0] * co, O[i][1] * co);
      ow[2 * i + 1] = pack_bf16(O[i][2] * co, O[i][3] * co);
    }
    const uint4 ov = turned(gown + ring, own + ring, ow, t0w, lane);
    if (tok < ck.n) put_out(o + ((ck.b + tok) * s.H + h) * s.P + p0 + 8 * (lane & 1), ovec, ov);
    if (kSave)
      *reinterpret_cast<uint4 *>(t.E16 + (ht * kChunk + tok) * s.P + p0 + 8 * (lane & 1)) =
          turned(gown + ring, own + ring, ew, t0w, lane);
    move(rescale(strip_top(mx + 4 * (c & 1)), dn));
  }
  cp_wait<0>();
  if (live && a.fin != nullptr) store_state<kTiles>(S, a.fin + row, up, N, lane);
}

// The reverse recurrence; writes dv, dinit, and for the gradient kernel dS leaving each chunk (D16), F (F16) and dO (X16).
template <int N, int kStrips>
__global__ void __launch_bounds__(128 * kStrips) chain_bwd_kernel(Shape s, Args a, Tiles t, BwdTiles o, int gvec, int ovec) {
  using L = Layout<N, 1>;
  constexpr int kTiles = N / 32, NB = 2 * N;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, strip = threadIdx.x >> 7, w = (threadIdx.x >> 5) & 3;
  const int h = blockIdx.y, p0 = (blockIdx.x * kStrips + strip) * 16, n0 = w * (N / 4), t0w = 16 * w;
  const bool live = p0 < s.P;
  const int64_t seq = blockIdx.z, tok_stride = int64_t(s.H) * s.P;
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0), nc = (te - t0 + kChunk - 1) / kChunk;
  const __nv_bfloat16 *go = static_cast<const __nv_bfloat16 *>(a.dout);
  __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv);
  const uint32_t base = smem_at(smem), own = base + kStages * L::kStage + strip * L::kStrip;
  uint8_t *gown = smem + kStages * L::kStage + strip * L::kStrip;
  float *mx = reinterpret_cast<float *>(gown + L::kMax);
  // step i of the sweep takes chunk nc - 1 - i of the sequence
  auto chunk = [&](int64_t i) {
    const int64_t c = nc - 1 - i;
    return Chunk{min(slot0 + c, s.slots - 1), t0 + c * kChunk, int(min(int64_t(kChunk), te - t0 - c * kChunk))};
  };
  auto fetch_x = [&](int64_t c) {
    if (c < nc && live) {
      const int at = int(c % kRing) * kBlock;
      fetch_rows(chunk(c), go, tok_stride, h * s.P + p0, gvec, own + at, gown + at);
    }
  };
  auto fetch = [&](int64_t c) {
    if (c < nc) fetch_tiles<N, 1, 128 * kStrips>(s, t, chunk(c).slot, h, base + int(c % kStages) * L::kStage);
    fetch_x(c + 1);
    cp_commit();
  };
  float D[kTiles][4], up = 1.f, dn = 1.f;
  const int64_t row = ((seq * s.H + h) * s.P + p0) * N + n0;
  load_state<kTiles>(D, a.dfinal + row, live && a.dfinal != nullptr, N, lane);
  fetch_x(0);
  cp_commit();
  fetch(0);
  fetch(1);
  // dO of this warp's tokens in units of the strip's scale; its fp16 takes the place of dO in the ring
  float X[2][4];
  auto take_x = [&](const uint32_t (&x)[4], int64_t c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v0 = unpack_bf16(x[2 * i]), v1 = unpack_bf16(x[2 * i + 1]);
      X[i][0] = v0.x * dn;
      X[i][1] = v0.y * dn;
      X[i][2] = v1.x * dn;
      X[i][3] = v1.y * dn;
    }
    uint32_t xa[1][4];
    to_a<1>(X[0], X[1], xa);
    stsm4t(block_addr(own + int(c % kRing) * kBlock, t0w, lane), xa[0]);
  };
  auto load_x = [&](uint32_t (&x)[4], int64_t c) { ldsm4t(x, block_addr(own + int(c % kRing) * kBlock, t0w, lane)); };
  auto move = [&](float f) {
    if (f != 1.f) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) D[i][r] *= f;
      dn *= f;
      up *= pow2_inv(f);
    }
  };
  if (nc > 0) {
    cp_wait<2>();
    __syncthreads();
    if (live) {
      uint32_t x[4];
      load_x(x, 0);
      const float m = fmaxf(__uint_as_float(top_of(x)), __uint_as_float(top_of<kTiles>(D)));
      if (lane == 0) mx[4 + w] = m;
      strip_sync(strip);
      move(rescale(strip_top(mx + 4), 1.f));
      take_x(x, 0);
    }
  }
  for (int64_t c = 0; c < nc; ++c) {
    if (live) put_state<1, kTiles>(D, own + L::kS, 0, n0, NB, lane);
    cp_wait<1>();
    __syncthreads();   // tiles of c, rows of c + 1, dS and dO of every warp; everyone is done with chunk c - 1
    fetch(c + 2);
    if (!live) continue;
    const Chunk ck = chunk(c);
    const int64_t ht = ck.slot * s.H + h;
    const int stage = int(c % kStages) * L::kStage, ring = int(c % kRing) * kBlock;
    const uint32_t ks = base + stage + L::kK, qs = base + stage + L::kQ, ys = base + stage + L::kY, ps = base + stage + L::kP;
    const float *vec = reinterpret_cast<const float *>(smem + stage + L::kVecAt);
    const float ka = vec[kVecKa], last = vec[kVecEg + kChunk - 1], co = a.scale * ka;
    float F[2][4] = {}, A[2][4] = {};
#pragma unroll
    for (int j = 0; j < N / 16; ++j) {
      uint32_t da[1][4];
      ldsm4(da[0], a_addr(own + L::kS, 0, 16 * j, NB, lane));
      mul_n<1>(F, da, ks, t0w, 16 * j, NB, lane);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j >= w) {
        uint32_t xa[1][4];
        ldsm4t(xa[0], block_addr(own + ring, 16 * j, lane));
        mul_t<1, 2>(A, xa, ps, t0w, 16 * j, 128, lane);
      }
    const float2 eg[2] = {vec2(vec + kVecEg + t0w, 0, lane), vec2(vec + kVecEg + t0w, 1, lane)};
    float2 be[2];
    {
      float B[2][4];
      uint32_t fa[1][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 tl = vec2(vec + kVecTail + t0w, i, lane), tau = vec2(vec + kVecTau + t0w, i, lane);
        be[i] = vec2(vec + kVecBeta + t0w, i, lane);
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          F[i][r] = ka * fmaf(tl.x, F[i][r], co * A[i][r]);
          F[i][r + 1] = ka * fmaf(tl.y, F[i][r + 1], co * A[i][r + 1]);
          B[i][r] = F[i][r] * (be[i].x * tau.x);
          B[i][r + 1] = F[i][r + 1] * (be[i].y * tau.y);
        }
      }
      to_a<1>(B[0], B[1], fa);
      stsm4(a_addr(own + L::kR, 0, t0w, 128, lane), fa[0]);
    }
    strip_sync(strip);
    {
      float C[2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= w) {
          uint32_t fa[1][4];
          ldsm4(fa[0], a_addr(own + L::kR, 0, 16 * j, 128, lane));
          mul_t<1, 2>(C, fa, ys, t0w, 16 * j, 128, lane);
        }
      float W[2][4], Z[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float c0 = -eg[i].x * ka, c1 = -eg[i].y * ka;
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          F[i][r] -= C[i][r];
          F[i][r + 1] -= C[i][r + 1];
          W[i][r] = F[i][r] * (be[i].x * c0);
          W[i][r + 1] = F[i][r + 1] * (be[i].y * c1);
          Z[i][r] = X[i][r] * eg[i].x;
          Z[i][r + 1] = X[i][r + 1] * eg[i].y;
        }
      }
      uint32_t wa[1][4];
      to_a<1>(W[0], W[1], wa);
      stsm4(a_addr(own + L::kW, 0, t0w, 128, lane), wa[0]);
      to_a<1>(Z[0], Z[1], wa);
      stsm4(a_addr(own + L::kU, 0, t0w, 128, lane), wa[0]);
    }
    uint32_t x[4] = {0, 0, 0, 0};
    {
      if (c + 1 < nc) load_x(x, c + 1);
      const float m = fmaxf(__uint_as_float(top_of(x)) * dn, __uint_as_float(top_of<kTiles>(D)));
      if (lane == 0) mx[4 * (c & 1) + w] = m;
    }
    {
      uint8_t *to = reinterpret_cast<uint8_t *>(o.D16 + (ht * s.P + p0) * N);
#pragma unroll
      for (int i = 0; i < 2 * N; i += 128) {
        const int at = 16 * (i + (threadIdx.x & 127));
        *reinterpret_cast<uint4 *>(to + at) = *reinterpret_cast<const uint4 *>(gown + L::kS + at);
      }
      if ((threadIdx.x & 127) == 0) o.ub[(ht * s.P + p0) >> 4] = up;
    }
    strip_sync(strip);
    {
      float Z[kTiles][4] = {};
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) D[i][r] *= last;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t wa[1][4], ya[1][4];
        ldsm4(wa[0], a_addr(own + L::kW, 0, 16 * j, 128, lane));
        ldsm4(ya[0], a_addr(own + L::kU, 0, 16 * j, 128, lane));
        mul_t<1, kTiles>(D, wa, ks, n0, 16 * j, NB, lane);
        mul_t<1, kTiles>(Z, ya, qs, n0, 16 * j, NB, lane);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) D[i][r] = fmaf(co, Z[i][r], D[i][r]);
    }
    const int tok = t0w + (lane >> 1);
    uint32_t rw[4], vw[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        rw[2 * i + r] = pack(F[i][2 * r], F[i][2 * r + 1]);
        vw[2 * i + r] = pack_bf16(F[i][2 * r] * (be[i].x * up), F[i][2 * r + 1] * (be[i].y * up));
      }
    const int64_t at = (ht * kChunk + tok) * s.P + p0 + 8 * (lane & 1);
    *reinterpret_cast<uint4 *>(o.X16 + at) = *reinterpret_cast<const uint4 *>(gown + ring + row_at(tok, lane & 1));
    *reinterpret_cast<uint4 *>(o.F16 + at) = turned(gown + ring, own + ring, rw, t0w, lane);
    const uint4 vv = turned(gown + ring, own + ring, vw, t0w, lane);
    if (tok < ck.n) put_out(dv + (ck.b + tok) * tok_stride + h * s.P + p0 + 8 * (lane & 1), ovec, vv);
    move(rescale(strip_top(mx + 4 * (c & 1)), dn));
    if (c + 1 < nc) take_x(x, c + 1);
  }
  cp_wait<0>();
  if (live && a.dinit != nullptr) store_state<kTiles>(D, a.dinit + row, up, N, lane);
}

bool vec16(const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

// Strips of a CTA: several share one copy of the chunk's tiles, fewer spread over more SMs.  At most `most`, and
// only while that still gives 120 of the 152 SMs a CTA.
int strips_of(const Shape &s, int most) {
  const int strips = (s.P + 15) / 16;
  int n = most;
  while (n > 1 && (n >= 2 * strips || s.nseq * s.H * ((strips + n - 1) / n) < 120)) n /= 2;
  return n;
}
dim3 chain_grid(const Shape &s, int n) {
  return dim3(unsigned(((s.P + 15) / 16 + n - 1) / n), unsigned(s.H), unsigned(s.nseq));
}

template <int N, int kTerms, int kStrips, bool kSave>
cudaError_t go_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  auto kernel = chain_fwd_kernel<N, kTerms, kStrips, kSave>;
  constexpr int smem = Layout<N, kTerms>::bytes(kStrips);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<chain_grid(s, kStrips), 128 * kStrips, smem, st>>>(s, a, t, vec16(a.v, s.vs), vec16(a.o, 8));
  return cudaGetLastError();
}

template <int N, int kTerms, bool kSave>
cudaError_t pick_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  // four strips with two terms would need more shared memory than an SM has
  const int n = strips_of(s, kTerms == 2 && N == 128 ? 2 : 4);
  if constexpr (kTerms == 1 || N == 64)
    if (n == 4) return go_fwd<N, kTerms, 4, kSave>(s, a, t, st);
  return n >= 2 ? go_fwd<N, kTerms, 2, kSave>(s, a, t, st) : go_fwd<N, kTerms, 1, kSave>(s, a, t, st);
}

template <int N>
cudaError_t fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  const bool save = t.S16 != nullptr;
  if (a.fin != nullptr) return save ? pick_fwd<N, 2, true>(s, a, t, st) : pick_fwd<N, 2, false>(s, a, t, st);
  return save ? pick_fwd<N, 1, true>(s, a, t, st) : pick_fwd<N, 1, false>(s, a, t, st);
}

template <int N, int kStrips>
cudaError_t go_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  auto kernel = chain_bwd_kernel<N, kStrips>;
  constexpr int smem = Layout<N, 1>::bytes(kStrips);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<chain_grid(s, kStrips), 128 * kStrips, smem, st>>>(s, a, t, b, vec16(a.dout, 8), vec16(a.dv, 8));
  return cudaGetLastError();
}

template <int N>
cudaError_t bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  const int n = strips_of(s, 4);
  return n == 4 ? go_bwd<N, 4>(s, a, t, b, st) : n == 2 ? go_bwd<N, 2>(s, a, t, b, st) : go_bwd<N, 1>(s, a, t, b, st);
}

}  // namespace

cudaError_t launch_chain_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  return s.N == 64 ? fwd<64>(s, a, t, st) : fwd<128>(s, a, t, st);
}

cudaError_t launch_chain_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  return s.N == 64 ? bwd<64>(s, a, t, b, st) : bwd<128>(s, a, t, b, st);
}

}  // namespace delta
}  // namespace ssd
