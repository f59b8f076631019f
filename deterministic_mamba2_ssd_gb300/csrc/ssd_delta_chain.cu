// ssd_delta_chain.cu -- the gated delta rule from chunk to chunk: the forward
// recurrence of S with the outputs, and the reverse recurrence of dS.
//
// Rows of S (one for each element of v) never mix, so a warp takes 16 of them
// through the whole sequence, kept as the fp32 accumulators [16 rows x
// dstate] of its own matrix products, and shares with the other warps of the
// CTA only the tiles it reads (k, q, T, P of the chunk).  Every product of a
// chunk has rows p on its left:
//
//   forward    X = S K16^T                    (p x t)   R = V - exp(G) 2^a X
//              E = R T16^T 2^tau              (p x t)   U = beta 2^a E
//              O = (exp(G) S Q16^T + U P16^T) scale 2^b
//              S = exp(G_C) S + (U exp(G_C - G)) K16
//   backward   F = (exp(G_C - G) dS K16^T + dO' P16) 2^a,   dO' = scale 2^b dO
//              dR = (beta 2^tau F) T16
//              dS = exp(G_C) dS + (exp(G) dO') Q16 - (exp(G) 2^a dR) K16
//
// so an accumulator, scaled column by column, rounded and packed, is the left
// operand of the next product, and the chain of a chunk runs from register to
// register with one CTA barrier a chunk (for the tiles, which arrive by
// asynchronous copies one or two chunks ahead).
//
// Operands are fp16 with power-of-two scales: k and q rows carry theirs (exact
// for bf16 input), rows of S, V, dO and everything between share one running
// scale a row, moved only when the row's largest value leaves [2^2, 2^12].
// One fp16 term is 11 bits (2^-12): enough for what leaves as bf16.  Where the
// fp32 state itself is asked for, S, R, U and T are carried as two terms (22
// bits); k and q are exact either way, and the sums are fp32.
//
// Why warp-level products: the chain S -> X -> R -> E -> U -> S is sequential,
// and at 16 rows a warp its tiles are small (16 x 64 x 128).  Keeping S in
// registers costs no barrier, no TMEM round trip and no copy of S through
// shared memory between the five dependent products of a chunk.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"

namespace ssd {
namespace delta {
namespace {

using namespace mma16;

constexpr float kLow = 4.f, kHigh = 4096.f, kMid = 64.f;   // window and centre of a row's running scale

__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <int N, int kTerms>
struct Layout {
  static constexpr int kK = 0, kQ = kChunk * N * 2, kT = 2 * kQ, kP = kT + 8192 * kTerms, kVecAt = kP + 8192,
                       kRows = kVecAt + (kVecChain * 4 + 127) / 128 * 128;
  static constexpr int kRowBytes = kChunk * 32;   // 64 tokens x 16 rows of one warp
  __host__ __device__ static constexpr int stage(int warps) { return kRows + warps * kRowBytes; }
};

// Byte offset of 16-byte half `j` of token t in a warp's 64 x 16 block.
__device__ __forceinline__ uint32_t row_at(int t, int j) { return t * 32 + ((j ^ ((t >> 2) & 1)) << 4); }

struct Chunk {
  int64_t slot, b;   // chunk slot, first token
  int n;             // tokens
};

// Asynchronous copies of one chunk's tiles (all threads) and of this warp's 64 x 16 block of v or dout.
template <int N, int kTerms>
__device__ __forceinline__ void load_chunk(const Shape &s, const Tiles &t, const Chunk &c, int h, const __nv_bfloat16 *x,
                                           int64_t xs, int col, bool live, bool vec, uint32_t stage, uint8_t *gstage) {
  using L = Layout<N, kTerms>;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int64_t kt = (c.slot * s.G + h / s.hpg) * kChunk * N, ht = c.slot * s.H + h;
  const uint8_t *K = reinterpret_cast<const uint8_t *>(t.K16 + kt), *Q = reinterpret_cast<const uint8_t *>(t.Q16 + kt);
  const uint8_t *T = reinterpret_cast<const uint8_t *>(t.T16 + ht * 2 * kTri);
  const uint8_t *P = reinterpret_cast<const uint8_t *>(t.P16 + ht * kTri);
  const uint8_t *V = reinterpret_cast<const uint8_t *>(t.vec + ht * kVec);
  for (int i = tid; i < kChunk * N / 8; i += nt) {
    cp16(stage + L::kK + 16 * i, K + 16 * i);
    cp16(stage + L::kQ + 16 * i, Q + 16 * i);
  }
  for (int i = tid; i < 512 * kTerms; i += nt) cp16(stage + L::kT + 16 * i, T + 16 * i);
  for (int i = tid; i < 512; i += nt) cp16(stage + L::kP + 16 * i, P + 16 * i);
  for (int i = tid; i < kVecChain / 4; i += nt) cp16(stage + L::kVecAt + 16 * i, V + 16 * i);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (lane >> 1) + 16 * i, j = lane & 1;
    const uint32_t at = L::kRows + warp * L::kRowBytes + row_at(r, j);
    const __nv_bfloat16 *src = x + (c.b + r) * xs + col + 8 * j;
    if (vec) {
      cp16_or_zero(stage + at, r < c.n ? src : x, r < c.n);
    } else {
      __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(gstage + at);
#pragma unroll
      for (int e = 0; e < 8; ++e) dst[e] = r < c.n ? src[e] : __float2bfloat16_rn(0.f);
    }
  }
}

// This warp's 64 x 16 block as packed pairs in accumulator layout: w[i][0], [1] of token tile 2 i (rows g, g + 8), w[i][2], [3] of 2 i + 1.
__device__ __forceinline__ uint32_t block_addr(uint32_t block, int i, int lane) {
  return block + row_at(16 * i + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
}
__device__ __forceinline__ void load_block(uint32_t block, uint32_t (&w)[4][4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) ldsm4t(w[i], block_addr(block, i, lane));
}

// The block back to [token][16 rows] in the warp's staging space, then 16-byte pieces to `put(token, half, value)`.
template <class Put>
__device__ __forceinline__ void store_block(uint8_t *gblock, uint32_t block, const uint32_t (&w)[4][4], int lane,
                                            Put put) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) stsm4t(block_addr(block, i, lane), w[i]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (lane >> 1) + 16 * i, j = lane & 1;
    put(r, j, *reinterpret_cast<const uint4 *>(gblock + row_at(r, j)));
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

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
  return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}

// One row's factor that brings its largest value `need` back to kMid (1 while it is inside the window, zero or not finite).
__device__ __forceinline__ float rescale(float need, float dn) {
  if (!(need > kHigh || (need < kLow && need > 0.f)) || isinf(need)) return 1.f;
  const float f = kMid * pow2_inv(pow2_above(need));
  const float lim = 1.0e33f;   // keeps 2^-r and 2^r finite; values below 1e-31 of 1 may then underflow
  return dn * f > lim ? 1.f : (dn * f < 1.f / lim ? 1.f : f);
}

// d[i] += A(a) * B over one 16-step of the contraction, for the tile pairs i2 in [lo, hi): B from rows [n][k].
template <int kPairs, int kTerms>
__device__ __forceinline__ void step_n(float (*d)[4], const uint32_t (&a)[kTerms][4], uint32_t tile, int k0, int bytes,
                                       int lane, int lo) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    if (i >= lo) {
      uint32_t b[4];
      ldsm4(b, b_addr(tile, 16 * i, k0, bytes, lane));
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        mma(d[2 * i], a[t], b[0], b[1]);
        mma(d[2 * i + 1], a[t], b[2], b[3]);
      }
    }
}
// The same with B from rows [k][n], tile pairs [0, hi].
template <int kPairs, int kTerms>
__device__ __forceinline__ void step_t(float (*d)[4], const uint32_t (&a)[kTerms][4], uint32_t tile, int k0, int bytes,
                                       int lane, int hi) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    if (i <= hi) {
      uint32_t b[4];
      ldsm4t(b, bt_addr(tile, 16 * i, k0, bytes, lane));
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        mma(d[2 * i], a[t], b[0], b[1]);
        mma(d[2 * i + 1], a[t], b[2], b[3]);
      }
    }
}

// Accumulator tiles 2 j, 2 j + 1 as the A operand of step j.
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

template <int N>
__device__ __forceinline__ void load_state(float (*S)[4], const float *p, bool on, int lane) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 v = on ? *reinterpret_cast<const float2 *>(p + int64_t((lane >> 2) + 8 * r) * N + 8 * i + 2 * (lane & 3))
                          : make_float2(0.f, 0.f);
      S[i][2 * r] = v.x;
      S[i][2 * r + 1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ void store_state(const float (*S)[4], float *p, const float (&up)[2], int lane) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float2 *>(p + int64_t((lane >> 2) + 8 * r) * N + 8 * i + 2 * (lane & 3)) =
          make_float2(S[i][2 * r] * up[r], S[i][2 * r + 1] * up[r]);
}

// Brings the rows' running scale to the chunk: the largest of |S| (already scaled) and of the incoming values `m`.
template <int N>
__device__ __forceinline__ void fit_rows(float (*S)[4], float (&up)[2], float (&dn)[2], float m0, float m1) {
  float need[2] = {m0 * dn[0], m1 * dn[1]};
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    need[0] = fmaxf(need[0], fmaxf(fabsf(S[i][0]), fabsf(S[i][1])));
    need[1] = fmaxf(need[1], fmaxf(fabsf(S[i][2]), fabsf(S[i][3])));
  }
  float f[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) f[r] = rescale(quad_max(need[r]), dn[r]);
  if (__any_sync(~0u, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      S[i][0] *= f[0];
      S[i][1] *= f[0];
      S[i][2] *= f[1];
      S[i][3] *= f[1];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      dn[r] *= f[r];
      up[r] *= pow2_inv(f[r]);
    }
  }
}

// This warp's rows of the state tile, [p][n] fp16 in the swizzled layout, and their scales.
template <int N, int kTerms>
__device__ __forceinline__ void save_state(const uint32_t (&a)[N / 16][kTerms][4], __half *tile, float *scales,
                                           const float (&up)[2], int lane) {
  uint8_t *p = reinterpret_cast<uint8_t *>(tile);
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int j = 0; j < N / 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint32_t *>(p + swz(g + 8 * (i & 1), 2 * j + (i >> 1), 2 * N) + 4 * q) = a[j][0][i];
  if (q == 0) {
    scales[g] = up[0];
    scales[g + 8] = up[1];
  }
}

__device__ __forceinline__ float2 vec2(const float *v, int i, int lane) {
  return *reinterpret_cast<const float2 *>(v + 8 * i + 2 * (lane & 3));
}

// CTA (16 * warps rows, head, sequence).
template <int N, int kTerms, int kStages, bool kSave>
__global__ void __launch_bounds__(256) chain_fwd_kernel(Shape s, Args a, Tiles t, int vvec, int ovec) {
  using L = Layout<N, kTerms>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, p0 = (blockIdx.x * warps + warp) * 16;
  const bool live = p0 < s.P;
  const int64_t seq = blockIdx.z;
  const uint32_t base = smem_at(smem);
  const int stage = L::stage(warps);
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0), nc = (te - t0 + kChunk - 1) / kChunk;
  const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v);
  __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o);
  auto chunk = [&](int64_t c) {
    return Chunk{min(slot0 + c, s.slots - 1), t0 + c * kChunk, int(min(int64_t(kChunk), te - t0 - c * kChunk))};
  };
  auto fetch = [&](int64_t c) {
    if (c < nc) {
      const int at = int(c % kStages) * stage;
      load_chunk<N, kTerms>(s, t, chunk(c), h, v, s.vs, h * s.P + p0, live, vvec, base + at, smem + at);
    }
    cp_commit();
  };
  float S[N / 8][4], up[2] = {1.f, 1.f}, dn[2] = {1.f, 1.f};
  const int64_t row = ((seq * s.H + h) * s.P + p0) * N;
  load_state<N>(S, a.init + row, live && a.init != nullptr, lane);
#pragma unroll
  for (int c = 0; c < kStages - 1; ++c) fetch(c);
  for (int64_t c = 0; c < nc; ++c) {
    cp_wait<kStages - 2>();
    __syncthreads();
    fetch(c + kStages - 1);
    if (!live) continue;
    const Chunk ck = chunk(c);
    const int at = int(c % kStages) * stage;
    const uint32_t ks = base + at + L::kK, qs = base + at + L::kQ, ts = base + at + L::kT, ps = base + at + L::kP;
    const uint32_t block = base + at + L::kRows + warp * L::kRowBytes;
    uint8_t *gblock = smem + at + L::kRows + warp * L::kRowBytes;
    const float *vec = reinterpret_cast<const float *>(smem + at + L::kVecAt);
    const float ka = vec[kVecKa], co = a.scale * vec[kVecQa];
    uint32_t vw[4][4];
    load_block(block, vw, lane);
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_bf16(vw[i][j]);
        m[j & 1] = fmaxf(m[j & 1], fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    fit_rows<N>(S, up, dn, m[0], m[1]);
    float R[8][4] = {}, O[8][4] = {};
    {
      uint32_t sa[N / 16][kTerms][4];
#pragma unroll
      for (int j = 0; j < N / 16; ++j) to_a<kTerms>(S[2 * j], S[2 * j + 1], sa[j]);
      if (kSave) {
        const int64_t ht = ck.slot * s.H + h;
        save_state<N, kTerms>(sa, t.S16 + (ht * s.P + p0) * N, t.up + ht * s.P + p0, up, lane);
      }
#pragma unroll
      for (int j = 0; j < N / 16; ++j) {
        step_n<4, kTerms>(R, sa[j], ks, 16 * j, 2 * N, lane, 0);
        uint32_t one[1][4] = {{sa[j][0][0], sa[j][0][1], sa[j][0][2], sa[j][0][3]}};
        step_n<4, 1>(O, one, qs, 16 * j, 2 * N, lane, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 eg = vec2(vec + kVecEg, i, lane);
      const float2 v0 = unpack_bf16(vw[i >> 1][2 * (i & 1)]), v1 = unpack_bf16(vw[i >> 1][2 * (i & 1) + 1]);
      const float c0 = eg.x * ka, c1 = eg.y * ka;
      R[i][0] = fmaf(-c0, R[i][0], v0.x * dn[0]);
      R[i][1] = fmaf(-c1, R[i][1], v0.y * dn[0]);
      R[i][2] = fmaf(-c0, R[i][2], v1.x * dn[1]);
      R[i][3] = fmaf(-c1, R[i][3], v1.y * dn[1]);
      O[i][0] *= eg.x;
      O[i][1] *= eg.y;
      O[i][2] *= eg.x;
      O[i][3] *= eg.y;
    }
    float E[8][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t ra[kTerms][4];
      to_a<kTerms>(R[2 * j], R[2 * j + 1], ra);
      step_n<4, kTerms>(E, ra, ts, 16 * j, 128, lane, j);
      if constexpr (kTerms == 2) {
        uint32_t one[1][4] = {{ra[0][0], ra[0][1], ra[0][2], ra[0][3]}};
        step_n<4, 1>(E, one, ts + 8192, 16 * j, 128, lane, j);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 tau = vec2(vec + kVecTau, i, lane);
      E[i][0] *= tau.x;
      E[i][1] *= tau.y;
      E[i][2] *= tau.x;
      E[i][3] *= tau.y;
    }
    if (kSave) {
      uint32_t w[4][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i >> 1][2 * (i & 1)] = pack(E[i][0], E[i][1]);
        w[i >> 1][2 * (i & 1) + 1] = pack(E[i][2], E[i][3]);
      }
      uint8_t *e16 = reinterpret_cast<uint8_t *>(t.E16 + (ck.slot * s.H + h) * kChunk * s.P);
      store_block(gblock, block, w, lane, [&](int r, int j, uint4 x) {
        *reinterpret_cast<uint4 *>(e16 + (int64_t(r) * s.P + p0 + 8 * j) * 2) = x;
      });
    }
    // U = beta 2^a E, then the outputs and the state
    const float last = vec[kVecEg + kChunk - 1];
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] *= last;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        const float2 be = vec2(vec + kVecBeta, i, lane);
        const float c0 = be.x * ka, c1 = be.y * ka;
        E[i][0] *= c0;
        E[i][1] *= c1;
        E[i][2] *= c0;
        E[i][3] *= c1;
      }
      uint32_t ua[1][4];
      to_a<1>(E[2 * j], E[2 * j + 1], ua);
      step_n<4, 1>(O, ua, ps, 16 * j, 128, lane, j);
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        const float2 tl = vec2(vec + kVecTail, i, lane);
        E[i][0] *= tl.x;
        E[i][1] *= tl.y;
        E[i][2] *= tl.x;
        E[i][3] *= tl.y;
      }
      uint32_t wa[kTerms][4];
      to_a<kTerms>(E[2 * j], E[2 * j + 1], wa);
      step_t<N / 16, kTerms>(S, wa, ks, 16 * j, 2 * N, lane, N / 16);
    }
    uint32_t w[4][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i >> 1][2 * (i & 1)] = pack_bf16(O[i][0] * co * up[0], O[i][1] * co * up[0]);
      w[i >> 1][2 * (i & 1) + 1] = pack_bf16(O[i][2] * co * up[1], O[i][3] * co * up[1]);
    }
    __nv_bfloat16 *op = o + (ck.b * s.H + h) * s.P + p0;
    store_block(gblock, block, w, lane, [&](int r, int j, uint4 x) {
      if (r < ck.n) put_out(op + int64_t(r) * s.H * s.P + 8 * j, ovec, x);
    });
  }
  cp_wait<0>();
  if (live && a.fin != nullptr) store_state<N>(S, a.fin + row, up, lane);
}

// The reverse recurrence; writes dv, the gradients of the states leaving the chunks (D16), dR (R16) and dinit.
template <int N, int kStages>
__global__ void __launch_bounds__(256) chain_bwd_kernel(Shape s, Args a, Tiles t, BwdTiles o, int gvec, int ovec) {
  using L = Layout<N, 1>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, p0 = (blockIdx.x * warps + warp) * 16;
  const bool live = p0 < s.P;
  const int64_t seq = blockIdx.z;
  const uint32_t base = smem_at(smem);
  const int stage = L::stage(warps);
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0), nc = (te - t0 + kChunk - 1) / kChunk;
  const __nv_bfloat16 *go = static_cast<const __nv_bfloat16 *>(a.dout);
  __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv);
  const int64_t tok = int64_t(s.H) * s.P;
  // chunk i of this sweep is chunk nc - 1 - i of the sequence
  auto chunk = [&](int64_t i) {
    const int64_t c = nc - 1 - i;
    return Chunk{min(slot0 + c, s.slots - 1), t0 + c * kChunk, int(min(int64_t(kChunk), te - t0 - c * kChunk))};
  };
  auto fetch = [&](int64_t i) {
    if (i < nc) {
      const int at = int(i % kStages) * stage;
      load_chunk<N, 1>(s, t, chunk(i), h, go, tok, h * s.P + p0, live, gvec, base + at, smem + at);
    }
    cp_commit();
  };
  float D[N / 8][4], up[2] = {1.f, 1.f}, dn[2] = {1.f, 1.f};
  const int64_t row = ((seq * s.H + h) * s.P + p0) * N;
  load_state<N>(D, a.dfinal + row, live && a.dfinal != nullptr, lane);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  for (int64_t c = 0; c < nc; ++c) {
    cp_wait<kStages - 2>();
    __syncthreads();
    fetch(c + kStages - 1);
    if (!live) continue;
    const Chunk ck = chunk(c);
    const int64_t ht = ck.slot * s.H + h;
    const int at = int(c % kStages) * stage;
    const uint32_t ks = base + at + L::kK, qs = base + at + L::kQ, ts = base + at + L::kT, ps = base + at + L::kP;
    const uint32_t block = base + at + L::kRows + warp * L::kRowBytes;
    uint8_t *gblock = smem + at + L::kRows + warp * L::kRowBytes;
    const float *vec = reinterpret_cast<const float *>(smem + at + L::kVecAt);
    const float ka = vec[kVecKa], co = a.scale * vec[kVecQa];
    float X[8][4];   // dO' = scale 2^b dO, then in units of the rows' scale
    {
      uint32_t w[4][4];
      load_block(block, w, lane);
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v0 = unpack_bf16(w[i >> 1][2 * (i & 1)]), v1 = unpack_bf16(w[i >> 1][2 * (i & 1) + 1]);
        X[i][0] = v0.x * co;
        X[i][1] = v0.y * co;
        X[i][2] = v1.x * co;
        X[i][3] = v1.y * co;
        m[0] = fmaxf(m[0], fmaxf(fabsf(X[i][0]), fabsf(X[i][1])));
        m[1] = fmaxf(m[1], fmaxf(fabsf(X[i][2]), fabsf(X[i][3])));
      }
      fit_rows<N>(D, up, dn, m[0], m[1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        X[i][0] *= dn[0];
        X[i][1] *= dn[0];
        X[i][2] *= dn[1];
        X[i][3] *= dn[1];
      }
    }
    float F[8][4] = {};
    {
      uint32_t da[N / 16][1][4];
#pragma unroll
      for (int j = 0; j < N / 16; ++j) to_a<1>(D[2 * j], D[2 * j + 1], da[j]);
      save_state<N, 1>(da, o.D16 + (ht * s.P + p0) * N, o.ub + ht * s.P + p0, up, lane);
#pragma unroll
      for (int j = 0; j < N / 16; ++j) step_n<4, 1>(F, da[j], ks, 16 * j, 2 * N, lane, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 tl = vec2(vec + kVecTail, i, lane);
      F[i][0] *= tl.x;
      F[i][1] *= tl.y;
      F[i][2] *= tl.x;
      F[i][3] *= tl.y;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t xa[1][4];
      to_a<1>(X[2 * j], X[2 * j + 1], xa);
      step_t<4, 1>(F, xa, ps, 16 * j, 128, lane, j);
    }
    float R[8][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        const float2 be = vec2(vec + kVecBeta, i, lane), tau = vec2(vec + kVecTau, i, lane);
        const float c0 = be.x * ka * tau.x, c1 = be.y * ka * tau.y;
        F[i][0] *= c0;
        F[i][1] *= c1;
        F[i][2] *= c0;
        F[i][3] *= c1;
      }
      uint32_t fa[1][4];
      to_a<1>(F[2 * j], F[2 * j + 1], fa);
      step_t<4, 1>(R, fa, ts, 16 * j, 128, lane, j);
    }
    {
      uint32_t w[4][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i >> 1][2 * (i & 1)] = pack(R[i][0], R[i][1]);
        w[i >> 1][2 * (i & 1) + 1] = pack(R[i][2], R[i][3]);
      }
      uint8_t *r16 = reinterpret_cast<uint8_t *>(o.R16 + ht * kChunk * s.P);
      store_block(gblock, block, w, lane, [&](int r, int j, uint4 x) {
        *reinterpret_cast<uint4 *>(r16 + (int64_t(r) * s.P + p0 + 8 * j) * 2) = x;
      });
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i >> 1][2 * (i & 1)] = pack_bf16(R[i][0] * up[0], R[i][1] * up[0]);
        w[i >> 1][2 * (i & 1) + 1] = pack_bf16(R[i][2] * up[1], R[i][3] * up[1]);
      }
      __nv_bfloat16 *vp = dv + (ck.b * s.H + h) * s.P + p0;
      store_block(gblock, block, w, lane, [&](int r, int j, uint4 x) {
        if (r < ck.n) put_out(vp + r * tok + 8 * j, ovec, x);
      });
    }
    const float last = vec[kVecEg + kChunk - 1];
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) D[i][r] *= last;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 2 * j; i < 2 * j + 2; ++i) {
        const float2 eg = vec2(vec + kVecEg, i, lane);
        const float c0 = -eg.x * ka, c1 = -eg.y * ka;
        X[i][0] *= eg.x;
        X[i][1] *= eg.y;
        X[i][2] *= eg.x;
        X[i][3] *= eg.y;
        R[i][0] *= c0;
        R[i][1] *= c1;
        R[i][2] *= c0;
        R[i][3] *= c1;
      }
      uint32_t xa[1][4], ra[1][4];
      to_a<1>(X[2 * j], X[2 * j + 1], xa);
      to_a<1>(R[2 * j], R[2 * j + 1], ra);
      step_t<N / 16, 1>(D, xa, qs, 16 * j, 2 * N, lane, N / 16);
      step_t<N / 16, 1>(D, ra, ks, 16 * j, 2 * N, lane, N / 16);
    }
  }
  cp_wait<0>();
  if (live && a.dinit != nullptr) store_state<N>(D, a.dinit + row, up, lane);
}

// Warps of a CTA: as many of a head's 16-row strips as leave every SM a CTA
// (more warps share one copy of the chunk's tiles; fewer spread over the SMs).
int chain_warps(const Shape &s) {
  const int strips = (s.P + 15) / 16;
  int w = 8;
  while (w > 2 && (w >= 2 * strips || s.nseq * s.H * ((strips + w - 1) / w) < 120)) w /= 2;
  return w;
}

template <class K>
cudaError_t launch(K kernel, int warps, int smem, const Shape &s, cudaStream_t st, dim3 &grid) {
  grid = dim3(unsigned(((s.P + 15) / 16 + warps - 1) / warps), unsigned(s.H), unsigned(s.nseq));
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

bool vec16(const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

template <int N, int kTerms, int kStages, bool kSave>
cudaError_t go_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  const int warps = chain_warps(s), smem = kStages * Layout<N, kTerms>::stage(warps);
  auto kernel = chain_fwd_kernel<N, kTerms, kStages, kSave>;
  dim3 grid;
  const cudaError_t e = launch(kernel, warps, smem, s, st, grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * warps, smem, st>>>(s, a, t, vec16(a.v, s.vs), vec16(a.o, 8));
  return cudaGetLastError();
}

template <int N>
cudaError_t pick_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  const bool save = t.S16 != nullptr, two = a.fin != nullptr;
  if (two) return save ? go_fwd<N, 2, 3, true>(s, a, t, st) : go_fwd<N, 2, 3, false>(s, a, t, st);
  return save ? go_fwd<N, 1, 3, true>(s, a, t, st) : go_fwd<N, 1, 3, false>(s, a, t, st);
}

template <int N>
cudaError_t go_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  const int warps = chain_warps(s), smem = 3 * Layout<N, 1>::stage(warps);
  auto kernel = chain_bwd_kernel<N, 3>;
  dim3 grid;
  const cudaError_t e = launch(kernel, warps, smem, s, st, grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * warps, smem, st>>>(s, a, t, b, vec16(a.dout, 8), vec16(a.dv, 8));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chain_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  return s.N == 64 ? pick_fwd<64>(s, a, t, st) : pick_fwd<128>(s, a, t, st);
}

cudaError_t launch_chain_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  return s.N == 64 ? go_bwd<64>(s, a, t, b, st) : go_bwd<128>(s, a, t, b, st);
}

}  // namespace delta
}  // namespace ssd
