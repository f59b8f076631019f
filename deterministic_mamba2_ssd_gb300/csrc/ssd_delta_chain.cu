// ssd_delta_chain.cu -- the gated delta rule from chunk to chunk on the tensor
// cores: the forward recurrence of S with the outputs, and the reverse
// recurrence of dS.  What chunks can do side by side has been done before
// (ssd_delta_prep.cu), so that a chunk's step is, with rows p of the state on
// the left of every product,
//
//   forward    E = V' - S W^T        (p x t)    U = beta E
//              O = scale (exp(G) S Q^T + U P^T)
//              S = exp(G_C) S + (exp(G_C - G) U)^ K
//   backward   F = A + dS B^T        (p x t)    dv = beta F
//              dS = exp(G_C) dS + scale (exp(G) dO)^T Q - (exp(G) beta F)^ K
//
// One CTA takes one head through one sequence.  The state's rows are the 128
// lanes of tensor memory: S itself stays in registers (fp32, a row and a
// quarter of dstate a thread, 16 warps), its fp16 goes to tensor memory as the
// left operand, W, K, Q, P come as shared-memory tiles.  E and U likewise go
// from the accumulator through registers back to tensor memory as a left
// operand, so nothing that a thread computes passes through shared memory.
// Warp 16 copies the tiles (bulk copies, two or three chunks ahead), warp 17
// issues the products.
//
// What bounds the kernel is the chain of a chunk, which is sequential: product
// with W, E and U, product with K, the new S -- about 1.4k cycles.  All that the
// next chunk does not wait for (O, records) is issued behind it.
//
// Operands are fp16 with power-of-two scales: the tiles carry theirs, S and all
// that is in its units share one running scale a head, moved when the largest
// value leaves [2^-2, 2^6] (by powers of 2^8; looked at one chunk late, which
// 2^10 of head room allows).  One fp16 term is 11 bits (2^-12): enough for what
// leaves as bf16.  Where the fp32 state itself is asked for, S, W, V' and U are
// carried as two terms (22 bits); the sums are fp32 either way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ssd_delta_tiles.cuh"
#include "umma.cuh"

namespace ssd {
namespace delta {
namespace {

using mma16::pack;
using mma16::pow2_inv;
using mma16::split;
using mma16::unpack;

constexpr int kEpi = 16;                       // warps that hold the state
constexpr int kThreads = 32 * (kEpi + 2);
constexpr float kLow = 0.25f, kHigh = 64.f;    // window of the state's largest value; four times that with two terms
constexpr uint32_t kWait = 1u << 22;           // polls before a wait gives up

// Columns of tensor memory: the state's fp16 terms, accumulators, and the other left operands.
template <int kTerms>
struct Tmem {
  static constexpr uint32_t kS = 0, kX = 64 * kTerms, kO = kX + 64, kW = kO + 64, kD = kW + 32 * kTerms,
                            kO2 = kTerms == 2 ? kX : kD + 128,       // two terms leave no room: X has been read by then
                            kU = kTerms == 2 ? kS + 64 : kD + 192;   // and S's second term has been multiplied
  static constexpr uint32_t kAlloc = 512;
};
static_assert(Tmem<2>::kD + 128 <= 512 && Tmem<1>::kU + 32 <= 512, "tensor memory");

template <int N, int kTerms>
struct Fwd {
  static constexpr int kTile = kChunk * N * 2;
  static constexpr int kStages = kTerms == 2 ? 2 : 3;
  static constexpr int kW = 0, kK = kTerms * kTile, kQ = kK + kTile, kP = kQ + kTile, kV = kP + 8192,
                       kVecAt = kV + kTerms * kChunk * 128 * 2, kStage = kVecAt + 1024;
};
template <int N>
struct Bwd {
  static constexpr int kTile = kChunk * N * 2, kRows = kChunk * 128 * 2;
  static constexpr int kStages = 2;
  static constexpr int kB = 0, kK = kTile, kQ = kK + kTile, kX2 = kQ + kTile, kA = kX2 + kRows, kVecAt = kA + kRows,
                       kStage = kVecAt + 1024;
};

// Barriers and the other words of a CTA, after the stages.
struct Control {
  uint64_t full[3], free[3];   // tiles of a stage have come; all that reads them is done
  uint64_t state, left;        // the state's fp16, and the other left operands, are in tensor memory
  uint64_t x, d, o;            // the products with W (B), K, and the outputs' are done
  uint32_t tmem;
  int dead;                    // a wait ran out: nothing is waited for any more
  float top[2][kEpi];          // largest |S| of each warp, by chunk parity
};

struct Waits {
  Control *c;
  int *status;
  __device__ __forceinline__ void operator()(uint64_t &bar, uint32_t parity) const {
    if (*reinterpret_cast<volatile int *>(&c->dead)) return;
    if (!umma::mbar_wait(&bar, parity & 1u, kWait)) {
      c->dead = 1;
      *status = 1;
    }
  }
};

// Factor that brings the largest value `need` back into the window (1 while it is inside, zero or not finite).  With two
// terms the window lies higher, where the second term of a state of like elements is still a normal fp16.
template <int kTerms>
__device__ __forceinline__ float rescale(float need, float dn) {
  if (kTerms == 2) need *= 0.25f;
  if (!(need > kHigh || (need < kLow && need > 0.f)) || isinf(need)) return 1.f;
  const int e = int(__float_as_uint(need) >> 23) - 127 + 2;   // need = 2^-2 2^e (1 to 2)
  const int k = e >= 0 ? e / 8 : (e - 7) / 8;
  const float f = __uint_as_float(uint32_t(127 - 8 * max(-12, min(12, k))) << 23);
  const float lim = 1.0e33f;   // keeps both scales finite
  return dn * f > lim || dn * f < 1.f / lim ? 1.f : f;
}
template <int n>
__device__ __forceinline__ float warp_top(const float (&v)[n]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < n; ++i) m = fmaxf(m, fabsf(v[i]));
  return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(m)));
}
__device__ __forceinline__ float head_top(const float *top, int warps) {
  float m = 0.f;
  for (int i = 0; i < warps; ++i) m = fmaxf(m, top[i]);
  return m;
}

__device__ __forceinline__ void epi_sync(int warps) { asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory"); }

// Arrives when this warp's stores to tensor memory are done.
__device__ __forceinline__ void stored(uint64_t &bar, int lane) {
  umma::tmem_wait_st();
  umma::fence_before_sync();
  __syncwarp();
  if (lane == 0) umma::mbar_arrive(&bar);
}

// 64 columns K steps of 16: descriptor of step k of a K-major panel tile [64][..], and of an MN-major one [64 = K][..].
__device__ __forceinline__ uint64_t desc_k(uint32_t tile, int k) {
  return umma::smem_desc_sw128(tile + (k / 4) * (kChunk * 128) + (k % 4) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int k) {
  return umma::smem_desc_sw128(tile + k * 16 * 128, kChunk * 128, 1024);
}

// Where a warp stands: rows of its tensor memory quadrant, and which quarter of the columns is its own.
struct Place {
  int warps;        // warps that hold rows of this head
  int p;            // row
  bool on, live;    // the warp has rows of the head; this thread has one
  int quarter;
  uint32_t lanes;   // its quadrant's lane field of a tensor memory address
};
__device__ __forceinline__ Place place(int P, int warp, int lane) {
  Place l;
  const int quads = (P + 31) / 32;
  l.warps = 4 * quads;
  l.p = 32 * (warp & 3) + lane;
  l.on = warp < kEpi && (warp & 3) < quads;
  l.live = l.on && l.p < P;
  l.quarter = warp >> 2;
  l.lanes = uint32_t(32 * (warp & 3)) << 16;
  return l;
}
// This warp's slot among those that hold rows.
__device__ __forceinline__ int slot_of(const Place &l, int warp) { return l.quarter * (l.warps / 4) + (warp & 3); }

// The swizzled tiles need 1 KB alignment; without it nothing is done.
__device__ __forceinline__ bool misaligned(const uint8_t *smem, int *status) {
  if ((umma::smem_u32(smem) & 1023u) == 0) return false;
  if (threadIdx.x == 0) *status = 2;
  return true;
}

__device__ __forceinline__ void set_up(Control &ct, int stages, int warps, int warp, int lane, uint32_t cols) {
  if (warp == 0) umma::tmem_alloc(&ct.tmem, cols);
  if (warp == 1 && lane == 0) {
    for (int i = 0; i < stages; ++i) {
      umma::mbar_init(&ct.full[i], 1);
      umma::mbar_init(&ct.free[i], warps);
    }
    umma::mbar_init(&ct.state, warps);
    umma::mbar_init(&ct.left, warps);
    umma::mbar_init(&ct.x, 1);
    umma::mbar_init(&ct.d, 1);
    umma::mbar_init(&ct.o, 1);
    umma::fence_mbar_init();
    ct.dead = 0;
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
}
// Every copy has landed before the CTA's shared memory is given up.
__device__ __forceinline__ void drain(Control &ct, int stages, int issued) {
  for (int c = max(0, issued - stages); c < issued; ++c) umma::mbar_wait(&ct.full[c % stages], (c / stages) & 1, kWait);
}
__device__ __forceinline__ void tear_down(Control &ct, int warp, uint32_t cols) {
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    umma::fence_after_sync();
    umma::tmem_relinquish();
    umma::tmem_dealloc(ct.tmem, cols);
  }
}

// The state's fp16 terms to tensor memory; the first term is left in `hi`.
template <int kTerms, int kCols>
__device__ __forceinline__ void put_state(const float (&S)[kCols], uint32_t at, uint32_t (&hi)[kCols / 2]) {
  uint32_t lo[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    uint32_t p[kTerms];
    split<kTerms>(S[2 * i], S[2 * i + 1], p);
    hi[i] = p[0];
    if (kTerms == 2) lo[i] = p[kTerms - 1];
  }
  umma::tmem_st(at, hi);
  if (kTerms == 2) umma::tmem_st(at + 64, lo);
}
// This thread's part of the fp16 state's row p to the record: 16-byte chunks j0.. of a panel tile of P rows.
template <int kWords>
__device__ __forceinline__ void save_state(const uint32_t (&hi)[kWords], __half *tile, int p, int j0, int P) {
  uint8_t *to = reinterpret_cast<uint8_t *>(tile);
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i)
    *reinterpret_cast<uint4 *>(to + pan(p, j0 + i, P)) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
}
template <int kCols>
__device__ __forceinline__ void load_d(uint32_t at, float (&v)[kCols]) {
  if constexpr (kCols == 32) umma::tmem_ld32(at, v);
  else umma::tmem_ld16(at, v);
}

// CTA (head, sequence).
template <int N, int kTerms, bool kSave>
__global__ void __launch_bounds__(kThreads, 1) chain_fwd_kernel(Shape s, Args a, Tiles t) {
  using L = Fwd<N, kTerms>;
  using M = Tmem<kTerms>;
  constexpr int kCols = N / 4, kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control &ct = *reinterpret_cast<Control *>(smem + kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x;
  const int64_t seq = blockIdx.y;
  const Place me = place(s.P, warp, lane);
  const Waits wait{&ct, t.status};
  if (misaligned(smem, t.status)) return;
  set_up(ct, kStages, me.warps, warp, lane, M::kAlloc);
  const uint32_t base = umma::smem_u32(smem), tm = ct.tmem;
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0);
  const int nc = int(min((te - t0 + kChunk - 1) / kChunk, s.slots - slot0));

  if (warp == kEpi) {   // copies
    if (lane == 0) {
      int issued = 0;
      const uint32_t vbytes = uint32_t(kTerms * kChunk * s.P * 2);
      for (int c = 0; c < nc; ++c) {
        const int st = c % kStages;
        if (c >= kStages) wait(ct.free[st], c / kStages - 1);
        if (*reinterpret_cast<volatile int *>(&ct.dead)) break;
        uint8_t *to = smem + st * L::kStage;
        const int64_t ht = (slot0 + c) * s.H + h, kt = ((slot0 + c) * s.G + h / s.hpg) * kChunk * N;
        umma::mbar_expect_tx(&ct.full[st], (kTerms + 2) * L::kTile + 8192 + vbytes + kVecChain * 4);
        umma::bulk_load(to + L::kW, t.W16 + ht * kTerms * kChunk * N, kTerms * L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kK, t.K16 + kt, L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kQ, t.Q16 + kt, L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kP, t.P16 + ht * kTri, 8192, &ct.full[st]);
        umma::bulk_load(to + L::kV, t.V16 + ht * kTerms * kChunk * s.P, vbytes, &ct.full[st]);
        umma::bulk_load(to + L::kVecAt, t.vec + ht * kVec, kVecChain * 4, &ct.full[st]);
        issued = c + 1;
      }
      drain(ct, kStages, issued);
    }
    __syncwarp();
  } else if (warp == kEpi + 1) {   // products
    if (lane == 0) {
      constexpr uint32_t to_t = umma::idesc_f16_f32(128, kChunk, 0, 0);   // columns t: tiles [t][k]
      constexpr uint32_t to_n = umma::idesc_f16_f32(128, N, 0, 1);        // columns n: tiles [t = k][n]
      for (int c = 0; c < nc; ++c) {
        const int st = c % kStages;
        const uint32_t tile = base + st * L::kStage;
        wait(ct.full[st], c / kStages);
        wait(ct.state, c);
        if (kTerms == 2 && c > 0) wait(ct.free[(c - 1) % kStages], (c - 1) / kStages);   // O has been read out of X's columns
        umma::fence_after_sync();
#pragma unroll
        for (int x = 0; x < (kTerms == 2 ? 3 : 1); ++x)   // S W, then S's second term, then W's
#pragma unroll
          for (int k = 0; k < N / 16; ++k)
            umma::mma_f16_ta(tm + M::kX, tm + M::kS + (x == 1 ? 64 : 0) + 8 * k,
                             desc_k(tile + L::kW + (x == 2 ? L::kTile : 0), k), to_t, x + k > 0);
        umma::mma_commit(&ct.x);
        if (kTerms == 1 && c > 0) wait(ct.free[(c - 1) % kStages], (c - 1) / kStages);
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          umma::mma_f16_ta(tm + M::kO, tm + M::kS + 8 * k, desc_k(tile + L::kQ, k), to_t, k > 0);
        wait(ct.left, c);
        umma::fence_after_sync();
        auto outputs = [&]() {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma::mma_f16_ta(tm + M::kO2, tm + M::kU + 8 * k, desc_k(tile + L::kP, k), to_t, k > 0);
        };
        if (kTerms == 2) outputs();   // its left operand lies where the new state will
#pragma unroll
        for (int x = 0; x < kTerms; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma::mma_f16_ta(tm + M::kD, tm + M::kW + 32 * x + 8 * k, desc_mn(tile + L::kK, k), to_n, x + k > 0);
        umma::mma_commit(&ct.d);
        if (kTerms == 1) {
          outputs();
          umma::mma_commit(&ct.o);
        }
      }
    }
    __syncwarp();
  } else if (me.on) {
    const int my = slot_of(me, warp), P = s.P, n0 = kCols * me.quarter, tq = 16 * me.quarter;
    const uint32_t lanes = tm + me.lanes;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + int64_t(h) * P + me.p;
    const int64_t row = ((seq * s.H + h) * P + me.p) * N + n0;
    float S[kCols], up = 1.f, dn = 1.f;
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 v = me.live && a.init != nullptr ? *reinterpret_cast<const float4 *>(a.init + row + i)
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i] = v.x, S[i + 1] = v.y, S[i + 2] = v.z, S[i + 3] = v.w;
    }
    // V's largest value is below 16 times its tile's scale
    auto incoming = [&](int c) { return c < nc ? 16.f * __ldg(t.vec + ((slot0 + c) * s.H + h) * kVec + kVecSv) : 0.f; };
    auto move = [&](float f) {
      if (f != 1.f) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) S[i] *= f;
        dn *= f;
        up *= pow2_inv(f);
      }
    };
    // the state entering chunk c: to tensor memory, and to the record behind it
    auto enter = [&](int c) {
      uint32_t hi[kCols / 2];
      put_state<kTerms, kCols>(S, lanes + M::kS + n0 / 2, hi);
      const float m = warp_top(S);
      if (lane == 0) ct.top[c & 1][my] = m;
      stored(ct.state, lane);
      if (kSave) {
        const int64_t ht = (slot0 + c) * s.H + h;
        if (me.live) save_state(hi, t.S16 + ht * P * N, me.p, n0 / 8, P);
        if (my == 0 && lane == 0) t.up[ht] = up;
      }
    };
    if (nc > 0) {
      const float m = warp_top(S);
      if (lane == 0) ct.top[1][my] = m;
      epi_sync(me.warps);
      move(rescale<kTerms>(fmaxf(head_top(ct.top[1], me.warps), incoming(0)), 1.f));
      enter(0);
    }
    for (int c = 0; c < nc; ++c) {
      const int st = c % kStages;
      const uint8_t *tile = smem + st * L::kStage;
      const float *vec = reinterpret_cast<const float *>(tile + L::kVecAt);
      const __half *V = reinterpret_cast<const __half *>(tile + L::kV);
      const int64_t ht = (slot0 + c) * s.H + h, b = t0 + int64_t(c) * kChunk;
      const int n = int(min(int64_t(kChunk), te - b));
      const float next = incoming(c + 1);
      wait(ct.full[st], c / kStages);
      const float ka = vec[kVecKa], sv = vec[kVecSv] * dn, last = vec[kVecEg + kChunk - 1];
      float E[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = 0.f;
        if (me.live) {
          x = __half2float(V[(tq + i) * P + me.p]);
          if (kTerms == 2) x += __half2float(V[(kChunk + tq + i) * P + me.p]);
        }
        E[i] = x * sv;
      }
      wait(ct.x, c);
      umma::fence_after_sync();
      uint32_t e16[8];
      {
        float X[16];
        umma::tmem_ld16(lanes + M::kX + tq, X);
        uint32_t u[8], w0[8], w1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 tl = *reinterpret_cast<const float2 *>(vec + kVecTail + tq + 2 * i);
          const float2 be = *reinterpret_cast<const float2 *>(vec + kVecBeta + tq + 2 * i);
          const float e0 = fmaf(-ka, X[2 * i], E[2 * i]), e1 = fmaf(-ka, X[2 * i + 1], E[2 * i + 1]);
          if (kSave) e16[i] = pack(e0, e1);
          const float u0 = e0 * be.x, u1 = e1 * be.y;
          u[i] = pack(u0, u1);
          uint32_t p[kTerms];
          split<kTerms>(u0 * tl.x, u1 * tl.y, p);
          w0[i] = p[0];
          w1[i] = p[kTerms - 1];
        }
        umma::tmem_st(lanes + M::kW + tq / 2, w0);
        if (kTerms == 2) umma::tmem_st(lanes + M::kW + 32 + tq / 2, w1);
        umma::tmem_st(lanes + M::kU + tq / 2, u);
        stored(ct.left, lane);
      }
      wait(ct.state, c);   // over long since: makes the other warps' `top` visible
      const float f = c + 1 < nc ? rescale<kTerms>(fmaxf(head_top(ct.top[c & 1], me.warps), next * dn), dn) : 1.f;
      if (kSave && me.live) {
        __half *e = t.E16 + (ht * kChunk + tq) * P + me.p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __half2 v = *reinterpret_cast<const __half2 *>(&e16[i]);
          e[2 * i * P] = __low2half(v);
          e[(2 * i + 1) * P] = __high2half(v);
        }
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) S[i] *= last;
      const float co = a.scale * ka * up;
      float O[16];
      auto outputs = [&]() {
        float o2[16];
        umma::tmem_ld16(lanes + M::kO + tq, O);
        umma::tmem_ld16(lanes + M::kO2 + tq, o2);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 eg = *reinterpret_cast<const float2 *>(vec + kVecEg + tq + i);
          O[i] = co * fmaf(eg.x, O[i], ka * o2[i]);
          O[i + 1] = co * fmaf(eg.y, O[i + 1], ka * o2[i + 1]);
        }
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&ct.free[st]);
      };
      wait(ct.d, c);
      umma::fence_after_sync();
      if (kTerms == 2) outputs();   // before X's columns are written again
      {
        float D[kCols];
        load_d(lanes + M::kD + n0, D);
#pragma unroll
        for (int i = 0; i < kCols; ++i) S[i] = me.live ? fmaf(ka, D[i], S[i]) : 0.f;
      }
      move(f);
      if (c + 1 < nc) enter(c + 1);
      if (kTerms == 1) {
        wait(ct.o, c);
        umma::fence_after_sync();
        outputs();
      }
      if (me.live) {
        __nv_bfloat16 *to = o + (b + tq) * s.H * P;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (tq + i < n) to[int64_t(i) * s.H * P] = __float2bfloat16_rn(O[i]);
      }
    }
    if (me.live && a.fin != nullptr) {
#pragma unroll
      for (int i = 0; i < kCols; i += 4)
        *reinterpret_cast<float4 *>(a.fin + row + i) = make_float4(S[i] * up, S[i + 1] * up, S[i + 2] * up, S[i + 3] * up);
    }
  }
  tear_down(ct, warp, M::kAlloc);
}

// The reverse recurrence; writes dv, dinit, and for the gradient kernel dS leaving each chunk (D16) and F (F16).
template <int N>
__global__ void __launch_bounds__(kThreads, 1) chain_bwd_kernel(Shape s, Args a, Tiles t, BwdTiles o) {
  using L = Bwd<N>;
  constexpr int kCols = N / 4, kStages = L::kStages;
  // columns: dS's fp16, F, the left operand of K, and the two terms of the change of dS
  constexpr uint32_t kS = 0, kX = 64, kW = 128, kD = 160, kD2 = 288, kAlloc = 512;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control &ct = *reinterpret_cast<Control *>(smem + kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x;
  const int64_t seq = blockIdx.y;
  const Place me = place(s.P, warp, lane);
  const Waits wait{&ct, o.status};
  if (misaligned(smem, o.status)) return;
  set_up(ct, kStages, me.warps, warp, lane, kAlloc);
  const uint32_t base = umma::smem_u32(smem), tm = ct.tmem;
  int64_t t0, te;
  seq_range(s, a.cu, seq, t0, te);
  const int64_t slot0 = first_slot(s, a.cu, seq, t0);
  const int nc = int(min((te - t0 + kChunk - 1) / kChunk, s.slots - slot0));
  auto slot_at = [&](int c) { return slot0 + nc - 1 - c; };   // step c takes the sequence's chunk nc - 1 - c

  if (warp == kEpi) {
    if (lane == 0) {
      int issued = 0;
      const uint32_t abytes = uint32_t(kChunk * s.P * 2), xbytes = uint32_t(kChunk * padded(s.P) * 2);
      for (int c = 0; c < nc; ++c) {
        const int st = c % kStages;
        if (c >= kStages) wait(ct.free[st], c / kStages - 1);
        if (*reinterpret_cast<volatile int *>(&ct.dead)) break;
        uint8_t *to = smem + st * L::kStage;
        const int64_t ht = slot_at(c) * s.H + h, kt = (slot_at(c) * s.G + h / s.hpg) * kChunk * N;
        umma::mbar_expect_tx(&ct.full[st], 3 * L::kTile + abytes + xbytes + kVecChain * 4 + kSide * 4);
        umma::bulk_load(to + L::kB, o.B16 + ht * kChunk * N, L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kK, t.K16 + kt, L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kQ, t.Q16 + kt, L::kTile, &ct.full[st]);
        umma::bulk_load(to + L::kX2, o.X2 + ht * kChunk * padded(s.P), xbytes, &ct.full[st]);
        umma::bulk_load(to + L::kA, o.A16 + ht * kChunk * s.P, abytes, &ct.full[st]);
        umma::bulk_load(to + L::kVecAt, t.vec + ht * kVec, kVecChain * 4, &ct.full[st]);
        umma::bulk_load(to + L::kVecAt + kVecChain * 4, o.side + ht * kSide, kSide * 4, &ct.full[st]);
        issued = c + 1;
      }
      drain(ct, kStages, issued);
    }
    __syncwarp();
  } else if (warp == kEpi + 1) {
    if (lane == 0) {
      constexpr uint32_t to_t = umma::idesc_f16_f32(128, kChunk, 0, 0);
      constexpr uint32_t to_n = umma::idesc_f16_f32(128, N, 0, 1);
      constexpr uint32_t from_x = umma::idesc_f16_f32(128, N, 1, 1);   // left operand: tile [t = k][p]
      for (int c = 0; c < nc; ++c) {
        const int st = c % kStages;
        const uint32_t tile = base + st * L::kStage;
        wait(ct.full[st], c / kStages);
        wait(ct.state, c);
        umma::fence_after_sync();
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          umma::mma_f16_ta(tm + kX, tm + kS + 8 * k, desc_k(tile + L::kB, k), to_t, k > 0);
        umma::mma_commit(&ct.x);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma::mma_f16(tm + kD2, desc_mn(tile + L::kX2, k), desc_mn(tile + L::kQ, k), from_x, k > 0);
        wait(ct.left, c);
        umma::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma::mma_f16_ta(tm + kD, tm + kW + 8 * k, desc_mn(tile + L::kK, k), to_n, k > 0);
        umma::mma_commit(&ct.d);
      }
    }
    __syncwarp();
  } else if (me.on) {
    const int my = slot_of(me, warp), P = s.P, n0 = kCols * me.quarter, tq = 16 * me.quarter;
    const uint32_t lanes = tm + me.lanes;
    __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv) + int64_t(h) * P + me.p;
    const int64_t row = ((seq * s.H + h) * P + me.p) * N + n0;
    float D[kCols], up = 1.f, dn = 1.f;
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 v = me.live && a.dfinal != nullptr ? *reinterpret_cast<const float4 *>(a.dfinal + row + i)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
      D[i] = v.x, D[i + 1] = v.y, D[i + 2] = v.z, D[i + 3] = v.w;
    }
    // A's largest value is below 16 times its tile's scale
    auto incoming = [&](int c) { return c < nc ? 16.f * fabsf(__ldg(o.side + (slot_at(c) * s.H + h) * kSide)) : 0.f; };
    auto move = [&](float f) {
      if (f != 1.f) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) D[i] *= f;
        dn *= f;
        up *= pow2_inv(f);
      }
    };
    // the gradient of the state leaving the chunk of step c: to tensor memory, and to the record behind it
    auto leave = [&](int c) {
      uint32_t hi[kCols / 2];
      put_state<1, kCols>(D, lanes + kS + n0 / 2, hi);
      const float m = warp_top(D);
      if (lane == 0) ct.top[c & 1][my] = m;
      stored(ct.state, lane);
      const int64_t ht = slot_at(c) * s.H + h;
      if (me.live) save_state(hi, o.D16 + ht * P * N, me.p, n0 / 8, P);
      if (my == 0 && lane == 0) o.ub[ht] = up;
    };
    if (nc > 0) {
      const float m = warp_top(D);
      if (lane == 0) ct.top[1][my] = m;
      epi_sync(me.warps);
      move(rescale<1>(fmaxf(head_top(ct.top[1], me.warps), incoming(0)), 1.f));
      leave(0);
    }
    for (int c = 0; c < nc; ++c) {
      const int st = c % kStages;
      const uint8_t *tile = smem + st * L::kStage;
      const float *vec = reinterpret_cast<const float *>(tile + L::kVecAt);
      const __half *A = reinterpret_cast<const __half *>(tile + L::kA);
      const int64_t ht = slot_at(c) * s.H + h, b = t0 + int64_t(nc - 1 - c) * kChunk;
      const int n = int(min(int64_t(kChunk), te - b));
      const float next = incoming(c + 1);
      wait(ct.full[st], c / kStages);
      const float ka = vec[kVecKa], sa = vec[kVecChain] * dn, sx = vec[kVecChain + 1] * dn, last = vec[kVecEg + kChunk - 1];
      float F[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) F[i] = me.live ? sa * __half2float(A[(tq + i) * P + me.p]) : 0.f;
      wait(ct.x, c);
      umma::fence_after_sync();
      {
        float X[16];
        umma::tmem_ld16(lanes + kX + tq, X);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 eg = *reinterpret_cast<const float2 *>(vec + kVecEg + tq + 2 * i);
          const float2 be = *reinterpret_cast<const float2 *>(vec + kVecBeta + tq + 2 * i);
          F[2 * i] = fmaf(ka, X[2 * i], F[2 * i]);
          F[2 * i + 1] = fmaf(ka, X[2 * i + 1], F[2 * i + 1]);
          w[i] = pack(F[2 * i] * (-ka * eg.x * be.x), F[2 * i + 1] * (-ka * eg.y * be.y));
        }
        umma::tmem_st(lanes + kW + tq / 2, w);
        stored(ct.left, lane);
      }
      wait(ct.state, c);   // over long since: makes the other warps' `top` visible
      const float f = c + 1 < nc ? rescale<1>(fmaxf(head_top(ct.top[c & 1], me.warps), next * dn), dn) : 1.f;
      if (me.live) {
        __nv_bfloat16 *to = dv + (b + tq) * s.H * P;
        __half *f16 = o.F16 + (ht * kChunk + tq) * P + me.p;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f16[i * P] = __float2half_rn(F[i]);
          if (tq + i < n) to[int64_t(i) * s.H * P] = __float2bfloat16_rn(F[i] * (vec[kVecBeta + tq + i] * up));
        }
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) D[i] *= last;
      const float co = a.scale * ka * sx;
      wait(ct.d, c);
      umma::fence_after_sync();
      {
        float d[kCols];
        load_d(lanes + kD2 + n0, d);
#pragma unroll
        for (int i = 0; i < kCols; ++i) D[i] = fmaf(co, d[i], D[i]);
        load_d(lanes + kD + n0, d);
#pragma unroll
        for (int i = 0; i < kCols; ++i) D[i] = me.live ? D[i] + d[i] : 0.f;   // lanes past the head hold anything
      }
      move(f);
      umma::fence_before_sync();
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(&ct.free[st]);
      if (c + 1 < nc) leave(c + 1);
    }
    if (me.live && a.dinit != nullptr) {
#pragma unroll
      for (int i = 0; i < kCols; i += 4)
        *reinterpret_cast<float4 *>(a.dinit + row + i) = make_float4(D[i] * up, D[i + 1] * up, D[i + 2] * up, D[i + 3] * up);
    }
  }
  tear_down(ct, warp, kAlloc);
}

template <int N, int kTerms, bool kSave>
cudaError_t go_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  auto kernel = chain_fwd_kernel<N, kTerms, kSave>;
  constexpr int smem = Fwd<N, kTerms>::kStages * Fwd<N, kTerms>::kStage + sizeof(Control);
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(unsigned(s.H), unsigned(s.nseq)), kThreads, smem, st>>>(s, a, t);
  return cudaGetLastError();
}
template <int N, int kTerms>
cudaError_t fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  return t.S16 != nullptr ? go_fwd<N, kTerms, true>(s, a, t, st) : go_fwd<N, kTerms, false>(s, a, t, st);
}
template <int N>
cudaError_t bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  auto kernel = chain_bwd_kernel<N>;
  constexpr int smem = Bwd<N>::kStages * Bwd<N>::kStage + sizeof(Control);
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(unsigned(s.H), unsigned(s.nseq)), kThreads, smem, st>>>(s, a, t, b);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chain_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st) {
  if (s.N == 64) return t.planes == 2 ? fwd<64, 2>(s, a, t, st) : fwd<64, 1>(s, a, t, st);
  return t.planes == 2 ? fwd<128, 2>(s, a, t, st) : fwd<128, 1>(s, a, t, st);
}

cudaError_t launch_chain_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st) {
  return s.N == 64 ? bwd<64>(s, a, t, b, st) : bwd<128>(s, a, t, b, st);
}

}  // namespace delta
}  // namespace ssd
