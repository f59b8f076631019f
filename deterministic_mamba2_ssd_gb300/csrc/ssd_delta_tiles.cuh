// ssd_delta_tiles.cuh -- what the tensor-core kernels of the gated delta rule
// hand to one another: per chunk and head (or group) fp16 tiles, each with the
// power-of-two scale that keeps its values inside fp16's range.
//
// With G_t the running sum of g in the chunk, L_ts = exp(G_t - G_s) (k_t . k_s)
// for s < t and Y = (I + L diag(beta))^-1 L:
//
//   K16, Q16 (slot, group)  k, q of 64 tokens, rows [token][dstate], times 2^-a:
//                           the larger tile's largest element in [8, 16), so
//                           that bf16 input is exact down to 2^-21 of it and no
//                           sum of 128 products leaves fp16's range
//   W16 (slot, head)        rows [t][dstate] of (I - Y diag(beta)) diag(exp(G)) K16;
//                           one plane, or two with the rounding left over
//   V16 (slot, head)        rows [t][p] (plain) of (I - Y diag(beta)) V times
//                           2^-v; one plane or two
//   P16 (slot, head)        exp(G_t - G_s) (q16_t . k16_s), s <= t
//   Y16 (slot, head)        beta_t Y_ts, s < t
//   vec (slot, head)        kVec floats, see the offsets below
//   S16 (slot, head)        state entering the chunk, rows [p][n], times 2^-r
//   E16 (slot, head)        e of the chunk, rows [t][p] (plain), times 2^-r
//   up  (slot, head)        2^r
// and for the backward, made before its chain:
//   B16 (slot, head)        rows [t][dstate] of (I - Y diag(beta))^T ... of tail K16:
//                           exp(G_C - G_s) k_s - sum_t beta_t Y_ts exp(G_C - G_t) k_t
//   A16 (slot, head)        rows [t][p] (plain): the same of scale 2^a P16^T dO, times 2^-f
//   X16 (slot, head)        dO, rows [t][p], times 2^-x
//   X2  (slot, head)        exp(G_t) dO_t, likewise
// and by it, with a scale ub of its own: D16 like S16, the gradient of the
// state leaving the chunk, and F16 like E16, F = dS k.
//
// "Rows [r][c]" are panels of 64 columns, [panel][row][128 bytes], with the
// 16-byte chunk j of row r at j ^ (r % 8): what both the tensor cores' shared
// memory descriptors and ldmatrix read without bank conflicts, as a K-major or
// an MN-major operand.
#pragma once

#include <cuda_fp16.h>

#include "mma16.cuh"
#include "ssd_delta.h"

namespace ssd {
namespace delta {

constexpr int kVecEg = 0;       // exp(G_t)
constexpr int kVecTail = 64;    // exp(G_C - G_t)
constexpr int kVecBeta = 128;
constexpr int kVecKa = 192;     // 2^a
constexpr int kVecSv = 193;     // 2^v
constexpr int kVecG = 200;      // G_t
constexpr int kVecGl = 264;     // and what its rounding left over
constexpr int kVec = 328;
constexpr int kVecChain = 196;  // the part that the chains read
constexpr int kSide = 4;        // floats of a backward record: 2^f, 2^x
constexpr int kTri = kChunk * kChunk;   // elements of a Y16 or P16 tile

// Byte offset of 16-byte chunk j of row r in a tile of `rows` rows.
__host__ __device__ __forceinline__ uint32_t pan(uint32_t r, uint32_t j, uint32_t rows) {
  return (j >> 3) * rows * 128u + r * 128u + (((j & 7u) ^ (r & 7u)) << 4);
}

// Columns of a panel tile of P columns.
__host__ __device__ __forceinline__ int64_t padded(int64_t P) { return (P + 63) / 64 * 64; }

struct Tiles {
  int *status;   // set where a bounded wait ran out
  __half *K16, *Q16, *W16, *V16, *P16, *Y16, *S16, *E16;
  float *vec, *up;
  size_t rec_bytes, work_bytes;
  int planes;    // of W16 and V16
};

// What the forward makes: in `rec`, with the parts that a backward reads, and the rest in `work`; without rec all that is
// needed in `work`.  planes: 2 where the fp32 state is asked for.
inline Tiles carve_tiles(const Shape &s, void *rec, void *work, bool record, int planes) {
  Carver r(rec), w(work);
  Carver &c = record ? r : w;
  Tiles t{};
  t.planes = planes;
  t.status = c.take<int>(4);
  t.K16 = c.take<__half>(s.slots * s.G * kChunk * s.N);
  t.Q16 = c.take<__half>(s.slots * s.G * kChunk * s.N);
  t.P16 = c.take<__half>(s.slots * s.H * kTri);
  t.vec = c.take<float>(s.slots * s.H * kVec);
  if (record) {
    t.Y16 = c.take<__half>(s.slots * s.H * kTri);
    t.S16 = c.take<__half>(s.slots * s.H * s.P * s.N);
    t.E16 = c.take<__half>(s.slots * s.H * kChunk * s.P);
    t.up = c.take<float>(s.slots * s.H);
  }
  t.W16 = w.take<__half>(s.slots * s.H * planes * kChunk * s.N);
  t.V16 = w.take<__half>(s.slots * s.H * planes * kChunk * s.P);
  t.rec_bytes = r.bytes();
  t.work_bytes = w.bytes();
  return t;
}

struct BwdTiles {
  int *status;
  __half *B16, *A16, *X16, *X2, *D16, *F16;
  float *side, *ub;
  size_t bytes;
};
inline BwdTiles carve_bwd_tiles(const Shape &s, void *p) {
  Carver c(p);
  BwdTiles t{};
  t.status = c.take<int>(4);
  t.B16 = c.take<__half>(s.slots * s.H * kChunk * s.N);
  t.A16 = c.take<__half>(s.slots * s.H * kChunk * s.P);
  t.X16 = c.take<__half>(s.slots * s.H * kChunk * padded(s.P));
  t.X2 = c.take<__half>(s.slots * s.H * kChunk * padded(s.P));
  t.D16 = c.take<__half>(s.slots * s.H * s.P * s.N);
  t.F16 = c.take<__half>(s.slots * s.H * kChunk * s.P);
  t.side = c.take<float>(s.slots * s.H * kSide);
  t.ub = c.take<float>(s.slots * s.H);
  t.bytes = c.bytes();
  return t;
}

// Kernel launches (ssd_delta_prep.cu, ssd_delta_chain.cu, ssd_delta_grads.cu).
cudaError_t launch_prep(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st);
cudaError_t launch_prep_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st);
cudaError_t launch_chain_fwd(const Shape &s, const Args &a, const Tiles &t, cudaStream_t st);
cudaError_t launch_chain_bwd(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st);
cudaError_t launch_grads(const Shape &s, const Args &a, const Tiles &t, const BwdTiles &b, cudaStream_t st);

}  // namespace delta
}  // namespace ssd
