// Building blocks of the gated delta rule kernels: warp matrix fragments,
// power-of-two scaled fp16 splits and the chunk table.
//
// The rule (per value head, state S [dv][dk]) over a chunk of C = 64 tokens,
// with c_i = g_1 + ... + g_i, D_ij = exp(c_i - c_j) and S the state before it:
//     L_ij = D_ij k_i.k_j (j < i),   P_ij = D_ij q_i.k_j (j <= i)
//     (I + L diag(beta)) Y = -L      (Y strictly lower)
//     R = V - e^c K S^T,   E = R + Y (beta R),   U = beta E
//     O = e^c Q S^T + P U,           S' = e^{c_C} S + (e^{c_C - c} U)^T K
// E holds the prediction errors v_t - S~_t k_t, U the written values.
//
// Every product runs on fp16 operands with fp32 accumulation and keeps fp32's
// precision, because the state is carried over the whole sequence: a bf16
// token row times a power of two is exact in fp16 (down to 2^-25 of the row's
// largest element), and an fp32 operand is split as x = hi + lo, hi = fp16(x),
// lo = fp16(x - hi), after its row is scaled by a power of two to [2^12, 2^13):
// what is dropped is below 2^-22 of an element and 2^-36 of the row.  A token operand
// times an fp32 one takes 2 products (hi, lo), two fp32 ones 3 (hi hi, lo hi,
// hi lo).  bf16 pieces would need 3 and 6 for the same precision.  The per-chunk
// gradients, which have no scales at hand, take TF32 parts in the same way.
#pragma once

#include "common.cuh"

namespace ttt {

constexpr int DR_C = 64;           // tokens of a chunk
constexpr int DR_TOK_EXP = 8;      // token rows are scaled to [2^8, 2^9)
constexpr int DR_ROW_EXP = 12;     // split fp32 rows are scaled to [2^12, 2^13)
constexpr int DR_TILE = DR_C * DR_C * 2;  // bytes of a 64 x 64 fp16 tile

// Per-chunk vectors of a value head, float [DR_NVEC][64].
enum {
  DV_AR = 0,    // e^{c_j} f_k : factor of K16 S^T in R
  DV_BETA = 1,
  DV_YS = 2,    // inverse row scale of Y
  DV_AO = 3,    // scale e^{c_i} f_q : factor of Q16 S^T in O
  DV_PS = 4,    // inverse row scale of P
  DV_AK = 5,    // e^{c_C - c_j} f_k : factor of U in S'
  DV_EG = 6,    // e^{c_C} (64 times)
  DV_C = 7,     // c_j, and what fp32 leaves of it (differences of far-off c's keep their digits)
  DV_CLO = 8,
  DR_NVEC = 9
};
// A value head's chunk block: Y hi | Y lo | vectors | P hi | P lo.  The scan takes what stands before P.
constexpr int DR_VEC = 2 * DR_TILE;                          // byte offset of the vectors
constexpr int DR_P = DR_VEC + DR_NVEC * DR_C * 4;            // ... and of P
constexpr int DR_BLK = DR_P + 2 * DR_TILE;

// A sequence, or a segment of one: first token, tokens in it (-1: nothing to do), first chunk, the sequence's
// number, the segment's number in it and how many it has, its number among the segments of cut sequences.
struct DrSeq {
  int tok, len, chunk0, id, seg, nseg, cut, pad;
};
struct DrChunk {  // one chunk: first token, tokens in it (-1: unused entry)
  int tok, len;
};

// ---- warp matrix fragments (m16n8k16): accumulators c[0..1] = (row g, cols 2t, 2t+1),
// c[2..3] = (row g + 8, the same), with g = lane / 4, t = lane % 4.

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four neighbouring 8-wide tiles: independent products in a row, so that the next four on the same accumulators
// do not wait for them (a product's latency is that of four issues of one warp).
__device__ __forceinline__ void mma_f16x4(float (*c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2][4]) {
  mma_f16(c[0], a, b[0][0], b[0][1]);
  mma_f16(c[1], a, b[0][2], b[0][3]);
  mma_f16(c[2], a, b[1][0], b[1][1]);
  mma_f16(c[3], a, b[1][2], b[1][3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// Untiled bulk copy global -> shared; both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// This lane's arrival on `bar` once its cp.async copies so far have landed (counted in the barrier's init).
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 2^n for -126 <= n <= 127
__device__ __forceinline__ float pow2i(int n) { return __int_as_float((n + 127) << 23); }

// Exponent of a power of two (-127 for one that has underflowed to zero or below the normal range).
__device__ __forceinline__ int exp_of(float x) { return ((__float_as_int(x) >> 23) & 0xff) - 127; }

// Exponent n of a power of two 2^n that takes |m| (a row's largest magnitude) to [2^to, 2^(to+1));
// 0 for a zero, infinite or NaN row.
__device__ __forceinline__ int row_exp(float m, int to) {
  const int e = (__float_as_int(m) >> 23) & 0xff;
  if (e == 0xff || m == 0.f) return 0;
  const int n = to - (e - 127);
  return n > 120 ? 120 : n;  // the smallest rows stay below the target rather than overflow the factor
}

__device__ __forceinline__ float max_abs2(float m, float a, float b) { return fmaxf(m, fmaxf(fabsf(a), fabsf(b))); }
__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// (x, y) -> packed fp16 hi and lo parts
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// A fragment (16 rows x 16 k) from two neighbouring accumulator tiles, rows scaled by s0 (g) and s1 (g + 8).
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], float s0, float s1,
                                        uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c0[0] * s0, c0[1] * s0, hi[0], lo[0]);
  split2(c0[2] * s1, c0[3] * s1, hi[1], lo[1]);
  split2(c1[0] * s0, c1[1] * s0, hi[2], lo[2]);
  split2(c1[2] * s1, c1[3] * s1, hi[3], lo[3]);
}

// Byte offset of 16-byte chunk `ch` of row `row` in an image of rows of `row_bytes` (a multiple of 128).
__device__ __forceinline__ uint32_t img_off(int row, int ch, int row_bytes) {
  return (uint32_t)(row * row_bytes + ((ch ^ (row & 7)) << 4));
}

// ldmatrix addresses, all of one form: lane l reads row (l % 8) of 8x8 matrix l / 8.
//   B operand with n along the image's rows (n0 + 8 (m / 2)), k along its columns (chunk k0/8 + m % 2)
__device__ __forceinline__ uint32_t addr_bn(uint32_t base, int lane, int n0, int kch, int row_bytes) {
  return base + img_off(n0 + ((lane >> 4) << 3) + (lane & 7), kch + ((lane >> 3) & 1), row_bytes);
}
//   B operand with k along the image's rows, n along its columns (to be read with .trans); also an A
//   operand with rows along the image's rows, k along its columns (without .trans)
__device__ __forceinline__ uint32_t addr_bk(uint32_t base, int lane, int k0, int nch, int row_bytes) {
  return base + img_off(k0 + (((lane >> 3) & 1) << 3) + (lane & 7), nch + (lane >> 4), row_bytes);
}

}  // namespace ttt
