// Gated delta rule, gradient of the chunked form (bf16 tokens).
//
// With the symbols of delta_common.cuh and S' the state after the chunk, from dO and dS':
//     dU = P^T dO + e^{c_C - c} K dS'^T,     Z = dU + Y^T (beta dU)   (= M^-T dU)
//     dV = beta Z,   dbeta = E . Z
//     dS = e^{c_C} dS' + (e^c dO)^T Q - (e^c beta Z)^T K
//     F_ij = D_ij dO_i.U_j (j <= i),   W_ij = D_ij beta_i Z_i.U_j (j < i)
//     dQ = e^c dO S + F K
//     dK = -e^c beta Z S - W K + e^{c_C - c} U dS' + F^T Q - W^T K
// Scaling S by exp(g_t) at token t scales every later o and read error alike, so
//     dg_t = <S~_t, dS~_t> = <S', dS'> + sum_{i >= t} (dO_i.O_i - dV_i.V_i)
//     <S', dS'> = e^{c_C} <S, dS'> + sum_j U_j . e^{c_C - c_j} dS' k_j
// with <S', dS'> taken at each chunk's end: no sum runs over more than a chunk.  Where dg is zero by itself (a token
// that resets the state, or a chunk's first one behind a state of zeros) the sums of that chunk start there,
//     dg_t = -sum_{a <= i < t} (...)_i for t >= a,   sum_{t <= i < a} (...)_i before it,
// so that it is zero exactly and not a difference of sums.
//
// Passes: the chunk preparation and the state pass again (they keep S, E and
// dO.O), the reverse pass over the chunks (dS in registers as the state pass
// has S; it keeps dS' and Z and writes dV), and one block per chunk and
// query/key head for dQ, dK and the gates.
#pragma once

#include "kernels_delta.cuh"

namespace ttt {

struct ReverseArgs {
  const __nv_bfloat16 *V, *dO;
  __nv_bfloat16* dV;
  int64_t ldv, ldo;
  const float* dS;  // gradient of the state after each sequence (null: zeros)
  float* dS0;       // gradient of the state before it (null: not wanted)
  int hk, hv, dk, dv;
  const DrSeq* seqs;
  const uint8_t* kq;
  const uint8_t* blk;
  Guard guard;
  const float* keep_e;
  float* keep_ds;  // [chunk][hv][dv][dk] dS'
  float* keep_z;   // [chunk][hv][dv][64] Z^T
  float* w_part;   // [chunk][hv][dv / 16][64]: dO.O in, dO.O - dV.V out
  float* b_part;   // [chunk][hv][dv / 16][64] E.Z
  float* x_part;   // [chunk][hv][dv / 16] sum_j U_j . e^{c_C - c_j} dS' k_j
  // segments of cut sequences: [cut][hv][dv][dk] gradients at their ends (of the segments before the last) and scan results
  float *seg_ds, *seg_n;
};

// As the state pass: a warp owns 16 value channels and keeps dS [16][dk] in registers.  SCAN: only what a segment
// adds to the gradient that passes through it (from zero; the last segment from dS).
template <int DK, bool SCAN>
__global__ void __launch_bounds__(160, 1) k_delta_reverse(const ReverseArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int STAGE = state_stage<DK, PASS_BACK>();
  constexpr int KQ = 2 * DR_C * DK * 2;
  constexpr int WSM = state_warp_smem<PASS_BACK>();
  constexpr int NT = DK / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = (blockDim.x >> 5) - 1;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* vbuf = smem + 2 * STAGE + warp * WSM;
  float* etile = reinterpret_cast<float*>(smem + 2 * STAGE + nwarp * WSM);  // [16 nwarp][64] E of one chunk
  uint64_t* full = reinterpret_cast<uint64_t*>(etile + nwarp * (DR_ETILE / 4));  // [2] stages, [1] E have landed
  uint64_t* empty = full + 3;                                                    // [2] stages, [1] E are read
  const int vblocks = (a.dv + nwarp * 16 - 1) / (nwarp * 16);
  const int h = blockIdx.x / vblocks % a.hv, hq = h / (a.hv / a.hk);
  const int vfirst = blockIdx.x % vblocks * nwarp * 16, v0 = vfirst + warp * 16;
  const int n16 = (a.dv + 15) / 16;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&full[i], i < 2 ? 33 : 1);
      mbar_init(&empty[i], nwarp);
    }
    fence_mbar_init();
  }
  pdl_wait();
  const int si = blockIdx.x / (vblocks * a.hv);
  const DrSeq sq = a.seqs[si];
  __syncthreads();
  if (sq.len < 0) return;
  const int nchunk = (sq.len + DR_C - 1) / DR_C;

  if (warp == nwarp) {  // the last warp brings the chunks, the last one first
#pragma unroll 1
    for (int it = 0; it < nchunk; ++it) {
      const int n = nchunk - 1 - it, buf = it & 1;
      const int64_t ci = sq.chunk0 + n;
      uint64_t* bar = &full[buf];
      if (it >= 2) mbar_wait(&empty[buf], ((it >> 1) - 1) & 1, a.guard);
      if (lane == 0) {
        uint8_t* st = smem + buf * STAGE;
        mbar_expect_tx(bar, STAGE);
        bulk_load(st, a.kq + (ci * a.hk + hq) * KQ, KQ, bar);
        bulk_load(st + KQ, a.blk + (ci * a.hv + h) * DR_BLK, DR_BLK, bar);
      }
      for (int w = 0; w < nwarp; ++w) {
        const uint32_t dst = smem_u32(smem + 2 * STAGE + w * WSM + buf * DR_VTILE);
        if constexpr (!SCAN) load_vtile(dst, a.V, a.ldv, sq, n, h * a.dv, vfirst + w * 16, a.dv, lane);
        load_vtile(dst + 2 * DR_VTILE, a.dO, a.ldo, sq, n, h * a.dv, vfirst + w * 16, a.dv, lane);
      }
      cp_arrive(bar);
      if constexpr (!SCAN) {  // one E tile: free from the middle of the chunk before
        if (it >= 1) mbar_wait(&empty[2], (it - 1) & 1, a.guard);
        if (lane == 0) {
          const uint32_t bytes = min(nwarp * 16, a.dv - vfirst) * DR_C * 4;
          mbar_expect_tx(&full[2], bytes);
          bulk_load(etile, a.keep_e + ((ci * a.hv + h) * a.dv + vfirst) * DR_C, bytes, &full[2]);
        }
      }
    }
    return;
  }

  float s[NT][4];
  const int64_t srow = ((int64_t)sq.id * a.hv + h) * a.dv, grow = ((int64_t)sq.cut * a.hv + h) * a.dv;
  const float* from = sq.seg == sq.nseg - 1 ? (a.dS ? a.dS + srow * a.dk : nullptr) : SCAN ? nullptr
                                                                                         : a.seg_ds + grow * a.dk;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = v0 + g + 8 * p, col = n * 8 + 2 * t;
      float2 x = make_float2(0.f, 0.f);
      if (from && r < a.dv && col < a.dk) x = *reinterpret_cast<const float2*>(from + (int64_t)r * a.dk + col);
      s[n][2 * p] = x.x;
      s[n][2 * p + 1] = x.y;
    }
  float inv0 = 1.f, inv1 = 1.f;  // dS = s * inv

#pragma unroll 1
  for (int it = 0; it < nchunk; ++it) {
    const int n = nchunk - 1 - it, buf = it & 1;
    mbar_wait(&full[buf], (it >> 1) & 1, a.guard);  // (as in the state pass)
    const uint32_t st = smem_u32(smem + buf * STAGE);
    const uint32_t kb = st, qb = st + DR_C * DK * 2, yh = st + KQ, yl = yh + DR_TILE, ph = yh + DR_P, pl = ph + DR_TILE;
    const float* vec = reinterpret_cast<const float*>(smem + buf * STAGE + KQ + DR_VEC);
    const uint32_t vb = smem_u32(vbuf + buf * DR_VTILE), db = smem_u32(vbuf + (2 + buf) * DR_VTILE);
    const int64_t blk = (int64_t)(sq.chunk0 + n) * a.hv + h;

    if constexpr (!SCAN) store_rows<NT>(a.keep_ds + (blk * a.dv + v0) * a.dk, s, inv0, inv1, a.dv - v0, a.dk, lane);
    // dS' K^T
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      m0 = max_abs2(m0, s[k][0], s[k][1]);
      m1 = max_abs2(m1, s[k][2], s[k][3]);
    }
    const int e0 = row_exp(quad_max(m0), DR_ROW_EXP), e1 = row_exp(quad_max(m1), DR_ROW_EXP);
    const float sc0 = pow2i(e0), sc1 = pow2i(e1);
    const float is0 = inv0 * pow2i(-e0), is1 = inv1 * pow2i(-e1);
    float r[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k][j] = 0.f;
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
      uint32_t hi[4], lo[4];
      split_a(s[2 * kt], s[2 * kt + 1], sc0, sc1, hi, lo);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b[4];
        ldsm4(b, addr_bn(kb, lane, np * 16, kt * 2, DK * 2));
        mma_f16(r[2 * np], hi, b[0], b[1]);
        mma_f16(r[2 * np + 1], hi, b[2], b[3]);
        mma_f16(r[2 * np], lo, b[0], b[1]);
        mma_f16(r[2 * np + 1], lo, b[2], b[3]);
      }
    }
    // the dO tile in the accumulator layout (bf16 pairs)
    uint32_t d[8][2];
    m0 = m1 = 0.f;
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t v[4];
      ldsm4t(v, vtile_addr(db, lane, np * 16));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = 2 * np + q;
        d[k][0] = v[2 * q];
        d[k][1] = v[2 * q + 1];
        const float2 ps = *reinterpret_cast<const float2*>(vec + DV_PS * DR_C + k * 8 + 2 * t);
        m0 = max_abs2(m0, __uint_as_float(d[k][0] << 16) * ps.x, __uint_as_float(d[k][0] & 0xffff0000u) * ps.y);
        m1 = max_abs2(m1, __uint_as_float(d[k][1] << 16) * ps.x, __uint_as_float(d[k][1] & 0xffff0000u) * ps.y);
      }
    }
    // dU = P^T dO + e^{c_C - c} K dS'^T; dO times P's row scale is exact in fp16
    {
      const int f0 = row_exp(quad_max(m0), DR_ROW_EXP), f1 = row_exp(quad_max(m1), DR_ROW_EXP);
      const float w0 = pow2i(f0), w1 = pow2i(f1), i0 = pow2i(-f0), i1 = pow2i(-f1);
      float x[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        uint32_t hi[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 ps = *reinterpret_cast<const float2*>(vec + DV_PS * DR_C + (2 * kt + q) * 8 + 2 * t);
          const uint32_t a0 = d[2 * kt + q][0], a1 = d[2 * kt + q][1];
          hi[2 * q] = pack_f16x2(__uint_as_float(a0 << 16) * ps.x * w0, __uint_as_float(a0 & 0xffff0000u) * ps.y * w0);
          hi[2 * q + 1] =
              pack_f16x2(__uint_as_float(a1 << 16) * ps.x * w1, __uint_as_float(a1 & 0xffff0000u) * ps.y * w1);
        }
#pragma unroll
        for (int np = 0; np <= kt; ++np) {
          uint32_t p[4];
          ldsm4t(p, addr_bk(ph, lane, kt * 16, np * 2, 128));
          mma_f16(x[2 * np], hi, p[0], p[1]);
          mma_f16(x[2 * np + 1], hi, p[2], p[3]);
          ldsm4t(p, addr_bk(pl, lane, kt * 16, np * 2, 128));
          mma_f16(x[2 * np], hi, p[0], p[1]);
          mma_f16(x[2 * np + 1], hi, p[2], p[3]);
        }
      }
      float kept = 0.f;
      if constexpr (!SCAN) mbar_wait(&full[2], it & 1, a.guard);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = k * 8 + 2 * t;
        const float2 ak = *reinterpret_cast<const float2*>(vec + DV_AK * DR_C + col);
        const float h00 = ak.x * (r[k][0] * is0), h01 = ak.y * (r[k][1] * is0);
        const float h10 = ak.x * (r[k][2] * is1), h11 = ak.y * (r[k][3] * is1);
        if constexpr (!SCAN) {  // U = beta E (what lies past dv is not read: dS' is zero there, E is not)
          const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + col);
          if (v0 + g < a.dv) {
            const float2 e = *reinterpret_cast<const float2*>(etile + (warp * 16 + g) * DR_C + etile_col(g, col));
            kept += be.x * e.x * h00 + be.y * e.y * h01;
          }
          if (v0 + g + 8 < a.dv) {
            const float2 e = *reinterpret_cast<const float2*>(etile + (warp * 16 + g + 8) * DR_C + etile_col(g, col));
            kept += be.x * e.x * h10 + be.y * e.y * h11;
          }
        }
        r[k][0] = x[k][0] * i0 + h00;
        r[k][1] = x[k][1] * i0 + h01;
        r[k][2] = x[k][2] * i1 + h10;
        r[k][3] = x[k][3] * i1 + h11;
      }
      if constexpr (!SCAN) {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) kept += __shfl_xor_sync(0xffffffffu, kept, m);
        if (lane == 0 && v0 < a.dv) a.x_part[blk * n16 + v0 / 16] = kept;
      }
    }
    // Z = dU + Y^T (beta dU); Y's row scale goes to the other factor
    {
      m0 = m1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + k * 8 + 2 * t);
        const float2 ys = *reinterpret_cast<const float2*>(vec + DV_YS * DR_C + k * 8 + 2 * t);
        m0 = max_abs2(m0, r[k][0] * (be.x * ys.x), r[k][1] * (be.y * ys.y));
        m1 = max_abs2(m1, r[k][2] * (be.x * ys.x), r[k][3] * (be.y * ys.y));
      }
      const int f0 = row_exp(quad_max(m0), DR_ROW_EXP), f1 = row_exp(quad_max(m1), DR_ROW_EXP);
      const float w0 = pow2i(f0), w1 = pow2i(f1), i0 = pow2i(-f0), i1 = pow2i(-f1);
      float x[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        float b[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int k = 2 * kt + q;
          const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + k * 8 + 2 * t);
          const float2 ys = *reinterpret_cast<const float2*>(vec + DV_YS * DR_C + k * 8 + 2 * t);
#pragma unroll
          for (int j = 0; j < 4; ++j) b[q][j] = r[k][j] * (j & 1 ? be.y * ys.y : be.x * ys.x);
        }
        uint32_t hi[4], lo[4];
        split_a(b[0], b[1], w0, w1, hi, lo);
#pragma unroll
        for (int np = 0; np <= kt; ++np) {
          uint32_t y[4];
          ldsm4t(y, addr_bk(yh, lane, kt * 16, np * 2, 128));
          mma_f16(x[2 * np], hi, y[0], y[1]);
          mma_f16(x[2 * np + 1], hi, y[2], y[3]);
          mma_f16(x[2 * np], lo, y[0], y[1]);
          mma_f16(x[2 * np + 1], lo, y[2], y[3]);
          ldsm4t(y, addr_bk(yl, lane, kt * 16, np * 2, 128));
          mma_f16(x[2 * np], hi, y[0], y[1]);
          mma_f16(x[2 * np + 1], hi, y[2], y[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[k][0] += x[k][0] * i0;
        r[k][1] += x[k][1] * i0;
        r[k][2] += x[k][2] * i1;
        r[k][3] += x[k][3] * i1;
      }
    }
    // keep Z, the gates' row sums, dV = beta Z
    if constexpr (!SCAN) {
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t v[4], y[4];
        ldsm4t(v, vtile_addr(vb, lane, np * 16));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int k = 2 * np + q, col = k * 8 + 2 * t;
          const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + col);
          float ex = 0.f, ey = 0.f;
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (v0 + g + 8 * p < a.dv) {
              *reinterpret_cast<float2*>(a.keep_z + (blk * a.dv + v0 + g + 8 * p) * DR_C + col) =
                  make_float2(r[k][2 * p], r[k][2 * p + 1]);
              const float2 e =
                  *reinterpret_cast<const float2*>(etile + (warp * 16 + g + 8 * p) * DR_C + etile_col(g, col));
              ex += e.x * r[k][2 * p];
              ey += e.y * r[k][2 * p + 1];
            }
          const float d00 = be.x * r[k][0], d01 = be.y * r[k][1], d10 = be.x * r[k][2], d11 = be.y * r[k][3];
          const uint32_t x0 = v[2 * q], x1 = v[2 * q + 1];
          float wx = d00 * __uint_as_float(x0 << 16) + d10 * __uint_as_float(x1 << 16);
          float wy = d01 * __uint_as_float(x0 & 0xffff0000u) + d11 * __uint_as_float(x1 & 0xffff0000u);
#pragma unroll
          for (int m = 4; m < 32; m <<= 1) {
            ex += __shfl_xor_sync(0xffffffffu, ex, m);
            ey += __shfl_xor_sync(0xffffffffu, ey, m);
            wx += __shfl_xor_sync(0xffffffffu, wx, m);
            wy += __shfl_xor_sync(0xffffffffu, wy, m);
          }
          if (g == 0 && v0 < a.dv) {
            const int64_t at = (blk * n16 + v0 / 16) * DR_C + col;
            const float2 oo = *reinterpret_cast<const float2*>(a.w_part + at);
            *reinterpret_cast<float2*>(a.w_part + at) = make_float2(oo.x - wx, oo.y - wy);
            *reinterpret_cast<float2*>(a.b_part + at) = make_float2(ex, ey);
          }
          y[2 * q] = pack_bf16x2(d00, d01);
          y[2 * q + 1] = pack_bf16x2(d10, d11);
        }
        __syncwarp();  // every lane has read these tokens of the V tile; dV takes their place
        stsm4t(vtile_addr(vb, lane, np * 16), y[0], y[1], y[2], y[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[2]);  // E is read
      store_vtile(vbuf + buf * DR_VTILE, a.dV, a.ldv, sq, n, (int64_t)h * a.dv, v0, a.dv, lane);
    }
    // dS = e^{c_C} dS' + (e^c dO)^T Q - (e^c beta Z)^T K
    {
      m0 = m1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = k * 8 + 2 * t;
        const float2 ar = *reinterpret_cast<const float2*>(vec + DV_AR * DR_C + col);
        const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + col);
        const float2 ao = *reinterpret_cast<const float2*>(vec + DV_AO * DR_C + col);
        r[k][0] *= -ar.x * be.x;
        r[k][1] *= -ar.y * be.y;
        r[k][2] *= -ar.x * be.x;
        r[k][3] *= -ar.y * be.y;
        m0 = max_abs2(max_abs2(m0, r[k][0], r[k][1]), ao.x * __uint_as_float(d[k][0] << 16),
                      ao.y * __uint_as_float(d[k][0] & 0xffff0000u));
        m1 = max_abs2(max_abs2(m1, r[k][2], r[k][3]), ao.x * __uint_as_float(d[k][1] << 16),
                      ao.y * __uint_as_float(d[k][1] & 0xffff0000u));
      }
      const int f0 = min(row_exp(quad_max(m0), DR_ROW_EXP), 87 - exp_of(is0));
      const int f1 = min(row_exp(quad_max(m1), DR_ROW_EXP), 87 - exp_of(is1));
      const float w0 = pow2i(f0), w1 = pow2i(f1);
      const float eg = vec[DV_EG * DR_C];
      const float d0 = eg * inv0 * w0, d1 = eg * inv1 * w1;
      inv0 = pow2i(-f0);
      inv1 = pow2i(-f1);
      uint32_t hi[4][4], lo[4][4], ho[4][4], lp[4][4];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        split_a(r[2 * kt], r[2 * kt + 1], w0, w1, hi[kt], lo[kt]);
        float b[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 ao = *reinterpret_cast<const float2*>(vec + DV_AO * DR_C + (2 * kt + q) * 8 + 2 * t);
          const uint32_t a0 = d[2 * kt + q][0], a1 = d[2 * kt + q][1];
          b[q][0] = ao.x * __uint_as_float(a0 << 16);
          b[q][1] = ao.y * __uint_as_float(a0 & 0xffff0000u);
          b[q][2] = ao.x * __uint_as_float(a1 << 16);
          b[q][3] = ao.y * __uint_as_float(a1 & 0xffff0000u);
        }
        split_a(b[0], b[1], w0, w1, ho[kt], lp[kt]);
      }
      // (accumulators of their own, as in the state pass)
#pragma unroll
      for (int np = 0; np < DK / 16; np += 2) {
        float acc[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[k][j] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          uint32_t b[2][4], c[2][4];
          ldsm4t(b[0], addr_bk(kb, lane, kt * 16, np * 2, DK * 2));
          ldsm4t(b[1], addr_bk(kb, lane, kt * 16, np * 2 + 2, DK * 2));
          ldsm4t(c[0], addr_bk(qb, lane, kt * 16, np * 2, DK * 2));
          ldsm4t(c[1], addr_bk(qb, lane, kt * 16, np * 2 + 2, DK * 2));
          mma_f16x4(acc, lo[kt], b);
          mma_f16x4(acc, lp[kt], c);
          mma_f16x4(acc, hi[kt], b);
          mma_f16x4(acc, ho[kt], c);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[2 * np + k][0] = fmaf(s[2 * np + k][0], d0, acc[k][0]);
          s[2 * np + k][1] = fmaf(s[2 * np + k][1], d0, acc[k][1]);
          s[2 * np + k][2] = fmaf(s[2 * np + k][2], d1, acc[k][2]);
          s[2 * np + k][3] = fmaf(s[2 * np + k][3], d1, acc[k][3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[buf]);  // this warp has read the stage and its tiles
  }
  // the gradient of the state before the sequence; in the scan, that at the end of the segment before the last or
  // what a segment adds
  float* to = a.dS0 && sq.seg == 0 ? a.dS0 + srow * a.dk : nullptr;
  if (SCAN) to = sq.seg == sq.nseg - 1 ? a.seg_ds + (grow - (int64_t)a.hv * a.dv) * a.dk : a.seg_n + grow * a.dk;
  if (to) store_rows<NT>(to + (int64_t)v0 * a.dk, s, inv0, inv1, a.dv - v0, a.dk, lane);
}

// ---------------------------------------------------------------------------
// dQ, dK and the gates: one block per (chunk, query/key head), over the value
// heads that share it.  The products take fp32 operands as they lie in memory in
// two TF32 parts (no scaling: TF32 has fp32's range), three products for each,
// two where an operand is exact (dO, K16, Q16); the factors of token rows go to
// the other operand.  One part each is 2.5 times fewer products (packed
// documents 279 us instead of 440), but keeps 2^-11 of the terms where they
// cancel, as behind a key that is written again.  32 value channels at a time
// are copied in while the 32 before are multiplied.
// Bound by the tensor cores and one block's phases on an SM (255 registers):
// 55% tensor pipe, 0.31 issue slots.
struct GradArgs {
  const __nv_bfloat16 *dO;
  int64_t ldo, ldq, ldk;
  __nv_bfloat16 *dQ, *dK;
  float *dg, *dbeta;  // [T][hv]
  int hk, hv, dk, dv;
  const DrChunk* chunks;
  const uint8_t* kq;
  const uint8_t* blk;
  const float* tok;
  const float *keep_s, *keep_e, *keep_ds, *keep_z, *w_part, *b_part, *x_part;
};

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo in two TF32 parts (what the products drop of lo is below 2^-21 of x)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void split_tf32(float x0, float x1, float x2, float x3, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split_tf32(x0, hi[0], lo[0]);
  split_tf32(x1, hi[1], lo[1]);
  split_tf32(x2, hi[2], lo[2]);
  split_tf32(x3, hi[3], lo[3]);
}
// A in two parts times B in two parts (h0, h1), (l0, l1)
__device__ __forceinline__ void mma_tf32x3(float (&c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint32_t h0,
                                           uint32_t h1, uint32_t l0, uint32_t l1) {
  mma_tf32(c, lo, h0, h1);
  mma_tf32(c, hi, l0, l1);
  mma_tf32(c, hi, h0, h1);
}

constexpr int GR_V = 32;     // value channels of a tile
constexpr int GR_LDT = 72;   // floats per row of [channels][64] tiles: fragment reads k-major (4 rows x 8 columns) hit 32 banks
constexpr int GR_LDA = 68;   // ... of [64][64] tiles read row-major (8 rows x 4 columns)
constexpr int GR_LDO = 40;   // bf16 per row of a dO tile [64][32]
template <int DK>
constexpr int grad_stage() {  // S, dS' | E, Z | dO
  return (2 * GR_V * (DK + 8) + 2 * GR_V * GR_LDT) * 4 + DR_C * GR_LDO * 2;
}
template <int DK>
constexpr int grad_smem() {
  constexpr int stages = 2 * grad_stage<DK>(), kq = 2 * DR_C * (DK + 8) * 4;  // K~, Q~ take the stages' place
  return (stages > kq ? stages : kq) + (2 * DR_C * GR_LDA + 5 * DR_C + 16 + 8 * DR_C + TF_N * DR_C) * 4;
}

template <int DK>
__global__ void __launch_bounds__(256, 1) k_delta_grad(const GradArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int LDS = DK + 8, STAGE = grad_stage<DK>();
  constexpr int KQ_BYTES = 2 * DR_C * LDS * 4;
  constexpr int NH = DK / 16;  // n-tiles of a warp's half of the dk columns
  float* Km = reinterpret_cast<float*>(smem);  // K16 [64][LDS] and Q16, once the tiles are done
  float* Qm = Km + DR_C * LDS;
  float* Fm = reinterpret_cast<float*>(smem + (2 * STAGE > KQ_BYTES ? 2 * STAGE : KQ_BYTES));  // F [64][GR_LDA]
  float* Wm = Fm + DR_C * GR_LDA;                                                              // W
  float* vc = Wm + DR_C * GR_LDA;  // c, beta, beta e^c, beta e^{c_C - c} of the value head, c's low part
  float* red = vc + 5 * DR_C;        // [16]
  float* part = red + 16;            // [2][4][64] partial sums of w and E.Z
  float* tfs = part + 8 * DR_C;      // the token factors (TF_*)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rg = warp >> 1, ch = warp & 1;  // this warp's 16 token rows and half of the columns
  const int ci = blockIdx.x, hq = blockIdx.y, rep = a.hv / a.hk, n16 = (a.dv + 15) / 16;
  pdl_wait();
  const DrChunk cu = a.chunks[ci];
  if (cu.len < 0) return;
  const int ntiles = (a.dv + GR_V - 1) / GR_V;

  // tile q (value head q / ntiles, channels 32 (q % ntiles)..) into stage q % 2, zero past dv, dk and the tokens
  auto load_tile = [&](int q) {
    const int h = hq * rep + q / ntiles, d0 = q % ntiles * GR_V;
    const int64_t row0 = ((int64_t)ci * a.hv + h) * a.dv + d0;
    const uint32_t st = smem_u32(smem + (q & 1) * STAGE);
    const int rows = a.dv - d0;
#pragma unroll
    for (int i = tid; i < GR_V * (DK / 4); i += 256) {
      const int r = i / (DK / 4), c = i % (DK / 4) * 4;
      const bool live = r < rows && c < a.dk;
      const int64_t at = live ? (row0 + r) * a.dk + c : 0;
      cp_async16(st + (r * LDS + c) * 4, a.keep_s + at, live);
      cp_async16(st + ((GR_V + r) * LDS + c) * 4, a.keep_ds + at, live);
    }
    const uint32_t et = st + 2 * GR_V * LDS * 4, zt = et + GR_V * GR_LDT * 4, ot = zt + GR_V * GR_LDT * 4;
#pragma unroll
    for (int i = tid; i < GR_V * 16; i += 256) {
      const int r = i >> 4, c = i & 15;
      const bool live = r < rows;
      const int64_t at = live ? (row0 + r) * DR_C : 0;
      // (the pairs of a kept E row are permuted in fours of tokens: 16-byte pieces stay whole)
      cp_async16(et + (r * GR_LDT + c * 4) * 4, a.keep_e + at + (live ? (c ^ (((d0 + r) & 7) << 1)) * 4 : 0), live);
      cp_async16(zt + (r * GR_LDT + c * 4) * 4, a.keep_z + at + (live ? c * 4 : 0), live);
    }
    {
      const int r = tid >> 2, c = (tid & 3) * 8;
      const bool live = r < cu.len && c < rows;
      const __nv_bfloat16* src = live ? a.dO + (int64_t)(cu.tok + r) * a.ldo + (int64_t)h * a.dv + d0 + c : a.dO;
      cp_async16(ot + (r * GR_LDO + c) * 2, src, live);
    }
    cp_commit();
  };

  float q[NH][4], k[NH][4];  // dQ~ and dK~, rows 16 rg + {g, g + 8}, columns ch DK/2 + 8 n + {2t, 2t + 1}
#pragma unroll
  for (int n = 0; n < NH; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) q[n][j] = k[n][j] = 0.f;
  const int r0 = rg * 16 + g;

  load_tile(0);
  float tf_in[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (tid + i * 256 < TF_N * DR_C) tf_in[i] = a.tok[((int64_t)ci * a.hk + hq) * TF_N * DR_C + tid + i * 256];
#pragma unroll 1
  for (int hr = 0; hr < rep; ++hr) {
    const int h = hq * rep + hr;
    const int64_t blk = (int64_t)ci * a.hv + h;
    const float* vec = reinterpret_cast<const float*>(a.blk + blk * DR_BLK + DR_VEC);
    // the gates' sums of the two passes (a quarter of the channel slices to each 64 threads) and the head's vectors:
    // every load is issued before the first is waited for
    const int tok = tid & (DR_C - 1), grp = tid >> 6;
    float w4[4], b4[4], x_sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = grp + 4 * i;
      w4[i] = p < n16 ? a.w_part[(blk * n16 + p) * DR_C + tok] : 0.f;
      b4[i] = p < n16 ? a.b_part[(blk * n16 + p) * DR_C + tok] : 0.f;
    }
    if (lane < n16) x_sum = a.x_part[blk * n16 + lane];
    const float c_in = vec[DV_C * DR_C + tok], c_lo = vec[DV_CLO * DR_C + tok], be = vec[DV_BETA * DR_C + tok];
    const float G = vec[DV_C * DR_C + DR_C - 1], G_lo = vec[DV_CLO * DR_C + DR_C - 1];
    float w = (w4[0] + w4[1]) + (w4[2] + w4[3]), b = (b4[0] + b4[1]) + (b4[2] + b4[3]);
    for (int p = grp + 16; p < n16; p += 4) {
      w += a.w_part[(blk * n16 + p) * DR_C + tok];
      b += a.b_part[(blk * n16 + p) * DR_C + tok];
    }
    for (int p = lane + 32; p < n16; p += 32) x_sum += a.x_part[blk * n16 + p];
#pragma unroll
    for (int o = 16; o; o >>= 1) x_sum += __shfl_xor_sync(0xffffffffu, x_sum, o);
    part[grp * DR_C + tok] = w;
    part[(4 + grp) * DR_C + tok] = b;
    if (tid < DR_C) {
      vc[tid] = c_in;
      vc[DR_C + tid] = be;
      vc[2 * DR_C + tid] = be * expf(c_in);
      vc[3 * DR_C + tid] = be * expf((G - c_in) + (G_lo - c_lo));
      vc[4 * DR_C + tid] = c_lo;
    }
    if (hr == 0)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (tid + i * 256 < TF_N * DR_C) tfs[tid + i * 256] = tf_in[i];
    float f[4][4], wm[4][4], sd = 0.f;  // F, W; this thread's part of <S, dS'>
    uint32_t s_bits = 0;                // ... and what is set in its part of S
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) f[n][j] = wm[n][j] = 0.f;
    __syncthreads();
    const float bc0 = -vc[2 * DR_C + r0], bc1 = -vc[2 * DR_C + r0 + 8];
    const float bl0 = vc[3 * DR_C + r0], bl1 = vc[3 * DR_C + r0 + 8];
    const float ec0 = expf(vc[r0]), ec1 = expf(vc[r0 + 8]);

#pragma unroll 1
    for (int tile = 0; tile < ntiles; ++tile) {
      const int at = hr * ntiles + tile;
      // (after a head's last tile K~ and Q~ take the stages' place, so the next head's first tile waits for them)
      if (tile + 1 < ntiles) {
        load_tile(at + 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      __syncthreads();
      const float* Sm = reinterpret_cast<const float*>(smem + (at & 1) * STAGE);
      const float *Dm = Sm + GR_V * LDS, *Em = Dm + GR_V * LDS, *Zm = Em + GR_V * GR_LDT;
      const __nv_bfloat16* Om = reinterpret_cast<const __nv_bfloat16*>(Zm + GR_V * GR_LDT);
#pragma unroll
      for (int i = tid; i < GR_V * (DK / 4); i += 256) {
        const int o = i / (DK / 4) * LDS + i % (DK / 4) * 4;
        const float4 x = *reinterpret_cast<const float4*>(Sm + o), y = *reinterpret_cast<const float4*>(Dm + o);
        sd += (x.x * y.x + x.y * y.y) + (x.z * y.z + x.w * y.w);
        s_bits |= __float_as_uint(x.x) | __float_as_uint(x.y) | __float_as_uint(x.z) | __float_as_uint(x.w);
      }
#pragma unroll
      for (int kk = 0; kk < GR_V; kk += 8) {
        const float o0 = __bfloat162float(Om[r0 * GR_LDO + kk + t]), o1 = __bfloat162float(Om[(r0 + 8) * GR_LDO + kk + t]);
        const float o2 = __bfloat162float(Om[r0 * GR_LDO + kk + t + 4]),
                    o3 = __bfloat162float(Om[(r0 + 8) * GR_LDO + kk + t + 4]);
        const float z0 = Zm[(kk + t) * GR_LDT + r0], z1 = Zm[(kk + t) * GR_LDT + r0 + 8];
        const float z2 = Zm[(kk + t + 4) * GR_LDT + r0], z3 = Zm[(kk + t + 4) * GR_LDT + r0 + 8];
        const float u0 = Em[(kk + t) * GR_LDT + r0], u1 = Em[(kk + t) * GR_LDT + r0 + 8];
        const float u2 = Em[(kk + t + 4) * GR_LDT + r0], u3 = Em[(kk + t + 4) * GR_LDT + r0 + 8];
        uint32_t h0, h1, l0, l1;
        if (ch * 32 <= rg * 16 + 15) {
          const uint32_t oa[4] = {__float_as_uint(o0), __float_as_uint(o1), __float_as_uint(o2), __float_as_uint(o3)};
          uint32_t zh[4], zl[4];
          split_tf32(z0, z1, z2, z3, zh, zl);
#pragma unroll
          for (int n = 0; n < 4; ++n) {  // F, W: columns j = 32 ch + 8 n + g
            const int j = ch * 32 + n * 8 + g;
            split_tf32(Em[(kk + t) * GR_LDT + j], h0, l0);
            split_tf32(Em[(kk + t + 4) * GR_LDT + j], h1, l1);
            mma_tf32(f[n], oa, l0, l1);  // (dO is exact)
            mma_tf32x3(wm[n], zh, zl, h0, h1, l0, l1);
            mma_tf32(f[n], oa, h0, h1);
          }
        }
        uint32_t oh[4], ol[4], zh[4], zl[4], uh[4], ul[4];
        split_tf32(o0 * ec0, o1 * ec1, o2 * ec0, o3 * ec1, oh, ol);
        split_tf32(z0 * bc0, z1 * bc1, z2 * bc0, z3 * bc1, zh, zl);
        split_tf32(u0 * bl0, u1 * bl1, u2 * bl0, u3 * bl1, uh, ul);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const int c = ch * (DK / 2) + n * 8 + g;
          split_tf32(Sm[(kk + t) * LDS + c], h0, l0);
          split_tf32(Sm[(kk + t + 4) * LDS + c], h1, l1);
          mma_tf32x3(q[n], oh, ol, h0, h1, l0, l1);
          mma_tf32x3(k[n], zh, zl, h0, h1, l0, l1);
          split_tf32(Dm[(kk + t) * LDS + c], h0, l0);
          split_tf32(Dm[(kk + t + 4) * LDS + c], h1, l1);
          mma_tf32x3(k[n], uh, ul, h0, h1, l0, l1);
        }
      }
      __syncthreads();  // the stage is read
    }
    // F and -W with their decays, gates and masks
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int j = ch * 32 + n * 8 + 2 * t;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = r0 + (p >> 1) * 8, jj = j + (p & 1);
        const float d =
            jj <= i ? expf((vc[i] - vc[jj]) + (vc[4 * DR_C + i] - vc[4 * DR_C + jj])) * vc[DR_C + jj] : 0.f;
        Fm[i * GR_LDA + jj] = jj <= i ? d * f[n][p] : 0.f;
        Wm[i * GR_LDA + jj] = jj < i ? -d * vc[DR_C + i] * wm[n][p] : 0.f;
      }
    }
    // K16, Q16 (exact; their rows' factors go to the other operand)
    const uint8_t* kq = a.kq + ((int64_t)ci * a.hk + hq) * (2 * DR_C * DK * 2);
    {
      uint4 raw[DK / 16];  // 2 x 64 rows of DK / 8 pieces, all in flight
#pragma unroll
      for (int n = 0; n < DK / 16; ++n) raw[n] = __ldg(reinterpret_cast<const uint4*>(kq) + tid + n * 256);
#pragma unroll
      for (int n = 0; n < DK / 16; ++n) {
        const int i = tid + n * 256, isq = n >= DK / 32;  // pieces as they lie: swizzled within the row
        const int r = i / (DK / 8) - isq * DR_C, c = (i % (DK / 8)) ^ (r & 7);
        float* dst = (isq ? Qm : Km) + r * LDS + c * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<float2*>(dst + 2 * j) = unpack_f16x2((&raw[n].x)[j]);
        }
      }
    }
    // <S, dS'> of the block, for the gates: dg_t = <S', dS'> + sum_{i >= t} w_i (from the tokens where it is zero, if
    // there are such), dbeta = E.Z
#pragma unroll
    for (int m = 16; m; m >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, m);
    if (lane == 0) red[warp] = sd;
    float w_sum = 0.f, b_sum = 0.f;
    if (tid < DR_C) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w_sum += part[i * DR_C + tid];
        b_sum += part[(4 + i) * DR_C + tid];
      }
    }
    float sum = w_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (tid < DR_C) {
      part[tid] = sum - w_sum;  // (of the warp's tokens before this one; this thread has read its sums there)
      const float step = tid ? (vc[tid] - vc[tid - 1]) + (vc[4 * DR_C + tid] - vc[4 * DR_C + tid - 1]) : vc[0];
      const uint32_t resets = __ballot_sync(0xffffffffu, expf(step) == 0.f);
      if (lane == 31) red[8 + warp] = sum;
      if (lane == 0) red[10 + warp] = __uint_as_float(resets);
    }
    const bool zero_state = !__syncthreads_or((s_bits << 1) != 0);
    if (tid < cu.len) {
      const float half = red[8];
      auto before = [&](int t) { return part[t] + (t >= 32 ? half : 0.f); };
      const unsigned long long zeros = __float_as_uint(red[10]) |
                                       (unsigned long long)__float_as_uint(red[11]) << 32 | (zero_state ? 1ull : 0ull);
      const unsigned long long upto = zeros & (~0ull >> (DR_C - 1 - tid));
      float dg;
      if (upto) {
        dg = before(DR_C - 1 - __clzll(upto)) - before(tid);
      } else if (zeros) {
        dg = before(__ffsll(zeros) - 1) - before(tid);
      } else {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) d += red[i];
        dg = expf(vc[DR_C - 1]) * d + x_sum + ((half + red[9]) - before(tid));
      }
      const int64_t at = (int64_t)(cu.tok + tid) * a.hv + h;
      a.dg[at] = dg;
      a.dbeta[at] = b_sum;
    }
    // dQ~ += F K~, dK~ += F^T Q~ - W K~ - W^T K~ with K~_j = f_k(j) K16_j, Q~_j = f_q(j) Q16_j
    auto bits = [](float x) { return __float_as_uint(x); };
    auto mma2 = [](float (&c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint32_t b0, uint32_t b1) {
      mma_tf32(c, lo, b0, b1);
      mma_tf32(c, hi, b0, b1);
    };
#pragma unroll 2
    for (int kk = 0; kk < DR_C; kk += 8) {
      const bool lower = kk <= rg * 16 + 15, upper = kk + 7 >= rg * 16;  // tiles of F, W and of their transposes
      uint32_t fa[4], wa[4], ft[4], wt[4], fal[4], wal[4], ftl[4], wtl[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = r0 + (p & 1) * 8, j = kk + t + (p >> 1) * 4;
        const float fk = tfs[TF_FK * DR_C + j], fq = tfs[TF_FQ * DR_C + j];
        split_tf32(Fm[i * GR_LDA + j] * fk, fa[p], fal[p]);
        split_tf32(Wm[i * GR_LDA + j] * fk, wa[p], wal[p]);
        split_tf32(Fm[j * GR_LDA + i] * fq, ft[p], ftl[p]);
        split_tf32(Wm[j * GR_LDA + i] * fk, wt[p], wtl[p]);
      }
      const float *k0 = Km + (kk + t) * LDS + ch * (DK / 2) + g, *q0 = Qm + (kk + t) * LDS + ch * (DK / 2) + g;
      if (lower) {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const uint32_t b0 = bits(k0[n * 8]), b1 = bits(k0[n * 8 + 4 * LDS]);
          mma2(q[n], fa, fal, b0, b1);
          mma2(k[n], wa, wal, b0, b1);
        }
      }
      if (upper) {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          mma2(k[n], wt, wtl, bits(k0[n * 8]), bits(k0[n * 8 + 4 * LDS]));
          mma2(k[n], ft, ftl, bits(q0[n * 8]), bits(q0[n * 8 + 4 * LDS]));
        }
      }
    }
    __syncthreads();  // shared memory is free for the next value head
    if (hr + 1 < rep) load_tile((hr + 1) * ntiles);
  }

  // back through the norms: dk = h_k (dk~ - p_k K16 (K16 . dk~)) (p_k = 0 where nothing is normalised), the dot
  // over both column halves; the rows leave through shared memory, 16 bytes a store
  float* dots = part;  // [2 halves][2][64]
  __nv_bfloat16* rows = reinterpret_cast<__nv_bfloat16*>(Fm);
  constexpr int LDR = DK + 8;
#pragma unroll
  for (int isq = 0; isq < 2; ++isq)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = r0 + 8 * p;
      const float* x = (isq ? Qm : Km) + row * LDS + ch * (DK / 2) + 2 * t;
      float s = 0.f;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        const float2 y = *reinterpret_cast<const float2*>(x + n * 8);
        s += y.x * (isq ? q[n][2 * p] : k[n][2 * p]) + y.y * (isq ? q[n][2 * p + 1] : k[n][2 * p + 1]);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (t == 0) dots[(ch * 2 + isq) * DR_C + row] = s;
    }
  __syncthreads();
#pragma unroll
  for (int isq = 0; isq < 2; ++isq) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = r0 + 8 * p;
      const float hs = tfs[(isq ? TF_HQ : TF_HK) * DR_C + row];
      const float dot = (dots[isq * DR_C + row] + dots[(2 + isq) * DR_C + row]) * tfs[(isq ? TF_PQ : TF_PK) * DR_C + row];
      const float* x = (isq ? Qm : Km) + row * LDS + ch * (DK / 2) + 2 * t;
      __nv_bfloat16* out = rows + row * LDR + ch * (DK / 2) + 2 * t;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        const float2 y = *reinterpret_cast<const float2*>(x + n * 8);
        *reinterpret_cast<uint32_t*>(out + n * 8) = pack_bf16x2(hs * ((isq ? q[n][2 * p] : k[n][2 * p]) - y.x * dot),
                                                                hs * ((isq ? q[n][2 * p + 1] : k[n][2 * p + 1]) - y.y * dot));
      }
    }
    __syncthreads();
    __nv_bfloat16* out = (isq ? a.dQ + (int64_t)cu.tok * a.ldq : a.dK + (int64_t)cu.tok * a.ldk) + (int64_t)hq * a.dk;
    const int64_t ld = isq ? a.ldq : a.ldk;
#pragma unroll
    for (int i = tid; i < DR_C * (DK / 8); i += 256) {
      const int r = i / (DK / 8), c = i % (DK / 8) * 8;
      if (r < cu.len && c < a.dk)
        *reinterpret_cast<uint4*>(out + r * ld + c) = *reinterpret_cast<const uint4*>(rows + r * LDR + c);
    }
    if (!isq) __syncthreads();
  }
}

}  // namespace ttt
