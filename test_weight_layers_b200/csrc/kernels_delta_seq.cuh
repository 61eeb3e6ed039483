// Gated delta rule, token by token: decoding steps over a pool of states
// (both dtypes) and whole sequences in fp32.
#pragma once

#include "delta_common.cuh"

namespace ttt {

// VEC contiguous elements as floats
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float* x) {
  if constexpr (VEC == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float* x) {
  uint32_t w[VEC / 2];
  if constexpr (VEC == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  else w[0] = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float* x) {
  if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <typename T>
struct SeqArgs {
  const T *Q, *K, *V;
  T* O;
  int64_t ldq, ldk, ldv, ldo;
  const float *g, *beta;
  const float* S0;  // null: zeros
  float* S;         // null: not wanted
  int hk, hv, dk, dv, l2norm;
  float scale;
  const DrSeq* seqs;  // sequences (null: decoding step)
  const int* slots;   // decoding step: place of each row's state (null: the row itself)
  int n_slots, rows;  // decoding step
};

// A warp holds ROWS rows of S (value channels), lane l the columns VEC (32 i + l) + 0..VEC-1
// of each; a token costs one pass over the registers and one warp reduction of 2 ROWS + 3 sums.
// Bound by the state's bytes in a decoding step (read and written once), by the
// reduction's latency over a sequence.
template <typename T, int VEC, int NV, int ROWS>
__global__ void __launch_bounds__(128) k_delta_tokens(const SeqArgs<T> a) {
  __shared__ int next_row;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, hq = h / (a.hv / a.hk);
  const int r0 = (blockIdx.z * 4 + warp) * ROWS;
  int64_t tok = blockIdx.x, state = blockIdx.x;
  int len = 1;
  if (a.seqs) {
    pdl_wait();
    const DrSeq sq = a.seqs[blockIdx.x];
    if (sq.len < 0) return;
    tok = sq.tok;
    len = sq.len;
    state = sq.id;
  } else if (a.slots) {
    state = a.slots[blockIdx.x];
    if (state < 0 || state >= a.n_slots) return;
  }
  float s[ROWS][NV * VEC];
  const int64_t srow = (state * a.hv + h) * a.dv;
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = VEC * (32 * i + lane);
      if (a.S0 && r0 + r < a.dv && col < a.dk) {
        load_vec<VEC>(a.S0 + (srow + r0 + r) * a.dk + col, &s[r][i * VEC]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[r][i * VEC + j] = 0.f;
      }
    }
  // rows of one slot run in row order in the block of the first of them
  auto next_same = [&](int after) {
    if (threadIdx.x == 0) next_row = INT32_MAX;
    __syncthreads();
    for (int b = after + 1 + (int)threadIdx.x; b < a.rows; b += 128)
      if (a.slots[b] == (int)state) atomicMin(&next_row, b);
    __syncthreads();
    const int n = next_row;
    __syncthreads();
    return n;
  };
  if (!a.seqs && a.slots) {
    bool earlier = false;
    for (int b = threadIdx.x; b < (int)blockIdx.x; b += 128) earlier |= a.slots[b] == (int)state;
    if (__syncthreads_or(earlier)) return;
  }

#pragma unroll 1
  for (int n = 0; n < len;) {
    float k[NV * VEC], q[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = VEC * (32 * i + lane);
      if (col < a.dk) {
        load_vec<VEC>(a.K + tok * a.ldk + (int64_t)hq * a.dk + col, &k[i * VEC]);
        load_vec<VEC>(a.Q + tok * a.ldq + (int64_t)hq * a.dk + col, &q[i * VEC]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) k[i * VEC + j] = q[i * VEC + j] = 0.f;
      }
    }
    const float be = a.beta[tok * a.hv + h], al = expf(a.g[tok * a.hv + h]);
    float v = 0.f;
    if (lane < ROWS && r0 + lane < a.dv) v = load_one(a.V + tok * a.ldv + (int64_t)h * a.dv + r0 + lane);
    float p[2 * ROWS + 3];
#pragma unroll
    for (int j = 0; j < 2 * ROWS + 3; ++j) p[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
      p[2 * ROWS] += k[i] * k[i];
      p[2 * ROWS + 1] += q[i] * q[i];
      p[2 * ROWS + 2] += k[i] * q[i];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        p[2 * r] += s[r][i] * k[i];
        p[2 * r + 1] += s[r][i] * q[i];
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int j = 0; j < 2 * ROWS + 3; ++j) p[j] += __shfl_xor_sync(0xffffffffu, p[j], o);
    float fk = 1.f, fq = 1.f;
    if (a.l2norm) {
      fk = 1.f / fmaxf(sqrtf(p[2 * ROWS]), 1e-12f);
      fq = 1.f / fmaxf(sqrtf(p[2 * ROWS + 1]), 1e-12f);
    }
    fq *= a.scale;
    float out = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float u = be * (__shfl_sync(0xffffffffu, v, r) - al * (p[2 * r] * fk));
      const float uk = u * fk;
      const float o = fq * (al * p[2 * r + 1] + uk * p[2 * ROWS + 2]);
      if (lane == r) out = o;
#pragma unroll
      for (int i = 0; i < NV * VEC; ++i) s[r][i] = al * s[r][i] + uk * k[i];
    }
    if (lane < ROWS && r0 + lane < a.dv) store_one(a.O + tok * a.ldo + (int64_t)h * a.dv + r0 + lane, out);
    if (a.seqs) {
      ++n;
      ++tok;
    } else {
      const int nx = a.slots ? next_same((int)tok) : INT32_MAX;
      if (nx == INT32_MAX) break;
      tok = nx;
    }
  }
  if (a.S) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = VEC * (32 * i + lane);
        if (r0 + r < a.dv && col < a.dk) store_vec<VEC>(a.S + (srow + r0 + r) * a.dk + col, &s[r][i * VEC]);
      }
  }
}

}  // namespace ttt
