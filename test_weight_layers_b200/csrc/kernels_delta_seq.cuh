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

// A token as a warp needs it: lane l the columns VEC (32 i + l) + 0..VEC-1 of k and q, lane r < ROWS the value of
// row r, and the scalars that do not depend on the state.
template <int E>
struct Token {
  float k[E], q[E], v, beta, g;  // as loaded
  float fk, fq, kq, al;          // norms' factors, k . q, exp(g)
};

// A warp holds ROWS rows of S (value channels), lane l the columns VEC (32 i + l) + 0..VEC-1 of each; a token
// costs one pass over the registers and one warp reduction: of S k and S q per row, and of k.k, q.q, k.q.
//   Decoding step (SEQ = false): bound by the state's bytes, read and written once: 89 us, 5.6 TB/s
// for 235 rows of 16 heads of 128 x 128.
//   Sequences (SEQ): bound by the chain reduction -> update; the next token's norms are reduced beside this
// token's products and the one after it is being loaded: 0.37 us a token of
// 64 x 64 (two rows to a warp).
template <typename T, int VEC, int NV, int ROWS, bool SEQ>
__global__ void __launch_bounds__(128) k_delta_tokens(const SeqArgs<T> a) {
  __shared__ int next_row;
  constexpr int E = NV * VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, hq = h / (a.hv / a.hk);
  const int r0 = (blockIdx.z * 4 + warp) * ROWS;
  int64_t tok = blockIdx.x, state = blockIdx.x;
  int len = 1;
  if constexpr (SEQ) {
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
  float s[ROWS][E];
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
  auto load = [&](Token<E>& x, int64_t tok) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = VEC * (32 * i + lane);
      if (col < a.dk) {
        load_vec<VEC>(a.K + tok * a.ldk + (int64_t)hq * a.dk + col, &x.k[i * VEC]);
        load_vec<VEC>(a.Q + tok * a.ldq + (int64_t)hq * a.dk + col, &x.q[i * VEC]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.k[i * VEC + j] = x.q[i * VEC + j] = 0.f;
      }
    }
    x.beta = a.beta[tok * a.hv + h];
    x.g = a.g[tok * a.hv + h];
    x.v = 0.f;
    if (SEQ && lane < ROWS && r0 + lane < a.dv) x.v = load_one(a.V + tok * a.ldv + (int64_t)h * a.dv + r0 + lane);
  };
  auto dots = [&](const Token<E>& x, float* p) {  // k.k, q.q, k.q of this lane's columns
    p[0] = p[1] = p[2] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      p[0] += x.k[i] * x.k[i];
      p[1] += x.q[i] * x.q[i];
      p[2] += x.k[i] * x.q[i];
    }
  };
  auto factors = [&](Token<E>& x, const float* p) {
    x.fk = x.fq = 1.f;
    if (a.l2norm) {
      x.fk = fminf(rsqrtf(p[0]), 1e12f);  // 1 / max(||k||, 1e-12)
      x.fq = fminf(rsqrtf(p[1]), 1e12f);
    }
    x.fq *= a.scale;
    // a row whose norm overflows has a factor of zero and counts as zero: its products may have overflowed too
    x.kq = x.fk == 0.f || x.fq == 0.f ? 0.f : p[2];
    x.al = expf(x.g);
  };
  auto products = [&](const Token<E>& x, float* p) {  // S k and S q of this lane's columns
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      p[2 * r] = p[2 * r + 1] = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        p[2 * r] += s[r][i] * x.k[i];
        p[2 * r + 1] += s[r][i] * x.q[i];
      }
    }
  };
  constexpr int NP = 2 * ROWS + 3;
  float p[NP];
  if constexpr (SEQ) {
    // The 2 ROWS + 3 sums (padded to 8) over the warp by halving: a lane whose bit is set keeps the upper half of
    // the values and sends the lower, so 8 sums take 9 shuffles; then each is read from its lane by all.
    static_assert(ROWS == 2, "eight sums");
    auto reduce = [&] {
      float v[8];
#pragma unroll
      for (int i = 0; i < 7; ++i) v[i] = p[i];
      v[7] = 0.f;
#pragma unroll
      for (int half = 4; half; half >>= 1) {
        const bool upper = lane & (half * 4);
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, half * 4);
        }
      }
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
#pragma unroll
      for (int i = 0; i < 7; ++i) p[i] = __shfl_sync(0xffffffffu, v[0], i * 4);
    };
    // running pointers of the token to load next
    const T *pk = a.K + tok * a.ldk + (int64_t)hq * a.dk, *pq = a.Q + tok * a.ldq + (int64_t)hq * a.dk;
    const T* pv = a.V + tok * a.ldv + (int64_t)h * a.dv + r0 + lane;
    const float *pb = a.beta + tok * a.hv + h, *pg = a.g + tok * a.hv + h;
    T* po = a.O + tok * a.ldo + (int64_t)h * a.dv + r0 + lane;
    const bool own = lane < ROWS && r0 + lane < a.dv;
    int left = len;  // tokens from the pointers on
    auto load_next = [&](Token<E>& x) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = VEC * (32 * i + lane);
        if (col < a.dk) {
          load_vec<VEC>(pk + col, &x.k[i * VEC]);
          load_vec<VEC>(pq + col, &x.q[i * VEC]);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) x.k[i * VEC + j] = x.q[i * VEC + j] = 0.f;
        }
      }
      x.beta = *pb;
      x.g = *pg;
      x.v = own ? load_one(pv) : 0.f;
      if (--left > 0) pk += a.ldk, pq += a.ldq, pv += a.ldv, pb += a.hv, pg += a.hv;  // (else: the last one again)
    };
    Token<E> x, y;
    if (len > 0) {
      load_next(x);
      load_next(y);
#pragma unroll
      for (int i = 0; i < 2 * ROWS; ++i) p[i] = 0.f;
      dots(x, p + 2 * ROWS);
      reduce();
      factors(x, p + 2 * ROWS);
    }
#pragma unroll 3
    for (int n = 0; n < len; ++n) {  // (unrolled so that the three tokens change names, not registers)
      Token<E> z;
      load_next(z);
      products(x, p);
      dots(y, p + 2 * ROWS);
      reduce();
      float out = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float sk = x.fk == 0.f ? 0.f : p[2 * r] * x.fk;
        const float u = x.beta * (__shfl_sync(0xffffffffu, x.v, r) - x.al * sk);
        const float uk = u * x.fk;
        if (lane == r) out = x.fq == 0.f ? 0.f : x.fq * (x.al * p[2 * r + 1] + uk * x.kq);
#pragma unroll
        for (int i = 0; i < E; ++i) s[r][i] = x.al * s[r][i] + uk * x.k[i];
      }
      if (own) store_one(po, out);
      po += a.ldo;
      factors(y, p + 2 * ROWS);
      x = y;
      y = z;
    }
  } else {
    // rows of one slot run in row order in the block of the first of them
    if (a.slots) {
      bool earlier = false;
      for (int b = threadIdx.x; b < (int)blockIdx.x; b += 128) earlier |= a.slots[b] == (int)state;
      if (__syncthreads_or(earlier)) return;
    }
    // The 2 ROWS sums over the warp with the values halved at each step: the lanes whose bit is set keep the upper
    // half and send the lower, so that 16 sums take 16 shuffles instead of 80.  Then lane l has sum l / LPI, and the
    // 2 LPI lanes of a row do its scalar part.
    constexpr int M = 2 * ROWS, LPI = 32 / M;
    const int mine = lane / (2 * LPI);
    for (;;) {
      Token<E> x;
      load(x, tok);
      const float v = r0 + mine < a.dv ? load_one(a.V + tok * a.ldv + (int64_t)h * a.dv + r0 + mine) : 0.f;
      products(x, p);
      dots(x, p + M);
#pragma unroll
      for (int half = ROWS; half; half >>= 1) {
        const int o = half * LPI;
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float send = upper ? p[i] : p[i + half], keep = upper ? p[i + half] : p[i];
          p[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
#pragma unroll
      for (int o = LPI / 2; o; o >>= 1) p[0] += __shfl_xor_sync(0xffffffffu, p[0], o);
#pragma unroll
      for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) p[M + i] += __shfl_xor_sync(0xffffffffu, p[M + i], o);
      factors(x, p + M);
      const float other = __shfl_xor_sync(0xffffffffu, p[0], LPI);
      const float sk = lane & LPI ? other : p[0], sq = lane & LPI ? p[0] : other;
      const float uk = x.beta * (v - x.al * (x.fk == 0.f ? 0.f : sk * x.fk)) * x.fk;
      if (lane % (2 * LPI) == 0 && r0 + mine < a.dv)
        store_one(a.O + tok * a.ldo + (int64_t)h * a.dv + r0 + mine,
                  x.fq == 0.f ? 0.f : x.fq * (x.al * sq + uk * x.kq));
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float ur = __shfl_sync(0xffffffffu, uk, r * 2 * LPI);
#pragma unroll
        for (int i = 0; i < E; ++i) s[r][i] = x.al * s[r][i] + ur * x.k[i];
      }
      if (!a.slots) break;
      if (threadIdx.x == 0) next_row = INT32_MAX;
      __syncthreads();
      for (int b = (int)tok + 1 + (int)threadIdx.x; b < a.rows; b += 128)
        if (a.slots[b] == (int)state) atomicMin(&next_row, b);
      __syncthreads();
      tok = next_row;
      __syncthreads();
      if (tok == INT32_MAX) break;
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
