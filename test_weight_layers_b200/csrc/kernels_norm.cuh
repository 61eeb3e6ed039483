// Block norms: the norm after a block with its gate and residual scale, the
// residual sum and the norm before the next block in one pass, and its gradient.
//
// Per row of D columns (r_y over D, or over each group of `group` columns):
//     p = y r_y w_post s(z),  r_y = 1 / sqrt(mean(y^2) + eps),  s = SiLU
//     x' = x + lambda p,      n = x' r w_pre,  r = 1 / sqrt(mean(x'^2) + eps)
// Gradient, from dx' and dn (t = dn w_pre, everything recomputed from y, x, z):
//     D_x' = dx' + r (t - x' r^2 mean(t x'));   dx = D_x';   dp = lambda D_x'
//     dz = dp y r_y w_post s'(z);   u = dp w_post s;   dy = r_y (u - y r_y mean(u y r_y))
//     dw_pre = sum dn x' r;  dlambda = sum D_x' p;  dw_post = sum dp y r_y s
// The row stays in registers between its reductions, so each tensor crosses
// HBM once: the kernels are bound by those bytes.  All arithmetic is fp32, rounded
// once on the way out.
#pragma once

#include "common.cuh"

namespace ttt {

template <typename T>
struct NormArgs {
  const T *X, *Y, *Z, *dXo, *dN;
  T *Xo, *N, *dX, *dY, *dZ;
  int64_t ldx, ldy, ldz, ldxo, ldn;
  const float *w_post, *lam, *w_pre;
  int64_t rows;   // rows of the kernel: rows of the call times `split`
  int split;      // groups taken as rows of their own (no second norm, no lambda), else 1
  int D;          // columns of a kernel row
  int group;      // columns per mean of y
  float eps;
  int vec;        // rows are 16-byte aligned and D a multiple of 8
  int norm2;      // second norm present
  float* part;    // backward: [blocks][3][D] column sums of (w_post, lambda, w_pre)
};

// Raw registers of 8 consecutive elements.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
};
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = (&r.q[0].x)[j];
    x[2 * j] = __uint_as_float(w << 16);
    x[2 * j + 1] = __uint_as_float(w & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __uint_as_float((&r.q[j >> 2].x)[j & 3]);
}
__device__ __forceinline__ Raw8<__nv_bfloat16> pack8(const float (&x)[8], __nv_bfloat16) {
  Raw8<__nv_bfloat16> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) (&r.q[0].x)[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
  return r;
}
__device__ __forceinline__ Raw8<float> pack8(const float (&x)[8], float) {
  Raw8<float> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) (&r.q[j >> 2].x)[j & 3] = __float_as_uint(x[j]);
  return r;
}

// Columns [col, col + 8) of a row, zero past D.  Plain loads: an output may be one of the inputs.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int col, int D, int vec) {
  Raw8<T> r;
  if (vec) {
#pragma unroll
    for (int j = 0; j < (int)(sizeof(T) / 2); ++j)
      r.q[j] = col < D ? reinterpret_cast<const uint4*>(p + col)[j] : make_uint4(0, 0, 0, 0);
  } else {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = col + j < D ? (float)p[col + j] : 0.f;
    r = pack8(x, T());
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int col, int D, int vec, const float (&x)[8]) {
  const Raw8<T> r = pack8(x, T());
  if (vec) {
    if (col < D)
#pragma unroll
      for (int j = 0; j < (int)(sizeof(T) / 2); ++j) reinterpret_cast<uint4*>(p + col)[j] = r.q[j];
  } else {
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < D) p[col + j] = e[j];
  }
}
// 8 weights from column `col` of a vector of `n` (ones where there is none, zero past n)
__device__ __forceinline__ void weight8(const float* w, int col, int n, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
  } else if (col + 8 <= n && (reinterpret_cast<uintptr_t>(w + col) & 15u) == 0) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + col));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + col + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = col + j < n ? __ldg(w + col + j) : 0.f;
  }
}

// Sums over the TPR threads of a row (TPR = 32: a warp; else the whole block).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // the sums before are read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * W + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[i * W + w];
      v[i] = s;
    }
  }
}

// Per-chunk sums -> each chunk's group sum (group a multiple of 8).  `buf`: D / 8 floats of this row.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float (&v)[NV], int t, int D, int group, float* buf) {
  auto sync = [] {
    if constexpr (TPR > 32) __syncthreads();
    else __syncwarp();
  };
  sync();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TPR + t) * 8 < D) buf[i * TPR + t] = v[i];
  sync();
  const int n = group / 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * TPR + t;
    float s = 0.f;
    if (c * 8 < D) {
      const int g0 = c / n * n;
      for (int k = 0; k < n; ++k) s += buf[g0 + k];
    }
    v[i] = s;
  }
}

template <typename T>
__device__ __forceinline__ T* norm_row(T* p, int64_t row, int64_t ld, const NormArgs<std::remove_const_t<T>>& a) {
  if (!p) return nullptr;
  if (a.split == 1) return p + row * ld;
  return p + row / a.split * ld + row % a.split * a.D;
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// TPR threads to a row, NV chunks of 8 columns to a thread; GROUPS: several means of y to a row.
template <typename T, int TPR, int NV, bool GROUPS>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) k_block_norm(const NormArgs<T> a) {
  constexpr int BLOCK = TPR > 128 ? TPR : 128;
  constexpr int RPB = BLOCK / TPR;  // rows per block
  __shared__ float red[TPR / 32 + 1];
  extern __shared__ float gbuf[];
  const int t = threadIdx.x % TPR, rb = threadIdx.x / TPR;
  float* buf = gbuf + rb * ((a.D + 7) / 8);
  for (int64_t row = (int64_t)blockIdx.x * RPB + rb; row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const T *xr = norm_row(a.X, row, a.ldx, a), *yr = norm_row(a.Y, row, a.ldy, a), *zr = norm_row(a.Z, row, a.ldz, a);
    Raw8<T> y[NV], x[NV], z[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      y[i] = load8(yr, col, a.D, a.vec);
      if (zr) z[i] = load8(zr, col, a.D, a.vec);
      if (xr) x[i] = load8(xr, col, a.D, a.vec);
    }
    float sy[NV], s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
      unpack8(y[i], v);
      sy[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sy[i] += v[j] * v[j];
      s1[0] += sy[i];
    }
    if constexpr (GROUPS) group_sum<TPR>(sy, t, a.D, a.group, buf);
    else row_sum<TPR>(s1, red);
    float p[NV][8], s2[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      const float ry = rsqrtf((GROUPS ? sy[i] : s1[0]) / (float)a.group + a.eps);
      float w[8], l[8], v[8];
      unpack8(y[i], p[i]);
      weight8(a.w_post, GROUPS ? col % a.group : col, a.group, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) p[i][j] = p[i][j] * ry * w[j];
      if (zr) {
        unpack8(z[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= v[j] * sigmoid_f(v[j]);
      }
      if (a.lam) {
        weight8(a.lam, col, a.D, l);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= l[j];
      }
      if (xr) {
        unpack8(x[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] += v[j];
      }
      if (a.Xo) store8(norm_row(a.Xo, row, a.ldxo, a), col, a.D, a.vec, p[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s2[0] += p[i][j] * p[i][j];
    }
    if (a.N) {
      row_sum<TPR>(s2, red);
      const float r = rsqrtf(s2[0] / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        float w[8];
        weight8(a.w_pre, col, a.D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= r * w[j];
        store8(norm_row(a.N, row, a.ldn, a), col, a.D, a.vec, p[i]);
      }
    }
  }
}

template <typename T, int TPR, int NV, bool GROUPS>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) k_block_norm_bwd(const NormArgs<T> a) {
  constexpr int BLOCK = TPR > 128 ? TPR : 128;
  constexpr int RPB = BLOCK / TPR;
  __shared__ float red[2 * (TPR / 32) + 1];
  extern __shared__ float gbuf[];
  const int t = threadIdx.x % TPR, rb = threadIdx.x / TPR;
  float* buf = gbuf + rb * ((a.D + 7) / 8);
  float c_post[NV][8], c_lam[NV][8], c_pre[NV][8];  // this thread's column sums
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) c_post[i][j] = c_lam[i][j] = c_pre[i][j] = 0.f;

  for (int64_t row = (int64_t)blockIdx.x * RPB + rb; row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const T *xr = norm_row(a.X, row, a.ldx, a), *yr = norm_row(a.Y, row, a.ldy, a), *zr = norm_row(a.Z, row, a.ldz, a);
    const T *gr = norm_row(a.dXo, row, a.ldxo, a), *nr = norm_row(a.dN, row, a.ldn, a);
    Raw8<T> y[NV], x[NV], z[NV], gx[NV], gn[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      y[i] = load8(yr, col, a.D, a.vec);
      if (zr) z[i] = load8(zr, col, a.D, a.vec);
      if (gr) gx[i] = load8(gr, col, a.D, a.vec);
      if (nr) {
        gn[i] = load8(nr, col, a.D, a.vec);
        if (xr) x[i] = load8(xr, col, a.D, a.vec);
      }
    }
    float sy[NV], s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
      unpack8(y[i], v);
      sy[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sy[i] += v[j] * v[j];
      s1[0] += sy[i];
    }
    if constexpr (GROUPS) group_sum<TPR>(sy, t, a.D, a.group, buf);
    else row_sum<TPR>(s1, red);
    // x' again, and the two sums of its norm
    float s2[2] = {0.f, 0.f};  // sum x'^2, sum t x'
    float r = 0.f, m = 0.f;
    if (nr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        const float ry = rsqrtf((GROUPS ? sy[i] : s1[0]) / (float)a.group + a.eps);
        float p[8], w[8], l[8], v[8];
        unpack8(y[i], p);
        weight8(a.w_post, GROUPS ? col % a.group : col, a.group, w);
        weight8(a.lam, col, a.D, l);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] *= ry * w[j] * l[j];
        if (zr) {
          unpack8(z[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] *= v[j] * sigmoid_f(v[j]);
        }
        if (xr) {
          unpack8(x[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] += v[j];
        }
        unpack8(gn[i], v);
        weight8(a.w_pre, col, a.D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s2[0] += p[j] * p[j];
          s2[1] += v[j] * w[j] * p[j];
        }
      }
      row_sum<TPR>(s2, red);
      r = rsqrtf(s2[0] / (float)a.D + a.eps);
      m = r * r * (s2[1] / (float)a.D);
    }
    // column sums, dx, dz and the sums of u y r_y
    float u[NV][8], su[NV], s3[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      const float ry = rsqrtf((GROUPS ? sy[i] : s1[0]) / (float)a.group + a.eps);
      float yh[8], w[8], l[8], zz[8], d[8], v[8];
      unpack8(y[i], yh);
      weight8(a.w_post, GROUPS ? col % a.group : col, a.group, w);
      weight8(a.lam, col, a.D, l);
      if (zr) unpack8(z[i], zz);
      if (gr) {
        unpack8(gx[i], d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.f;
      }
      float sg[8], sl[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        yh[j] *= ry;
        sg[j] = zr ? sigmoid_f(zz[j]) : 1.f;
        sl[j] = zr ? zz[j] * sg[j] : 1.f;
      }
      if (nr) {
        float wp[8], xv[8];
        unpack8(gn[i], v);
        weight8(a.w_pre, col, a.D, wp);
        if (xr) unpack8(x[i], xv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xo = (xr ? xv[j] : 0.f) + l[j] * (yh[j] * w[j] * sl[j]);
          c_pre[i][j] += v[j] * (xo * r);
          d[j] += r * (v[j] * wp[j] - xo * m);
        }
      }
      su[i] = 0.f;
      float dz[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c_lam[i][j] += d[j] * (yh[j] * w[j] * sl[j]);
        const float dp = d[j] * l[j];
        c_post[i][j] += dp * yh[j] * sl[j];
        if (zr) dz[j] = dp * yh[j] * w[j] * sg[j] * (1.f + zz[j] * (1.f - sg[j]));
        u[i][j] = dp * w[j] * sl[j];
        su[i] += u[i][j] * yh[j];
      }
      s3[0] += su[i];
      if (a.dX) store8(norm_row(a.dX, row, a.ldx, a), col, a.D, a.vec, d);
      if (zr && a.dZ) store8(norm_row(a.dZ, row, a.ldz, a), col, a.D, a.vec, dz);
    }
    if (a.dY) {
      if constexpr (GROUPS) group_sum<TPR>(su, t, a.D, a.group, buf);
      else row_sum<TPR>(s3, red);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        const float ry = rsqrtf((GROUPS ? sy[i] : s1[0]) / (float)a.group + a.eps);
        const float mu = (GROUPS ? su[i] : s3[0]) / (float)a.group;
        float v[8];
        unpack8(y[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ry * (u[i][j] - v[j] * ry * mu);
        store8(norm_row(a.dY, row, a.ldy, a), col, a.D, a.vec, v);
      }
    }
  }

  // the block's column sums: its rows' threads in turn, in a fixed order
  if (a.part) {
    float* part = a.part + (int64_t)blockIdx.x * 3 * a.D;
#pragma unroll 1
    for (int q = 0; q < 3; ++q) {
      float* sum = RPB > 1 ? gbuf : part + q * a.D;
      if constexpr (RPB > 1) __syncthreads();
#pragma unroll 1
      for (int b = 0; b < RPB; ++b) {
        if (rb == b)
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int col = (i * TPR + t) * 8 + j;
              const float v = q == 0 ? c_post[i][j] : q == 1 ? c_lam[i][j] : c_pre[i][j];
              if (col < a.D) sum[col] = b ? sum[col] + v : v;
            }
        if constexpr (RPB > 1) __syncthreads();
      }
      if constexpr (RPB > 1)
        for (int col = threadIdx.x; col < a.D; col += BLOCK) part[q * a.D + col] = gbuf[col];
    }
  }
}

// Column sums over the blocks' partial sums in a fixed order; dw_post also over the row's groups.
// Block: 32 columns x 8 slices of the blocks.
__global__ void __launch_bounds__(256) k_norm_cols(const float* __restrict__ part, int blocks, int D, int group,
                                                   float* dw_post, float* dlam, float* dw_pre) {
  __shared__ float s[8][33];
  const int q = blockIdx.y, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  float* out = q == 0 ? dw_post : q == 1 ? dlam : dw_pre;
  const int n = q == 0 ? group : D;
  const int col = blockIdx.x * 32 + lane;
  if (!out || blockIdx.x * 32 >= n) return;
  pdl_wait();
  float v = 0.f;
  if (col < n)
    for (int b = slice; b < blocks; b += 8)
      for (int c = col; c < D; c += n) v += part[((int64_t)b * 3 + q) * D + c];
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && col < n) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i][lane];
    out[col] = t;
  }
}

}  // namespace ttt
