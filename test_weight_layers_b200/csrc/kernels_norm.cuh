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
// HBM once.  All arithmetic is fp32, rounded once on the way out.
//
// Share of the copy rate (6.46 TB/s) with all operands, bf16 | fp32:
//                         forward       gradient
//     131,072 x   768   0.89 | 0.68   0.62 | 0.58
//      65,536 x 2,048   0.83 | 0.97   0.79 | 0.51
//      16,384 x 8,192   0.57 | 0.61   0.25 | 0.21
// The bf16 forward and the bf16 gradient at 2,048 columns are bound by those bytes.
// What is far below spills registers in its row loop: the fp32 gradient (224 to 524
// bytes a thread), the gradient of more than 4,096 columns, whose 512 threads have
// 128 registers for two chunks each (976 to 1,592), and the fp32 forward with three
// chunks to a thread, as for 768 columns (148 to 392, under the bound of four blocks
// an SM); the bf16 gradient with one chunk to a thread spills 24 to 156.
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

// Two fp32 operations in one instruction (the gradient is bound by its instructions otherwise).
__device__ __forceinline__ unsigned long long bits(float2 x) { return *reinterpret_cast<unsigned long long*>(&x); }
__device__ __forceinline__ float2 from_bits(unsigned long long v) { return *reinterpret_cast<float2*>(&v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return from_bits(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return from_bits(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void unpack2(const Raw8<__nv_bfloat16>& r, float2 (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = (&r.q[0].x)[j];
    x[j] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}
__device__ __forceinline__ void unpack2(const Raw8<float>& r, float2 (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = make_float2(__uint_as_float((&r.q[j >> 1].x)[2 * (j & 1)]), __uint_as_float((&r.q[j >> 1].x)[2 * (j & 1) + 1]));
}

// Columns [col, col + 8) of a row, zero past D.  VEC: rows and weights are 16-byte aligned, D a multiple of 8.
// Plain loads: an output may be one of the inputs.
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int col, int D) {
  Raw8<T> r;
  if constexpr (VEC) {
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
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int col, int D, const float (&x)[8]);
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int col, int D, const float2 (&x)[4]) {
  const float y[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
  store8<VEC>(p, col, D, y);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int col, int D, const float (&x)[8]) {
  const Raw8<T> r = pack8(x, T());
  if constexpr (VEC) {
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
template <bool VEC>
__device__ __forceinline__ void weight8(const float* w, int col, int n, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = w ? 0.f : 1.f;
  if (!w) return;
  if constexpr (VEC) {
    if (col < n) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(w + col));
      const float4 b = __ldg(reinterpret_cast<const float4*>(w + col + 4));
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < n) x[j] = __ldg(w + col + j);
  }
}

template <bool VEC>
__device__ __forceinline__ void weight8(const float* w, int col, int n, float2 (&x)[4]) {
  float y[8];
  weight8<VEC>(w, col, n, y);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = make_float2(y[2 * j], y[2 * j + 1]);
}

// Sums over the TPR threads of a row (TPR = 32: a warp; else the whole block).  The sums of a row have a buffer
// each, so that one barrier does: a buffer is written again only after the barriers of the others.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[TPR / 32]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; w += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&red[i][w]);
        s += (x.x + x.y) + (x.z + x.w);
      }
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

// Where kernel row r starts: row r / split, part r % split of its columns, stepped without divisions.
struct RowAt {
  int64_t row;
  int part;
  __device__ __forceinline__ RowAt(int64_t r, int split) : row(split == 1 ? r : r / split), part(split == 1 ? 0 : (int)(r % split)) {}
  __device__ __forceinline__ void step(const RowAt& by, int split) {
    row += by.row;
    part += by.part;
    if (part >= split) part -= split, ++row;
  }
  template <typename T>
  __device__ __forceinline__ T* in(T* p, int64_t ld, int D) const {
    return p + row * ld + part * D;
  }
};

// The logistic function.  bf16 rows take the hardware's exponential and reciprocal (2^-21 for |z| below 8, 2^-17 at -88
// where it vanishes: far below the outputs' rounding, and what the weights' gradients take from it is that of single
// rows): the exact ones are a third of the instructions of a pass that is otherwise bound by HBM.
template <typename T>
__device__ __forceinline__ float sigmoid_f(float z) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}

// TPR threads to a row, NV chunks of 8 columns to a thread; GROUPS: several means of y to a row.
// Measured (131,072 x 768, bf16, all operands): 176 us, 5.73 TB/s; without the loads ahead 208 us.
template <typename T, int TPR, int NV, bool GROUPS, bool VEC>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128, NV <= 3 ? 4 * 128 / (TPR > 128 ? TPR : 128) : 1) k_block_norm(const NormArgs<T> a) {
  constexpr int BLOCK = TPR > 128 ? TPR : 128;
  constexpr int RPB = BLOCK / TPR;  // rows per block
  __shared__ __align__(16) float red[2][TPR / 32];
  extern __shared__ float gbuf[];
  const int t = threadIdx.x % TPR, rb = threadIdx.x / TPR;
  float* buf = gbuf + rb * ((a.D + 7) / 8);
  const bool xr = a.X != nullptr, zr = a.Z != nullptr;
  const float inv_group = 1.f / (float)a.group, inv_d = 1.f / (float)a.D;
  const int64_t r0 = (int64_t)blockIdx.x * RPB + rb, step = (int64_t)gridDim.x * RPB;
  RowAt at(r0, a.split), ahead = at;
  const RowAt by(step, a.split);
  Raw8<T> ny[NV], nx[NV], nz[NV];  // the next row, in flight while one is worked on
  auto load_row = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      ny[i] = load8<VEC>(ahead.in(a.Y, a.ldy, a.D), col, a.D);
      if (zr) nz[i] = load8<VEC>(ahead.in(a.Z, a.ldz, a.D), col, a.D);
      if (xr) nx[i] = load8<VEC>(ahead.in(a.X, a.ldx, a.D), col, a.D);
    }
    ahead.step(by, a.split);
  };
  if (r0 < a.rows) load_row();
  for (int64_t row = r0; row < a.rows; row += step, at.step(by, a.split)) {
    Raw8<T> y[NV], x[NV], z[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i] = ny[i], x[i] = nx[i], z[i] = nz[i];
    if (row + step < a.rows) load_row();
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
    const float ry1 = rsqrtf(s1[0] * inv_group + a.eps);
    float p[NV][8], s2[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      const float ry = GROUPS ? rsqrtf(sy[i] * inv_group + a.eps) : ry1;
      float w[8], v[8];
      unpack8(y[i], p[i]);
      weight8<VEC>(a.w_post, GROUPS ? col % a.group : col, a.group, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) p[i][j] = p[i][j] * ry * w[j];
      if (zr) {
        unpack8(z[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= v[j] * sigmoid_f<T>(v[j]);
      }
      if (a.lam) {
        weight8<VEC>(a.lam, col, a.D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= w[j];
      }
      if (xr) {
        unpack8(x[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] += v[j];
      }
      if (a.Xo) store8<VEC>(at.in(a.Xo, a.ldxo, a.D), col, a.D, p[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s2[0] += p[i][j] * p[i][j];
    }
    if (a.N) {
      row_sum<TPR>(s2, red + 1);
      const float r = rsqrtf(s2[0] * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        float w[8];
        weight8<VEC>(a.w_pre, col, a.D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] *= r * w[j];
        store8<VEC>(at.in(a.N, a.ldn, a.D), col, a.D, p[i]);
      }
    } else if (TPR > 32 && !GROUPS) {
      __syncthreads();  // a row with one sum only: its buffer is read
    }
  }
}

// The gradient.  A thread keeps its columns for all its rows: their weights and their sums stay in registers, and
// the next row's loads are in flight while one is worked on.
// Measured (65,536 x 2,048, bf16, all operands): 422 us, 5.1 TB/s, half of the issue slots busy.
template <typename T, int TPR, int NV, bool GROUPS, bool VEC>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128, NV == 1 ? (TPR > 128 ? 512 / TPR : 4) : 1)
    k_block_norm_bwd(const NormArgs<T> a) {
  constexpr int BLOCK = TPR > 128 ? TPR : 128;
  constexpr int RPB = BLOCK / TPR;
  __shared__ __align__(16) float red[4][TPR / 32];  // sum 0, the two of sum 1, sum 2
  extern __shared__ float gbuf[];
  const int t = threadIdx.x % TPR, rb = threadIdx.x / TPR;
  float* buf = gbuf + rb * ((a.D + 7) / 8);
  const bool xr = a.X != nullptr, zr = a.Z != nullptr, gr = a.dXo != nullptr, nr = a.dN != nullptr;
  const float inv_group = 1.f / (float)a.group, inv_d = 1.f / (float)a.D;
  float2 c_post[NV][4], c_lam[NV][4], c_pre[NV][4];  // this thread's column sums
  float2 wq[NV][4], lm[NV][4], wp[NV][4];            // and its columns' weights
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * 8;
    weight8<VEC>(a.w_post, GROUPS ? col % a.group : col, a.group, wq[i]);
    weight8<VEC>(a.lam, col, a.D, lm[i]);
    weight8<VEC>(a.w_pre, col, a.D, wp[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) c_post[i][j] = c_lam[i][j] = c_pre[i][j] = both(0.f);
  }
  const int64_t r0 = (int64_t)blockIdx.x * RPB + rb, step = (int64_t)gridDim.x * RPB;
  RowAt at(r0, a.split), ahead = at;
  const RowAt by(step, a.split);
  Raw8<T> ny[NV], nx[NV], nz[NV], ngx[NV], ngn[NV];
  auto load_row = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      ny[i] = load8<VEC>(ahead.in(a.Y, a.ldy, a.D), col, a.D);
      if (zr) nz[i] = load8<VEC>(ahead.in(a.Z, a.ldz, a.D), col, a.D);
      if (gr) ngx[i] = load8<VEC>(ahead.in(a.dXo, a.ldxo, a.D), col, a.D);
      if (nr) {
        ngn[i] = load8<VEC>(ahead.in(a.dN, a.ldn, a.D), col, a.D);
        if (xr) nx[i] = load8<VEC>(ahead.in(a.X, a.ldx, a.D), col, a.D);
      }
    }
    ahead.step(by, a.split);
  };
  if (r0 < a.rows) load_row();
  for (int64_t row = r0; row < a.rows; row += step, at.step(by, a.split)) {
    Raw8<T> x[NV], z[NV], gx[NV], gn[NV];
    float2 yh[NV][4];
    float sy[NV], s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack2(ny[i], yh[i]);
      x[i] = nx[i], z[i] = nz[i], gx[i] = ngx[i], gn[i] = ngn[i];
      float2 q = both(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) q = fma2(yh[i][j], yh[i][j], q);
      sy[i] = q.x + q.y;
      s1[0] += sy[i];
    }
    if (row + step < a.rows) load_row();
    if constexpr (GROUPS) group_sum<TPR>(sy, t, a.D, a.group, buf);
    else row_sum<TPR>(s1, red);
    // s(z), s'(z), x' again, and the two sums of its norm
    float2 sl[NV][4], ds[NV][4], xo[NV][4];
    float ry[NV], s2[2] = {0.f, 0.f};  // sum x'^2, sum t x'
    const float ry1 = rsqrtf(s1[0] * inv_group + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ry[i] = GROUPS ? rsqrtf(sy[i] * inv_group + a.eps) : ry1;
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) yh[i][j] = mul2(yh[i][j], both(ry[i])), sl[i][j] = both(1.f), ds[i][j] = both(0.f);
      if (zr) {
        unpack2(z[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 sg = make_float2(sigmoid_f<T>(v[j].x), sigmoid_f<T>(v[j].y));
          sl[i][j] = mul2(v[j], sg);
          ds[i][j] = fma2(sl[i][j], fma2(sg, both(-1.f), both(1.f)), sg);
        }
      }
      if (nr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) xo[i][j] = mul2(mul2(yh[i][j], sl[i][j]), mul2(lm[i][j], wq[i][j]));
        if (xr) {
          unpack2(x[i], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) xo[i][j] = fma2(v[j], both(1.f), xo[i][j]);
        }
        unpack2(gn[i], v);
        float2 q0 = both(0.f), q1 = q0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q0 = fma2(xo[i][j], xo[i][j], q0);
          q1 = fma2(mul2(v[j], wp[i][j]), xo[i][j], q1);
        }
        s2[0] += q0.x + q0.y;
        s2[1] += q1.x + q1.y;
      }
    }
    float r = 0.f, m = 0.f;
    if (nr) {
      row_sum<TPR>(s2, red + 1);
      r = rsqrtf(s2[0] * inv_d + a.eps);
      m = r * r * (s2[1] * inv_d);
    }
    // column sums, dx, dz and the sums of u y r_y
    float2 u[NV][4];
    float su[NV], s3[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * 8;
      float2 d[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = both(0.f);
      if (gr) unpack2(gx[i], d);
      if (nr) {
        unpack2(gn[i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c_pre[i][j] = fma2(v[j], mul2(xo[i][j], both(r)), c_pre[i][j]);
          const float2 e = fma2(xo[i][j], both(-m), mul2(v[j], wp[i][j]));
          d[j] = fma2(e, both(r), d[j]);
        }
      }
      float2 q = both(0.f), dz[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 ys = mul2(yh[i][j], sl[i][j]), dp = mul2(d[j], lm[i][j]), dw = mul2(dp, wq[i][j]);
        c_lam[i][j] = fma2(d[j], mul2(ys, wq[i][j]), c_lam[i][j]);
        c_post[i][j] = fma2(dp, ys, c_post[i][j]);
        dz[j] = mul2(mul2(dw, yh[i][j]), ds[i][j]);
        u[i][j] = mul2(dw, sl[i][j]);
        q = fma2(u[i][j], yh[i][j], q);
      }
      su[i] = q.x + q.y;
      s3[0] += su[i];
      if (a.dX) store8<VEC>(at.in(a.dX, a.ldx, a.D), col, a.D, d);
      if (zr && a.dZ) store8<VEC>(at.in(a.dZ, a.ldz, a.D), col, a.D, dz);
    }
    if (a.dY) {
      if constexpr (GROUPS) group_sum<TPR>(su, t, a.D, a.group, buf);
      else row_sum<TPR>(s3, red + 3);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * 8;
        const float mu = (GROUPS ? su[i] : s3[0]) * inv_group;
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(fma2(yh[i][j], both(-mu), u[i][j]), both(ry[i]));
        store8<VEC>(at.in(a.dY, a.ldy, a.D), col, a.D, v);
      }
    } else if (TPR > 32 && !GROUPS && !nr) {
      __syncthreads();  // a row with one sum only: its buffer is read
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
              const float2 v2 = q == 0 ? c_post[i][j / 2] : q == 1 ? c_lam[i][j / 2] : c_pre[i][j / 2];
              const float v = j % 2 ? v2.y : v2.x;
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
// Block: 32 columns x 32 slices of the blocks, four loads of a slice in flight.
__global__ void __launch_bounds__(1024) k_norm_cols(const float* __restrict__ part, int blocks, int D, int group,
                                                    float* dw_post, float* dlam, float* dw_pre) {
  __shared__ float s[32][33];
  const int q = blockIdx.y, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  float* out = q == 0 ? dw_post : q == 1 ? dlam : dw_pre;
  const int n = q == 0 ? group : D;
  const int col = blockIdx.x * 32 + lane;
  if (!out || blockIdx.x * 32 >= n) return;
  pdl_wait();
  float v = 0.f;
  if (col < n)
    for (int c = col; c < D; c += n) {
      const float* p = part + (int64_t)q * D + c;
      const int64_t ld = 3 * (int64_t)D;
      for (int b = slice; b < blocks; b += 128) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = b + 32 * k < blocks ? p[(b + 32 * k) * ld] : 0.f;
        v += (x[0] + x[1]) + (x[2] + x[3]);
      }
    }
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && col < n) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    out[col] = t;
  }
}

}  // namespace ttt
