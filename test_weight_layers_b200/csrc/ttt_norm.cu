// C ABI of the block norms (see include/ttt.h for the contract).
#include <algorithm>

#include "host.cuh"
#include "kernels_norm.cuh"
#include "ttt.h"

using namespace ttt;

namespace {

constexpr int kNormMaxD = 8192;
constexpr int kNormSms = 148;

// How a call's rows map to kernel rows: groups become rows of their own where nothing ties the columns of a
// row together but w_post (no second norm, no residual scale or gradient over all columns).
struct NormShape {
  int split, D, tpr, nv;
  bool groups;
};

// Threads of a row and chunks of 8 columns per thread.  Forward: a warp to a row up to 1024 columns (no barriers),
// but one chunk to a thread where the rows are too few to fill the card (7 rows of 768: 3.0 us against 6.6 us).
// Backward: up to ten tensors' registers and three column sums per chunk, so at most two chunks per thread; two
// rather than one, since the reductions cost a thread the same (65,536 x 2,048: 422 us with 2 chunks on 4 warps,
// 486 us with 1 on 8).
NormShape norm_shape(const ttt_norm_cfg& c, bool row_wide, bool back, int64_t T) {
  NormShape s{};
  s.split = !row_wide && c.group < c.D ? c.D / c.group : 1;
  s.D = c.D / s.split;
  s.groups = c.group < s.D;
  const int chunks = (s.D + 7) / 8;
  if (back) s.tpr = chunks <= 64 ? 32 : chunks <= 256 ? 128 : chunks <= 512 ? 256 : 512;
  else if (T * s.split <= 4 * kNormSms) s.tpr = chunks <= 32 ? 32 : chunks <= 128 ? 128 : chunks <= 256 ? 256 : 512;
  else s.tpr = chunks <= 128 ? 32 : chunks <= 512 ? 128 : 256;
  s.nv = (chunks + s.tpr - 1) / s.tpr;
  return s;
}

int64_t norm_blocks(const NormShape& s, int64_t T) {
  const int block = std::max(128, s.tpr), rpb = block / s.tpr;
  const int64_t rows = T * s.split;
  return std::max<int64_t>(1, std::min<int64_t>((rows + rpb - 1) / rpb, (int64_t)kNormSms * (512 / block)));
}

bool norm_cfg_ok(const ttt_norm_cfg* c) {
  return c && c->D >= 1 && c->group >= 1 && c->D % c->group == 0 && c->eps >= 0.f;
}
bool norm_cfg_supported(const ttt_norm_cfg& c) { return c.D <= kNormMaxD && (c.group == c.D || c.group % 8 == 0); }

int64_t eff(int64_t ld, int D) { return ld ? ld : D; }

bool vec_ok(const void* p, int64_t ld, ttt_dtype dt) {
  return !p || (aligned16(p) && (ld * (int64_t)esize(dt)) % 16 == 0);
}
bool elem_ok(const void* p, ttt_dtype dt) { return (reinterpret_cast<uintptr_t>(p) & (esize(dt) - 1)) == 0; }

template <typename T, int TPR, int NV, bool GROUPS, bool VEC>
int launch_norm(const NormArgs<T>& a, bool back, int64_t blocks, cudaStream_t s) {
  constexpr int block = TPR > 128 ? TPR : 128;
  const int chunks = (a.D + 7) / 8, rpb = block / TPR;
  size_t smem = GROUPS ? (size_t)rpb * chunks * 4 : 0;
  if (back) {
    if constexpr (NV <= 2) {
      if (rpb > 1) smem = std::max(smem, (size_t)a.D * 4);
      k_block_norm_bwd<T, TPR, NV, GROUPS, VEC><<<(unsigned)blocks, block, smem, s>>>(a);
    }
  } else {
    k_block_norm<T, TPR, NV, GROUPS, VEC><<<(unsigned)blocks, block, smem, s>>>(a);
  }
  TTT_LAUNCHED();
  return TTT_OK;
}

template <typename T, int TPR, int NV>
int launch_norm_any(const NormArgs<T>& a, const NormShape& sh, bool vec, bool back, int64_t blocks, cudaStream_t s) {
  if (sh.groups) {
    return vec ? launch_norm<T, TPR, NV, true, true>(a, back, blocks, s)
               : launch_norm<T, TPR, NV, true, false>(a, back, blocks, s);
  }
  return vec ? launch_norm<T, TPR, NV, false, true>(a, back, blocks, s)
             : launch_norm<T, TPR, NV, false, false>(a, back, blocks, s);
}

// The shapes that norm_shape gives.
template <typename T>
int run_norm(const NormArgs<T>& a, const NormShape& sh, bool vec, bool back, int64_t blocks, cudaStream_t s) {
  switch (sh.tpr * 8 + sh.nv) {
    case 32 * 8 + 1: return launch_norm_any<T, 32, 1>(a, sh, vec, back, blocks, s);
    case 32 * 8 + 2: return launch_norm_any<T, 32, 2>(a, sh, vec, back, blocks, s);
    case 32 * 8 + 3: return launch_norm_any<T, 32, 3>(a, sh, vec, back, blocks, s);
    case 32 * 8 + 4: return launch_norm_any<T, 32, 4>(a, sh, vec, back, blocks, s);
    case 128 * 8 + 1: return launch_norm_any<T, 128, 1>(a, sh, vec, back, blocks, s);
    case 128 * 8 + 2: return launch_norm_any<T, 128, 2>(a, sh, vec, back, blocks, s);
    case 128 * 8 + 3: return launch_norm_any<T, 128, 3>(a, sh, vec, back, blocks, s);
    case 128 * 8 + 4: return launch_norm_any<T, 128, 4>(a, sh, vec, back, blocks, s);
    case 256 * 8 + 1: return launch_norm_any<T, 256, 1>(a, sh, vec, back, blocks, s);
    case 256 * 8 + 2: return launch_norm_any<T, 256, 2>(a, sh, vec, back, blocks, s);
    case 256 * 8 + 3: return launch_norm_any<T, 256, 3>(a, sh, vec, back, blocks, s);
    case 256 * 8 + 4: return launch_norm_any<T, 256, 4>(a, sh, vec, back, blocks, s);
    case 512 * 8 + 1: return launch_norm_any<T, 512, 1>(a, sh, vec, back, blocks, s);
    case 512 * 8 + 2: return launch_norm_any<T, 512, 2>(a, sh, vec, back, blocks, s);
    default: return TTT_ERR_UNSUPPORTED;
  }
}

struct NormCall {
  const void *X, *Y, *Z, *dXo, *dN;
  void *Xo, *N, *dX, *dY, *dZ;
  const float *w_post, *lam, *w_pre;
};

// Strides, alignment and the vector rule: 16-byte accesses where every row allows them, else by element.
int check_norm(const NormCall& c, const ttt_norm_cfg& cfg, ttt_dtype dt, int64_t (&ld)[5], int& vec) {
  ld[0] = eff(cfg.ld_x, cfg.D);
  ld[1] = eff(cfg.ld_y, cfg.D);
  ld[2] = eff(cfg.ld_z, cfg.D);
  ld[3] = eff(cfg.ld_xout, cfg.D);
  ld[4] = eff(cfg.ld_n, cfg.D);
  for (int64_t l : ld)
    if (l < cfg.D) return TTT_ERR_INVALID;
  const struct {
    const void* p;
    int64_t ld;
  } t[] = {{c.X, ld[0]}, {c.dX, ld[0]},  {c.Y, ld[1]},   {c.dY, ld[1]}, {c.Z, ld[2]},
           {c.dZ, ld[2]}, {c.Xo, ld[3]}, {c.dXo, ld[3]}, {c.N, ld[4]},  {c.dN, ld[4]}};
  vec = cfg.D % 8 == 0 && cfg.group % 8 == 0;
  for (const auto& x : t) {
    if (!elem_ok(x.p, dt)) return TTT_ERR_ALIGN;
    if (!vec_ok(x.p, x.ld, dt)) vec = 0;
  }
  for (const void* p : {(const void*)c.w_post, (const void*)c.lam, (const void*)c.w_pre})
    if (!elem_ok(p, TTT_FP32)) return TTT_ERR_ALIGN;
    else if (!aligned16(p)) vec = 0;
  return TTT_OK;
}

template <typename T>
NormArgs<T> norm_args(const NormCall& c, const ttt_norm_cfg& cfg, const NormShape& sh, const int64_t (&ld)[5], int64_t rows) {
  NormArgs<T> a{};
  a.X = (const T*)c.X;
  a.Y = (const T*)c.Y;
  a.Z = (const T*)c.Z;
  a.dXo = (const T*)c.dXo;
  a.dN = (const T*)c.dN;
  a.Xo = (T*)c.Xo;
  a.N = (T*)c.N;
  a.dX = (T*)c.dX;
  a.dY = (T*)c.dY;
  a.dZ = (T*)c.dZ;
  a.ldx = ld[0];
  a.ldy = ld[1];
  a.ldz = ld[2];
  a.ldxo = ld[3];
  a.ldn = ld[4];
  a.w_post = c.w_post;
  a.lam = c.lam;
  a.w_pre = c.w_pre;
  a.rows = rows * sh.split;
  a.split = sh.split;
  a.D = sh.D;
  a.group = cfg.group;
  a.eps = cfg.eps;
  return a;
}

}  // namespace

extern "C" {

int ttt_block_norm(const void* X, const void* Y, const void* Z, const float* w_post, const float* res_scale,
                   const float* w_pre, void* Xout, void* N, int64_t T, const ttt_norm_cfg* cfg, ttt_dtype dtype,
                   void* stream) {
  if ((dtype != TTT_FP32 && dtype != TTT_BF16) || !norm_cfg_ok(cfg) || T < 0) return TTT_ERR_INVALID;
  if (!norm_cfg_supported(*cfg)) return TTT_ERR_UNSUPPORTED;
  const NormCall c{X, Y, Z, nullptr, nullptr, Xout, N, nullptr, nullptr, nullptr, w_post, res_scale, w_pre};
  int64_t ld[5];
  int vec;
  TTT_TRY(check_norm(c, *cfg, dtype, ld, vec));
  if (T == 0) return TTT_OK;
  if (!Y || (!Xout && !N)) return TTT_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  const NormShape sh = norm_shape(*cfg, N || res_scale, false, T);
  const int block = std::max(128, sh.tpr), rpb = block / sh.tpr;
  const int64_t blocks = std::min<int64_t>((T * sh.split + rpb - 1) / rpb, (int64_t)kNormSms * (512 / block));
  ProfScope ps(TTT_PROF_BNORM, s);
  if (dtype == TTT_FP32) return run_norm(norm_args<float>(c, *cfg, sh, ld, T), sh, vec != 0, false, blocks, s);
  return run_norm(norm_args<__nv_bfloat16>(c, *cfg, sh, ld, T), sh, vec != 0, false, blocks, s);
}

size_t ttt_block_norm_workspace_bytes(const ttt_norm_cfg* cfg, int64_t T) {
  if (!norm_cfg_ok(cfg) || !norm_cfg_supported(*cfg) || T < 0) return 0;
  size_t most = 0;
  for (bool wide : {false, true}) {
    const NormShape sh = norm_shape(*cfg, wide, true, T);
    most = std::max(most, (size_t)norm_blocks(sh, std::max<int64_t>(T, 1)) * 3 * sh.D * 4);
  }
  return up256(most);
}

int ttt_block_norm_backward(const void* X, const void* Y, const void* Z, const float* w_post, const float* res_scale,
                            const float* w_pre, const void* dXout, const void* dN, void* dX, void* dY, void* dZ,
                            float* dw_post, float* dres_scale, float* dw_pre, int64_t T, const ttt_norm_cfg* cfg,
                            ttt_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
  if ((dtype != TTT_FP32 && dtype != TTT_BF16) || !norm_cfg_ok(cfg) || T < 0) return TTT_ERR_INVALID;
  if (!norm_cfg_supported(*cfg)) return TTT_ERR_UNSUPPORTED;
  const NormCall c{X, Y, Z, dXout, dN, nullptr, nullptr, dX, dY, dZ, w_post, res_scale, w_pre};
  int64_t ld[5];
  int vec;
  TTT_TRY(check_norm(c, *cfg, dtype, ld, vec));
  if (!elem_ok(dw_post, TTT_FP32) || !elem_ok(dres_scale, TTT_FP32) || !elem_ok(dw_pre, TTT_FP32)) return TTT_ERR_ALIGN;
  const bool cols = dw_post || dres_scale || dw_pre;
  if (cols && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < ttt_block_norm_workspace_bytes(cfg, T)))
    return TTT_ERR_WORKSPACE;
  if (T > 0 && (!Y || (!dXout && !dN))) return TTT_ERR_INVALID;
  if ((dZ && !Z && T > 0) || (dX && !X && T > 0)) return TTT_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  const NormShape sh = norm_shape(*cfg, dN || res_scale || dres_scale || dw_pre, true, T);
  ProfScope ps(TTT_PROF_BNORM, s);
  int64_t blocks = 0;
  if (T > 0) {
    blocks = norm_blocks(sh, T);
    auto go = [&](auto a) {
      a.part = cols ? (float*)ws : nullptr;
      return run_norm(a, sh, vec != 0, true, blocks, s);
    };
    TTT_TRY(dtype == TTT_FP32 ? go(norm_args<float>(c, *cfg, sh, ld, T))
                              : go(norm_args<__nv_bfloat16>(c, *cfg, sh, ld, T)));
  }
  if (!cols) return TTT_OK;
  TTT_TRY(launch_pdl(k_norm_cols, dim3((sh.D + 31) / 32, 3), dim3(1024), 0, s, (const float*)ws, (int)blocks, sh.D,
                     cfg->group, dw_post, dres_scale, dw_pre));
  TTT_LAUNCHED();
  return TTT_OK;
}

}  // extern "C"
