// Gated delta rule, chunked form (bf16 tokens): chunk table, chunk preparation
// and the state pass.  The formulas and the operand scheme are in
// delta_common.cuh.
#pragma once

#include "delta_common.cuh"

namespace ttt {

// ---------------------------------------------------------------------------
// Chunk table.  One block: checks the offsets (0 <= cu[i] <= cu[i+1] <= T), cuts
// long sequences into segments (fill: sequences' passes that fit on the card; 0:
// none is cut), and writes the segments, those before and those behind a cut once
// more by themselves, and each chunk's first token and length.  Refused offsets, or an
// error already recorded in the status word, mark every segment with length -1:
// the kernels after it then write nothing.
//
// Uncut, the passes take as long as the longest sequence.  Cut into segments of k
// chunks they take about 3 k (the transitions are more rows than the states) and a
// join for each, so the longest is cut where it is at least three times the card's
// share of all chunks, k being that share; a join costs about as much as a chunk of
// both passes, so neither many joins nor long segments: 2 k^2 >= chunks.
constexpr int DR_CUT_CHUNKS = 12;  // shorter sequences are never cut
__global__ void __launch_bounds__(1024) k_delta_plan(const int* __restrict__ cu, int n_seq, int T, int fill,
                                                     int max_segs, int max_cuts, int max_chunks,
                                                     DrSeq* __restrict__ seqs, DrSeq* __restrict__ cuts,
                                                     DrChunk* __restrict__ chunks, unsigned int* status) {
  __shared__ long long warp_sum[32];
  __shared__ int warp_all[32], warp_max[32];
  __shared__ long long carry;
  __shared__ int listed;
  __shared__ int order[1024], key[1024];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = *(volatile unsigned int*)status != DEV_OK;
  const int even = n_seq > 0 ? T / n_seq : 0;  // without offsets: sequences of equal length
  int all = 0, most = 0;  // chunks of all sequences and of the longest one
  if (cu) {
    for (int i = tid; i < n_seq; i += 1024) {
      const int a = cu[i], b = cu[i + 1];
      if (a < 0 || b < a || b > T) {
        bad = true;
        atomicCAS(status, (unsigned int)DEV_OK, (unsigned int)DEV_INVALID);
      } else {
        const int n = (b - a) / DR_C + ((b - a) % DR_C != 0);
        all += n;
        most = max(most, n);
      }
    }
    all = __reduce_add_sync(0xffffffffu, all);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) warp_all[warp] = all, warp_max[warp] = most;
  }
  bad = __syncthreads_or(bad);
  int seg_chunks = 0;
  if (fill) {
    if (cu) {
      all = __reduce_add_sync(0xffffffffu, warp_all[lane]);
      most = __reduce_max_sync(0xffffffffu, warp_max[lane]);
    } else {
      most = (even + DR_C - 1) / DR_C;
      all = most * n_seq;
    }
    if (most >= DR_CUT_CHUNKS && 3 * all <= (long long)fill * most) {
      seg_chunks = (all + fill - 1) / fill;
      while (2 * (long long)seg_chunks * seg_chunks < most) ++seg_chunks;
    }
  }
  // up to 1024 sequences are taken longest first, so that the passes' long blocks start early
  const bool sorted = cu && n_seq > 1 && n_seq <= 1024;
  if (sorted) {
    int n = 2;
    while (n < n_seq) n <<= 1;
    if (tid < n) {
      order[tid] = tid;
      key[tid] = tid < n_seq ? cu[tid + 1] - cu[tid] : INT32_MIN;
    }
    for (int k = 2; k <= n; k <<= 1)
      for (int j = k >> 1; j; j >>= 1) {
        __syncthreads();
        const int o = tid ^ j;
        if (tid < n && o > tid) {
          const int a = key[tid], b = key[o], ia = order[tid], ib = order[o];
          const bool after = a < b || (a == b && ia > ib);  // a belongs behind b
          if (after == ((tid & k) == 0)) {
            key[tid] = b, key[o] = a;
            order[tid] = ib, order[o] = ia;
          }
        }
      }
    __syncthreads();
  }
  if (tid == 0) carry = listed = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n_seq; i0 += 1024) {
    const int i = i0 + tid;
    int tok = 0, len = 0, id = i;
    if (i < n_seq) {
      if (sorted) id = order[i];
      tok = cu ? cu[id] : id * even;
      len = bad ? -1 : (cu ? cu[id + 1] - tok : even);
    }
    const int n = len > 0 ? (len + DR_C - 1) / DR_C : 0;
    const int ns = i >= n_seq ? 0 : seg_chunks > 0 && n > 0 ? (n + seg_chunks - 1) / seg_chunks : 1;
    // segments of cut sequences (up to 296), segments and chunks (each below 2^27), scanned together
    const long long own = (long long)(ns > 1 ? ns : 0) << 54 | (long long)ns << 27 | n;
    long long sum = own;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      long long w = warp_sum[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += v;
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    const long long first = carry + sum - own + (warp ? warp_sum[warp - 1] : 0);
    const int chunk0 = (int)(first & 0x7ffffff), seg0 = (int)(first >> 27 & 0x7ffffff), cut0 = (int)(first >> 54);
    const int at = ns > 1 ? atomicAdd(&listed, ns - 1) : 0;  // (the list's order does not matter)
    for (int k = 0; k < ns; ++k) {
      const int c0 = k * seg_chunks;
      const int l = ns == 1 ? len : min(seg_chunks * DR_C, len - c0 * DR_C);
      const DrSeq s{tok + c0 * DR_C, l, chunk0 + c0, id, k, ns, cut0 + k, 0};
      seqs[seg0 + k] = s;
      if (k < ns - 1) cuts[at + k] = s;
      if (k > 0) cuts[max_cuts + at + k - 1] = s;
    }
    __syncthreads();
    if (tid == 1023) carry = first + own;
    __syncthreads();
  }
  const int total = (int)(carry & 0x7ffffff), nsegs = (int)(carry >> 27 & 0x7ffffff);
  for (int i = nsegs + tid; i < max_segs; i += 1024) seqs[i] = DrSeq{0, -1, 0, 0, 0, 1, 0, 0};
  for (int i = listed + tid; i < max_cuts; i += 1024)
    cuts[i] = cuts[max_cuts + i] = DrSeq{0, -1, 0, 0, 0, 1, 0, 0};
  __threadfence_block();
  __syncthreads();
  for (int c = tid; c < max_chunks; c += 1024) {
    DrChunk e{0, -1};
    if (c < total) {
      int lo = 0, hi = nsegs - 1;  // the last segment whose first chunk is <= c (empty ones before it share it)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seqs[mid].chunk0 <= c) lo = mid;
        else hi = mid - 1;
      }
      const DrSeq s = seqs[lo];
      const int at = (c - s.chunk0) * DR_C;
      e.tok = s.tok + at;
      e.len = min(DR_C, s.len - at);
    }
    chunks[c] = e;
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// Chunk preparation: one block per (chunk, query/key head), for all value heads
// that share it.  Writes K16 and Q16 (the token rows, exact in fp16, as
// shared-memory images for the next kernels' bulk copies) and per value head
// Y and P (hi, lo) and the chunk vectors.
struct PrepArgs {
  const __nv_bfloat16 *Q, *K;
  const float *g, *beta;  // [T][heads_v]
  int64_t ldq, ldk;
  int hk, hv, dk, l2norm;
  float scale;
  const DrChunk* chunks;
  uint8_t* kq;   // [chunk][hk][K16 | Q16]
  uint8_t* blk;  // [chunk][hv][DR_BLK]
  float* tok;    // [chunk][hk][6][64] token factors (TF_*), backward pass only
};

// Token factors for the way back through the norm: k~ = f_k K16 with f_k = scale 2^-e / n, so
// dk = h_k (dk~ - p_k K16 (K16 . dk~)), h_k = f_k 2^e, p_k = 1 / ||K16||^2 (0 where nothing is normalised).
enum { TF_FK = 0, TF_FQ = 1, TF_HK = 2, TF_HQ = 3, TF_PK = 4, TF_PQ = 5, TF_N = 6 };

constexpr int PREP_LD = 68;  // floats per row of the fp32 64 x 64 tiles

// The fp16 images are dead once their products are taken; the fp32 tiles L and Y take their place.
template <int DK>
constexpr int prep_smem() {
  constexpr int images = 2 * DR_C * DK * 2, tiles = 2 * DR_C * PREP_LD * 4;
  return (images > tiles ? images : tiles) + DR_C * 8 + 5 * DR_C * 4;
}

// Row scale (a power of two) of row `i`'s 64 floats at `p`, over both half-row threads.
__device__ __forceinline__ int half_row_exp(const float* p, int half) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + half * 32 + j);
    m = max_abs2(max_abs2(m, v.x, v.y), v.z, v.w);
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return row_exp(m, DR_ROW_EXP);
}

// Writes row i (this thread's half) of a 64 x 64 fp32 tile as fp16 hi and lo images.
__device__ __forceinline__ void store_half_row(const float* p, int i, int half, float s, uint8_t* hi, uint8_t* lo) {
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const float4 a = *reinterpret_cast<const float4*>(p + half * 32 + ch * 8);
    const float4 b = *reinterpret_cast<const float4*>(p + half * 32 + ch * 8 + 4);
    uint4 h, l;
    split2(a.x * s, a.y * s, h.x, l.x);
    split2(a.z * s, a.w * s, h.y, l.y);
    split2(b.x * s, b.y * s, h.z, l.z);
    split2(b.z * s, b.w * s, h.w, l.w);
    const uint32_t off = img_off(i, half * 4 + ch, 128);
    *reinterpret_cast<uint4*>(hi + off) = h;
    *reinterpret_cast<uint4*>(lo + off) = l;
  }
}

// (I + L beta) Y = -L for the strictly lower L, in 16 x 16 blocks (128 threads).  The diagonal blocks by
// forward substitution, a thread to a column; then, by their distance from the diagonal,
//     Y_ij = T + Y_ii beta_i T,   T = -L_ij - sum_{j <= k < i} L_ik beta_k Y_kj
// since (I + L_ii beta_i)^-1 = I + Y_ii beta_i.  Substitution over all 64 rows at once is a chain four times
// as long that only half of the threads share: 16,700 cycles a block against 6,700.
__device__ __forceinline__ void solve_y(const float* Lm, float* Ym, const float* bet, int tid) {
  if (tid < DR_C) {
    const int b0 = tid & ~15, cc = tid & 15;
    float w[16];  // beta_j Y_j of this column
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float* L = Lm + (b0 + r) * PREP_LD + b0;
      float s0 = -L[cc], s1 = 0.f;  // L is zero on and above the diagonal
#pragma unroll
      for (int j = 0; j < r; j += 4) {
        const float4 l = *reinterpret_cast<const float4*>(L + j);
        s0 -= l.x * w[j];
        if (j + 1 < r) s1 -= l.y * w[j + 1];
        if (j + 2 < r) s0 -= l.z * w[j + 2];
        if (j + 3 < r) s1 -= l.w * w[j + 3];
      }
      const float y = cc < r ? s0 + s1 : 0.f;
      w[r] = bet[b0 + r] * y;
      Ym[(b0 + r) * PREP_LD + tid] = y;
#pragma unroll
      for (int d = 16; d < DR_C; d += 16)  // P lay here: zero the blocks above the diagonal
        if (b0 >= d) Ym[(b0 - d + r) * PREP_LD + tid] = 0.f;
    }
  }
  const int r = tid >> 3, c2 = (tid & 7) * 2;  // this thread's row and two columns of each block
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    float2 v[3];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4 - d; ++n) {  // block (n + d, n)
      const float* L = Lm + ((n + d) * 16 + r) * PREP_LD;
      float2 s = *reinterpret_cast<const float2*>(L + n * 16 + c2);
      s.x = -s.x, s.y = -s.y;
#pragma unroll
      for (int k = 0; k < d; ++k)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int kj = (n + k) * 16 + j;
          const float4 l = *reinterpret_cast<const float4*>(L + kj);
          const float4 b = *reinterpret_cast<const float4*>(bet + kj);
          const float lb[4] = {l.x * b.x, l.y * b.y, l.z * b.z, l.w * b.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 y = *reinterpret_cast<const float2*>(Ym + (kj + q) * PREP_LD + n * 16 + c2);
            s.x -= lb[q] * y.x;
            s.y -= lb[q] * y.y;
          }
        }
      *reinterpret_cast<float2*>(Ym + ((n + d) * 16 + r) * PREP_LD + n * 16 + c2) = s;  // T
      v[n] = s;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4 - d; ++n) {
      const int i0 = (n + d) * 16;
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 l = *reinterpret_cast<const float4*>(Ym + (i0 + r) * PREP_LD + i0 + j);
        const float4 b = *reinterpret_cast<const float4*>(bet + i0 + j);
        const float lb[4] = {l.x * b.x, l.y * b.y, l.z * b.z, l.w * b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 y = *reinterpret_cast<const float2*>(Ym + (i0 + j + q) * PREP_LD + n * 16 + c2);
          v[n].x += lb[q] * y.x;
          v[n].y += lb[q] * y.y;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4 - d; ++n)
      *reinterpret_cast<float2*>(Ym + ((n + d) * 16 + r) * PREP_LD + n * 16 + c2) = v[n];
  }
}

template <int DK, bool BACK>
__global__ void __launch_bounds__(128, 4) k_delta_prep(const PrepArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int IMAGES = 2 * DR_C * DK * 2, TILES = 2 * DR_C * PREP_LD * 4;
  uint8_t* k16 = smem;
  uint8_t* q16 = k16 + DR_C * DK * 2;
  float* Lm = reinterpret_cast<float*>(smem);
  float* Ym = Lm + DR_C * PREP_LD;  // P first, then Y
  double* c = reinterpret_cast<double*>(smem + (IMAGES > TILES ? IMAGES : TILES));
  float* fk = reinterpret_cast<float*>(c + DR_C);
  float* fq = fk + DR_C;
  float* bet = fq + DR_C;
  float* rowm = bet + DR_C;  // [128] row maxima
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int ci = blockIdx.x, hq = blockIdx.y;
  pdl_wait();
  const DrChunk ch = a.chunks[ci];
  if (ch.len < 0) return;

  // the first value head's gates, read ahead
  const int rep = a.hv / a.hk;
  float g_next = 0.f, b_next = 0.f;
  const int64_t gate0 = (int64_t)(ch.tok + tid) * a.hv + hq * rep;
  if (tid < ch.len) {
    g_next = __ldg(a.g + gate0);
    b_next = __ldg(a.beta + gate0);
  }
  // token rows -> scaled fp16 images: LPR lanes to a row, BATCH rows of a lane group in flight, each step taken
  // for all of them before the next (the reductions' latency is what this phase costs)
  uint8_t* kq = a.kq + ((int64_t)ci * a.hk + hq) * (2 * DR_C * DK * 2);
  constexpr int LPR = DK <= 64 ? 8 : DK <= 128 ? 16 : 32, RPI = 32 / LPR, ITERS = 32 / RPI;
  constexpr int BATCH = ITERS < 8 ? ITERS : 8;
  const int rl = lane % LPR, rsub = lane / LPR;
#pragma unroll 1
  for (int b0 = 0; b0 < ITERS; b0 += BATCH) {
    uint4 raw[BATCH];
    float m[BATCH], ss[BATCH];
    // rows 0..63 are K's, 64..127 Q's; a warp has 32 rows of one of them
    const bool isq = warp >= 2;
    const int rb = (warp & 1) * 32 + b0 * RPI + rsub;
    const __nv_bfloat16* src = (isq ? a.Q + (int64_t)ch.tok * a.ldq : a.K + (int64_t)ch.tok * a.ldk) +
                               (int64_t)hq * a.dk + rl * 8;
    const int64_t ld = isq ? a.ldq : a.ldk;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int row = rb + b * RPI;
      raw[b] = make_uint4(0, 0, 0, 0);
      if (row < ch.len && rl * 8 < a.dk) raw[b] = __ldg(reinterpret_cast<const uint4*>(src + row * ld));
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      m[b] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = (&raw[b].x)[j];
        m[b] = max_abs2(m[b], __uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
      }
    }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1)
#pragma unroll
      for (int b = 0; b < BATCH; ++b) m[b] = fmaxf(m[b], __shfl_xor_sync(0xffffffffu, m[b], o));
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const float s = pow2i(row_exp(m[b], DR_TOK_EXP));
      ss[b] = 0.f;
      uint4 h;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = (&raw[b].x)[j];
        const float x = __uint_as_float(w << 16) * s, y = __uint_as_float(w & 0xffff0000u) * s;
        ss[b] += x * x + y * y;
        (&h.x)[j] = pack_f16x2(x, y);
      }
      if (rl * 8 < DK) {
        const uint32_t off = img_off(rb + b * RPI, rl, DK * 2);
        *reinterpret_cast<uint4*>((isq ? q16 : k16) + off) = h;
        *reinterpret_cast<uint4*>(kq + (isq ? DR_C * DK * 2 : 0) + off) = h;
      }
    }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1)
#pragma unroll
      for (int b = 0; b < BATCH; ++b) ss[b] += __shfl_xor_sync(0xffffffffu, ss[b], o);
    if (rl == 0)
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        rowm[(isq ? DR_C : 0) + rb + b * RPI] = m[b];
        fk[(isq ? DR_C : 0) + rb + b * RPI] = ss[b];
      }
  }
  __syncthreads();
  {
    // the rows' factors, one thread to a row: k^ = k / max(||k||, 1e-12) with ||k|| = 2^-e sqrt(ss)
    const bool isq = tid >= DR_C;
    const int row = tid & (DR_C - 1);
    const float mm = rowm[tid], ss = fk[tid];
    const int e = row_exp(mm, DR_TOK_EXP);
    const float inv = pow2i(-e), norm = sqrtf(ss);
    const bool normed = a.l2norm && norm * inv > 1e-12f;
    float f = normed ? 1.f / norm : a.l2norm ? inv * 1e12f : inv;
    if (isq) f *= a.scale;
    const float back = f * pow2i(e);  // 1 / max(||k||, 1e-12) (or 1), for the way back
    // a zero row has no scale to undo; its factor would only set the scale of what it is multiplied with
    if (row >= ch.len || mm == 0.f) f = 0.f;
    fk[tid] = f;  // (fq follows fk)
    if constexpr (BACK) {
      float* tf = a.tok + ((int64_t)ci * a.hk + hq) * TF_N * DR_C + row;
      tf[(isq ? TF_FQ : TF_FK) * DR_C] = f;
      tf[(isq ? TF_HQ : TF_HK) * DR_C] = back;
      tf[(isq ? TF_PQ : TF_PK) * DR_C] = normed ? 1.f / ss : 0.f;
    }
  }

  // K16 K16^T and Q16 K16^T on and below the diagonal; warp w has rows [16 w, 16 w + 16)
  float ak[8][4], aq[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) ak[n][j] = aq[n][j] = 0.f;
  {
    const uint32_t kb = smem_u32(k16), qb = smem_u32(q16);
#pragma unroll 2
    for (int kt = 0; kt < DK / 16; ++kt) {
      uint32_t fa[4], fb[4];
      ldsm4(fa, addr_bk(kb, lane, warp * 16, kt * 2, DK * 2));
      ldsm4(fb, addr_bk(qb, lane, warp * 16, kt * 2, DK * 2));
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np > warp) break;
        uint32_t b[4];
        ldsm4(b, addr_bn(kb, lane, np * 16, kt * 2, DK * 2));
        mma_f16(ak[2 * np], fa, b[0], b[1]);
        mma_f16(ak[2 * np + 1], fa, b[2], b[3]);
        mma_f16(aq[2 * np], fb, b[0], b[1]);
        mma_f16(aq[2 * np + 1], fb, b[2], b[3]);
      }
    }
  }

#pragma unroll 1
  for (int hr = 0; hr < rep; ++hr) {
    const int h = hq * rep + hr;
    uint8_t* blk = a.blk + ((int64_t)ci * a.hv + h) * DR_BLK;
    float* vec = reinterpret_cast<float*>(blk + DR_VEC);
    // c in 64 bits: the exponents reach hundreds below zero, and only their differences count
    // lower values than -400 (-inf: a reset) are taken as that, so that the sums of the tokens behind them keep their
    // digits: exp of it is zero in fp32 (below -104) even where gates behind it grow to fp32's largest (88)
    double s = g_next < -400.f ? -400.0 : (double)g_next;
    const float b_now = b_next;
    if (tid < ch.len && hr + 1 < rep) {
      g_next = __ldg(a.g + gate0 + hr + 1);
      b_next = __ldg(a.beta + gate0 + hr + 1);
    }
    if (tid < DR_C) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
    }
    __syncthreads();  // the images, or the tiles of the value head before, are read
    if (tid < DR_C) {
      c[tid] = s;
      bet[tid] = b_now;
    }
    __syncthreads();
    const double c31 = c[31];
    // L and P in the products' layout
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int i = warp * 16 + g + 8 * p;
      const double cii = c[i] + (i >= 32 ? c31 : 0.0);
      const float fki = fk[i], fqi = fq[i];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int j = n * 8 + 2 * t;
        float2 l = make_float2(0.f, 0.f), y = l;
        if (n * 8 <= warp * 16 + 15) {
          const double2 cj = *reinterpret_cast<const double2*>(c + j);
          const double base = n >= 4 ? c31 : 0.0;
          const float2 fj = *reinterpret_cast<const float2*>(fk + j);
          if (j <= i) {
            const float d = expf((float)(cii - (cj.x + base))) * fj.x;
            y.x = d * fqi * aq[n][2 * p];
            if (j < i) l.x = d * fki * ak[n][2 * p];
          }
          if (j + 1 <= i) {
            const float d = expf((float)(cii - (cj.y + base))) * fj.y;
            y.y = d * fqi * aq[n][2 * p + 1];
            if (j + 1 < i) l.y = d * fki * ak[n][2 * p + 1];
          }
        }
        *reinterpret_cast<float2*>(Lm + i * PREP_LD + j) = l;
        *reinterpret_cast<float2*>(Ym + i * PREP_LD + j) = y;
      }
    }
    __syncthreads();
    const int i = tid >> 1, half = tid & 1;
    {
      const float* P = Ym + i * PREP_LD;
      const int e = half_row_exp(P, half);
      store_half_row(P, i, half, pow2i(e), blk + DR_P, blk + DR_P + DR_TILE);
      if (!half) {
        const double G = c[DR_C - 1] + c31, cii = c[i] + (i >= 32 ? c31 : 0.0);
        const float ec = expf((float)cii), el = expf((float)(G - cii));
        const float fki = fk[i], fqi = fq[i];
        vec[DV_PS * DR_C + i] = pow2i(-e);
        vec[DV_AR * DR_C + i] = ec * fki;
        vec[DV_BETA * DR_C + i] = bet[i];
        vec[DV_AO * DR_C + i] = ec * fqi;
        vec[DV_AK * DR_C + i] = el * fki;
        vec[DV_EG * DR_C + i] = expf((float)G);
        vec[DV_C * DR_C + i] = (float)cii;
        vec[DV_CLO * DR_C + i] = (float)(cii - (double)(float)cii);
      }
    }
    __syncthreads();
    solve_y(Lm, Ym, bet, tid);
    __syncthreads();
    const int e = half_row_exp(Ym + i * PREP_LD, half);
    store_half_row(Ym + i * PREP_LD, i, half, pow2i(e), blk, blk + DR_TILE);
    if (!half) vec[DV_YS * DR_C + i] = pow2i(-e);
  }
  pdl_trigger();
}

// ---------------------------------------------------------------------------
// State pass: the recurrence over the chunks of a sequence.  The rows of S
// (value channels) do not meet, so a warp owns 16 of them and keeps them in
// registers for the whole sequence: S [16][dk] as accumulators is at once the A
// operand of S K^T, the errors R^T [16][64] that of (beta R)^T Y^T, the writes U^T
// that of U^T K and U^T P^T.  No row warp waits for another inside a chunk; shared
// memory holds only what all of them read (K16, Q16, Y, P), brought one to two
// chunks ahead by a warp of its own, or by the warps that make the outputs beside
// the chain (forward; they take S's parts and U from the row warps).
// Bound by the chain's latency: 6,900 cycles a chunk at dk = 128, 9,500 at 192, of
// which the row warp's and its output warp's 504 and 696 products are 4,000 and 5,600.
// (The outputs' share with one part of S, U and P each was 104 and 136 products fewer and
// the pass a tenth faster, 239 us for 265 of packed prompts; but an output whose terms cancel,
// as where a key is written again, then keeps 2^-11 of the terms instead of its own bits.)
//
// Few heads leave most SMs idle while a long sequence runs chunk by chunk.  S' is linear in S, so the sequence is
// then cut into segments: the scan pass runs each from a zero state (N, its end) and from the unit matrix without
// values (Phi, its transition, dk more rows of the same kind), the join pass chains S <- S Phi + N over the
// segments, and the state pass proper starts each segment from its own state.  2.6 times the products of one pass
// (dk = dv), on as many SMs as there are segments.
struct StateArgs {
  const __nv_bfloat16* V;
  __nv_bfloat16* O;
  int64_t ldv, ldo;
  const float* S0;
  float* S;
  int hk, hv, dk, dv;
  const DrSeq* seqs;
  const uint8_t* kq;
  const uint8_t* blk;
  Guard guard;
  // segments of cut sequences (the scan's seqs are those before a cut): [cut][hv][dv][dk] states at their starts and scan
  // results, [cut][hv] transitions (fp16 hi and lo images [DK][DK], rows scaled) and their rows' inverse scales
  // [cut][hv][DK]
  float *seg_s, *seg_n;
  uint8_t* phi;
  float* phi_scale;
  // backward pass: recompute the states, keep them and the errors, and sum dO . O
  const __nv_bfloat16* dO;  // rows of stride ldo
  float* keep_s;            // [chunk][hv][dv][dk]
  float* keep_e;            // [chunk][hv][dv][64] E^T
  float* w_part;            // [chunk][hv][dv / 16][64]
};

// A warp's V, dO or O tile: 64 token rows of 16 channels, 32 bytes each, the halves of rows 4..7 of every 8 swapped
// so that the 8 rows of an 8x8 tile lie in different banks.
constexpr int DR_VTILE = DR_C * 32;
__device__ __forceinline__ uint32_t vtile_off(int row, int half) {
  return (uint32_t)(row * 32 + ((half ^ ((row >> 2) & 1)) << 4));
}

enum { PASS_OUT = 0, PASS_BACK = 1, PASS_SCAN = 2 };  // what a state pass is for

// Outputs of their own warps where shared memory holds the hand-over (dk <= 192): per warp S's parts as A
// fragments with their row scales, U, and a tile for O.
template <int DK, int PASS>
constexpr bool state_split() {
  return PASS == PASS_OUT && DK <= 192;
}
template <int DK>
constexpr int state_hand() {
  return DK / 16 * 1024 + 256 + 4096 + DR_VTILE;
}
// A stage (two of them): K16, Q16 and the chunk's block; without Q16 and P in the scan, which has no outputs, and
// where the output warps keep those in one buffer of their own (they have the row warps' state update to refill it).
template <int DK, int PASS>
constexpr int state_stage() {
  return PASS == PASS_SCAN || state_split<DK, PASS>() ? DR_C * DK * 2 + DR_P : 2 * DR_C * DK * 2 + DR_BLK;
}
template <int DK, int PASS>
constexpr int state_obuf() {
  return state_split<DK, PASS>() ? DR_C * DK * 2 + 2 * DR_TILE : 0;
}
// per warp two V tiles, and two dO tiles for the backward pass
template <int PASS>
constexpr int state_warp_smem() {
  return (PASS == PASS_BACK ? 4 : 2) * DR_VTILE;
}
constexpr int DR_ETILE = 16 * DR_C * 4;  // a warp's E rows (reverse pass)
template <int DK, int PASS>
constexpr int state_smem(int warps, bool etile = false) {
  return 2 * state_stage<DK, PASS>() + state_obuf<DK, PASS>() + 64 +
         warps * (state_warp_smem<PASS>() + (etile ? DR_ETILE : 0) + (state_split<DK, PASS>() ? state_hand<DK>() + 32 : 0));
}
template <int DK, int PASS>
constexpr int state_threads() {  // at most four warps of rows, and as many for their outputs or one that copies
  return state_split<DK, PASS>() ? 256 : 160;  // (a ninth warp would leave 168 registers)
}

// A warp's 64 x 16 tile of token rows `p` (first channel v0 of head h), zero outside the sequence and the head.
__device__ __forceinline__ void load_vtile(uint32_t dst, const __nv_bfloat16* p, int64_t ld, const DrSeq& sq, int n,
                                           int col0, int v0, int dv, int lane) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int row = it * 16 + (lane >> 1), half = lane & 1;
    const int at = n * DR_C + row;
    const bool live = at < sq.len && v0 + half * 8 < dv;
    cp_async16(dst + vtile_off(row, half), live ? p + (int64_t)(sq.tok + at) * ld + col0 + v0 + half * 8 : p, live);
  }
}
// ... and its counterpart: a tile in shared memory -> token rows.
__device__ __forceinline__ void store_vtile(const uint8_t* src, __nv_bfloat16* p, int64_t ld, const DrSeq& sq, int n,
                                            int64_t col0, int v0, int dv, int lane) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int row = it * 16 + (lane >> 1), half = lane & 1;
    const int at = n * DR_C + row;
    if (at < sq.len && v0 + half * 8 < dv)
      *reinterpret_cast<uint4*>(p + (int64_t)(sq.tok + at) * ld + col0 + v0 + half * 8) =
          *reinterpret_cast<const uint4*>(src + vtile_off(row, half));
  }
}
// Address of 8x8 matrix lane/8 of token rows n0..n0+15 of such a tile: (tokens n0 + 8 (m / 2), channels 8 (m % 2));
// read with .trans it gives the accumulator layout of two neighbouring 8-token tiles (rows = channels).
__device__ __forceinline__ uint32_t vtile_addr(uint32_t base, int lane, int n0) {
  return base + vtile_off(n0 + ((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);
}

// x += P U in the accumulator layout (rows of U^T = r at scales w0, w1), all parts.
__device__ __forceinline__ void mul_pu(float (&x)[8][4], const float (&r)[8][4], float w0, float w1, uint32_t ph,
                                       uint32_t pl, int lane) {
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    uint32_t hi[4], lo[4];
    split_a(r[2 * kt], r[2 * kt + 1], w0, w1, hi, lo);
#pragma unroll
    for (int np = kt; np < 4; ++np) {
      uint32_t p[4];
      ldsm4(p, addr_bn(ph, lane, np * 16, kt * 2, 128));
      mma_f16(x[2 * np], hi, p[0], p[1]);
      mma_f16(x[2 * np + 1], hi, p[2], p[3]);
      mma_f16(x[2 * np], lo, p[0], p[1]);
      mma_f16(x[2 * np + 1], lo, p[2], p[3]);
      ldsm4(p, addr_bn(pl, lane, np * 16, kt * 2, 128));
      mma_f16(x[2 * np], hi, p[0], p[1]);
      mma_f16(x[2 * np + 1], hi, p[2], p[3]);
    }
  }
}

// O's tile in the accumulator layout, o (Q S^T at scales is) and x (P U at scales iu), to the rows of a tile.
__device__ __forceinline__ void store_o(const float (&o)[8][4], const float (&x)[8][4], float is0, float is1, float iu0,
                                        float iu1, const float* vec, uint32_t tile, int lane) {
  const int t = lane & 3;
#pragma unroll
  for (int np = 0; np < 4; ++np) {
    uint32_t y[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 2 * np + q, col = k * 8 + 2 * t;
      const float2 ao = *reinterpret_cast<const float2*>(vec + DV_AO * DR_C + col);
      const float2 ps = *reinterpret_cast<const float2*>(vec + DV_PS * DR_C + col);
      y[2 * q] = pack_bf16x2(ao.x * (o[k][0] * is0) + ps.x * (x[k][0] * iu0),
                             ao.y * (o[k][1] * is0) + ps.y * (x[k][1] * iu0));
      y[2 * q + 1] = pack_bf16x2(ao.x * (o[k][2] * is1) + ps.x * (x[k][2] * iu1),
                                 ao.y * (o[k][3] * is1) + ps.y * (x[k][3] * iu1));
    }
    stsm4t(vtile_addr(tile, lane, np * 16), y[0], y[1], y[2], y[3]);
  }
}

// A warp's 16 rows of dk floats, rows scaled back, to `out`; `rows` of them exist.
template <int NT>
__device__ __forceinline__ void store_rows(float* out, const float (&s)[NT][4], float i0, float i1, int rows, int dk,
                                           int lane) {
  const int g = lane >> 2, t = lane & 3;
  float* p0 = out + (int64_t)g * dk + 2 * t;
  float* p1 = p0 + 8 * (int64_t)dk;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n * 8 + 8 > dk) break;  // (dk is a multiple of 8)
    if (g < rows) *reinterpret_cast<float2*>(p0 + n * 8) = make_float2(s[n][0] * i0, s[n][1] * i0);
    if (g + 8 < rows) *reinterpret_cast<float2*>(p1 + n * 8) = make_float2(s[n][2] * i1, s[n][3] * i1);
  }
}

// Column of an even token index in a row of the kept E: pairs are permuted by the row (mod 8), so that 8 rows' pairs
// lie in different banks once a tile is copied to shared memory as it is.
__device__ __forceinline__ int etile_col(int row, int col) { return (((col >> 1) ^ ((row & 7) << 2)) << 1) | (col & 1); }

template <int DK, int PASS>
__global__ void __launch_bounds__(state_threads<DK, PASS>(), 1) k_delta_state(const StateArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr bool BACK = PASS == PASS_BACK, SCAN = PASS == PASS_SCAN, SPLIT = state_split<DK, PASS>();
  constexpr int STAGE = state_stage<DK, PASS>();
  constexpr int KB = DR_C * DK * 2;                  // bytes of K16, and of Q16
  constexpr int YB = SPLIT || SCAN ? KB : 2 * KB;    // offset of Y in a stage
  constexpr int TILES = 2 * STAGE + state_obuf<DK, PASS>();  // offset of the warps' tiles
  constexpr int WSM = state_warp_smem<PASS>();
  constexpr int NT = DK / 8;
  const int tid = threadIdx.x, lane = tid & 31;
  const int nwarp = SPLIT ? blockDim.x >> 6 : (blockDim.x >> 5) - 1;  // warps that own rows
  const bool outer = SPLIT && tid >> 5 >= nwarp;
  const int warp = outer ? (tid >> 5) - nwarp : tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* vbuf = smem + TILES + warp * WSM;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + TILES + nwarp * WSM);  // [2] stage and tiles have landed
  uint64_t* empty = full + 2;                                                // [2] every warp has read them
  uint64_t *ofull = full + 4, *oempty = full + 5;  // the output warps' Q16 and P have landed, every one has read them
  // hand-over from a row warp to its output warp: S's parts written, read, U written, read
  uint64_t* hand = full + 6 + 4 * warp;
  uint8_t* hbuf = smem + TILES + nwarp * (WSM + 32) + 64 + warp * state_hand<DK>();
  uint4* h_s = reinterpret_cast<uint4*>(hbuf);  // [dk / 16][hi, lo][32]
  float4* h_u = reinterpret_cast<float4*>(h_s + DK / 16 * 64);
  float2* h_ss = reinterpret_cast<float2*>(h_u + 8 * 32);
  uint8_t* obuf = reinterpret_cast<uint8_t*>(h_ss + 32);
  const int nblocks = (a.dv + nwarp * 16 - 1) / (nwarp * 16);
  const int vblocks = nblocks + (SCAN ? (DK + nwarp * 16 - 1) / (nwarp * 16) : 0);
  const int h = blockIdx.x / vblocks % a.hv, hq = h / (a.hv / a.hk);
  const int vb0 = blockIdx.x % vblocks;
  const bool phi = SCAN && vb0 >= nblocks;  // rows of the transition instead of value channels
  const int vfirst = (phi ? vb0 - nblocks : vb0) * nwarp * 16;
  const int v0 = vfirst + warp * 16;  // first row of this warp (may lie past the end)
  const int dv_in = phi ? 0 : a.dv;  // the transition's rows take no values
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1 + 32 * (SPLIT ? nwarp : 1));  // the bulk copies, and each copying lane's tile copies
      mbar_init(&empty[i], nwarp * (SPLIT ? 2 : 1));
    }
    if (SPLIT) {
      mbar_init(ofull, 1);
      mbar_init(oempty, nwarp);
      for (int i = 0; i < 4 * nwarp; ++i) mbar_init(&full[6 + i], 1);
    }
    fence_mbar_init();
  }
  pdl_wait();
  const int si = blockIdx.x / (vblocks * a.hv);
  const DrSeq sq = a.seqs[si];
  __syncthreads();
  if (sq.len < 0) return;
  if (phi && sq.seg == 0) return;  // a first segment's transition has no use (nor has a last one's scan)
  const int nchunk = (sq.len + DR_C - 1) / DR_C;

  auto load_stage = [&](int n) {  // one thread: the chunk's shared operands
    uint64_t* bar = &full[n & 1];
    const int64_t ci = sq.chunk0 + n;
    uint8_t* st = smem + (n & 1) * STAGE;
    mbar_expect_tx(bar, STAGE);
    bulk_load(st, a.kq + (ci * a.hk + hq) * 2 * KB, YB, bar);
    bulk_load(st + YB, a.blk + (ci * a.hv + h) * DR_BLK, STAGE - YB, bar);
  };
  auto load_tiles = [&](int n, int w) {  // one warp: row warp w's tiles
    const uint32_t dst = smem_u32(smem + TILES + w * WSM + (n & 1) * DR_VTILE);
    load_vtile(dst, a.V, a.ldv, sq, n, h * a.dv, vfirst + w * 16, dv_in, lane);
    if constexpr (BACK) load_vtile(dst + 2 * DR_VTILE, a.dO, a.ldo, sq, n, h * a.dv, vfirst + w * 16, dv_in, lane);
  };
  if (!SPLIT && warp == nwarp) {  // the last warp brings the chunks, two ahead at most
#pragma unroll 1
    for (int n = 0; n < nchunk; ++n) {
      if (n >= 2) mbar_wait(&empty[n & 1], ((n >> 1) - 1) & 1, a.guard);
      if (lane == 0) load_stage(n);
      for (int w = 0; w < nwarp; ++w) load_tiles(n, w);
      cp_arrive(&full[n & 1]);
    }
    return;
  }

  if constexpr (SPLIT) {
    if (outer) {
      // O = e^c Q S^T + P U beside the row warp's chain, from both parts of S, U and P: what is read from the state and
      // what is written over it can cancel; and the next chunk's copies, once every warp is done with the stage
      auto copy = [&](int n) {
        if (warp == 0 && lane == 0) load_stage(n);
        load_tiles(n, warp);
        cp_arrive(&full[n & 1]);
      };
      uint8_t* ob = smem + 2 * STAGE;
      const uint32_t qb = smem_u32(ob), ph = qb + KB, pl = ph + DR_TILE;
      auto copy_o = [&](int n) {
        const int64_t ci = sq.chunk0 + n;
        mbar_expect_tx(ofull, KB + 2 * DR_TILE);
        bulk_load(ob, a.kq + (ci * a.hk + hq) * 2 * KB + KB, KB, ofull);
        bulk_load(ob + KB, a.blk + (ci * a.hv + h) * DR_BLK + DR_P, 2 * DR_TILE, ofull);
      };
      if (nchunk > 0) {
        copy(0);
        if (warp == 0 && lane == 0) copy_o(0);
      }
#pragma unroll 1
      for (int n = 0; n < nchunk; ++n) {
        if (warp == 0 && n > 0) {
          mbar_wait(oempty, (n - 1) & 1, a.guard);
          if (lane == 0) copy_o(n);
        }
        if (n + 1 < nchunk) {
          if (n > 0) mbar_wait(&empty[(n + 1) & 1], ((n - 1) >> 1) & 1, a.guard);
          copy(n + 1);
        }
        mbar_wait(&full[n & 1], (n >> 1) & 1, a.guard);
        mbar_wait(ofull, n & 1, a.guard);
        const float* vec = reinterpret_cast<const float*>(smem + (n & 1) * STAGE + YB + DR_VEC);
        float o[8][4], x[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[k][j] = x[k][j] = 0.f;
        mbar_wait(&hand[0], n & 1, a.guard);
        const float2 is = h_ss[lane];
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
          const uint4 v = h_s[kt * 64 + lane], w = h_s[kt * 64 + 32 + lane];
          const uint32_t hi[4] = {v.x, v.y, v.z, v.w}, lo[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int np = 0; np < 4; np += 2) {
            uint32_t c[2][4];
            ldsm4(c[0], addr_bn(qb, lane, np * 16, kt * 2, DK * 2));
            ldsm4(c[1], addr_bn(qb, lane, np * 16 + 16, kt * 2, DK * 2));
            mma_f16x4(o + 2 * np, hi, c);
            mma_f16x4(o + 2 * np, lo, c);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&hand[1]);
        mbar_wait(&hand[2], n & 1, a.guard);
        float r[8][4], m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 v = h_u[k * 32 + lane];
          r[k][0] = v.x, r[k][1] = v.y, r[k][2] = v.z, r[k][3] = v.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&hand[3]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m0 = max_abs2(m0, r[k][0], r[k][1]);
          m1 = max_abs2(m1, r[k][2], r[k][3]);
        }
        const int f0 = row_exp(quad_max(m0), DR_ROW_EXP), f1 = row_exp(quad_max(m1), DR_ROW_EXP);
        mul_pu(x, r, pow2i(f0), pow2i(f1), ph, pl, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty);
        store_o(o, x, is.x, is.y, pow2i(-f0), pow2i(-f1), vec, smem_u32(obuf), lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[n & 1]);
        store_vtile(obuf, a.O, a.ldo, sq, n, (int64_t)h * a.dv, v0, a.dv, lane);
        __syncwarp();  // the tile is read
      }
      return;
    }
  }

  float s[NT][4];
  const int64_t srow = ((int64_t)sq.id * a.hv + h) * a.dv, grow = ((int64_t)sq.cut * a.hv + h) * a.dv;
  // a first segment starts from S0 (which the scan keeps: S may be S0, and a last segment may end before the first one
  // starts), the others from the join's state, or in the scan from zero or the unit matrix
  const float* from = sq.nseg > 1 && !SCAN ? a.seg_s + grow * a.dk
                      : sq.seg == 0        ? (a.S0 ? a.S0 + srow * a.dk : nullptr)
                                           : nullptr;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = v0 + g + 8 * p, col = n * 8 + 2 * t;
      float2 x = make_float2(0.f, 0.f);
      if (phi) {
        if (r < a.dk) x = make_float2(col == r ? 1.f : 0.f, col + 1 == r ? 1.f : 0.f);
      } else if (from && r < a.dv && col < a.dk) {
        x = *reinterpret_cast<const float2*>(from + (int64_t)r * a.dk + col);
      }
      s[n][2 * p] = x.x;
      s[n][2 * p + 1] = x.y;
    }
  float inv0 = 1.f, inv1 = 1.f;  // S = s * inv: rows g and g + 8 carry a power of two
  if (SCAN && sq.seg == 0) store_rows<NT>(a.seg_s + (grow + v0) * a.dk, s, 1.f, 1.f, a.dv - v0, a.dk, lane);

#pragma unroll 1
  for (int n = 0; n < nchunk; ++n) {
    // a wait that gives up records the error; the pass then runs on (bounded) with what the stage holds
    mbar_wait(&full[n & 1], (n >> 1) & 1, a.guard);
    const uint32_t st = smem_u32(smem + (n & 1) * STAGE);
    const uint32_t kb = st, qb = st + KB, yh = st + YB, yl = yh + DR_TILE, ph = yh + DR_P, pl = ph + DR_TILE;
    const float* vec = reinterpret_cast<const float*>(smem + (n & 1) * STAGE + YB + DR_VEC);
    const uint32_t vb = smem_u32(vbuf + (n & 1) * DR_VTILE);
    const int64_t blk = (int64_t)(sq.chunk0 + n) * a.hv + h;  // this chunk's block of the kept arrays

    if constexpr (BACK) {
      store_rows<NT>(a.keep_s + (blk * a.dv + v0) * a.dk, s, inv0, inv1, a.dv - v0, a.dk, lane);
    }
    // S K^T and S Q^T
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      m0 = max_abs2(m0, s[k][0], s[k][1]);
      m1 = max_abs2(m1, s[k][2], s[k][3]);
    }
    const int e0 = row_exp(quad_max(m0), DR_ROW_EXP), e1 = row_exp(quad_max(m1), DR_ROW_EXP);
    const float sc0 = pow2i(e0), sc1 = pow2i(e1);
    float r[8][4], o[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k][j] = o[k][j] = 0.f;
    if (SPLIT && n > 0) mbar_wait(&hand[1], (n - 1) & 1, a.guard);  // the output warp has read the S before
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
      uint32_t hi[4], lo[4];
      split_a(s[2 * kt], s[2 * kt + 1], sc0, sc1, hi, lo);
      if constexpr (SPLIT) {
        h_s[kt * 64 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        h_s[kt * 64 + 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
#pragma unroll
      for (int np = 0; np < 4; np += 2) {
        uint32_t b[2][4], c[2][4];
        ldsm4(b[0], addr_bn(kb, lane, np * 16, kt * 2, DK * 2));
        ldsm4(b[1], addr_bn(kb, lane, np * 16 + 16, kt * 2, DK * 2));
        mma_f16x4(r + 2 * np, hi, b);
        if constexpr (!SCAN && !SPLIT) {
          ldsm4(c[0], addr_bn(qb, lane, np * 16, kt * 2, DK * 2));
          ldsm4(c[1], addr_bn(qb, lane, np * 16 + 16, kt * 2, DK * 2));
          mma_f16x4(o + 2 * np, hi, c);
        }
        mma_f16x4(r + 2 * np, lo, b);
        if constexpr (!SCAN && !SPLIT) mma_f16x4(o + 2 * np, lo, c);
      }
    }
    // R = V - e^c K S^T, then the scale of beta R
    const float is0 = inv0 * pow2i(-e0), is1 = inv1 * pow2i(-e1);
    if constexpr (SPLIT) {
      h_ss[lane] = make_float2(is0, is1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&hand[0]);
    }
    m0 = m1 = 0.f;
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t v[4];
      ldsm4t(v, vtile_addr(vb, lane, np * 16));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = 2 * np + q, col = k * 8 + 2 * t;
        const float2 ar = *reinterpret_cast<const float2*>(vec + DV_AR * DR_C + col);
        const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + col);
        const uint32_t x0 = v[2 * q], x1 = v[2 * q + 1];
        r[k][0] = __uint_as_float(x0 << 16) - ar.x * (r[k][0] * is0);
        r[k][1] = __uint_as_float(x0 & 0xffff0000u) - ar.y * (r[k][1] * is0);
        r[k][2] = __uint_as_float(x1 << 16) - ar.x * (r[k][2] * is1);
        r[k][3] = __uint_as_float(x1 & 0xffff0000u) - ar.y * (r[k][3] * is1);
        m0 = max_abs2(m0, be.x * r[k][0], be.y * r[k][1]);
        m1 = max_abs2(m1, be.x * r[k][2], be.y * r[k][3]);
      }
    }
    // E = R + Y (beta R); the diagonal is not part of Y, so only tiles with i >= j
    {
      const int f0 = row_exp(quad_max(m0), DR_ROW_EXP), f1 = row_exp(quad_max(m1), DR_ROW_EXP);
      const float w0 = pow2i(f0), w1 = pow2i(f1);
      float x[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = 0.f;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        float b0[4], b1[4];
        const float2 ba = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + kt * 16 + 2 * t);
        const float2 bb = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + kt * 16 + 8 + 2 * t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b0[j] = r[2 * kt][j] * (j & 1 ? ba.y : ba.x);
          b1[j] = r[2 * kt + 1][j] * (j & 1 ? bb.y : bb.x);
        }
        uint32_t hi[4], lo[4];
        split_a(b0, b1, w0, w1, hi, lo);
#pragma unroll
        for (int np = kt; np < 4; ++np) {
          uint32_t y[4];
          ldsm4(y, addr_bn(yh, lane, np * 16, kt * 2, 128));
          mma_f16(x[2 * np], hi, y[0], y[1]);
          mma_f16(x[2 * np + 1], hi, y[2], y[3]);
          mma_f16(x[2 * np], lo, y[0], y[1]);
          mma_f16(x[2 * np + 1], lo, y[2], y[3]);
          ldsm4(y, addr_bn(yl, lane, np * 16, kt * 2, 128));
          mma_f16(x[2 * np], hi, y[0], y[1]);
          mma_f16(x[2 * np + 1], hi, y[2], y[3]);
        }
      }
      const float i0 = pow2i(-f0), i1 = pow2i(-f1);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = k * 8 + 2 * t;
        const float2 ys = *reinterpret_cast<const float2*>(vec + DV_YS * DR_C + col);
        const float2 be = *reinterpret_cast<const float2*>(vec + DV_BETA * DR_C + col);
        r[k][0] = r[k][0] + ys.x * (x[k][0] * i0);
        r[k][1] = r[k][1] + ys.y * (x[k][1] * i0);
        r[k][2] = r[k][2] + ys.x * (x[k][2] * i1);
        r[k][3] = r[k][3] + ys.y * (x[k][3] * i1);
        if constexpr (BACK) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (v0 + g + 8 * p < a.dv)
              *reinterpret_cast<float2*>(a.keep_e + (blk * a.dv + v0 + g + 8 * p) * DR_C + etile_col(g, col)) =
                  make_float2(r[k][2 * p], r[k][2 * p + 1]);
        }
        r[k][0] *= be.x;  // r becomes U
        r[k][1] *= be.y;
        r[k][2] *= be.x;
        r[k][3] *= be.y;
      }
    }
    if constexpr (SPLIT) {  // U for the output warp
      if (n > 0) mbar_wait(&hand[3], (n - 1) & 1, a.guard);
#pragma unroll
      for (int k = 0; k < 8; ++k) h_u[k * 32 + lane] = make_float4(r[k][0], r[k][1], r[k][2], r[k][3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&hand[2]);
    }
    // O = e^c Q S^T + P U, accumulated in U's scale over P's row scales
    if constexpr (!SCAN && !SPLIT) {
      m0 = m1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m0 = max_abs2(m0, r[k][0], r[k][1]);
        m1 = max_abs2(m1, r[k][2], r[k][3]);
      }
      const int f0 = row_exp(quad_max(m0), DR_ROW_EXP), f1 = row_exp(quad_max(m1), DR_ROW_EXP);
      const float w0 = pow2i(f0), w1 = pow2i(f1), i0 = pow2i(-f0), i1 = pow2i(-f1);
      float x[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = 0.f;
      mul_pu(x, r, w0, w1, ph, pl, lane);
      if constexpr (BACK) {  // this warp's part of dO . O for each token
        const uint32_t db = smem_u32(vbuf + (2 + (n & 1)) * DR_VTILE);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t d[4];
          ldsm4t(d, vtile_addr(db, lane, np * 16));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int k = 2 * np + q, col = k * 8 + 2 * t;
            const float2 ao = *reinterpret_cast<const float2*>(vec + DV_AO * DR_C + col);
            const float2 ps = *reinterpret_cast<const float2*>(vec + DV_PS * DR_C + col);
            const uint32_t d0 = d[2 * q], d1 = d[2 * q + 1];
            float sx = (ao.x * (o[k][0] * is0) + ps.x * (x[k][0] * i0)) * __uint_as_float(d0 << 16) +
                       (ao.x * (o[k][2] * is1) + ps.x * (x[k][2] * i1)) * __uint_as_float(d1 << 16);
            float sy = (ao.y * (o[k][1] * is0) + ps.y * (x[k][1] * i0)) * __uint_as_float(d0 & 0xffff0000u) +
                       (ao.y * (o[k][3] * is1) + ps.y * (x[k][3] * i1)) * __uint_as_float(d1 & 0xffff0000u);
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) {
              sx += __shfl_xor_sync(0xffffffffu, sx, m);
              sy += __shfl_xor_sync(0xffffffffu, sy, m);
            }
            if (g == 0 && v0 < a.dv)
              *reinterpret_cast<float2*>(a.w_part + (blk * ((a.dv + 15) / 16) + v0 / 16) * DR_C + col) =
                  make_float2(sx, sy);
          }
        }
      } else {
        __syncwarp();  // every lane has read its V tile; O takes its place
        store_o(o, x, is0, is1, i0, i1, vec, vb, lane);
        __syncwarp();
        store_vtile(vbuf + (n & 1) * DR_VTILE, a.O, a.ldo, sq, n, (int64_t)h * a.dv, v0, a.dv, lane);
      }
    }
    // S' = e^{c_C} S + (e^{c_C - c} U)^T K, with S brought to the scale of the added term
    {
      m0 = m1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 ak = *reinterpret_cast<const float2*>(vec + DV_AK * DR_C + k * 8 + 2 * t);
        r[k][0] *= ak.x;
        r[k][1] *= ak.y;
        r[k][2] *= ak.x;
        r[k][3] *= ak.y;
        m0 = max_abs2(m0, r[k][0], r[k][1]);
        m1 = max_abs2(m1, r[k][2], r[k][3]);
      }
      // (a state far larger than what is added bounds the scale, so that it cannot overflow)
      const int f0 = min(row_exp(quad_max(m0), DR_ROW_EXP), 87 - exp_of(is0));
      const int f1 = min(row_exp(quad_max(m1), DR_ROW_EXP), 87 - exp_of(is1));
      const float w0 = pow2i(f0), w1 = pow2i(f1);
      const float eg = vec[DV_EG * DR_C];
      const float d0 = eg * inv0 * w0, d1 = eg * inv1 * w1;
      inv0 = pow2i(-f0);
      inv1 = pow2i(-f1);
      uint32_t hi[4][4], lo[4][4];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) split_a(r[2 * kt], r[2 * kt + 1], w0, w1, hi[kt], lo[kt]);
      // The products have accumulators of their own: the tensor cores cut off what falls below the sum, and S, which
      // is carried over all chunks, takes the result with one rounding to nearest.
#pragma unroll
      for (int np = 0; np < DK / 16; np += 2) {
        float acc[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[k][j] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          uint32_t b[2][4];
          ldsm4t(b[0], addr_bk(kb, lane, kt * 16, np * 2, DK * 2));
          ldsm4t(b[1], addr_bk(kb, lane, kt * 16, np * 2 + 2, DK * 2));
          mma_f16x4(acc, lo[kt], b);
          mma_f16x4(acc, hi[kt], b);
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
    if (lane == 0) mbar_arrive(&empty[n & 1]);  // this warp has read the stage and its tiles
  }
  if (phi) {  // Phi as split images, each row at its own scale
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m0 = max_abs2(m0, s[n][0], s[n][1]);
      m1 = max_abs2(m1, s[n][2], s[n][3]);
    }
    const int e0 = row_exp(quad_max(m0), DR_ROW_EXP), e1 = row_exp(quad_max(m1), DR_ROW_EXP);
    if (v0 < DK) {
      uint8_t* img = a.phi + ((int64_t)sq.cut * a.hv + h) * (2 * DK * DK * 2);
      float* sc = a.phi_scale + ((int64_t)sq.cut * a.hv + h) * DK;
      if (t == 0) {
        sc[v0 + g] = inv0 * pow2i(-e0);
        sc[v0 + g + 8] = inv1 * pow2i(-e1);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t hi, lo;
          const float w = pow2i(p ? e1 : e0);
          split2(s[n][2 * p] * w, s[n][2 * p + 1] * w, hi, lo);
          const uint32_t off = img_off(v0 + g + 8 * p, n, DK * 2) + 4 * t;
          *reinterpret_cast<uint32_t*>(img + off) = hi;
          *reinterpret_cast<uint32_t*>(img + DK * DK * 2 + off) = lo;
        }
    }
    return;
  }
  // the state after the sequence; in the scan, the start of the second segment or what a segment adds
  float* to = a.S ? a.S + srow * a.dk : nullptr;
  if (SCAN) to = sq.seg == 0 ? a.seg_s + (grow + (int64_t)a.hv * a.dv) * a.dk : a.seg_n + grow * a.dk;
  else if (sq.seg < sq.nseg - 1) to = nullptr;
  if (to) store_rows<NT>(to + (int64_t)v0 * a.dk, s, inv0, inv1, a.dv - v0, a.dk, lane);
}

// ---------------------------------------------------------------------------
// Join pass: the states at the segments' starts, from what the scan left,
//     S_{k+1} = S_k Phi_k + N_k                (state pass)
//     dS_{k-1} = dS_k Phi_k^T + N'_k           (REVERSE: gradient at the segments' ends)
// A warp owns 16 rows and keeps them in registers over the segments; Phi comes in blocks of 64 rows
// (of 64 columns of its transpose: the same bytes' rows hold them) through a ring of two stages, and what a
// segment adds is copied in while its products run: nothing in a step waits for a load of its own.
struct JoinArgs {
  const DrSeq* seqs;   // the segments before a cut
  int hv, dk, dv;
  float* seg_s;        // [cut][hv][dv][dk]: start states, or gradients at the ends
  const float* seg_n;  // what each segment adds
  const uint8_t* phi;
  const float* phi_scale;
  Guard guard;
};

template <int DK>
constexpr int join_smem() {
  return 2 * 2 * DR_C * DK * 2 + 2 * DK * 4 + DR_C * DK * 4 + 64;
}

template <int DK, bool REVERSE>
__global__ void __launch_bounds__(128, 1) k_delta_join(const JoinArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NT = DK / 8, KB = DK / DR_C, BLK = DR_C * DK * 2;  // BLK: bytes of 64 rows of an image
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  float* scale = reinterpret_cast<float*>(smem + 4 * BLK);  // [2][DK] inverse row scales of Phi, by segment parity
  float* add = scale + 2 * DK;  // [64][dk] N of the step
  uint64_t* full = reinterpret_cast<uint64_t*>(add + DR_C * DK);  // [2] ring, [1] N
  const int vblocks = (a.dv + 63) / 64;
  const int h = blockIdx.x / vblocks % a.hv, row0 = blockIdx.x % vblocks * 64, v0 = row0 + warp * 16;
  const uint32_t add_bytes = min(64, a.dv - row0) * a.dk * 4;
  const int si = blockIdx.x / (vblocks * a.hv);
  if (tid == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    mbar_init(&full[2], 1);
    fence_mbar_init();
  }
  pdl_wait();
  const DrSeq sq = a.seqs[si];
  __syncthreads();
  if (sq.len < 0 || sq.seg != 0 || sq.nseg < 3) return;
  const int steps = sq.nseg - 2, total = steps * KB;  // segments 1 .. nseg - 2, in this order or from the last
  auto seg_of = [&](int q) { return sq.cut + (REVERSE ? sq.nseg - 2 - q : 1 + q); };
  auto load = [&](int q) {  // one thread: 64 rows of Phi, hi and lo
    const uint8_t* img = a.phi + ((int64_t)seg_of(q / KB) * a.hv + h) * (2 * DK * DK * 2) + q % KB * BLK;
    uint8_t* st = smem + (q & 1) * 2 * BLK;
    const bool first = q % KB == 0;  // the step's row scales come with its first block
    mbar_expect_tx(&full[q & 1], 2 * BLK + (first ? DK * 4 : 0));
    bulk_load(st, img, BLK, &full[q & 1]);
    bulk_load(st + BLK, img + DK * DK * 2, BLK, &full[q & 1]);
    if (first)
      bulk_load(scale + (q / KB & 1) * DK, a.phi_scale + ((int64_t)seg_of(q / KB) * a.hv + h) * DK, DK * 4,
                &full[q & 1]);
  };
  float s[NT][4];
  auto rows = [&](float* base, int seg, int n, int p) {  // this thread's pair of row 8 p, tile n; null past the end
    const int r = v0 + g + 8 * p, col = n * 8 + 2 * t;
    return r < a.dv && col < a.dk ? base + (((int64_t)seg * a.hv + h) * a.dv + r) * a.dk + col : nullptr;
  };
  auto load_s = [&](int seg) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float* x = rows(a.seg_s, seg, n, p);
        const float2 v = x ? *reinterpret_cast<const float2*>(x) : make_float2(0.f, 0.f);
        s[n][2 * p] = v.x;
        s[n][2 * p + 1] = v.y;
      }
  };
  load_s(REVERSE ? sq.cut + sq.nseg - 2 : sq.cut + 1);
  if (tid == 0) load(0);
#pragma unroll 1
  for (int q = 0; q < steps; ++q) {
    const int seg = seg_of(q), to = REVERSE ? seg - 1 : seg + 1;
    const float* sc = scale + (q & 1) * DK;
    if (tid == 0) {
      mbar_expect_tx(&full[2], add_bytes);
      bulk_load(add, a.seg_n + (((int64_t)seg * a.hv + h) * a.dv + row0) * a.dk, add_bytes, &full[2]);
    }
    mbar_wait(&full[(q * KB) & 1], ((q * KB) >> 1) & 1, a.guard);
    // forward: Phi's row scales meet S's columns; reverse: the result's columns
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (!REVERSE) {
        const float2 f = *reinterpret_cast<const float2*>(sc + n * 8 + 2 * t);
        s[n][0] *= f.x, s[n][1] *= f.y, s[n][2] *= f.x, s[n][3] *= f.y;
      }
      m0 = max_abs2(m0, s[n][0], s[n][1]);
      m1 = max_abs2(m1, s[n][2], s[n][3]);
    }
    const int e0 = row_exp(quad_max(m0), DR_ROW_EXP), e1 = row_exp(quad_max(m1), DR_ROW_EXP);
    const float w0 = pow2i(e0), w1 = pow2i(e1), i0 = pow2i(-e0), i1 = pow2i(-e1);
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int at = q * KB + kb;
      if (tid == 0 && at + 1 < total) load(at + 1);
      mbar_wait(&full[at & 1], (at >> 1) & 1, a.guard);
      const uint32_t ph = smem_u32(smem + (at & 1) * 2 * BLK), pl = ph + BLK;
      if constexpr (!REVERSE) {  // rows kb 64.. of Phi: 64 of the sum's terms, all columns
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kt = kb * 4 + k4;
          uint32_t hi[4], lo[4];
          split_a(s[2 * kt], s[2 * kt + 1], w0, w1, hi, lo);
#pragma unroll
          for (int np = 0; np < DK / 16; np += 2) {
            uint32_t b[2][4], c[2][4];
            ldsm4t(b[0], addr_bk(ph, lane, k4 * 16, np * 2, DK * 2));
            ldsm4t(b[1], addr_bk(ph, lane, k4 * 16, np * 2 + 2, DK * 2));
            ldsm4t(c[0], addr_bk(pl, lane, k4 * 16, np * 2, DK * 2));
            ldsm4t(c[1], addr_bk(pl, lane, k4 * 16, np * 2 + 2, DK * 2));
            mma_f16x4(acc + 2 * np, hi, b);
            mma_f16x4(acc + 2 * np, lo, b);
            mma_f16x4(acc + 2 * np, hi, c);
          }
        }
      } else {  // rows kb 64.. of Phi are these columns of the result: all terms
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
          uint32_t hi[4], lo[4];
          split_a(s[2 * kt], s[2 * kt + 1], w0, w1, hi, lo);
#pragma unroll
          for (int np = 0; np < 4; np += 2) {
            uint32_t b[2][4], c[2][4];
            ldsm4(b[0], addr_bn(ph, lane, np * 16, kt * 2, DK * 2));
            ldsm4(b[1], addr_bn(ph, lane, np * 16 + 16, kt * 2, DK * 2));
            ldsm4(c[0], addr_bn(pl, lane, np * 16, kt * 2, DK * 2));
            ldsm4(c[1], addr_bn(pl, lane, np * 16 + 16, kt * 2, DK * 2));
            mma_f16x4(acc + kb * 8 + 2 * np, hi, b);
            mma_f16x4(acc + kb * 8 + 2 * np, lo, b);
            mma_f16x4(acc + kb * 8 + 2 * np, hi, c);
          }
        }
      }
      __syncthreads();  // the stage is read
    }
    mbar_wait(&full[2], q & 1, a.guard);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 f = REVERSE ? *reinterpret_cast<const float2*>(sc + n * 8 + 2 * t) : make_float2(1.f, 1.f);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float i = p ? i1 : i0;
        const int r = v0 + g + 8 * p, col = n * 8 + 2 * t;
        const float2 v = r < a.dv && col < a.dk ? *reinterpret_cast<const float2*>(add + (r - row0) * a.dk + col)
                                                : make_float2(0.f, 0.f);
        s[n][2 * p] = acc[n][2 * p] * i * f.x + v.x;
        s[n][2 * p + 1] = acc[n][2 * p + 1] * i * f.y + v.y;
        float* out = rows(a.seg_s, to, n, p);
        if (out) *reinterpret_cast<float2*>(out) = make_float2(s[n][2 * p], s[n][2 * p + 1]);
      }
    }
    __syncthreads();  // N is read
  }
}

}  // namespace ttt
