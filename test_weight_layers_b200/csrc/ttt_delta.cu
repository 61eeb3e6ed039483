// C ABI of the gated delta rule (see include/ttt.h for the contract): argument
// checks, workspace carving and the launch sequences.
#include <algorithm>
#include <initializer_list>

#include "host.cuh"
#include "kernels_delta.cuh"
#include "kernels_delta_bwd.cuh"
#include "kernels_delta_seq.cuh"
#include "ttt.h"

using namespace ttt;

namespace {

struct DeltaWs {
  unsigned int* status;
  DrSeq* seqs;
  DrChunk* chunks;
  uint8_t* kq;
  uint8_t* blk;
  int64_t max_chunks;
  DrSeq* cuts;  // [2][max_cuts] the segments before and behind each cut
  int fill, max_segs, max_cuts;
  float *seg_s, *seg_n, *phi_scale;
  uint8_t* phi;
  // backward pass
  float *tok, *keep_s, *keep_ds, *keep_e, *keep_z, *w_part, *b_part, *x_part;
  size_t total;
};

// bf16 calls of so few tokens run token by token: one short kernel instead of the chunks' three (4 heads of 192: 19 us
// against 33 us for 32 tokens, 33 and 33 for 64; 16 heads of 128: 19 against 27, 31 and 27).
constexpr int64_t kTokensMost = 40;
constexpr int kDeltaMaxSeqs = 1 << 24;

int dk_pad(int dk) { return (dk + 63) / 64 * 64; }

bool delta_dims_ok(const ttt_delta_dims& d) {
  return d.heads_qk >= 1 && d.heads_v >= 1 && d.dk >= 1 && d.dv >= 1 && d.heads_v % d.heads_qk == 0;
}

bool delta_dims_supported(const ttt_delta_dims& d) {
  return d.dk % 8 == 0 && d.dv % 8 == 0 && d.dk <= 256 && d.dv <= 1024 && d.heads_v <= 4096;
}

// Blocks of 4 warps (64 value channels) that the passes have for each sequence.
int64_t pass_blocks(const ttt_delta_dims& d) { return (int64_t)d.heads_v * ((d.dv + 63) / 64); }

// Segments.  Uncut, the passes have n_seq * pass_blocks blocks, each on its own SM for the length of a sequence; few
// heads and a long sequence leave most SMs idle.  Such sequences are cut into segments (2.6 times the products, a scan
// and a join; the rule, which needs the lengths, is k_delta_plan's): 131,072 tokens, 4 heads of 192, take 10.7 ms
// uncut, 2.56 ms in 12 segments, 1,374 tokens 138 us, and 101 us in 6; 32,768 tokens beside four prompts of 100 take
// 2.71 ms uncut, 0.76 in 12 segments; 16 heads of 128, 32,768 tokens and 100: 2.29 ms, 1.49 in 4.  Where no sequence
// is cut after all, the scan and the join end at once (4 and 3 us of packed prompts' 388; four prompts of 700 tokens, 4
// heads of 192: 86 us without them, 92 with).
constexpr int kDeltaSms = 148;

struct SegRoom {
  int fill = 0;   // pass_blocks that fit on the card (0: no sequence can be cut)
  int cuts = 0;   // cuts, at most
  int segs = 0;   // segments of cut sequences, at most
};

// With k chunks to a segment, k >= chunks of all sequences / fill and 2 k^2 >= those of the longest: a sequence of n
// chunks has at most n / k segments beyond the first, so all have `fill` at most, and each sqrt(2 n); fewer than
// `fill` sequences are longer than k.
SegRoom seg_room(const ttt_delta_dims& d, int64_t T, int n_seq, ttt_dtype dt) {
  SegRoom r;
  const int64_t fill = dt == TTT_BF16 ? kDeltaSms / pass_blocks(d) : 0;
  if (fill < 3 || T <= (DR_CUT_CHUNKS - 1) * DR_C) return r;
  const int64_t chunks = (T + DR_C - 1) / DR_C, some = std::min<int64_t>(n_seq, fill);
  int64_t root = 1;
  while (root < fill && root * root < 2 * chunks) ++root;
  r.fill = (int)fill;
  r.cuts = (int)std::min(fill, some * root);
  r.segs = (int)some + r.cuts;
  return r;
}

DeltaWs delta_carve(void* base, const ttt_delta_dims& d, int64_t T, int n_seq, ttt_dtype dt, bool backward) {
  DeltaWs w{};
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = b + off;
    off = up256(off + bytes);
    return p;
  };
  w.max_chunks = T / DR_C + n_seq;
  const SegRoom room = seg_room(d, T, n_seq, dt);
  w.fill = room.fill;
  w.max_segs = n_seq + room.cuts;
  w.max_cuts = room.cuts;
  w.status = reinterpret_cast<unsigned int*>(take(256));
  w.seqs = reinterpret_cast<DrSeq*>(take(((size_t)w.max_segs + 2 * w.max_cuts) * sizeof(DrSeq)));
  w.cuts = w.seqs + w.max_segs;
  w.chunks = reinterpret_cast<DrChunk*>(take((size_t)std::max<int64_t>(w.max_chunks, 1) * sizeof(DrChunk)));
  if (dt == TTT_BF16) {
    w.kq = take((size_t)w.max_chunks * d.heads_qk * 2 * DR_C * dk_pad(d.dk) * 2);
    w.blk = take((size_t)w.max_chunks * d.heads_v * DR_BLK);
  }
  if (w.max_cuts) {
    const size_t segs = (size_t)room.segs * d.heads_v, dkp = dk_pad(d.dk);
    w.seg_s = reinterpret_cast<float*>(take(segs * d.dv * d.dk * 4));
    w.seg_n = reinterpret_cast<float*>(take(segs * d.dv * d.dk * 4));
    w.phi = take(segs * 2 * dkp * dkp * 2);
    w.phi_scale = reinterpret_cast<float*>(take(segs * dkp * 4));
  }
  if (dt == TTT_BF16 && backward) {
    const size_t blocks = (size_t)w.max_chunks * d.heads_v, n16 = (d.dv + 15) / 16;
    w.tok = reinterpret_cast<float*>(take((size_t)w.max_chunks * d.heads_qk * TF_N * DR_C * 4));
    w.keep_s = reinterpret_cast<float*>(take(blocks * d.dv * d.dk * 4));
    w.keep_ds = reinterpret_cast<float*>(take(blocks * d.dv * d.dk * 4));
    w.keep_e = reinterpret_cast<float*>(take(blocks * d.dv * DR_C * 4));
    w.keep_z = reinterpret_cast<float*>(take(blocks * d.dv * DR_C * 4));
    w.w_part = reinterpret_cast<float*>(take(blocks * n16 * DR_C * 4));
    w.b_part = reinterpret_cast<float*>(take(blocks * n16 * DR_C * 4));
    w.x_part = reinterpret_cast<float*>(take(blocks * n16 * 4));
  }
  w.total = off;
  return w;
}

struct DeltaIo {
  int64_t ldq, ldk, ldv, ldo;
  int l2norm;
};

int check_rows(const void* p, int64_t ld, int64_t width, ttt_dtype dt) {
  if (!p || ld < width) return TTT_ERR_INVALID;
  if (!aligned16(p) || (ld * (int64_t)esize(dt)) % 16) return TTT_ERR_ALIGN;
  return TTT_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks shared by the entry points (O: the outputs' rows, or their gradient's); fills the row strides.
int delta_check(const void* Q, const void* K, const void* V, const float* g, const float* beta, const void* O,
                const ttt_delta_dims& d, const ttt_io_cfg* io, ttt_dtype dt, bool any_tokens, DeltaIo& out) {
  const int64_t nq = (int64_t)d.heads_qk * d.dk, nv = (int64_t)d.heads_v * d.dv;
  out.ldq = io->ld_q ? io->ld_q : nq;
  out.ldk = io->ld_k ? io->ld_k : nq;
  out.ldv = io->ld_v ? io->ld_v : nv;
  out.ldo = io->ld_o ? io->ld_o : nv;
  out.l2norm = io->qk_l2norm;
  if (out.ldq < nq || out.ldk < nq || out.ldv < nv || out.ldo < nv) return TTT_ERR_INVALID;
  if (!any_tokens) return TTT_OK;
  TTT_TRY(check_rows(Q, out.ldq, nq, dt));
  TTT_TRY(check_rows(K, out.ldk, nq, dt));
  TTT_TRY(check_rows(V, out.ldv, nv, dt));
  TTT_TRY(check_rows(O, out.ldo, nv, dt));
  if (!g || !beta) return TTT_ERR_INVALID;
  return aligned4(g) && aligned4(beta) ? TTT_OK : TTT_ERR_ALIGN;
}

bool is_one_of(const void* out, std::initializer_list<const void*> in) {
  return std::find(in.begin(), in.end(), out) != in.end();
}

// Opts kernel K in to all the shared memory a block can have, once per device.
template <auto K>
int smem_opt_in() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  TTT_CHECK(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return TTT_OK;
  TTT_CHECK(cudaFuncSetAttribute((const void*)K, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
  done.fetch_or(bit, std::memory_order_relaxed);
  return TTT_OK;
}

// Sequences of equal length need not be looked at to see that none is cut.
void even_cuts(DeltaWs& w, int64_t T, int n_seq) {
  if (!w.fill || ((T / n_seq + DR_C - 1) / DR_C >= DR_CUT_CHUNKS && 3ll * n_seq <= w.fill)) return;
  w.fill = w.max_cuts = 0;
  w.max_segs = n_seq;
}

int launch_plan(const int32_t* cu, int n_seq, int64_t T, const DeltaWs& w, cudaStream_t s) {
  k_delta_plan<<<1, 1024, 0, s>>>(cu, n_seq, (int)T, w.fill, w.max_segs, w.max_cuts, (int)w.max_chunks, w.seqs, w.cuts,
                                  w.chunks, w.status);
  TTT_LAUNCHED();
  return TTT_OK;
}

// Row warps of a pass block (16 value channels each): four, one to a sub-partition of the SM.  A warp's chain of
// products is bound by its own latency, so eight on an SM ran at 0.6 of the speed each (state pass of packed prompts
// of 16 heads, taken with the row warps making the outputs as well: 435 us with 8, 260 with 4; with 2, which share a
// staged copy of the operands with fewer, 353); two where shared memory holds no more (dk = 256 on the way back).
template <int DK>
constexpr int pass_warps(bool back) {
  return back && DK > 192 ? 2 : 4;
}
int pass_warps_for(int most, int dv) { return std::min(most, (dv + 15) / 16); }

// Launches a pass over the chunks of each segment (`warps` with the one that copies).
template <auto K, typename Args>
int launch_pass(const Args& a, int segs, int64_t blocks_per_head, int warps, int smem, cudaStream_t s) {
  if (blocks_per_head * a.hv * segs > INT32_MAX) return TTT_ERR_UNSUPPORTED;
  TTT_TRY(smem_opt_in<K>());
  TTT_TRY(launch_pdl(K, dim3((unsigned)(blocks_per_head * a.hv * segs)), dim3(warps * 32), smem, s, a));
  TTT_LAUNCHED();
  return TTT_OK;
}

int64_t blocks_of(int rows, int warps) { return (rows + 16 * warps - 1) / (16 * warps); }

template <int DK, bool REVERSE>
int launch_join(const StateArgs& sa, float* seg_s, const DeltaWs& w, cudaStream_t s) {
  JoinArgs ja{w.cuts, sa.hv, sa.dk, sa.dv, seg_s, w.seg_n, w.phi, w.phi_scale, sa.guard};
  return launch_pass<k_delta_join<DK, REVERSE>>(ja, w.max_cuts, (sa.dv + 63) / 64, 4, join_smem<DK>(), s);
}

// The states at the starts of cut sequences' segments.
template <int DK>
int run_scan(StateArgs sa, const DeltaWs& w, cudaStream_t s) {
  if (!w.max_cuts) return TTT_OK;
  const int warps = pass_warps<DK>(false);
  sa.seqs = w.cuts;
  TTT_TRY((launch_pass<k_delta_state<DK, PASS_SCAN>>(sa, w.max_cuts, blocks_of(sa.dv, warps) + blocks_of(DK, warps),
                                                   warps + 1, state_smem<DK, PASS_SCAN>(warps), s)));
  return launch_join<DK, false>(sa, w.seg_s, w, s);
}

template <int DK, bool BACK>
int launch_prep(const PrepArgs& pa, const DeltaWs& w, cudaStream_t s) {
  TTT_TRY((smem_opt_in<k_delta_prep<DK, BACK>>()));
  TTT_TRY(launch_pdl(k_delta_prep<DK, BACK>, dim3((unsigned)w.max_chunks, pa.hk), dim3(128), prep_smem<DK>(), s, pa));
  TTT_LAUNCHED();
  return TTT_OK;
}

template <int DK>
int run_delta_fwd(const PrepArgs& pa, StateArgs sa, const DeltaWs& w, cudaStream_t s) {
  TTT_TRY((launch_prep<DK, false>(pa, w, s)));
  TTT_TRY(run_scan<DK>(sa, w, s));
  const int warps = pass_warps_for(pass_warps<DK>(false), sa.dv);
  return launch_pass<k_delta_state<DK, PASS_OUT>>(sa, w.max_segs, blocks_of(sa.dv, warps),
                                                  state_split<DK, PASS_OUT>() ? 2 * warps : warps + 1,
                                                  state_smem<DK, PASS_OUT>(warps), s);
}

template <int DK>
int run_delta_bwd(const PrepArgs& pa, const StateArgs& sa, const ReverseArgs& ra, const GradArgs& ga, const DeltaWs& w,
                  cudaStream_t s) {
  TTT_TRY((launch_prep<DK, true>(pa, w, s)));
  TTT_TRY(run_scan<DK>(sa, w, s));
  const int warps = pass_warps_for(pass_warps<DK>(true), sa.dv), smem = state_smem<DK, PASS_BACK>(warps, true);
  const int64_t blocks = blocks_of(sa.dv, warps);
  TTT_TRY((launch_pass<k_delta_state<DK, PASS_BACK>>(sa, w.max_segs, blocks, warps + 1, smem, s)));
  if (w.max_cuts) {  // the transitions are the state pass's, transposed
    ReverseArgs scan = ra;
    scan.seqs = w.cuts + w.max_cuts;
    TTT_TRY((launch_pass<k_delta_reverse<DK, true>>(scan, w.max_cuts, blocks, warps + 1, smem, s)));
    TTT_TRY((launch_join<DK, true>(sa, w.seg_s, w, s)));
  }
  TTT_TRY((launch_pass<k_delta_reverse<DK, false>>(ra, w.max_segs, blocks, warps + 1, smem, s)));
  TTT_TRY(smem_opt_in<k_delta_grad<DK>>());
  TTT_TRY(launch_pdl(k_delta_grad<DK>, dim3((unsigned)w.max_chunks, ga.hk), dim3(256), grad_smem<DK>(), s, ga));
  TTT_LAUNCHED();
  return TTT_OK;
}

template <typename T, int VEC, int NV, int ROWS, bool SEQ>
int launch_tokens_rows(const SeqArgs<T>& a, unsigned blocks, cudaStream_t s) {
  const dim3 grid(blocks, a.hv, (a.dv + 4 * ROWS - 1) / (4 * ROWS));
  if constexpr (SEQ) {
    TTT_TRY(launch_pdl(k_delta_tokens<T, VEC, NV, ROWS, SEQ>, grid, dim3(128), 0, s, a));
  } else {
    k_delta_tokens<T, VEC, NV, ROWS, SEQ><<<grid, 128, 0, s>>>(a);
  }
  TTT_LAUNCHED();
  return TTT_OK;
}

// Rows of S per warp: many where the state's bytes count (a decoding step that fills the card: loads of 4 to 8 rows
// in flight), two where the latency of the reduction does (sequences, a few rows).
template <typename T, int VEC, int NV>
int launch_tokens(const SeqArgs<T>& a, unsigned blocks, cudaStream_t s) {
  constexpr int MANY = NV * VEC > 4 ? 4 : 8;
  if (a.seqs) return launch_tokens_rows<T, VEC, NV, 2, true>(a, blocks, s);
  if ((int64_t)blocks * a.hv * a.dv < 148 * 64) return launch_tokens_rows<T, VEC, NV, 2, false>(a, blocks, s);
  return launch_tokens_rows<T, VEC, NV, MANY, false>(a, blocks, s);
}

template <typename T>
int run_tokens(const SeqArgs<T>& a, unsigned blocks, cudaStream_t s) {
  if (a.dk == 128) return launch_tokens<T, 4, 1>(a, blocks, s);
  if (a.dk == 256) return launch_tokens<T, 4, 2>(a, blocks, s);
  switch ((a.dk + 63) / 64) {
    case 1: return launch_tokens<T, 2, 1>(a, blocks, s);
    case 2: return launch_tokens<T, 2, 2>(a, blocks, s);
    case 3: return launch_tokens<T, 2, 3>(a, blocks, s);
    default: return launch_tokens<T, 2, 4>(a, blocks, s);
  }
}

template <typename T>
SeqArgs<T> seq_args(const void* Q, const void* K, const void* V, const float* g, const float* beta, const float* S0,
                    float* S, void* O, float scale, const ttt_delta_dims& d, const DeltaIo& io) {
  SeqArgs<T> a{};
  a.Q = (const T*)Q;
  a.K = (const T*)K;
  a.V = (const T*)V;
  a.O = (T*)O;
  a.ldq = io.ldq;
  a.ldk = io.ldk;
  a.ldv = io.ldv;
  a.ldo = io.ldo;
  a.g = g;
  a.beta = beta;
  a.S0 = S0;
  a.S = S;
  a.hk = d.heads_qk;
  a.hv = d.heads_v;
  a.dk = d.dk;
  a.dv = d.dv;
  a.l2norm = io.l2norm;
  a.scale = scale;
  return a;
}

PrepArgs prep_args(const void* Q, const void* K, const float* g, const float* beta, float scale,
                   const ttt_delta_dims& d, const DeltaIo& x, const DeltaWs& w) {
  PrepArgs a{};
  a.Q = (const __nv_bfloat16*)Q;
  a.K = (const __nv_bfloat16*)K;
  a.g = g;
  a.beta = beta;
  a.ldq = x.ldq;
  a.ldk = x.ldk;
  a.hk = d.heads_qk;
  a.hv = d.heads_v;
  a.dk = d.dk;
  a.l2norm = x.l2norm;
  a.scale = scale;
  a.chunks = w.chunks;
  a.kq = w.kq;
  a.blk = w.blk;
  a.tok = w.tok;
  return a;
}

// What the passes over the chunks share (StateArgs, ReverseArgs).
template <typename Args>
void pass_args(Args& a, const void* V, const ttt_delta_dims& d, const DeltaIo& x, const DeltaWs& w) {
  a.V = (const __nv_bfloat16*)V;
  a.ldv = x.ldv;
  a.ldo = x.ldo;
  a.hk = d.heads_qk;
  a.hv = d.heads_v;
  a.dk = d.dk;
  a.dv = d.dv;
  a.seqs = w.seqs;
  a.kq = w.kq;
  a.blk = w.blk;
  a.guard = Guard{w.status, wait_timeout_ns()};
  a.keep_e = w.keep_e;
  a.w_part = w.w_part;
  a.seg_n = w.seg_n;
}

StateArgs state_args(const void* V, const float* S0, const ttt_delta_dims& d, const DeltaIo& x, const DeltaWs& w) {
  StateArgs a{};
  pass_args(a, V, d, x, w);
  a.S0 = S0;
  a.keep_s = w.keep_s;
  a.seg_s = w.seg_s;
  a.phi = w.phi;
  a.phi_scale = w.phi_scale;
  return a;
}

int delta_check_call(const ttt_delta_dims& d, ttt_dtype dt, int64_t T, int n_seq, bool packed, const ttt_io_cfg* io,
                     bool backward, void* ws, size_t ws_bytes) {
  if ((dt != TTT_FP32 && dt != TTT_BF16) || !delta_dims_ok(d) || T < 0 || n_seq < 0 || !io) return TTT_ERR_INVALID;
  if (!delta_dims_supported(d) || T > INT32_MAX - DR_C || n_seq > kDeltaMaxSeqs) return TTT_ERR_UNSUPPORTED;
  if (n_seq == 0 ? T > 0 && !packed : !packed && T % n_seq) return TTT_ERR_INVALID;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return TTT_ERR_WORKSPACE;
  return ws_bytes < delta_carve(nullptr, d, T, n_seq, dt, backward).total ? TTT_ERR_WORKSPACE : TTT_OK;
}

}  // namespace

extern "C" {

size_t ttt_delta_workspace_bytes(ttt_delta_dims dims, int64_t T, int n_seq, ttt_dtype dtype, int backward) {
  if ((dtype != TTT_FP32 && dtype != TTT_BF16) || !delta_dims_ok(dims) || !delta_dims_supported(dims) || T < 0 ||
      T > INT32_MAX - DR_C || n_seq < 0 || n_seq > kDeltaMaxSeqs)
    return 0;
  return delta_carve(nullptr, dims, T, n_seq, dtype, backward != 0).total;
}

int ttt_delta_chunked(const void* Q, const void* K, const void* V, const float* g, const float* beta, const float* S0,
                      float* S, void* O, const int32_t* cu_seqlens, int n_seq, int64_t T, float scale,
                      ttt_delta_dims dims, const ttt_io_cfg* io, ttt_dtype dtype, void* ws, size_t ws_bytes,
                      void* stream) {
  TTT_TRY(delta_check_call(dims, dtype, T, n_seq, cu_seqlens != nullptr, io, false, ws, ws_bytes));
  DeltaIo x;
  const bool any = T > 0 && n_seq > 0;
  TTT_TRY(delta_check(Q, K, V, g, beta, O, dims, io, dtype, any, x));
  if (any && is_one_of(O, {Q, K, V})) return TTT_ERR_INVALID;
  if ((S0 && !aligned16(S0)) || (S && !aligned16(S)) || !aligned4(cu_seqlens)) return TTT_ERR_ALIGN;
  if (n_seq == 0) return TTT_OK;
  cudaStream_t s = (cudaStream_t)stream;
  DeltaWs w = delta_carve(ws, dims, T, n_seq, dtype, false);
  if (!cu_seqlens) even_cuts(w, T, n_seq);
  ProfScope ps(TTT_PROF_DELTA, s);
  TTT_TRY(launch_plan(cu_seqlens, n_seq, T, w, s));
  if (dtype == TTT_FP32 || T <= kTokensMost) {
    auto go = [&](auto a) {
      a.seqs = w.seqs;
      return run_tokens(a, (unsigned)n_seq, s);
    };
    if (dtype == TTT_FP32) return go(seq_args<float>(Q, K, V, g, beta, S0, S, O, scale, dims, x));
    return go(seq_args<__nv_bfloat16>(Q, K, V, g, beta, S0, S, O, scale, dims, x));
  }
  const PrepArgs pa = prep_args(Q, K, g, beta, scale, dims, x, w);
  StateArgs sa = state_args(V, S0, dims, x, w);
  sa.O = (__nv_bfloat16*)O;
  sa.S = S;
  switch (dk_pad(dims.dk)) {
    case 64: return run_delta_fwd<64>(pa, sa, w, s);
    case 128: return run_delta_fwd<128>(pa, sa, w, s);
    case 192: return run_delta_fwd<192>(pa, sa, w, s);
    default: return run_delta_fwd<256>(pa, sa, w, s);
  }
}

int ttt_delta_chunked_backward(const void* Q, const void* K, const void* V, const float* g, const float* beta,
                               const float* S0, const void* dO, const float* dS, void* dQ, void* dK, void* dV,
                               float* dg, float* dbeta, float* dS0, const int32_t* cu_seqlens, int n_seq, int64_t T,
                               float scale, ttt_delta_dims dims, const ttt_io_cfg* io, ttt_dtype dtype, void* ws,
                               size_t ws_bytes, void* stream) {
  if (dtype == TTT_FP32) return TTT_ERR_UNSUPPORTED;
  TTT_TRY(delta_check_call(dims, dtype, T, n_seq, cu_seqlens != nullptr, io, true, ws, ws_bytes));
  DeltaIo x;
  const bool any = T > 0 && n_seq > 0;
  TTT_TRY(delta_check(Q, K, V, g, beta, dO, dims, io, dtype, any, x));
  for (const void* p : {(const void*)S0, (const void*)dS, (const void*)dS0})
    if (!aligned16(p)) return TTT_ERR_ALIGN;
  if (!aligned4(cu_seqlens) || !aligned4(dg) || !aligned4(dbeta)) return TTT_ERR_ALIGN;
  if (dS0 && (dS0 == dS || dS0 == S0)) return TTT_ERR_INVALID;
  if (any) {
    TTT_TRY(check_rows(dQ, x.ldq, (int64_t)dims.heads_qk * dims.dk, dtype));
    TTT_TRY(check_rows(dK, x.ldk, (int64_t)dims.heads_qk * dims.dk, dtype));
    TTT_TRY(check_rows(dV, x.ldv, (int64_t)dims.heads_v * dims.dv, dtype));
    if (!dg || !dbeta) return TTT_ERR_INVALID;
    for (const void* out : {(const void*)dQ, (const void*)dK, (const void*)dV})
      if (is_one_of(out, {Q, K, V, dO})) return TTT_ERR_INVALID;
  }
  if (n_seq == 0) return TTT_OK;
  cudaStream_t s = (cudaStream_t)stream;
  DeltaWs w = delta_carve(ws, dims, T, n_seq, dtype, true);
  if (!cu_seqlens) even_cuts(w, T, n_seq);
  ProfScope ps(TTT_PROF_DELTA, s);
  TTT_TRY(launch_plan(cu_seqlens, n_seq, T, w, s));
  const PrepArgs pa = prep_args(Q, K, g, beta, scale, dims, x, w);
  StateArgs sa = state_args(V, S0, dims, x, w);
  sa.dO = (const __nv_bfloat16*)dO;
  ReverseArgs ra{};
  pass_args(ra, V, dims, x, w);
  ra.dO = (const __nv_bfloat16*)dO;
  ra.dV = (__nv_bfloat16*)dV;
  ra.dS = dS;
  ra.dS0 = dS0;
  ra.keep_ds = w.keep_ds;
  ra.keep_z = w.keep_z;
  ra.b_part = w.b_part;
  ra.x_part = w.x_part;
  ra.seg_ds = w.seg_s;  // (the start states are read by then)
  GradArgs ga{};
  ga.dO = (const __nv_bfloat16*)dO;
  ga.ldo = x.ldo;
  ga.ldq = x.ldq;
  ga.ldk = x.ldk;
  ga.dQ = (__nv_bfloat16*)dQ;
  ga.dK = (__nv_bfloat16*)dK;
  ga.dg = dg;
  ga.dbeta = dbeta;
  ga.hk = dims.heads_qk;
  ga.hv = dims.heads_v;
  ga.dk = dims.dk;
  ga.dv = dims.dv;
  ga.chunks = w.chunks;
  ga.kq = w.kq;
  ga.blk = w.blk;
  ga.tok = w.tok;
  ga.keep_s = w.keep_s;
  ga.keep_e = w.keep_e;
  ga.keep_ds = w.keep_ds;
  ga.keep_z = w.keep_z;
  ga.w_part = w.w_part;
  ga.b_part = w.b_part;
  ga.x_part = w.x_part;
  switch (dk_pad(dims.dk)) {
    case 64: return run_delta_bwd<64>(pa, sa, ra, ga, w, s);
    case 128: return run_delta_bwd<128>(pa, sa, ra, ga, w, s);
    case 192: return run_delta_bwd<192>(pa, sa, ra, ga, w, s);
    default: return run_delta_bwd<256>(pa, sa, ra, ga, w, s);
  }
}

int ttt_delta_step(const void* Q, const void* K, const void* V, const float* g, const float* beta, float* S,
                   int n_slots, const int32_t* slots, void* O, int64_t B, float scale, ttt_delta_dims dims,
                   const ttt_io_cfg* io, ttt_dtype dtype, void* stream) {
  if ((dtype != TTT_FP32 && dtype != TTT_BF16) || !delta_dims_ok(dims) || B < 0 || n_slots < 0 || !io)
    return TTT_ERR_INVALID;
  if (!delta_dims_supported(dims) || B > INT32_MAX / 2) return TTT_ERR_UNSUPPORTED;
  if (!slots && B > n_slots) return TTT_ERR_INVALID;
  DeltaIo x;
  TTT_TRY(delta_check(Q, K, V, g, beta, O, dims, io, dtype, B > 0, x));
  if (B == 0) return TTT_OK;
  if (is_one_of(O, {Q, K, V})) return TTT_ERR_INVALID;
  if (n_slots == 0 && slots) return TTT_OK;  // every row is padding (and an empty pool may be NULL)
  if (!S) return TTT_ERR_INVALID;
  if (!aligned16(S) || !aligned4(slots)) return TTT_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope ps(TTT_PROF_DELTA, s);
  auto go = [&](auto a) {
    a.slots = slots;
    a.n_slots = n_slots;
    a.rows = (int)B;
    return run_tokens(a, (unsigned)B, s);
  };
  if (dtype == TTT_FP32) return go(seq_args<float>(Q, K, V, g, beta, S, S, O, scale, dims, x));
  return go(seq_args<__nv_bfloat16>(Q, K, V, g, beta, S, S, O, scale, dims, x));
}

}  // extern "C"
