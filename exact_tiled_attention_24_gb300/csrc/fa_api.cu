// C ABI of the exact tiled attention library: argument checks, TMA
// descriptor construction and kernel dispatch. Declarations and the full
// contract are in include/fa.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_common.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared size/scale checks. Returns FA_OK or the status to report.
int check_sizes(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const long long bh = static_cast<long long>(B) * H;
  // Grid sizes and row indices are 32-bit: BH * N rows must fit in int32.
  if (bh * N > INT_MAX) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Grouped-query heads: Hkv K/V heads, each shared by H / Hkv query heads.
int check_heads(int H, int Hkv) {
  if (Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int check_scale(float scale) {
  if (!std::isfinite(scale) || scale <= 0.f) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int map_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace

extern "C" {

const char* fa_version(void) { return "0.1.0"; }

int fa_debug_checks(void) {
#ifdef FA_DEBUG
  return 1;
#else
  return 0;
#endif
}

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_MISALIGNED: return "FA_ERR_MISALIGNED";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_BAD_INDEX: return "FA_ERR_BAD_INDEX";
    case FA_ERR_BOUNDS: return "FA_ERR_BOUNDS";
    default: return "FA_ERR_UNKNOWN";
  }
}

int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int Hkv, int N, int d, float scale, int causal, void* stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_fwd(q, k, v, o, lse, B * H, H / Hkv, N, d, scale, causal != 0,
                                 static_cast<cudaStream_t>(stream)));
}

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
           int d, float scale, int causal, void* stream) {
  return fa_fwd_gqa(q, k, v, o, lse, B, H, H, N, d, scale, causal, stream);
}

size_t fa_bwd_workspace_bytes(int B, int H, int N, int d) {
  if (check_sizes(B, H, N, d) != FA_OK) return 0;
  return static_cast<size_t>(B) * H * N * sizeof(float);
}

int fa_bwd_preprocess(const void* o, const void* dO, float* Dvec, int B, int H, int N, int d,
                      void* stream) {
  if (!o || !dO || !Dvec) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if (!aligned16(o) || !aligned16(dO) || !aligned16(Dvec)) return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_bwd_preprocess(static_cast<const __nv_bfloat16*>(o),
                                            static_cast<const __nv_bfloat16*>(dO), Dvec, B * H, N,
                                            d, static_cast<cudaStream_t>(stream)));
}

int fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO, const float* lse,
                const float* Dvec, void* dk, void* dv, int B, int H, int Hkv, int N, int d,
                float scale, int causal, void* stream) {
  if (!q || !k || !v || !dO || !lse || !Dvec || !dk || !dv) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(lse) ||
      !aligned16(Dvec) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_bwd_dkdv(q, k, v, dO, dk, dv, lse, Dvec, B * H, H / Hkv, N, d, scale,
                                      causal != 0, static_cast<cudaStream_t>(stream)));
}

int fa_bwd_dq(const void* q, const void* k, const void* v, const void* dO, const float* lse,
              const float* Dvec, void* dq, int B, int H, int Hkv, int N, int d, float scale,
              int causal, void* stream) {
  if (!q || !k || !v || !dO || !lse || !Dvec || !dq) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(lse) ||
      !aligned16(Dvec) || !aligned16(dq))
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_bwd_dq(q, k, v, dO, dq, lse, Dvec, B * H, H / Hkv, N, d, scale,
                                    causal != 0, static_cast<cudaStream_t>(stream)));
}

int fa_bwd_dq_d(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                float* Dvec, void* dq, int B, int H, int Hkv, int N, int d, float scale, int causal,
                void* stream) {
  if (!q || !k || !v || !o || !dO || !lse || !Dvec || !dq) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(lse) ||
      !aligned16(Dvec) || !aligned16(dq))
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_bwd_dq_d(q, k, v, o, dO, dq, lse, Dvec, B * H, H / Hkv, N, d, scale, causal != 0,
                                      static_cast<cudaStream_t>(stream)));
}

int fa_bwd_fuses_d(int B, int H, int Hkv, int N, int d) {
  if (check_sizes(B, H, N, d) != FA_OK || check_heads(H, Hkv) != FA_OK) return 0;
  return fa::bwd_fuse_d(B * H, H / Hkv, N) ? 1 : 0;
}

int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dO,
               const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes,
               int B, int H, int Hkv, int N, int d, float scale, int causal, void* stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_heads(H, Hkv)) != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!workspace || ws_bytes < fa_bwd_workspace_bytes(B, H, N, d)) return FA_ERR_WORKSPACE;
  // Every pointer is checked here, before the preprocess is launched, so
  // that an error leaves nothing queued (the stages repeat these checks).
  const void* ptrs[] = {q, k, v, o, dO, lse, dq, dk, dv, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_MISALIGNED;
  float* Dvec = static_cast<float*>(workspace);
  if (fa::bwd_fuse_d(B * H, H / Hkv, N)) {  // D inside the dQ sweep, then dK/dV
    st = fa_bwd_dq_d(q, k, v, o, dO, lse, Dvec, dq, B, H, Hkv, N, d, scale, causal, stream);
    if (st != FA_OK) return st;
    return fa_bwd_dkdv(q, k, v, dO, lse, Dvec, dk, dv, B, H, Hkv, N, d, scale, causal, stream);
  }
  st = fa_bwd_preprocess(o, dO, Dvec, B, H, N, d, stream);
  if (st != FA_OK) return st;
  // The dQ sweep needs only D: it runs on the library's side stream, forked
  // from `stream` after the preprocess and joined back at the end, beside
  // the dK/dV sweep (the two grids then share one tail).
  cudaStream_t cs = static_cast<cudaStream_t>(stream), side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  bool forked = fa::side_stream(&side) == cudaSuccess &&
                cudaEventCreateWithFlags(&fork, cudaEventDisableTiming) == cudaSuccess &&
                cudaEventCreateWithFlags(&join, cudaEventDisableTiming) == cudaSuccess &&
                cudaEventRecord(fork, cs) == cudaSuccess && cudaStreamWaitEvent(side, fork, 0) == cudaSuccess;
  if (!forked) {  // no side stream: the three stages in order on `stream`
    if (fork) cudaEventDestroy(fork);
    if (join) cudaEventDestroy(join);
    st = fa_bwd_dkdv(q, k, v, dO, lse, Dvec, dk, dv, B, H, Hkv, N, d, scale, causal, stream);
    if (st != FA_OK) return st;
    return fa_bwd_dq(q, k, v, dO, lse, Dvec, dq, B, H, Hkv, N, d, scale, causal, stream);
  }
  const int st_dkdv = fa_bwd_dkdv(q, k, v, dO, lse, Dvec, dk, dv, B, H, Hkv, N, d, scale, causal, stream);
  const int st_dq = fa_bwd_dq(q, k, v, dO, lse, Dvec, dq, B, H, Hkv, N, d, scale, causal, side);
  // Join even after a failed launch, so `stream` stays ordered after the side work.
  cudaError_t ej = cudaEventRecord(join, side);
  if (ej == cudaSuccess) ej = cudaStreamWaitEvent(cs, join, 0);
  cudaEventDestroy(fork);
  cudaEventDestroy(join);
  if (st_dkdv != FA_OK) return st_dkdv;
  if (st_dq != FA_OK) return st_dq;
  return map_cuda(ej);
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
           const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes,
           int B, int H, int N, int d, float scale, int causal, void* stream) {
  return fa_bwd_gqa(q, k, v, o, dO, lse, dq, dk, dv, workspace, ws_bytes, B, H, H, N, d, scale,
                    causal, stream);
}

static int softmax_rows(const float* x, float* y, long long rows, int n, bool online, void* stream) {
  if (!x || !y || rows < 1 || n < 1) return FA_ERR_INVALID_ARG;
  if (rows > INT_MAX) return FA_ERR_UNSUPPORTED;  // one CTA per row in a 1-D grid
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 3u) != 0)
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_softmax(x, y, rows, n, online, static_cast<cudaStream_t>(stream)));
}

int fa_softmax_safe(const float* x, float* y, long long rows, int n, void* stream) {
  return softmax_rows(x, y, rows, n, false, stream);
}

int fa_softmax_online(const float* x, float* y, long long rows, int n, void* stream) {
  return softmax_rows(x, y, rows, n, true, stream);
}

// ------------------------------------------------------------------ decode

size_t fa_decode_workspace_bytes(int B, int H, int d, int n_splits) {
  if (B < 1 || H < 1 || n_splits < 1 || (d != 64 && d != 128)) return 0;
  const size_t rows = static_cast<size_t>(n_splits) * B * H;
  const size_t o_bytes = (rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255);
  return o_bytes + rows * sizeof(float);
}

int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                    const int* seq_lens, void* o, float* lse, void* workspace, size_t ws_bytes, int B,
                    int H, int Hkv, int d, int num_blocks, int block_size, int max_blocks_per_seq,
                    float scale, int n_splits, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o || !lse) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || num_blocks < 1 || block_size < 1 || max_blocks_per_seq < 1 || n_splits < 1)
    return FA_ERR_INVALID_ARG;
  int st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<long long>(Hkv) * ((H / Hkv + 15) / 16) > 65535 || n_splits > 4096)
    return FA_ERR_UNSUPPORTED;
  const long long ctx = static_cast<long long>(max_blocks_per_seq) * block_size;
  // The cache's token rows (num_blocks * Hkv * block_size) are indexed in
  // 32 bits on the device: fewer than 2^32 - 1 (512 GB of cache at d = 64).
  if (ctx > INT_MAX / 2 || static_cast<long long>(num_blocks) * Hkv * block_size >= 0xffffffffll)
    return FA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < fa_decode_workspace_bytes(B, H, d, n_splits)) return FA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_MISALIGNED;
  const size_t rows = static_cast<size_t>(n_splits) * B * H;
  float* o_part = static_cast<float*>(workspace);
  float* lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                             ((rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255)));
  return map_cuda(fa::launch_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, o_part,
                                          lse_part, B, H, Hkv, d, num_blocks, block_size,
                                          max_blocks_per_seq, scale, n_splits,
                                          static_cast<cudaStream_t>(stream)));
}

int fa_attn_merge(const float* o_parts, const float* lse_parts, int n_parts, void* o, float* lse,
                  long long rows, int d, void* stream) {
  if (!o_parts || !lse_parts || !o || !lse || n_parts < 1 || rows < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((rows + 7) / 8 > INT_MAX) return FA_ERR_UNSUPPORTED;
  if (!aligned16(o_parts) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse_parts) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FA_ERR_MISALIGNED;
  return map_cuda(fa::launch_attn_merge(o_parts, lse_parts, n_parts, o, lse, rows, d,
                                        static_cast<cudaStream_t>(stream)));
}

// ------------------------------------- norms, rotation and paged appends

// Rotation tables and norm weights, shared by the entry points below.
static int check_rope(const float* cos, const float* sin, int d, int rot, int n_pos, const void* q_weight,
                      const void* k_weight, int weight_fp32, float eps) {
  if (rot < 0 || (weight_fp32 != 0 && weight_fp32 != 1)) return FA_ERR_INVALID_ARG;
  if (rot > 0 && (!cos || !sin || n_pos < 1)) return FA_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && (!std::isfinite(eps) || eps < 0.f)) return FA_ERR_INVALID_ARG;
  if (rot % 16 != 0 || rot > d) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}
static bool rope_aligned(const float* cos, const float* sin, int rot, const void* q_weight, const void* k_weight) {
  return (rot == 0 || (aligned16(cos) && aligned16(sin))) && aligned16(q_weight) && aligned16(k_weight);
}

static bool heads_strides_ok(const fa_heads* t) { return t->stride_b >= 0 && t->stride_h >= 0 && t->stride_n >= 0; }
static bool heads_aligned(const fa_heads* t) {
  return aligned16(t->ptr) && t->stride_b % 8 == 0 && t->stride_h % 8 == 0 && t->stride_n % 8 == 0;
}
static fa::HeadRows head_rows(const fa_heads* t, int B, int H, int N, int d) {
  return {static_cast<__nv_bfloat16*>(t->ptr), t->stride_b, t->stride_h, t->stride_n,
          t->stride_b * (B - 1) + t->stride_h * (H - 1) + t->stride_n * (N - 1) + d};
}

// Checks of the training form; on FA_OK fills p.
static int norm_rope_args(fa::NormRope* p, const fa_norm_rope_args* a, const fa_heads* q, const fa_heads* k) {
  const fa_heads* ts[] = {q, k, &a->q_out, &a->k_out};
  for (const fa_heads* t : ts)
    if (!t->ptr || !heads_strides_ok(t)) return FA_ERR_INVALID_ARG;
  if (a->Hkv < 1 || (!a->q_weight) != (!a->k_weight)) return FA_ERR_INVALID_ARG;
  int st = check_sizes(a->B, a->H, a->N, a->d);
  if (st == FA_OK) st = check_sizes(a->B, a->Hkv, a->N, a->d);
  if (st != FA_OK) return st;
  if ((st = check_rope(a->cos, a->sin, a->d, a->rot, a->n_pos, a->q_weight, a->k_weight, a->weight_fp32, a->eps)) !=
      FA_OK)
    return st;
  if (a->rot == 0 && !a->q_weight) return FA_ERR_INVALID_ARG;                     // nothing to do
  if (a->rot > 0 && !a->positions && a->n_pos < a->N) return FA_ERR_INVALID_ARG;  // token n is at position n
  if (a->H > 65536 || a->Hkv > 65536) return FA_ERR_UNSUPPORTED;
  for (const fa_heads* t : ts)
    if (!heads_aligned(t)) return FA_ERR_MISALIGNED;
  if (!rope_aligned(a->cos, a->sin, a->rot, a->q_weight, a->k_weight) ||
      (reinterpret_cast<uintptr_t>(a->positions) & 3u))
    return FA_ERR_MISALIGNED;
  *p = fa::NormRope{};
  p->q = head_rows(q, a->B, a->H, a->N, a->d);
  p->k = head_rows(k, a->B, a->Hkv, a->N, a->d);
  p->q_out = head_rows(&a->q_out, a->B, a->H, a->N, a->d);
  p->k_out = head_rows(&a->k_out, a->B, a->Hkv, a->N, a->d);
  p->cos = a->cos, p->sin = a->sin;
  p->positions = a->rot > 0 ? a->positions : nullptr;
  p->pos_sb = a->positions_per_batch ? a->N : 0;
  p->q_weight = a->q_weight, p->k_weight = a->k_weight;
  p->w32 = a->weight_fp32 != 0, p->interleaved = a->interleaved != 0;
  p->B = a->B, p->H = a->H, p->Hkv = a->Hkv, p->N = a->N, p->rot = a->rot, p->n_pos = a->n_pos;
  p->eps = a->eps;
  return FA_OK;
}

int fa_qk_norm_rope(const fa_norm_rope_args* a, void* stream) {
  if (!a) return FA_ERR_INVALID_ARG;
  fa::NormRope p;
  const int st = norm_rope_args(&p, a, &a->q, &a->k);
  if (st != FA_OK) return st;
  return map_cuda(fa::launch_norm_rope(p, a->d, static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int B, int N, int d) {
  if (B < 1 || N < 1 || (d != 64 && d != 128) || static_cast<long long>(B) * N > INT_MAX) return 0;
  return fa::norm_rope_bwd_partial_bytes(d);
}

int fa_qk_norm_rope_bwd(const fa_norm_rope_args* a, const fa_norm_rope_grads* g, void* stream) {
  if (!a || !g) return FA_ERR_INVALID_ARG;
  const bool norm = a->q_weight || a->k_weight;
  fa::NormRope p;
  // no norm: q and k are not read
  const int st = norm_rope_args(&p, a, norm ? &a->q : &a->q_out, norm ? &a->k : &a->k_out);
  if (st != FA_OK) return st;
  if (!g->dq.ptr || !g->dk.ptr || !heads_strides_ok(&g->dq) || !heads_strides_ok(&g->dk)) return FA_ERR_INVALID_ARG;
  if (norm && (!g->dq_weight || !g->dk_weight)) return FA_ERR_INVALID_ARG;
  if (norm && (!g->workspace || g->ws_bytes < fa_qk_norm_rope_bwd_workspace_bytes(a->B, a->N, a->d)))
    return FA_ERR_WORKSPACE;
  if (!heads_aligned(&g->dq) || !heads_aligned(&g->dk) || !aligned16(g->workspace) || !aligned16(g->dq_weight) ||
      !aligned16(g->dk_weight))
    return FA_ERR_MISALIGNED;
  p.dq = head_rows(&g->dq, a->B, a->H, a->N, a->d);
  p.dk = head_rows(&g->dk, a->B, a->Hkv, a->N, a->d);
  return map_cuda(fa::launch_norm_rope_bwd(p, a->d, static_cast<float*>(g->workspace), g->dq_weight, g->dk_weight,
                                           static_cast<cudaStream_t>(stream)));
}

// Sizes of a paged cache: its token rows are indexed in 32 bits.
static int check_cache(int Hkv, int num_blocks, int block_size, int max_blocks) {
  if (Hkv < 1 || num_blocks < 1 || block_size < 1 || max_blocks < 1) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks) * block_size > INT_MAX / 2 ||
      static_cast<long long>(num_blocks) * Hkv >= (0xffffffffll + block_size - 1) / block_size)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

static bool tokens_strides_ok(const fa_tokens* t) { return t->stride_t >= 0 && t->stride_h >= 0; }
static bool tokens_aligned(const fa_tokens* t) {
  return aligned16(t->ptr) && t->stride_t % 8 == 0 && t->stride_h % 8 == 0;
}
static fa::TokenRows token_rows(const fa_tokens* t, int T, int H, int d) {
  return {static_cast<__nv_bfloat16*>(t->ptr), t->stride_t, t->stride_h,
          t->stride_t * (T - 1) + t->stride_h * (H - 1) + d};
}

static int append(const fa_append_args* a, bool q4, void* stream) {
  if (!a || !a->k.ptr || !a->v.ptr || !a->k_cache || !a->v_cache || !a->block_table || !a->positions)
    return FA_ERR_INVALID_ARG;
  if (!tokens_strides_ok(&a->k) || !tokens_strides_ok(&a->v)) return FA_ERR_INVALID_ARG;
  if (q4 && (!a->k_scale || !a->v_scale || (!a->k_values) != (!a->v_values))) return FA_ERR_INVALID_ARG;
  const bool queries = a->q.ptr != nullptr;
  if (queries != (a->q_out.ptr != nullptr)) return FA_ERR_INVALID_ARG;
  if (queries && (a->H < 1 || !tokens_strides_ok(&a->q) || !tokens_strides_ok(&a->q_out))) return FA_ERR_INVALID_ARG;
  if (!queries && a->q_weight) return FA_ERR_INVALID_ARG;
  if (queries && (!a->q_weight) != (!a->k_weight)) return FA_ERR_INVALID_ARG;
  if (a->T < 1 || a->B < 1 || (!a->requests && a->T > a->B)) return FA_ERR_INVALID_ARG;
  int st = check_cache(a->Hkv, a->num_blocks, a->block_size, a->max_blocks_per_seq);
  if (st != FA_OK) return st;
  if (a->d != 64 && a->d != 128) return FA_ERR_UNSUPPORTED;
  const int w32 = a->weight_fp32 & ~FA_ZERO_SKIPPED;
  if ((st = check_rope(a->cos, a->sin, a->d, a->rot, a->n_pos, a->q_weight, a->k_weight, w32, a->eps)) != FA_OK)
    return st;
  if (a->H > 16384 || a->Hkv > 16384) return FA_ERR_UNSUPPORTED;
  if (!tokens_aligned(&a->k) || !tokens_aligned(&a->v) ||
      (queries && (!tokens_aligned(&a->q) || !tokens_aligned(&a->q_out))) || !aligned16(a->k_cache) ||
      !aligned16(a->v_cache) || !rope_aligned(a->cos, a->sin, a->rot, a->q_weight, a->k_weight) ||
      ((reinterpret_cast<uintptr_t>(a->block_table) | reinterpret_cast<uintptr_t>(a->positions) |
        reinterpret_cast<uintptr_t>(a->requests)) & 3u))
    return FA_ERR_MISALIGNED;
  if (q4 && (!aligned16(a->k_scale) || !aligned16(a->v_scale) || !aligned16(a->k_values) || !aligned16(a->v_values)))
    return FA_ERR_MISALIGNED;
  fa::Append p{};
  if (queries) {
    p.q = token_rows(&a->q, a->T, a->H, a->d);
    p.q_out = token_rows(&a->q_out, a->T, a->H, a->d);
  }
  p.k = token_rows(&a->k, a->T, a->Hkv, a->d);
  p.v = token_rows(&a->v, a->T, a->Hkv, a->d);
  p.k_cache = a->k_cache, p.v_cache = a->v_cache;
  if (q4) {
    p.k_scale = static_cast<__nv_bfloat16*>(a->k_scale), p.v_scale = static_cast<__nv_bfloat16*>(a->v_scale);
    p.k_values = static_cast<__nv_bfloat16*>(a->k_values), p.v_values = static_cast<__nv_bfloat16*>(a->v_values);
  }
  p.block_table = a->block_table, p.positions = a->positions, p.requests = a->requests;
  p.cos = a->cos, p.sin = a->sin;
  p.q_weight = a->q_weight, p.k_weight = a->k_weight;
  p.w32 = w32 != 0, p.interleaved = a->interleaved != 0, p.zero_skipped = (a->weight_fp32 & FA_ZERO_SKIPPED) != 0;
  p.T = a->T, p.B = a->B, p.H = queries ? a->H : 0, p.Hkv = a->Hkv;
  p.num_blocks = a->num_blocks, p.bs = a->block_size, p.max_blocks = a->max_blocks_per_seq;
  p.rot = a->rot, p.n_pos = a->n_pos;
  p.eps = a->eps;
  return map_cuda(fa::launch_append(p, a->d, q4, static_cast<cudaStream_t>(stream)));
}

int fa_append_paged(const fa_append_args* a, void* stream) { return append(a, false, stream); }
int fa_append_paged_q4(const fa_append_args* a, void* stream) { return append(a, true, stream); }

int fa_decode_q4_splits(int B, int H, int Hkv, int block_size, int max_blocks_per_seq) {
  if (B < 1 || H < 1 || check_heads(H, Hkv) != FA_OK || check_cache(Hkv, 1, block_size, max_blocks_per_seq) != FA_OK)
    return 0;
  return fa::decode_q4_splits(B, H, Hkv, static_cast<long long>(max_blocks_per_seq) * block_size);
}

int fa_decode_paged_q4(const fa_decode_q4_args* a, void* stream) {
  if (!a || !a->q || !a->k_cache || !a->k_scale || !a->v_cache || !a->v_scale || !a->block_table || !a->seq_lens ||
      !a->o || !a->lse)
    return FA_ERR_INVALID_ARG;
  const int B = a->B, H = a->H, Hkv = a->Hkv, d = a->d, S = a->n_splits;
  if (B < 1 || H < 1 || S < 1) return FA_ERR_INVALID_ARG;
  int st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  if ((st = check_scale(a->scale)) != FA_OK) return st;
  if ((st = check_cache(Hkv, a->num_blocks, a->block_size, a->max_blocks_per_seq)) != FA_OK) return st;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<long long>(Hkv) * ((H / Hkv + 7) / 8) > 65535 || S > 4096) return FA_ERR_UNSUPPORTED;
  if (S > 1 && (!a->workspace || a->ws_bytes < fa_decode_workspace_bytes(B, H, d, S))) return FA_ERR_WORKSPACE;
  if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->k_scale) || !aligned16(a->v_cache) ||
      !aligned16(a->v_scale) || !aligned16(a->o) || !aligned16(a->workspace) ||
      ((reinterpret_cast<uintptr_t>(a->lse) | reinterpret_cast<uintptr_t>(a->block_table) |
        reinterpret_cast<uintptr_t>(a->seq_lens)) & 3u))
    return FA_ERR_MISALIGNED;
  fa::DecodeQ4 p{};
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.k_cache = static_cast<const uint8_t*>(a->k_cache), p.v_cache = static_cast<const uint8_t*>(a->v_cache);
  p.k_scale = static_cast<const uint32_t*>(a->k_scale), p.v_scale = static_cast<const uint32_t*>(a->v_scale);
  p.block_table = a->block_table, p.seq_lens = a->seq_lens;
  p.o = static_cast<__nv_bfloat16*>(a->o), p.lse = a->lse;
  if (S > 1) {
    const size_t rows = static_cast<size_t>(S) * B * H;
    p.o_part = static_cast<float*>(a->workspace);
    p.lse_part = reinterpret_cast<float*>(static_cast<char*>(a->workspace) +
                                          ((rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255)));
  }
  p.B = B, p.H = H, p.Hkv = Hkv;
  p.num_blocks = a->num_blocks, p.bs = a->block_size, p.max_blocks = a->max_blocks_per_seq;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  return map_cuda(fa::launch_decode_q4(p, d, S, static_cast<cudaStream_t>(stream)));
}

int fa_selftest_wait_limit(void* stream) {
  return map_cuda(fa::launch_wait_limit_selftest(static_cast<cudaStream_t>(stream)));
}

int fa_last_device_error(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t ef = 0, eb = 0, ed = 0, et = 0, es = 0, er = 0, ea = 0, eq = 0;
  if (fa::read_and_clear_fwd_error(&ef, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_bwd_error(&eb, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_decode_error(&ed, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_selftest_error(&et, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_softmax_error(&es, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_rope_error(&er, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_append_error(&ea, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::read_and_clear_decode_q4_error(&eq, s) != cudaSuccess) return FA_ERR_CUDA;
  if (ef == 1 || eb == 1 || ed == 1 || et == 1 || eq == 1) return FA_ERR_TIMEOUT;
  if (ef == 3 || eb == 3 || ed == 3 || es == 3 || er == 3 || ea == 3 || eq == 3) return FA_ERR_BOUNDS;
  if (ed == 2 || er == 2 || ea == 2 || eq == 2) return FA_ERR_BAD_INDEX;
  if (ef || eb || ed || et || es || er || ea || eq) return FA_ERR_TIMEOUT;
  return FA_OK;
}

}  // extern "C"
