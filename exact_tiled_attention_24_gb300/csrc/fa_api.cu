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

// Checks of the training form; on FA_OK fills p (tensors in q, k and their
// counterparts a, b: the outputs, or the output gradients).
static int norm_rope_args(fa::NormRope* p, const fa_heads* q, const fa_heads* k, const fa_heads* a, const fa_heads* b,
                          const float* cos, const float* sin, const int* positions, int positions_per_batch,
                          const void* q_weight, const void* k_weight, int weight_fp32, int B, int H, int Hkv, int N,
                          int d, int rot, int n_pos, float eps, int interleaved) {
  const fa_heads* ts[] = {q, k, a, b};
  for (const fa_heads* t : ts)
    if (!t || !t->ptr || !heads_strides_ok(t)) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || (!q_weight) != (!k_weight)) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_rope(cos, sin, d, rot, n_pos, q_weight, k_weight, weight_fp32, eps)) != FA_OK) return st;
  if (rot == 0 && !q_weight) return FA_ERR_INVALID_ARG;               // nothing to do
  if (rot > 0 && !positions && n_pos < N) return FA_ERR_INVALID_ARG;  // token n is at position n
  if (H > 65536 || Hkv > 65536) return FA_ERR_UNSUPPORTED;
  for (const fa_heads* t : ts)
    if (!heads_aligned(t)) return FA_ERR_MISALIGNED;
  if (!rope_aligned(cos, sin, rot, q_weight, k_weight) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_MISALIGNED;
  *p = fa::NormRope{};
  p->q = head_rows(q, B, H, N, d);
  p->k = head_rows(k, B, Hkv, N, d);
  p->q_out = head_rows(a, B, H, N, d);
  p->k_out = head_rows(b, B, Hkv, N, d);
  p->cos = cos, p->sin = sin;
  p->positions = rot > 0 ? positions : nullptr;
  p->pos_sb = positions_per_batch ? N : 0;
  p->q_weight = q_weight, p->k_weight = k_weight;
  p->w32 = weight_fp32 != 0, p->interleaved = interleaved != 0;
  p->B = B, p->H = H, p->Hkv = Hkv, p->N = N, p->rot = rot, p->n_pos = n_pos;
  p->eps = eps;
  return FA_OK;
}

int fa_qk_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* q_out, const fa_heads* k_out,
                    const float* cos, const float* sin, const int* positions, int positions_per_batch,
                    const void* q_weight, const void* k_weight, int weight_fp32, int B, int H, int Hkv, int N, int d,
                    int rot, int n_pos, float eps, int interleaved, void* stream) {
  fa::NormRope p;
  const int st = norm_rope_args(&p, q, k, q_out, k_out, cos, sin, positions, positions_per_batch, q_weight, k_weight,
                                weight_fp32, B, H, Hkv, N, d, rot, n_pos, eps, interleaved);
  if (st != FA_OK) return st;
  return map_cuda(fa::launch_norm_rope(p, d, static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int B, int N, int d) {
  if (B < 1 || N < 1 || (d != 64 && d != 128) || static_cast<long long>(B) * N > INT_MAX) return 0;
  return static_cast<size_t>(2) * fa::norm_rope_bwd_parts(B, N, d) * d * sizeof(float);
}

int fa_qk_norm_rope_bwd(const fa_heads* dq_out, const fa_heads* dk_out, const fa_heads* q, const fa_heads* k,
                        const fa_heads* dq, const fa_heads* dk, float* dq_weight, float* dk_weight, const float* cos,
                        const float* sin, const int* positions, int positions_per_batch, const void* q_weight,
                        const void* k_weight, int weight_fp32, void* workspace, size_t ws_bytes, int B, int H, int Hkv,
                        int N, int d, int rot, int n_pos, float eps, int interleaved, void* stream) {
  if (!q_weight && !k_weight) q = dq_out, k = dk_out;  // no norm: q and k are not read
  fa::NormRope p;
  const int st = norm_rope_args(&p, q, k, dq_out, dk_out, cos, sin, positions, positions_per_batch, q_weight, k_weight,
                                weight_fp32, B, H, Hkv, N, d, rot, n_pos, eps, interleaved);
  if (st != FA_OK) return st;
  if (!dq || !dk || !dq->ptr || !dk->ptr || !heads_strides_ok(dq) || !heads_strides_ok(dk)) return FA_ERR_INVALID_ARG;
  if (q_weight && (!dq_weight || !dk_weight)) return FA_ERR_INVALID_ARG;
  if (q_weight && (!workspace || ws_bytes < fa_qk_norm_rope_bwd_workspace_bytes(B, N, d))) return FA_ERR_WORKSPACE;
  if (!heads_aligned(dq) || !heads_aligned(dk) || !aligned16(workspace) || !aligned16(dq_weight) ||
      !aligned16(dk_weight))
    return FA_ERR_MISALIGNED;
  p.dq = head_rows(dq, B, H, N, d);
  p.dk = head_rows(dk, B, Hkv, N, d);
  return map_cuda(fa::launch_norm_rope_bwd(p, d, static_cast<float*>(workspace), dq_weight, dk_weight,
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

static int append_args(fa::Append* p, const fa_tokens* q, const fa_tokens* k, const fa_tokens* v,
                       const fa_tokens* q_out, void* k_cache, void* v_cache, const int* block_table,
                       const int* positions, const int* requests, const float* cos, const float* sin,
                       const void* q_weight, const void* k_weight, int weight_fp32, int T, int B, int H, int Hkv, int d,
                       int num_blocks, int block_size, int max_blocks, int rot, int n_pos, float eps,
                       int interleaved) {
  if (!k || !v || !k->ptr || !v->ptr || !k_cache || !v_cache || !block_table || !positions) return FA_ERR_INVALID_ARG;
  if (!tokens_strides_ok(k) || !tokens_strides_ok(v)) return FA_ERR_INVALID_ARG;
  const bool queries = q != nullptr;
  if (queries != (q_out != nullptr)) return FA_ERR_INVALID_ARG;
  if (queries && (!q->ptr || !q_out->ptr || H < 1 || !tokens_strides_ok(q) || !tokens_strides_ok(q_out)))
    return FA_ERR_INVALID_ARG;
  if (!queries && q_weight) return FA_ERR_INVALID_ARG;
  if (queries && (!q_weight) != (!k_weight)) return FA_ERR_INVALID_ARG;
  if (T < 1 || B < 1 || (!requests && T > B)) return FA_ERR_INVALID_ARG;
  int st = check_cache(Hkv, num_blocks, block_size, max_blocks);
  if (st != FA_OK) return st;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((st = check_rope(cos, sin, d, rot, n_pos, q_weight, k_weight, weight_fp32, eps)) != FA_OK) return st;
  if (H > 16384 || Hkv > 16384) return FA_ERR_UNSUPPORTED;
  if (!tokens_aligned(k) || !tokens_aligned(v) || (queries && (!tokens_aligned(q) || !tokens_aligned(q_out))) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !rope_aligned(cos, sin, rot, q_weight, k_weight) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(positions) |
        reinterpret_cast<uintptr_t>(requests)) & 3u))
    return FA_ERR_MISALIGNED;
  *p = fa::Append{};
  if (queries) {
    p->q = token_rows(q, T, H, d);
    p->q_out = token_rows(q_out, T, H, d);
  }
  p->k = token_rows(k, T, Hkv, d);
  p->v = token_rows(v, T, Hkv, d);
  p->k_cache = k_cache, p->v_cache = v_cache;
  p->block_table = block_table, p->positions = positions, p->requests = requests;
  p->cos = cos, p->sin = sin;
  p->q_weight = q_weight, p->k_weight = k_weight;
  p->w32 = weight_fp32 != 0, p->interleaved = interleaved != 0;
  p->T = T, p->B = B, p->H = queries ? H : 0, p->Hkv = Hkv;
  p->num_blocks = num_blocks, p->bs = block_size, p->max_blocks = max_blocks, p->rot = rot, p->n_pos = n_pos;
  p->eps = eps;
  return FA_OK;
}

int fa_append_paged(const fa_tokens* q, const fa_tokens* k, const fa_tokens* v, const fa_tokens* q_out, void* k_cache,
                    void* v_cache, const int* block_table, const int* positions, const int* requests, const float* cos,
                    const float* sin, const void* q_weight, const void* k_weight, int weight_fp32, int T, int B, int H,
                    int Hkv, int d, int num_blocks, int block_size, int max_blocks_per_seq, int rot, int n_pos,
                    float eps, int interleaved, void* stream) {
  fa::Append p;
  const int st = append_args(&p, q, k, v, q_out, k_cache, v_cache, block_table, positions, requests, cos, sin,
                             q_weight, k_weight, weight_fp32, T, B, H, Hkv, d, num_blocks, block_size,
                             max_blocks_per_seq, rot, n_pos, eps, interleaved);
  if (st != FA_OK) return st;
  return map_cuda(fa::launch_append(p, d, false, static_cast<cudaStream_t>(stream)));
}

int fa_append_paged_q4(const fa_tokens* q, const fa_tokens* k, const fa_tokens* v, const fa_tokens* q_out,
                       void* k_cache, void* k_scale, void* v_cache, void* v_scale, void* k_values, void* v_values,
                       const int* block_table, const int* positions, const int* requests, const float* cos,
                       const float* sin, const void* q_weight, const void* k_weight, int weight_fp32, int T, int B,
                       int H, int Hkv, int d, int num_blocks, int block_size, int max_blocks_per_seq, int rot,
                       int n_pos, float eps, int interleaved, void* stream) {
  if (!k_scale || !v_scale || (!k_values) != (!v_values)) return FA_ERR_INVALID_ARG;
  fa::Append p;
  const int st = append_args(&p, q, k, v, q_out, k_cache, v_cache, block_table, positions, requests, cos, sin,
                             q_weight, k_weight, weight_fp32, T, B, H, Hkv, d, num_blocks, block_size,
                             max_blocks_per_seq, rot, n_pos, eps, interleaved);
  if (st != FA_OK) return st;
  if (!aligned16(k_scale) || !aligned16(v_scale) || !aligned16(k_values) || !aligned16(v_values))
    return FA_ERR_MISALIGNED;
  p.k_scale = static_cast<__nv_bfloat16*>(k_scale), p.v_scale = static_cast<__nv_bfloat16*>(v_scale);
  p.k_values = static_cast<__nv_bfloat16*>(k_values), p.v_values = static_cast<__nv_bfloat16*>(v_values);
  return map_cuda(fa::launch_append(p, d, true, static_cast<cudaStream_t>(stream)));
}

int fa_decode_q4_splits(int B, int H, int Hkv, int block_size, int max_blocks_per_seq) {
  if (B < 1 || H < 1 || check_heads(H, Hkv) != FA_OK || check_cache(Hkv, 1, block_size, max_blocks_per_seq) != FA_OK)
    return 0;
  return fa::decode_q4_splits(B, H, Hkv, static_cast<long long>(max_blocks_per_seq) * block_size);
}

int fa_decode_paged_q4(const void* q, const void* k_cache, const void* k_scale, const void* v_cache,
                       const void* v_scale, const int* block_table, const int* seq_lens, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int d, int num_blocks, int block_size,
                       int max_blocks_per_seq, float scale, int n_splits, void* stream) {
  if (!q || !k_cache || !k_scale || !v_cache || !v_scale || !block_table || !seq_lens || !o || !lse)
    return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || n_splits < 1) return FA_ERR_INVALID_ARG;
  int st = check_heads(H, Hkv);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = check_cache(Hkv, num_blocks, block_size, max_blocks_per_seq)) != FA_OK) return st;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<long long>(Hkv) * ((H / Hkv + 7) / 8) > 65535 || n_splits > 4096)
    return FA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < fa_decode_workspace_bytes(B, H, d, n_splits)) return FA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(k_scale) || !aligned16(v_cache) || !aligned16(v_scale) ||
      !aligned16(o) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_MISALIGNED;
  const size_t rows = static_cast<size_t>(n_splits) * B * H;
  fa::DecodeQ4 p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache), p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = static_cast<const uint32_t*>(k_scale), p.v_scale = static_cast<const uint32_t*>(v_scale);
  p.block_table = block_table, p.seq_lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o), p.lse = lse;
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        ((rows * d * sizeof(float) + 255) & ~static_cast<size_t>(255)));
  p.B = B, p.H = H, p.Hkv = Hkv, p.num_blocks = num_blocks, p.bs = block_size, p.max_blocks = max_blocks_per_seq;
  p.scale_log2 = scale * 1.4426950408889634f;
  return map_cuda(fa::launch_decode_q4(p, d, n_splits, static_cast<cudaStream_t>(stream)));
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
