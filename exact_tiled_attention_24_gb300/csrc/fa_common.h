// Declarations shared by the C-ABI layer and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

// Heads whose tiles are scheduled together: the CTAs resident at one time
// then re-read one group's shared operand (K and V in the forward and the
// dQ sweep, Q and dO in the dK/dV sweep), and the group is sized so that
// operand stays in L2 (about 40 MB of the 129 MB). `bytes_per_head` is the
// shared operand's size per scheduled head.
constexpr long long kL2GroupBytes = 40ll << 20;
inline int head_group_for(long long bytes_per_head, int max_group) {
  long long g = bytes_per_head > 0 ? kL2GroupBytes / bytes_per_head : max_group;
  if (g > max_group) g = max_group;
  return g < 1 ? 1 : static_cast<int>(g);
}

// Kernel launchers. Pointers are device pointers to contiguous [BH][N][d]
// bf16 tensors (lse, Dvec: [BH][N] fp32); k, v, dk and dv hold BH / G heads,
// query head h reading K/V head h / G (G = 1: one K/V head per query head).
// Each launcher builds the TMA descriptors its kernel needs. Arguments are
// assumed validated by the caller. Return the launch (or descriptor) error.
cudaError_t launch_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int BH,
                       int G, int N, int d, float scale, bool causal, cudaStream_t stream);
cudaError_t launch_bwd_preprocess(const __nv_bfloat16* o, const __nv_bfloat16* dO, float* Dvec,
                                  int BH, int N, int d, cudaStream_t stream);
cudaError_t launch_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO, void* dk,
                            void* dv, const float* lse, const float* Dvec, int BH, int G, int N, int d,
                            float scale, bool causal, cudaStream_t stream);
cudaError_t launch_bwd_dq(const void* q, const void* k, const void* v, const void* dO, void* dq,
                          const float* lse, const float* Dvec, int BH, int G, int N, int d, float scale,
                          bool causal, cudaStream_t stream);
// Whether the full backward forms D inside the dQ sweep and runs the dK/dV
// sweep after it, instead of a separate D pass and the two sweeps side by
// side: with one K/V head per query head (G = 1) and a dK/dV grid of at
// least four CTAs per SM. Measured: c4 2.354 against 2.382 ms, B=16 H=16
// N=2048 causal 0.795 against 0.821; with grouped-query heads or small
// grids the two sweeps sharing one tail is worth more than the D pass.
bool bwd_fuse_d(int BH, int G, int N);
// The dQ sweep that also forms D = rowsum(dO ∘ O) of its query tiles from o
// and writes it to Dvec (for a dK/dV sweep launched after it).
cudaError_t launch_bwd_dq_d(const void* q, const void* k, const void* v, const void* o, const void* dO,
                            void* dq, const float* lse, float* Dvec, int BH, int G, int N, int d, float scale,
                            bool causal, cudaStream_t stream);

// Row softmax of x [rows][n] fp32 into y (may alias x): three passes (safe)
// or two (online). One CTA per row.
cudaError_t launch_softmax(const float* x, float* y, long long rows, int n, bool online,
                           cudaStream_t stream);

// Decode of one new query row per request against a paged KV cache
// (k_cache, v_cache [num_blocks][Hkv][block_size][d] bf16), split over the
// context into S parts, partial results in o_part [S][B*H][d] fp32 and
// lse_part [S][B*H], then merged into o [B*H][d] bf16 and lse [B*H].
cudaError_t launch_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                                const int* block_table, const int* seq_lens, void* o, float* lse,
                                float* o_part, float* lse_part, int B, int H, int Hkv, int d,
                                int num_blocks, int block_size, int max_blocks, float scale, int S,
                                cudaStream_t stream);
// Merge S partial attention results per row: o_parts [S][rows][d] fp32,
// lse_parts [S][rows] -> o [rows][d] bf16, lse [rows].
cudaError_t launch_attn_merge(const float* o_parts, const float* lse_parts, int S, void* o, float* lse,
                              long long rows, int d, cudaStream_t stream);

// ---- between the projections and the attention kernels (fa_rope.cu)
// A [B][heads][N][d] bf16 tensor with unit stride in d: strides of the other
// dimensions in elements, and the elements from p to the last one's end.
struct HeadRows {
  __nv_bfloat16* p;
  long long sb, sh, sn;
  long long extent;
};
// Rotations with several position axes: pair i of a token's rotated dimensions
// turns by its position on one axis. n = 0: one position a token.
struct Axes {
  const int* positions;  // [n][stride]
  long long stride;
  int n;
  unsigned long long of_pair[2];  // two bits a pair: its axis
};
// Arguments of the norm and rotation kernels. No norm: the weights are null.
// No rotation: rot = 0. The backward takes dy in q_out and k_out.
struct NormRope {
  HeadRows q, k, q_out, k_out, dq, dk;
  const float* cos;      // [n_pos][rot / 2]
  const float* sin;
  const int* positions;  // [N], or [B][N] with pos_sb = N; null: token n is at position n
  long long pos_sb;
  const void* q_weight;  // [d], bf16, or fp32 with w32
  const void* k_weight;
  bool w32, interleaved;
  int B, H, Hkv, N, rot, n_pos;
  float eps;
  Axes axes;  // with n > 0: positions as [n][B][N] (pos_sb = N) or [n][N] in place of `positions`
  int q_sections, k_sections;  // set by the launcher: parts that the heads are cut into
};
cudaError_t launch_norm_rope(const NormRope& p, int d, cudaStream_t stream);
// Workspace of the weight gradients' partial rows.
size_t norm_rope_bwd_partial_bytes(int d);
cudaError_t launch_norm_rope_bwd(const NormRope& p, int d, float* partial, float* dqw, float* dkw,
                                 cudaStream_t stream);

// ---- appending to a paged cache (fa_append.cu)
// A [T][heads][d] bf16 tensor with unit stride in d.
struct TokenRows {
  __nv_bfloat16* p;
  long long st, sh;
  long long extent;
};
struct Append {
  TokenRows q, k, v, q_out;  // q.p null: no queries (H = 0)
  void* k_cache;             // bf16 [num_blocks][Hkv][bs][d], or codes [...][d / 2]
  void* v_cache;
  __nv_bfloat16* k_scale;    // [num_blocks][Hkv][bs][d / 64][2], 4-bit caches only
  __nv_bfloat16* v_scale;
  __nv_bfloat16* k_values;   // [T][Hkv][d] values held, or null
  __nv_bfloat16* v_values;
  const int* block_table;    // [B][max_blocks]
  const int* positions;      // [T]
  const int* requests;       // [T], or null: token t is request t's
  const float* cos;
  const float* sin;
  const void* q_weight;
  const void* k_weight;
  bool w32, interleaved, zero_skipped;
  int T, B, H, Hkv, num_blocks, bs, max_blocks, rot, n_pos;
  float eps;
  Axes axes;  // with n > 0: the tokens' rotary positions, [n][T]; `positions` are slots only
  int q_sections, kv_sections;  // set by the launcher: parts that the heads are cut into
};
cudaError_t launch_append(const Append& p, int d, bool q4, cudaStream_t stream);

// ---- decode over a cache in 4-bit codes (fa_decode_q4.cu)
struct DecodeQ4 {
  const __nv_bfloat16* q;    // [B][H][d]
  const uint8_t* k_cache;    // [num_blocks][Hkv][bs][d / 2]
  const uint8_t* v_cache;
  const uint32_t* k_scale;   // (s, z) pairs, [num_blocks][Hkv][bs][d / 64]
  const uint32_t* v_scale;
  const int* block_table;
  const int* seq_lens;
  __nv_bfloat16* o;
  float* lse;
  float* o_part;             // [S][B·H][d], [S][B·H]: partial results, S > 1
  float* lse_part;
  int B, H, Hkv, num_blocks, bs, max_blocks;
  float scale_log2;
};
int decode_q4_splits(int B, int H, int Hkv, long long max_ctx);
cudaError_t launch_decode_q4(const DecodeQ4& p, int d, int S, cudaStream_t stream);

// ---- attention of chunks of new tokens over a paged cache (fa_extend.cu)
// An item of work that a CTA's share begins within.
struct ItemCut {
  int parts;  // 0: none
  int nth;    // the CTA's place among those that share it (0 has its first tile)
  int tok0, ntok, head0, heads;
};
struct Extend {
  const void* k_cache;       // bf16 [num_blocks][Hkv][bs][d], or codes [...][d / 2]
  const void* v_cache;
  const uint32_t* k_scale;   // (s, z) pairs, [num_blocks][Hkv][bs][d / 64], 4-bit caches only
  const uint32_t* v_scale;
  const int* block_table;    // [B][max_blocks]
  const int* seq_lens;       // [B]
  const int* q_starts;       // [B + 1]
  __nv_bfloat16* o;          // [T][H][d]
  float* lse;                // [T][H]
  float* o_part;             // [n_slots][d / 4][256][4]: normalised parts of cut items
  float* lse_part;           // [n_slots][256]
  ItemCut* cuts;             // [ctas]
  int T, B, H, Hkv, num_blocks, bs, max_blocks;
  int heads, hv;             // query heads a tile holds (at most 128), K/V heads times the parts its query heads are cut into
  int tpt;                   // tokens a query tile holds: 128 / heads
  int ctas, lc, may_chunk, chunk_halves;  // see fa_extend_plan.cuh
  unsigned bs_inverse;       // 2^32 / bs, rounded up (bs = 1: 1)
  int n_slots, n_long;       // workspace parts; long items there may be
  bool causal, zero_skipped;
  float scale_log2;
  // The block of a key below 2^30: the product is at most key / 2^32 < 1 too
  // large, so one too many at most.
  __host__ __device__ int block_of(int key) const {
    if (bs == 1) return key;
    const int q = static_cast<int>((static_cast<unsigned long long>(bs_inverse) * static_cast<unsigned>(key)) >> 32);
    return q * bs > key ? q - 1 : q;
  }
};
// Sets the fields from `heads` to `n_long` from the sizes; returns the workspace's bytes.
size_t extend_sizes(Extend* p, int d, bool q4);
cudaError_t launch_extend(const Extend& p, const void* q, int d, bool q4, cudaStream_t stream);

// The calling host thread's side stream on the current device (a
// non-blocking stream the library creates on first use and keeps).
cudaError_t side_stream(cudaStream_t* out);

// Device error words (one per translation unit): read, then clear.
cudaError_t launch_wait_limit_selftest(cudaStream_t stream);
cudaError_t read_and_clear_selftest_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_fwd_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_bwd_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_decode_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_softmax_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_rope_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_append_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_decode_q4_error(uint32_t* out, cudaStream_t stream);
cudaError_t read_and_clear_extend_error(uint32_t* out, cudaStream_t stream);

}  // namespace fa
