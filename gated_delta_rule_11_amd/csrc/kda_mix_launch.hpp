// kda_mix_launch.hpp -- argument blocks between the C ABI layer and the launchers of the
// linear-attention, prompt-attention and cache-attention kernels.  All pointers are device
// pointers already validated by the ABI layer.
#pragma once

#include "kda_launch.hpp"

namespace kda {

// ---- linear attention with a decay per head -------------------------------------------

// Tokens of a chunk: the fp32 kernels' tiles of 64 tokens would not fit the LDS.
__host__ __device__ constexpr int linear_chunk(bool bf16) { return bf16 ? 64 : 32; }

// Threads of a walk's workgroup: a wavefront for every 16 value columns, of up to 64, and one for every
// 16 tokens of a chunk (fewer where only the state is wanted).
__host__ __device__ constexpr int linear_threads(bool bf16, int dv) {
  return 64 * ((dv < 64 ? dv : 64) / 16 + linear_chunk(bf16) / 16);
}
__host__ __device__ constexpr int linear_slices(int dv) { return dv > 64 ? 2 : 1; }

// Chunks between the states that the backward keeps for dg.  Within a block dg is a difference of
// sums over the block's tokens.  B = 4, H = 32, T = 4001, d = 128, forward and backward: 773 us and dg within
// 1.0e-6 of the 64-bit result at 8 chunks, 793 us and 0.67e-6 at 4, 832 us and 0.48e-6 at 2.
constexpr int kBlockChunks = 4;

// A walk over the chunks (kda_linear_walk.hpp); q, k, v are roles there: dk is q's and k's size, dv v's.
struct LinearArgs {
  const void *q, *k, *v;  // [B, T, H, d]
  const float* g;         // [B, T, H], or [H] when g_head
  const float* S_in;      // entry states (see S_in_seg), or nullptr
  void* o;                // [B, T, H, dv]; nullptr: no outputs
  float* S_out;           // [B, H, nseg, dk, dv] (S_out_seg) or [B, H, dk, dv] of the last segment, or nullptr
  int B, T, H, dk, dv;
  float scale;
  bool in_bf16, out_bf16, g_head;
  bool reverse = false;           // from the last chunk to the first
  bool state_tr = false;          // S_in (not a segment's) is [B, H, dv, dk]
  int nseg = 1, seg_chunks = 0;   // segments of a sequence, chunks of each
  bool S_in_seg = false, S_out_seg = false;
  float* seg_decay = nullptr;     // [B, H, nseg]: each segment's total decay (written with S_out_seg)
  // For dg: the outputs' dot products with `dot` ([B, T, H, dv]) into x [dv / 16, B, H, T]; a forward walk
  // keeps its states every kBlockChunks chunks in ckpt [B, H, blocks + 1, dk dv], a reverse walk
  // multiplies its own with them into bsum [B, H, blocks, dv / 16].
  const void* dot = nullptr;
  float *x = nullptr, *ckpt = nullptr, *bsum = nullptr;
};
hipError_t launch_linear_fwd_bf16(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_fwd_f32(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_rev_bf16(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_rev_f32(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_walk(const LinearArgs& a, hipStream_t st);

struct LinearScanArgs {
  const float *S_in, *St, *decay;  // [BH, dk dv] or nullptr, [BH, nseg, dk dv], [BH, nseg]
  float* E;                        // [BH, nseg, dk dv]
  int64_t BH;
  int nseg, dk, dv;
  bool state_tr;  // S_in is [BH, dv, dk]
};
hipError_t launch_linear_scan(const LinearScanArgs& a, hipStream_t st);

struct LinearDgArgs {
  const float *xq, *xk, *bsum;  // [parts, BH, T], [BH, blocks, parts]
  float* dg;                    // [B, T, H]
  double* block_sum;            // [BH, blocks]: the blocks' sums of dg instead, or nullptr
  int64_t BH;
  int T, H, parts, block;       // block: tokens, at most 256
};
hipError_t launch_linear_dg(const LinearDgArgs& a, hipStream_t st);
// dg [H] = sums of x [B, H, blocks] over batch and blocks
hipError_t launch_linear_dg_sum(const double* x, float* dg, int64_t B, int H, int64_t blocks, hipStream_t st);

struct LinearStepArgs {
  const void *q, *k, *v;  // [N, H, d]
  const float* g;         // [N, H] or [H]
  const float* S_in;
  float* S_out;  // may equal S_in
  void* o;
  int N, H, dk, dv;
  float scale;
  bool in_bf16, out_bf16, g_head;
};
hipError_t launch_linear_step(const LinearStepArgs& a, hipStream_t st);

// ---- causal attention over packed prompts ---------------------------------------------

struct PromptArgs {
  const void *q, *k, *v;  // [n, Hq, d], [n, Hkv, d]
  const int* cu;          // [nseq + 1]
  void* o;                // [n, Hq, d]
  float* lse;             // [n, Hq] or nullptr
  int n, nseq, Hq, Hkv, d;
  float scale;
  bool in_bf16, out_bf16;
  bool zero_tail;  // outputs of rows behind the last sequence: set to zero, or left
};
hipError_t launch_prompt_fwd(const PromptArgs& a, hipStream_t st);

struct PromptBwdArgs {
  const void *q, *k, *v, *o, *d_o;
  const float* lse;
  const int* cu;
  float* D;     // [n, Hq] scratch
  float* part;  // [parts, 2, n, Hkv, d] scratch when parts > 1
  void *dq, *dk, *dv;
  int n, nseq, Hq, Hkv, d, parts;
  float scale;
  bool in_bf16, o_bf16, grad_bf16;  // d_o is in the inputs' type
  bool zero_tail;
};
int prompt_bwd_parts(int n, int Hq, int Hkv);
hipError_t launch_prompt_bwd(const PromptBwdArgs& a, hipStream_t st);

// ---- attention over a paged cache in 8 bits -------------------------------------------

struct CacheAppendArgs {
  const void *k, *v;  // [n, Hkv, d]
  const int *cu, *ctx, *table;
  uint8_t *kc, *vc;  // [pages, Hkv, page, d], [pages, Hkv, d, page]
  float *ks, *vs;    // [pages, Hkv]
  int n, N, Hkv, d, page, pages, max_pages;
  bool in_bf16;
};
hipError_t launch_cache_append(const CacheAppendArgs& a, hipStream_t st);

struct CacheStepArgs {
  const void* q;  // [N, Hq, d]
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int *table, *ctx;
  void* o;
  float* lse;   // [N, Hq] or nullptr
  float* part;  // [N, Hq, splits, d + 2] when splits > 1
  int N, Hq, Hkv, d, page, pages, max_pages, splits;
  float scale;
  bool in_bf16, out_bf16;
};
int cache_step_splits(int N, int Hq, int Hkv, int page, int max_pages);
hipError_t launch_cache_step(const CacheStepArgs& a, hipStream_t st);

}  // namespace kda
