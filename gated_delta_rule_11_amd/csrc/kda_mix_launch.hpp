// kda_mix_launch.hpp -- argument blocks between the C ABI layer and the launchers of the
// linear-attention, prompt-attention and cache-attention kernels.  All pointers are device
// pointers already validated by the ABI layer.
#pragma once

#include "kda_launch.hpp"

namespace kda {

// ---- linear attention with a decay per head -------------------------------------------

// Tokens of a chunk: the fp32 kernels' tiles of 64 tokens would not fit the LDS.
__host__ __device__ constexpr int linear_chunk(bool bf16) { return bf16 ? 64 : 32; }

struct LinearArgs {
  const void *q, *k, *v;  // [B, T, H, d]
  const float* g;         // [B, T, H], or [H] when g_head
  const float* S_in;      // entry states (see S_in_seg), or nullptr
  void* o;                // [B, T, H, dv]; nullptr: no outputs
  float* S_out;           // [B, H, nseg, dk, dv] (S_out_seg) or [B, H, dk, dv] of the last segment, or nullptr
  float* ckpt;            // [B, H, chunks, dk, dv]: the state entering each chunk, or nullptr
  int B, T, H, dk, dv;
  float scale;
  bool in_bf16, out_bf16, g_head;
  int nseg = 1, seg_chunks = 0;  // segments of a sequence, chunks of each
  bool S_in_seg = false, S_out_seg = false;
  float* seg_decay = nullptr;  // [B, H, nseg]: each segment's total decay (written with S_out_seg)
  // the backward's state: walks the chunks from the last to the first, adding
  // scale e^G q do^T (k = q, v = do), segment 0 being the sequence's last
  bool reverse = false;
};
hipError_t launch_linear_walk(const LinearArgs& a, hipStream_t st);

// E_0 = S_in (or 0), E_{p+1} = decay_p E_p + St_p over a sequence's segments.
struct LinearScanArgs {
  const float *S_in, *St, *decay;  // [BH, n] or nullptr, [BH, nseg, n], [BH, nseg]
  float* E;                        // [BH, nseg, n]
  int64_t BH;
  int nseg, n;
};
hipError_t launch_linear_scan(const LinearScanArgs& a, hipStream_t st);

struct LinearBwdArgs {
  const void *q, *k, *v, *d_o;
  const float* g;
  const float *S, *R;  // [B, H, chunks, dk, dv]: the state entering, and the gradient leaving, each chunk
  void *dq, *dk_, *dv_;
  float* dg;  // [B, T, H]
  int B, T, H, dk, dv;
  float scale;
  bool in_bf16, grad_bf16, g_head;
};
hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t st);
// dg [H] = sums of x [B, T, H] over batch and tokens
hipError_t launch_linear_dg_sum(const float* x, float* dg, int64_t rows, int H, hipStream_t st);

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
};
hipError_t launch_prompt_fwd(const PromptArgs& a, hipStream_t st);

struct PromptBwdArgs {
  const void *q, *k, *v, *o, *d_o;
  const float* lse;
  const int* cu;
  float* D;  // [n, Hq] scratch
  void *dq, *dk, *dv;
  int n, nseq, Hq, Hkv, d;
  float scale;
  bool in_bf16, o_bf16, grad_bf16;  // d_o is in the inputs' type
};
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
