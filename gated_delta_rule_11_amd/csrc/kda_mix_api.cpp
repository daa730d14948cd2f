// kda_mix_api.cpp -- the C ABI of the mixers beside the delta rule (declared in
// include/kda.h): linear attention with a decay per head, causal attention over packed prompts,
// attention over a paged cache in 8 bits.  As everywhere in the library, arguments are validated
// on the host first, on any error nothing is launched, and launches are asynchronous on the
// caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_checks.hpp"
#include "kda_mix_launch.hpp"

using namespace kda;

namespace {

// A launch holds fewer than 2^32 threads.  In workgroups of 256, which all kernels here have but the
// linear walks (linear_threads; see walk_grid_ok):
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

// ---- linear attention -------------------------------------------------------------------

struct LinearForm {
  int64_t nch;      // chunks of a sequence
  int nseg;         // segments, 1: one walk
  int seg_chunks;
};

// A walk runs one workgroup per (b, h, slice of up to 64 value columns), chunk after chunk.  Where
// that leaves compute units without work the sequence is cut into segments of at least
// kMinSegChunks chunks, as many as keep to one workgroup per compute unit: the end states then
// cost one more pass over k and v.  Measured, at most 128 : 256 : 512 workgroups, us: bf16, d = 128,
// 8 heads of 131072 tokens 759 : 462 : 463; 32 of 16384 385 : 239 : 248; 128 of 8192 294 : 297 : 466
// (512 cuts them in two); fp32, 8 of 16384 342 : 193 : 205; with gradients, 8 of 16384 524 : 327 :
// 372.  Segments of at least 2 : 4 : 16 chunks, us: bf16, 8 heads of 512 tokens 24 : 24 : 19 and of
// 2048 27 : 28 : 57; fp32, 4 heads of 1024 27 : 35 : 93.
constexpr int64_t kUnits = 256;
// A chunk's rows of all heads stay within the 32-bit offsets of its copies.
constexpr int64_t kMaxRow = int64_t(1) << 22;
bool linear_sizes_ok(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv) {
  return sizes_ok(B, T, H, dk, dv) && H * dk <= kMaxRow && H * dv <= kMaxRow;
}
constexpr int64_t kMinSegChunks = 4;
// Nor is a sequence of fewer chunks than this cut: two more launches cost what they save.  Measured,
// cut : whole, us, 8 heads: 8 chunks, bf16, 24 : 19 (d = 128) and 23 : 16 (64), fp32 33 : 34 and 22 : 15
// (32), with gradients 107 : 102, 86 : 84, 137 : 146 and 69 : 61; 12 chunks 24 : 27, 23 : 21, 34 : 49,
// with gradients 110 : 144, 87 : 118, 140 : 210.  Fewer heads are alike (one of 12 chunks, d = 128: 23 : 25
// and, gradients alone, 82 : 117); at 64, with two segments each, cutting gains little or costs up to a
// third: 12 chunks, d = 128, bf16 36 : 27 and 131 : 125, fp32 50 : 50 and 160 : 170, d = 64 23 : 22 and 82 : 102.
constexpr int64_t kMinCutChunks = 12;
LinearForm linear_form(int64_t B, int64_t T, int64_t H, int dv, bool bf16) {
  const int C = linear_chunk(bf16);
  LinearForm f{(T + C - 1) / C, 1, 0};
  f.seg_chunks = int(f.nch);
  const int64_t units = B * H * linear_slices(dv);
  if (units <= 0 || f.nch < kMinCutChunks) return f;
  int64_t segs = kUnits / units;
  segs = segs < f.nch / kMinSegChunks ? segs : f.nch / kMinSegChunks;
  if (segs < 2) return f;
  f.seg_chunks = int((f.nch + segs - 1) / segs);
  f.nseg = int((f.nch + f.seg_chunks - 1) / f.seg_chunks);
  return f;
}

int64_t align4(int64_t floats) { return (floats + 3) & ~int64_t(3); }

// Floats of a segmented walk: end states, entry states, decays.
int64_t seg_floats(const LinearForm& f, int64_t bh, int64_t state) {
  return f.nseg <= 1 ? 0 : bh * f.nseg * 2 * state + align4(bh * f.nseg);
}

// Every segment's entry state into the workspace (a.S_in_seg set), or nothing for one segment.
hipError_t enter_segments(LinearArgs& a, const LinearForm& f, float* ws, hipStream_t st) {
  a.nseg = f.nseg;
  a.seg_chunks = f.seg_chunks;
  if (f.nseg <= 1) return hipSuccess;
  const int64_t bh = int64_t(a.B) * a.H, state = int64_t(a.dk) * a.dv;
  float* St = ws;
  float* E = St + bh * f.nseg * state;
  float* decay = E + bh * f.nseg * state;
  LinearArgs p = a;  // end states from zero
  p.o = nullptr; p.S_in = nullptr; p.dot = nullptr;
  p.S_out = St; p.S_out_seg = true; p.seg_decay = decay;
  hipError_t e = launch_linear_walk(p, st);
  if (e != hipSuccess) return e;
  e = launch_linear_scan(LinearScanArgs{a.S_in, St, decay, E, bh, f.nseg, a.dk, a.dv, a.state_tr}, st);
  a.S_in = E;
  a.S_in_seg = true;
  return e;
}

// A walk's launch: one workgroup per (b, h, slice), or up to kUnits of them where sequences are cut.  (The
// scan between walks runs for cut sequences only, at most kUnits / 2 heads.)
bool walk_grid_ok(int64_t B, int64_t H, int dv, bool bf16) {
  return B * H * linear_slices(dv) * linear_threads(bf16, dv) <= 0xffffffffLL;
}

// The launches of a backward (the walks' value columns are those of k for dq and dk; dg has one workgroup
// per block), and sizes that keep its layout within 64 bits.
bool bwd_grid_ok(int64_t B, int64_t T, int64_t H, int dk, int dv, bool bf16) {
  const int64_t nblk = (T + linear_chunk(bf16) * kBlockChunks - 1) / (linear_chunk(bf16) * kBlockChunks);
  return walk_grid_ok(B, H, dk, bf16) && walk_grid_ok(B, H, dv, bf16) && B * H * nblk <= kMaxGrid / 2;
}

// Workspace of the backward, in floats: kept states, dot products and boundary terms for dg, one
// walk's segments at a time, the blocks' sums of dg (64 bits) when g is per head.
struct BwdLayout {
  LinearForm fk, fv;  // walks over value columns of dk, and of dv
  int64_t nblk, ckpt, x, bsum, seg, dg, total;
};
BwdLayout bwd_layout(int64_t B, int64_t T, int64_t H, int dk, int dv, bool bf16, bool g_head) {
  BwdLayout l{};
  l.fk = linear_form(B, T, H, dk, bf16);
  l.fv = linear_form(B, T, H, dv, bf16);
  const int64_t bh = B * H, state = int64_t(dk) * dv;
  l.nblk = (l.fk.nch + kBlockChunks - 1) / kBlockChunks;
  l.ckpt = bh * (l.nblk + 1) * state;
  l.x = align4(bh * T * (dk / 16));
  l.bsum = align4(bh * l.nblk * (dk / 16));
  const int64_t a = seg_floats(l.fk, bh, state), b = seg_floats(l.fv, bh, state);
  l.seg = align4(a > b ? a : b);
  l.dg = g_head ? align4(bh * l.nblk * 2) : 0;
  l.total = T > 0 ? l.ckpt + 2 * l.x + l.bsum + l.seg + l.dg : 0;
  return l;
}

// ---- prompts and cache ------------------------------------------------------------------

bool attn_dim_ok(int d) { return d == 64 || d == 128; }
bool page_ok(int p) { return p == 16 || p == 32 || p == 64; }

// n rows (or N sequences) of Hq heads in groups over Hkv, d wide.
kda_status heads_ok(int64_t n, int64_t Hq, int64_t Hkv, int64_t d) {
  // the last tile of rows ends within 32 bits
  if (!sizes_ok(n, 1, Hq, d, d) || Hkv < 1 || n > 0x7fffffffLL - 256) return KDA_ERR_SHAPE;
  if (!attn_dim_ok(int(d)) || Hq % Hkv != 0) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// Workspace of the prompts' backward: D, and the parts of dk and dv.
int64_t prompt_bwd_floats(int n, int Hq, int Hkv, int d) {
  const int parts = prompt_bwd_parts(n, Hq, Hkv);
  return align4(int64_t(n) * Hq) + (parts > 1 ? int64_t(parts) * 2 * n * Hkv * d : 0);
}

}  // namespace

extern "C" {

size_t kda_linear_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, kda_dtype in_dtype) {
  if (!dtype_ok(in_dtype) || !linear_sizes_ok(B, T, H, dk, dv) || !dim_ok(dk) || !dim_ok(dv)) return 0;
  return size_t(seg_floats(linear_form(B, T, H, dv, in_dtype == KDA_BF16), int64_t(B) * H, int64_t(dk) * dv)) * 4;
}

kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, kda_dtype in_dtype, const float* g,
                                int g_per_head, const float* S_in, void* o, kda_dtype o_dtype, float* S_out, int B,
                                int T, int H, int dk, int dv, float scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype)) return KDA_ERR_DTYPE;
  if (!linear_sizes_ok(B, T, H, dk, dv)) return KDA_ERR_SHAPE;
  if (!dim_ok(dk) || !dim_ok(dv) || !isfinite(scale) || (g_per_head != 0 && g_per_head != 1))
    return KDA_ERR_UNSUPPORTED;
  const bool bf16 = in_dtype == KDA_BF16;
  const LinearForm f = linear_form(B, T, H, dv, bf16);
  const int64_t bh = int64_t(B) * H, ntok = bh * T, state = int64_t(dk) * dv;
  if (bh == 0) return KDA_OK;
  if (!walk_grid_ok(B, H, dv, bf16)) return KDA_ERR_SHAPE;
  const int64_t need = seg_floats(f, bh, state) * 4;
  if (ntok > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_NULL;
  if (need > 0 && !workspace) return KDA_ERR_NULL;
  if (!all_aligned({q, k, v, o, S_in, S_out, need > 0 ? workspace : nullptr}, g, 4)) return KDA_ERR_ALIGN;
  if (workspace_bytes < size_t(need)) return KDA_ERR_WORKSPACE;
  const int64_t e = int64_t(esize(in_dtype));
  const Range rSi{S_in, bh * state * 4}, rSo{S_out, bh * state * 4}, ro{o, ntok * dv * int64_t(esize(o_dtype))},
      rw{need > 0 ? workspace : nullptr, need};
  const Range ins[] = {{q, ntok * dk * e}, {k, ntok * dk * e}, {v, ntok * dv * e}, {g, g_per_head ? H * 4 : ntok * 4}};
  for (const Range& in : ins)
    if (overlap(ro, in) || overlap(rSo, in) || overlap(rw, in)) return KDA_ERR_ALIAS;
  if (overlap(ro, rSi) || overlap(ro, rSo) || overlap(rw, ro) || overlap(rw, rSi) || overlap(rw, rSo))
    return KDA_ERR_ALIAS;
  if (overlap(rSo, rSi) && S_out != S_in) return KDA_ERR_ALIAS;
  LinearArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.S_in = S_in; a.o = o; a.S_out = S_out;
  a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.scale = scale;
  a.in_bf16 = bf16; a.out_bf16 = o_dtype == KDA_BF16; a.g_head = g_per_head != 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) a.o = nullptr;  // only the state passes through
  const hipError_t err = enter_segments(a, f, static_cast<float*>(workspace), st);
  if (err != hipSuccess) return from_hip(err);
  return from_hip(launch_linear_walk(a, st));
}

size_t kda_linear_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, kda_dtype in_dtype, int g_per_head) {
  if (!dtype_ok(in_dtype) || !linear_sizes_ok(B, T, H, dk, dv) || !dim_ok(dk) || !dim_ok(dv) ||
      !bwd_grid_ok(B, T, H, dk, dv, in_dtype == KDA_BF16))
    return 0;
  return size_t(bwd_layout(B, T, H, dk, dv, in_dtype == KDA_BF16, g_per_head != 0).total) * 4;
}

kda_status kda_linear_chunk_bwd(const void* q, const void* k, const void* v, kda_dtype in_dtype, const float* g,
                                int g_per_head, const float* S_in, const void* d_o, const float* dS_out, void* dq,
                                void* dk, void* dv, kda_dtype grad_dtype, float* dg, float* dS_in, int B, int T, int H,
                                int dk_dim, int dv_dim, float scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(grad_dtype)) return KDA_ERR_DTYPE;
  if (!linear_sizes_ok(B, T, H, dk_dim, dv_dim)) return KDA_ERR_SHAPE;
  if (!dim_ok(dk_dim) || !dim_ok(dv_dim) || !isfinite(scale) || (g_per_head != 0 && g_per_head != 1))
    return KDA_ERR_UNSUPPORTED;
  const bool bf16 = in_dtype == KDA_BF16;
  if (!bwd_grid_ok(B, T, H, dk_dim, dv_dim, bf16)) return KDA_ERR_SHAPE;
  const BwdLayout l = bwd_layout(B, T, H, dk_dim, dv_dim, bf16, g_per_head != 0);
  const int64_t bh = int64_t(B) * H, ntok = bh * T, state = int64_t(dk_dim) * dv_dim;
  if (bh == 0 && !g_per_head) return KDA_OK;
  if (ntok > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk || !dv || !dg)) return KDA_ERR_NULL;
  if (g_per_head && !dg) return KDA_ERR_NULL;
  const int64_t need = l.total * 4;
  if (need > 0 && !workspace) return KDA_ERR_NULL;
  if (!all_aligned({q, k, v, d_o, dq, dk, dv, S_in, dS_out, dS_in, need > 0 ? workspace : nullptr}, g, 4) ||
      !aligned(dg, 4))
    return KDA_ERR_ALIGN;
  if (workspace_bytes < size_t(need)) return KDA_ERR_WORKSPACE;
  const int64_t e = int64_t(esize(in_dtype)), eg = int64_t(esize(grad_dtype));
  const int64_t ng = g_per_head ? H : ntok;
  const Range ins[] = {{q, ntok * dk_dim * e}, {k, ntok * dk_dim * e}, {v, ntok * dv_dim * e}, {g, ng * 4},
                       {S_in, bh * state * 4}, {d_o, ntok * dv_dim * e}, {dS_out, bh * state * 4}};
  const Range outs[] = {{dq, ntok * dk_dim * eg}, {dk, ntok * dk_dim * eg}, {dv, ntok * dv_dim * eg}, {dg, ng * 4},
                        {dS_in, bh * state * 4}, {need > 0 ? workspace : nullptr, need}};
  for (const Range& o : outs) {
    for (const Range& in : ins)
      if (overlap(o, in)) return KDA_ERR_ALIAS;
    for (const Range& o2 : outs)
      if (&o2 != &o && overlap(o, o2)) return KDA_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* ckpt = static_cast<float*>(workspace);
  float* xq = ckpt + l.ckpt;
  float* xk = xq + l.x;
  float* bsum = xk + l.x;
  float* seg = bsum + l.bsum;
  double* block_sum = g_per_head ? reinterpret_cast<double*>(seg + l.seg) : nullptr;
  LinearArgs w{};
  w.B = B; w.T = T; w.H = H; w.scale = scale; w.g = g;
  w.in_bf16 = bf16; w.out_bf16 = grad_dtype == KDA_BF16; w.g_head = g_per_head != 0;
  w.ckpt = ckpt; w.bsum = bsum;
  hipError_t err = hipSuccess;
  auto walk = [&](LinearArgs x, const LinearForm& f) {
    if (T == 0) x.o = nullptr;  // only the state passes through
    err = enter_segments(x, f, seg, st);
    if (err == hipSuccess) err = launch_linear_walk(x, st);
  };
  if (bh > 0) {
    // dv, and the gradient of the entry state
    LinearArgs x = w;
    x.q = k; x.k = q; x.v = d_o; x.dk = dk_dim; x.dv = dv_dim; x.o = dv; x.reverse = true;
    x.S_in = dS_out; x.S_out = dS_in;
    if (T > 0 || dS_in) walk(x, l.fv);
    if (err == hipSuccess && T > 0) {  // dq, and the states
      LinearArgs y = w;
      y.q = d_o; y.k = v; y.v = k; y.dk = dv_dim; y.dv = dk_dim; y.o = dq;
      y.S_in = S_in; y.state_tr = true; y.dot = q; y.x = xq;
      walk(y, l.fk);
    }
    if (err == hipSuccess && T > 0) {  // dk, and the states' products with their gradients
      LinearArgs y = w;
      y.q = v; y.k = d_o; y.v = q; y.dk = dv_dim; y.dv = dk_dim; y.o = dk; y.reverse = true;
      y.S_in = dS_out; y.state_tr = true; y.dot = k; y.x = xk;
      walk(y, l.fk);
    }
    if (err == hipSuccess && T > 0)
      err = launch_linear_dg(LinearDgArgs{xq, xk, bsum, dg, block_sum, bh, T, H, dk_dim / 16, linear_chunk(bf16) * kBlockChunks}, st);
  }
  if (err == hipSuccess && g_per_head) err = launch_linear_dg_sum(block_sum, dg, B, H, l.nblk, st);
  return from_hip(err);
}

kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, kda_dtype in_dtype, const float* g,
                                  int g_per_head, const float* S_in, float* S_out, void* o, kda_dtype o_dtype, int N,
                                  int H, int dk, int dv, float scale, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype)) return KDA_ERR_DTYPE;
  if (!sizes_ok(N, 1, H, dk, dv)) return KDA_ERR_SHAPE;
  if (!dim_ok(dk) || !dim_ok(dv) || !isfinite(scale) || (g_per_head != 0 && g_per_head != 1))
    return KDA_ERR_UNSUPPORTED;
  const int64_t nh = int64_t(N) * H;
  if (nh == 0) return KDA_OK;
  if (nh > kMaxGrid) return KDA_ERR_SHAPE;
  if (!q || !k || !v || !g || !S_in || !S_out || !o) return KDA_ERR_NULL;
  if (!all_aligned({q, k, v, S_in, S_out, o}, g, 4)) return KDA_ERR_ALIGN;
  const int64_t e = int64_t(esize(in_dtype)), ns = nh * dk * dv * 4;
  const Range rSi{S_in, ns}, rSo{S_out, ns}, ro{o, nh * dv * int64_t(esize(o_dtype))};
  const Range ins[] = {{q, nh * dk * e}, {k, nh * dk * e}, {v, nh * dv * e}, {g, (g_per_head ? H : nh) * 4}};
  for (const Range& in : ins)
    if (overlap(rSo, in) || overlap(ro, in)) return KDA_ERR_ALIAS;
  if (overlap(rSo, ro) || overlap(rSi, ro) || (overlap(rSi, rSo) && S_in != S_out)) return KDA_ERR_ALIAS;
  return from_hip(launch_linear_step(LinearStepArgs{q, k, v, g, S_in, S_out, o, N, H, dk, dv, scale,
                                                    in_dtype == KDA_BF16, o_dtype == KDA_BF16, g_per_head != 0},
                                     static_cast<hipStream_t>(stream)));
}

kda_status kda_attn_prompt_fwd(const void* q, const void* k, const void* v, kda_dtype in_dtype, const int* cu_seqlens,
                               void* o, kda_dtype o_dtype, float* lse, int n, int n_seqs, int Hq, int Hkv, int d,
                               float scale, int zero_tail, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype)) return KDA_ERR_DTYPE;
  const kda_status s = heads_ok(n, Hq, Hkv, d);
  if (s == KDA_ERR_SHAPE || n_seqs < 0) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !isfinite(scale) || (zero_tail != 0 && zero_tail != 1)) return KDA_ERR_UNSUPPORTED;
  if (n == 0 || (n_seqs == 0 && !zero_tail)) return KDA_OK;
  if ((int64_t(n) + 127) / 128 * Hq > kMaxGrid) return KDA_ERR_SHAPE;
  if (!q || !k || !v || !cu_seqlens || !o) return KDA_ERR_NULL;
  if (!all_aligned({q, k, v, o}, cu_seqlens, 4) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
  const int64_t e = int64_t(esize(in_dtype)), nq = int64_t(n) * Hq, nk = int64_t(n) * Hkv;
  const Range ro{o, nq * d * int64_t(esize(o_dtype))}, rl{lse, nq * 4};
  const Range ins[] = {{q, nq * d * e}, {k, nk * d * e}, {v, nk * d * e}, {cu_seqlens, (int64_t(n_seqs) + 1) * 4}};
  for (const Range& in : ins)
    if (overlap(ro, in) || overlap(rl, in)) return KDA_ERR_ALIAS;
  if (overlap(ro, rl)) return KDA_ERR_ALIAS;
  return from_hip(launch_prompt_fwd(PromptArgs{q, k, v, cu_seqlens, o, lse, n, n_seqs, Hq, Hkv, d, scale,
                                               in_dtype == KDA_BF16, o_dtype == KDA_BF16, zero_tail != 0},
                                    static_cast<hipStream_t>(stream)));
}

size_t kda_attn_prompt_bwd_workspace_bytes(int n, int Hq, int Hkv, int d) {
  if (heads_ok(n, Hq, Hkv, d) != KDA_OK) return 0;
  return size_t(prompt_bwd_floats(n, Hq, Hkv, d)) * 4;
}

kda_status kda_attn_prompt_bwd(const void* q, const void* k, const void* v, kda_dtype in_dtype, const int* cu_seqlens,
                               const void* o, kda_dtype o_dtype, const float* lse, const void* d_o, void* dq, void* dk,
                               void* dv, kda_dtype grad_dtype, int n, int n_seqs, int Hq, int Hkv, int d, float scale,
                               int zero_tail, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype) || !dtype_ok(grad_dtype)) return KDA_ERR_DTYPE;
  const kda_status s = heads_ok(n, Hq, Hkv, d);
  if (s == KDA_ERR_SHAPE || n_seqs < 0) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !isfinite(scale) || (zero_tail != 0 && zero_tail != 1)) return KDA_ERR_UNSUPPORTED;
  if (n == 0 || (n_seqs == 0 && !zero_tail)) return KDA_OK;
  const int64_t nq = int64_t(n) * Hq, nk = int64_t(n) * Hkv;
  if ((int64_t(n) + 127) / 128 * Hq > kMaxGrid || (nq + 31) / 32 > kMaxGrid || nk * d / 1024 >= kMaxGrid)
    return KDA_ERR_SHAPE;
  if (!q || !k || !v || !cu_seqlens || !o || !lse || !d_o || !dq || !dk || !dv || !workspace) return KDA_ERR_NULL;
  if (!all_aligned({q, k, v, o, d_o, dq, dk, dv, workspace}, cu_seqlens, 4) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
  const int64_t need = prompt_bwd_floats(n, Hq, Hkv, d) * 4;
  if (workspace_bytes < size_t(need)) return KDA_ERR_WORKSPACE;
  const int64_t e = int64_t(esize(in_dtype)), eg = int64_t(esize(grad_dtype)), eo = int64_t(esize(o_dtype));
  const Range ins[] = {{q, nq * d * e}, {k, nk * d * e}, {v, nk * d * e}, {cu_seqlens, (int64_t(n_seqs) + 1) * 4},
                       {o, nq * d * eo}, {lse, nq * 4}, {d_o, nq * d * e}};
  const Range outs[] = {{dq, nq * d * eg}, {dk, nk * d * eg}, {dv, nk * d * eg}, {workspace, need}};
  for (const Range& x : outs) {
    for (const Range& in : ins)
      if (overlap(x, in)) return KDA_ERR_ALIAS;
    for (const Range& y : outs)
      if (&y != &x && overlap(x, y)) return KDA_ERR_ALIAS;
  }
  return from_hip(launch_prompt_bwd(PromptBwdArgs{q, k, v, o, d_o, lse, cu_seqlens, static_cast<float*>(workspace),
                                                  static_cast<float*>(workspace) + align4(nq), dq, dk, dv, n, n_seqs,
                                                  Hq, Hkv, d, prompt_bwd_parts(n, Hq, Hkv), scale, in_dtype == KDA_BF16,
                                                  o_dtype == KDA_BF16, grad_dtype == KDA_BF16, zero_tail != 0},
                                    static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_cache_append(const void* k, const void* v, kda_dtype in_dtype, const int* cu_seqlens,
                               const int* context_len, const int* block_table, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, int n, int N, int Hkv, int d, int page, int n_pages,
                               int max_pages, void* stream) {
  if (!dtype_ok(in_dtype)) return KDA_ERR_DTYPE;
  const kda_status s = heads_ok(n, Hkv, Hkv, d);
  if (s == KDA_ERR_SHAPE || N < 0 || n_pages < 0 || max_pages < 0 || page < 1) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !page_ok(page)) return KDA_ERR_UNSUPPORTED;
  if (n == 0 || N == 0 || n_pages == 0 || max_pages == 0) return KDA_OK;
  const int64_t ph = int64_t(n_pages) * Hkv;
  if ((int64_t(n) / page + 2 * int64_t(N)) * Hkv > kMaxGrid) return KDA_ERR_SHAPE;
  if (!k || !v || !cu_seqlens || !context_len || !block_table || !k_cache || !v_cache || !k_scale || !v_scale)
    return KDA_ERR_NULL;
  if (!all_aligned({k, v, k_cache, v_cache}, cu_seqlens, 4) || !aligned(context_len, 4) || !aligned(block_table, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return KDA_ERR_ALIGN;
  const int64_t e = int64_t(esize(in_dtype)), nk = int64_t(n) * Hkv * d;
  const Range ins[] = {{k, nk * e}, {v, nk * e}, {cu_seqlens, (int64_t(N) + 1) * 4}, {context_len, int64_t(N) * 4},
                       {block_table, int64_t(N) * max_pages * 4}};
  const Range outs[] = {{k_cache, ph * page * d}, {v_cache, ph * page * d}, {k_scale, ph * 4}, {v_scale, ph * 4}};
  for (const Range& x : outs) {
    for (const Range& in : ins)
      if (overlap(x, in)) return KDA_ERR_ALIAS;
    for (const Range& y : outs)
      if (&y != &x && overlap(x, y)) return KDA_ERR_ALIAS;
  }
  return from_hip(launch_cache_append(
      CacheAppendArgs{k, v, cu_seqlens, context_len, block_table, static_cast<uint8_t*>(k_cache),
                      static_cast<uint8_t*>(v_cache), k_scale, v_scale, n, N, Hkv, d, page, n_pages, max_pages,
                      in_dtype == KDA_BF16},
      static_cast<hipStream_t>(stream)));
}

size_t kda_attn_decode_step_workspace_bytes(int N, int Hq, int Hkv, int d, int page, int max_pages) {
  if (heads_ok(N, Hq, Hkv, d) != KDA_OK || !page_ok(page) || max_pages < 0 || N == 0) return 0;
  const int splits = cache_step_splits(N, Hq, Hkv, page, max_pages);
  return splits == 1 ? 0 : size_t(N) * Hq * splits * (size_t(d) + 2) * 4;
}

kda_status kda_attn_decode_step(const void* q, kda_dtype in_dtype, const void* k_cache, const void* v_cache,
                                const float* k_scale, const float* v_scale, const int* block_table,
                                const int* context_len, void* o, kda_dtype o_dtype, float* lse, int N, int Hq, int Hkv,
                                int d, int page, int n_pages, int max_pages, float scale, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype)) return KDA_ERR_DTYPE;
  const kda_status s = heads_ok(N, Hq, Hkv, d);
  if (s == KDA_ERR_SHAPE || n_pages < 0 || max_pages < 0 || page < 1) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !page_ok(page) || !isfinite(scale)) return KDA_ERR_UNSUPPORTED;
  if (N == 0) return KDA_OK;
  const int splits = cache_step_splits(N, Hq, Hkv, page, max_pages);
  const int64_t nq = int64_t(N) * Hq;
  if (nq * splits > kMaxGrid) return KDA_ERR_SHAPE;
  const size_t need = kda_attn_decode_step_workspace_bytes(N, Hq, Hkv, d, page, max_pages);
  if (!q || !context_len || !o || (need > 0 && !workspace)) return KDA_ERR_NULL;
  if (n_pages > 0 && max_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale || !block_table))
    return KDA_ERR_NULL;
  if (!all_aligned({q, o, k_cache, v_cache, need > 0 ? workspace : nullptr}, block_table, 4) ||
      !aligned(context_len, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lse, 4))
    return KDA_ERR_ALIGN;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  const int64_t ph = int64_t(n_pages) * Hkv;
  const Range ins[] = {{q, nq * d * int64_t(esize(in_dtype))}, {k_cache, ph * page * d}, {v_cache, ph * page * d},
                       {k_scale, ph * 4}, {v_scale, ph * 4}, {block_table, int64_t(N) * max_pages * 4},
                       {context_len, int64_t(N) * 4}};
  const Range outs[] = {{o, nq * d * int64_t(esize(o_dtype))}, {lse, nq * 4},
                        {need > 0 ? workspace : nullptr, int64_t(need)}};
  for (const Range& x : outs) {
    for (const Range& in : ins)
      if (overlap(x, in)) return KDA_ERR_ALIAS;
    for (const Range& y : outs)
      if (&y != &x && overlap(x, y)) return KDA_ERR_ALIAS;
  }
  // a cache of no pages leaves every token out: the kernel then sees a table of no pages and does not
  // read it (it may be NULL)
  return from_hip(launch_cache_step(
      CacheStepArgs{q, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), k_scale, v_scale,
                    block_table, context_len, o, lse, static_cast<float*>(workspace), N, Hq, Hkv, d, page, n_pages,
                    n_pages > 0 ? max_pages : 0, splits, scale, in_dtype == KDA_BF16, o_dtype == KDA_BF16},
      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
