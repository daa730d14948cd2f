// kda_serve_api.cpp -- the C ABI of what a serving step over the paged cache needs beside it
// (declared in include/kda.h): rotary positions, appending with the rotation on the way, attention
// of a chunk of new tokens.
// As everywhere in the library, arguments are validated on the host first, on any
// error nothing is launched, and launches are asynchronous on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_checks.hpp"
#include "kda_mix_launch.hpp"

using namespace kda;

namespace {

// n rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t n, stride, width;
};
Range span(const Rows& r) { return {r.p, r.n > 0 ? (r.n - 1) * r.stride + r.width : 0}; }
bool overlap(const Rows& a, const Range& b) { return kda::overlap(span(a), b); }
// Views of one buffer whose rows alternate share a range of memory but no byte.
bool overlap(const Rows& a, const Rows& b) {
  if (!kda::overlap(span(a), span(b))) return false;
  if (a.stride != b.stride || a.n < 2 || b.n < 2) return true;
  const int64_t off = int64_t(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const int64_t at = ((off % a.stride) + a.stride) % a.stride;  // b's rows within a's
  return at < a.width || at + b.width > a.stride;
}

// Rows of H heads of d: apart by at least their width, each on 16 bytes.
kda_status stride_ok(int64_t stride, int64_t H, int64_t d, size_t e) {
  if (stride < H * d || stride > (int64_t(1) << 28)) return KDA_ERR_SHAPE;  // (below: products of 64 bits)
  return (stride * int64_t(e)) % 16 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}

bool flag_ok(int x) { return x == 0 || x == 1; }
constexpr int kMaxAxes = 8, kMaxRopeDim = 256;
bool turn_ok(int rot, int d, int n_axes, int interleaved) {
  return rot >= 16 && rot % 16 == 0 && rot <= d && n_axes >= 1 && n_axes <= kMaxAxes && flag_ok(interleaved);
}

// What one wavefront turns: with `many`, so many rows that its lanes, a unit of 16 channels each, come out even with
// the heads (24 heads of 64 channels: two rows of eight heads at a time, 55 us for 65 by whole rows); all of the rows'
// heads, or fewer where that leaves the GPU short of wavefronts (256 rows of 32 heads of 128: 3.6 us in four parts, 4.6
// whole; 2000 rows 7.0 whole, 8.2 in four parts).
void rope_waves(RopeArgs& a, bool many) {
  const int most = 64 / (a.d / 16);
  a.side = most;
  a.rows = 1;
  if (many) {
    while (a.H % a.side != 0) --a.side;
    a.rows = most / a.side;
  }
  const int64_t all = (a.H + a.side - 1) / a.side, groups = (int64_t(a.n) + a.rows - 1) / a.rows;
  const int64_t want = groups < 1 ? 1 : (2048 + groups - 1) / groups, parts = want < all ? want : all;
  a.heads = int((all + parts - 1) / parts * a.side);
}

// Query heads that share a key head: the costs by which workgroups divide the work stay in 64 bits.
constexpr int kMaxGroup = 1024;

}  // namespace

extern "C" {

kda_status kda_rope(const void* x, kda_dtype in_dtype, int64_t x_stride, const int* positions, int n_axes,
                    const float* inv_freq, const int* axes, int rot, int interleaved, int inverse, void* y,
                    kda_dtype y_dtype, int64_t y_stride, int n, int H, int d, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(y_dtype)) return KDA_ERR_DTYPE;
  if (!sizes_ok(n, 1, H, d, d)) return KDA_ERR_SHAPE;
  if (d % 16 != 0 || d > kMaxRopeDim || !turn_ok(rot, d, n_axes, interleaved) || !flag_ok(inverse))
    return KDA_ERR_UNSUPPORTED;
  const size_t ex = esize(in_dtype), ey = esize(y_dtype);
  kda_status s = stride_ok(x_stride, H, d, ex), t = stride_ok(y_stride, H, d, ey);
  if (s == KDA_ERR_SHAPE || t == KDA_ERR_SHAPE) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  RopeArgs args{x, y, x_stride, y_stride, Rotation{positions, inv_freq, axes, n_axes, rot / 2, interleaved != 0}, n, H, d, 1, 1, 1,
                inverse != 0, in_dtype == KDA_BF16, y_dtype == KDA_BF16};
  rope_waves(args, true);
  if ((rope_items(args) + 3) / 4 > kMaxGrid) return KDA_ERR_SHAPE;
  if (!x || !positions || !inv_freq || !y) return KDA_ERR_NULL;
  if (s != KDA_OK || t != KDA_OK || !all_aligned({x, y}, positions, 4) || !aligned(inv_freq, 4) || !aligned(axes, 4))
    return KDA_ERR_ALIGN;
  const Rows rx{x, n, x_stride * int64_t(ex), int64_t(H) * d * int64_t(ex)};
  const Rows ry{y, n, y_stride * int64_t(ey), int64_t(H) * d * int64_t(ey)};
  const bool same = x == y && in_dtype == y_dtype && x_stride == y_stride;
  if (!same && overlap(ry, rx)) return KDA_ERR_ALIAS;
  const Range ins[] = {{positions, int64_t(n) * n_axes * 4}, {inv_freq, int64_t(rot) * 2}, {axes, int64_t(rot) * 2}};
  for (const Range& in : ins)
    if (overlap(ry, in)) return KDA_ERR_ALIAS;
  return from_hip(launch_rope(args, static_cast<hipStream_t>(stream)));
}

kda_status kda_kv_cache_append_rope(const void* k, int64_t k_stride, const void* v, int64_t v_stride, kda_dtype in_dtype,
                                    const void* q, int64_t q_stride, void* q_out, kda_dtype q_out_dtype,
                                    int64_t q_out_stride, const int* positions, int n_axes, const float* inv_freq,
                                    const int* axes, int rot, int interleaved, const int* cu_seqlens,
                                    const int* context_len, const int* block_table, void* k_cache, void* v_cache,
                                    float* k_scale, float* v_scale, int n, int N, int Hq, int Hkv, int d, int page,
                                    int n_pages, int max_pages, int zero_tail, void* stream) {
  if (!dtype_ok(in_dtype) || (q && !dtype_ok(q_out_dtype))) return KDA_ERR_DTYPE;
  kda_status s = heads_ok(n, q ? Hq : Hkv, Hkv, d);
  if (s == KDA_ERR_SHAPE || N < 0 || n_pages < 0 || max_pages < 0 || page < 1) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !page_ok(page) || !turn_ok(rot, d, n_axes, interleaved) || !flag_ok(zero_tail))
    return KDA_ERR_UNSUPPORTED;
  const size_t e = esize(in_dtype), eo = q ? esize(q_out_dtype) : e;
  const kda_status strides[] = {stride_ok(k_stride, Hkv, d, e), stride_ok(v_stride, Hkv, d, e),
                                q ? stride_ok(q_stride, Hq, d, e) : KDA_OK, q ? stride_ok(q_out_stride, Hq, d, eo) : KDA_OK};
  for (const kda_status t : strides)
    if (t == KDA_ERR_SHAPE) return t;
  const bool cache = N > 0 && n_pages > 0 && max_pages > 0, turns = q && (N > 0 || zero_tail);
  if (n == 0 || (!cache && !turns)) return KDA_OK;
  RopeArgs queries{turns ? q : nullptr, q_out, q_stride, q_out_stride,
                   Rotation{positions, inv_freq, axes, n_axes, rot / 2, interleaved != 0}, n, Hq, d, 1, 1, 1, false,
                   in_dtype == KDA_BF16, q_out_dtype == KDA_BF16};
  if (q) rope_waves(queries, false);
  const int64_t items = q ? (rope_items(queries) + 3) / 4 : 0;
  if ((int64_t(n) / page + 2 * int64_t(N)) * Hkv + items > kMaxGrid) return KDA_ERR_SHAPE;
  if (!inv_freq || !cu_seqlens || (N > 0 && !context_len) || (!positions && n_axes != 1) || (q && !q_out)) return KDA_ERR_NULL;
  if (cache && (!k || !v || !block_table || !k_cache || !v_cache || !k_scale || !v_scale)) return KDA_ERR_NULL;
  for (const kda_status t : strides)
    if (t != KDA_OK) return t;
  if (!all_aligned({k, v, q, q ? q_out : nullptr, k_cache, v_cache}, cu_seqlens, 4) || !aligned(context_len, 4) ||
      !aligned(block_table, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(positions, 4) ||
      !aligned(inv_freq, 4) || !aligned(axes, 4))
    return KDA_ERR_ALIGN;
  const int64_t ph = int64_t(n_pages) * Hkv, es = int64_t(e);
  const Rows rk{k, n, k_stride * es, Hkv * int64_t(d) * es}, rv{v, n, v_stride * es, Hkv * int64_t(d) * es};
  const Rows rq{q, n, q_stride * es, Hq * int64_t(d) * es};
  const Rows ro{q ? q_out : nullptr, n, q_out_stride * int64_t(eo), Hq * int64_t(d) * int64_t(eo)};
  const Range ins[] = {{cu_seqlens, (int64_t(N) + 1) * 4}, {context_len, int64_t(N) * 4},
                       {block_table, int64_t(N) * max_pages * 4}, {positions, int64_t(n) * n_axes * 4},
                       {inv_freq, int64_t(rot) * 2}, {axes, int64_t(rot) * 2}};
  const Range outs[] = {{k_cache, ph * page * d}, {v_cache, ph * page * d}, {k_scale, ph * 4}, {v_scale, ph * 4}};
  for (const Range& x : outs) {
    for (const Range& in : ins)
      if (kda::overlap(x, in)) return KDA_ERR_ALIAS;
    for (const Range& y : outs)
      if (&y != &x && kda::overlap(x, y)) return KDA_ERR_ALIAS;
    for (const Rows& r : {rk, rv, rq, ro})
      if (overlap(r, x)) return KDA_ERR_ALIAS;
  }
  for (const Range& in : ins)
    if (overlap(ro, in)) return KDA_ERR_ALIAS;
  const bool same = q && q == q_out && in_dtype == q_out_dtype && q_stride == q_out_stride;
  if (overlap(ro, rk) || overlap(ro, rv) || (!same && overlap(ro, rq))) return KDA_ERR_ALIAS;
  return from_hip(launch_cache_append_rope(
      CacheRopeArgs{CacheAppendArgs{k, v, cu_seqlens, context_len, block_table, static_cast<uint8_t*>(k_cache),
                                    static_cast<uint8_t*>(v_cache), k_scale, v_scale, n, cache ? N : 0, Hkv, d, page, n_pages,
                                    max_pages, in_dtype == KDA_BF16},
                    k_stride, v_stride, queries, N, zero_tail != 0},
      static_cast<hipStream_t>(stream)));
}

size_t kda_attn_chunk_fwd_workspace_bytes(int n, int N, int Hq, int Hkv, int d, int page, int max_pages,
                                          kda_dtype in_dtype) {
  if (!dtype_ok(in_dtype) || heads_ok(n, Hq, Hkv, d) != KDA_OK || Hq / Hkv > kMaxGroup || !page_ok(page) || N < 1 || n < 1 ||
      max_pages < 1)
    return 0;
  return size_t(cache_chunk_workspace_floats(cache_chunk_most_groups(n, N, Hq, Hkv, page, max_pages, in_dtype == KDA_BF16), d)) * 4;
}

kda_status kda_attn_chunk_fwd(const void* q, int64_t q_stride, kda_dtype in_dtype, const int* cu_seqlens,
                              const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                              const int* block_table, const int* context_len, void* o, kda_dtype o_dtype, float* lse, int n,
                              int N, int Hq, int Hkv, int d, int page, int n_pages, int max_pages, float scale, int zero_tail,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(o_dtype)) return KDA_ERR_DTYPE;
  const kda_status s = heads_ok(n, Hq, Hkv, d);
  if (s == KDA_ERR_SHAPE || N < 0 || n_pages < 0 || max_pages < 0 || page < 1) return KDA_ERR_SHAPE;
  if (s != KDA_OK || !page_ok(page) || Hq / Hkv > kMaxGroup || !isfinite(scale) || !flag_ok(zero_tail))
    return KDA_ERR_UNSUPPORTED;
  const kda_status st = stride_ok(q_stride, Hq, d, esize(in_dtype));
  if (st == KDA_ERR_SHAPE) return st;
  if (n == 0 || (N == 0 && !zero_tail)) return KDA_OK;
  if (cache_chunk_slots(n, N, Hq, Hkv) * Hkv > kMaxGrid) return KDA_ERR_SHAPE;
  const int used = n_pages > 0 ? max_pages : 0;  // a cache of no pages leaves every token out
  const int groups = N > 0 && used > 0 ? cache_chunk_groups(n, N, Hq, Hkv, page, used, in_dtype == KDA_BF16) : 0;
  const size_t need = size_t(cache_chunk_workspace_floats(groups, d)) * 4;
  if (!q || !o || (N > 0 && (!cu_seqlens || !context_len)) || (need > 0 && !workspace)) return KDA_ERR_NULL;
  if (N > 0 && used > 0 && (!k_cache || !v_cache || !k_scale || !v_scale || !block_table)) return KDA_ERR_NULL;
  if (st != KDA_OK || !all_aligned({q, o, k_cache, v_cache, need > 0 ? workspace : nullptr}, block_table, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(context_len, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lse, 4))
    return KDA_ERR_ALIGN;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  const int64_t ph = int64_t(n_pages) * Hkv, nq = int64_t(n) * Hq, e = int64_t(esize(in_dtype));
  const Rows rq{q, n, q_stride * e, int64_t(Hq) * d * e};
  const Range ins[] = {span(rq), {k_cache, ph * page * d}, {v_cache, ph * page * d}, {k_scale, ph * 4}, {v_scale, ph * 4},
                       {block_table, int64_t(N) * max_pages * 4}, {context_len, int64_t(N) * 4},
                       {cu_seqlens, (int64_t(N) + 1) * 4}};
  const Range outs[] = {{o, nq * d * int64_t(esize(o_dtype))}, {lse, nq * 4}, {need > 0 ? workspace : nullptr, int64_t(need)}};
  for (const Range& x : outs) {
    for (const Range& in : ins)
      if (kda::overlap(x, in)) return KDA_ERR_ALIAS;
    for (const Range& y : outs)
      if (&y != &x && kda::overlap(x, y)) return KDA_ERR_ALIAS;
  }
  return from_hip(launch_cache_chunk(
      CacheChunkArgs{q, q_stride, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), k_scale, v_scale,
                     cu_seqlens, block_table, context_len, o, lse, static_cast<float*>(workspace), n, N, Hq, Hkv, d, page,
                     n_pages, used, groups, scale, in_dtype == KDA_BF16, o_dtype == KDA_BF16, zero_tail != 0},
      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
