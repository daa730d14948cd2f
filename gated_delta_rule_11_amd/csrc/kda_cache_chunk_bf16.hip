// kda_cache_chunk_bf16.hip -- attention of a chunk over the cache, bf16 queries; the division of the work.
#include "kda_cache_chunk.hpp"

namespace kda {

hipError_t launch_cache_chunk_bf16(const CacheChunkArgs& a, hipStream_t st) { return launch_chunk_any<bf16_t>(a, st); }

hipError_t launch_cache_chunk(const CacheChunkArgs& a, hipStream_t st) {
  return a.in_bf16 ? launch_cache_chunk_bf16(a, st) : launch_cache_chunk_f32(a, st);
}

int64_t cache_chunk_slots(int n, int N, int Hq, int Hkv) { return int64_t(n) * (Hq / Hkv) / kChunkRows + N; }

// Workgroups that share the work, 0 for one to a tile.
int cache_chunk_groups(int n, int N, int Hq, int Hkv, int page, int max_pages, bool bf16) {
  const int64_t tiles = cache_chunk_slots(n, N, Hq, Hkv) * Hkv;
  const int64_t steps = (int64_t(max_pages) * page + 63) / 64;
  if (steps <= 8) return 0;
  const int64_t most = bf16 ? 512 : 256;
  const int64_t want = tiles > most || steps > most ? most : tiles * steps / 4;
  return int(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace kda
