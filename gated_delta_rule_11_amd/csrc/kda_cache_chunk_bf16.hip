// kda_cache_chunk_bf16.hip -- attention of a chunk over the cache, bf16 queries; the division of the work.
#include "kda_cache_chunk.hpp"

namespace kda {

hipError_t launch_cache_chunk_bf16(const CacheChunkArgs& a, hipStream_t st) { return launch_chunk_any<bf16_t>(a, st); }

hipError_t launch_cache_chunk(const CacheChunkArgs& a, hipStream_t st) {
  return a.in_bf16 ? launch_cache_chunk_bf16(a, st) : launch_cache_chunk_f32(a, st);
}

int64_t cache_chunk_slots(int n, int N, int Hq, int Hkv) { return int64_t(n) * (Hq / Hkv) / kChunkRows + N; }

// Workgroups that share the work, 0 for one to a tile.  Dividing tiles costs parts, a second launch and a start for each
// cut; not dividing costs where one long tile ends late, and how long one may be is known by the table's room, how much
// else there is by the number of tiles.  One to a tile against the division, us, 32 heads on 8 of 128, bf16:
//   room 1000:  4 single tokens 12.5, 20.3;  256 of them 71, 78;  one prompt 33, 49
//   room 2000:  one prompt 63, 74;  16 prompts 306, 330;  two chunks of 40 tokens 55, 42
//   room 4000:  one prompt 150, 176;  26 single tokens among 6 chunks 110, 84
// fp32, a third of the steps' rate and half the workgroups at once, 24 heads on 4 of 64 in a room of 2048, at about 64, 236,
// 404 and 804 tiles:
//   whole prompts 19, 25;  48, 47;  65, 72;  96, 102;  single tokens 17, 24;  21, 26;  35, 34;  56, 51
//   pieces of 64 to 512 tokens behind up to 2000: 26, 31;  69, 64;  103, 90;  159, 131
// Neither is the faster at all lengths, which the host does not know; from 100 to 800 tiles the three together differ by a
// tenth at most (with d = 128, 32 heads on 8 or a room of 1500 by less than a fifth, to either side).  The border, 12 tiles
// to a step, is 384 here.
int cache_chunk_groups(int n, int N, int Hq, int Hkv, int page, int max_pages, bool bf16) {
  const int64_t tiles = cache_chunk_slots(n, N, Hq, Hkv) * Hkv;
  const int64_t steps = (int64_t(max_pages) * page + 63) / 64;
  const int64_t few = (bf16 ? 4 : 12) * steps;
  if ((steps <= 32 && tiles >= few) || (steps <= 64 && tiles >= 4 * few)) return 0;
  return cache_chunk_most_groups(n, N, Hq, Hkv, page, max_pages, bf16);
}

// The same for as many tokens or fewer in the same table's room, where the division needs a workspace.
int cache_chunk_most_groups(int n, int N, int Hq, int Hkv, int page, int max_pages, bool bf16) {
  const int64_t tiles = cache_chunk_slots(n, N, Hq, Hkv) * Hkv;
  const int64_t steps = (int64_t(max_pages) * page + 63) / 64;
  if (steps <= 16) return 0;
  const int64_t most = bf16 ? 512 : 256;
  const int64_t want = tiles > most || steps > most ? most : tiles * steps / 4;
  return int(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace kda
