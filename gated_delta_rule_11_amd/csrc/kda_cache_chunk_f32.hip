// kda_cache_chunk_f32.hip -- attention of a chunk over the cache, fp32 queries.
#include "kda_cache_chunk.hpp"

namespace kda {

hipError_t launch_cache_chunk_f32(const CacheChunkArgs& a, hipStream_t st) { return launch_chunk_any<float>(a, st); }

}  // namespace kda
