// The tiled cached attention with keys in two parts (a shared prefix, then each sequence's own): a
// translation unit of its own, so that both compile at the same time.
#define CACHE_TILE_SIDE true
#include "fwd_cache_tile.cu"
