// Decode attention over chosen blocks of 16-bit caches: instantiations.
#include "decode_blocks.cuh"

namespace pkv {

int launch_blocks_16(const pkv_pool *pool, const blk::Params &p, int64_t max_tiles,
                     cudaStream_t s)
{
    return pool->kv_dtype == PKV_F16 ? blk::launch_d<PKV_F16>(pool, p, s, max_tiles)
                                     : blk::launch_d<PKV_BF16>(pool, p, s, max_tiles);
}

}  // namespace pkv
