// Decode attention over 8-bit float caches (PKV_F8), and over chosen blocks
// of them: instantiations and launch.
#include "decode_blocks.cuh"

namespace pkv {

// What the dense and the block-list calls have in common.
blk::Params block_params(const pkv_pool *pool, const void *q, pkv_dtype q_dtype, int num_q_heads,
                         const void *k_cache, const void *v_cache, const void *k_scales,
                         const void *v_scales, const int32_t *seq_lens, int batch,
                         int64_t len_cap, float scale, float *out, void *workspace)
{
    blk::Params p{};
    p.q = q;
    p.k_cache = static_cast<const unsigned char *>(k_cache);
    p.v_cache = static_cast<const unsigned char *>(v_cache);
    p.k_scales = static_cast<const float *>(k_scales);
    p.v_scales = static_cast<const float *>(v_scales);
    p.seq_lens = seq_lens;
    p.out = out;
    p.counters = static_cast<int *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                           block_counter_bytes(pool));
    p.err = pool->d_err;
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = pool->num_kv_heads;
    p.block_size = pool->block_size;
    p.bs_log2 = log2_of(pool->block_size);
    p.num_blocks = pool->num_blocks;
    p.len_cap = (int)len_cap;
    p.q_dtype = q_dtype;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);  // log2(e)
    return p;
}

int launch_decode_f8(const pkv_pool *pool, const void *q, pkv_dtype q_dtype, int num_q_heads,
                     const void *k_cache, const void *v_cache, const void *k_scales,
                     const void *v_scales, const int32_t *tables, int max_blocks,
                     const int32_t *seq_lens, int batch, int max_seq_len, int window, float scale,
                     float *out, void *workspace, pkv_stream_t stream)
{
    const int64_t cap = (int64_t)max_blocks * pool->block_size;
    const int64_t len_cap = max_seq_len < cap ? max_seq_len : cap;
    const int64_t max_tiles =
        (int64_t)batch * pool->num_kv_heads * ((len_cap + blk::TILE - 1) / blk::TILE);
    if (max_tiles >= ((int64_t)1 << 31))
        return PKV_ERR_UNSUPPORTED;
    blk::Params p = block_params(pool, q, q_dtype, num_q_heads, k_cache, v_cache, k_scales,
                                 v_scales, seq_lens, batch, len_cap, scale, out, workspace);
    p.tables = tables;
    p.table_stride = max_blocks;
    p.window = window > 0 ? window : 0;
    return blk::launch_d<PKV_F8>(pool, p, reinterpret_cast<cudaStream_t>(stream), max_tiles);
}

int launch_blocks_f8(const pkv_pool *pool, const blk::Params &p, int64_t max_tiles,
                     cudaStream_t s)
{
    return blk::launch_d<PKV_F8>(pool, p, s, max_tiles);
}

}  // namespace pkv
