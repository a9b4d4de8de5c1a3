// paged_decode_attention_sparse: which blocks of each (sequence, KV head) a
// query attends to, by a score from the blocks' key bounds, and the launch of
// the attention over them.
//
// Score.  Channel d of every key of block j lies in [lo, hi] = [l, h] 2^e with
// the stored int8 l, h, so q . k <= sum_d max(q_d lo_d, q_d hi_d).  With the
// group's query values in steps of one power of two, qi = rint(q 2^-eq) in
// [-127, 127], the sum is of whole numbers, qi+ . h + qi- . l with the
// positive and the negative parts of qi (sum_d max(qi l, qi h), as l <= h), below 2^22,
// and the block's score, its largest over the group's heads times 2^e, is
// exact in fp32: which blocks are chosen does not depend on the order of any
// sum.  2^eq is common to the blocks and left out.
//
// Work.  Bounds are read once, 2 D + 4 bytes a (block, KV head): a CTA scores
// a chunk of one (sequence, KV head)'s blocks, 16 bytes a lane, with dp4a;
// the last CTA of that (sequence, KV head) finds the budget-th largest score
// by a search over the bits of the (order-preserving) score keys, held in
// registers, and writes the chosen blocks in ascending order.
#include <algorithm>

#include "decode_blocks.cuh"

namespace pkv {

int launch_blocks_f8(const pkv_pool *pool, const blk::Params &p, int64_t max_tiles,
                     cudaStream_t s);
int launch_blocks_16(const pkv_pool *pool, const blk::Params &p, int64_t max_tiles,
                     cudaStream_t s);
blk::Params block_params(const pkv_pool *pool, const void *q, pkv_dtype q_dtype, int num_q_heads,
                         const void *k_cache, const void *v_cache, const void *k_scales,
                         const void *v_scales, const int32_t *seq_lens, int batch,
                         int64_t len_cap, float scale, float *out, void *workspace);

namespace {

using namespace dev;

constexpr int NT = 512;              // threads of a CTA
constexpr int NW = NT / 32;
constexpr int MAX_KEYS = 32;         // keys a thread holds in registers (16384 blocks in all)

struct SelectArgs {
    const void *q;
    const int8_t *bounds;            // [NB][Hkv][2][D]
    const int32_t *exps;             // [NB][Hkv]
    const int32_t *tables;
    const int32_t *seq_lens;
    int32_t *selected;               // [B][Hkv][budget] logical blocks, -1 past the last
    int32_t *phys;                   // the same as physical blocks
    uint32_t *keys;                  // [B][Hkv][max_n]
    int *counters;                   // [B][Hkv]
    unsigned int *err;
    int batch, num_kv_heads, num_blocks, block_size, bs_log2, max_blocks, len_cap;
    int max_n;                       // blocks of the longest sequence allowed
    int chunk, chunks;               // blocks a CTA scores; CTAs a (sequence, KV head)
    int budget, q_dtype;
};

// Order-preserving map of fp32 to unsigned; 0 is below every number's.
__device__ __forceinline__ uint32_t sort_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int x, int *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = __reduce_add_sync(FULL_MASK, x);
    __syncthreads();
    if (lane == 0)
        scratch[warp] = x;
    __syncthreads();
    return __reduce_add_sync(FULL_MASK, lane < NW ? scratch[lane] : 0);
}

// The `want` largest of n keys (ties: lowest index first), 0 < want < n: their
// indices, ascending, to sel / phys.  Key i is held by thread i % NT.
template <int K>
__device__ __forceinline__ void pick(const SelectArgs &a, const volatile uint32_t *keys, int n,
                                     int want, int32_t *sel, int32_t *phys, const int32_t *row,
                                     int *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t key[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
        key[j] = tid + j * NT < n ? keys[tid + j * NT] : 0u;
    // t = the want-th largest key: the largest t that at least `want` reach
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = t | (1u << bit);
        int c = 0;
#pragma unroll
        for (int j = 0; j < K; ++j)
            c += key[j] >= cand;
        if (block_sum(c, scratch) >= want)
            t = cand;
    }
    int above = 0;
#pragma unroll
    for (int j = 0; j < K; ++j)
        above += key[j] > t;
    const int ties = want - block_sum(above, scratch);     // equal keys to take, lowest index first
    // ranks in index order (index i = j * NT + tid)
    int base_gt = 0, base_eq = 0;
#pragma unroll 1
    for (int j = 0; j < K; ++j) {
        if (j * NT >= n)
            break;
        const int i = j * NT + tid;
        uint32_t kj = 0;
#pragma unroll
        for (int u = 0; u < K; ++u)
            if (u == j)
                kj = key[u];
        const bool gt = i < n && kj > t, eq = i < n && kj == t;
        const unsigned mg = __ballot_sync(FULL_MASK, gt), me = __ballot_sync(FULL_MASK, eq);
        __syncthreads();
        if (lane == 0)
            scratch[warp] = __popc(mg) | (__popc(me) << 16);
        __syncthreads();
        int bg = 0, be = 0, tg = 0, te = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int v = scratch[w];
            if (w < warp) {
                bg += v & 0xffff;
                be += v >> 16;
            }
            tg += v & 0xffff;
            te += v >> 16;
        }
        const unsigned below = (1u << lane) - 1u;
        const int rg = base_gt + bg + __popc(mg & below), re = base_eq + be + __popc(me & below);
        if (gt || (eq && re < ties)) {
            const int at = rg + min(re, ties);
            sel[at] = i;
            phys[at] = __ldg(row + i);
        }
        base_gt += tg;
        base_eq += te;
    }
}

// The same for more keys than registers hold: the keys are read again for
// every bit.
__device__ __forceinline__ void pick_many(const SelectArgs &a, const volatile uint32_t *keys,
                                          int n, int want, int32_t *sel, int32_t *phys,
                                          const int32_t *row, int *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = t | (1u << bit);
        int c = 0;
#pragma unroll 4
        for (int i = tid; i < n; i += NT)
            c += keys[i] >= cand;
        if (block_sum(c, scratch) >= want)
            t = cand;
    }
    int above = 0;
#pragma unroll 4
    for (int i = tid; i < n; i += NT)
        above += keys[i] > t;
    const int ties = want - block_sum(above, scratch);
    int base_gt = 0, base_eq = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const uint32_t kj = i < n ? keys[i] : 0u;
        const bool gt = i < n && kj > t, eq = i < n && kj == t;
        const unsigned mg = __ballot_sync(FULL_MASK, gt), me = __ballot_sync(FULL_MASK, eq);
        __syncthreads();
        if (lane == 0)
            scratch[warp] = __popc(mg) | (__popc(me) << 16);
        __syncthreads();
        int bg = 0, be = 0;
        for (int w = 0; w < NW; ++w) {
            const int v = scratch[w];
            if (w < warp) {
                bg += v & 0xffff;
                be += v >> 16;
            }
        }
        const unsigned below = (1u << lane) - 1u;
        const int rg = base_gt + bg + __popc(mg & below), re = base_eq + be + __popc(me & below);
        if (gt || (eq && re < ties)) {
            const int at = rg + min(re, ties);
            sel[at] = i;
            phys[at] = __ldg(row + i);
        }
        for (int w = 0; w < NW; ++w) {
            base_gt += scratch[w] & 0xffff;
            base_eq += scratch[w] >> 16;
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(NT) select_kernel(const SelectArgs a)
{
    constexpr int LPB = 2 * D / 16;          // lanes that read one block's bounds
    constexpr int BPW = 32 / LPB;            // blocks a warp reads at once
    __shared__ __align__(16) int8_t s_q[2][G][D];   // negative parts, positive parts
    __shared__ int s_part[32 * NW];          // a warp's 32 block sums
    __shared__ int scratch[NW + 1];
    __shared__ float s_max[NW];
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x / a.chunks, part = blockIdx.x - seg * a.chunks;
    const int H = a.num_kv_heads, b = seg / H, kvh = seg - b * H;
    int L = __ldg(a.seq_lens + b);
    if (L < 0 || L > a.len_cap)
        L = 0;                               // (the attention records it)
    const int n = (L + a.block_size - 1) >> a.bs_log2;
    const int nsel = min(n, a.budget);
    const int32_t *row = a.tables + (int64_t)b * a.max_blocks;
    int32_t *sel = a.selected + (int64_t)seg * a.budget;
    int32_t *phys = a.phys + (int64_t)seg * a.budget;
    const int j_begin = part * a.chunk;
    if (part > 0 && (j_begin >= n || n <= a.budget))
        return;
    if (part == 0)
        for (int i = nsel + tid; i < a.budget; i += NT)
            sel[i] = -1;
    if (n <= a.budget) {
        for (int i = tid; i < n; i += NT) {
            sel[i] = i;
            phys[i] = __ldg(row + i);
        }
        return;
    }
    if (part == 0 && tid == 0) {             // the newest block, always
        sel[nsel - 1] = n - 1;
        phys[nsel - 1] = __ldg(row + n - 1);
    }
    if (a.budget == 1)
        return;

    // ---- the group's query values in whole steps of 2^eq
    const uint16_t *qsrc =
        static_cast<const uint16_t *>(a.q) + ((int64_t)b * H + kvh) * G * D;
    auto q_at = [&](int i) {
        const uint16_t w = __ldg(qsrc + i);
        return a.q_dtype == PKV_BF16 ? bf16lo(w) : __half2float(__ushort_as_half(w));
    };
    float amax = 0.0f;
    for (int i = tid; i < G * D; i += NT)
        amax = fmaxf(amax, fabsf(q_at(i)));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, m));
    if (lane == 0)
        s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w)
        amax = fmaxf(amax, s_max[w]);
    const float f = pow2_f32(-int8_exponent(amax));
    for (int i = tid; i < G * D; i += NT) {
        const int v = max(-127, min(127, __float2int_rn(q_at(i) * f)));
        s_q[0][i / D][i % D] = (int8_t)min(v, 0);
        s_q[1][i / D][i % D] = (int8_t)max(v, 0);
    }
    __syncthreads();
    // the lane's 16 channels of the lower (first half of the lanes) or upper bounds
    const int c = lane % LPB, sub = lane / LPB;
    int qr[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int4 w = *reinterpret_cast<const int4 *>(
            &s_q[c / (LPB / 2)][g][(c % (LPB / 2)) * 16]);
        qr[g][0] = w.x; qr[g][1] = w.y; qr[g][2] = w.z; qr[g][3] = w.w;
    }

    // ---- scores of this CTA's blocks (the newest one is not scored): 32
    // blocks a warp at a time
    uint32_t *keys = a.keys + (int64_t)seg * a.max_n;
    const int j_end = min(n - 1, j_begin + a.chunk);
    for (int j0 = j_begin + warp * 32; j0 < j_end; j0 += NW * 32) {
        const int j = j0 + lane;
        int id = j < j_end ? __ldg(row + j) : 0;
        const bool ok = id >= 0 && id < a.num_blocks;
        if (!ok) {
            atomicOr(a.err, PKV_EBIT_BLOCK);
            id = 0;
        }
        const int e = __ldg(a.exps + (int64_t)id * H + kvh);
        constexpr int STEP = 4;              // blocks' loads in flight: STEP * BPW
#pragma unroll 1
        for (int u0 = 0; u0 < LPB; u0 += STEP) {
            uint4 x[STEP];
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int id_u = __shfl_sync(FULL_MASK, id, (u0 + u) * BPW + sub);
                x[u] = __ldg(reinterpret_cast<const uint4 *>(
                                 a.bounds + ((int64_t)id_u * H + kvh) * 2 * D) + c);
            }
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                int best = INT_MIN;
                int s[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    int v = __dp4a((int)x[u].x, qr[g][0], 0);
                    v = __dp4a((int)x[u].y, qr[g][1], v);
                    v = __dp4a((int)x[u].z, qr[g][2], v);
                    s[g] = __dp4a((int)x[u].w, qr[g][3], v);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
#pragma unroll
                    for (int m = LPB / 2; m >= 1; m >>= 1)
                        s[g] += __shfl_xor_sync(FULL_MASK, s[g], m);
                    best = max(best, s[g]);
                }
                if (c == 0)
                    s_part[warp * 32 + (u0 + u) * BPW + sub] = best;
            }
        }
        __syncwarp();
        if (j < j_end) {
            const int ec = min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
            keys[j] = ok ? sort_key((float)s_part[warp * 32 + lane] * pow2_f32(ec)) : 0u;
        }
        __syncwarp();
    }

    // ---- the last CTA of this (sequence, KV head) chooses
    const int parts = (n + a.chunk - 1) / a.chunk;
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        const int old = parts > 1 ? atomicAdd(a.counters + seg, 1) : 0;
        scratch[NW] = old == parts - 1;
        if (old == parts - 1 && parts > 1)
            a.counters[seg] = 0;
        __threadfence();
    }
    __syncthreads();
    if (!scratch[NW])
        return;
    const int m = n - 1, want = a.budget - 1;
    if (m <= 4 * NT)
        pick<4>(a, keys, m, want, sel, phys, row, scratch);
    else if (m <= 8 * NT)
        pick<8>(a, keys, m, want, sel, phys, row, scratch);
    else if (m <= MAX_KEYS * NT)
        pick<MAX_KEYS>(a, keys, m, want, sel, phys, row, scratch);
    else
        pick_many(a, keys, m, want, sel, phys, row, scratch);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The regions of the workspace behind the attention's own.
struct Regions {
    size_t counters, phys, keys, total;
};

Regions regions(const pkv_pool *pool, int batch, int num_q_heads, int max_seq_len, int budget)
{
    const size_t segs = (size_t)batch * pool->num_kv_heads;
    const size_t n = ((size_t)max_seq_len + pool->block_size - 1) / pool->block_size;
    Regions r;
    r.counters = up256(decode_workspace_bytes(pool, batch, num_q_heads));
    r.phys = r.counters + up256(segs * sizeof(int));
    r.keys = r.phys + up256(segs * budget * sizeof(int32_t));
    r.total = r.keys + up256(segs * n * sizeof(uint32_t));
    return r;
}

template <int D>
cudaError_t launch_select(const SelectArgs &a, int G, unsigned grid, cudaStream_t s)
{
    switch (G) {
    case 1: return launch_pdl(select_kernel<D, 1>, dim3(grid), dim3(NT), 0, s, a);
    case 2: return launch_pdl(select_kernel<D, 2>, dim3(grid), dim3(NT), 0, s, a);
    case 4: return launch_pdl(select_kernel<D, 4>, dim3(grid), dim3(NT), 0, s, a);
    default: return launch_pdl(select_kernel<D, 8>, dim3(grid), dim3(NT), 0, s, a);
    }
}

}  // namespace

size_t sparse_workspace_bytes(const pkv_pool *pool, int batch, int num_q_heads, int max_seq_len,
                              int budget)
{
    return regions(pool, batch, num_q_heads, max_seq_len, budget).total;
}

int launch_sparse(const pkv_pool *pool, const void *q, pkv_dtype q_dtype, int num_q_heads,
                  const void *k_cache, const void *v_cache, const void *k_scales,
                  const void *v_scales, const int8_t *bounds, const int32_t *exps,
                  const int32_t *tables, int max_blocks, const int32_t *seq_lens, int batch,
                  int max_seq_len, int budget, float scale, float *out, int32_t *selected,
                  void *workspace, pkv_stream_t stream)
{
    const Regions r = regions(pool, batch, num_q_heads, max_seq_len, budget);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const int H = pool->num_kv_heads, bs = pool->block_size;
    const int64_t cap = std::min<int64_t>((int64_t)max_blocks * bs, max_seq_len);
    SelectArgs a{};
    a.q = q;
    a.bounds = bounds;
    a.exps = exps;
    a.tables = tables;
    a.seq_lens = seq_lens;
    a.selected = selected;
    a.phys = reinterpret_cast<int32_t *>(ws + r.phys);
    a.keys = reinterpret_cast<uint32_t *>(ws + r.keys);
    a.counters = reinterpret_cast<int *>(ws + r.counters);
    a.err = pool->d_err;
    a.batch = batch;
    a.num_kv_heads = H;
    a.num_blocks = pool->num_blocks;
    a.block_size = bs;
    a.bs_log2 = log2_of(bs);
    a.max_blocks = max_blocks;
    a.len_cap = (int)cap;
    a.max_n = (int)((max_seq_len + (int64_t)bs - 1) / bs);
    a.budget = budget;
    a.q_dtype = q_dtype;
    // a CTA's chunk: whole warps' groups of 32 blocks, a few CTAs a SM over the batch
    const int64_t segs = (int64_t)batch * H, n = (cap + bs - 1) / bs;
    const int64_t per = (segs * n + (int64_t)pool->num_sms * 4 - 1) / ((int64_t)pool->num_sms * 4);
    const int64_t span = 32 * NW;
    a.chunk = (int)std::max<int64_t>(span, (per + span - 1) / span * span);
    a.chunks = (int)std::max<int64_t>(1, (n + a.chunk - 1) / a.chunk);
    const int64_t tiles_a_head =
        (std::min<int64_t>(cap, (int64_t)budget * bs) + blk::TILE - 1) / blk::TILE;
    const int64_t max_tiles = segs * tiles_a_head;
    if (segs * a.chunks > INT32_MAX || max_tiles > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(segs * a.chunks);
    const int G = num_q_heads / H;
    const cudaError_t e = pool->head_dim == 64 ? launch_select<64>(a, G, grid, s)
                                               : launch_select<128>(a, G, grid, s);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess)
        return PKV_ERR_CUDA;
    blk::Params p = block_params(pool, q, q_dtype, num_q_heads, k_cache, v_cache, k_scales,
                                 v_scales, seq_lens, batch, cap, scale, out, workspace);
    p.tables = a.phys;
    p.table_stride = budget;
    p.per_head = 1;
    p.budget = budget;
    return pool->kv_dtype == PKV_F8 ? launch_blocks_f8(pool, p, max_tiles, s)
                                    : launch_blocks_16(pool, p, max_tiles, s);
}

}  // namespace pkv
