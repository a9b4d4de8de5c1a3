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
// Work.  Bounds are read once, 2 D + 4 bytes a (block, KV head), 16 bytes a
// lane, and multiplied with dp4a; every warp scores whole groups of 32 blocks
// with its own copy of the query values in registers, so scoring needs no
// barrier.  The last CTA of a (sequence, KV head) then finds the budget-th
// largest score key (an order-preserving map of the score) digit by digit: the
// keys, staged in shared memory, are counted by 8-bit digits of their
// distance to the smallest, counted from the top bit that any of them has, so
// that the first digit already spreads them; and it writes the chosen
// blocks in ascending order.
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

constexpr int NT = 256;              // threads of a CTA
constexpr int NW = NT / 32;
constexpr int SMEM_KEYS = 49152;     // score keys that are staged in shared memory

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
    int stage;                       // shared memory holds a (sequence, KV head)'s keys
    int budget, q_dtype;
};

// Order-preserving map of fp32 to unsigned; 0 is below every number's.
__device__ __forceinline__ uint32_t sort_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The `want` largest of n keys (ties: lowest index first), 0 < want < n: their
// indices, ascending, to sel / phys.  `keys` may be staged or in the workspace.
struct Pick {
    int hist[256];
    uint32_t lo[NW], hi[NW];
    int gt[NW], eq[NW];
    int bin, left;
};

__device__ __forceinline__ void pick(const volatile uint32_t *keys, int n, int want, int32_t *sel,
                                     int32_t *phys, const int32_t *row, Pick &s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the keys' range
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 4
    for (int i = tid; i < n; i += NT) {
        const uint32_t k = keys[i];
        lo = min(lo, k);
        hi = max(hi, k);
    }
    lo = __reduce_min_sync(FULL_MASK, lo);
    hi = __reduce_max_sync(FULL_MASK, hi);
    if (lane == 0) {
        s.lo[warp] = lo;
        s.hi[warp] = hi;
    }
    s.hist[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        lo = min(lo, s.lo[w]);
        hi = max(hi, s.hi[w]);
    }
    // t, relative to lo: the want-th largest key, a digit of up to 8 bits at a
    // time; `left` of the keys that share t's digits so far are still to take
    int top = hi > lo ? 32 - __clz(hi - lo) : 0;      // bits not decided yet
    uint32_t t = 0;
    int left = want;
    while (top > 0) {
        const int shift = max(top - 8, 0);
#pragma unroll 4
        for (int i = tid; i < n; i += NT) {
            const uint32_t k = keys[i] - lo;
            if (top >= 32 || (k >> top) == (t >> top))
                atomicAdd(&s.hist[(k >> shift) & ((1u << (top - shift)) - 1u)], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // bins from the top: lane l holds bins 255 - 8 l .. 248 - 8 l
            int c[8], sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                c[u] = s.hist[255 - 8 * lane - u];
                sum += c[u];
            }
            int inc = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(FULL_MASK, inc, off);
                if (lane >= off)
                    inc += x;
            }
            int above = inc - sum;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (above < left && above + c[u] >= left) {
                    s.bin = 255 - 8 * lane - u;
                    s.left = left - above;
                }
                above += c[u];
            }
        }
        __syncthreads();
        t |= (uint32_t)s.bin << shift;
        left = s.left;
        top = shift;
        s.hist[tid] = 0;
        __syncthreads();
    }
    t += lo;
    // keys above t, and the first `left` equal ones, in index order: each warp
    // ranks a contiguous run of indices, 32 at a time
    const int per = ((n + NW - 1) / NW + 31) & ~31;
    const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
    const unsigned below = (1u << lane) - 1u;
    int g = 0, e = 0;
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? keys[i + lane] : 0u;
        g += __popc(__ballot_sync(FULL_MASK, i + lane < i1 && k > t));
        e += __popc(__ballot_sync(FULL_MASK, i + lane < i1 && k == t));
    }
    if (lane == 0) {
        s.gt[warp] = g;
        s.eq[warp] = e;
    }
    __syncthreads();
    g = e = 0;
    for (int w = 0; w < warp; ++w) {
        g += s.gt[w];
        e += s.eq[w];
    }
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? keys[i + lane] : 0u;
        const bool gt = i + lane < i1 && k > t, eq = i + lane < i1 && k == t;
        const unsigned mg = __ballot_sync(FULL_MASK, gt), me = __ballot_sync(FULL_MASK, eq);
        const int rg = g + __popc(mg & below), re = e + __popc(me & below);
        if (gt || (eq && re < left)) {
            const int at = rg + min(re, left);
            sel[at] = i + lane;
            phys[at] = __ldg(row + i + lane);
        }
        g += __popc(mg);
        e += __popc(me);
    }
}

// The largest over the G heads of s[g] summed over the LPB lanes of a block.
// While a lane holds several heads, each level of the sum halves them (the
// lane whose mask bit is set keeps the upper half); the remaining levels add.
template <int G, int LPB>
__device__ __forceinline__ int sum_heads(int (&s)[G], int lane)
{
    int mask = LPB / 2;
#pragma unroll
    for (int h = G / 2; h >= 1; h >>= 1, mask >>= 1) {
        const bool up = (lane & mask) != 0;
#pragma unroll
        for (int g = 0; g < h; ++g) {
            const int send = up ? s[g] : s[g + h], keep = up ? s[g + h] : s[g];
            s[g] = keep + __shfl_xor_sync(FULL_MASK, send, mask);
        }
    }
    const int below = mask;
#pragma unroll
    for (; mask >= 1; mask >>= 1)
        s[0] += __shfl_xor_sync(FULL_MASK, s[0], mask);
    int best = s[0];
#pragma unroll
    for (int m = LPB / 2; m > below; m >>= 1)
        best = max(best, __shfl_xor_sync(FULL_MASK, best, m));
    return best;
}

template <int D, int G>
__global__ void __launch_bounds__(NT) select_kernel(const SelectArgs a)
{
    constexpr int LPB = 2 * D / 16;          // lanes that read one block's bounds
    constexpr int BPW = 32 / LPB;            // blocks a warp reads at once
    extern __shared__ uint32_t s_keys[];
    __shared__ int s_part[32 * NW];          // a warp's 32 block sums
    __shared__ Pick s_pick;
    __shared__ int s_last;
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

    // ---- the group's query values in whole steps of 2^eq: the lane's 16
    // channels, negative parts for the lanes of the lower bounds, positive for
    // the upper
    const int c = lane % LPB, sub = lane / LPB;
    const bool upper = c >= LPB / 2;
    int qr[G][4];
    {
        const uint4 *qsrc = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(a.q) + ((int64_t)b * H + kvh) * G * D +
            (c % (LPB / 2)) * 16);
        uint32_t raw[G][8];
        float amax = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 x = __ldg(qsrc + g * (D / 8) + h);
                raw[g][4 * h] = x.x; raw[g][4 * h + 1] = x.y;
                raw[g][4 * h + 2] = x.z; raw[g][4 * h + 3] = x.w;
            }
        auto pair = [&](uint32_t w) {
            return a.q_dtype == PKV_BF16 ? make_float2(bf16lo(w), bf16hi(w)) : half2_to_float2(w);
        };
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = pair(raw[g][i]);
                amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, m));
        const float f = pow2_f32(-int8_exponent(amax));
        auto step = [&](float x) {
            const int v = max(-127, min(127, __float2int_rn(x * f)));
            return (upper ? max(v, 0) : min(v, 0)) & 0xff;
        };
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = pair(raw[g][2 * i]), y = pair(raw[g][2 * i + 1]);
                qr[g][i] = step(x.x) | step(x.y) << 8 | step(y.x) << 16 | step(y.y) << 24;
            }
    }

    // ---- scores of this CTA's blocks (the newest one is not scored): 32
    // blocks a warp at a time
    uint32_t *keys = a.keys + (int64_t)seg * a.max_n;
    const int parts = (n + a.chunk - 1) / a.chunk;
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
        constexpr int STEP = 8;              // loads of a lane in flight
        static_assert(LPB % STEP == 0, "whole steps");
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
                int s[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    int v = __dp4a((int)x[u].x, qr[g][0], 0);
                    v = __dp4a((int)x[u].y, qr[g][1], v);
                    v = __dp4a((int)x[u].z, qr[g][2], v);
                    s[g] = __dp4a((int)x[u].w, qr[g][3], v);
                }
                // sums over the block's lanes: halving the heads a lane keeps
                // at each level until one is left, then its largest head
                int best = sum_heads<G, LPB>(s, lane);
                if (c == 0)
                    s_part[warp * 32 + (u0 + u) * BPW + sub] = best;
            }
        }
        __syncwarp();
        if (j < j_end) {
            const int ec = min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
            const uint32_t k = ok ? sort_key((float)s_part[warp * 32 + lane] * pow2_f32(ec)) : 0u;
            if (parts == 1 && a.stage)
                s_keys[j] = k;
            else
                keys[j] = k;
        }
        __syncwarp();
    }

    // ---- the last CTA of this (sequence, KV head) chooses
    __syncthreads();
    if (parts > 1) {
        if (tid == 0) {
            __threadfence();
            const int old = atomicAdd(a.counters + seg, 1);
            s_last = old == parts - 1;
            if (old == parts - 1) {
                a.counters[seg] = 0;
                __threadfence();
            }
        }
        __syncthreads();
        if (!s_last)
            return;
        if (a.stage) {
#pragma unroll 4
            for (int i = tid; i < n - 1; i += NT)
                s_keys[i] = __ldcg(keys + i);
            __syncthreads();
        }
    }
    pick(a.stage ? s_keys : keys, n - 1, a.budget - 1, sel, phys, row, s_pick);
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

template <int D, int G>
cudaError_t launch_select_t(const SelectArgs &a, unsigned grid, size_t smem, cudaStream_t s)
{
    if (smem > 40000) {
        const cudaError_t e = cudaFuncSetAttribute(
            select_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(select_kernel<D, G>, dim3(grid), dim3(NT), smem, s, a);
}

template <int D>
cudaError_t launch_select(const SelectArgs &a, int G, unsigned grid, size_t smem, cudaStream_t s)
{
    switch (G) {
    case 1: return launch_select_t<D, 1>(a, grid, smem, s);
    case 2: return launch_select_t<D, 2>(a, grid, smem, s);
    case 4: return launch_select_t<D, 4>(a, grid, smem, s);
    default: return launch_select_t<D, 8>(a, grid, smem, s);
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
    // a CTA's chunk: whole groups of 32 blocks for its warps, four CTAs a SM over the batch
    const int64_t segs = (int64_t)batch * H, n = (cap + bs - 1) / bs;
    const int64_t per = (segs * n + (int64_t)pool->num_sms * 4 - 1) / ((int64_t)pool->num_sms * 4);
    const int64_t span = 32 * NW;
    a.chunk = (int)std::max<int64_t>(span, (per + span - 1) / span * span);
    a.chunks = (int)std::max<int64_t>(1, (n + a.chunk - 1) / a.chunk);
    a.stage = n <= SMEM_KEYS;
    const size_t smem = a.stage ? (size_t)n * 4 : 0;
    const int64_t tiles_a_head =
        (std::min<int64_t>(cap, (int64_t)budget * bs) + blk::TILE - 1) / blk::TILE;
    const int64_t max_tiles = segs * tiles_a_head;
    if (segs * a.chunks > INT32_MAX || max_tiles > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(segs * a.chunks);
    const int G = num_q_heads / H;
    const cudaError_t e = pool->head_dim == 64 ? launch_select<64>(a, G, grid, smem, s)
                                               : launch_select<128>(a, G, grid, smem, s);
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
