// kv_device_reserve / kv_device_release: block tables, slot mapping and token
// offsets built on the device from request lengths, so that a decode step
// needs no host round trip and can be captured in a graph.
//
// With L_b rows cached and n_b new tokens, sequence b holds ceil(L_b / bs)
// blocks and needs ceil((L_b + n_b) / bs); the k-th new block of the call
// (sequences in order, each one's blocks in order) is the k-th from the top
// of the free list, and token j of sequence b gets slot
// table[b][(L_b + j) / bs] * bs + (L_b + j) % bs (KV cache visualization page,
// "PagedAttention: the cache in blocks": a sequence gains a block only when
// its tokens need one).
//
// Work: two exclusive prefix sums over the batch (tokens, new blocks), then one
// independent entry per token and per new block.  A decode step's call is
// bound by its launch and by the dependent chain lengths -> sums -> table entry
// -> slot, a prompt batch's by writing the slots.  Every CTA computes the sums
// for itself (at most 4096 lengths, read from L2) and takes a slice of the
// entries, which needs no second kernel and no grid barrier: what a CTA reads
// (lengths, free count, old table entries, ids below the count) no CTA
// writes.  Lengths and free count may be updated in place, so the last CTA to
// finish (a ticket) writes them.
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int NT = 512;            // threads of a CTA
constexpr int NW = NT / 32;
constexpr int MAX_SEQS = 4096;     // both prefix arrays fit static shared memory

// Exclusive prefix of (a, b) over the CTA's threads, and the totals.
struct Sums {
    long long a[NW], b[NW];
};

__device__ __forceinline__ void block_scan(long long &a, long long &b, long long &ta,
                                           long long &tb, Sums &s)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(FULL_MASK, ia, off);
        const long long y = __shfl_up_sync(FULL_MASK, ib, off);
        if (lane >= off) {
            ia += x;
            ib += y;
        }
    }
    if (lane == 31) {
        s.a[warp] = ia;
        s.b[warp] = ib;
    }
    __syncthreads();
    long long ba = 0, bb = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) {
            ba += s.a[w];
            bb += s.b[w];
        }
        ta += s.a[w];
        tb += s.b[w];
    }
    a = ba + ia - a;
    b = bb + ib - b;
}

// Largest b with start[b] <= x, given start[0] = 0 <= x < start[n].  Where
// several sequences start at x it is the last of them, the one that is not
// empty.
__device__ __forceinline__ int find(const int *start, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// True in every thread of the last CTA to get here (all of whose CTAs' reads
// and writes are then done); the ticket is left at zero.  bad: in the last CTA,
// whether any thread of any CTA came with it set (each CTA with one counts
// 2^16 on the ticket; there are at most 3 a SM).
__device__ __forceinline__ bool last_cta(int32_t *ticket, bool &bad)
{
    __shared__ int last, any;
    bad = __syncthreads_or(bad) != 0;
    if (gridDim.x == 1)
        return true;
    if (threadIdx.x == 0) {
        __threadfence();
        const int old = atomicAdd(ticket, 1 + (bad ? 1 << 16 : 0));
        last = (old & 0xffff) == (int)gridDim.x - 1;
        any = bad || (old >> 16) != 0;
        if (last) {
            __threadfence();
            *ticket = 0;
        }
    }
    __syncthreads();
    bad = any != 0;
    return last != 0;
}

struct TableArgs {
    const int32_t *free_in;
    int32_t *free_out;          // [0] count, [1] ticket
    int free_capacity;
    const int32_t *lens;
    int32_t *lens_out;
    int batch, max_blocks, block_size, bs_log2, num_blocks;
    unsigned int *err;
};

__global__ void __launch_bounds__(NT) reserve_kernel(TableArgs a, const int32_t *free_ids,
                                                     const int32_t *num_new, int32_t *tables,
                                                     int32_t *slots, int max_tokens,
                                                     int32_t *q_start)
{
    __shared__ int s_tok[MAX_SEQS + 1], s_blk[MAX_SEQS + 1];
    __shared__ Sums sums;
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, B = a.batch, bs = a.block_size, lg = a.bs_log2;
    const int count = a.free_in[0];
    const int per = (B + NT - 1) / NT;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const long long cap = (long long)a.max_blocks * bs;

    // tokens and new blocks of this thread's sequences; a length or a count
    // out of range refuses the whole call
    bool bad = false;
    long long nt = 0, nb = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = a.lens[b], n = num_new ? num_new[b] : 1;
        if (L < 0 || n < 0 || (long long)L + n > cap || (long long)L + n > INT32_MAX) {
            bad = true;
            continue;
        }
        nt += n;
        nb += (((long long)L + n + bs - 1) >> lg) - (((long long)L + bs - 1) >> lg);
    }
    long long at = nt, ab = nb, total_t, total_b;
    block_scan(at, ab, total_t, total_b, sums);
    bad |= total_t > max_tokens || count < 0 || count > a.free_capacity;
    const bool any_bad = __syncthreads_or(bad) != 0;
    const bool full = !any_bad && total_b > count;
    const bool ok = !any_bad && !full;
    if (!ok && blockIdx.x == 0 && tid == 0)
        atomicOr(a.err, any_bad ? PKV_EBIT_SEQLEN : PKV_EBIT_NO_BLOCKS);
    if (ok) {
        for (int b = b0; b < b1; ++b) {
            const int L = a.lens[b], n = num_new ? num_new[b] : 1;
            s_tok[b] = (int)at;
            s_blk[b] = (int)ab;
            at += n;
            ab += (((long long)L + n + bs - 1) >> lg) - (((long long)L + bs - 1) >> lg);
        }
        if (tid == 0) {
            s_tok[B] = (int)total_t;
            s_blk[B] = (int)total_b;
        }
    }
    __syncthreads();
    const int T = ok ? (int)total_t : 0, NB = ok ? (int)total_b : 0;
    const int stride = gridDim.x * NT, first = blockIdx.x * NT + tid;

    // a new block's id, or -1 (recorded) for one outside the pool
    auto fresh = [&](int k) {
        const int id = free_ids[count - 1 - k];
        if (id < 0 || id >= a.num_blocks) {
            atomicOr(a.err, PKV_EBIT_BLOCK);
            return -1;
        }
        return id;
    };
    // (the first new block's id is on its way while the slots are worked out)
    int id = first < NB ? fresh(first) : 0;
    // four consecutive tokens a thread: one search, then along the batch
    for (int64_t i4 = (int64_t)first * 4; i4 < max_tokens; i4 += (int64_t)stride * 4) {
        int b = i4 < T ? find(s_tok, B, (int)i4) : B;
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i4 + u;
            v[u] = -1;
            if (i < T) {
                while (i >= s_tok[b + 1])
                    ++b;
                const int L = a.lens[b];
                const int pos = L + (int)(i - s_tok[b]);
                const int old = (int)(((long long)L + bs - 1) >> lg);
                const int j = pos >> lg;
                int blk;
                if (j >= old) {
                    blk = fresh(s_blk[b] + j - old);
                } else {
                    blk = tables[(int64_t)b * a.max_blocks + j];
                    if (blk < 0 || blk >= a.num_blocks) {
                        atomicOr(a.err, PKV_EBIT_BLOCK);
                        blk = -1;
                    }
                }
                if (blk >= 0)
                    v[u] = blk * bs + (pos & (bs - 1));
            }
        }
        if (i4 + 4 <= max_tokens && (reinterpret_cast<uintptr_t>(slots) & 15u) == 0) {
            *reinterpret_cast<int4 *>(slots + i4) = make_int4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i4 + u < max_tokens)
                    slots[i4 + u] = v[u];
        }
    }
    for (int k = first; k < NB; k += stride) {
        const int b = find(s_blk, B, k);
        const int old = (int)(((long long)a.lens[b] + bs - 1) >> lg);
        if (k != first)
            id = fresh(k);
        tables[(int64_t)b * a.max_blocks + old + (k - s_blk[b])] = id;
    }
    if (q_start)
        for (int b = first; b <= B; b += stride)
            q_start[b] = ok ? s_tok[b] : 0;

    bool none = false;
    if (last_cta(a.free_out + 1, none)) {
        for (int b = tid; b < B; b += NT)
            a.lens_out[b] = a.lens[b] + (ok ? s_tok[b + 1] - s_tok[b] : 0);
        if (tid == 0)
            a.free_out[0] = count - NB;
    }
}

__global__ void __launch_bounds__(NT) release_kernel(TableArgs a, int32_t *free_ids,
                                                     const int32_t *done, const int32_t *tables)
{
    __shared__ int s_blk[MAX_SEQS + 1];
    __shared__ Sums sums;
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, B = a.batch, bs = a.block_size, lg = a.bs_log2;
    const int count = a.free_in[0];
    const int per = (B + NT - 1) / NT;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const long long cap = (long long)a.max_blocks * bs;

    bool bad = false;
    long long nb = 0, unused = 0, tu;
    for (int b = b0; b < b1; ++b) {
        const int L = a.lens[b];
        if (done[b] == 0)
            continue;
        if (L < 0 || L > cap)
            bad = true;
        else
            nb += ((long long)L + bs - 1) >> lg;
    }
    long long ab = nb, total;
    block_scan(ab, unused, total, tu, sums);
    bad |= count < 0 || count + total > a.free_capacity;
    const bool ok = __syncthreads_or(bad) == 0;
    if (!ok && blockIdx.x == 0 && tid == 0)
        atomicOr(a.err, PKV_EBIT_SEQLEN);
    if (ok) {
        for (int b = b0; b < b1; ++b) {
            s_blk[b] = (int)ab;
            ab += done[b] != 0 ? ((long long)a.lens[b] + bs - 1) >> lg : 0;
        }
        if (tid == 0)
            s_blk[B] = (int)total;
    }
    __syncthreads();
    const int R = ok ? (int)total : 0;
    bool bad_id = false;
    for (int k = blockIdx.x * NT + tid; k < R; k += gridDim.x * NT) {
        const int b = find(s_blk, B, k);
        const int id = tables[(int64_t)b * a.max_blocks + (k - s_blk[b])];
        if (id < 0 || id >= a.num_blocks) {
            atomicOr(a.err, PKV_EBIT_BLOCK);
            bad_id = true;
        }
        free_ids[count + k] = id;          // (counted only below, if all are good)
    }
    if (last_cta(a.free_out + 1, bad_id)) {
        for (int b = tid; b < B; b += NT)
            a.lens_out[b] = ok && !bad_id && done[b] != 0 ? 0 : a.lens[b];
        if (tid == 0)
            a.free_out[0] = count + (bad_id ? 0 : R);
    }
}

TableArgs table_args(const pkv_pool *pool, const int32_t *free_in, int32_t *free_out,
                     int free_capacity, const int32_t *lens, int32_t *lens_out, int batch,
                     int max_blocks)
{
    TableArgs a;
    a.free_in = free_in;
    a.free_out = free_out;
    a.free_capacity = free_capacity;
    a.lens = lens;
    a.lens_out = lens_out;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.block_size = pool->block_size;
    a.bs_log2 = log2_of(pool->block_size);
    a.num_blocks = pool->num_blocks;
    a.err = pool->d_err;
    return a;
}

// CTAs for this many threads' work, at most three a SM (what their shared
// memory and threads let be resident): a thread then has one or two rounds of
// dependent loads.
int grid_for(int64_t items, int num_sms)
{
    const int64_t g = (items + NT - 1) / NT, cap = (int64_t)num_sms * 3;
    return (int)(g < 1 ? 1 : g > cap ? cap : g);
}

}  // namespace

int launch_device_reserve(const pkv_pool *pool, const int32_t *free_ids, int free_capacity,
                          const int32_t *free_in, int32_t *free_out, const int32_t *lens,
                          const int32_t *num_new, int batch, int32_t *tables, int max_blocks,
                          int32_t *slots, int max_tokens, int32_t *q_start, int32_t *lens_out,
                          pkv_stream_t stream)
{
    const TableArgs a = table_args(pool, free_in, free_out, free_capacity, lens, lens_out, batch,
                                   max_blocks);
    if (launch_pdl(reserve_kernel, dim3(grid_for(max_tokens / 4, pool->num_sms)), dim3(NT), 0,
                   reinterpret_cast<cudaStream_t>(stream), a, free_ids, num_new, tables, slots,
                   max_tokens, q_start) != cudaSuccess)
        return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int launch_device_release(const pkv_pool *pool, int32_t *free_ids, int free_capacity,
                          const int32_t *free_in, int32_t *free_out, const int32_t *lens,
                          const int32_t *done, int batch, const int32_t *tables, int max_blocks,
                          int32_t *lens_out, pkv_stream_t stream)
{
    const TableArgs a = table_args(pool, free_in, free_out, free_capacity, lens, lens_out, batch,
                                   max_blocks);
    // a quarter of the tables' entries at once: few sequences finish together
    if (launch_pdl(release_kernel,
                   dim3(grid_for((int64_t)batch * max_blocks / 4, pool->num_sms)), dim3(NT), 0,
                   reinterpret_cast<cudaStream_t>(stream), a, free_ids, done,
                   tables) != cudaSuccess)
        return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
