// paged_decode_attention_sparse: which blocks of each (sequence, KV head) a
// query attends to, by a score from the blocks' key bounds, and the launch of
// the attention over them.
//
// Score.  Channel d of every key of block j lies in [lo, hi] = [l, h] 2^e with
// the stored int8 l, h, so q . k <= sum_d max(q_d lo_d, q_d hi_d).  With the
// group's query values in steps of one power of two, qi = rint(q 2^-eq) in
// [-127, 127], the sum is of whole numbers, qi+ . h + qi- . l with the
// positive and the negative parts of qi (sum_d max(qi l, qi h), as l <= h), below 2^22,
// and the block's score, its largest over the group's heads times 2^(e - 22),
// is exact in fp32 for every e of a block (-96 to 120): which blocks are chosen
// does not depend on the order of any sum.  2^(eq + 22) is common to the blocks
// and left out.
//
// Work.  Bounds are read once, 2 D + 4 bytes a (block, KV head).  The scores
// of 16 blocks and all heads of the group are warp-level MMAs on fp16 (int8
// values and their sums below 2^24 are exact there; an int8 MMA of this GPU
// takes 65 clocks to the fp16 one's 8, and dp4a with its sums over lanes made
// the kernel issue-bound: 18 us of scoring on 16 x 2048 blocks x 8 heads
// where the bytes take 10).  Every warp scores whole groups of 32 blocks with
// its own copy of the query values in registers, so scoring needs no barrier.
// The last CTA of a (sequence, KV head) then finds the budget-th
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

constexpr int RANKED = 256;          // keys left open that are ranked among one another
constexpr int SMEM_KEYS = 24576;     // score keys that are staged in shared memory, with their ids

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
    int stage;                       // keys (and as many ids) staged in shared memory, or 0
    int budget, q_dtype;
};

// Order-preserving map of fp32 to unsigned; 0 is below every number's.
__device__ __forceinline__ uint32_t sort_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The `want` largest of n keys (ties: lowest index first), 0 < want < n: their
// indices, ascending, to sel, their ids to phys.  Keys and ids may be staged, or in
// the workspace and the block table.
template <int NT>
struct Pick {
    static constexpr int NW = NT / 32;
    int hist[3][256];                    // counts of digit d in d mod 3
    uint32_t cand[RANKED];                   // the keys that the digits so far leave open
    uint32_t lo[NW], hi[NW];
    int gt[NW], eq[NW];
    int ncand, left;
    uint32_t t;
};

template <int NT, bool STAGED>
__device__ __forceinline__ void pick(const uint32_t *keys, const int32_t *ids, int n, int want,
                                     int32_t *sel, int32_t *phys, Pick<NT> &s)
{
    constexpr int NW = NT / 32;
    constexpr int BATCH = 4;             // keys a thread loads before it uses them
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto key = [&](int i) { return STAGED ? keys[i] : __ldcg(keys + i); };
    // f(key) for every key, in no particular order
    auto for_keys = [&](auto f) {
#pragma unroll 1
        for (int i0 = tid; i0 < n; i0 += NT * BATCH) {
            uint32_t k[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                k[u] = key(min(i0 + u * NT, n - 1));
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                if (i0 + u * NT < n)
                    f(k[u]);
        }
    };
    // the keys' range
    uint32_t lo = 0xffffffffu, hi = 0u;
    for_keys([&](uint32_t k) {
        lo = min(lo, k);
        hi = max(hi, k);
    });
    lo = __reduce_min_sync(FULL_MASK, lo);
    hi = __reduce_max_sync(FULL_MASK, hi);
    if (lane == 0) {
        s.lo[warp] = lo;
        s.hi[warp] = hi;
    }
    if (tid < 256)
        s.hist[0][tid] = s.hist[1][tid] = 0;
    if (tid == 0)
        s.ncand = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        lo = min(lo, s.lo[w]);
        hi = max(hi, s.hi[w]);
    }
    // t, relative to lo: the want-th largest key, by digits of up to 8 bits; `left`
    // of the keys that share t's digits so far are still to take.  Once few are
    // open, their ranks among one another say the rest.
    int top = hi > lo ? 32 - __clz(hi - lo) : 0;      // bits not decided yet
    uint32_t t = 0;
    int left = want, open = n;
#pragma unroll 1
    for (int d = 0; top > 0 && open > RANKED; ++d) {
        int *hist = s.hist[d % 3];
        const int shift = max(top - 8, 0);
        const uint32_t mask = (1u << (top - shift)) - 1u;
        for_keys([&](uint32_t k) {
            k -= lo;
            if (top >= 32 || (k >> top) == (t >> top))
                atomicAdd(&hist[(k >> shift) & mask], 1);
        });
        // the next digit's counts at zero; digit d - 2's, in the same place, were
        // read before the last barrier
        if (tid < 256)
            s.hist[(d + 1) % 3][tid] = 0;
        __syncthreads();
        // every warp finds the digit for itself, bins from the top: lane l
        // holds bins 255 - 8 l .. 248 - 8 l
        int c[8], sum = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            c[u] = hist[255 - 8 * lane - u];
            sum += c[u];
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(FULL_MASK, inc, off);
            if (lane >= off)
                inc += x;
        }
        const int l = __ffs(__ballot_sync(FULL_MASK, inc >= left)) - 1;
        int above = inc - sum, bin = 0, rest = 0, in = 0;
        bool found = false;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (!found && above + c[u] >= left) {
                found = true;
                bin = 255 - 8 * lane - u;
                rest = left - above;
                in = c[u];
            }
            above += c[u];
        }
        t |= (uint32_t)__shfl_sync(FULL_MASK, bin, l) << shift;
        left = __shfl_sync(FULL_MASK, rest, l);
        open = __shfl_sync(FULL_MASK, in, l);
        top = shift;
    }
    if (top > 0) {
        for_keys([&](uint32_t k) {
            k -= lo;
            if (top >= 32 || (k >> top) == (t >> top))
                s.cand[atomicAdd(&s.ncand, 1)] = k;
        });
        __syncthreads();
        if (tid < open) {
            // keys above this one, and as large: it is the one sought if the
            // left-th largest falls among the latter
            const uint32_t mine = s.cand[tid];
            int gt = 0, ge = 0;
#pragma unroll 8
            for (int i = 0; i < open; ++i) {
                const uint32_t k = s.cand[i];
                gt += k > mine;
                ge += k >= mine;
            }
            if (gt < left && left <= ge) {   // (equal keys write the same)
                s.t = mine;
                s.left = left - gt;
            }
        }
        __syncthreads();
        t = s.t;
        left = s.left;
    }
    t += lo;
    // keys above t, and the first `left` equal ones, in index order: each warp
    // ranks a contiguous run of indices, 32 at a time
    const int per = ((n + NW - 1) / NW + 31) & ~31;
    const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
    const unsigned below = (1u << lane) - 1u;
    // f(index, key) for the warp's run, 32 indices at a time in order
    auto for_run = [&](auto f) {
#pragma unroll 1
        for (int i = i0; i < i1; i += 32 * BATCH) {
            uint32_t k[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                k[u] = key(min(i + 32 * u + lane, i1 - 1));
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                f(i + 32 * u + lane, k[u]);
        }
    };
    int g = 0, e = 0;
    for_run([&](int i, uint32_t k) {
        g += __popc(__ballot_sync(FULL_MASK, i < i1 && k > t));
        e += __popc(__ballot_sync(FULL_MASK, i < i1 && k == t));
    });
    if (lane == 0) {
        s.gt[warp] = g;
        s.eq[warp] = e;
    }
    __syncthreads();
    g = e = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        if (w < warp) {
            g += s.gt[w];
            e += s.eq[w];
        }
    for_run([&](int i, uint32_t k) {
        const bool gt = i < i1 && k > t, eq = i < i1 && k == t;
        const unsigned mg = __ballot_sync(FULL_MASK, gt), me = __ballot_sync(FULL_MASK, eq);
        const int re = e + __popc(me & below);
        if (gt || (eq && re < left)) {
            const int at = g + __popc(mg & below) + min(re, left);
            sel[at] = i;
            phys[at] = ids[i];
        }
        g += __popc(mg);
        e += __popc(me);
    });
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) select_kernel(const SelectArgs a)
{
    constexpr int NW = NT / 32;
    constexpr int NC = D / 32;               // 16-byte chunks a lane reads of a block's bounds
    extern __shared__ uint32_t s_keys[];     // keys, then (from a.stage on) ids
    __shared__ Pick<NT> s_pick;
    __shared__ int s_last;
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x / a.chunks, part = blockIdx.x - seg * a.chunks;
    const int H = a.num_kv_heads, b = seg / H, kvh = seg - b * H;
    int L = a.seq_lens[b];
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
            phys[i] = row[i];
        }
        return;
    }
    if (part == 0 && tid == 0) {             // the newest block, always
        sel[nsel - 1] = n - 1;
        phys[nsel - 1] = row[n - 1];
    }
    if (a.budget == 1)
        return;

    // ---- the group's query values in whole steps of 2^eq, as B fragments: lane
    // (gid, tig) holds head gid mod G and the channels of its chunks 4 c + tig of
    // the bounds: negative parts for the lower bounds (c < NC / 2), positive
    // parts for the upper ones
    const int gid = lane >> 2, tig = lane & 3;
    uint32_t qf[4 * NC][2];
    {
        const uint4 *qsrc = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(a.q) + (((int64_t)b * H + kvh) * G + gid % G) * D) +
            2 * tig;
        uint32_t raw[NC / 2][8];
        float amax = 0.0f;
        auto pair = [&](uint32_t w) {
            return a.q_dtype == PKV_BF16 ? make_float2(bf16lo(w), bf16hi(w)) : half2_to_float2(w);
        };
#pragma unroll
        for (int c = 0; c < NC / 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 x = qsrc[8 * c + h];
                raw[c][4 * h] = x.x; raw[c][4 * h + 1] = x.y;
                raw[c][4 * h + 2] = x.z; raw[c][4 * h + 3] = x.w;
            }
#pragma unroll
        for (int c = 0; c < NC / 2; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = pair(raw[c][i]);
                amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, m));
        const float f = pow2_f32(-int8_exponent(amax));
        auto step = [&](float x) { return fminf(fmaxf(rintf(x * f), -127.0f), 127.0f); };
        const __half2 zero = __floats2half2_rn(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < NC / 2; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = pair(raw[c][i]);
                const __half2 v = __floats2half2_rn(step(x.x), step(x.y));
                const __half2 neg = __hmin2(v, zero), pos = __hmax2(v, zero);
                qf[4 * c + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t *>(&neg);
                qf[4 * (c + NC / 2) + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t *>(&pos);
            }
    }

    // ---- scores of this CTA's blocks (the newest one is not scored): 32
    // blocks a warp at a time
    uint32_t *keys = a.keys + (int64_t)seg * a.max_n;
    const int parts = (n + a.chunk - 1) / a.chunk;
    const int j_end = min(n - 1, j_begin + a.chunk);
    constexpr int STEP = NW * 32;
    // the block ids of the lane's block of a group, its exponent, and the
    // bounds of rows gid, gid + 8 of a 16-block tile (the lane's chunks)
    auto load_id = [&](int j0) {
        return j0 + lane < j_end ? row[j0 + lane] : 0;
    };
    auto valid_id = [&](int id) {
        if (id >= 0 && id < a.num_blocks)
            return id;
        atomicOr(a.err, PKV_EBIT_BLOCK);
        return 0;
    };
    auto load_tile = [&](uint4 (&x)[2][NC], int id, int t) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int id_r = __shfl_sync(FULL_MASK, id, 16 * t + 8 * r + gid);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.bounds + ((int64_t)id_r * H + kvh) * 2 * D) + tig;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                x[r][c] = src[4 * c];
        }
    };
    // a tile's scores: lane l gets that of row l mod 16
    auto score_tile = [&](const uint4 (&x)[2][NC]) {
        float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t u[4] = {x[0][c].x, x[0][c].y, x[0][c].z, x[0][c].w};
            const uint32_t v[4] = {x[1][c].x, x[1][c].y, x[1][c].z, x[1][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t ub = u[i] ^ 0x80808080u, vb = v[i] ^ 0x80808080u;
                kern::mma_16816<false>(s[i & 1], kern::i8pair_to_half2<0x4140u>(ub),
                                       kern::i8pair_to_half2<0x4140u>(vb),
                                       kern::i8pair_to_half2<0x4342u>(ub),
                                       kern::i8pair_to_half2<0x4342u>(vb), qf[4 * c + i][0],
                                       qf[4 * c + i][1]);
            }
        }
        // rows gid and gid + 8: the largest over the columns (heads)
        float m0 = fmaxf(s[0][0] + s[1][0], s[0][1] + s[1][1]);
        float m1 = fmaxf(s[0][2] + s[1][2], s[0][3] + s[1][3]);
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(FULL_MASK, m0, m));
            m1 = fmaxf(m1, __shfl_xor_sync(FULL_MASK, m1, m));
        }
        const float r0 = __shfl_sync(FULL_MASK, m0, 4 * (lane & 7));
        const float r1 = __shfl_sync(FULL_MASK, m1, 4 * (lane & 7));
        return lane & 8 ? r1 : r0;
    };
    int j0 = j_begin + warp * 32;
    if (j0 < j_end) {
        // a tile's bounds are on their way while the one before is scored
        int raw = load_id(j0), raw_next = load_id(j0 + STEP);
        int id = valid_id(raw);
        int e = a.exps[(int64_t)id * H + kvh];
        uint4 x0[2][NC], x1[2][NC];
        load_tile(x0, id, 0);
#pragma unroll 1
        for (;;) {
            load_tile(x1, id, 1);
            const float even = score_tile(x0);
            const bool ok = raw == id;
            const int raw_now = raw, e_now = e, j = j0 + lane;
            j0 += STEP;
            const bool more = j0 < j_end;
            if (more) {
                raw = raw_next;
                id = valid_id(raw);
                raw_next = load_id(j0 + STEP);
                e = a.exps[(int64_t)id * H + kvh];
                load_tile(x0, id, 0);
            }
            const float odd = score_tile(x1);
            if (j < j_end) {
                const int ec = min(max(e_now, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
                const uint32_t k =
                    ok ? sort_key((lane < 16 ? even : odd) * pow2_f32(ec - 22)) : 0u;
                if (parts == 1 && a.stage) {
                    s_keys[j] = k;
                    s_keys[a.stage + j] = raw_now;
                } else {
                    keys[j] = k;
                }
            }
            if (!more)
                break;
        }
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
            for (int i = tid; i < n - 1; i += NT) {
                s_keys[i] = __ldcg(keys + i);
                s_keys[a.stage + i] = row[i];
            }
            __syncthreads();
        }
    }
    if (a.stage)
        pick<NT, true>(s_keys, reinterpret_cast<const int32_t *>(s_keys + a.stage), n - 1,
                       a.budget - 1, sel, phys, s_pick);
    else
        pick<NT, false>(keys, row, n - 1, a.budget - 1, sel, phys, s_pick);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The regions of the workspace behind the counters (which the choice and the
// attention use one after the other, each leaving them zero) and the partials.
struct Regions {
    size_t phys, keys, total;
};

Regions regions(const pkv_pool *pool, int batch, int num_q_heads, int max_seq_len, int budget)
{
    const size_t segs = (size_t)batch * pool->num_kv_heads;
    const size_t n = ((size_t)max_seq_len + pool->block_size - 1) / pool->block_size;
    Regions r;
    r.phys = block_workspace_bytes(pool, batch, num_q_heads);
    r.keys = r.phys + up256(segs * budget * sizeof(int32_t));
    r.total = r.keys + up256(segs * n * sizeof(uint32_t));
    return r;
}

template <int D, int G, int NT>
cudaError_t launch_select_t(const SelectArgs &a, unsigned grid, size_t smem, cudaStream_t s)
{
    // The limit belongs to the kernel, not to the launch: the most that any call asks for,
    // so that a call from another host thread between this one's setting and its launch
    // changes nothing.
    cudaError_t e = cudaFuncSetAttribute(select_kernel<D, G, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SMEM_KEYS * 8);
    if (e != cudaSuccess)
        return e;
    // of the SM's 228 KB for shared memory and L1 no more than the CTAs use as shared
    // memory: up to 128 KB of bounds are in flight through the L1, and without this
    // the kernel runs with the division that the one before it had (behind the
    // attention with all of it as shared memory, 54 instead of 46 us for the choice
    // of 128 of 2048 blocks of 16 sequences and the attention over them).  A preference:
    // another thread's call in between costs time, not the launch.
    const size_t used = 512 / NT * (smem + sizeof(Pick<NT>) + 1280);
    const int percent = (int)std::min<size_t>(100, (used * 100 + 233471) / 233472);
    e = cudaFuncSetAttribute(select_kernel<D, G, NT>,
                             cudaFuncAttributePreferredSharedMemoryCarveout, percent);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(select_kernel<D, G, NT>, dim3(grid), dim3(NT), smem, s, a);
}

// 16 warps a CTA where every CTA has an SM to itself, else 8 and two CTAs a SM
// (256 CTAs on 152 SMs: 38 instead of 43 us with the attention behind them).
template <int D, int G>
cudaError_t launch_select_g(const SelectArgs &a, int num_sms, unsigned grid, size_t smem,
                            cudaStream_t s)
{
    return (int64_t)grid <= num_sms ? launch_select_t<D, G, 512>(a, grid, smem, s)
                                    : launch_select_t<D, G, 256>(a, grid, smem, s);
}

template <int D>
cudaError_t launch_select(const SelectArgs &a, int G, int num_sms, unsigned grid, size_t smem,
                          cudaStream_t s)
{
    switch (G) {
    case 1: return launch_select_g<D, 1>(a, num_sms, grid, smem, s);
    case 2: return launch_select_g<D, 2>(a, num_sms, grid, smem, s);
    case 4: return launch_select_g<D, 4>(a, num_sms, grid, smem, s);
    default: return launch_select_g<D, 8>(a, num_sms, grid, smem, s);
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
    a.counters = reinterpret_cast<int *>(ws);
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
    // a CTA's chunk: all of a (sequence, KV head)'s blocks where there are enough
    // of those for most SMs (nothing is handed from CTA to CTA then), else in
    // steps of 8 warps' groups what gives every SM a CTA
    const int64_t segs = (int64_t)batch * H, n = (cap + bs - 1) / bs;
    const int64_t per = (segs * n + pool->num_sms - 1) / pool->num_sms;
    const int64_t span = 256;
    a.chunk = (int)std::max<int64_t>(span, (per + span - 1) / span * span);
    if (segs * 3 >= (int64_t)pool->num_sms * 2 && n <= SMEM_KEYS)
        a.chunk = (int)std::max<int64_t>(a.chunk, n);
    a.chunks = (int)std::max<int64_t>(1, (n + a.chunk - 1) / a.chunk);
    a.stage = n <= SMEM_KEYS ? (int)n : 0;
    const size_t smem = (size_t)a.stage * 8;
    const int64_t tiles_a_head =
        (std::min<int64_t>(cap, (int64_t)budget * bs) + blk::TILE - 1) / blk::TILE;
    const int64_t max_tiles = segs * tiles_a_head;
    if (segs * a.chunks > INT32_MAX || max_tiles > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(segs * a.chunks);
    const int G = num_q_heads / H;
    const cudaError_t e = pool->head_dim == 64 ? launch_select<64>(a, G, pool->num_sms, grid, smem, s)
                                               : launch_select<128>(a, G, pool->num_sms, grid, smem, s);
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
