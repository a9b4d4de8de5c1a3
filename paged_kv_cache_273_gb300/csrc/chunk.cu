// paged_chunk_attention: attention of each sequence's new tokens over its cached rows
// (the new ones among them): a piece of a prompt, a whole one, or a few drafted tokens.
//
// softmax(scale q K^T) V of "KV cache: the engine behind fast LLM inference",
// "Concept", in tiles of 128 keys with a running maximum and sum ("Flash attention:
// don't build the giant matrix" in the guide), on the fifth-generation tensor cores.
//
// A (token, query head) pair is a row; the G query heads of a KV head are packed, so
// one read of K and V serves them all, and n tokens make n G rows.  An item is up to 256
// (or 128) rows of one (sequence, KV head); chunk_schedule.h cuts all items' key tiles
// into one share a CTA, so that one long sequence fills the GPU as well as a large batch
// does.  An item that is cut leaves one state (weighted sum, maximum, sum) a
// piece, which chunk_join_kernel joins in the order of the keys: the result does not depend on
// timing.
//
// Within a CTA two softmax groups of 128 threads, a thread a row, alternate on the
// tensor cores.  Of an item of more than 128 rows each group has its own rows, and both read
// each K and V tile; of a smaller one both have the same rows, and every other
// key tile each: the first group joins the two states at the piece's end, out of tensor memory.
//
// Bound: few new tokens read K and V once for n G rows, so memory is the floor (n G below
// about 290 rows of 16-bit keys, half that of e4m3); long pieces are bound by the tensor cores
// and by the softmax between a group's two products.  Measured on a GB300 (a call in a
// captured chain, both kernels): 8 drafted tokens each of 16 sequences' 271 MB of rows 56 us
// (4.8 TB/s); whole prompts of 550 GFLOP 435 to 453 us on several GPUs (1.21 to 1.26 PFLOP/s, the tensor
// cores 55% busy); pieces over e4m3 of 756 GFLOP 880 us (0.86 PFLOP/s, 45%); 32 tokens of 64 heads over
// 131000 e4m3 rows 140 us.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "blocks_common.cuh"
#include "chunk_schedule.h"
#include "tc_common.cuh"

namespace pkv {
namespace {

using namespace dev;
using chunk::Piece;
using chunk::Place;
using chunk::Rules;
using chunk::Seq;
using chunk::TILE;
using chunk::Walk;

struct ChunkParams {
    CUtensorMap tm_q;             // q [T][Hq][D]: boxes of 64 columns x G heads x 128 / G tokens
    CUtensorMap tm_k, tm_v;       // 16-bit caches: boxes of box_rows whole rows
    const void *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *tables, *q_start, *seq_lens;
    const uint64_t *visible;
    void *out;
    int32_t *places;              // [0]: shares; from [8] on a share's pieces to join; from
                                  // [items_at] on their item: token, rows, KV head
    int items_at;
    uint32_t share_step;          // 2^32 / the grid's CTAs
    float *part;                  // 2 states a CTA: that of its first piece, and of its last
    unsigned int *err;
    int batch, num_tokens, max_q_len, num_q_heads, num_kv_heads, lg_g;
    int block_size, bs_log2, max_blocks, num_blocks;
    int box_rows;                 // min(block_size, 128): rows of a tile from one block
    float scale_log2;
    Rules rules;
};

// Warps: the softmax groups; then, of a 16-bit cache, one that brings K, one V, one that
// hands out the pieces and brings their q, and one that issues the MMAs; of an 8-bit cache,
// four that bring and convert tiles, the MMA warp, the one for pieces and q, and one that
// brings the tiles' scales.
template <int D, bool F8, bool BF, int NQ>
struct Cfg {
    static constexpr int ROWS = NQ * TILE_M;
    static constexpr int Q_BYTES = TILE_M * D * 2;                       // one half
    static constexpr int KV_BYTES = TILE * D * 2;
    // ring slots: what shared memory holds
    static constexpr int NS = D == 64 ? 4 : NQ == 1 && !F8 ? 3 : 2;
    // tiles' scales: read until the tile's softmax, when NS + 1 tiles more may be there
    static constexpr int RING = 8;
    static_assert(RING >= NS + 2, "scales in use");
    static constexpr int OFF_K = NQ * Q_BYTES;
    static constexpr int OFF_V = OFF_K + NS * KV_BYTES;
    static constexpr int OFF_ML = OFF_V + NS * KV_BYTES;                 // the second group's states
    // [RING][FAC / 16][16]: scales of K, exponents of V's, and two to minus these
    static constexpr int FAC = 48;
    static constexpr int OFF_SC = OFF_ML + (F8 ? 3 : 2) * TILE_M * 4;
    static constexpr int OFF_QE = OFF_SC + (F8 ? RING * FAC * 4 : 0);     // q's exponents, two pieces
    static constexpr int OFF_BAR = OFF_QE + (F8 ? 2 * TILE_M : 0);
    static constexpr int PIECES = 4;                                     // handed out and not done
    static constexpr int NBARS = 4 * NS + 8 + 6 + 2 * PIECES;
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;                 // tensor memory's address, flag, pieces
    static constexpr int SMEM_BYTES = OFF_MISC + 224;
    static constexpr int W0 = 8;                                         // the first warp behind the groups
    static constexpr int W_MMA = F8 ? W0 + 4 : W0 + 3, W_FEED = F8 ? W0 + 5 : W0 + 2;
    static constexpr int W_SCALES = W0 + 6;                              // of an 8-bit cache
    static constexpr int CONSUMERS = W0 + (F8 ? 6 : 3);                  // warps that a piece is for
    static constexpr bool QCONV = F8 && BF;
    static constexpr int NT = 32 * (F8 ? W0 + 8 : W0 + 4);
    // registers of a thread: at launch, and from then on in the softmax groups, the four
    // warps behind them, and the last four (the shares add up to what was there at launch)
    static constexpr int REGS = F8 ? 128 : 168;
    static constexpr int R_SOFT = F8 ? 168 : 216, R_2 = F8 ? 112 : 72, R_3 = F8 ? 64 : 0;
    static_assert(2 * R_SOFT + R_2 + R_3 <= NT / 128 * REGS, "registers");
    static constexpr int GROUP_COLS = 256;                               // S, then O, of a group
    // a K or V tile: eight rows of 64 columns are 1024 bytes (128-byte swizzled); a group of
    // eight rows holds its panels one after the other, so that one tensor copy brings
    // a block's whole rows (two of 64 columns each cost the warp that issues them
    // twice as long, more than a tile's time on the tensor cores)
    static constexpr int GROUP8 = 1024 * (D / 64);
    // P in the caches' 16-bit type; over an 8-bit cache, whose codes become fp16, in fp16.  One
    // rounding of a weight, no second part for the rest: it moves an output by about what the
    // output's own rounding to q's type does (bf16 2.1e-3 of its size rather than 1.6e-3, fp16
    // 2.7e-4 rather than 2.1e-4), and P V of two parts would add half as many MMAs again
    // (prefill.cu, whose fp32 output shows the rest, takes 717 us for these prompts).
    static constexpr bool PBF = BF && !F8;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// Byte offset of 16-byte chunk ch of row r in a K or V tile.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int ch)
{
    return (uint32_t)((r >> 3) * (1024 * (D / 64)) + (ch >> 3) * 1024 + (r & 7) * 128 +
                      (((ch & 7) ^ (r & 7)) << 4));
}

// Rows that a sequence may have: positions of a tile's keys stay below 2^31.
constexpr int MAX_LEN = 1 << 30;

// What a wait for the end of a piece may take for each of its tiles, beside WAIT_LIMIT_NS.
constexpr uint64_t TILE_LIMIT_NS = 1 << 17;

// Sequence b's lengths; false if it has no work.
__device__ __forceinline__ bool lengths(const ChunkParams &p, int b, Seq &q, int &q0, bool &bad)
{
    q0 = p.q_start[b];
    const int64_t n = (int64_t)p.q_start[b + 1] - q0;
    const int L = p.seq_lens[b];
    bad = n < 0 || (n > 0 && (q0 < 0 || n > p.max_q_len || q0 + n > p.num_tokens || L < n ||
                              (int64_t)L > (int64_t)p.max_blocks * p.block_size || L > MAX_LEN ||
                              (p.rules.tree && n > 64)));
    q.n = bad ? 0 : (int)n;
    q.L = L;
    return q.n > 0;
}

// What a group does of a piece: its rows, and its s-th key tile.
__device__ __forceinline__ bool shared_rows(const Piece &c) { return c.rows <= TILE_M; }
__device__ __forceinline__ int group_tiles(const ChunkParams &p, const Piece &c, int g)
{
    const int nt = c.t1 - c.t0;
    if (shared_rows(c))
        return (nt + 1 - g) / 2;
    if (g == 1 || p.rules.tree)
        return nt;
    // the first half's last token sees fewer keys
    const int last = c.first + (TILE_M >> p.lg_g) - 1;
    return min(nt, max(0, last / TILE + 1 - c.t0));
}
__device__ __forceinline__ int tile_at(const Piece &c, int g, int s)
{
    return shared_rows(c) ? 2 * s + g : s;            // behind t0
}

// Where this share starts and ends: the sequences' costs are summed over the CTA, and the
// threads whose sequences hold the two positions place them.
template <int NT>
__device__ __forceinline__ bool find_share(const ChunkParams &p, Place *places, int64_t *sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.batch + NT - 1) / NT;
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    const int c = blockIdx.x;
    int64_t mine = 0, before = 0, U = 0;
    int n = 0;
    // first the sum, then the two places (one body, for the instruction cache's sake)
#pragma unroll 1
    for (int k = -1; k < 2; ++k) {
        int64_t x = k < 0 ? -1 : chunk::share_start(U, n, c + k, gridDim.x, p.share_step) - before;
        if (k >= 0 && (x < 0 || x >= mine))
            continue;
        int64_t sum = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            Seq q;
            int q0;
            bool bad;
            if (lengths(p, b, q, q0, bad)) {
                const int64_t one = chunk::cost_of(p.rules, q), cost = p.num_kv_heads * one;
                if (k >= 0 && x < sum + cost) {
                    places[k] = chunk::place_in(p.rules, q, b, x - sum, one);
                    break;
                }
                sum += cost;
            }
            if (bad && k < 0 && c == 0)
                atomicOr(p.err, PKV_EBIT_SEQLEN);
        }
        if (k >= 0)
            continue;
        mine = sum;
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(FULL_MASK, upto, m);
            if (lane >= m)
                upto += o;
        }
        if (lane == 31)
            sums[warp] = upto;
        __syncthreads();
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp)
                before += sums[w];
            U += sums[w];
        }
        before += upto - mine;
        n = chunk::shares(U, gridDim.x);
        if (c == 0 && tid == 0)
            p.places[0] = U > 0 ? n : 0;
        if (U == 0 || c >= n)
            return false;
        if (tid == 0 && c + 1 == n) {
            Place e{};
            e.b = p.batch;
            places[1] = e;
        }
    }
    if (tid == 0)
        sums[NT / 32] = U;
    __syncthreads();
    return true;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// One block's rows (or 128 of them) of one KV head, from its group `y` of eight on.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int y, int z,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// For the joining (one thread, of a warp that is done): the item that this share starts within,
// if the share is the first to do so, its pieces, its first token and its rows.
__device__ __forceinline__ void note_item(const ChunkParams &p, const Place &a, int64_t U)
{
    const int c = blockIdx.x, n = chunk::shares(U, gridDim.x);
    int4 item = make_int4(0, 0, 0, 0);
    int pieces = 0;
    if (a.split) {
        Seq q;
        int q0;
        bool bad;
        lengths(p, a.b, q, q0, bad);
        pieces = chunk::pieces_to_join(p.rules, q, a, U, n, c, gridDim.x, p.share_step);
        item = make_int4(q0 + (a.rt << p.rules.lg_tpr),
                         min(1 << p.rules.lg_tpr, q.n - (a.rt << p.rules.lg_tpr)) << p.lg_g, a.h, 0);
    }
    p.places[8 + c] = pieces;
    reinterpret_cast<int4 *>(p.places + p.items_at)[c] = item;
}

// 16 e4m3 codes -> 16 fp16 values (exact), as two 16-byte chunks.
__device__ __forceinline__ void codes_to_half(const uint4 &w, uint4 &lo, uint4 &hi)
{
    f8x4_to_half2(w.x, lo.x, lo.y);
    f8x4_to_half2(w.y, lo.z, lo.w);
    f8x4_to_half2(w.z, hi.x, hi.y);
    f8x4_to_half2(w.w, hi.z, hi.w);
}

// Chunks 2j and 2j + 1 of a row: the second panel's lanes write their odd one first, so that
// eight lanes' stores fall on all banks.
template <int D>
__device__ __forceinline__ void put_chunks(unsigned char *tile, int row, int j, const uint4 &lo,
                                           const uint4 &hi)
{
    const int odd = j >> 2;
    *reinterpret_cast<uint4 *>(tile + tile_off<D>(row, 2 * j + odd)) = odd ? hi : lo;
    *reinterpret_cast<uint4 *>(tile + tile_off<D>(row, 2 * j + 1 - odd)) = odd ? lo : hi;
}

// fp16 weights are taken times 2^7: the running maximum moves when a score is 2^8 above it, so
// they stay below 2^15, and weights down to 2^-21 of the largest keep all their bits.
constexpr float P_SHIFT = 7.0f;

// O over an 8-bit cache is kept times 2^-16 outside of tensor memory (the sum over many keys
// of values near fp32's largest is beyond it; their quotient by the weights' sum is not).
constexpr int V_SHIFT = 16;

// Row r of a half of q (bf16, as the tensor copy left it) -> fp16 times 2^-e in place, the
// row's largest magnitude in [2^14, 2^15); returns e.
template <int D>
__device__ __forceinline__ int halve_row(unsigned char *q, int r)
{
    auto at = [&](int ch) {
        return reinterpret_cast<uint4 *>(q + (ch >> 3) * (TILE_M * 128) + r * 128 +
                                         (((ch & 7) ^ (r & 7)) << 4));
    };
    uint32_t top = 0;                              // magnitudes order as their bits
#pragma unroll
    for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 w = *at(ch);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            top = max(top, max(v[k] << 16 & 0x7fffffffu, v[k] & 0x7fff0000u));
    }
    const int e = max((int)(top >> 23) - 127 - 14, -126);
    const float f = pow2_f32(-e);
#pragma unroll
    for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 w = *at(ch);
        uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = pack2<__half>(bf16lo(v[k]) * f, bf16hi(v[k]) * f);
        *at(ch) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    return e;
}

template <int D, bool F8, bool BF, int NQ>
__global__ void __launch_bounds__((Cfg<D, F8, BF, NQ>::NT), 1)
    chunk_kernel(const __grid_constant__ ChunkParams p)
{
    using C = Cfg<D, F8, BF, NQ>;
    constexpr int NS = C::NS, W0 = C::W0;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *sQ = smem, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V;
    float *ml = reinterpret_cast<float *>(smem + C::OFF_ML);
    float *k_sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    signed char *q_exp = reinterpret_cast<signed char *>(smem + C::OFF_QE);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
    uint64_t *s_full = v_empty + NS, *p_full = s_full + 2, *o_done = p_full + 2, *o_free = o_done + 2;
    uint64_t *q_full = o_free + 2, *q_empty = q_full + 1, *ml_full = q_empty + 1, *ml_free = ml_full + 1;
    uint64_t *drain = ml_free + 1;
    uint64_t *pc_full = drain + 1, *pc_empty = pc_full + C::PIECES, *q_raw = pc_empty + C::PIECES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Place *places = reinterpret_cast<Place *>(smem + C::OFF_MISC + 16);
    int64_t *sums = reinterpret_cast<int64_t *>(smem + C::OFF_MISC + 64);
    Piece *pieces = reinterpret_cast<Piece *>(smem + C::OFF_MISC + 16);    // (over the two above)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_map(&p.tm_q);
        if (!F8 && p.box_rows >= 8) {              // (blocks of 4 rows have no map)
            prefetch_map(&p.tm_k);
            prefetch_map(&p.tm_v);
        }
    }
    grid_dependency_wait();
    grid_dependents_launch();
    if (!find_share<C::NT>(p, places, sums))
        return;
    const Place begin = places[0];
    const int64_t line = sums[C::NT / 32];
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], F8 ? 5 : 2);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], F8 ? 4 : 2);
            mbar_init(&v_empty[i], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&s_full[g], 1);
            mbar_init(&p_full[g], 4);      // (a lane a warp arrives)
            mbar_init(&o_done[g], 1);
            mbar_init(&o_free[g], 4);
        }
        mbar_init(q_full, C::QCONV ? 8 : 1);
        mbar_init(q_raw, 1);
        for (int i = 0; i < C::PIECES; ++i) {
            mbar_init(&pc_full[i], 1);
            mbar_init(&pc_empty[i], C::CONSUMERS);
        }
        mbar_init(q_empty, 1);
        mbar_init(ml_full, 4);
        mbar_init(ml_free, 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == C::W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(tmem_slot)),
                     "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Every role but the one that hands out the pieces waits for a few tiles' work at most.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return mbar_wait_or_abort(bar, parity & 1, abort_flag);
    };
    Piece c;
    // The item-th piece, and when this warp is done with it.
    auto take = [&](uint32_t item) -> bool {
        if (!__all_sync(FULL_MASK, wait(&pc_full[item % C::PIECES], item / C::PIECES)))
            return false;
        c = pieces[item % C::PIECES];
        return c.kind >= 0;
    };
    auto done = [&](uint32_t item) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&pc_empty[item % C::PIECES]);
    };

    if (warp < W0)
        more_registers<C::R_SOFT>();
    else if (warp < W0 + 4)
        fewer_registers<C::R_2>();
    else
        fewer_registers<F8 ? C::R_3 : 24>();
    if (warp < W0) {
        // ================= softmax: group g, one thread a row
        const int g = warp >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;
        const uint32_t t_s = tmem + g * C::GROUP_COLS + ((uint32_t)(quad * 32) << 16), t_o = t_s + TILE;
        // the parities of the phases that come next, of s_full, o_done, ml_full and (group 0)
        // the second group's o_done; and (group 1) whether its state is being read
        uint32_t ph = 0;
        constexpr uint32_t P_S = 1, P_O = 2, P_ML = 4, P_O1 = 8, LENT = 16;
        int gt = 0;                                // the CTA's tiles so far
        auto phase = [&](uint64_t *bar, uint32_t bit) -> bool {
            const bool ok = __all_sync(FULL_MASK, wait(bar, (ph & bit) ? 1u : 0u));
            ph ^= bit;
            return ok;
        };
        for (uint32_t item = 0; take(item); ++item) {
            const bool both = shared_rows(c);
            const int row = both ? r : g * TILE_M + r;
            const bool warp_live = (both ? quad * 32 : g * TILE_M + quad * 32) < c.rows;
            const int pos = c.first + (row >> p.lg_g);
            // keys in sight: up to `lim`, from `from`, and of the new ones those of the row's bits
            const bool valid = row < c.rows;
            const int lim = !valid ? -1 : p.visible ? c.len - 1 : pos;
            const int from = p.rules.window > 0 ? pos - p.rules.window + 1 : 0;
            const uint64_t *bits_at = p.visible + (p.visible && valid ? c.tok + (row >> p.lg_g) : 0);
            const int nt = group_tiles(p, c, g);
            // The running maximum and sum; and over an 8-bit cache, where a block's V has a
            // scale of 2^E, the running maximum of score + E: what P (p 2^E) is taken
            // relative to, so that fp16 holds all that matters to this row however far apart
            // the scales are.
            float m_run = -INFINITY, l_run = 0.0f, x_run = -INFINITY, rs = p.scale_log2;
            if constexpr (C::QCONV) {
                // bf16 q over an 8-bit cache becomes fp16 times a power of two a row (K's
                // codes are fp16; what a row's small values lose is below 2^-38 of its
                // largest), in place
                // (a group whose rows the other converts waits all the same: its arrival
                // counts once an item)
                if (!__all_sync(FULL_MASK, wait(q_raw, item)))
                    goto softmax_done;
                if (!both || g == 0) {
                    const int e = halve_row<D>(sQ + (both ? 0 : g) * C::Q_BYTES, r);
                    rs *= pow2_f32(e);
                    if (both)
                        q_exp[(item & 1) * TILE_M + r] = (signed char)e;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full);
            }
            for (int s = 0; s < nt; ++s) {
                const int tb = (c.t0 + tile_at(c, g, s)) * TILE;       // the tile's first key
                if (!phase(&s_full[g], P_S))
                    goto softmax_done;
                tc_fence_after();
                if (warp_live) {
                    if (C::QCONV && both && g == 1 && s == 0)
                        rs *= pow2_f32(q_exp[(item & 1) * TILE_M + r]);
                    const float *fac = k_sc + ((gt + tile_at(c, g, s)) & (C::RING - 1)) * C::FAC;
                    const bool masked = __any_sync(
                        FULL_MASK, tb + TILE - 1 > lim || tb < from ||
                                       (p.visible && tb + TILE > c.base));
                    // keys in sight among the 32 from c0 on
                    auto in_sight = [&](int c0) -> uint32_t {
                        const int k0 = tb + c0, u = lim - k0, d = from - k0;
                        uint32_t w = u >= 31 ? 0xffffffffu : u < 0 ? 0u : (2u << u) - 1u;
                        if (d > 0)
                            w = d < 32 ? w & (0xffffffffu << d) : 0u;
                        if (p.visible) {
                            const int e = k0 - c.base;
                            const uint64_t bits = *bits_at;
                            if (e >= 0)
                                w &= e < 64 ? (uint32_t)(bits >> e) : 0u;
                            else if (e > -32)
                                w &= (uint32_t)(bits << -e) | ((1u << -e) - 1u);
                        }
                        return w;
                    };
                    constexpr int HW = TILE / 2;
                    auto hide = [&](float *x, int h0) {
                        if (masked) {
#pragma unroll
                            for (int c0 = 0; c0 < HW; c0 += 32) {
                                const uint32_t w = in_sight(h0 + c0);
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    x[c0 + j] = (w >> j) & 1 ? x[c0 + j] : -INFINITY;
                            }
                        }
                    };
                    // The running maxima move only when a score exceeds them by more than
                    // 2^8 (or is the first in sight): below that the weights stay <= 2^8, and
                    // the quotient by the sum of the same weights is unchanged.
                    auto moved = [&](float &run, float mx) -> float {
                        const float was = run;
                        run = mx > was + 8.0f ? mx : was;
                        return run == was ? 1.0f : was == -INFINITY ? 0.0f : ex2_approx(was - run);
                    };
                    // O is idle at this point: the P V of the previous tile finished before
                    // this S did, the next one waits for p_full
                    auto rescale = [&](float corr) {
                        if (s == 0 || !__any_sync(FULL_MASK, corr != 1.0f))
                            return;
                        // (rare: few registers rather than few loads)
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 8) {
                            float o[8];
                            uint32_t w[8];
                            tmem_ld_begin<8>(t_o + c0, o);
                            tmem_ld_end<8>(o);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                w[j] = __float_as_uint(o[j] * corr);
                            tmem_st8(t_o + c0, w);
                        }
                    };
                    using PT = typename std::conditional<C::PBF, __nv_bfloat16, __half>::type;
                    float mx = -INFINITY;
                    if constexpr (!F8) {
                        // half of the scores, then their maximum under way while the others come
                        float v[TILE];
                        auto highest = [&](const float *x) {
                            float t[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int j = 4; j < HW; j += 8)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    t[k] = j + 4 < HW ? max3f(t[k], x[j + k], x[j + 4 + k])
                                                      : fmaxf(t[k], x[j + k]);
                            mx = fmaxf(mx, max3f(fmaxf(t[0], t[1]), t[2], t[3]));
                        };
                        tmem_ld_begin<HW>(t_s, v);
                        tmem_ld_end<HW>(v);
                        tmem_ld_begin<HW>(t_s + HW, v + HW);
                        hide(v, 0);
                        highest(v);
                        tmem_ld_end<HW>(v + HW);
                        hide(v + HW, HW);
                        highest(v + HW);
                        const float corr = moved(m_run, mx * rs);   // (scale > 0: the maximum commutes)
                        rescale(corr);
                        // Weights, their sum, and P over the S columns: of each 64 keys the
                        // 16-bit pairs in 32 columns.  Eight keys a step: the exponents of one
                        // eight, the exponentials of the one before, the rounding and summing
                        // of the one before that, so that the three units that they run on
                        // work at once.
                        const float off = (C::PBF ? 0.0f : P_SHIFT) - (m_run == -INFINITY ? 0.0f : m_run);
                        float sum[4] = {};
                        constexpr int E = TILE / 8;
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < E + 2; ++i) {
                            if (i < E)
#pragma unroll
                                for (int j = 8 * i; j < 8 * i + 8; j += 2)
                                    fma2_bc(v[j], v[j + 1], rs, off);
                            if (i >= 1 && i <= E)
#pragma unroll
                                for (int j = 8 * i - 8; j < 8 * i; ++j)
                                    v[j] = ex2_approx(v[j]);
                            if (i >= 2) {
                                const float *y = v + 8 * i - 16;
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    w[(i & 1) * 4 + j] = pack2<PT>(y[2 * j], y[2 * j + 1]);
                                add2(sum[0], sum[1], y[0], y[1]);
                                add2(sum[2], sum[3], y[2], y[3]);
                                add2(sum[0], sum[1], y[4], y[5]);
                                add2(sum[2], sum[3], y[6], y[7]);
                                if (i & 1)
                                    tmem_st8(t_s + (i - 2) / 8 * 64 + (i - 2) % 8 / 2 * 8, w);
                            }
                        }
                        l_run = l_run * corr + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
                    } else {
                        // One half of the scores after the other, the first one read again for its
                        // weights: registers are the conversion's too, and both halves written
                        // out (929 us rather than 880) take more of the instruction cache.
                        // A factor for eight keys: K's scale, the row's own and the softmax's
                        // (at least the smallest normal number: -inf times it is -inf).
                        float v[HW], mv = -INFINITY;
                        auto factor = [&](float ks) { return fmaxf(ks * rs, 0x1p-126f); };
                        auto eight = [&](float (&f)[8], int at) {
#pragma unroll
                            for (int k = 0; k < 8; k += 4)
                                *reinterpret_cast<float4 *>(f + k) = *reinterpret_cast<const float4 *>(fac + at + k);
                        };
#pragma unroll
                        for (int h0 = 0; h0 < TILE; h0 += HW) {
                            tmem_ld_begin<HW>(t_s + h0, v);
                            float kf[8], ve[8];
                            eight(kf, h0 / 8);
                            eight(ve, 16 + h0 / 8);
                            tmem_ld_end<HW>(v);
                            hide(v, h0);
#pragma unroll
                            for (int k = 0; k < HW / 8; ++k) {
                                const float *x = v + 8 * k;
                                const float a = max3f(max3f(x[0], x[1], x[2]), max3f(x[3], x[4], x[5]),
                                                      fmaxf(x[6], x[7])) * factor(kf[k]);
                                mx = fmaxf(mx, a);
                                mv = fmaxf(mv, a + ve[k]);
                            }
                        }
                        l_run *= moved(m_run, mx);
                        rescale(moved(x_run, mv));
                        const float x0 = x_run == -INFINITY ? 0.0f : x_run;
                        // The sum of p: of P = p 2^(E + 7 - x), by eights, times 2^-E and
                        // 2^(x - 7 - m).  (Where V's scales reach so high that fp32 does not
                        // hold the P of keys with small ones, of p itself.)
                        const float up = x_run == -INFINITY ? 0.0f : ex2_approx(x_run - P_SHIFT - m_run);
                        const bool far = __any_sync(FULL_MASK, x_run - m_run > 11.0f);
                        float lt = 0.0f;
#pragma unroll 1
                        for (int h0 = TILE - HW; h0 >= 0; h0 -= HW) {
                            float kf[8], ve[8];
                            eight(kf, h0 / 8);
                            eight(ve, 16 + h0 / 8);
                            if (h0 < TILE - HW) {          // (the last half is there)
                                tmem_ld_begin<HW>(t_s + h0, v);
                                tmem_ld_end<HW>(v);
                                hide(v, h0);
                            }
                            if (far) {
                                const float m0 = m_run == -INFINITY ? 0.0f : m_run;
#pragma unroll
                                for (int j = 0; j < HW; ++j)
                                    l_run += ex2_approx(fmaf(v[j], factor(kf[j / 8]), -m0));
                            }
                            constexpr int E = HW / 8;
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < E + 2; ++i) {      // (steps as above)
                                if (i < E) {
                                    const float f = factor(kf[i]);
                                    const float off = ve[i] + (P_SHIFT - x0);
#pragma unroll
                                    for (int j = 8 * i; j < 8 * i + 8; j += 2)
                                        fma2_bc(v[j], v[j + 1], f, off);
                                }
                                if (i >= 1 && i <= E)
#pragma unroll
                                    for (int j = 8 * i - 8; j < 8 * i; ++j)
                                        v[j] = ex2_approx(v[j]);
                                if (i >= 2) {
                                    float *y = v + 8 * i - 16;
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        w[(i & 1) * 4 + j] = pack2<PT>(y[2 * j], y[2 * j + 1]);
                                    add2(y[0], y[1], y[2], y[3]);
                                    add2(y[4], y[5], y[6], y[7]);
                                    add2(y[0], y[1], y[4], y[5]);
                                    lt = fmaf(y[0] + y[1], fac[32 + h0 / 8 + i - 2], lt);
                                    if (i & 1)
                                        tmem_st8(t_s + h0 + (i - 2) / 2 * 8, w);
                                }
                            }
                        }
                        if (!far)
                            l_run = fmaf(lt, up, l_run);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[g]);
            }
            gt += c.t1 - c.t0;
            // ---- the piece's end
            c = pieces[item % C::PIECES];          // (read again: not kept through the tiles)
            const int nt1 = both ? group_tiles(p, c, 1) : 0;
            if (nt > 0 && !phase(&o_done[g], P_O))
                goto softmax_done;
            // O to units of p: over an 8-bit cache it holds P's, and V_SHIFT below
            float a0 = !F8 ? 1.0f : x_run == -INFINITY ? 0.0f
                                  : ex2_approx(x_run - m_run - (P_SHIFT + V_SHIFT)), a1 = 0.0f;
            if (g == 1 && both) {
                // hand the state over: the first group reads it and this group's O
                if (nt > 0) {
                    if ((ph & LENT) && !__all_sync(FULL_MASK, wait(ml_free, (ph & P_ML) ? 0u : 1u)))
                        goto softmax_done;
                    ml[r] = l_run;
                    ml[TILE_M + r] = m_run;
                    if (F8)
                        ml[2 * TILE_M + r] = a0;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(ml_full);
                    ph = (ph ^ P_ML) | LENT;
                }
                done(item);
                continue;
            }
            if (g == 0 && !both)
                ph ^= P_O1;                        // (the second group waits for its own)
            if (nt1 > 0) {
                if (!phase(&o_done[1], P_O1) || !phase(ml_full, P_ML))
                    goto softmax_done;
                const float l1 = ml[r], n1 = ml[TILE_M + r], b1 = F8 ? ml[2 * TILE_M + r] : 1.0f;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(ml_free);
                const float m = fmaxf(m_run, n1);
                const float w0 = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m);
                const float w1 = n1 == -INFINITY ? 0.0f : ex2_approx(n1 - m);
                a0 *= w0;
                a1 = b1 * w1;
                m_run = m;
                l_run = l_run * w0 + l1 * w1;
            }
            tc_fence_after();
            if (warp_live) {
                if (c.kind == 0) {
                    const float inv = l_run == 0.0f ? 0.0f : (F8 ? (float)(1 << V_SHIFT) : 1.0f) / l_run;
                    a0 *= inv;
                    a1 *= inv;
                }
                T *out = static_cast<T *>(p.out) +
                         ((int64_t)(c.tok + (row >> p.lg_g)) * p.num_q_heads +
                          (c.h << p.lg_g) + (row & ((1 << p.lg_g) - 1))) * D;
                // a state: of each four columns all rows' side by side, then maxima and sums
                float *states = p.part + ((int64_t)blockIdx.x * 2 + (c.kind == 2)) * C::ROWS * (D + 2);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float o[32];
                    if (nt > 0) {
                        tmem_ld32(t_o + c0, o);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] *= a0;
                    }
                    if (nt1 > 0) {
                        float o1[32];
                        tmem_ld32(t_o + C::GROUP_COLS + c0, o1);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = fmaf(o1[j], a1, o[j]);
                    }
                    if (!valid || (c.kind && nt == 0)) {
                        // (padding rows, and a half that sees none of the piece's keys: its
                        // sum of 0 says so)
                    } else if (c.kind == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4 *>(out + c0 + 8 * j) = make_uint4(
                                pack2<T>(o[8 * j], o[8 * j + 1]), pack2<T>(o[8 * j + 2], o[8 * j + 3]),
                                pack2<T>(o[8 * j + 4], o[8 * j + 5]), pack2<T>(o[8 * j + 6], o[8 * j + 7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(states + ((c0 / 4 + j) * C::ROWS + row) * 4) =
                                make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
                if (c.kind && valid)
                    *reinterpret_cast<float2 *>(states + C::ROWS * D + 2 * row) = make_float2(m_run, l_run);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (nt > 0)
                    mbar_arrive(&o_free[g]);
                if (nt1 > 0)
                    mbar_arrive(&o_free[1]);
            }
            done(item);
        }
    softmax_done:;
    } else if (!F8 && warp < W0 + 2) {
        // ================= K or V tiles of a 16-bit cache
        const bool is_k = warp == W0;
        unsigned char *ring = is_k ? sK : sV;
        uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
        const CUtensorMap *tm = is_k ? &p.tm_k : &p.tm_v;
        const T *cache = static_cast<const T *>(is_k ? p.k_cache : p.v_cache);
        const int R = p.box_rows, nbox = TILE / R;
        const int oob = p.num_blocks * p.num_kv_heads;     // a block past the end: zeros
        constexpr int DCH = D / 8;
        uint32_t gt = 0;
        bool ok = true;
        for (uint32_t item = 0; ok && take(item); ++item) {
            const int32_t *table = p.tables + (int64_t)c.b * p.max_blocks;
            // lane j: rows [j R, j R + R) of a tile, from one block; ids a tile ahead
            auto block_of = [&](int t) -> int32_t {
                const int pos0 = t * TILE + lane * R;
                return lane < nbox && t < c.t1 && pos0 <= c.last && pos0 + R > c.sight
                           ? table[pos0 >> p.bs_log2] : -2;
            };
            int32_t ahead = block_of(c.t0);
            for (int t = c.t0; t < c.t1; ++t, ++gt) {
                const int slot = gt % NS;
                const int pos0 = t * TILE + lane * R;
                const int32_t blk = ahead;
                ahead = block_of(t + 1);
                if (!(ok = __all_sync(FULL_MASK, gt < NS || wait(&empty[slot], gt / NS + 1))))
                    break;
                const bool inbox = lane < nbox;
                int z = oob;
                if (inbox && blk != -2) {
                    if (blk < 0 || blk >= p.num_blocks)
                        atomicOr(p.err, PKV_EBIT_BLOCK);
                    else
                        z = blk * p.num_kv_heads + c.h;
                }
                const int y = pos0 & (p.block_size - 1);
                unsigned char *dst = ring + slot * C::KV_BYTES;
                // By a tensor copy where the box is of whole groups of eight rows and
                // holds no row past the last in sight (those are zeros: P is 0 there, but 0
                // times a stale NaN is not); by 16-byte copies otherwise.
                const bool by_tma = inbox && R >= 8 && (z == oob || pos0 + R - 1 <= c.last);
                const unsigned tma_boxes = __popc(__ballot_sync(FULL_MASK, by_tma));
                const unsigned cp_boxes = __ballot_sync(FULL_MASK, inbox && !by_tma);
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[slot], tma_boxes * (uint32_t)R * 2u * D);
                __syncwarp();
                if (by_tma)
                    tma_load_5d(dst + lane * R * 2 * D, tm, y >> 3, z, &full[slot]);
                if (cp_boxes) {
                    for (unsigned m = cp_boxes; m; m &= m - 1) {
                        const int bx = __ffs(m) - 1;
                        const int zb = __shfl_sync(FULL_MASK, z, bx);
                        const int yb = __shfl_sync(FULL_MASK, y, bx);
                        for (int idx = lane; idx < R * DCH; idx += 32) {
                            const int rr = bx * R + idx / DCH, ch = idx % DCH;
                            const bool in = zb != oob && t * TILE + rr <= c.last;
                            const int64_t row = in ? (int64_t)zb * p.block_size + yb + idx / DCH : 0;
                            cp_async16(dst + tile_off<D>(rr, ch), cache + row * D + ch * 8, in);
                        }
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[slot]);
            }
            done(item);
        }
        if (is_k && lane == 0)
            note_item(p, begin, line);
    } else if (F8 && warp < W0 + 4) {
        // ================= bring and convert tiles of an 8-bit cache: codes to fp16, this
        // warp's 32 rows.  The codes come through registers, asked for when the tile before
        // (V before the next K, K before V) has been converted: through shared memory they
        // would take as much of its bandwidth again as the converted tiles' writing does, and
        // room for a slot of each.  K and V take turns in one copy of the code: with one for each,
        // whose loads had twice as long, pieces of prompts took 914 us rather than 880.
        const int w0 = (warp - W0) * 32, H = p.num_kv_heads;
        constexpr int LPR = D / 16, RPI = 32 / LPR, NI = 32 / RPI;  // lanes a row, rows at once
        const int rr = lane / LPR, j = lane % LPR;
        const unsigned char *kc = static_cast<const unsigned char *>(p.k_cache);
        const unsigned char *vc = static_cast<const unsigned char *>(p.v_cache);
        uint32_t gt = 0;
        bool ok = true;
        for (uint32_t item = 0; ok && take(item); ++item) {
            const int32_t *table = p.tables + (int64_t)c.b * p.max_blocks;
            // lane q < 4: the block of rows w0 + 8 q .. w0 + 8 q + 7 of a tile (-2: none in sight)
            auto block_of = [&](int t) -> int32_t {
                const int pos0 = t * TILE + w0 + 8 * (lane & 3);
                const int first = pos0 & ~(p.block_size - 1);
                return t < c.t1 && pos0 <= c.last && first + p.block_size > c.sight
                           ? table[pos0 >> p.bs_log2] : -2;
            };
            auto good = [&](int32_t blk) { return blk >= 0 && blk < p.num_blocks; };
            // Where a tile's rows are (a row's 16 bytes of this lane, by groups of eight rows),
            // and which of them count: the others, of no block or behind the last key, come
            // from block 0 and become zeros (a load under a condition would be waited for
            // where the condition ends).
            int64_t at[4];
            auto find = [&](int t, int32_t ids) -> uint32_t {
                uint32_t count = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int32_t blk = __shfl_sync(FULL_MASK, ids, q);
                    const int pos = t * TILE + w0 + 8 * q + rr;
                    const bool in = good(blk);
                    at[q] = (((int64_t)(in ? blk : 0) * H + c.h) * p.block_size +
                             (pos & (p.block_size - 1))) * D + j * 16;
                    // (the rows of group q: pos, and with four lanes' rows at once pos + 4)
#pragma unroll
                    for (int u = 0; u < NI / 4; ++u)
                        count |= in && pos + 4 * u <= c.last ? 1u << (q * (NI / 4) + u) : 0u;
                }
                return count;
            };
            uint4 d[NI];
            auto bring = [&](const unsigned char *cache) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    d[i] = *reinterpret_cast<const uint4 *>(cache + at[i / (NI / 4)] +
                                                            i % (NI / 4) * 4 * D);
            };
            int32_t ids = block_of(c.t0), ids1 = block_of(c.t0 + 1);
            uint32_t count = find(c.t0, ids);
            bring(kc);
            // K and V in turn: one copy of the code
#pragma unroll 1
            for (int u = 2 * c.t0; u < 2 * c.t1; ++u) {
                const bool is_v = u & 1;
                const int slot = gt % NS;
                if (!(ok = __all_sync(FULL_MASK, gt < NS || wait((is_v ? v_empty : k_empty) + slot, gt / NS + 1))))
                    break;
                unsigned char *dst = (is_v ? sV : sK) + slot * C::KV_BYTES;
                if (!__all_sync(FULL_MASK, count == (1u << NI) - 1u)) {
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        if (!((count >> i) & 1))
                            d[i] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    uint4 lo, hi;
                    codes_to_half(d[i], lo, hi);
                    put_chunks<D>(dst, w0 + i * RPI + rr, j, lo, hi);
                }
                if (is_v) {
                    ids = ids1;
                    ids1 = block_of((u >> 1) + 2);
                    count = find((u >> 1) + 1, ids);
                    ++gt;
                }
                bring(is_v ? kc : vc);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive((is_v ? v_full : k_full) + slot);
            }
            done(item);
        }
        if (warp == W0 && lane == 0)
            note_item(p, begin, line);
    } else if (F8 && warp == C::W_SCALES) {
        // ================= a tile's scales, lane l those of its rows 8 l .. 8 l + 7: loaded
        // before the tile's slot is free.  (By the warps that convert, between their own
        // loads, pieces took 901 us rather than 879, and 32 tokens over 131000 rows 145 rather than 140.)
        const int H = p.num_kv_heads;
        uint32_t gt = 0;
        bool ok = true;
        for (uint32_t item = 0; ok && take(item); ++item) {
            const int32_t *table = p.tables + (int64_t)c.b * p.max_blocks;
            for (int t = c.t0; t < c.t1; ++t, ++gt) {
                const int pos0 = t * TILE + 8 * (lane & 15);
                const int first = pos0 & ~(p.block_size - 1);
                const bool in = pos0 <= c.last && first + p.block_size > c.sight;
                const int32_t blk = in ? table[pos0 >> p.bs_log2] : 0;
                const bool good = blk >= 0 && blk < p.num_blocks;
                const int64_t at = (int64_t)(good ? blk : 0) * H + c.h;
                const float kf = pow2_f32(block_exponent(p.k_scales[at]));
                const int ve = block_exponent(p.v_scales[at]);
                if (!good)
                    atomicOr(p.err, PKV_EBIT_BLOCK);
                if (!(ok = __all_sync(FULL_MASK, gt < NS || wait(&k_empty[gt % NS], gt / NS + 1))))
                    break;
                float *sc = k_sc + (gt & (C::RING - 1)) * C::FAC + (lane & 15);
                sc[0] = kf;
                sc[16] = (float)ve;
                sc[32] = pow2_f32(-ve);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&k_full[gt % NS]);
            }
            done(item);
        }
    } else if (warp == C::W_FEED) {
        // ================= hand out the share's pieces, one ahead of the one whose q is
        // brought (once the last S before has read its own)
        auto seq = [&](int b, Seq &q, int &q0) {
            bool bad;
            return lengths(p, b, q, q0, bad);
        };
        Walk walk;
        walk.start(p.batch, places, seq);
        __syncwarp();                              // (places lie where the pieces go)
        // A wait for the end of a piece: as long as its tiles take (1 to 4 us each), so its limit
        // grows with the tiles handed out.  Should another role hang, that role's own limit
        // ends this wait too.
        int64_t tiles = 0;
        auto wait_piece = [&](uint64_t *bar, uint32_t parity) -> bool {
            const bool ok = mbar_wait_bounded(bar, parity & 1, abort_flag,
                                              WAIT_LIMIT_NS + (uint64_t)tiles * TILE_LIMIT_NS);
            if (!ok)
                *abort_flag = 1;
            return __all_sync(FULL_MASK, ok);
        };
        auto hand_out = [&](uint32_t item, bool more) -> bool {
            const uint32_t slot = item % C::PIECES;
            if (item >= C::PIECES && !wait_piece(&pc_empty[slot], item / C::PIECES + 1))
                return false;
            if (more)
                tiles += c.t1 - c.t0;
            else
                c.kind = -1;
            if (lane == 0) {
                pieces[slot] = c;
                mbar_arrive(&pc_full[slot]);
            }
            return true;
        };
        bool more = walk.next(p.rules, p.batch, p.num_kv_heads, p.lg_g, c, seq), ok = hand_out(0, more);
        for (uint32_t item = 0; ok && more; ++item) {
            const int halves = shared_rows(c) ? 1 : 2, y = c.h << p.lg_g, z = c.tok;
            more = walk.next(p.rules, p.batch, p.num_kv_heads, p.lg_g, c, seq);
            if (!(ok = hand_out(item + 1, more)))
                break;
            if (item > 0 && !(ok = wait_piece(q_empty, item - 1)))
                break;
            if (lane == 0) {
                uint64_t *bar = C::QCONV ? q_raw : q_full;
                mbar_arrive_expect_tx(bar, halves * (uint32_t)C::Q_BYTES);
                for (int hh = 0; hh < halves; ++hh)
                    for (int pn = 0; pn < D / 64; ++pn)
                        tma_load_3d(sQ + hh * C::Q_BYTES + pn * (TILE_M * 128), &p.tm_q, pn * 64, y,
                                    z + hh * (TILE_M >> p.lg_g), bar);
            }
            __syncwarp();
        }
    } else if (warp == C::W_MMA) {
        // ================= MMA issue: the warp walks as one, an elected lane issues
        // S = Q K^T, both K-major, and O += P V, P in tensor memory, V MN-major; all of them
        // 128-byte swizzled panels of 64 channels: a row every 128 bytes, eight rows 1024
        // bytes.  q's next panel is 128 rows on; K's and V's lies beside the first, and the next
        // eight rows behind both.  A step of 16 along the contraction is 32 bytes into S's
        // rows, 16 rows of V.
        constexpr uint32_t Q_PANEL = TILE_M * 128;
        const uint32_t idesc_s = umma_idesc(C::PBF ? 1u : 0u, 0u, TILE);
        const uint32_t idesc_o = umma_idesc(C::PBF ? 1u : 0u, 1u, D);
        // (an allocation of all of tensor memory starts at its first column)
        constexpr uint32_t tm = 0;
        const uint32_t el = elect_lane();
        const uint64_t dq = umma_desc_sw128(smem_addr(sQ), 16, 1024);
        const uint64_t dk = umma_desc_sw128(smem_addr(sK), 16, C::GROUP8);
        const uint64_t dv = umma_desc_sw128(smem_addr(sV), 1024, C::GROUP8);
        const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
        const uint32_t q_hi = (uint32_t)(dq >> 32), k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
        // per group, a bit each: the parity of p_full's and o_free's next phase, and whether O
        // holds an earlier piece's
        uint32_t gt = 0, p_par = 0, of_par = 0, used = 0, k_seen = 0, v_seen = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(FULL_MASK, wait(bar, parity));
        };
        for (uint32_t item = 0; ok && take(item); ++item) {
            // (shuffled, so that what follows from them is known to be the warp's and is worked
            // out in uniform registers)
            const bool both = __shfl_sync(FULL_MASK, (int)shared_rows(c), 0) != 0;
            const int nt0 = __shfl_sync(FULL_MASK, group_tiles(p, c, 0), 0);
            const int nt1 = __shfl_sync(FULL_MASK, group_tiles(p, c, 1), 0);
            const int tiles = __shfl_sync(FULL_MASK, c.t1 - c.t0, 0);
            int s_left = nt0 + nt1;
            if (!(ok = wait_all(q_full, item)))
                break;
            // Step s of a group: O += P V of its tile s, and S of its tile s + 1, whose K is
            // waited for first: once P is there, nothing but the MMAs is left to do.  One
            // copy of the code for both groups and the first S: the instruction cache is
            // what roles that run long straight code at the same time contend for.
#pragma unroll 1
            for (int i = -2; i < 2 * max(nt0, nt1) && ok; ++i) {
                const int g = i & 1, s = i >> 1, nt = g ? nt1 : nt0;
                if (s >= nt)
                    continue;
                const bool more = s + 1 < nt;
                const uint32_t k = gt + (both ? 2 * s + g : s), slot = k % NS;
                const uint32_t k1 = k + (both ? 2 : 1), slot1 = k1 % NS;
                // (a tile that both groups read is waited for once)
                if (s >= 0 && (int)(k - v_seen) >= 0) {
                    if (!(ok = wait_all(&v_full[slot], k / NS)))
                        break;
                    v_seen = k + 1;
                }
                if (more && (int)(k1 - k_seen) >= 0) {
                    if (!(ok = wait_all(&k_full[slot1], k1 / NS)))
                        break;
                    k_seen = k1 + 1;
                }
                const uint32_t base = tm + g * C::GROUP_COLS;
                if (s >= 0) {
                    if (s == 0) {
                        // the softmax threads have read an earlier piece's O out
                        if ((used >> g) & 1) {
                            if (!(ok = wait_all(&o_free[g], (of_par >> g) & 1)))
                                break;
                            of_par ^= 1u << g;
                        }
                        used |= 1u << g;
                    }
                    if (!(ok = wait_all(&p_full[g], (p_par >> g) & 1)))
                        break;
                    p_par ^= 1u << g;
                    tc_fence_after();
                    const uint32_t vb = v_lo + slot * (C::KV_BYTES / 16);
#pragma unroll
                    for (int ks = 0; ks < TILE / 16; ++ks) {
                        const uint32_t pa = base + ks / 4 * 64 + ks % 4 * 8;
                        umma_f16_ta_elected(el, base + TILE, pa, vb + ks * (C::GROUP8 / 8), v_hi,
                                            idesc_o, s > 0 || ks > 0 ? 1u : 0u);
                    }
                    if (both || g == 1)            // the tile's last reader
                        umma_commit_elected(el, &v_empty[slot]);
                    if (!more)
                        umma_commit_elected(el, &o_done[g]);
                }
                if (more) {
                    tc_fence_after();
                    const uint32_t kb = k_lo + slot1 * (C::KV_BYTES / 16);
                    const uint32_t qb = q_lo + (both ? 0 : g) * (C::Q_BYTES / 16);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_f16_elected(el, base, qb + (ks / 4) * (Q_PANEL / 16) + (ks % 4) * 2, q_hi,
                                         kb + (ks / 4) * (1024 / 16) + (ks % 4) * 2, k_hi, idesc_s,
                                         ks > 0 ? 1u : 0u);
                    umma_commit_elected(el, &s_full[g]);
                    if (both || g == 1)
                        umma_commit_elected(el, &k_empty[slot1]);
                    if (--s_left == 0)
                        umma_commit_elected(el, q_empty);
                }
            }
            gt += tiles;
            done(item);
        }
        // every issued MMA has finished before tensor memory is released
        umma_commit_elected(el, drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0u) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (tid == 0)
            atomicOr(p.err, PKV_EBIT_TIMEOUT);
        // copies in flight land before the shared memory is another CTA's
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) {
        }
    }
    if (warp == C::W_MMA) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
    }
}

// Items that were cut: the states of an item's pieces joined in the order of the keys, eight
// columns of 32 rows a warp, a lane a row.  Warps count off the shares that an item to join is
// noted with, so that those without cost a look at a word each, and take their units in turn.
// Bound by latency: 6 us of a call with its launch where the states are 128 rows, 14 where they
// are 256 (two states a CTA then: 40 MB written and read, mostly in L2).
template <int D, typename T>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p,
                                                         int item_rows, int row_blocks, float v_scale)
{
    grid_dependency_wait();
    grid_dependents_launch();
    const int n = p.places[0], lane = threadIdx.x & 31;
    const int warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
    const int64_t state = (int64_t)item_rows * (D + 2);
    constexpr int CG = D / 8;                              // groups of eight columns
    const int per = row_blocks * CG;                       // units of an item
    int u = warp;                                          // this warp's next unit, from here on
    for (int s0 = 0; s0 < n; s0 += 32) {
        const int mine = s0 + lane < n ? p.places[8 + s0 + lane] : 0;
        const unsigned some = __ballot_sync(FULL_MASK, mine > 0);
        const int units = __popc(some) * per;
        for (; u < units; u += warps) {
            const int k = u / per, v = u - k * per;
            const int row = v / CG * 32 + lane, col = v % CG;
            // the k-th share's lane
            const int src = __ffs(__ballot_sync(FULL_MASK, mine > 0 && __popc(some & ((1u << lane) - 1)) == k)) - 1;
            const int pieces = __shfl_sync(FULL_MASK, mine, src), c = s0 + src;
            const int4 item = reinterpret_cast<const int4 *>(p.places + p.items_at)[c];
            if (row >= item.y)
                continue;                                  // (no exchange from here on)
            // piece i: the last state of share c - 1, then the first ones of c, c + 1, ..
            const float *start = p.part + (2 * (int64_t)(c - 1) + 1) * state;
            auto piece = [&](int i) -> const float * {
                return i == 0 ? start : start + (2 * (int64_t)i - 1) * state;
            };
            float m = -INFINITY, l = 0.0f, acc[8] = {};
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) {
                const float2 ml = *reinterpret_cast<const float2 *>(piece(i) + item_rows * D + 2 * row);
                m = ml.y != 0.0f ? fmaxf(m, ml.x) : m;
            }
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) {
                const float *s = piece(i);
                const float2 ml = *reinterpret_cast<const float2 *>(s + item_rows * D + 2 * row);
                const float4 o0 = *reinterpret_cast<const float4 *>(s + (2 * col * item_rows + row) * 4);
                const float4 o1 = *reinterpret_cast<const float4 *>(s + ((2 * col + 1) * item_rows + row) * 4);
                // (a piece that has none of the row's keys in sight may have written no O)
                const bool none = ml.y == 0.0f;
                const float w = none || ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
                l = fmaf(w, ml.y, l);
                const float x[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    acc[d] = none ? acc[d] : fmaf(w, x[d], acc[d]);
            }
            const float inv = l == 0.0f ? 0.0f : v_scale / l;
            T *out = static_cast<T *>(p.out) +
                     ((int64_t)(item.x + (row >> p.lg_g)) * p.num_q_heads + (item.z << p.lg_g) +
                      (row & ((1 << p.lg_g) - 1))) * D + 8 * col;
            *reinterpret_cast<uint4 *>(out) =
                make_uint4(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv),
                           pack2<T>(acc[4] * inv, acc[5] * inv), pack2<T>(acc[6] * inv, acc[7] * inv));
        }
        u -= units;
    }
}

// q [T][Hq][D] as the tensor {D, Hq, T}, boxes of 64 x G x 128 / G: a half's rows.
bool encode_q_map(CUtensorMap *m, const pkv_pool *pool, const void *q, int num_q_heads,
                  int num_tokens, int G, bool bf)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint64_t D = pool->head_dim;
    const cuuint64_t dims[3] = {D, (cuuint64_t)num_q_heads, (cuuint64_t)num_tokens};
    const cuuint64_t strides[2] = {D * 2, D * 2 * (cuuint64_t)num_q_heads};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(TILE_M / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void *>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache [NB][Hkv][bs][D] of 16-bit elements as the tensor {64, 8, D / 64, bs / 8, NB * Hkv}:
// columns of a panel, rows of a group of eight, panels, groups, (block, KV head)s; boxes of
// up to 128 rows.  (Blocks of 4 rows have no group and no map.)
bool encode_tile_map(CUtensorMap *m, const pkv_pool *pool, const void *base, bool bf)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint64_t D = pool->head_dim, groups = pool->block_size / 8;
    const cuuint64_t dims[5] = {64, 8, D / 64, groups,
                                (cuuint64_t)pool->num_blocks * pool->num_kv_heads};
    const cuuint64_t strides[4] = {D * 2, 128, D * 16, (cuuint64_t)pool->block_size * D * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)(D / 64),
                               (cuuint32_t)std::min<cuuint64_t>(groups, TILE / 8), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F8, bool BF, int NQ>
int launch_chunk_t(const pkv_pool *pool, const ChunkParams &p, cudaStream_t s)
{
    using C = Cfg<D, F8, BF, NQ>;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    // set per call (for the current device, from any host thread)
    if (cudaFuncSetAttribute(chunk_kernel<D, F8, BF, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_BYTES) != cudaSuccess)
        return PKV_ERR_CUDA;
    const int sms = pool->num_sms;
    if (sms < 1)
        return PKV_ERR_CUDA;
    if (launch_pdl(chunk_kernel<D, F8, BF, NQ>, dim3((unsigned)sms), dim3(C::NT),
                   (size_t)C::SMEM_BYTES, s, p) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (sms > 1 && launch_pdl(chunk_join_kernel<D, T>, dim3((unsigned)(4 * sms)), dim3(256),
                              0, s, p, (int)C::ROWS,
                              (int)((std::min<int64_t>(C::ROWS, (int64_t)p.max_q_len << p.lg_g) + 31) / 32), F8 ? (float)(1 << V_SHIFT) : 1.0f) != cudaSuccess)
        return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// Rows of an item: 128 where every sequence's rows fit (its keys are then read by both
// softmax groups in turn), else 256.
int item_rows(int max_q_len, int G) { return (int64_t)max_q_len * G <= TILE_M ? TILE_M : 2 * TILE_M; }

int items_at(const pkv_pool *pool) { return (8 + std::max(1, pool->num_sms) + 3) / 4 * 4; }

size_t places_bytes(const pkv_pool *pool)
{
    // a word a share, and 16 bytes
    return ((size_t)items_at(pool) * 4 + (size_t)16 * std::max(1, pool->num_sms) + 255) / 256 * 256;
}

}  // namespace

size_t chunk_workspace_bytes(const pkv_pool *pool, int num_q_heads, int max_q_len)
{
    const int G = num_q_heads / pool->num_kv_heads;
    return places_bytes(pool) + (size_t)2 * std::max(1, pool->num_sms) * item_rows(max_q_len, G) *
                                    (pool->head_dim + 2) * sizeof(float);
}

int launch_chunk(const pkv_pool *pool, const void *q, pkv_dtype q_dtype, int num_q_heads,
                 int num_tokens, const void *k_cache, const void *v_cache, const void *k_scales,
                 const void *v_scales, const int32_t *tables, int max_blocks,
                 const int32_t *q_start, const int32_t *seq_lens, int batch, int max_q_len,
                 int window, const uint64_t *visible, float scale, void *out, void *workspace,
                 pkv_stream_t stream)
{
    ChunkParams p{};
    const int G = num_q_heads / pool->num_kv_heads;
    const bool f8 = pool->kv_dtype == PKV_F8, bf = q_dtype == PKV_BF16;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scales = static_cast<const float *>(k_scales);
    p.v_scales = static_cast<const float *>(v_scales);
    p.tables = tables;
    p.q_start = q_start;
    p.seq_lens = seq_lens;
    p.visible = visible;
    p.out = out;
    p.places = static_cast<int32_t *>(workspace);
    p.items_at = items_at(pool);
    p.share_step = chunk::share_step(std::max(1, pool->num_sms));
    p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + places_bytes(pool));
    p.err = pool->d_err;
    p.batch = batch;
    p.num_tokens = num_tokens;
    p.max_q_len = max_q_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = pool->num_kv_heads;
    p.lg_g = log2_of(G);
    p.block_size = pool->block_size;
    p.bs_log2 = log2_of(pool->block_size);
    p.max_blocks = max_blocks;
    p.num_blocks = pool->num_blocks;
    p.box_rows = std::min(pool->block_size, TILE);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const int rows = item_rows(max_q_len, G);
    p.rules.lg_tpr = log2_of(rows / G);
    p.rules.window = window;
    p.rules.tree = visible != nullptr;
    if (!encode_q_map(&p.tm_q, pool, q, num_q_heads, num_tokens, G, bf))
        return PKV_ERR_CUDA;
    if (!f8 && pool->block_size >= 8 && (!encode_tile_map(&p.tm_k, pool, k_cache, bf) ||
                                         !encode_tile_map(&p.tm_v, pool, v_cache, bf)))
        return PKV_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PKV_CHUNK(D, F)                                                                          \
    (bf ? (rows == TILE_M ? launch_chunk_t<D, F, true, 1>(pool, p, s)                            \
                          : launch_chunk_t<D, F, true, 2>(pool, p, s))                           \
        : (rows == TILE_M ? launch_chunk_t<D, F, false, 1>(pool, p, s)                           \
                          : launch_chunk_t<D, F, false, 2>(pool, p, s)))
    if (pool->head_dim == 128)
        return f8 ? PKV_CHUNK(128, true) : PKV_CHUNK(128, false);
    return f8 ? PKV_CHUNK(64, true) : PKV_CHUNK(64, false);
#undef PKV_CHUNK
}

}  // namespace pkv
