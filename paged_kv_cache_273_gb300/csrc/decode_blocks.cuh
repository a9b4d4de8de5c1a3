// Decode attention with a copy ring for every warp: over 8-bit float caches
// (PKV_F8, one scale a (block, KV head)), and over lists of chosen blocks
// (paged_decode_attention_sparse) of 8-bit float and 16-bit caches.
//
// What it computes ("KV cache: the engine behind fast LLM inference",
// "Concept"): out = softmax(scale * q . K^T) . V for each sequence and query
// head, the G query heads of a KV head together.
//
// How:
//  * The work is one list of 16-token tiles, ordered by (sequence, KV head,
//    tile).  CTA c of P takes the tiles [c T / P, (c + 1) T / P), or, of
//    sequences about as long as one another, whole (sequence, KV head)s; its
//    warps take equal parts of those: every warp streams a contiguous run of tiles
//    through a ring of its own (cp.async, completion counted per thread), so
//    no warp waits for another and nothing waits on a flag or barrier until
//    the CTA's end.
//  * A warp keeps the online softmax state of its current (sequence, KV
//    head) in registers.  A piece that lies inside one warp's run is written
//    straight to the output.  At most two pieces of a run are shared with
//    neighbours; their states go to shared memory, the CTA joins the states
//    of its warps at its end, and a piece shared with other CTAs is left in
//    the workspace and joined, in CTA order, by the last of them to finish
//    (the result does not depend on timing).  A state that is handed on holds
//    2^-24 of its weighted sum, which is in range for any V over 2^24 rows, where
//    the sum itself is not; what that takes from the small end is below 2^-125.
//  * Tile math: warp-level MMAs as in the kernel for the other caches; e4m3
//    codes become fp16 exactly, q becomes fp16 exactly (a bf16 q is brought
//    to [2^14, 2^15) by a power of two first), products are exact and sums
//    fp32.  With x a row's score * log2(e) and m a whole number at or above the
//    largest x so far, a row's weight is p = 2^(x - m) <= 1; the denominator
//    sums p, the numerator p times the row of V, as an MMA for each tile whose
//    sum is added to the running one in fp32.
//  * Weights are split into two fp16 or three bf16 parts.  fp16 parts are taken
//    of 2^15 p: at 1 both parts of a small weight would lie on the one grid of
//    fp16's subnormal numbers (2^-24), and rows 17 nats below a sequence's
//    largest would weigh up to half as much again, or nothing.  At 2^15 the grid
//    leaves 2^-40 of the largest weight.
//  * A V scale 2^ev stays out of the weights: a tile's sum of p and codes is
//    multiplied by 2^(ev - r) as it joins the running sum, r the largest exponent
//    so far, so that blocks may be 2^126 apart.  A tile of two blocks (of 8 rows)
//    takes the larger of two scales up to 2^4 apart, the other block's weights
//    brought to it, and else is summed block by block.
//  * Every rescaling is by a power of two.
//  * Rows outside the attended range are filled with zeros by the copies, so
//    that whatever they hold (NaN codes of an earlier owner) is never read.
#pragma once

#include "blocks_common.cuh"
#include "decode_kernel.cuh"

namespace pkv {
namespace kern {

template <> struct KvBits<PKV_F8> { static constexpr int v = 8; };

}  // namespace kern

namespace blk {

using namespace dev;
using kern::round_up;

constexpr int TILE = 16;
constexpr int MAX_BATCH = 4096;
// Tiles a warp is given at least, where the batch has fewer than one share of
// that for every warp of the GPU.
constexpr int MIN_TILES = 2;
// Tiles a warp takes of a piece that is not worth joining across CTAs.
constexpr int SHORT_TILES = 8;

template <int D, int G, int KV>
struct Cfg {
    static constexpr bool F8 = KV == PKV_F8;
    static constexpr int ROWB = D * kern::KvBits<KV>::v / 8;
    static constexpr int CH = ROWB / 16;            // 16-byte chunks of a row
    static constexpr int RPI = 32 / CH;             // rows a warp copies at once
    static constexpr int NI = TILE / RPI;           // copies of a tile of K (or V)
    static constexpr int TILE_BYTES = TILE * ROWB;
    static constexpr int SC_BYTES = F8 ? 2 * TILE * 4 : 0;   // each row's K scale, then V scale
    static constexpr int STAGE = 2 * TILE_BYTES + SC_BYTES;
    // warps: a multiple of the SM's four partitions, as many as the registers
    // allow (8-bit rows of 128, 16 x 4096 tokens, 32 / 8 heads: 28.0 us with 12
    // warps, 29.0 with 11, 32.3 with 13)
    static constexpr int W = F8 ? (D == 64 ? 16 : 12) : 8;
    // two tiles of a piece computed together: where the registers allow it
    // beside as many warps (rows of 64: 33.8 instead of 34.5 us on 64
    // sequences of up to 2048 tokens, 12 heads; rows of 128 in pairs, with 8
    // warps for the registers, 30.0 instead of 28.0 us on the shape above)
    static constexpr bool PAIR = F8 && D == 64;
    static constexpr int NT = W * 32;
    static constexpr int STATE = G * (D + 2);       // floats of one softmax state
    // ring stages that fit beside the states and the tile prefix, at most 5 (e4m3
    // rows of 64, 64 sequences of up to 2048 tokens, 12 heads: 33.8 us with 5, 34.1
    // with 6, 34.6 with 4)
    static constexpr int FIXED = W * STATE * 4 + (MAX_BATCH + 1) * 4 + W * 6 * 16 + W * 16 + 256;
    static constexpr int FIT = (232448 - FIXED) / (W * STAGE);
    static constexpr int NST = FIT > 5 ? 5 : FIT;
    static_assert(NST >= (PAIR ? 3 : 2), "ring");
    static_assert(NST * STAGE >= STATE * 4, "a warp's last state takes its ring's place");
    static_assert(TILE_BYTES % 1024 == 0 || STAGE % 128 == 0, "swizzle period");
};

struct Params {
    const void *q;
    const unsigned char *k_cache;
    const unsigned char *v_cache;
    const float *k_scales;       // [NB][Hkv], 8-bit float caches
    const float *v_scales;
    // physical blocks: row b of [B][table_stride], or with per_head row
    // b * Hkv + kvh of a list of chosen blocks
    const int32_t *tables;
    const int32_t *seq_lens;
    float *out;
    float *partials;
    int *counters;
    unsigned int *err;
    int batch, num_q_heads, num_kv_heads;
    int block_size, bs_log2, num_blocks;
    int64_t table_stride;
    int len_cap;
    int window;
    int per_head;                // tables rows are lists of chosen blocks
    int budget;                  // per_head: entries of a list
    int q_dtype;
    int pieces_each;             // even split: (sequence, KV head)s a CTA, and the CTAs
    int whole_ctas;
    float scale_log2;
};

// Shared memory: the rings, the warps' first states, what the rings' tiles
// are, the tile prefix (and, for up to half the largest batch, the sequences'
// lengths), the states' pieces.
template <int D, int G, int KV>
struct Smem {
    using C = Cfg<D, G, KV>;
    static constexpr int RING = 0;
    static constexpr int STATES = C::W * C::NST * C::STAGE;
    static constexpr int INFO = round_up(STATES + C::W * C::STATE * 4, 16);
    static constexpr int TSTART = INFO + C::W * C::NST * 16;
    __host__ __device__ static bool has_lens(int batch) { return 2 * batch <= MAX_BATCH; }
    __host__ __device__ static int meta(int batch)
    {
        return round_up(TSTART + ((has_lens(batch) ? 2 : 1) * batch + 1) * 4, 16);
    }
    __host__ __device__ static int total(int batch)
    {
        return meta(batch) + (2 * C::W + 2 * C::W + 16) * 4;
    }
};

// Rows a sequence's length leaves to attend: the length itself, or the rows of
// the chosen blocks (all of them full but the newest, which comes last).
__device__ __forceinline__ int attended_len(const Params &p, int L)
{
    if (!p.per_head || L <= 0)
        return L;
    const int n = (L + p.block_size - 1) >> p.bs_log2;
    return L - ((n - min(n, p.budget)) << p.bs_log2);
}

__device__ __forceinline__ int first_row(const Params &p, int L)
{
    return p.window > 0 && L > p.window ? L - p.window : 0;
}

// A sequence's attended length, 0 for one out of range.
__device__ __forceinline__ int seq_len(const Params &p, int b)
{
    const int L = p.seq_lens[b];
    return L < 0 || L > p.len_cap ? 0 : attended_len(p, L);
}

__device__ __forceinline__ int num_tiles(int L, int lo)
{
    return L > lo ? (L + TILE - 1) / TILE - lo / TILE : 0;
}

__device__ __forceinline__ void cp16_zfill(void *dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp4_zfill(void *dst, const void *src, bool valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src),
                 "r"(valid ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

static __device__ __noinline__ int long_quotient(int x, int d) { return x / d; }

// x / d of non-negative ints; a fraction of an integer division's latency where
// both the quotient's distance to the next whole number, at least 1 / (2 d), and
// fp32's error in it, at most (x / d) 2^-22, leave no doubt: x < 2^20.
__device__ __forceinline__ int quotient(int x, int d)
{
    return x < (1 << 20) ? (int)__fdividef((float)x + 0.5f, (float)d) : long_quotient(x, d);
}

// A tile of the list: what a lane holds of each of the warp's next 32 tiles.
struct Tile {
    int id[4];           // block of each quarter of the rows (blocks of >= 16 rows: all in id[0])
    int b, kvh;
    int bits;            // rows in the sequence (1..16), first attended row << 5, first / last
                         // tile of the piece << 10 / 11, first row's place in its block << 12
};
constexpr int FIRST = 1 << 10, LAST = 1 << 11;

__device__ __forceinline__ int rows_of(int bits) { return bits & 31; }
__device__ __forceinline__ int skip_of(int bits) { return (bits >> 5) & 31; }
__device__ __forceinline__ bool is_full(int bits) { return (bits & 1023) == TILE; }

template <int D, int G, int KV>
__device__ __forceinline__ Tile tile_at(const Params &p, const int *tstart, int x)
{
    Tile t;
    t.b = kern::find_seq(tstart, p.batch, x);
    const int L = Smem<D, G, KV>::has_lens(p.batch) ? tstart[p.batch + 1 + t.b] : seq_len(p, t.b);
    const int lo = first_row(p, L);
    const int nt = num_tiles(L, lo);
    const int off = x - tstart[t.b];
    t.kvh = quotient(off, nt);
    const int i = off - t.kvh * nt;
    const int t0 = TILE * (lo / TILE + i);
    t.bits = min(TILE, L - t0) | max(0, lo - t0) << 5 | (i == 0 ? FIRST : 0) |
             (i + 1 == nt ? LAST : 0) | (t0 & (p.block_size - 1)) << 12;
    const int32_t *row =
        p.tables + (p.per_head ? (int64_t)t.b * p.num_kv_heads + t.kvh : (int64_t)t.b) *
                       p.table_stride;
    // blocks that hold attended rows (no other entry is looked at)
    const int n = p.block_size >= TILE ? 1 : TILE >> p.bs_log2;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int r0 = u << p.bs_log2;
        t.id[u] = -1;
        if (u < n && (n == 1 || (r0 < rows_of(t.bits) &&
                                 r0 + p.block_size > skip_of(t.bits)))) {
            const int id = row[(t0 >> p.bs_log2) + u];
            if (id < 0 || id >= p.num_blocks)
                atomicOr(p.err, PKV_EBIT_BLOCK);
            else
                t.id[u] = id;
        }
    }
    return t;
}

// Copies of the tile that lane j describes into a stage, one commit group.
template <int D, int G, int KV>
__device__ __forceinline__ void issue_tile(const Params &p, const Tile &d, int j,
                                           unsigned char *stage, int4 *info, int lane)
{
    using C = Cfg<D, G, KV>;
    const int r0 = lane / C::CH, c = lane % C::CH;
    const int bits = __shfl_sync(FULL_MASK, d.bits, j), kvh = __shfl_sync(FULL_MASK, d.kvh, j);
    const int b = __shfl_sync(FULL_MASK, d.b, j), id0 = __shfl_sync(FULL_MASK, d.id[0], j);
    const int rows = rows_of(bits), skip = skip_of(bits), bs = p.block_size;
    if (lane == 0)
        *info = make_int4(bits, b, kvh, 0);
    // copy i goes 512 bytes behind copy i - 1, and the swizzle's row bits flip one
    // bit of the chunk from copy to copy
    const uint32_t dst0 = kern::swz_off(r0 * C::ROWB + c * 16, true);
    auto dst_of = [&](int i) { return (dst0 ^ ((i & 1) * 0x40u)) + i * 512u; };
    static_assert(C::RPI * C::ROWB == 512, "a warp's copy");
    if (bs >= TILE) {
        const int64_t head = (int64_t)max(id0, 0) * p.num_kv_heads + kvh;
        const int64_t base = (head * bs + (bits >> 12) + r0) * C::ROWB + c * 16;
        const unsigned char *k = p.k_cache + base, *v = p.v_cache + base;
        if (is_full(bits) && id0 >= 0) {
#pragma unroll
            for (int i = 0; i < C::NI; ++i) {
                cp_async_16b(stage + dst_of(i), k + i * 512);
                cp_async_16b(stage + C::TILE_BYTES + dst_of(i), v + i * 512);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < C::NI; ++i) {
                const int r = r0 + i * C::RPI;
                const bool in = id0 >= 0 && r < rows && r >= skip;
                cp16_zfill(stage + dst_of(i), k + i * 512, in);
                cp16_zfill(stage + C::TILE_BYTES + dst_of(i), v + i * 512, in);
            }
        }
        if constexpr (C::F8)
            cp4_zfill(stage + 2 * C::TILE_BYTES + lane * 4,
                      (lane < TILE ? p.k_scales : p.v_scales) + head, id0 >= 0);
    } else {
        const int id1 = __shfl_sync(FULL_MASK, d.id[1], j);
        const int id2 = __shfl_sync(FULL_MASK, d.id[2], j);
        const int id3 = __shfl_sync(FULL_MASK, d.id[3], j);
        auto head_of = [&](int r, bool &v) -> int64_t {
            const int u = r >> p.bs_log2;
            const int id = u == 0 ? id0 : u == 1 ? id1 : u == 2 ? id2 : id3;
            v = id >= 0 && r < rows && r >= skip;
            return (int64_t)max(id, 0) * p.num_kv_heads + kvh;
        };
#pragma unroll 1
        for (int i = 0; i < C::NI; ++i) {
            const int r = r0 + i * C::RPI;
            bool v;
            const int64_t head = head_of(r, v);
            const int64_t off = (head * bs + (r & (bs - 1))) * C::ROWB + c * 16;
            cp16_zfill(stage + dst_of(i), p.k_cache + off, v);
            cp16_zfill(stage + C::TILE_BYTES + dst_of(i), p.v_cache + off, v);
        }
        if constexpr (C::F8) {
            // (of a block with attended rows: all of its rows' entries)
            const int u = (lane & (TILE - 1)) >> p.bs_log2, id = u == 0 ? id0 : id1;
            const int64_t head = (int64_t)max(id, 0) * p.num_kv_heads + kvh;
            cp4_zfill(stage + 2 * C::TILE_BYTES + lane * 4,
                      (lane < TILE ? p.k_scales : p.v_scales) + head, id >= 0);
        }
    }
}

template <int D, int G, int KV>
struct State : kern::MmaState<D, G, KV, false> {
    int r;               // largest exponent of a V scale so far: acc's unit is 2^(r - 15)
};

// The lane's quarter of q's row for its head column (head gid mod G: the
// columns beyond G repeat the heads, as in the other kernel), raw.
template <int D, int G>
__device__ __forceinline__ void fetch_q(uint32_t (&w)[D / 8], const Params &p, int b, int kvh,
                                        int lane)
{
    const int gid = lane >> 2, tig = lane & 3;
    const uint4 *src = reinterpret_cast<const uint4 *>(
        static_cast<const uint16_t *>(p.q) +
        ((int64_t)b * p.num_q_heads + kvh * G + gid % G) * D + tig * (D / 4));
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const uint4 x = src[c];
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
    }
}

// What turns an MMA sum of the lane's two heads into a log2-domain score:
// * first, * the K scale, * second, in this order.  second (8-bit float caches) is
// the part of a bf16 q's power of two beyond 2^-60 or 2^60, 1 for most: a first
// product is then in range whatever q is, and the next one leaves it only where
// the score does.
template <int KV>
struct QScale {
    float first[2];
    float second[2];
};

// Raw q -> B fragments of the score MMAs, and those factors.
template <int D, int G, int KV>
__device__ __forceinline__ void use_q(State<D, G, KV> &st, QScale<KV> &qscale,
                                      uint32_t (&w)[D / 8], const Params &p, int lane)
{
    constexpr bool F8 = KV == PKV_F8;
    constexpr int NQ = D / 32;                       // 16-byte chunks of the lane's quarter row
    const int tig = lane & 3;
    float unscale = p.scale_log2, rest = 1.0f;
    if (F8 && p.q_dtype == PKV_BF16) {
        // fp16 has bf16's 8 significant bits but not its exponents: bring the
        // head's largest magnitude to [2^14, 2^15); values down to 2^-28 of it
        // stay exact
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ * 4; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
        amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(FULL_MASK, amax, 2));
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
        const float f = pow2_f32(14 - e);
#pragma unroll
        for (int i = 0; i < NQ * 4; ++i) {
            const __half2 h = __floats2half2_rn(bf16lo(w[i]) * f, bf16hi(w[i]) * f);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        const int near = min(max(e - 14, -60), 60);
        unscale = p.scale_log2 * pow2_f32(near);
        rest = pow2_f32(e - 14 - near);
    }
    // word 2 ks + h of the fragment order
    const int rot = kern::MmaCfg<D, KV>::ROTATE ? (tig >> 1) * 2 : 0;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (F8) {
                st.qh[ks][h] = w[2 * ks + h];
            } else {
                // chunk (ks / 2 + rot) mod chunks, word 2 (ks % 2) + h: rot is
                // 0 or 2, picked without indexing registers by a variable
                const int a = 4 * (ks >> 1) + 2 * (ks & 1) + h;
                const int bb = 4 * (((ks >> 1) + 2) & (kern::MmaCfg<D, KV>::KCH - 1)) +
                               2 * (ks & 1) + h;
                st.qh[ks][h] = rot ? w[bb] : w[a];
            }
        }
    // the heads of columns 2 tig, 2 tig + 1 (lane 4 n holds column n's head)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        qscale.first[r] = __shfl_sync(FULL_MASK, unscale, 8 * tig + 4 * r);
        if constexpr (F8)
            qscale.second[r] = __shfl_sync(FULL_MASK, rest, 8 * tig + 4 * r);
    }
}

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// The reference of a state that has seen no score above -inf, the least fp32
// number rather than -inf: such scores (products beyond fp32, infinite keys) then
// weigh 2^(-inf - m) = 0, not 2^(-inf + inf).
constexpr float NO_SCORE = -3.402823466e38f;

// 2^(m - top), the weight of a state in a join.
__device__ __forceinline__ float join_weight(float m, float top)
{
    return kern::exp2_approx(m - top);
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        x += __shfl_xor_sync(FULL_MASK, x, m);
    return x;
}

// Parts a weight is split into, each of the MMA's type: two of fp16 leave
// 2^-22 of it and 2^-25 whatever it is, three of bf16 2^-27 (two would leave
// 2^-18).  The largest weight is 2^weight_top_log2: 2^15 for fp16, whose largest
// number is 65504.
template <int KV>
__host__ __device__ constexpr int weight_parts() { return KV == PKV_BF16 ? 3 : 2; }
template <int KV>
__host__ __device__ constexpr int weight_top_log2() { return KV == PKV_BF16 ? 0 : 15; }

// What a state's weighted sum is kept by once it leaves the registers.
constexpr float STATE_UNIT = 16777216.0f;

// 2^d for d <= 0, 0 where that is not a normal number.
__device__ __forceinline__ float pow2_down(int d)
{
    return d < -126 ? 0.0f : pow2_f32(d);
}

// The B fragments of a tile's weights.  The MMA's 8 head columns take 8 / G
// parts of the weights at a time: column c holds part c / G of head c mod G (the
// columns repeat the heads), so that G < 8 needs one or two MMAs for all parts.
template <int KV, int G>
__host__ __device__ constexpr int weight_mmas() { return (weight_parts<KV>() * G + 7) / 8; }

template <int G, int KV>
__device__ __forceinline__ void split_weights(uint32_t (&bf)[weight_mmas<KV, G>()][2], float p0,
                                              float p1, float p2, float p3, int lane)
{
    constexpr bool BF = kern::MmaBf16<KV>::v;
    constexpr int NP = weight_parts<KV>();
    const int tig = lane & 3;
    uint32_t part[2][NP];                         // heads 2 tig, 2 tig + 1 of token gid | gid + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float x = h ? p2 : p0, y = h ? p3 : p1;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (BF) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
                x -= __low2float(v);
                y -= __high2float(v);
                part[h][i] = *reinterpret_cast<const uint32_t *>(&v);
            } else {
                const __half2 v = __floats2half2_rn(x, y);
                x -= __low2float(v);
                y -= __high2float(v);
                part[h][i] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < weight_mmas<KV, G>(); ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v = 0u;
            if constexpr (G == 1) {
                // columns 2 tig, 2 tig + 1 are parts 2 tig, 2 tig + 1 of the one head
                if (tig == 0)
                    v = __byte_perm(part[h][0], part[h][1], 0x7610u);
                else if (tig == 1 && NP > 2)
                    v = part[h][NP - 1] & 0xffffu;
            } else {
                const int mine = (2 * tig) / G + m * (8 / G);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    if (mine == i)
                        v = part[h][i];
            }
            bf[m][h] = kern::transpose8x8(v);
        }
}

// O^T += V^T P^T of NS tiles, tile n's in units of g[n].  A tile's sum starts at
// zero and is added to the running one in fp32: an MMA truncates what it adds to
// its accumulator, and over a long run of tiles that would show (3e-6 of the
// result at 230 tiles a warp).
template <int D, int G, int KV, int NS>
__device__ __forceinline__ void weigh_v(State<D, G, KV> &st,
                                        const uint32_t (&vw)[NS][4][kern::VFrag<D, KV>::VW],
                                        const uint32_t (&bf)[NS][weight_mmas<KV, G>()][2],
                                        const float (&g)[NS])
{
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t a0, a1, a2, a3;
            if constexpr (KV == PKV_F8) {
                const int w = j >> 1;
                const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                f8x4_to_half2(__byte_perm(vw[n][0][w], vw[n][1][w], sel), a0, a1);
                f8x4_to_half2(__byte_perm(vw[n][2][w], vw[n][3][w], sel), a2, a3);
            } else {
                a0 = __byte_perm(vw[n][0][j], vw[n][1][j], 0x5410u);
                a1 = __byte_perm(vw[n][0][j], vw[n][1][j], 0x7632u);
                a2 = __byte_perm(vw[n][2][j], vw[n][3][j], 0x5410u);
                a3 = __byte_perm(vw[n][2][j], vw[n][3][j], 0x7632u);
            }
#pragma unroll
            for (int m = 0; m < weight_mmas<KV, G>(); ++m)
                kern::mma_16816<kern::MmaBf16<KV>::v>(t, a0, a1, a2, a3, bf[n][m][0], bf[n][m][1]);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                st.acc[j][u] = KV == PKV_F8 ? fmaf(t[u], g[n], st.acc[j][u]) : st.acc[j][u] + t[u];
        }
}

// At a piece's end: the sums of a head's parts, in the head's own columns.
template <int D, int G, int KV>
__device__ __forceinline__ void join_parts(State<D, G, KV> &st)
{
    constexpr int NP = weight_parts<KV>();
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        if constexpr (G == 1) {
            st.acc[j][0] += st.acc[j][1];
            st.acc[j][2] += st.acc[j][3];
            if constexpr (NP > 2) {
                st.acc[j][0] += __shfl_down_sync(FULL_MASK, st.acc[j][0], 1);
                st.acc[j][2] += __shfl_down_sync(FULL_MASK, st.acc[j][2], 1);
            }
        } else if constexpr (G < 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x = st.acc[j][u];
                st.acc[j][u] += __shfl_down_sync(FULL_MASK, x, G / 2);
                if constexpr (G == 2 && NP > 2)
                    st.acc[j][u] += __shfl_down_sync(FULL_MASK, x, 2);
            }
        }
    }
}

// S^T = K q^T of the tile at sK, rows gid and gid + 8 and the lane's quarter of d
// (the fragments of the kernel for the other caches): e4m3 codes become fp16
// exactly, word ks of a quarter row being the pairs of k-step ks.
template <int D, int G, int KV>
__device__ __forceinline__ void tile_scores(float (&s)[4], const State<D, G, KV> &st,
                                            const unsigned char *sK, int lane)
{
    if constexpr (KV == PKV_F8) {
        using M = kern::MmaCfg<D, KV>;
        const int gid = lane >> 2, tig = lane & 3;
        const uint32_t k0 = gid * M::ROWB + tig * M::KQB, k1 = k0 + 8 * M::ROWB;
        // two chains, so that a tile's MMAs wait for half as many others
        float s2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < M::KCH; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(sK + kern::swz_off(k0 + c * 16, true));
            const uint4 y = *reinterpret_cast<const uint4 *>(sK + kern::swz_off(k1 + c * 16, true));
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ks = 4 * c + i;
                uint32_t a0, a1, a2, a3;
                f8x4_to_half2(xw[i], a0, a2);
                f8x4_to_half2(yw[i], a1, a3);
                kern::mma_16816<false>((i & 1) ? s2 : s, a0, a1, a2, a3, st.qh[ks][0],
                                       st.qh[ks][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i] += s2[i];
    } else {
        kern::mma_scores<D, G, KV, false>(s, st, sK, lane, true);
    }
}

// The lane's eighth of the V rows of tokens 2 tig, + 1, + 8, + 9 of the tile at sV.
template <int D, int KV>
__device__ __forceinline__ void tile_values(uint32_t (&vw)[4][kern::VFrag<D, KV>::VW],
                                            const unsigned char *sV, int lane)
{
    using M = kern::MmaCfg<D, KV>;
    if constexpr (M::VB >= 16) {
        kern::load_v_frag<D, KV>(vw, sV, lane, true);
    } else {
        const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v0 = (2 * tig + (i & 1) + 8 * (i >> 1)) * M::ROWB + gid * M::VB;
            const uint2 x = *reinterpret_cast<const uint2 *>(
                sV + kern::swz_off(v0 & ~15u, true) + (v0 & 15u));
            vw[i][0] = x.x;
            vw[i][1] = x.y;
        }
    }
}

// x * f, y * g, packed.
__device__ __forceinline__ void scale2(float &x, float &y, float f, float g)
{
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(f), "f"(g));
}

// NS tiles of a piece: scores, online softmax, weighted V (see the head of the
// file).  ONE: a tile's rows are of one block.
template <int D, int G, int KV, int NS, bool ONE>
__device__ __forceinline__ void tiles(State<D, G, KV> &st, const QScale<KV> &qscale,
                                      const unsigned char *const (&stage)[NS],
                                      const int (&bits)[NS], int lane)
{
    using C = Cfg<D, G, KV>;
    const int gid = lane >> 2;
    uint32_t vw[NS][4][kern::VFrag<D, KV>::VW];
    float x[NS][4];                    // (token gid | gid + 8, heads 2 tig, 2 tig + 1)
    int ev[NS][2], top = BLOCK_MIN_EXP;   // exponents of the V scales of rows 0..7, 8..15
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        tile_scores<D, G, KV>(s, st, stage[n], lane);
        tile_values<D, KV>(vw[n], stage[n] + C::TILE_BYTES, lane);
        if constexpr (C::F8) {
            // the scales of rows 0..7 and 8..15 (of one block, unless blocks are
            // smaller than a tile)
            const float *sc = reinterpret_cast<const float *>(stage[n] + 2 * C::TILE_BYTES);
            const float k0 = sc[0];
            float k1 = k0;
            ev[n][0] = ev[n][1] = block_exponent(sc[TILE]);
            if constexpr (!ONE) {
                k1 = sc[8];
                // (a block without an attended row has no say)
                if (rows_of(bits[n]) > 8)
                    ev[n][1] = block_exponent(sc[TILE + 8]);
                if (skip_of(bits[n]) >= 8)
                    ev[n][0] = ev[n][1];
            }
            top = max(top, max(ev[n][0], ev[n][1]));
            scale2(s[0], s[1], qscale.first[0], qscale.first[1]);
            scale2(s[2], s[3], qscale.first[0], qscale.first[1]);
            scale2(s[0], s[1], k0, k0);
            scale2(s[2], s[3], k1, k1);
            scale2(s[0], s[1], qscale.second[0], qscale.second[1]);
            scale2(s[2], s[3], qscale.second[0], qscale.second[1]);
        } else {
            scale2(s[0], s[1], qscale.first[0], qscale.first[1]);
            scale2(s[2], s[3], qscale.first[0], qscale.first[1]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[n][u] = s[u];
        if (!is_full(bits[n])) {
            const int rows = rows_of(bits[n]), skip = skip_of(bits[n]);
            if (gid >= rows || gid < skip)
                x[n][0] = x[n][1] = -INFINITY;
            if (gid + 8 >= rows || gid + 8 < skip)
                x[n][2] = x[n][3] = -INFINITY;
        }
        mx0 = fmaxf(mx0, fmaxf(x[n][0], x[n][2]));
        mx1 = fmaxf(mx1, fmaxf(x[n][1], x[n][3]));
    }
    bool above = mx0 > st.m[0] || mx1 > st.m[1];
    if constexpr (C::F8)
        above |= top > st.r;
    if (__any_sync(FULL_MASK, above)) {
#pragma unroll
        for (int mask = 4; mask < 32; mask <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, mask));
            mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, mask));
        }
        const float t0 = fmaxf(st.m[0], ceilf(mx0)), t1 = fmaxf(st.m[1], ceilf(mx1));
        const float c0 = kern::exp2_approx(st.m[0] - t0);
        const float c1 = kern::exp2_approx(st.m[1] - t1);
        st.m[0] = t0;
        st.m[1] = t1;
        st.l[0] *= c0;
        st.l[1] *= c1;
        float a0 = c0, a1 = c1;
        if constexpr (C::F8) {
            const int r = max(st.r, top);
            const float u = pow2_down(st.r - r);
            a0 *= u;
            a1 *= u;
            st.r = r;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            st.acc[j][0] *= a0;
            st.acc[j][2] *= a0;
            st.acc[j][1] *= a1;
            st.acc[j][3] *= a1;
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        x[n][0] = kern::exp2_approx(x[n][0] - st.m[0]);
        x[n][1] = kern::exp2_approx(x[n][1] - st.m[1]);
        x[n][2] = kern::exp2_approx(x[n][2] - st.m[0]);
        x[n][3] = kern::exp2_approx(x[n][3] - st.m[1]);
        st.l[0] += x[n][0] + x[n][2];
        st.l[1] += x[n][1] + x[n][3];
    }
    constexpr float TOP = (float)(1 << weight_top_log2<KV>());
    uint32_t bf[NS][weight_mmas<KV, G>()][2];
    float g[NS];
    if constexpr (!C::F8 || ONE) {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if constexpr (weight_top_log2<KV>() != 0) {
                scale2(x[n][0], x[n][1], TOP, TOP);
                scale2(x[n][2], x[n][3], TOP, TOP);
            }
            if constexpr (C::F8)
                g[n] = pow2_down(ev[n][0] - st.r);
            split_weights<G, KV>(bf[n], x[n][0], x[n][1], x[n][2], x[n][3], lane);
        }
        weigh_v<D, G, KV, NS>(st, vw, bf, g);
    } else {
        // two blocks a tile: together where their scales are close, else one by one
        bool again = false;
#pragma unroll 1
        for (int pass = 0;; ++pass) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int far = max(ev[n][0], ev[n][1]);
                int e = far;
                float f0, f1;              // of rows 0..7 and 8..15
                if (far - min(ev[n][0], ev[n][1]) > 4) {
                    e = pass ? ev[n][1] : ev[n][0];
                    f0 = pass ? 0.0f : TOP;
                    f1 = pass ? TOP : 0.0f;
                    again = true;
                } else {
                    f0 = pass ? 0.0f : TOP * pow2_f32(ev[n][0] - far);
                    f1 = pass ? 0.0f : TOP * pow2_f32(ev[n][1] - far);
                }
                g[n] = pow2_down(e - st.r);
                split_weights<G, KV>(bf[n], x[n][0] * f0, x[n][1] * f0, x[n][2] * f1,
                                     x[n][3] * f1, lane);
            }
            weigh_v<D, G, KV, NS>(st, vw, bf, g);
            if (!again || pass == 1)
                break;
        }
    }
}

// ONE: a tile's rows are of one block (16-bit caches: nothing of the math asks).
// A kernel of its own for 8-bit float blocks of 8 rows: its tile math beside the
// other's in one kernel costs registers (64 sequences of up to 4096 tokens, 32 / 8
// heads of 64, blocks of 16: 46.7 instead of 40.5 us).
template <int D, int G, int KV, bool ONE>
__global__ void __launch_bounds__(Cfg<D, G, KV>::NT, 1)
    decode_blocks_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<D, G, KV>;
    using S = Smem<D, G, KV>;
    constexpr int W = C::W, NT = C::NT, NST = C::NST;
    extern __shared__ __align__(1024) unsigned char smem[];
    float *states = reinterpret_cast<float *>(smem + S::STATES);
    int *tstart = reinterpret_cast<int *>(smem + S::TSTART);
    int *meta = reinterpret_cast<int *>(smem + S::meta(p.batch));   // [W][2] pieces, -1 = none
    int *scan = meta + 2 * W;                                       // [W] warp sums, [W] maxima
    int *flag = scan + 2 * W;                                       // [2] pieces to join here
    int *edge = flag + 2;        // the CTA's first and last piece: index, its first and last CTA
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.batch, Hkv = p.num_kv_heads, Hq = p.num_q_heads;
    const int cta = blockIdx.x;

    // Over chosen blocks the kernel before this one is the one that chose them: of
    // what this kernel reads it writes their list alone, and it let this kernel
    // start only after all before it had completed, so that the lengths may be
    // read ahead of the wait.
    if (!p.per_head) {
        grid_dependency_wait();
        grid_dependents_launch();
    }

    // ---- exclusive prefix of the sequences' tiles (all KV heads')
    {
        const int per = (B + NT - 1) / NT;
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int n = 0, most = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int raw = p.seq_lens[b];
            if ((raw < 0 || raw > p.len_cap) && cta == 0)
                atomicOr(p.err, PKV_EBIT_SEQLEN);
            const int L = raw < 0 || raw > p.len_cap ? 0 : attended_len(p, raw);
            if (S::has_lens(B))
                tstart[B + 1 + b] = L;
            const int nt = num_tiles(L, first_row(p, L));
            n += nt * Hkv;
            // (a sequence without tiles counts as one too long for the even split)
            most = max(most, nt > 0 ? nt : INT_MAX);
        }
        most = __reduce_max_sync(FULL_MASK, most);
        int inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(FULL_MASK, inc, off);
            if (lane >= off)
                inc += x;
        }
        if (lane == 31) {
            scan[warp] = inc;
            scan[W + warp] = most;
        }
        if (tid < 2 * W)
            meta[tid] = -1;
        if (tid < 2)
            flag[tid] = -1;
        __syncthreads();
        int at = inc - n;
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (w < warp)
                at += scan[w];
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            tstart[b] = at;
            const int L = S::has_lens(B) ? tstart[B + 1 + b] : seq_len(p, b);
            at += num_tiles(L, first_row(p, L)) * Hkv;
        }
        if (tid == NT - 1)
            tstart[B] = at;
        __syncthreads();
    }
    const int T = tstart[B];
    // ---- this CTA's tiles [c0, c1), and how many CTAs have any (P).  Where the
    // sequences are about as long as one another, a CTA takes `each` whole
    // pieces, so that none is joined across CTAs: if that leaves at most a
    // fifth of the CTAs idle (joining costs more than they would take over: 16 x
    // 4096 e4m3 tokens of 8 KV heads on 128 of 152 SMs 28.0 us, shared out over
    // all 30.0; 128 chosen blocks of 16 bf16 sequences 45.1 and 49.4), or if the
    // pieces are so short that joining costs more than it spreads.
    // Else every CTA takes an equal part of the list, but no fewer than
    // MIN_TILES tiles a warp.
    int most = scan[W];
#pragma unroll
    for (int w = 1; w < W; ++w)
        most = max(most, scan[W + w]);
    const bool even = (int64_t)most * B * Hkv <= (int64_t)T + T / 8 &&
                      (p.whole_ctas * 5 >= (int)gridDim.x * 4 || most <= SHORT_TILES * W);
    const int P = even ? p.whole_ctas : max(1, min((int)gridDim.x, T / (W * MIN_TILES)));
    // tiles of one KV head of sequence b
    auto tiles_a_head = [&](int b) { return quotient(tstart[b + 1] - tstart[b], Hkv); };
    // an uneven split's boundaries, floor(c T / P), and the CTA with tile x
    // (cut(c) is at least c TP, and more than that by less than c)
    const int TP = T / P, TR = T - TP * P;
    auto cut = [&](int c) { return c * TP + quotient(c * TR, P); };
    auto owner = [&](int x) {
        int c = min(P - 1, quotient(x, TP));
        while (cut(c) > x)
            --c;
        return c;
    };
    int c0 = T, c1 = T;
    if (cta < P) {
        if (even) {
            int b = quotient(cta * p.pieces_each, Hkv);
            c0 = tstart[b] + (cta * p.pieces_each - b * Hkv) * tiles_a_head(b);
            if (cta + 1 < P) {
                b = quotient((cta + 1) * p.pieces_each, Hkv);
                c1 = tstart[b] + ((cta + 1) * p.pieces_each - b * Hkv) * tiles_a_head(b);
            }
        } else {
            c0 = cut(cta);
            c1 = cut(cta + 1);
        }
    }
    const int r0 = c0 + (int)((int64_t)warp * (c1 - c0) / W);
    const int r1 = c0 + (int)((int64_t)(warp + 1) * (c1 - c0) / W);
    if (p.per_head) {
        grid_dependency_wait();
        grid_dependents_launch();
    }
    unsigned char *ring = smem + S::RING + warp * NST * C::STAGE;
    int4 *info = reinterpret_cast<int4 *>(smem + S::INFO) + warp * NST;
    if (r0 < r1) {
        const int n = r1 - r0;
        // the lanes describe the run's tiles 32 at a time: one round trip to the
        // block tables for all of them
        int base = 0;
        Tile d = tile_at<D, G, KV>(p, tstart, min(r0 + lane, r1 - 1));
        uint32_t qraw[D / 8];
        fetch_q<D, G>(qraw, p, __shfl_sync(FULL_MASK, d.b, 0), __shfl_sync(FULL_MASK, d.kvh, 0),
                      lane);
        int issued = 0;
        auto issue = [&]() {
            if (issued < n) {
                if (issued - base == 32) {
                    base = issued;
                    d = tile_at<D, G, KV>(p, tstart, min(r0 + base + lane, r1 - 1));
                }
                issue_tile<D, G, KV>(p, d, issued - base, ring + (issued % NST) * C::STAGE,
                                     info + issued % NST, lane);
                ++issued;
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i)
            issue();

        State<D, G, KV> st;
        QScale<KV> qscale;
        bool fresh = true;
        bool whole = true;                 // the piece began in this run
        const int gid = lane >> 2, tig = lane & 3;
#pragma unroll 1
        for (int k = 0, step = 1; k < n; k += step) {
            __syncwarp();              // the last tiles are read; this one's info is there
            const int4 it = info[k % NST];
            // two tiles of the piece at a time, while it has them
            const bool two = C::PAIR && !(it.x & LAST) && k + 1 < n;
            step = two ? 2 : 1;
            if (two)
                cp_wait<C::PAIR ? NST - 3 : 0>();
            else
                cp_wait<NST - 2>();
            __syncwarp();              // the lanes' copies have landed
            const int bits1 = two ? info[(k + 1) % NST].x : it.x;
            if (fresh) {
                whole = (it.x & FIRST) != 0;
                use_q<D, G, KV>(st, qscale, qraw, p, lane);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    st.m[r] = NO_SCORE;
                    st.l[r] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        st.acc[j][u] = 0.0f;
                st.r = BLOCK_MIN_EXP;
                fresh = false;
            }
            issue();
            const bool ends = (bits1 & LAST) != 0;
            if (ends && k + step < n) {
                // q of the next piece, on its way while this piece's last tile is computed
                __syncwarp();
                const int4 next = info[(k + step) % NST];
                fetch_q<D, G>(qraw, p, next.y, next.z, lane);
            }
            const unsigned char *s0 = ring + (k % NST) * C::STAGE;
            if (two) {
                if constexpr (C::PAIR) {
                    const unsigned char *const st2[2] = {s0, ring + ((k + 1) % NST) * C::STAGE};
                    const int b2[2] = {it.x, bits1};
                    tiles<D, G, KV, 2, ONE>(st, qscale, st2, b2, lane);
                    __syncwarp();      // the first tile's stage may be filled again
                    issue();
                }
            } else {
                const unsigned char *const st1[1] = {s0};
                const int b1[1] = {it.x};
                tiles<D, G, KV, 1, ONE>(st, qscale, st1, b1, lane);
            }
            if (ends || k + step == n) {
                // ---- the piece's end, or the run's
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int mask = 4; mask < 32; mask <<= 1)
                        st.l[r] += __shfl_xor_sync(FULL_MASK, st.l[r], mask);
                join_parts<D, G, KV>(st);
                const bool out_now = whole && ends;
                if (!out_now)
                    __syncwarp();      // the ring may be overwritten
                float *dst;
                if (out_now) {
                    dst = p.out + ((int64_t)it.y * Hq + it.z * G) * D;
                } else {
                    // a piece that began before the run is its first one and
                    // has a place of its own; one that goes on behind it is
                    // its last one and takes the drained ring's
                    dst = whole ? reinterpret_cast<float *>(ring) : states + warp * C::STATE;
                    if (lane == 0)
                        meta[2 * warp + (whole ? 1 : 0)] = it.y * Hkv + it.z;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = 2 * tig + r;
                    if (h < G) {
                        // from acc's unit to values
                        const float f = pow2_f32((C::F8 ? st.r : 0) - weight_top_log2<KV>());
                        const float inv = out_now ? 1.0f / st.l[r] : 1.0f / STATE_UNIT;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
                            *reinterpret_cast<float2 *>(dst + h * D + gid * (D / 8) + 2 * j) =
                                make_float2(st.acc[j][r] * inv * f, st.acc[j][r + 2] * inv * f);
                        if (!out_now && gid == 0) {
                            dst[G * D + h] = st.m[r];
                            dst[G * D + G + h] = st.l[r];
                        }
                    }
                }
                fresh = true;
            }
        }
        cp_wait<0>();
    }
    if (warp == W - 1 && lane < 2 && !even && c0 < c1) {
        // the CTAs of this one's first and last piece
        const int x = lane ? c1 - 1 : c0;
        const int b = kern::find_seq(tstart, B, x), nt = tiles_a_head(b);
        const int kvh = quotient(x - tstart[b], nt), x0 = tstart[b] + kvh * nt;
        edge[3 * lane] = b * Hkv + kvh;
        edge[3 * lane + 1] = owner(x0);
        edge[3 * lane + 2] = owner(x0 + nt - 1);
    }

    // rows of sequences without a row to attend: zeros
#pragma unroll 1
    for (int b = cta; b < B; b += gridDim.x)
        if (tstart[b + 1] == tstart[b])
#pragma unroll 1
            for (int i = tid; i < Hq * D; i += NT)
                p.out[(int64_t)b * Hq * D + i] = 0.0f;
    if (c0 >= c1)
        return;
    __syncthreads();

    // ---- join the warps' states of each piece (they lie in list order)
    // lane f: state f (warp f / 2's first or last piece)
    static_assert(2 * W <= 32, "a lane a state");
    const float *mine_state = lane & 1 ? reinterpret_cast<const float *>(
                                             smem + S::RING + (lane >> 1) % W * NST * C::STAGE)
                                       : states + (lane >> 1) % W * C::STATE;
    const int mine_seg = lane < 2 * W ? meta[lane] : -1;
    const unsigned valid = __ballot_sync(FULL_MASK, mine_seg >= 0);
    const unsigned before = valid & ((1u << lane) - 1u);
    const int prev_seg = __shfl_sync(FULL_MASK, mine_seg, before ? 31 - __clz(before) : 0);
    unsigned starts = __ballot_sync(FULL_MASK,
                                    mine_seg >= 0 && (before == 0 || prev_seg != mine_seg));
    constexpr int MO = (G * D + NT - 1) / NT;   // elements of a piece's output a thread joins
    int shared_pieces = 0;
    while (starts) {
        const int f = __ffs(starts) - 1;
        starts &= starts - 1;
        const unsigned members =
            valid & ~((1u << f) - 1u) & (starts ? (starts & (~starts + 1u)) - 1u : ~0u);
        const int seg = __shfl_sync(FULL_MASK, mine_seg, f);
        // shared with other CTAs: 1 as this CTA's first piece, 2 as its last
        int edges = 0;
        if (!even)
            for (int t = 0; t < 2; ++t)
                if (edge[3 * t] == seg && edge[3 * t + 1] != edge[3 * t + 2])
                    edges = t + 1;
        const bool mine = edges == 0;
        float *dst = mine ? p.out + (int64_t)seg * G * D
                          : p.partials + (int64_t)(cta + seg) * C::STATE;
        const bool member = (members >> lane) & 1u;
        // a warp's 32 elements belong to one head: the lanes weigh the states
        float w[MO], den[MO], top[MO], num[MO];
#pragma unroll
        for (int o = 0; o < MO; ++o) {
            const int g = min((o * NT + tid) / D, G - 1);
            const float m = member ? mine_state[G * D + g] : -INFINITY;
            const float l = member ? mine_state[G * D + G + g] : 0.0f;
            top[o] = warp_max(m);
            w[o] = member ? join_weight(m, top[o]) : 0.0f;
            den[o] = warp_sum(w[o] * l);
            num[o] = 0.0f;
        }
#pragma unroll 1
        for (unsigned left = members; left;) {
            // four states at a time; past the last one it is read again, with weight 0
            int u[4];
            float v[4][MO];
            bool there[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                there[t] = left != 0u;
                u[t] = there[t] ? __ffs(left) - 1 : u[0];
                left &= left - 1u;
                const float *sp = (u[t] & 1 ? reinterpret_cast<const float *>(
                                                  smem + S::RING + (u[t] >> 1) * NST * C::STAGE)
                                            : states + (u[t] >> 1) * C::STATE) + tid;
#pragma unroll
                for (int o = 0; o < MO; ++o)
                    v[t][o] = tid + o * NT < G * D ? sp[o * NT] : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int o = 0; o < MO; ++o) {
                    const float wu = __shfl_sync(FULL_MASK, w[o], u[t]);
                    num[o] = fmaf(there[t] ? wu : 0.0f, v[t][o], num[o]);
                }
        }
#pragma unroll
        for (int o = 0; o < MO; ++o) {
            const int i = o * NT + tid, g = i / D;
            if (i < G * D) {
                dst[i] = mine ? num[o] / den[o] * STATE_UNIT : num[o];
                if (!mine && i % D == 0) {
                    dst[G * D + g] = top[o];
                    dst[G * D + G + g] = den[o];
                }
            }
        }
        shared_pieces |= edges;        // bit t: the piece edge[3 t] is
    }
    if (shared_pieces == 0)
        return;
    __syncthreads();
    if (tid < 2 && (shared_pieces >> tid & 1)) {
        const int seg = edge[3 * tid];
        __threadfence();               // every thread's partials, ordered before the count
        if (atomicAdd(p.counters + seg, 1) == edge[3 * tid + 2] - edge[3 * tid + 1]) {
            flag[tid] = seg;
            p.counters[seg] = 0;
            __threadfence();
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        const int seg = flag[j];
        if (seg < 0)
            continue;
        const int o0 = edge[3 * j + 1], o1 = edge[3 * j + 2];
        const float *part = p.partials + (int64_t)(o0 + seg) * C::STATE;
        const int np = o1 - o0 + 1;
        float num[MO], den[MO], top[MO];
#pragma unroll
        for (int o = 0; o < MO; ++o) {
            num[o] = den[o] = 0.0f;
            top[o] = -INFINITY;
        }
        // 16 partials at a time, all their loads on the way together
        constexpr int BATCH = 16;
#pragma unroll 1
        for (int q0 = 0; q0 < np; q0 += BATCH) {
            const int qn = min(BATCH, np - q0);
            float v[BATCH][MO], m[MO], l[MO];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const float *sp = part + (int64_t)(q0 + min(u, qn - 1)) * C::STATE + tid;
#pragma unroll
                for (int o = 0; o < MO; ++o)
                    v[u][o] = tid + o * NT < G * D ? __ldcg(sp + o * NT) : 0.0f;
            }
#pragma unroll
            for (int o = 0; o < MO; ++o) {
                const int g = min((o * NT + tid) / D, G - 1);
                const float *sp = part + (int64_t)(q0 + min(lane, qn - 1)) * C::STATE + G * D + g;
                m[o] = __ldcg(sp);
                l[o] = __ldcg(sp + G);
            }
#pragma unroll
            for (int o = 0; o < MO; ++o) {
                const bool in = lane < qn;
                const float mn = fmaxf(top[o], warp_max(in ? m[o] : -INFINITY));
                const float a = join_weight(top[o], mn);
                const float w = in ? join_weight(m[o], mn) : 0.0f;
                den[o] = fmaf(den[o], a, warp_sum(in ? w * l[o] : 0.0f));
                num[o] *= a;
                top[o] = mn;
#pragma unroll
                for (int u = 0; u < BATCH; ++u)
                    num[o] = fmaf(__shfl_sync(FULL_MASK, w, u), v[u][o], num[o]);
            }
        }
#pragma unroll
        for (int o = 0; o < MO; ++o)
            if (tid + o * NT < G * D)
                p.out[(int64_t)seg * G * D + o * NT + tid] =
                    num[o] / den[o] * STATE_UNIT;
    }
}

// ---- host side ---------------------------------------------------------------

template <int D, int G, int KV, bool ONE>
int launch_k(const pkv_pool *pool, const Params &base, cudaStream_t stream, int64_t max_tiles)
{
    Params prm = base;
    using C = Cfg<D, G, KV>;
    const int smem = Smem<D, G, KV>::total(prm.batch);
    if (smem > pool->max_smem_optin)
        return PKV_ERR_UNSUPPORTED;
    // The limit belongs to the kernel, not to the launch: the largest batch's, the same
    // from every call, so that a call from another host thread between this one's
    // setting and its launch changes nothing.
    if (cudaFuncSetAttribute(decode_blocks_kernel<D, G, KV, ONE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem<D, G, KV>::total(MAX_BATCH)) != cudaSuccess)
        return PKV_ERR_CUDA;
    // a CTA for each piece, or one for the least its warps take
    int64_t P = max_tiles / (C::W * MIN_TILES);
    if (P < (int64_t)prm.batch * prm.num_kv_heads)
        P = (int64_t)prm.batch * prm.num_kv_heads;
    if (P > pool->num_sms)
        P = pool->num_sms;
    if (P < 1)
        P = 1;
    const int64_t pieces = (int64_t)prm.batch * prm.num_kv_heads;
    prm.pieces_each = (int)((pieces + P - 1) / P);
    prm.whole_ctas = (int)((pieces + prm.pieces_each - 1) / prm.pieces_each);
    if (launch_pdl(decode_blocks_kernel<D, G, KV, ONE>, dim3((unsigned)P), dim3(C::NT),
                   (size_t)smem, stream, prm) != cudaSuccess)
        return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, int G, int KV>
int launch_t(const pkv_pool *pool, const Params &prm, cudaStream_t s, int64_t max_tiles)
{
    if constexpr (KV == PKV_F8)
        if (prm.block_size < TILE)
            return launch_k<D, G, KV, false>(pool, prm, s, max_tiles);
    return launch_k<D, G, KV, true>(pool, prm, s, max_tiles);
}

template <int D, int KV>
int launch_g(const pkv_pool *pool, const Params &prm, cudaStream_t s, int64_t max_tiles)
{
    switch (prm.num_q_heads / prm.num_kv_heads) {
    case 1: return launch_t<D, 1, KV>(pool, prm, s, max_tiles);
    case 2: return launch_t<D, 2, KV>(pool, prm, s, max_tiles);
    case 4: return launch_t<D, 4, KV>(pool, prm, s, max_tiles);
    case 8: return launch_t<D, 8, KV>(pool, prm, s, max_tiles);
    }
    return PKV_ERR_UNSUPPORTED;
}

template <int KV>
int launch_d(const pkv_pool *pool, const Params &prm, cudaStream_t s, int64_t max_tiles)
{
    return pool->head_dim == 64 ? launch_g<64, KV>(pool, prm, s, max_tiles)
                                : launch_g<128, KV>(pool, prm, s, max_tiles);
}

}  // namespace blk
}  // namespace pkv
