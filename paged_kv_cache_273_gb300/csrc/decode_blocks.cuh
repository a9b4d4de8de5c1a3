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
//    tile).  CTA c of P takes the tiles [c T / P, (c + 1) T / P), and its
//    warps equal parts of those: every warp streams a contiguous run of tiles
//    through a ring of its own (cp.async, completion counted per thread), so
//    no warp waits for another and nothing waits on a flag or barrier until
//    the CTA's end.
//  * A warp keeps the online softmax state of its current (sequence, KV
//    head) in registers.  A piece that lies inside one warp's run is written
//    straight to the output.  At most two pieces of a run are shared with
//    neighbours; their states go to shared memory, the CTA joins the states
//    of its warps at its end, and a piece shared with other CTAs is left in
//    the workspace and joined, in CTA order, by the last of them to finish
//    (the result does not depend on timing).
//  * Tile math: warp-level MMAs as in the kernel for the other caches; e4m3
//    codes become fp16 exactly, q becomes fp16 exactly (a bf16 q is brought
//    to [2^14, 2^15) by a power of two first), products are exact and sums
//    fp32.  A V scale 2^ev is part of the weight's exponent: with x a row's
//    score * log2(e), the denominator sums 2^(x - m) and the weighted V sums
//    w c with w = 2^(x - m + ev - (n - m)) <= 1, c the V codes, where m and n
//    are whole numbers at or above the largest x and the largest x + ev so
//    far.  So a weight needs no multiplication by its scale and stays in
//    fp16's range whatever the scales are, both sums come from the same
//    rounded x - m, and every rescaling is by a power of two.  Weights are
//    split into a high and a low fp16 part (2^-22 relative; bf16 caches: two
//    bf16 parts, 2^-18).
//  * Rows outside the attended range are filled with zeros by the copies, so
//    that whatever they hold (NaN codes of an earlier owner) is never read.
#pragma once

#include "decode_kernel.cuh"

namespace pkv {
namespace blk {

using namespace dev;
using kern::round_up;

constexpr int TILE = 16;
constexpr int MAX_BATCH = 4096;
// Tiles a warp is given at least, where the batch has fewer than one share of
// that for every warp of the GPU.
constexpr int MIN_TILES = 2;

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
    static constexpr int W = 8;                     // warps
    static constexpr int NT = W * 32;
    static constexpr int STATE = G * (D + 2);       // floats of one softmax state
    // ring stages that fit beside the states and the tile prefix, at most 6
    static constexpr int FIXED = W * STATE * 4 + (MAX_BATCH + 1) * 4 + W * 8 + 256;
    static constexpr int FIT = (232448 - FIXED) / (W * STAGE);
    static constexpr int NST = FIT > 6 ? 6 : FIT;
    static_assert(NST >= 2, "ring");
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
    float scale_log2;
};

// Shared memory: the rings, the warps' first states, the tile prefix, the
// states' pieces.
template <int D, int G, int KV>
struct Smem {
    using C = Cfg<D, G, KV>;
    static constexpr int RING = 0;
    static constexpr int STATES = C::W * C::NST * C::STAGE;
    static constexpr int TSTART = STATES + C::W * C::STATE * 4;
    __host__ __device__ static int meta(int batch)
    {
        return round_up(TSTART + (batch + 1) * 4, 16);
    }
    __host__ __device__ static int total(int batch)
    {
        return meta(batch) + (2 * C::W + C::W + 8) * 4;
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
    const int L = __ldg(p.seq_lens + b);
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

// A position in the tile list.
struct Pos {
    int b, kvh, ti;      // sequence, KV head, 16-row tile of the sequence
    int L, lo;           // rows attended: [lo, L)
    int end;             // one past the piece's last tile
};

template <int D, int G, int KV>
__device__ __forceinline__ Pos pos_at(const Params &p, const int *tstart, int x)
{
    Pos s;
    s.b = kern::find_seq(tstart, p.batch, x);
    s.L = seq_len(p, s.b);
    s.lo = first_row(p, s.L);
    const int nt = num_tiles(s.L, s.lo);
    const int off = x - tstart[s.b];
    s.kvh = off / nt;
    s.ti = off - s.kvh * nt + s.lo / TILE;
    s.end = s.lo / TILE + nt;
    return s;
}

// To the next tile (only called when the list has one).
__device__ __forceinline__ void advance(const Params &p, const int *tstart, Pos &s)
{
    if (++s.ti < s.end)
        return;
    if (++s.kvh == p.num_kv_heads) {
        s.kvh = 0;
        do
            ++s.b;
        while (tstart[s.b + 1] == tstart[s.b]);
        s.L = seq_len(p, s.b);
        s.lo = first_row(p, s.L);
        s.end = (s.L + TILE - 1) / TILE;
    }
    s.ti = s.lo / TILE;
}

// Copies of one tile into a stage, one commit group.
template <int D, int G, int KV>
__device__ __forceinline__ void issue_tile(const Params &p, const Pos &s, unsigned char *stage,
                                           int lane)
{
    using C = Cfg<D, G, KV>;
    const int r0 = lane / C::CH, c = lane % C::CH;
    const int bs = p.block_size;
    const int32_t *row =
        p.tables + (p.per_head ? (int64_t)s.b * p.num_kv_heads + s.kvh : (int64_t)s.b) *
                       p.table_stride;
    const int t0 = TILE * s.ti;
    auto block_of = [&](int t, bool &ok) {
        int id = ok ? __ldg(row + (t >> p.bs_log2)) : 0;
        if (id < 0 || id >= p.num_blocks) {
            atomicOr(p.err, PKV_EBIT_BLOCK);
            id = 0;
            ok = false;
        }
        return id;
    };
    if (bs >= TILE) {
        // the tile lies in one block (its first attended row says which)
        bool ok = true;
        const int id = block_of(t0, ok);
        const int64_t head = (int64_t)id * p.num_kv_heads + s.kvh;
        const int64_t base = (head * bs + (t0 & (bs - 1)) + r0) * C::ROWB + c * 16;
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            const int r = r0 + i * C::RPI;
            const bool v = ok && t0 + r < s.L && t0 + r >= s.lo;
            const uint32_t dst = kern::swz_off(r * C::ROWB + c * 16, true);
            cp16_zfill(stage + dst, p.k_cache + base + i * C::RPI * C::ROWB, v);
            cp16_zfill(stage + C::TILE_BYTES + dst, p.v_cache + base + i * C::RPI * C::ROWB, v);
        }
        if constexpr (C::F8)
            cp4_zfill(stage + 2 * C::TILE_BYTES + lane * 4,
                      (lane < TILE ? p.k_scales : p.v_scales) + head, ok);
    } else {
#pragma unroll
        for (int i = 0; i < C::NI; ++i) {
            const int r = r0 + i * C::RPI, t = t0 + r;
            bool v = t < s.L && t >= s.lo;
            const int id = block_of(t, v);
            const int64_t off =
                (((int64_t)id * p.num_kv_heads + s.kvh) * bs + (t & (bs - 1))) * C::ROWB + c * 16;
            const uint32_t dst = kern::swz_off(r * C::ROWB + c * 16, true);
            cp16_zfill(stage + dst, p.k_cache + off, v);
            cp16_zfill(stage + C::TILE_BYTES + dst, p.v_cache + off, v);
        }
        if constexpr (C::F8) {
            const int t = t0 + (lane & (TILE - 1));
            bool v = t < s.L && t >= s.lo;
            const int id = block_of(t, v);
            cp4_zfill(stage + 2 * C::TILE_BYTES + lane * 4,
                      (lane < TILE ? p.k_scales : p.v_scales) +
                          ((int64_t)id * p.num_kv_heads + s.kvh),
                      v);
        }
    }
}

template <int D, int G, int KV>
struct State : kern::MmaState<D, G, KV, false> {
    float n[2];          // whole numbers >= x + ev of heads 2 tig, 2 tig + 1 (m: >= x)
};

// q of the G heads of (b, kvh) -> B fragments of the score MMAs (the head
// columns beyond G repeat the heads, as in the other kernel), and the factors
// that turn an MMA sum over the lane's two heads into a log2-domain score.
template <int D, int G, int KV>
__device__ __forceinline__ void load_q(State<D, G, KV> &st, float (&qscale)[2], const Params &p,
                                       int b, int kvh, int lane)
{
    constexpr bool F8 = KV == PKV_F8;
    constexpr int NQ = D / 32;                       // 16-byte chunks of the lane's quarter row
    const int gid = lane >> 2, tig = lane & 3;
    const int head = gid % G;
    const uint4 *src = reinterpret_cast<const uint4 *>(
        static_cast<const uint16_t *>(p.q) +
        ((int64_t)b * p.num_q_heads + kvh * G + head) * D + tig * (D / 4));
    uint32_t w[NQ * 4];
#pragma unroll
    for (int c = 0; c < NQ; ++c) {
        const uint4 x = __ldg(src + c);
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
    }
    float unscale = p.scale_log2;
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
        unscale = p.scale_log2 * pow2_f32(max(e, -112) - 14);
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
    qscale[0] = __shfl_sync(FULL_MASK, unscale, 8 * tig);
    qscale[1] = __shfl_sync(FULL_MASK, unscale, 8 * tig + 4);
}

// One tile: scores, online softmax, weighted V (see the head of the file).
template <int D, int G, int KV>
__device__ __forceinline__ void tile(State<D, G, KV> &st, const float (&qscale)[2],
                                     const unsigned char *stage, int nvalid, int tlo, int lane)
{
    using C = Cfg<D, G, KV>;
    const int gid = lane >> 2;
    const unsigned char *sK = stage, *sV = stage + C::TILE_BYTES;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    kern::mma_scores<D, G, KV, false>(s, st, sK, lane, true);
    uint32_t vw[4][kern::VFrag<D, KV>::VW];
    kern::load_v_frag<D, KV>(vw, sV, lane, true);
    const bool v0 = gid < nvalid && gid >= tlo;
    const bool v1 = gid + 8 < nvalid && gid + 8 >= tlo;
    float x0, x1, x2, x3, f0 = 0.0f, f1 = 0.0f;
    if constexpr (C::F8) {
        const float *sc = reinterpret_cast<const float *>(stage + 2 * C::TILE_BYTES);
        const float k0 = pow2_f32(block_exponent(sc[gid]));
        const float k1 = pow2_f32(block_exponent(sc[gid + 8]));
        f0 = (float)block_exponent(sc[TILE + gid]);
        f1 = (float)block_exponent(sc[TILE + gid + 8]);
        s[0] *= k0;
        s[1] *= k0;
        s[2] *= k1;
        s[3] *= k1;
    }
    x0 = v0 ? s[0] * qscale[0] : -INFINITY;       // token gid, head 2 tig
    x1 = v0 ? s[1] * qscale[1] : -INFINITY;       // token gid, head 2 tig + 1
    x2 = v1 ? s[2] * qscale[0] : -INFINITY;       // token gid + 8, head 2 tig
    x3 = v1 ? s[3] * qscale[1] : -INFINITY;       // token gid + 8, head 2 tig + 1
    float mx0 = fmaxf(x0, x2), mx1 = fmaxf(x1, x3);
    float my0 = mx0, my1 = mx1;
    bool above = mx0 > st.m[0] || mx1 > st.m[1];
    if constexpr (C::F8) {
        my0 = fmaxf(x0 + f0, x2 + f1);
        my1 = fmaxf(x1 + f0, x3 + f1);
        above |= my0 > st.n[0] || my1 > st.n[1];
    }
    if (__any_sync(FULL_MASK, above)) {
#pragma unroll
        for (int mask = 4; mask < 32; mask <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, mask));
            mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, mask));
            if constexpr (C::F8) {
                my0 = fmaxf(my0, __shfl_xor_sync(FULL_MASK, my0, mask));
                my1 = fmaxf(my1, __shfl_xor_sync(FULL_MASK, my1, mask));
            }
        }
        const float m0 = fmaxf(st.m[0], ceilf(mx0)), m1 = fmaxf(st.m[1], ceilf(mx1));
        const float c0 = kern::exp2_approx(st.m[0] - m0), c1 = kern::exp2_approx(st.m[1] - m1);
        st.m[0] = m0;
        st.m[1] = m1;
        st.l[0] *= c0;
        st.l[1] *= c1;
        float a0 = c0, a1 = c1;
        if constexpr (C::F8) {
            const float n0 = fmaxf(st.n[0], ceilf(my0)), n1 = fmaxf(st.n[1], ceilf(my1));
            a0 = kern::exp2_approx(st.n[0] - n0);
            a1 = kern::exp2_approx(st.n[1] - n1);
            st.n[0] = n0;
            st.n[1] = n1;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            st.acc[j][0] *= a0;
            st.acc[j][2] *= a0;
            st.acc[j][1] *= a1;
            st.acc[j][3] *= a1;
        }
    }
    x0 -= st.m[0];
    x1 -= st.m[1];
    x2 -= st.m[0];
    x3 -= st.m[1];
    float p0 = kern::exp2_approx(x0), p1 = kern::exp2_approx(x1);
    float p2 = kern::exp2_approx(x2), p3 = kern::exp2_approx(x3);
    st.l[0] += p0 + p2;
    st.l[1] += p1 + p3;
    if constexpr (C::F8) {
        const float d0 = st.n[0] - st.m[0], d1 = st.n[1] - st.m[1];
        p0 = kern::exp2_approx(x0 + (f0 - d0));
        p1 = kern::exp2_approx(x1 + (f0 - d1));
        p2 = kern::exp2_approx(x2 + (f1 - d0));
        p3 = kern::exp2_approx(x3 + (f1 - d1));
    }
    kern::mma_pv<D, G, KV, false>(st, vw, p0, p1, p2, p3, lane);
}

template <int D, int G, int KV>
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
    int *scan = meta + 2 * W;                                       // [W] warp sums
    int *flag = scan + W;                                           // [2] pieces to join here
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.batch, Hkv = p.num_kv_heads, Hq = p.num_q_heads;
    const int cta = blockIdx.x;

    grid_dependency_wait();
    grid_dependents_launch();

    // ---- exclusive prefix of the sequences' tiles (all KV heads')
    {
        const int per = (B + NT - 1) / NT;
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int n = 0;
        for (int b = b0; b < b1; ++b) {
            const int raw = __ldg(p.seq_lens + b);
            if ((raw < 0 || raw > p.len_cap) && cta == 0)
                atomicOr(p.err, PKV_EBIT_SEQLEN);
            const int L = seq_len(p, b);
            n += num_tiles(L, first_row(p, L)) * Hkv;
        }
        int inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(FULL_MASK, inc, off);
            if (lane >= off)
                inc += x;
        }
        if (lane == 31)
            scan[warp] = inc;
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
        for (int b = b0; b < b1; ++b) {
            tstart[b] = at;
            const int L = seq_len(p, b);
            at += num_tiles(L, first_row(p, L)) * Hkv;
        }
        if (tid == NT - 1)
            tstart[B] = at;
        __syncthreads();
    }
    const int T = tstart[B];
    // CTAs that share the list: no more than leave every warp MIN_TILES
    const int P = max(1, min((int)gridDim.x, T / (W * MIN_TILES)));

    // rows of sequences without a row to attend: zeros
    for (int b = cta; b < B; b += gridDim.x)
        if (tstart[b + 1] == tstart[b])
            for (int i = tid; i < Hq * D; i += NT)
                p.out[(int64_t)b * Hq * D + i] = 0.0f;
    if (cta >= P || T == 0)
        return;

    const int c0 = (int)((int64_t)cta * T / P), c1 = (int)((int64_t)(cta + 1) * T / P);
    const int r0 = c0 + (int)((int64_t)warp * (c1 - c0) / W);
    const int r1 = c0 + (int)((int64_t)(warp + 1) * (c1 - c0) / W);
    unsigned char *ring = smem + S::RING + warp * NST * C::STAGE;
    if (r0 < r1) {
        const int n = r1 - r0;
        Pos cs = pos_at<D, G, KV>(p, tstart, r0);
        Pos is = cs;
        int issued = 0;
        auto issue = [&]() {
            if (issued < n) {
                issue_tile<D, G, KV>(p, is, ring + (issued % NST) * C::STAGE, lane);
                if (++issued < n)
                    advance(p, tstart, is);
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i)
            issue();

        State<D, G, KV> st;
        float qscale[2];
        bool fresh = true;
        bool whole = cs.ti == cs.lo / TILE;       // the piece began in this run
        const int gid = lane >> 2, tig = lane & 3;
        for (int k = 0; k < n; ++k) {
            if (fresh) {
                load_q<D, G, KV>(st, qscale, p, cs.b, cs.kvh, lane);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    st.m[r] = st.n[r] = -INFINITY;
                    st.l[r] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        st.acc[j][u] = 0.0f;
                fresh = false;
            }
            cp_wait<NST - 2>();
            __syncwarp();              // the lanes' copies have landed, the last tile is read
            issue();
            tile<D, G, KV>(st, qscale, ring + (k % NST) * C::STAGE, cs.L - TILE * cs.ti,
                           cs.lo - TILE * cs.ti, lane);
            const bool ends = cs.ti + 1 == cs.end;
            if (ends || k + 1 == n) {
                // ---- the piece's end, or the run's
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int mask = 4; mask < 32; mask <<= 1)
                        st.l[r] += __shfl_xor_sync(FULL_MASK, st.l[r], mask);
                if constexpr (G == 1) {
                    // column 1 holds the low-part sums of column 0's head
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        st.acc[j][0] += st.acc[j][1];
                        st.acc[j][2] += st.acc[j][3];
                    }
                } else if constexpr (G < 8) {
                    // columns 2 tig + G, + 1 (lane + G / 2) hold the low-part
                    // sums of the lane's heads
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            st.acc[j][u] += __shfl_down_sync(FULL_MASK, st.acc[j][u], G / 2);
                }
                const bool out_now = whole && ends;
                if (!out_now)
                    __syncwarp();      // the ring may be overwritten
                float *dst;
                if (out_now) {
                    dst = p.out + ((int64_t)cs.b * Hq + cs.kvh * G) * D;
                } else {
                    // a piece that began before the run is its first one and
                    // has a place of its own; one that goes on behind it is
                    // its last one and takes the drained ring's
                    dst = whole ? reinterpret_cast<float *>(ring) : states + warp * C::STATE;
                    if (lane == 0)
                        meta[2 * warp + (whole ? 1 : 0)] = cs.b * Hkv + cs.kvh;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = 2 * tig + r;
                    if (h < G) {
                        // (8-bit float: from units of 2^(n - m) codes to values)
                        float f = C::F8 ? pow2_f32(min(max((int)(st.n[r] - st.m[r]), -126), 127))
                                        : 1.0f;
                        if (out_now)
                            f = f / st.l[r];
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
                            *reinterpret_cast<float2 *>(dst + h * D + gid * (D / 8) + 2 * j) =
                                make_float2(st.acc[j][r] * f, st.acc[j][r + 2] * f);
                        if (!out_now && gid == 0) {
                            dst[G * D + h] = st.m[r];
                            dst[G * D + G + h] = st.l[r];
                        }
                    }
                }
                fresh = true;
                whole = true;
            }
            if (k + 1 < n)
                advance(p, tstart, cs);
        }
        cp_wait<0>();
    }
    __syncthreads();

    // ---- join the warps' states of each piece (they lie in list order)
    auto state_of = [&](int f) {
        return f & 1 ? reinterpret_cast<const float *>(smem + S::RING +
                                                       (f >> 1) * NST * C::STAGE)
                     : states + (f >> 1) * C::STATE;
    };
    auto tiles_of = [&](int seg, int &x0, int &x1) {
        const int b = seg / Hkv, kvh = seg - b * Hkv;
        const int nt = (tstart[b + 1] - tstart[b]) / Hkv;
        x0 = tstart[b] + kvh * nt;
        x1 = x0 + nt;
    };
    int shared_pieces = 0;
    for (int f = 0; f < 2 * W;) {
        const int seg = meta[f];
        if (seg < 0) {
            ++f;
            continue;
        }
        int e = f + 1;
        while (e < 2 * W && (meta[e] == seg || meta[e] < 0))
            ++e;
        int x0, x1;
        tiles_of(seg, x0, x1);
        const bool mine = x0 >= c0 && x1 <= c1;
        float *dst = mine ? p.out + ((int64_t)(seg / Hkv) * Hq + (seg % Hkv) * G) * D
                          : p.partials + (int64_t)(cta + seg) * C::STATE;
        for (int i = tid; i < G * D; i += NT) {
            const int g = i / D;
            float M = -INFINITY;
            for (int u = f; u < e; ++u)
                if (meta[u] >= 0)
                    M = fmaxf(M, state_of(u)[G * D + g]);
            float num = 0.0f, den = 0.0f;
            for (int u = f; u < e; ++u)
                if (meta[u] >= 0) {
                    const float *sp = state_of(u);
                    const float w = kern::exp2_approx(sp[G * D + g] - M);
                    num = fmaf(w, sp[i], num);
                    den = fmaf(w, sp[G * D + G + g], den);
                }
            if (mine) {
                dst[i] = num / den;
            } else {
                dst[i] = num;
                if (i % D == 0) {
                    dst[G * D + g] = M;
                    dst[G * D + G + g] = den;
                }
            }
        }
        if (!mine) {
            if (tid == 0)
                scan[shared_pieces] = seg;
            ++shared_pieces;           // at most two: the CTA's first and last piece
        }
        f = e;
    }
    if (shared_pieces == 0)
        return;
    __syncthreads();
    if (tid == 0) {
        __threadfence();               // every thread's partials, ordered before the counts
        for (int i = 0; i < shared_pieces; ++i) {
            const int seg = scan[i];
            int x0, x1;
            tiles_of(seg, x0, x1);
            const int others = kern::owner_of(x1 - 1, T, P) - kern::owner_of(x0, T, P);
            if (atomicAdd(p.counters + seg, 1) == others) {
                flag[i] = seg;
                p.counters[seg] = 0;
            }
        }
        __threadfence();
    }
    __syncthreads();
    for (int j = 0; j < 2; ++j) {
        const int seg = flag[j];
        if (seg < 0)
            continue;
        int x0, x1;
        tiles_of(seg, x0, x1);
        const int o0 = kern::owner_of(x0, T, P), o1 = kern::owner_of(x1 - 1, T, P);
        for (int i = tid; i < G * D; i += NT) {
            const int g = i / D;
            float m = -INFINITY, num = 0.0f, den = 0.0f;
#pragma unroll 4
            for (int c = o0; c <= o1; ++c) {
                const float *sp = p.partials + (int64_t)(c + seg) * C::STATE;
                const float mp = __ldcg(sp + G * D + g), np = __ldcg(sp + i),
                            dp = __ldcg(sp + G * D + G + g);
                const float mn = fmaxf(m, mp);
                const float a = kern::exp2_approx(m - mn), w = kern::exp2_approx(mp - mn);
                num = fmaf(num, a, np * w);
                den = fmaf(den, a, dp * w);
                m = mn;
            }
            p.out[((int64_t)(seg / Hkv) * Hq + (seg % Hkv) * G) * D + i] = num / den;
        }
    }
}

// ---- host side ---------------------------------------------------------------

template <int D, int G, int KV>
int launch_t(const pkv_pool *pool, const Params &prm, cudaStream_t stream, int64_t max_tiles)
{
    using C = Cfg<D, G, KV>;
    const int smem = Smem<D, G, KV>::total(prm.batch);
    if (smem > pool->max_smem_optin)
        return PKV_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(decode_blocks_kernel<D, G, KV>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return PKV_ERR_CUDA;
    int64_t P = max_tiles / (C::W * MIN_TILES);
    if (P > pool->num_sms)
        P = pool->num_sms;
    if (P < 1)
        P = 1;
    if (launch_pdl(decode_blocks_kernel<D, G, KV>, dim3((unsigned)P), dim3(C::NT), (size_t)smem,
                   stream, prm) != cudaSuccess)
        return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
