// Rotary positions: kv_rope_rotate (rotated heads of a projection's output) and
// kv_rope_append (the same rotation of q and K on the way to the attention's q and
// to the paged cache, V beside it).
//
// Pair i of a head's first rot_dim channels, (a, b), at position p becomes
//   m (a cos - b sin, b cos + a sin),  angle = p * theta_i.
// theta_i comes as a 64-bit fraction of a turn, so p * theta_i modulo 2^64 is the
// angle modulo a turn, exactly, however far p is: one integer multiply instead of a
// reduction of a rounded product, and no table of angles in memory (a table of fp32
// sines and cosines would be read again for every token: 512 bytes beside the 12 KB
// of a 32 + 8 + 8 head token).
//
// Both are bound by memory: every row is read once and written once, 16 bytes a
// lane.  A thread takes one unit (two 16-byte chunks that hold the pairs' both
// halves) of one token through several heads, so that its sines and cosines are
// computed once for them.  Measured on a GB300: prompts of 32 + 8 heads rotated, 671 MB, 116 us
// (5.8 TB/s); q, K and V of prompts to q_out and an fp16 cache, 806 MB, 120 us (6.7 TB/s); 64 + 8 + 8
// heads into e4m3, 1.5 GB, 256 us.  A decode step takes 2.2 us, a launch's time; into e4m3 5.2: there a
// CTA works out a chunk's angles, waits for them at a barrier and only then looks at its slots.
#include <cuda_runtime.h>

#include "blocks_common.cuh"

namespace pkv {
namespace {

using namespace dev;

struct RopeParams {
    const void *q, *k, *v;        // rows [T][heads][D], a token's first element stride apart
    int64_t q_stride, k_stride, v_stride;
    const uint64_t *freqs;        // [rot / 2] turns a position, in units of 2^-64
    const int32_t *positions;     // [T]
    const int32_t *slots;         // [T]; null: rotate only
    void *q_out;                  // rotated q, a token's first element q_out_stride apart
    int64_t q_out_stride;
    void *k_cache, *v_cache;
    float *k_scales, *v_scales;   // 8-bit float caches
    unsigned int *err;
    int64_t num_tokens, num_slots;
    int rot, num_q_heads, num_kv_heads, block_size;
    float magnitude;
    float sign;                   // -1: the transposed rotation
    int slices;                   // threads that share a token's heads, for each unit
    int run_ctas;                 // CTAs of an 8-bit float cache's runs (the others: rotated rows)
    int every;                    // one of them among so many CTAs
    int parts;                    // of them, to a chunk of tokens: 8 (K or V, head)s each
    int chunk;                    // tokens that are looked at for runs
};

// Tokens whose sines and cosines a CTA of runs keeps in shared memory: those of its chunk and
// of a run that goes on behind it (of blocks of up to 32 tokens; of larger ones the tokens
// behind are worked out by each warp).
constexpr int TABLE_TOKENS = 64;

// A unit: V pairs of channels, in two 16-byte chunks at elements a and b of the
// head.  Halves: the chunks are V channels of either half.  Interleaved: they are
// neighbours, and each holds whole pairs.
template <typename T, int D>
struct Unit {
    static constexpr int V = 16 / (int)sizeof(T);
    static constexpr int N = D / (2 * V);              // units of a head
};

template <typename T, int D, bool IL>
__device__ __forceinline__ void unit_at(int u, int rot, int &a, int &b, bool &turned)
{
    constexpr int V = Unit<T, D>::V;
    const int nrot = rot / (2 * V);
    turned = u < nrot;
    if (IL || !turned) {                               // (channels behind the rotated ones likewise)
        a = 2 * u * V;
        b = a + V;
    } else {
        a = u * V;
        b = rot / 2 + a;
    }
}

__device__ __forceinline__ void get_row16(const uint4 &w, float (&x)[8], __half)
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = half2_to_float2(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void get_row16(const uint4 &w, float (&x)[8], __nv_bfloat16)
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(v[i]);
        x[2 * i + 1] = bf16hi(v[i]);
    }
}
__device__ __forceinline__ void get_row16(const uint4 &w, float (&x)[4], float)
{
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ uint32_t two(float lo, float hi, __half)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t two(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 put_row16(const float (&x)[8])
{
    return make_uint4(two(x[0], x[1], T()), two(x[2], x[3], T()), two(x[4], x[5], T()),
                      two(x[6], x[7], T()));
}
template <typename T>
__device__ __forceinline__ uint4 put_row16(const float (&x)[4])
{
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
}

// Cosines and sines (times the magnitude) of V pairs, or of a unit's, at a position.  The
// angle is taken as a number of quarter turns and a rest of at most an eighth, 32 bits of it
// (cut off below 2^-34 turns: 3.7e-10 in a sine): rounded to fp32 the rest is within 2.4e-8, half
// a step of a sine's own (a fraction of a whole turn would be off by four times that).
template <int V>
__device__ __forceinline__ void turns_at(const RopeParams &p, int pair, int32_t pos, float (&c)[V],
                                         float (&s)[V])
{
    const uint64_t *f = p.freqs + pair;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(f + i);
        const uint64_t t[2] = {w.x * (uint64_t)(int64_t)pos, w.y * (uint64_t)(int64_t)pos};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t n = ((uint32_t)(t[j] >> 32) + 0x20000000u) >> 30;     // quarters, 0..3
            const float x = (float)(int32_t)(uint32_t)(t[j] >> 30) * 0x1p-33f;   // half turns
            float sn, cs;
            sincospif(x, &sn, &cs);
            const uint32_t a = __float_as_uint(n & 1 ? sn : cs), b = __float_as_uint(n & 1 ? cs : sn);
            c[i + j] = __uint_as_float(a ^ ((n + 1) & 2) << 30) * p.magnitude;
            s[i + j] = __uint_as_float(b ^ (n & 2) << 30) * (p.magnitude * p.sign);
        }
    }
}

template <int V>
__device__ __forceinline__ void turns(const RopeParams &p, int u, int32_t pos, float (&c)[V],
                                      float (&s)[V])
{
    turns_at<V>(p, u * V, pos, c, s);
}

// The unit's pairs in xa, xb (its two chunks), rotated in place.
template <int V, bool IL>
__device__ __forceinline__ void turn(float (&xa)[V], float (&xb)[V], const float (&c)[V],
                                     const float (&s)[V])
{
    if constexpr (IL) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float a = xa[2 * i], b = xa[2 * i + 1];
            xa[2 * i] = fmaf(a, c[i], -(b * s[i]));
            xa[2 * i + 1] = fmaf(b, c[i], a * s[i]);
            const float d = xb[2 * i], e = xb[2 * i + 1];
            xb[2 * i] = fmaf(d, c[V / 2 + i], -(e * s[V / 2 + i]));
            xb[2 * i + 1] = fmaf(e, c[V / 2 + i], d * s[V / 2 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = xa[i], b = xb[i];
            xa[i] = fmaf(a, c[i], -(b * s[i]));
            xb[i] = fmaf(b, c[i], a * s[i]);
        }
    }
}

// Heads of one token, unit by unit: q's to q_out and, over a cache of T itself
// (HEADS_KV), K's and V's to their slot.
template <typename T, int D, bool IL, bool HEADS_KV>
__device__ __forceinline__ void rope_rows(const RopeParams &p, int cta)
{
    using U = Unit<T, D>;
    constexpr int V = U::V, UNROLL = 4;
    const int64_t g = (int64_t)cta * blockDim.x + threadIdx.x;
    const int u = (int)(g % U::N);
    const int64_t rest = g / U::N;
    const int64_t t = rest / p.slices;
    if (t >= p.num_tokens)
        return;
    const int slice = (int)(rest - t * p.slices);
    int slot = 0;
    if (p.slots) {
        slot = p.slots[t];
        if (slot < 0)
            return;
        if ((int64_t)slot >= p.num_slots) {
            if (u == 0 && slice == 0)
                atomicOr(p.err, PKV_EBIT_SLOT);
            return;
        }
    }
    int a, b;
    bool turned;
    unit_at<T, D, IL>(u, p.rot, a, b, turned);
    const int Hq = p.num_q_heads, H = p.num_kv_heads;
    const int heads = HEADS_KV ? Hq + 2 * H : Hq;
    const T *q = static_cast<const T *>(p.q) + t * p.q_stride;
    const T *k = HEADS_KV ? static_cast<const T *>(p.k) + t * p.k_stride : nullptr;
    const T *v = HEADS_KV ? static_cast<const T *>(p.v) + t * p.v_stride : nullptr;
    T *qo = static_cast<T *>(p.q_out) + t * p.q_out_stride;
    // the cached row of KV head 0
    const int64_t row = HEADS_KV ? ((int64_t)(slot / p.block_size) * H * p.block_size +
                                    slot % p.block_size) * D
                                 : 0;
    const int64_t head_step = (int64_t)p.block_size * D;
    T *kc = HEADS_KV ? static_cast<T *>(p.k_cache) + row : nullptr;
    T *vc = HEADS_KV ? static_cast<T *>(p.v_cache) + row : nullptr;
    float c[V], s[V];
    if (turned)
        turns<V>(p, u, p.positions[t], c, s);
    for (int h0 = slice; h0 < heads; h0 += UNROLL * p.slices) {
        uint4 wa[UNROLL], wb[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int h = h0 + i * p.slices;
            if (h < heads) {
                const T *src = h < Hq ? q + (int64_t)h * D
                               : h < Hq + H ? k + (int64_t)(h - Hq) * D : v + (int64_t)(h - Hq - H) * D;
                wa[i] = *reinterpret_cast<const uint4 *>(src + a);
                wb[i] = *reinterpret_cast<const uint4 *>(src + b);
            }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int h = h0 + i * p.slices;
            if (h < heads) {
                if (turned && h < Hq + H) {
                    float xa[V], xb[V];
                    get_row16(wa[i], xa, T());
                    get_row16(wb[i], xb, T());
                    turn<V, IL>(xa, xb, c, s);
                    wa[i] = put_row16<T>(xa);          // rounded once, to the rows' own type
                    wb[i] = put_row16<T>(xb);
                }
                T *dst = h < Hq ? qo + (int64_t)h * D
                         : h < Hq + H ? kc + (h - Hq) * head_step : vc + (h - Hq - H) * head_step;
                *reinterpret_cast<uint4 *>(dst + a) = wa[i];
                *reinterpret_cast<uint4 *>(dst + b) = wb[i];
            }
        }
    }
}

template <typename T, int D, bool IL, bool HEADS_KV>
__global__ void __launch_bounds__(256) rope_rows_kernel(const __grid_constant__ RopeParams p)
{
    grid_dependency_wait();
    grid_dependents_launch();
    rope_rows<T, D, IL, HEADS_KV>(p, blockIdx.x);
}

// K or V rows of one run into an 8-bit float cache, by one warp: as kv_append does
// (the run's largest magnitude gives the exponent, a block's exponent only grows),
// but of K's rotated values, in fp32: they are rounded once, to their codes.  The
// rows of a run of up to 16 stay in registers between the maximum and the codes;
// of a longer run they are read and rotated twice.
template <typename T, int D, bool IL>
__device__ __forceinline__ void rope_run(const RopeParams &p, const float2 *table, int64_t t0,
                                         bool is_v, int h, int64_t t, int blk, int off, int n)
{
    using U = Unit<T, D>;
    constexpr int V = U::V, RPI = 32 / U::N, ROWS = 16, NR = ROWS / RPI;
    const int lane = threadIdx.x & 31, u = lane % U::N, r0 = lane / U::N;
    int a, b;
    bool turned;
    unit_at<T, D, IL>(u, p.rot, a, b, turned);
    turned = turned && !is_v;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const T *src = static_cast<const T *>(is_v ? p.v : p.k) + t * stride + (int64_t)h * D;
    const int64_t head = (int64_t)blk * p.num_kv_heads + h;
    uint8_t *rows = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + head * p.block_size * D;
    float *scale = (is_v ? p.v_scales : p.k_scales) + head;
    const int e_old = off > 0 ? block_exponent(*scale) : BLOCK_MIN_EXP;
    float xa[NR][V], xb[NR][V];
    auto load = [&](int k0) {
        uint4 wa[NR], wb[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int k = k0 + i * RPI + r0;
            const T *row = src + k * stride;
            wa[i] = k < n ? *reinterpret_cast<const uint4 *>(row + a) : make_uint4(0u, 0u, 0u, 0u);
            wb[i] = k < n ? *reinterpret_cast<const uint4 *>(row + b) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int k = k0 + i * RPI + r0;
            get_row16(wa[i], xa[i], T());
            get_row16(wb[i], xb[i], T());
            if (turned && k < n) {
                float c[V], s[V];
                const int row = (int)(t - t0) + k;
                if (row < TABLE_TOKENS) {
                    const float4 *w = reinterpret_cast<const float4 *>(table + row * (p.rot / 2) + u * V);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        const float4 f = w[e];
                        c[2 * e] = f.x; s[2 * e] = f.y; c[2 * e + 1] = f.z; s[2 * e + 1] = f.w;
                    }
                } else {
                    turns<V>(p, u, p.positions[t + k], c, s);
                }
                turn<V, IL>(xa[i], xb[i], c, s);
            }
        }
    };
    float amax = 0.0f;
    for (int k0 = n > ROWS ? (n - 1) / ROWS * ROWS : 0; k0 >= 0; k0 -= ROWS) {
        load(k0);
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                amax = fmaxf(amax, fmaxf(fabsf(xa[i][j]), fabsf(xb[i][j])));
    }
    int e = code_exponent(warp_max(amax));
    if (off > 0) {
        if (e > e_old)
            rescale_rows(rows, off * (D / 16), e_old - e);
        else
            e = e_old;
    }
    __syncwarp();                                          // every lane has read the scale
    if (lane == 0)
        *scale = pow2_f32(e);
    const float f = pow2_f32(-e);
    for (int k0 = 0; k0 < n; k0 += ROWS) {
        if (k0 > 0)
            load(k0);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int k = k0 + i * RPI + r0;
            if (k < n) {
                uint8_t *dst = rows + (off + k) * D;
                uint32_t wa[V / 4], wb[V / 4];
#pragma unroll
                for (int j = 0; j < V / 4; ++j) {
                    wa[j] = f8_pack(xa[i][4 * j] * f, xa[i][4 * j + 1] * f) |
                            f8_pack(xa[i][4 * j + 2] * f, xa[i][4 * j + 3] * f) << 16;
                    wb[j] = f8_pack(xb[i][4 * j] * f, xb[i][4 * j + 1] * f) |
                            f8_pack(xb[i][4 * j + 2] * f, xb[i][4 * j + 3] * f) << 16;
                }
                if constexpr (V == 8) {
                    *reinterpret_cast<uint2 *>(dst + a) = make_uint2(wa[0], wa[1]);
                    *reinterpret_cast<uint2 *>(dst + b) = make_uint2(wb[0], wb[1]);
                } else {
                    *reinterpret_cast<uint32_t *>(dst + a) = wa[0];
                    *reinterpret_cast<uint32_t *>(dst + b) = wb[0];
                }
            }
        }
    }
}

// One launch for both: in some CTAs a warp takes runs of a chunk of tokens for one (K or
// V, head), the others rotate q.  They are spread evenly over the grid, so that the arithmetic of
// the runs goes beside the rows' memory traffic.  A chunk's sines and cosines are worked
// out once for all its heads.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(256, 2) rope_append_f8_kernel(const __grid_constant__ RopeParams p)
{
    extern __shared__ __align__(16) float2 table[];        // [TABLE_TOKENS][rot / 2]: cosine, sine
    grid_dependency_wait();
    grid_dependents_launch();
    // every `every`-th CTA until there are run_ctas of them
    const int cta = (int)blockIdx.x, run = cta / p.every;
    if (run * p.every != cta || run >= p.run_ctas) {
        rope_rows<T, D, IL, false>(p, cta - min(p.run_ctas, run + 1));
        return;
    }
    const int H = p.num_kv_heads, warp = threadIdx.x >> 5;
    const int64_t chunk = run / p.parts, t0 = chunk * p.chunk;
    const int r0 = (int)(run - chunk * p.parts) * 8;
    if (r0 < H) {                                          // (K among them)
        const int pairs = p.rot / 2;
        const int rows = (int)min((int64_t)min(TABLE_TOKENS, p.chunk + p.block_size - 1),
                                  p.num_tokens - t0);
        for (int i = threadIdx.x; i < rows * pairs / 2; i += 256) {
            const int row = 2 * i / pairs, pair = 2 * i - row * pairs;
            float c[2], s[2];
            turns_at<2>(p, pair, p.positions[t0 + row], c, s);
            *reinterpret_cast<float4 *>(table + 2 * i) = make_float4(c[0], s[0], c[1], s[1]);
        }
    }
    __syncthreads();
    const int r = r0 + warp;
    if (r >= 2 * H)
        return;
    const bool is_v = r >= H;
    for_runs(p.slots, t0, p.chunk, p.num_tokens, p.block_size, p.num_slots, r == 0, p.err,
             [&](int64_t t, int blk, int off, int n) {
                 rope_run<T, D, IL>(p, table, t0, is_v, is_v ? r - H : r, t, blk, off, n);
             });
}

// How many threads share a token's heads.  A thread's sines and cosines cost it about
// as much as five heads' rows, so a large batch gives each thread several heads (8); a small one
// spreads them, for the latency, until about 2048 threads an SM are there.
int head_slices(int64_t tokens, int units, int heads, int num_sms)
{
    int s = (heads + 7) / 8;
    while (s < heads && tokens * units * s < (int64_t)num_sms * 2048)
        s = s * 2 < heads ? s * 2 : heads;
    return s;
}

template <typename T, int D, bool IL>
int launch_rows(RopeParams &p, int num_sms, cudaStream_t s)
{
    const int heads = p.num_q_heads + (p.slots ? 2 * p.num_kv_heads : 0);
    p.slices = head_slices(p.num_tokens, Unit<T, D>::N, heads, num_sms);
    const int64_t ctas = (p.num_tokens * Unit<T, D>::N * p.slices + 255) / 256;
    if (ctas > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    const cudaError_t e =
        p.slots ? launch_pdl(rope_rows_kernel<T, D, IL, true>, dim3((unsigned)ctas), dim3(256), 0, s, p)
                : launch_pdl(rope_rows_kernel<T, D, IL, false>, dim3((unsigned)ctas), dim3(256), 0, s, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, int D, bool IL>
int launch_f8(RopeParams &p, int num_sms, cudaStream_t s)
{
    p.slices = p.num_q_heads ? head_slices(p.num_tokens, Unit<T, D>::N, p.num_q_heads, num_sms) : 0;
    const int64_t rows = (p.num_tokens * Unit<T, D>::N * p.slices + 255) / 256;
    // as kv_append: a token at a time while that keeps the warps few, else 32
    p.chunk = p.num_tokens * 2 * p.num_kv_heads <= (int64_t)num_sms * 64 ? 1 : 32;
    p.parts = (2 * p.num_kv_heads + 7) / 8;
    const int64_t runs = (p.num_tokens + p.chunk - 1) / p.chunk * p.parts;
    if (rows + runs > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    p.run_ctas = (int)runs;
    p.every = (int)((rows + runs) / runs);
    const size_t smem = (size_t)TABLE_TOKENS * (p.rot / 2) * sizeof(float2);   // at most 32 KB
    const cudaError_t e = launch_pdl(rope_append_f8_kernel<T, D, IL>, dim3((unsigned)(rows + runs)),
                                     dim3(256), smem, s, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, int D>
int launch_layout(RopeParams &p, bool interleaved, bool f8, int num_sms, cudaStream_t s)
{
    if (f8)
        return interleaved ? launch_f8<T, D, true>(p, num_sms, s) : launch_f8<T, D, false>(p, num_sms, s);
    return interleaved ? launch_rows<T, D, true>(p, num_sms, s) : launch_rows<T, D, false>(p, num_sms, s);
}

int launch_typed(RopeParams &p, pkv_dtype dtype, int head_dim, bool interleaved, bool f8,
                 int num_sms, cudaStream_t s)
{
    if (head_dim == 128) {
        if (dtype == PKV_F16) return launch_layout<__half, 128>(p, interleaved, f8, num_sms, s);
        if (dtype == PKV_BF16) return launch_layout<__nv_bfloat16, 128>(p, interleaved, f8, num_sms, s);
        return launch_layout<float, 128>(p, interleaved, f8, num_sms, s);
    }
    if (dtype == PKV_F16) return launch_layout<__half, 64>(p, interleaved, f8, num_sms, s);
    if (dtype == PKV_BF16) return launch_layout<__nv_bfloat16, 64>(p, interleaved, f8, num_sms, s);
    return launch_layout<float, 64>(p, interleaved, f8, num_sms, s);
}

RopeParams rope_params(const pkv_rope *rope, const int32_t *positions, int num_tokens)
{
    RopeParams p{};
    p.freqs = rope->freqs;
    p.rot = rope->rot_dim;
    p.magnitude = rope->magnitude;
    p.sign = 1.0f;
    p.positions = positions;
    p.num_tokens = num_tokens;
    return p;
}

}  // namespace

int launch_rope_rotate(const pkv_rope *rope, const void *x, int64_t x_stride, pkv_dtype dtype,
                       int num_heads, int head_dim, const int32_t *positions, int num_tokens,
                       bool transposed, void *out, int64_t out_stride, int num_sms,
                       pkv_stream_t stream)
{
    RopeParams p = rope_params(rope, positions, num_tokens);
    p.q = x;
    p.q_stride = x_stride;
    p.num_q_heads = num_heads;
    p.q_out = out;
    p.q_out_stride = out_stride;
    p.sign = transposed ? -1.0f : 1.0f;
    return launch_typed(p, dtype, head_dim, rope->layout == PKV_ROPE_INTERLEAVED, false, num_sms,
                        reinterpret_cast<cudaStream_t>(stream));
}

int launch_rope_append(const pkv_pool *pool, const pkv_rope *rope, const void *q,
                       int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                       int64_t v_stride, pkv_dtype in_dtype, int num_q_heads,
                       const int32_t *positions, const int32_t *slots, int num_tokens,
                       void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
                       void *k_scales, void *v_scales, pkv_stream_t stream)
{
    RopeParams p = rope_params(rope, positions, num_tokens);
    p.q = q;
    p.q_stride = q_stride;
    p.num_q_heads = num_q_heads;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.k = k;
    p.k_stride = k_stride;
    p.v = v;
    p.v_stride = v_stride;
    p.num_kv_heads = pool->num_kv_heads;
    p.block_size = pool->block_size;
    p.num_slots = (int64_t)pool->num_blocks * pool->block_size;
    p.slots = slots;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scales = static_cast<float *>(k_scales);
    p.v_scales = static_cast<float *>(v_scales);
    p.err = pool->d_err;
    return launch_typed(p, in_dtype, pool->head_dim, rope->layout == PKV_ROPE_INTERLEAVED,
                        pool->kv_dtype == PKV_F8, pool->num_sms,
                        reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace pkv
