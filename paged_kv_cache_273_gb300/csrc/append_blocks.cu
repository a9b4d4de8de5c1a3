// Appends that keep state per block rather than per row: kv_append on 8-bit
// float caches (PKV_F8: e4m3 codes, one power-of-two scale for each (block, KV
// head) of K and of V; "KV cache: the engine behind fast LLM inference",
// "Quantized KV cache") and kv_bounds_append (int8 lower and upper bounds of a
// block's keys).
//
// A run is the call's consecutive new rows of one block.  One warp handles a
// run of one head: the run's largest magnitude gives an exponent; a run that
// starts a block sets the block's, a later one can only raise it, and when it
// does, what the block holds is brought to the new exponent first.  Powers of
// two make that step lossless for e4m3 codes down to their subnormals, and
// for the bounds it commutes with their rounding (a floor of a floor by powers
// of two is the floor of the whole), so the bounds do not depend on how a
// prompt was cut into calls.
//
// Bytes moved are the rows in and the codes (bounds) out, once each: a run's
// rows stay in registers between the maximum and the rounding.
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pkv {
namespace {

using namespace dev;

// The least e >= BLOCK_MIN_EXP with amax <= 448 * 2^e, the largest e4m3 value
// being 448 = 1.75 * 2^8 (amax finite, >= 0).
__device__ __forceinline__ int code_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, BLOCK_MIN_EXP), BLOCK_MAX_EXP);
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        x = fmaxf(x, __shfl_xor_sync(FULL_MASK, x, m));
    return x;
}

// E consecutive input values of a row, raw, and as floats.
template <typename T, int E>
struct alignas(sizeof(T) * E) Raw {
    T v[E];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Rows of a run that are held in registers at once.
constexpr int ROWS = 16;

// For every run that starts at a token of [t0, t0 + C) (C <= 32), in order:
// f(first token, block, first offset in the block, rows).  All lanes call f
// together.  `report`: record slots beyond the cache.
template <typename F>
__device__ __forceinline__ void for_runs(const int32_t *slots, int64_t t0, int C, int64_t T,
                                         int bs, int64_t num_slots, bool report,
                                         unsigned int *err, F f)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = t0 + lane;
    const int s = lane < C && t < T ? __ldg(slots + t) : -1;
    int before = __shfl_up_sync(FULL_MASK, s, 1);
    if (lane == 0)
        before = t0 > 0 ? __ldg(slots + t0 - 1) : -1;
    if (report && s >= 0 && (int64_t)s >= num_slots)
        atomicOr(err, PKV_EBIT_SLOT);
    const bool starts = s >= 0 && (int64_t)s < num_slots &&
                        (before != s - 1 || (s & (bs - 1)) == 0);
    unsigned todo = __ballot_sync(FULL_MASK, starts);
    while (todo) {
        const int i = __ffs(todo) - 1;
        todo &= todo - 1;
        const int slot = __shfl_sync(FULL_MASK, s, i);
        const int off = slot & (bs - 1);
        int n = 1;                                   // rows of the run
        for (;;) {
            const int64_t tn = t0 + i + n + lane;
            const bool more = off + n + lane < bs && tn < T && __ldg(slots + tn) == slot + n + lane;
            const unsigned gap = ~__ballot_sync(FULL_MASK, more);
            if (gap) {
                n += __ffs(gap) - 1;
                break;
            }
            n += 32;
        }
        f(t0 + i, slot / bs, off, n);
    }
}

// One warp per (chunk of C tokens, K or V, head).
template <typename T, int E>
__global__ void __launch_bounds__(256) append_f8_kernel(
    const T *__restrict__ k_new, const T *__restrict__ v_new, const int32_t *__restrict__ slots,
    int64_t num_tokens, int C, int num_kv_heads, int block_size, int64_t num_slots,
    uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache, float *__restrict__ k_scales,
    float *__restrict__ v_scales, unsigned int *__restrict__ err)
{
    constexpr int D = 32 * E;
    using R = Raw<T, E>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int H = num_kv_heads;
    const int64_t chunks = (num_tokens + C - 1) / C;
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < chunks * 2 * H;
         w += nwarps) {
        const int64_t chunk = w / (2 * H);
        const int r = (int)(w - chunk * 2 * H);
        const bool is_v = r >= H;
        const int h = is_v ? r - H : r;
        const T *src = (is_v ? v_new : k_new);
        uint8_t *cache = is_v ? v_cache : k_cache;
        float *scales = is_v ? v_scales : k_scales;
        auto encode = [&](const float (&x)[E], uint8_t *dst) {
            uint32_t word = f8_pack(x[0], x[1]);
            if constexpr (E == 4) {
                word |= (uint32_t)f8_pack(x[2], x[3]) << 16;
                *reinterpret_cast<uint32_t *>(dst) = word;
            } else {
                *reinterpret_cast<uint16_t *>(dst) = (uint16_t)word;
            }
        };
        for_runs(slots, chunk * C, C, num_tokens, block_size, num_slots, r == 0, err,
                 [&](int64_t t, int blk, int off, int n) {
            const R *in = reinterpret_cast<const R *>(src + (t * H + h) * D) + lane;
            const int64_t step = (int64_t)H * 32;              // R's from row to row
            const int64_t head = (int64_t)blk * H + h;
            uint8_t *rows = cache + head * block_size * D + lane * E;
            R x[ROWS];
            float amax = 0.0f;
            // the largest magnitude of the run; its first ROWS rows stay in x
            for (int k0 = n > ROWS ? (n - 1) / ROWS * ROWS : 0; k0 >= 0; k0 -= ROWS) {
#pragma unroll
                for (int k = 0; k < ROWS; ++k)
                    if (k0 + k < n)
                        x[k] = in[(k0 + k) * step];
#pragma unroll
                for (int k = 0; k < ROWS; ++k)
                    if (k0 + k < n)
#pragma unroll
                        for (int u = 0; u < E; ++u)
                            amax = fmaxf(amax, fabsf(to_f(x[k].v[u])));
            }
            int e = code_exponent(warp_max(amax));
            if (off > 0) {
                const int e_old = block_exponent(scales[head]);
                if (e > e_old) {
                    // the block's older rows at its new scale
                    const float f = pow2_f32(max(e_old - e, -126));
                    for (int k = 0; k < off; ++k) {
                        uint8_t *p = rows + k * D;
                        float y[E];
                        if constexpr (E == 4) {
                            const uint32_t word = *reinterpret_cast<const uint32_t *>(p);
                            f8_unpack(word & 0xffffu, y[0], y[1]);
                            f8_unpack(word >> 16, y[2], y[3]);
                        } else {
                            f8_unpack(*reinterpret_cast<const uint16_t *>(p), y[0], y[1]);
                        }
#pragma unroll
                        for (int u = 0; u < E; ++u)
                            y[u] *= f;
                        encode(y, p);
                    }
                } else {
                    e = e_old;
                }
            }
            __syncwarp();                                      // every lane has read the scale
            if (lane == 0)
                scales[head] = pow2_f32(e);
            const float f = pow2_f32(-e);
            for (int k0 = 0; k0 < n; k0 += ROWS) {
                if (k0 > 0) {
#pragma unroll
                    for (int k = 0; k < ROWS; ++k)
                        if (k0 + k < n)
                            x[k] = in[(k0 + k) * step];
                }
#pragma unroll
                for (int k = 0; k < ROWS; ++k)
                    if (k0 + k < n) {
                        float y[E];
#pragma unroll
                        for (int u = 0; u < E; ++u)
                            y[u] = to_f(x[k].v[u]) * f;
                        encode(y, rows + (off + k0 + k) * D);
                    }
            }
        });
    }
}

// One warp per (chunk of C tokens, head).  bounds [NB][Hkv][2][D]: the
// minima rounded down, then the maxima rounded up, in units of 2^exps.
template <typename T, int E>
__global__ void __launch_bounds__(256) append_bounds_kernel(
    const T *__restrict__ k_new, const int32_t *__restrict__ slots, int64_t num_tokens, int C,
    int num_kv_heads, int block_size, int64_t num_slots, int8_t *__restrict__ bounds,
    int32_t *__restrict__ exps, unsigned int *__restrict__ err)
{
    constexpr int D = 32 * E;
    using R = Raw<T, E>;
    using C8 = Raw<int8_t, E>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int H = num_kv_heads;
    const int64_t chunks = (num_tokens + C - 1) / C;
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < chunks * H;
         w += nwarps) {
        const int64_t chunk = w / H;
        const int h = (int)(w - chunk * H);
        for_runs(slots, chunk * C, C, num_tokens, block_size, num_slots, h == 0, err,
                 [&](int64_t t, int blk, int off, int n) {
            const R *in = reinterpret_cast<const R *>(k_new + (t * H + h) * D) + lane;
            const int64_t step = (int64_t)H * 32;
            const int64_t head = (int64_t)blk * H + h;
            C8 *lo_p = reinterpret_cast<C8 *>(bounds + head * 2 * D) + lane;
            C8 *hi_p = lo_p + 32;
            float lo[E], hi[E];
#pragma unroll
            for (int u = 0; u < E; ++u) {
                lo[u] = INFINITY;
                hi[u] = -INFINITY;
            }
            for (int k0 = 0; k0 < n; k0 += 8) {
                R x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < n)
                        x[k] = in[(k0 + k) * step];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < n)
#pragma unroll
                        for (int u = 0; u < E; ++u) {
                            const float y = to_f(x[k].v[u]);
                            lo[u] = fminf(lo[u], y);
                            hi[u] = fmaxf(hi[u], y);
                        }
            }
            float amax = 0.0f;
#pragma unroll
            for (int u = 0; u < E; ++u)
                amax = fmaxf(amax, fmaxf(fabsf(lo[u]), fabsf(hi[u])));
            int e = int8_exponent(warp_max(amax));
            int e_old = e;
            if (off > 0) {
                e_old = min(max(exps[head], BLOCK_MIN_EXP), BLOCK_MAX_EXP);
                e = max(e, e_old);
            }
            __syncwarp();
            if (lane == 0)
                exps[head] = e;
            const float f = pow2_f32(-e);
            C8 l8, h8;
            int il[E], ih[E];
#pragma unroll
            for (int u = 0; u < E; ++u) {
                il[u] = __float2int_rd(lo[u] * f);
                ih[u] = __float2int_ru(hi[u] * f);
            }
            if (off > 0) {
                const C8 lw = *lo_p, hw = *hi_p;
                const int down = min(e - e_old, 31);
#pragma unroll
                for (int u = 0; u < E; ++u) {
                    il[u] = min(il[u], (int)lw.v[u] >> down);
                    ih[u] = max(ih[u], -((-(int)hw.v[u]) >> down));
                }
            }
#pragma unroll
            for (int u = 0; u < E; ++u) {
                l8.v[u] = (int8_t)max(il[u], -128);
                h8.v[u] = (int8_t)min(ih[u], 127);
            }
            *lo_p = l8;
            *hi_p = h8;
        });
    }
}

// Tokens a warp looks for runs in: one while that keeps every SM's warps few
// (a decode step: every token is a run of its own), else 32, so that a bulk
// write's warps find a whole block's run each and few find none.
int chunk_tokens(int64_t warps_at_one, int num_sms)
{
    return warps_at_one <= (int64_t)num_sms * 64 ? 1 : 32;
}

int grid_for(int64_t warps, int num_sms)
{
    const int64_t blocks = (warps + 7) / 8, cap = (int64_t)num_sms * 8;
    return (int)(blocks < 1 ? 1 : blocks > cap ? cap : blocks);
}

}  // namespace

int launch_append_f8(const pkv_pool *pool, const void *k_new, const void *v_new,
                     pkv_dtype in_dtype, const int32_t *slots, int num_tokens, void *k_cache,
                     void *v_cache, void *k_scales, void *v_scales, pkv_stream_t stream)
{
    const int H = pool->num_kv_heads, bs = pool->block_size;
    const int64_t T = num_tokens, num_slots = (int64_t)pool->num_blocks * bs;
    const int C = chunk_tokens(T * 2 * H, pool->num_sms);
    const int grid = grid_for((T + C - 1) / C * 2 * H, pool->num_sms);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PKV_A8(T_, E)                                                                            \
    launch_pdl(append_f8_kernel<T_, E>, dim3(grid), dim3(256), 0, s,                              \
               static_cast<const T_ *>(k_new), static_cast<const T_ *>(v_new), slots, T, C, H,    \
               bs, num_slots, static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache),   \
               static_cast<float *>(k_scales), static_cast<float *>(v_scales), pool->d_err)
    if (pool->head_dim == 128) {
        if (in_dtype == PKV_F16) PKV_A8(__half, 4);
        else if (in_dtype == PKV_BF16) PKV_A8(__nv_bfloat16, 4);
        else PKV_A8(float, 4);
    } else {
        if (in_dtype == PKV_F16) PKV_A8(__half, 2);
        else if (in_dtype == PKV_BF16) PKV_A8(__nv_bfloat16, 2);
        else PKV_A8(float, 2);
    }
#undef PKV_A8
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int launch_append_bounds(const pkv_pool *pool, const void *k_new, pkv_dtype in_dtype,
                         const int32_t *slots, int num_tokens, int8_t *bounds, int32_t *exps,
                         pkv_stream_t stream)
{
    const int H = pool->num_kv_heads, bs = pool->block_size;
    const int64_t T = num_tokens, num_slots = (int64_t)pool->num_blocks * bs;
    const int C = chunk_tokens(T * H, pool->num_sms);
    const int grid = grid_for((T + C - 1) / C * H, pool->num_sms);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PKV_B8(T_, E)                                                                            \
    launch_pdl(append_bounds_kernel<T_, E>, dim3(grid), dim3(256), 0, s,                          \
               static_cast<const T_ *>(k_new), slots, T, C, H, bs, num_slots, bounds, exps,       \
               pool->d_err)
    if (pool->head_dim == 128) {
        if (in_dtype == PKV_F16) PKV_B8(__half, 4);
        else if (in_dtype == PKV_BF16) PKV_B8(__nv_bfloat16, 4);
        else PKV_B8(float, 4);
    } else {
        if (in_dtype == PKV_F16) PKV_B8(__half, 2);
        else if (in_dtype == PKV_BF16) PKV_B8(__nv_bfloat16, 2);
        else PKV_B8(float, 2);
    }
#undef PKV_B8
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
