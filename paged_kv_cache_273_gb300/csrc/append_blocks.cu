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

#include "blocks_common.cuh"

namespace pkv {
namespace {

using namespace dev;

// 16 bytes of a row: 8 (16-bit types) or 4 (fp32) consecutive values.
template <typename T>
struct Row16;

// 16-bit types two to a word, minima and maxima on the packed pairs.
template <typename T2, bool BF>
struct Row16Pairs {
    static constexpr int N = 8;
    uint4 w;
    __device__ __forceinline__ static T2 as(uint32_t x) { return *reinterpret_cast<T2 *>(&x); }
    __device__ __forceinline__ static uint32_t bits(T2 x) { return *reinterpret_cast<uint32_t *>(&x); }
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) { return bits(__hmax2(as(a), as(b))); }
    __device__ __forceinline__ static uint32_t min2(uint32_t a, uint32_t b) { return bits(__hmin2(as(a), as(b))); }
    __device__ __forceinline__ static float2 pair(uint32_t x)
    {
        return BF ? make_float2(bf16lo(x), bf16hi(x)) : half2_to_float2(x);
    }
    __device__ __forceinline__ float amax() const
    {
        const uint32_t m = max2(max2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                max2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        const float2 f = pair(m);
        return fmaxf(f.x, f.y);
    }
    __device__ __forceinline__ void lower(const Row16Pairs &o)
    {
        w = make_uint4(min2(w.x, o.w.x), min2(w.y, o.w.y), min2(w.z, o.w.z), min2(w.w, o.w.w));
    }
    __device__ __forceinline__ void raise(const Row16Pairs &o)
    {
        w = make_uint4(max2(w.x, o.w.x), max2(w.y, o.w.y), max2(w.z, o.w.z), max2(w.w, o.w.w));
    }
    __device__ __forceinline__ void get(float (&x)[N]) const
    {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pair(v[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <> struct Row16<__half> : Row16Pairs<__half2, false> {};
template <> struct Row16<__nv_bfloat16> : Row16Pairs<__nv_bfloat162, true> {};

template <>
struct Row16<float> {
    static constexpr int N = 4;
    uint4 w;
    __device__ __forceinline__ void get(float (&x)[N]) const
    {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    __device__ __forceinline__ float amax() const
    {
        float x[4];
        get(x);
        return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    }
    __device__ __forceinline__ static uint32_t lo(uint32_t a, uint32_t b)
    {
        return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ __forceinline__ static uint32_t hi(uint32_t a, uint32_t b)
    {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ __forceinline__ void lower(const Row16 &o)
    {
        w = make_uint4(lo(w.x, o.w.x), lo(w.y, o.w.y), lo(w.z, o.w.z), lo(w.w, o.w.w));
    }
    __device__ __forceinline__ void raise(const Row16 &o)
    {
        w = make_uint4(hi(w.x, o.w.x), hi(w.y, o.w.y), hi(w.z, o.w.z), hi(w.w, o.w.w));
    }
};

__device__ __forceinline__ uint4 shfl_xor4(uint4 x, int m)
{
    return make_uint4(__shfl_xor_sync(FULL_MASK, x.x, m), __shfl_xor_sync(FULL_MASK, x.y, m),
                      __shfl_xor_sync(FULL_MASK, x.z, m), __shfl_xor_sync(FULL_MASK, x.w, m));
}

// How a warp reads rows: LPR lanes a row, 16 bytes each, RPI rows at once;
// NR such reads hold the 16 rows that stay in registers.
template <typename T, int D>
struct Rows {
    static constexpr int LPR = D * (int)sizeof(T) / 16;
    static constexpr int RPI = 32 / LPR;
    static constexpr int ROWS = 16;
    static constexpr int NR = ROWS / RPI;
};

// One warp per (chunk of C tokens, K or V, head).
template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) append_f8_kernel(
    const T *k_new, const T *v_new, const int32_t *slots, int64_t num_tokens, int C,
    int num_kv_heads, int block_size, int64_t num_slots, uint8_t *k_cache, uint8_t *v_cache,
    float *k_scales, float *v_scales, unsigned int *err)
{
    using A = Rows<T, D>;
    using X = Row16<T>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int r0 = lane / A::LPR, c = lane % A::LPR;
    const int H = num_kv_heads;
    const int64_t chunks = (num_tokens + C - 1) / C;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t chunk = w / (2 * H);
    if (chunk >= chunks)
        return;
    const int r = (int)(w - chunk * 2 * H);
    const bool is_v = r >= H;
    const int h = is_v ? r - H : r;
    const T *src = is_v ? v_new : k_new;
    uint8_t *cache = is_v ? v_cache : k_cache;
    float *scales = is_v ? v_scales : k_scales;
    for_runs(slots, chunk * C, C, num_tokens, block_size, num_slots, r == 0, err,
             [&](int64_t t, int blk, int off, int n) {
        const uint4 *in = reinterpret_cast<const uint4 *>(src + (t * H + h) * D) + c;
        const int64_t step = (int64_t)H * A::LPR;          // uint4s from row to row
        const int64_t head = (int64_t)blk * H + h;
        uint8_t *rows = cache + head * block_size * D;
        const int e_old = off > 0 ? block_exponent(scales[head]) : BLOCK_MIN_EXP;
        X x[A::NR];
        float amax = 0.0f;
        // the largest magnitude of the run; its first rows stay in x
        for (int k0 = n > A::ROWS ? (n - 1) / A::ROWS * A::ROWS : 0; k0 >= 0; k0 -= A::ROWS) {
#pragma unroll
            for (int i = 0; i < A::NR; ++i) {
                const int k = k0 + i * A::RPI + r0;
                x[i].w = k < n ? in[k * step] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < A::NR; ++i)
                amax = fmaxf(amax, x[i].amax());
        }
        int e = code_exponent(warp_max(amax));
        if (off > 0) {
            if (e > e_old) {
                rescale_rows(rows, off * (D / 16), e_old - e);
            } else {
                e = e_old;
            }
        }
        __syncwarp();                                      // every lane has read the scale
        if (lane == 0)
            scales[head] = pow2_f32(e);
        const float f = pow2_f32(-e);
        for (int k0 = 0; k0 < n; k0 += A::ROWS) {
            if (k0 > 0) {
#pragma unroll
                for (int i = 0; i < A::NR; ++i) {
                    const int k = k0 + i * A::RPI + r0;
                    if (k < n)
                        x[i].w = in[k * step];
                }
            }
#pragma unroll
            for (int i = 0; i < A::NR; ++i) {
                const int k = k0 + i * A::RPI + r0;
                if (k < n) {
                    float y[X::N];
                    x[i].get(y);
                    uint32_t v[X::N / 4];
#pragma unroll
                    for (int u = 0; u < X::N / 4; ++u)
                        v[u] = f8_pack(y[4 * u] * f, y[4 * u + 1] * f) |
                               f8_pack(y[4 * u + 2] * f, y[4 * u + 3] * f) << 16;
                    uint8_t *dst = rows + (off + k) * D + c * X::N;
                    if constexpr (X::N == 8)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(v[0], v[1]);
                    else
                        *reinterpret_cast<uint32_t *>(dst) = v[0];
                }
            }
        }
    });
}

// One warp per (chunk of C tokens, head).  bounds [NB][Hkv][2][D]: the
// minima rounded down, then the maxima rounded up, in units of 2^exps.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_bounds_kernel(
    const T *k_new, const int32_t *slots, int64_t num_tokens, int C, int num_kv_heads,
    int block_size, int64_t num_slots, int8_t *bounds, int32_t *exps, unsigned int *err)
{
    using A = Rows<T, D>;
    using X = Row16<T>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    const int r0 = lane / A::LPR, c = lane % A::LPR;
    const int H = num_kv_heads;
    const int64_t chunks = (num_tokens + C - 1) / C;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t chunk = w / H;
    if (chunk >= chunks)
        return;
    const int h = (int)(w - chunk * H);
    for_runs(slots, chunk * C, C, num_tokens, block_size, num_slots, h == 0, err,
             [&](int64_t t, int blk, int off, int n) {
        const uint4 *in = reinterpret_cast<const uint4 *>(k_new + (t * H + h) * D) + c;
        const int64_t step = (int64_t)H * A::LPR;
        const int64_t head = (int64_t)blk * H + h;
        // a lane group's bounds: N channels, r0 picks the lower or the upper ones
        int8_t *mine = bounds + (head * 2) * D + c * X::N;
        int e_old = 0;
        if (off > 0)
            e_old = min(max(exps[head], BLOCK_MIN_EXP), BLOCK_MAX_EXP);
        X lo, hi;
        for (int k0 = 0; k0 < n; k0 += A::ROWS) {
            X x[A::NR];
#pragma unroll
            for (int i = 0; i < A::NR; ++i)
                // (past the run's end its last row again: loads that no test holds back;
                // read once, evict first: 49 instead of 52 us for 131k rows)
                x[i].w = __ldcs(in + min(k0 + i * A::RPI + r0, n - 1) * step);
            if (k0 == 0)
                lo = hi = x[0];
#pragma unroll
            for (int i = 0; i < A::NR; ++i) {
                lo.lower(x[i]);
                hi.raise(x[i]);
            }
        }
#pragma unroll
        for (int m = A::LPR; m < 32; m <<= 1) {
            X l, u;
            l.w = shfl_xor4(lo.w, m);
            u.w = shfl_xor4(hi.w, m);
            lo.lower(l);
            hi.raise(u);
        }
        int e = int8_exponent(warp_max(fmaxf(lo.amax(), hi.amax())));
        if (off > 0)
            e = max(e, e_old);
        __syncwarp();
        if (lane == 0)
            exps[head] = e;
        if (r0 != 0)
            return;
        const float f = pow2_f32(-e);
        float l[X::N], u[X::N];
        lo.get(l);
        hi.get(u);
        int il[X::N], iu[X::N];
#pragma unroll
        for (int i = 0; i < X::N; ++i) {
            il[i] = __float2int_rd(l[i] * f);
            iu[i] = __float2int_ru(u[i] * f);
        }
        if (off > 0) {
            const int down = min(e - e_old, 31);
#pragma unroll
            for (int q = 0; q < X::N / 4; ++q) {
                const uint32_t wl = reinterpret_cast<const uint32_t *>(mine)[q];
                const uint32_t wu = reinterpret_cast<const uint32_t *>(mine + D)[q];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ol = (int8_t)(wl >> (8 * i)), ou = (int8_t)(wu >> (8 * i));
                    il[4 * q + i] = min(il[4 * q + i], ol >> down);
                    iu[4 * q + i] = max(iu[4 * q + i], -((-ou) >> down));
                }
            }
        }
#pragma unroll
        for (int q = 0; q < X::N / 4; ++q) {
            uint32_t wl = 0u, wu = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wl |= (uint32_t)(max(il[4 * q + i], -128) & 0xff) << (8 * i);
                wu |= (uint32_t)(min(iu[4 * q + i], 127) & 0xff) << (8 * i);
            }
            reinterpret_cast<uint32_t *>(mine)[q] = wl;
            reinterpret_cast<uint32_t *>(mine + D)[q] = wu;
        }
    });
}

// One thread a 16-byte chunk of a block's bounds, or a head's exponent: a copied
// block is a few KB, the launch is what it costs.
__global__ void __launch_bounds__(256) bounds_copy_kernel(
    const int32_t *src, const int32_t *dst, int64_t items, int chunks, int num_kv_heads,
    int num_blocks, uint4 *bounds, int32_t *exps, unsigned int *err)
{
    grid_dependency_wait();
    grid_dependents_launch();
    const int per = chunks + num_kv_heads;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < items; c += stride) {
        const int64_t i = c / per;
        const int r = (int)(c - i * per);
        const int32_t s = src[i], d = dst[i];
        if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
            if (r == 0)
                atomicOr(err, PKV_EBIT_BLOCK);
        } else if (r < chunks) {
            bounds[(int64_t)d * chunks + r] = bounds[(int64_t)s * chunks + r];
        } else {
            const int h = r - chunks;
            exps[(int64_t)d * num_kv_heads + h] = exps[(int64_t)s * num_kv_heads + h];
        }
    }
}

// Tokens a warp looks for runs in: one while that keeps every SM's warps few
// (a decode step: every token is a run of its own), else 32, so that a bulk
// write's warps find a run or two each and few find none (131k rows of 8 heads:
// 128 us at 32, 139 at 16).
int chunk_tokens(int64_t warps_at_one, int num_sms)
{
    return warps_at_one <= (int64_t)num_sms * 64 ? 1 : 32;
}

}  // namespace

int launch_append_f8(const pkv_pool *pool, const void *k_new, const void *v_new,
                     pkv_dtype in_dtype, const int32_t *slots, int num_tokens, void *k_cache,
                     void *v_cache, void *k_scales, void *v_scales, pkv_stream_t stream)
{
    const int H = pool->num_kv_heads, bs = pool->block_size;
    const int64_t T = num_tokens, num_slots = (int64_t)pool->num_blocks * bs;
    const int C = chunk_tokens(T * 2 * H, pool->num_sms);
    const int64_t grid = ((T + C - 1) / C * 2 * H + 7) / 8;     // 8 warps a CTA
    if (grid > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PKV_A8(T_, D)                                                                            \
    launch_pdl(append_f8_kernel<T_, D>, dim3((unsigned)grid), dim3(256), 0, s,                              \
               static_cast<const T_ *>(k_new), static_cast<const T_ *>(v_new), slots, T, C, H,    \
               bs, num_slots, static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache),   \
               static_cast<float *>(k_scales), static_cast<float *>(v_scales), pool->d_err)
    if (pool->head_dim == 128) {
        if (in_dtype == PKV_F16) PKV_A8(__half, 128);
        else if (in_dtype == PKV_BF16) PKV_A8(__nv_bfloat16, 128);
        else PKV_A8(float, 128);
    } else {
        if (in_dtype == PKV_F16) PKV_A8(__half, 64);
        else if (in_dtype == PKV_BF16) PKV_A8(__nv_bfloat16, 64);
        else PKV_A8(float, 64);
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
    const int64_t grid = ((T + C - 1) / C * H + 7) / 8;
    if (grid > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define PKV_B8(T_, D)                                                                            \
    launch_pdl(append_bounds_kernel<T_, D>, dim3((unsigned)grid), dim3(256), 0, s,                          \
               static_cast<const T_ *>(k_new), slots, T, C, H, bs, num_slots, bounds, exps,       \
               pool->d_err)
    if (pool->head_dim == 128) {
        if (in_dtype == PKV_F16) PKV_B8(__half, 128);
        else if (in_dtype == PKV_BF16) PKV_B8(__nv_bfloat16, 128);
        else PKV_B8(float, 128);
    } else {
        if (in_dtype == PKV_F16) PKV_B8(__half, 64);
        else if (in_dtype == PKV_BF16) PKV_B8(__nv_bfloat16, 64);
        else PKV_B8(float, 64);
    }
#undef PKV_B8
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int launch_bounds_copy(const pkv_pool *pool, const int32_t *src, const int32_t *dst, int n,
                       int8_t *bounds, int32_t *exps, pkv_stream_t stream)
{
    const int H = pool->num_kv_heads, chunks = H * 2 * pool->head_dim / 16;
    const int64_t items = (int64_t)n * (chunks + H);
    const int64_t grid = (items + 255) / 256, most = (int64_t)pool->num_sms * 8;
    launch_pdl(bounds_copy_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0,
               reinterpret_cast<cudaStream_t>(stream), src, dst, items, chunks, H,
               pool->num_blocks, reinterpret_cast<uint4 *>(bounds), exps, pool->d_err);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
