// K9a -- values to e4m3 with one fp32 scale per block of 1 x 128 or 128 x 128
// elements:
//   amax = max(max |x|, 2^-64) over the block,
//   scale = amax / 448,  q = e4m3(x * (448 / amax))       (448 = largest e4m3 value)
// with IEEE fp32 divisions and one rounding to nearest even, so the bytes are a
// function of the values alone.  The lower bound of amax keeps 448 / amax finite (a
// block of zeros gives zeros).  The maximum is taken over the bits of |x|, where a
// NaN is larger than every number: a block with a NaN gets a NaN scale.
//
// Memory-bound: x read once, q written once.  By rows, eight lanes hold a row block in
// 16-element pieces, so its maximum needs three shuffles and its bytes leave 16 at a time;
// two row blocks a lane are in flight at once.  The 128 x 128 block stays in registers (64
// values a thread, 8 side by side) between its maximum and its conversion.
// 16384 x 2048 bf16 by rows: 16.7 us in a graph (100.8 MB: 15.4 at the copy rate); 8513 x
// 2064 fp32 by tiles: 15.7 us (88 MB: 13.4; with 16 values side by side 16.4).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr float kFp8Max = 448.f;
constexpr float kTiny = 5.421010862427522e-20f;   // 2^-64

__device__ __forceinline__ uint32_t amax8(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ uint2 to_e4m3x8(const float (&x)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ float block_amax(uint32_t bits) {
    return __uint_as_float(max(bits, __float_as_uint(kTiny)));
}

// Eight elements as they were loaded (half the registers of their floats for bf16, so
// that more loads are in flight), and as floats.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    uint4 u;
    __device__ __forceinline__ void load(const bf16 *p) { u = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16lo(w[e]);
            x[2 * e + 1] = bf16hi(w[e]);
        }
    }
};
template <> struct Raw8<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p) { load8(p, v); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[e];
    }
};

// Eight lanes hold a row block, 16 elements each: two row blocks a lane 16.7 us (16384 x
// 2048 bf16), one 18.4, four 17.0; sixteen lanes of 8 elements, two row blocks: 20.2.
constexpr int QB = 2;

template <typename T>
__global__ void __launch_bounds__(256)
quant_rows_kernel(const T *__restrict__ x, long long ld_x, uint32_t n_blocks, int cols, uint32_t cb,
                  uint8_t *__restrict__ q, long long ld_q, float *__restrict__ scale) {
    const int sub = threadIdx.x & 7;
    const uint32_t first = (blockIdx.x * 32 + (threadIdx.x >> 3)) * QB;
    // row and column of these lanes' row blocks, which follow one another
    uint32_t r[QB], c[QB];
    r[0] = first / cb;
    c[0] = first - r[0] * cb;
#pragma unroll
    for (int i = 1; i < QB; ++i) {
        const bool wrap = c[i - 1] + 1 == cb;
        r[i] = r[i - 1] + wrap;
        c[i] = wrap ? 0 : c[i - 1] + 1;
    }
    Raw8<T> raw[QB][2];
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const int col = (int)c[i] * 128 + 16 * sub;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (first + i < n_blocks && col < cols) raw[i][k].load(x + r[i] * ld_x + col + 8 * k);
            else raw[i][k].zero();
        }
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        float v[2][8];
        raw[i][0].floats(v[0]);
        raw[i][1].floats(v[1]);
        uint32_t m = max(amax8(v[0]), amax8(v[1]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float amax = block_amax(m);
        const int col = (int)c[i] * 128 + 16 * sub;
        if (first + i < n_blocks) {
            if (sub == 0) scale[first + i] = __fdiv_rn(amax, kFp8Max);
            const float inv = __fdiv_rn(kFp8Max, amax);
            if (col < cols) {
                const uint2 a = to_e4m3x8(v[0], inv), b = to_e4m3x8(v[1], inv);
                *reinterpret_cast<uint4 *>(q + r[i] * ld_q + col) = make_uint4(a.x, a.y, b.x, b.y);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
quant_tiles_kernel(const T *__restrict__ x, long long ld_x, int rows, int cols, uint8_t *__restrict__ q,
                   long long ld_q, float *__restrict__ scale) {
    __shared__ uint32_t part[8];
    const int sub = threadIdx.x & 15, c = blockIdx.x * 128 + 8 * sub;
    const long long r0 = (long long)blockIdx.y * 128 + (threadIdx.x >> 4);
    Raw8<T> raw[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + 16 * i < rows && c < cols) raw[i].load(x + (r0 + 16 * i) * ld_x + c);
        else raw[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        raw[i].floats(v);
        m = max(m, amax8(v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, part[w]);
    const float amax = block_amax(m), inv = __fdiv_rn(kFp8Max, amax);
    if (threadIdx.x == 0) scale[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = __fdiv_rn(amax, kFp8Max);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (r0 + 16 * i < rows && c < cols) {
            float v[8];
            raw[i].floats(v);
            *reinterpret_cast<uint2 *>(q + (r0 + 16 * i) * ld_q + c) = to_e4m3x8(v, inv);
        }
}

template <typename T>
cudaError_t launch_quant(int rows, int cols, const void *x, long long ld_x, int block_rows, void *q, long long ld_q,
                         float *scale, cudaStream_t stream) {
    const int cb = (cols + 127) / 128;
    if (block_rows == 1) {
        const long long n = (long long)rows * cb, per_cta = 32 * QB;
        quant_rows_kernel<T><<<(unsigned)((n + per_cta - 1) / per_cta), 256, 0, stream>>>(
            static_cast<const T *>(x), ld_x, (uint32_t)n, cols, (uint32_t)cb, static_cast<uint8_t *>(q), ld_q, scale);
    } else {
        quant_tiles_kernel<T><<<dim3(cb, (rows + 127) / 128), 256, 0, stream>>>(
            static_cast<const T *>(x), ld_x, rows, cols, static_cast<uint8_t *>(q), ld_q, scale);
    }
    return launched();
}

}  // namespace

cudaError_t launch_quant_fp8(int rows, int cols, const void *x, long long ld_x, bool bf16_in, int block_rows,
                             void *q, long long ld_q, float *scale, cudaStream_t stream) {
    return bf16_in ? launch_quant<bf16>(rows, cols, x, ld_x, block_rows, q, ld_q, scale, stream)
                   : launch_quant<float>(rows, cols, x, ld_x, block_rows, q, ld_q, scale, stream);
}

}  // namespace gdn
