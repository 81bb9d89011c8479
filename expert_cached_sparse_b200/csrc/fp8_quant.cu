// e4m3 codes with float32 block scales: 1 x 128 blocks of activation rows
// (optionally of silu(gate) * up) and 128 x 128 blocks of weights.
// s = m / 448 for a block of largest magnitude m, or 1 when m < 2^-100;
// q = e4m3(x / s), nearest, ties to even.
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyBlock = 7.888609052210118e-31f;   // 2^-100
constexpr int64_t kMaxDim = 1 << 20;

__device__ __forceinline__ float block_scale(float m) { return m < kTinyBlock ? 1.0f : __fdiv_rn(m, kE4m3Max); }

// Eight consecutive elements, widened to fp32.
template <bool XF32>
__device__ __forceinline__ void load8(const void* p, float (&v)[8])
{
    if (XF32) {
        const float4 a = __ldg(static_cast<const float4*>(p)), b = __ldg(static_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 u = __ldg(static_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
        }
    }
}

__device__ __forceinline__ float max8(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));   // fmaxf leaves NaN out
    return m;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 r = make_float2(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
        w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// 16 lanes per 1 x 128 block, eight columns each; consecutive half-warps take
// consecutive rows of one block column, so that their scales are adjacent.
template <bool XF32, bool SWIGLU>
__global__ void __launch_bounds__(256) quant_act_kernel(const void* __restrict__ x, int64_t ldx, int rows, int cols,
                                                        uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s)
{
    const int kb = (cols + 127) / 128, sub = threadIdx.x & 15;
    const int64_t total = (int64_t)((rows + 15) / 16) * 16 * kb;   // rows of whole 16-row groups, so warps stay whole
    const int64_t step = (int64_t)gridDim.x * 16;
    for (int64_t i = blockIdx.x * (int64_t)16 + (threadIdx.x >> 4); i < total; i += step) {
        const int64_t g = i / (16 * kb);
        const int r = (int)(g * 16 + (i & 15)), b = (int)((i >> 4) % kb), c = b * 128 + sub * 8;
        const bool live = r < rows && c < cols;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = 0.0f;
        if (live) {
            const int64_t at = (int64_t)r * ldx + c;
            const char* p = static_cast<const char*>(x);
            const int sz = XF32 ? 4 : 2;
            load8<XF32>(p + at * sz, v);
            if (SWIGLU) {
                float u[8];
                load8<XF32>(p + (at + cols) * sz, u);
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] = v[j] / (1.0f + expf(-v[j])) * u[j];
            }
        }
        float m = max8(v);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = block_scale(m);
        if (live) {
            *reinterpret_cast<uint2*>(q + (int64_t)r * ldq + c) = codes8(v, sc);
            if (sub == 0) s[(int64_t)b * rows + r] = sc;
        }
    }
}

// One CTA per 128 x 128 block; each thread holds eight runs of eight columns.
template <bool XF32>
__global__ void __launch_bounds__(256) quant_weight_kernel(const void* __restrict__ w, int64_t blocks, int out, int in,
                                                           uint8_t* __restrict__ q, float* __restrict__ s)
{
    __shared__ float s_m[8];
    const int nb = (out + 127) / 128, kb = (in + 127) / 128;
    const int tr = threadIdx.x >> 4, c8 = (threadIdx.x & 15) * 8;
    for (int64_t i = blockIdx.x; i < blocks; i += gridDim.x) {
        const int b = (int)(i % kb);
        const int64_t en = i / kb;
        const int64_t e = en / nb;
        const int r0 = (int)(en % nb) * 128 + tr, c = b * 128 + c8;
        float v[8][8];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int r = r0 + 16 * j;
            if (r < out && c < in) {
                load8<XF32>(static_cast<const char*>(w) + ((e * out + r) * in + c) * (XF32 ? 4 : 2), v[j]);
                m = fmaxf(m, max8(v[j]));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, s_m[j]);
        const float sc = block_scale(m);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int r = r0 + 16 * j;
            if (r < out && c < in) *reinterpret_cast<uint2*>(q + (e * out + r) * in + c) = codes8(v[j], sc);
        }
        if (threadIdx.x == 0) s[i] = sc;
        __syncthreads();
    }
}

int sm_count()
{
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_quantize_act(const void* d_x, int32_t x_dtype, int64_t ldx, int32_t rows, int32_t cols,
                                    int32_t swiglu, uint8_t* d_q, int64_t ldq, float* d_s, void* stream)
{
    if (rows < 0 || cols <= 0 || cols % 8) return MOE_ERR_INVALID_ARG;
    if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (cols > kMaxDim || rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    const int64_t width = swiglu ? 2 * (int64_t)cols : cols;
    if (ldx < width || ldq < cols || ldx % (x_dtype == MOE_DT_F32 ? 4 : 8) || ldq % 8) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!d_x || !d_q || !d_s) return MOE_ERR_INVALID_ARG;
    if (((uintptr_t)d_x & 15) || ((uintptr_t)d_q & 7) || ((uintptr_t)d_s & 3)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    ProfScope ps(MOE_PROF_QUANT, st);
    prof_count(MOE_PROF_QUANT, 1);
    const int64_t want = (int64_t)((rows + 15) / 16) * ((cols + 127) / 128);
    const int cap = sm_count() * 8;
    const int grid = (int)(want < cap ? want : cap);
    const bool f32 = x_dtype == MOE_DT_F32;
    auto* kern = f32 ? (swiglu ? quant_act_kernel<true, true> : quant_act_kernel<true, false>)
                     : (swiglu ? quant_act_kernel<false, true> : quant_act_kernel<false, false>);
    kern<<<grid, 256, 0, st>>>(d_x, ldx, rows, cols, d_q, ldq, d_s);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
}

extern "C" int moe_fp8_quantize_weight(const void* d_w, int32_t w_dtype, int32_t experts, int32_t out, int32_t in,
                                       uint8_t* d_q, float* d_s, void* stream)
{
    if (experts <= 0 || out <= 0 || in <= 0 || in % 8) return MOE_ERR_INVALID_ARG;
    if (w_dtype != MOE_DT_F32 && w_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (experts > kMaxExperts || out > kMaxDim || in > kMaxDim) return MOE_ERR_UNSUPPORTED;
    if (!d_w || !d_q || !d_s) return MOE_ERR_INVALID_ARG;
    if (((uintptr_t)d_w & 15) || ((uintptr_t)d_q & 7) || ((uintptr_t)d_s & 3)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    ProfScope ps(MOE_PROF_QUANT, st);
    prof_count(MOE_PROF_QUANT, 1);
    const int64_t blocks = (int64_t)experts * ((out + 127) / 128) * ((in + 127) / 128);
    const int cap = sm_count() * 8;
    const int grid = (int)(blocks < cap ? blocks : cap);
    auto* kern = w_dtype == MOE_DT_F32 ? quant_weight_kernel<true> : quant_weight_kernel<false>;
    kern<<<grid, 256, 0, st>>>(d_w, blocks, out, in, d_q, d_s);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
}
