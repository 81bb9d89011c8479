// e4m3 codes with float32 block scales: 1 x 128 blocks of activation rows
// (optionally of silu(gate) * up) and 128 x 128 blocks of weights.
// s = m / 448 for a block of largest magnitude m, or 1 when m < 2^-100;
// q = e4m3(x / s), nearest, ties to even.
#include <cuda_fp8.h>

#include "common.cuh"
#include "overlap.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyBlock = 7.888609052210118e-31f;   // 2^-100
constexpr int64_t kMaxDim = 1 << 20;

// Two floats at a time: one instruction for both, each rounded by itself.
struct Two {
    unsigned long long v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two add2(Two a, Two b)
{
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// Quotients by Markstein's method (P. W. Markstein, IBM J. Res. Dev. 34, 1990):
// with y the correctly rounded 1 / s, q0 = v y and the exact residual
// r = v - q0 s, q0 + r y rounds to the correctly rounded v / s: three
// instructions an element against about forty of a division.
__device__ __forceinline__ float quotient(float v, float s, float y)
{
    const float q = __fmul_rn(v, y);
    return __fmaf_rn(__fmaf_rn(-q, s, v), y, q);
}
__device__ __forceinline__ float block_scale(float m)
{
    if (isinf(m)) return m;
    return m < kTinyBlock ? 1.0f : quotient(m, kE4m3Max, 1.0f / kE4m3Max);
}
// 1 / s, correctly rounded, for 2^-90 <= s < 2^120: two Newton steps from the
// hardware's reciprocal; the second one rounds correctly unless the
// significand of s is all ones (the same paper).
__device__ __forceinline__ float reciprocal(float s)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    y = __fmaf_rn(__fmaf_rn(-s, y, 1.0f), y, y);
    y = __fmaf_rn(__fmaf_rn(-s, y, 1.0f), y, y);
    return (__float_as_uint(s) & 0x7FFFFF) == 0x7FFFFF ? __fdiv_rn(1.0f, s) : y;
}

// Eight consecutive elements as they lie in memory; bf16 ones stay packed
// (four registers instead of eight while loads are in flight).
template <bool XF32>
struct Run8;

template <>
struct Run8<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p)
    {
        a = static_cast<const float4*>(p)[0];
        b = static_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void forget() {}
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

template <>
struct Run8<false> {
    uint4 u;
    __device__ __forceinline__ void load(const void* p) { u = *static_cast<const uint4*>(p); }
    // keeps the compiler from holding the widened values instead of the packed ones
    __device__ __forceinline__ void forget() { asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

__device__ __forceinline__ float max8(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));   // fmaxf leaves NaN out
    return m;
}

// silu(g) * u with the hardware's 2^x (relative error 2^-22) and reciprocal
// (2^-23): with the roundings of -g log2(e), of the sum and of the products
// the relative error is below (10 + 1.5 |g|) 2^-24, far inside an e4m3 step of
// 2^-4.  Four instructions an element; expf and a division took 32 in all, and
// this kernel is bound by its instructions.
__device__ __forceinline__ Two swiglu2(Two g, Two u)
{
    float a, b;
    mul2(g, Two(-1.4426950408889634f, -1.4426950408889634f)).get(a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    add2(Two(a, b), Two(1.0f, 1.0f)).get(a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return mul2(mul2(g, Two(a, b)), u);
}

// The block's divisor: v / s for its 128 or 16384 elements.  An infinite s
// gives y = 0 and takes the part of a zero in the residual, so that
// finite / inf is 0 and inf / inf NaN.  The residual's last bit is worth
// 2^-46 times the leading ones of s and of the quotient: no less than 2^-149,
// so exact, where s >= 2^-92 and the quotient is at least 2^-11 (codes of
// smaller ones are 0 either way).  Smaller s, and their v, are scaled up.
constexpr float kLift = 1.8446744073709552e19f;        // 2^64
constexpr float kSmallScale = 8.077935669463161e-28f;   // 2^-90
struct Divisor {
    Two s, y;    // -s twice, 1 / s twice
    bool lift;
    __device__ __forceinline__ explicit Divisor(float scale)
    {
        lift = scale < kSmallScale;
        if (lift) scale *= kLift;
        const float t = isinf(scale) ? 0.0f : scale, r = isinf(scale) ? 0.0f : reciprocal(scale);
        s = Two(-t, -t);
        y = Two(r, r);
    }
    __device__ __forceinline__ Two operator()(Two v) const
    {
        const Two q = mul2(v, y);
        return fma2(fma2(q, s, v), y, q);
    }
};

template <bool LIFT>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Divisor& d)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        Two t(v[2 * i], v[2 * i + 1]);
        if (LIFT) t = mul2(t, Two(kLift, kLift));
        float2 r;
        d(t).get(r.x, r.y);
        w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}
// (Two bodies: the lift as predicated instructions took 30 us beside 528 for
// 64 x 4096 x 4096 weights.)
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Divisor& d)
{
    return d.lift ? codes8<true>(v, d) : codes8<false>(v, d);
}

// A CTA takes 16 rows by BPT block columns at a time: half a warp per row
// (eight columns a lane), all BPT loads in flight before the first block is
// worked on.  The 16 rows' scales of a block column are adjacent.
template <bool XF32, bool SWIGLU, int BPT>
__global__ void __launch_bounds__(256) quant_act_kernel(const void* x, int64_t ldx, int rows, int cols,
                                                        uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s)
{
    constexpr int SZ = XF32 ? 4 : 2;
    const int kb = (cols + 127) / 128, per = (kb + BPT - 1) / BPT, sub = threadIdx.x & 15;
    const int total = (rows + 15) / 16 * per;
    start_next();
    wait_before();
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
        const int r = i / per * 16 + (threadIdx.x >> 4), b0 = i % per * BPT;
        const char* p = static_cast<const char*>(x) + (int64_t)r * ldx * SZ;
        Run8<XF32> x8[BPT], u8[SWIGLU ? BPT : 1];
#pragma unroll
        for (int j = 0; j < BPT; j++) {
            const int c = (b0 + j) * 128 + sub * 8;
            if (r < rows && c < cols) {
                x8[j].load(p + (int64_t)c * SZ);
                if (SWIGLU) u8[j].load(p + ((int64_t)cols + c) * SZ);
            } else {
                x8[j].zero();
                if (SWIGLU) u8[j].zero();
            }
        }
#pragma unroll
        for (int j = 0; j < BPT; j++) {
            const int b = b0 + j, c = b * 128 + sub * 8;
            float v[8];
            x8[j].get(v);
            if (SWIGLU) {
                float u[8];
                u8[j].get(u);
#pragma unroll
                for (int k = 0; k < 8; k += 2) swiglu2(Two(v[k], v[k + 1]), Two(u[k], u[k + 1])).get(v[k], v[k + 1]);
            }
            float m = max8(v);
#pragma unroll
            for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float sc = block_scale(m);
            if (r < rows && c < cols) {
                *reinterpret_cast<uint2*>(q + (int64_t)r * ldq + c) = codes8(v, Divisor(sc));
                if (sub == 0) s[(int64_t)b * rows + r] = sc;
            }
        }
    }
}

// One CTA per 128 x 128 block; each thread holds eight runs of eight columns
// between the maximum and the codes, so the block is read once.
template <bool XF32>
__global__ void __launch_bounds__(256, XF32 ? 2 : 4)
    quant_weight_kernel(const void* w, int blocks, int out, int in, uint8_t* __restrict__ q,
                        float* __restrict__ s)
{
    __shared__ float s_m[2][8];
    const int nb = (out + 127) / 128, kb = (in + 127) / 128;
    const int tr = threadIdx.x >> 4, c8 = (threadIdx.x & 15) * 8;
    int flip = 0;
    start_next();
    wait_before();
    for (int i = blockIdx.x; i < blocks; i += gridDim.x, flip ^= 1) {
        const int en = i / kb, b = i - en * kb;
        const int64_t e = en / nb;
        const int r0 = en % nb * 128 + tr, c = b * 128 + c8;
        Run8<XF32> w8[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int r = r0 + 16 * j;
            if (r < out && c < in)
                w8[j].load(static_cast<const char*>(w) + ((e * out + r) * in + c) * (XF32 ? 4 : 2));
            else
                w8[j].zero();
        }
        float v[8], m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            w8[j].get(v);
            m = fmaxf(m, max8(v));
            w8[j].forget();
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) s_m[flip][threadIdx.x >> 5] = m;   // two sets: one barrier a block
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, s_m[flip][j]);
        const float sc = block_scale(m);
        const Divisor div(sc);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int r = r0 + 16 * j;
            if (r < out && c < in) {
                w8[j].get(v);
                *reinterpret_cast<uint2*>(q + (e * out + r) * in + c) = codes8(v, div);
            }
        }
        if (threadIdx.x == 0) s[i] = sc;
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
    // four blocks a thread once that still gives every SM several CTAs
    const int64_t groups = (rows + 15) / 16, kb = (cols + 127) / 128;
    const int sms = sm_count();
    const bool wide = groups * ((kb + 3) / 4) >= 4 * sms;
    const int64_t want = groups * (wide ? (kb + 3) / 4 : kb);
    // CTAs of one item or few, so that they end together (8 an SM: 49 us
    // instead of 46 for SwiGLU on 24576 x 2048)
    if (want > 0x7fffffff - 64 * sms) return MOE_ERR_UNSUPPORTED;
    const int grid = (int)(want < 64 * sms ? want : 64 * sms);
    const bool f32 = x_dtype == MOE_DT_F32;
    auto* kern = wide ? (f32 ? (swiglu ? quant_act_kernel<true, true, 4> : quant_act_kernel<true, false, 4>)
                             : (swiglu ? quant_act_kernel<false, true, 4> : quant_act_kernel<false, false, 4>))
                      : (f32 ? (swiglu ? quant_act_kernel<true, true, 1> : quant_act_kernel<true, false, 1>)
                             : (swiglu ? quant_act_kernel<false, true, 1> : quant_act_kernel<false, false, 1>));
    MOE_CUDA_TRY(launch_overlapped(kern, grid, 1, 256, 0, st, d_x, ldx, (int)rows, (int)cols, d_q, ldq, d_s));
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
    // CTAs of a few blocks, so that they end together (all of them resident at
    // once: 527 us instead of 495 for 64 x 4096 x 4096; one block each: 503)
    const int cap = sm_count() * (w_dtype == MOE_DT_F32 ? 64 : 128);
    if (blocks > 0x7fffffff - cap) return MOE_ERR_UNSUPPORTED;   // 35 TB of bf16
    const int grid = (int)(blocks < cap ? blocks : cap);
    auto* kern = w_dtype == MOE_DT_F32 ? quant_weight_kernel<true> : quant_weight_kernel<false>;
    MOE_CUDA_TRY(launch_overlapped(kern, grid, 1, 256, 0, st, d_w, (int)blocks, (int)out, (int)in, d_q, d_s));
    return MOE_OK;
}
