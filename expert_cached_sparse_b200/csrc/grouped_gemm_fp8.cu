// Matrix products of e4m3 codes with block scales, grouped by expert (see
// include/moe.h).  First form: 64 x 64 output tiles, fp32 FMAs
// from shared memory, one expert per grid plane.
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int64_t kMaxDim = 1 << 20;

enum Mode { FWD, DX, DW, FP8 };

struct Args {
    const void* a;          // row matrix: x (FWD, FP8) or dy (DX, DW)
    int64_t lda;
    const void* w;          // weights, or x (DW)
    int64_t ldw;
    const float* xs;
    const float* ws;
    const int32_t* offsets;
    void* out;
    int64_t ldo;
    int out_dtype, accumulate;
    int experts, in, outs, rows;
};

__device__ __forceinline__ float ld_bf16(const void* p, int64_t i)
{
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ float ld_e4m3(const void* p, int64_t i)
{
    __nv_fp8_e4m3 v;
    v.__x = static_cast<const uint8_t*>(p)[i];
    return (float)v;
}

template <int MODE>
__global__ void __launch_bounds__(256) gg8_kernel(const Args g)
{
    __shared__ float sa[16][65], sb[16][65];
    const int e = blockIdx.z;
    int r0 = g.offsets[e], r1 = g.offsets[e + 1];
    if (r0 < 0 || r1 > g.rows || r1 < r0) r0 = r1 = 0;
    const int m = MODE == DW ? g.outs : r1 - r0;                       // output rows
    const int n = MODE == FWD || MODE == FP8 ? g.outs : g.in;          // output columns
    const int kk = MODE == DW ? r1 - r0 : (MODE == DX ? g.outs : g.in);
    if (MODE == DW && g.accumulate && kk == 0) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int nb = (g.outs + 127) / 128, kb = (g.in + 127) / 128;
    for (int i0 = blockIdx.y * 64; i0 < m; i0 += gridDim.y * 64)
        for (int j0 = blockIdx.x * 64; j0 < n; j0 += gridDim.x * 64) {
            float acc[4][4] = {};
            for (int k0 = 0; k0 < kk; k0 += 16) {
                for (int t = threadIdx.x; t < 1024; t += 256) {
                    const int k = k0 + (t & 15), i = i0 + (t >> 4), j = j0 + (t >> 4);
                    float va = 0.0f, vb = 0.0f;
                    if (k < kk && i < m) {
                        if (MODE == FP8)
                            va = ld_e4m3(g.a, (int64_t)(r0 + i) * g.lda + k) * g.xs[(int64_t)(k / 128) * g.rows + r0 + i];
                        else if (MODE == DW)
                            va = ld_bf16(g.a, (int64_t)(r0 + k) * g.lda + i);
                        else
                            va = ld_bf16(g.a, (int64_t)(r0 + i) * g.lda + k);
                    }
                    if (k < kk && j < n) {
                        if (MODE == FP8)
                            vb = ld_e4m3(g.w, ((int64_t)e * n + j) * kk + k) * g.ws[((int64_t)e * nb + j / 128) * kb + k / 128];
                        else if (MODE == FWD)
                            vb = ld_bf16(g.w, ((int64_t)e * n + j) * kk + k);
                        else if (MODE == DX)
                            vb = ld_bf16(g.w, ((int64_t)e * kk + k) * n + j);
                        else
                            vb = ld_bf16(g.w, (int64_t)(r0 + k) * g.ldw + j);
                    }
                    sa[t & 15][t >> 4] = va;
                    sb[t & 15][t >> 4] = vb;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 16; k++)
#pragma unroll
                    for (int p = 0; p < 4; p++)
#pragma unroll
                        for (int q = 0; q < 4; q++) acc[p][q] = fmaf(sa[k][ty * 4 + p], sb[k][tx + 16 * q], acc[p][q]);
                __syncthreads();
            }
            for (int p = 0; p < 4; p++)
                for (int q = 0; q < 4; q++) {
                    const int i = i0 + ty * 4 + p, j = j0 + tx + 16 * q;
                    if (i >= m || j >= n) continue;
                    const int64_t at = MODE == DW ? ((int64_t)e * m + i) * n + j : (int64_t)(r0 + i) * g.ldo + j;
                    float v = acc[p][q];
                    if (g.out_dtype == MOE_DT_F32) {
                        float* o = static_cast<float*>(g.out) + at;
                        *o = MODE == DW && g.accumulate ? *o + v : v;
                    } else {
                        uint16_t* o = static_cast<uint16_t*>(g.out) + at;
                        if (MODE == DW && g.accumulate) v += bf16_bits_to_f32(*o);
                        *o = f32_to_bf16_bits(v);
                    }
                }
        }
}

template <int MODE>
int launch(const Args& g, void* stream)
{
    cudaStream_t st = as_stream(stream);
    ProfScope ps(MOE_PROF_GEMM, st);
    prof_count(MOE_PROF_GEMM, 1);
    const int m = MODE == DW ? g.outs : g.rows, n = MODE == FWD || MODE == FP8 ? g.outs : g.in;
    const int gx = (n + 63) / 64, gy = (m + 63) / 64;
    const dim3 grid(gx < 64 ? gx : 64, gy < 16 ? gy : 16, g.experts);
    gg8_kernel<MODE><<<grid, 256, 0, st>>>(g);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
}

// Checks common to the products; MOE_OK to go on.
int check_sizes(int experts, int in, int out, int rows, int in_mult)
{
    if (experts <= 0 || in <= 0 || in % in_mult || out <= 0 || out % 8 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (experts > kMaxExperts || in > kMaxDim || out > kMaxDim || rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
// A matrix of 16-byte aligned rows of `width` elements of `size` bytes.
bool rows_ok(const void* p, int64_t ld, int64_t width, int size)
{
    return p && !((uintptr_t)p & 15) && ld >= width && ld < ((int64_t)1 << 36) && (ld * size) % 16 == 0;
}
static bool out_dtype_ok(int t) { return t == MOE_DT_F32 || t == MOE_DT_BF16; }
int dtype_size(int t) { return t == MOE_DT_F32 ? 4 : 2; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm_fp8(int32_t experts, int32_t in, int32_t out, const uint8_t* d_xq, int64_t ldxq,
                                    const float* d_xs, const uint8_t* d_wq, const float* d_ws,
                                    const int32_t* d_offsets, int32_t rows, void* d_y, int64_t ldy, int32_t y_dtype,
                                    void* stream)
{
    if (int rc = check_sizes(experts, in, out, rows, 16)) return rc;
    if (!out_dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!d_offsets || !d_xs || !d_ws || ((uintptr_t)d_xs & 3) || ((uintptr_t)d_ws & 3) || !rows_ok(d_xq, ldxq, in, 1) ||
        !rows_ok(d_wq, in, in, 1) || !rows_ok(d_y, ldy, out, dtype_size(y_dtype)))
        return MOE_ERR_INVALID_ARG;
    return launch<FP8>({d_xq, ldxq, d_wq, in, d_xs, d_ws, d_offsets, d_y, ldy, y_dtype, 0, experts, in, out, rows},
                       stream);
}
