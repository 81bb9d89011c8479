// Matrix products of e4m3 codes grouped by expert, with a float32 scale per
// 1 x 128 block of the rows and per 128 x 128 block of the weights (see
// include/moe.h):
//   y[r][o] = sum_b (xs[b][r] ws[e][o / 128][b]) sum_{j in block b} xq[r][j] wq[e][o][j]
//
// The scales are arbitrary, so they cannot go into the tensor core (its block
// scales are powers of two): each 128-column block is a product of its own in
// tensor memory, and the epilogue adds it, scaled, to fp32 sums in registers.
// With 128 features of one weight block as the tensor core's M and NB rows as
// its N, a block's weight scale is one number per tile and a row's scale one
// number per column, so the two multiply once per column and each element
// costs a single FMA.  An expert's rows are never padded beyond 16.
//
// One persistent CTA per SM: warp 0 copies (one 128-column block of both
// operands per stage, TMA into the 128-byte swizzle), warp 1 issues the MMAs
// of a block into one of four accumulators, warps 2-3 bring the products of
// scales into a ring in shared memory, four blocks at a time, and warps 4-11
// (two per tensor-memory lane quarter, half of the columns each) add.  Waits
// are bounded as in grouped_gemm.cu.
#include "tc.cuh"

namespace moe {

__device__ int g_gemm8_error;   // first device-side error of the FP8 products (0: none)

namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kMaxStages = 12;
constexpr int kABytes = 128 * 128;   // 128 features x 128 columns
constexpr int kBufs = 4;             // accumulators
constexpr int kGroup = 4;            // blocks per scale slot
constexpr int kSlots = 3;
constexpr int kEpi = 8;              // epilogue warps

struct Args {
    const int32_t* offsets;
    const float* xs;   // [blocks][rows]
    const float* ws;   // [E][nb][blocks]
    void* out;
    int64_t ldo;
    int out_f32;
    int E, rows;
    int M, blocks;     // features; 128-column blocks
    int stages;
    int box;           // smallest height of a copy of the row operand
    long long wait;    // limit of every bounded wait, in SM clock cycles
    int withhold;      // testing: CTA 0 leaves its first stage unfilled
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 1)
    gg8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ RowMaps tm_b, const Args a)
{
    constexpr int STAGE = kABytes + NB * 128;
    constexpr int CW = NB / 2;                    // columns of one epilogue warp
    constexpr uint32_t TMEM = kBufs * NB;
    static_assert(CW % 16 == 0, "columns are read 16 at a time");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kBufs], acc_empty[kBufs];
    __shared__ __align__(8) uint64_t sc_full[kSlots], sc_empty[kSlots], fin;
    __shared__ __align__(16) float s_scale[kSlots][kGroup][NB];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_scan[2 * kThreads / 32];
    unsigned char* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    LiveExpert* tab = reinterpret_cast<LiveExpert*>(ring + (size_t)a.stages * STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_v = &s_abort;
    int* err = &g_gemm8_error;

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < a.stages; i++) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < kBufs; i++) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), kEpi);
        }
        for (int i = 0; i < kSlots; i++) {
            mbar_init(smem_u32(&sc_full[i]), 2);
            mbar_init(smem_u32(&sc_empty[i]), kEpi);
        }
        mbar_init(smem_u32(&fin), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tma_prefetch(&tm_a);
        for (int i = 0; i < kRowMaps && a.box << i <= NB; i++) tma_prefetch(&tm_b.m[i]);
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(&s_tmem), TMEM);
    fence_before();
    const int live = build_live(a.offsets, a.E, a.rows, NB, tab, s_scan);
    fence_after();
    const uint32_t tmem = s_tmem;
    RowUnits<NB, 1> units(tab, live, a.M);
    RowUnit v;

    if (warp == 0) {
        // ============ copies
        int st = 0, withheld = -1;
        uint32_t ph = 0;
        long long issued = 0;
        bool ok = true;
        if (elect1()) {
        while (ok && units.next(v)) {
            const int ub = row_units(v.n, a.box);
            const uint32_t bytes = kABytes + (uint32_t)(ub * a.box * 128);
            for (int b = 0; b < a.blocks; b++) {
                if (!(ok = mbar_wait(smem_u32(&empty[st]), ph ^ 1, abort_v, a.wait, err))) break;
                const uint32_t bar = smem_u32(&full[st]), sa = smem_u32(ring + (size_t)st * STAGE), sb = sa + kABytes;
                if (a.withhold && blockIdx.x == 0 && issued == 0) {
                    withheld = st;   // testing: never filled, so the wait for it runs out
                } else {
                    mbar_expect_tx(bar, bytes);
                    tma_3d(sa, &tm_a, 128 * b, v.m0, v.e, bar);
                    tma_rows(sb, tm_b, 128 * b, v.r0, ub, a.box, bar);
                }
                issued++;
                if (++st == a.stages) { st = 0; ph ^= 1; }
            }
        }
        // every issued copy lands before the CTA exits
        for (int i = 0; i < a.stages && i < issued; i++)
            if (i != withheld) mbar_drain(smem_u32(&full[i]), i < st ? ph : (ph ^ 1), err);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ============ MMAs: one accumulator per block
        int st = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool ok = true;
        if (elect1()) {
        while (ok && units.next(v)) {
            const uint32_t id = idesc_e4m3<1>((v.n + 15) & ~15);
            for (int b = 0; b < a.blocks; b++) {
                if (!(ok = mbar_wait(smem_u32(&acc_empty[buf]), bph ^ 1, abort_v, a.wait, err))) break;
                if (!(ok = mbar_wait(smem_u32(&full[st]), ph, abort_v, a.wait, err))) break;
                fence_after();
                const uint32_t sa = smem_u32(ring + (size_t)st * STAGE);
                const uint64_t da = desc_k(sa), db = desc_k(sa + kABytes);
#pragma unroll
                for (int k = 0; k < 4; k++) mma_e4m3<1>(tmem + (uint32_t)(buf * NB), da + 2 * k, db + 2 * k, id, k > 0);
                commit<1>(smem_u32(&empty[st]));
                commit<1>(smem_u32(&acc_full[buf]));
                if (++st == a.stages) { st = 0; ph ^= 1; }
                if (++buf == kBufs) { buf = 0; bph ^= 1; }
            }
        }
        commit<1>(smem_u32(&fin));
        mbar_drain(smem_u32(&fin), 0, err);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ============ scales: xs * ws of four blocks by NB rows per slot
        constexpr int PER = kGroup * NB / 64;
        const int t = tid - 64, nb = (a.M + 127) / 128;
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
        while (ok && units.next(v)) {
            const float* wsp = a.ws + ((int64_t)v.e * nb + v.m0 / 128) * a.blocks;
            for (int b0 = 0; b0 < a.blocks; b0 += kGroup) {
                float s[PER];
#pragma unroll
                for (int i = 0; i < PER; i++) {
                    const int at = t + 64 * i, b = b0 + at / NB, c = at % NB;
                    s[i] = 0.0f;
                    if (b < a.blocks && c < v.n)
                        s[i] = __ldg(a.xs + (int64_t)b * a.rows + v.r0 + c) * __ldg(wsp + b);
                }
                if (!(ok = mbar_wait_warp(smem_u32(&sc_empty[slot]), ph ^ 1, abort_v, a.wait, err))) break;
#pragma unroll
                for (int i = 0; i < PER; i++) (&s_scale[slot][0][0])[t + 64 * i] = s[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sc_full[slot]));
                if (++slot == kSlots) { slot = 0; ph ^= 1; }
            }
        }
    } else {
        // ============ sums: lane quarter warp % 4, columns CW * half on, one feature per thread
        const int q = warp & 3, half = (warp - 4) >> 2;
        int slot = 0, buf = 0;
        uint32_t sph = 0, bph = 0;
        bool ok = true;
        while (ok && units.next(v)) {
            float acc[CW];
#pragma unroll
            for (int c = 0; c < CW; c++) acc[c] = 0.0f;
            const int c0 = CW * half;
            for (int b = 0; b < a.blocks; b++) {
                const int g = b % kGroup;
                if (g == 0 && !(ok = mbar_wait_warp(smem_u32(&sc_full[slot]), sph, abort_v, a.wait, err))) break;
                if (!(ok = mbar_wait_warp(smem_u32(&acc_full[buf]), bph, abort_v, a.wait, err))) break;
                fence_after();
                const uint32_t src = tmem + (uint32_t)(buf * NB + c0) + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int c = 0; c < CW; c += 16) {
                    if (c0 + c >= v.n) break;
                    uint32_t d[16];
                    tmem_ld16(src + c, d);
                    wait_ld();
                    const float4* s4 = reinterpret_cast<const float4*>(&s_scale[slot][g][c0 + c]);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float4 s = s4[j];
                        acc[c + 4 * j] = fmaf(__uint_as_float(d[4 * j]), s.x, acc[c + 4 * j]);
                        acc[c + 4 * j + 1] = fmaf(__uint_as_float(d[4 * j + 1]), s.y, acc[c + 4 * j + 1]);
                        acc[c + 4 * j + 2] = fmaf(__uint_as_float(d[4 * j + 2]), s.z, acc[c + 4 * j + 2]);
                        acc[c + 4 * j + 3] = fmaf(__uint_as_float(d[4 * j + 3]), s.w, acc[c + 4 * j + 3]);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&acc_empty[buf]));
                    if (g == kGroup - 1 || b == a.blocks - 1) mbar_arrive(smem_u32(&sc_empty[slot]));
                }
                if (++buf == kBufs) { buf = 0; bph ^= 1; }
                if ((g == kGroup - 1 || b == a.blocks - 1) && ++slot == kSlots) { slot = 0; sph ^= 1; }
            }
            if (!ok) break;
            const int f = v.m0 + 32 * q + lane;
            if (f < a.M) {
                const int64_t at = (int64_t)(v.r0 + c0) * a.ldo + f;
                float* of = static_cast<float*>(a.out) + at;
                uint16_t* oh = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
                for (int c = 0; c < CW; c++) {
                    if (c0 + c >= v.n) break;
                    if (a.out_f32) of[c * a.ldo] = acc[c];
                    else oh[c * a.ldo] = f32_to_bf16_bits(acc[c]);
                }
            }
            __syncwarp();
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem, TMEM);
    }
}

template <int NB>
int launch_nb(Args& a, const CUtensorMap& ta, const RowMaps& tb, cudaStream_t st)
{
    constexpr int STAGE = kABytes + NB * 128;
    int sms = 0;
    if (int rc = device_sms(&sms)) return rc;
    const int table = (int)align_up(sizeof(LiveExpert) * (a.E + 1), 128);
    const int fixed = kSlots * kGroup * NB * 4 + 1024;   // scale ring, barriers
    a.stages = (kSmemMax - fixed - 1024 - table) / STAGE;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const int smem = 1024 + a.stages * STAGE + table;
    auto* kern = gg8_kernel<NB>;
    MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    ProfScope ps(MOE_PROF_GEMM, st);
    prof_count(MOE_PROF_GEMM, 1);
    kern<<<sms, kThreads, smem, st>>>(ta, tb, a);
    MOE_LAUNCH_CHECK();
    return MOE_OK;
}

}  // namespace

int gemm8_device_error(int clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gemm8_error, sizeof v) != cudaSuccess) return MOE_ERR_CUDA;
    if (clear && v) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_gemm8_error, &z, sizeof z) != cudaSuccess) return MOE_ERR_CUDA;
    }
    return v;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm_fp8(int32_t experts, int32_t in, int32_t out, const uint8_t* d_xq, int64_t ldxq,
                                    const float* d_xs, const uint8_t* d_wq, const float* d_ws,
                                    const int32_t* d_offsets, int32_t rows, void* d_y, int64_t ldy, int32_t y_dtype,
                                    void* stream)
{
    if (int rc = check_gemm_sizes(experts, in, out, rows, 16)) return rc;
    if (!out_dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!d_offsets || !d_xs || !d_ws || ((uintptr_t)d_xs & 3) || ((uintptr_t)d_ws & 3) || !rows_ok(d_xq, ldxq, in, 1) ||
        !rows_ok(d_wq, in, in, 1) || !rows_ok(d_y, ldy, out, dtype_size(y_dtype)))
        return MOE_ERR_INVALID_ARG;
    Args a{};
    a.offsets = d_offsets;
    a.xs = d_xs;
    a.ws = d_ws;
    a.out = d_y;
    a.ldo = ldy;
    a.out_f32 = y_dtype == MOE_DT_F32;
    a.E = experts;
    a.rows = rows;
    a.M = out;
    a.blocks = (in + 127) / 128;
    a.wait = test_wait_cycles(kWaitCycles);
    a.withhold = test_withhold();
    const bool small = rows <= 16 * (int64_t)experts;
    a.box = small ? 16 : 32;
    CUtensorMap ta;
    RowMaps tb;
    const uint64_t wd[3] = {(uint64_t)in, (uint64_t)out, (uint64_t)experts};
    const uint64_t wst[2] = {(uint64_t)in, (uint64_t)in * out};
    const uint32_t wb[3] = {128, 128, 1};
    if (!encode_map(&ta, E_U8, 3, d_wq, wd, wst, wb) ||
        !encode_rows(&tb, E_U8, d_xq, ldxq, in, rows, a.box, small ? 32 : 128))
        return MOE_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    return small ? launch_nb<32>(a, ta, tb, st) : launch_nb<128>(a, ta, tb, st);
}
