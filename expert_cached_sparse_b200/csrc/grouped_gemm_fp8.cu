// Matrix products of e4m3 codes grouped by expert, with a float32 scale per
// 1 x 128 block of the rows and per 128 x 128 block of the weights (see
// include/moe.h):
//   y[r][o] = sum_b (xs[b][r] ws[e][o / 128][b]) sum_{j in block b} xq[r][j] wq[e][o][j]
//
// The scales are arbitrary, so they cannot go into the tensor core (its block
// scales are powers of two): each 128-column block is a product of its own in
// tensor memory, and the epilogue adds it, scaled, to fp32 sums in registers.
//
// MANY rows an expert: rows are the tensor core's M, one tensor-memory lane
// and one thread each, and 256 features its N: a thread's scale xs ws is then
// one number for all of its columns, and two elements cost one instruction
// (0.51 us a block of a tile; one FMA an element, 0.53).  With rows as N every
// column has its own scale, and reading those from shared memory takes as long
// as the FMAs (575 against 329 cycles for 128 x 256 elements, 16 warps).
// FEW: features are M and up to 32 rows N, as in grouped_gemm.cu, so that all
// warps have work on a tile of one row and the MMAs compute 16 rows and not
// 128: 120 W less at the same stream of weights, which the clock gets back.
//
// Roles, one persistent CTA per SM: warps 0 and 2 copy (one 128-column block
// of rows and of weights per stage, TMA into the 128-byte swizzle), warp 1
// issues the MMAs of a block into one of the accumulators, and warps 4 on add,
// a quarter of the lanes each (MANY: and half of the columns).  (On pairs of
// CTAs, as in grouped_gemm.cu, every block's accumulator has to be handed back
// across the cluster: 1.26 ms against 0.89 for 4096 tokens.)  Waits are
// bounded as in grouped_gemm.cu.
#include "tc.cuh"

namespace moe {

__device__ int g_gemm8_error;   // first device-side error of the FP8 products (0: none)

namespace {

using namespace tc;

template <bool FEW_>
struct Cfg {
    static constexpr bool FEW = FEW_;
    static constexpr int NF = FEW ? 128 : 256;              // features of a tile
    static constexpr int NR = FEW ? 32 : 128;               // most rows of a tile
    static constexpr int EPI = FEW ? 4 : 8;                 // epilogue warps
    static constexpr int THREADS = 128 + 32 * EPI;
    static constexpr int COLS = FEW ? NR : NF;              // tensor-memory columns of an accumulator
    static constexpr int BUFS = FEW ? 4 : 512 / COLS;       // accumulators
    static constexpr int CW = FEW ? COLS : COLS / 2;        // columns of one epilogue warp
    static constexpr int WEIGHTS = NF * 128, STAGE = WEIGHTS + NR * 128;
};
// Registers a thread of the control warps and of the epilogue's where the
// latter hold 128 sums each: together what the block is launched with,
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kRegs = 168, kControlRegs = 72, kSumRegs = 216;
static_assert(128 * kControlRegs + 32 * Cfg<false>::EPI * kSumRegs <= Cfg<false>::THREADS * kRegs,
              "a larger split never starts");
constexpr int kMaxStages = 12;
constexpr int kStatic = 4096;        // bytes of static shared memory at most

struct Args {
    const int32_t* offsets;
    const float* xs;   // [blocks][rows]
    const float* ws;   // [E][nb][blocks]
    void* out;
    int64_t ldo;
    int out_f32;
    int wide;          // output rows are 32-byte aligned
    int E, rows;
    int M, blocks;     // features; 128-column blocks
    int split;         // FEW: CTAs of a cluster that share a tile's blocks
    int stages;
    int box;           // smallest height of a copy of the rows
    long long wait;    // limit of every bounded wait, in SM clock cycles
    int withhold;      // testing: CTA 0 leaves its first stage unfilled
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A load that stays where it is written, far ahead of its use (the compiler
// would move a plain one down to the use and wait for it there); 0 if !in.
__device__ __forceinline__ float fetch_f32(const float* p, bool in)
{
    float v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
                 "@p ld.global.f32 %0, [%1];\n\t}" : "=f"(v) : "l"(p), "r"((int)in));
    return v;
}

// 32 adjacent bytes of a row: one whole sector where rows are aligned so.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        uint4* o = static_cast<uint4*>(p);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// a += x s, b += y s: one instruction, two products.
__device__ __forceinline__ void add2(float& a, float& b, uint32_t x, uint32_t y, float s)
{
    asm("{\n\t.reg .b64 p, q, t;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 t, {%4, %4};\n\t"
        "fma.rn.f32x2 p, q, t, p;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(x), "r"(y), "f"(s));
}

template <class CFG>
__global__ void __launch_bounds__(CFG::THREADS, 1)
    gg8_kernel(const __grid_constant__ RowMaps tm_rows, const __grid_constant__ CUtensorMap tm_w, const Args a)
{
    constexpr bool FEW = CFG::FEW;
    constexpr int NF = CFG::NF, CW = CFG::CW, BUFS = CFG::BUFS, STAGE = CFG::STAGE, WEIGHTS = CFG::WEIGHTS;
    constexpr uint32_t TMEM = BUFS * CFG::COLS;
    constexpr int GROUP = FEW ? 4 : 8;            // blocks whose scales are fetched together, a group ahead (MANY of 4:
                                                  // 885 us instead of 857 for 4096 tokens x 6 of 256 experts)
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[BUFS], acc_empty[BUFS], fin;
    __shared__ uint32_t s_tmem;
    __shared__ CopyPos s_copy[2];
    __shared__ int s_abort, s_live;
    __shared__ long long s_scan[CFG::EPI];
    __shared__ __align__(16) float s_scale[FEW ? CFG::EPI : 1][GROUP][32];   // FEW: a warp's scales of a group
    unsigned char* ring = smem_raw;
    PlanExpert* tab = reinterpret_cast<PlanExpert*>(ring + (size_t)a.stages * STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_v = &s_abort;
    int* err = &g_gemm8_error;

    if (smem_u32(ring) & 1023) {   // the swizzle counts on it; static shared memory is padded so
        wait_before();
        if (tid == 0) atomicCAS(err, 0, (int)MOE_ERR_UNSUPPORTED);
        return;
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < a.stages; i++) {
            mbar_init(smem_u32(&full[i]), 2);   // both copy warps
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < BUFS; i++) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), CFG::EPI);
        }
        mbar_init(smem_u32(&fin), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const RowBlocks blocks{CFG::NR};
    if (warp == 0) {
        for (int i = 0; i < kRowMaps && a.box << i <= CFG::NR; i++) tma_prefetch(&tm_rows.m[i]);
    } else if (warp == 2) {
        tma_prefetch(&tm_w);
    }
    wait_before();
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s_tmem), TMEM);   // (not before: it may wait for what the kernel before holds)
    } else if (warp >= 4) {
        build_plan<32 * CFG::EPI>(a.offsets, a.E, a.rows, blocks, tab, s_scan, &s_live);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    const int rank = FEW ? (int)cluster_rank() : 0;
    PlanWalk tiles(tab, s_live, blocks, (a.M + NF - 1) / NF, blockIdx.x / a.split, gridDim.x / a.split);
    int split = a.split, blo, bhi;   // this CTA's blocks [blo, bhi)
    tiles.split_steps(a.blocks, rank, split, blo, bhi);
    PlanTile v;

    if (warp < 4) {
        if (!FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        if (warp == 0) {
            // ============ copies of the rows
            if (elect1()) {
                // MANY: a tile's MMAs read 128 rows whatever it has.  Rows left over from a
                // taller tile, or from before the kernel, are overwritten with zeros (a copy
                // from behind the matrix) when the stage is next filled: the results do not
                // depend on them, but the tensor core's power does, and with it the clock.
                int u = 0;
                uint64_t tall = ~0ull;   // per stage, 4 bits: boxes that may hold something, less one
                copy_loop<STAGE, 1>(smem_u32(full), empty, ring, a.stages, abort_v, a.wait, a.withhold && blockIdx.x == 0,
                                 err, &s_copy[0],
                                 [&] {
                                     if (!tiles.next(v)) return -1;
                                     u = row_units(v.n, a.box);
                                     return bhi - blo;
                                 },
                                 [&](int s, uint32_t bar, uint32_t sa, int st) {
                                     int wipe = 0;
                                     if (!FEW) {
                                         wipe = max(0, min((int)(tall >> (4 * st) & 15) + 1, CFG::NR / a.box) - u);
                                         tall = (tall & ~(15ull << (4 * st))) | ((uint64_t)(u - 1) << (4 * st));
                                     }
                                     const uint32_t sr = sa + WEIGHTS;
                                     mbar_expect_tx(bar, (uint32_t)((u + wipe) * a.box * 128));
                                     tma_rows(sr, tm_rows, 128 * (blo + s), v.r0, u, a.box, bar);
                                     if (wipe) tma_rows(sr + u * a.box * 128, tm_rows, 0, a.rows, wipe, a.box, bar);
                                 });
            }
            __syncwarp();
            start_next();   // (at the kernel's start: the same within 1%, and SMs held for longer)
            drain_copies(full, a.stages, s_copy, 0, a.withhold && blockIdx.x == 0, err);
        } else if (warp == 2) {
            // ============ copies of the weights
            if (elect1())
                copy_loop<STAGE, 1>(smem_u32(full), empty, ring, a.stages, abort_v, a.wait, a.withhold && blockIdx.x == 0,
                                 err, &s_copy[1],
                                 [&] { return tiles.next(v) ? bhi - blo : -1; },
                                 [&](int s, uint32_t bar, uint32_t sa, int) {
                                     mbar_expect_tx(bar, WEIGHTS);
                                     tma_3d(sa, &tm_w, 128 * (blo + s), v.m * NF, v.e, bar);
                                 });
            __syncwarp();
            drain_copies(full, a.stages, s_copy, 1, a.withhold && blockIdx.x == 0, err);
        } else if (warp == 1) {
            // ============ MMAs: one accumulator per block
            if (elect1()) {
                int st = 0, buf = 0;
                uint32_t ph = 0, bph = 0;
                bool ok = true;
                while (ok && tiles.next(v)) {
                    const uint32_t id = idesc_e4m3(FEW ? mma_rows<1>(v.n) : NF);
                    for (int b = blo; b < bhi; b++) {
                        if (!(ok = mbar_wait(smem_u32(&full[st]), ph, abort_v, a.wait, err))) break;
                        if (!(ok = mbar_wait(smem_u32(&acc_empty[buf]), bph ^ 1, abort_v, a.wait, err))) break;
                        fence_after();
                        const uint32_t sa = smem_u32(ring + (size_t)st * STAGE);
                        const uint64_t da = desc_k(FEW ? sa : sa + WEIGHTS), db = desc_k(FEW ? sa + WEIGHTS : sa);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mma_e4m3<1>(tmem + (uint32_t)(buf * CFG::COLS), da + 2 * k, db + 2 * k, id, k > 0);
                        commit<1>(smem_u32(&empty[st]));
                        commit<1>(smem_u32(&acc_full[buf]));
                        if (++st == a.stages) { st = 0; ph ^= 1; }
                        if (++buf == BUFS) { buf = 0; bph ^= 1; }
                    }
                }
                commit<1>(smem_u32(&fin));   // every MMA completes before tensor memory is released
                mbar_drain(smem_u32(&fin), 0, err);
            }
            __syncwarp();
        }
        if (FEW && split > 1) split_others();
    } else {
        if (!FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // ============ sums.  MANY: rows 32 q + lane, CW features from c0 on; FEW: feature
        // 32 q + lane, every row
        const int q = warp & 3, c0 = CW * ((warp - 4) >> 2), nb = (a.M + 127) / 128;
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true, reduced = false;
        const int row = FEW ? lane : 32 * q + lane;   // whose scales the lane fetches
        const float *xsp, *wsp;
        bool scales;
        float xs[GROUP], ws[GROUP];
        auto of_tile = [&](const PlanTile& t) {
            const int m0 = t.m * NF + (FEW ? 32 * q : c0);
            scales = m0 < a.M && row < t.n;
            xsp = a.xs + t.r0 + row;
            wsp = a.ws + ((int64_t)t.e * nb + m0 / 128) * a.blocks;
        };
        auto fetch = [&](int b0) {
#pragma unroll
            for (int g = 0; g < GROUP; g++) {
                const bool in = scales && b0 + g < bhi;
                xs[g] = fetch_f32(xsp + (int64_t)(b0 + g) * a.rows, in);
                ws[g] = fetch_f32(wsp + b0 + g, in);
            }
        };
        // FEW: the first scales of a tile are fetched before the last blocks of the tile before it
        // (16 tokens x 6 of 256 experts, 4096 x 4096: 123.5 us against 128; MANY's tiles are long
        // and its registers few: 870 us against 857)
        PlanTile after;
        bool more = FEW && tiles.next(after);
        if (more) {
            of_tile(after);
            fetch(blo);
        }
        while (ok && (FEW ? more : tiles.next(v))) {
            if (FEW) {
                v = after;
            } else {
                of_tile(v);
                fetch(blo);
            }
            const int m0 = v.m * NF + (FEW ? 32 * q : c0);            // the warp's first feature
            const bool works = m0 < a.M && (FEW || 32 * q < v.n);     // the warp has features and rows
            float acc[CW];
#pragma unroll
            for (int c = 0; c < CW; c++) acc[c] = 0.0f;
            for (int b0 = blo; ok && b0 < bhi; b0 += GROUP) {
                float s[GROUP];
#pragma unroll
                for (int g = 0; g < GROUP; g++) {
                    s[g] = xs[g] * ws[g];
                    if (FEW) s_scale[warp - 4][g][lane] = s[g];   // of all rows, for all lanes
                }
                if (FEW) __syncwarp();
                if (!FEW || b0 + GROUP < bhi) {
                    fetch(b0 + GROUP);
                } else if ((more = tiles.next(after))) {
                    of_tile(after);
                    fetch(blo);
                }
#pragma unroll
                for (int g = 0; g < GROUP; g++) {
                    if (b0 + g >= bhi) break;
                    if (!(ok = mbar_wait_warp(smem_u32(&acc_full[buf]), bph, abort_v, a.wait, err))) break;
                    fence_after();
                    if (works) {
                        const uint32_t src = tmem + (uint32_t)(buf * CFG::COLS + (FEW ? 0 : c0)) + ((uint32_t)(32 * q) << 16);
                        if constexpr (FEW) {
#pragma unroll
                            for (int c = 0; c < CW; c += 16) {
                                if (c >= v.n) break;
                                uint32_t d[16];
                                tmem_ld16(src + c, d);
                                wait_ld(d);
#pragma unroll
                                for (int j = 0; j < 16; j += 4) {
                                    const float4 t = *reinterpret_cast<const float4*>(&s_scale[warp - 4][g][c + j]);
                                    acc[c + j] = fmaf(__uint_as_float(d[j]), t.x, acc[c + j]);
                                    acc[c + j + 1] = fmaf(__uint_as_float(d[j + 1]), t.y, acc[c + j + 1]);
                                    acc[c + j + 2] = fmaf(__uint_as_float(d[j + 2]), t.z, acc[c + j + 2]);
                                    acc[c + j + 3] = fmaf(__uint_as_float(d[j + 3]), t.w, acc[c + j + 3]);
                                }
                            }
                        } else {
                            uint32_t d[2][16];   // 16 columns on their way while 16 are added
                            tmem_ld16(src, d[0]);
#pragma unroll
                            for (int c = 0; c < CW; c += 16) {
                                wait_ld(d[(c / 16) & 1]);
                                if (c + 16 < CW) tmem_ld16(src + c + 16, d[(c / 16 + 1) & 1]);
#pragma unroll
                                for (int j = 0; j < 16; j += 2)
                                    add2(acc[c + j], acc[c + j + 1], d[(c / 16) & 1][j], d[(c / 16) & 1][j + 1], s[g]);
                            }
                        }
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
                    if (++buf == BUFS) { buf = 0; bph ^= 1; }
                }
            }
            if (!ok) break;
            if constexpr (FEW) {
                if (split > 1) {
                    split_reduce(acc, ring, rank, split, 32 * q + lane);
                    reduced = true;
                    if (rank) break;
                }
                if (m0 + lane < a.M) {
                    const int64_t at = (int64_t)v.r0 * a.ldo + m0 + lane;
                    // left at the last row: 32 predicated stores of either type, most of them none,
                    // took 3500 cycles
                    if (a.out_f32) {
                        float* o = static_cast<float*>(a.out) + at;
#pragma unroll
                        for (int c = 0; c < CW; c++, o += a.ldo) {
                            if (c >= v.n) break;
                            *o = acc[c];
                        }
                    } else {
                        uint16_t* o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
                        for (int c = 0; c < CW; c++, o += a.ldo) {
                            if (c >= v.n) break;
                            *o = f32_to_bf16_bits(acc[c]);
                        }
                    }
                }
            } else if (scales) {
                const int64_t at = (int64_t)(v.r0 + row) * a.ldo + m0;
                const int n = min(CW, a.M - m0);   // a multiple of 8
                if (a.out_f32) {
                    float* o = static_cast<float*>(a.out) + at;
#pragma unroll
                    for (int c = 0; c < CW; c += 8)
                        if (c < n) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; j++) w[j] = __float_as_uint(acc[c + j]);
                            store32(o + c, w, a.wide);
                        }
                } else {
                    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
                    for (int c = 0; c < CW; c += 16)
                        if (c < n) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; j++) w[j] = pack_bf16(acc[c + 2 * j], acc[c + 2 * j + 1]);
                            if (c + 8 < n) store32(o + c, w, a.wide);
                            else *reinterpret_cast<uint4*>(o + c) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
            }
            __syncwarp();
        }
        if (FEW && split > 1 && !reduced) split_others();   // no tile, or a wait that ran out
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem, TMEM);
    }
}

template <class CFG>
int launch(Args& a, int64_t tiles, int sms, int dev, const RowMaps& tr, const CUtensorMap& tw, cudaStream_t st)
{
    static std::atomic<int> smem_set[kMaxDevices];
    auto* kern = gg8_kernel<CFG>;
    if (int rc = allow_smem(kern, kSmemMax - kStatic, smem_set, dev)) return rc;
    const int fixed = plan_bytes(a.E);
    a.stages = (kSmemMax - kStatic - fixed) / CFG::STAGE;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const int smem = fixed + a.stages * CFG::STAGE;
    if (!CFG::FEW) {   // the register split counts on what the kernel was compiled to
        static const int regs = [] {
            cudaFuncAttributes at{};
            return cudaFuncGetAttributes(&at, gg8_kernel<CFG>) == cudaSuccess ? at.numRegs : 0;
        }();
        if (regs != kRegs) return MOE_ERR_UNSUPPORTED;
    }
    ProfScope ps(MOE_PROF_GEMM, st);
    prof_count(MOE_PROF_GEMM, 1);
    MOE_CUDA_TRY(launch_clusters(kern, sms, tiles, a.split, CFG::THREADS, smem, st, tr, tw, a));
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
    if (!words_ok(d_offsets) || !words_ok(d_xs) || !words_ok(d_ws) || !rows_ok(d_xq, ldxq, in, 1) ||
        !rows_ok(d_wq, in, in, 1) || !rows_ok(d_y, ldy, out, dtype_size(y_dtype)))
        return MOE_ERR_INVALID_ARG;
    Args a{};
    a.offsets = d_offsets;
    a.xs = d_xs;
    a.ws = d_ws;
    a.out = d_y;
    a.ldo = ldy;
    a.out_f32 = y_dtype == MOE_DT_F32;
    a.wide = !(((uintptr_t)d_y | (uintptr_t)(ldy * dtype_size(y_dtype))) & 31);
    a.E = experts;
    a.rows = rows;
    a.M = out;
    a.blocks = (in + 127) / 128;
    a.wait = test_wait_cycles(kWaitCycles);
    a.withhold = test_withhold();
    int sms = 0, dev = 0;
    if (int rc = device_sms(&sms, &dev)) return rc;
    // FEW where the experts have few rows, or where its small tiles fit the SMs at once
    const int64_t few_tiles = most_tiles(experts, rows, 32, (out + 127) / 128);
    const bool few = rows <= 16 * (int64_t)experts || few_tiles <= sms;
    a.split = few ? split_of(few_tiles, a.blocks, sms) : 1;
    a.box = few ? 16 : 32;
    RowMaps tr;
    CUtensorMap tw;
    const uint64_t wd[3] = {(uint64_t)in, (uint64_t)out, (uint64_t)experts};
    const uint64_t wst[2] = {(uint64_t)in, (uint64_t)in * out};
    const uint32_t wb[3] = {128, few ? 128u : 256u, 1};
    if (!encode_rows(&tr, E_U8, d_xq, ldxq, in, rows, a.box, few ? 32 : 128) ||
        !encode_map(&tw, E_U8, 3, d_wq, wd, wst, wb))
        return MOE_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    return few ? launch<Cfg<true>>(a, few_tiles, sms, dev, tr, tw, st)
               : launch<Cfg<false>>(a, most_tiles(experts, rows, 128, (out + 255) / 256), sms, dev, tr, tw, st);
}
