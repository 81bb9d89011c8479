// Matrix products grouped by expert with ragged row ranges, in bf16, and
// their gradients (see include/moe.h):
//   FWD  y[r][o]  = sum_i x[r][i] W_e[o][i]
//   DX   dx[r][i] = sum_o dy[r][o] W_e[o][i]
//   DW   dW_e[o][i] = sum_r dy[r][o] x[r][i]   over e's rows
//
// One kernel, three operand layouts.  A tile is 128 features (the tensor
// core's M, one tensor-memory lane each: `out` for FWD and DW, `in` for DX) by
// up to NB columns (N: rows for FWD and DX, `in` for DW), and the inner index
// advances 64 per pipeline stage.  The features are the operand that is never
// ragged, so M is always full and N takes any multiple of 16: an expert with
// one row costs a 128 x 16 tile, not a 128 x 128 one.  TMA brings each operand
// into the 128-byte swizzle as it lies in memory; where the inner index is
// not the contiguous one (W in DX, x and dy in DW) the tensor core reads the
// tile MN-major, so nothing is transposed.  What lies outside a matrix reads
// as zeros, so odd sizes need no other path.
//
// Rows are ragged: in FWD and DX a tile's surplus rows are another expert's
// (each N column is its own sum; they are not stored).  In DW rows are the
// inner index, so a last step's surplus rows are zeroed in shared memory, in
// both operands (a NaN there must not meet a zero), before the MMAs read them.
//
// Tiles of many columns run on pairs of CTAs (CG = 2, the two SMs of a
// cluster): 256 features by NB columns, each CTA holding its own 128 features
// and half of the columns, so a column's bytes cross from L2 once for 256
// features instead of once for 128.
//
// Roles, one persistent CTA or pair per SM or two: warps 0 and 2 copy the two
// operands (one warp for both issued too slowly), warp 1 (of the pair's first
// CTA) issues the MMAs into one of two accumulators, warps 4 on read the other
// one back and store it.  In DW warp 3 works between copies and MMAs: it zeroes
// the surplus rows.  The copies of a pair's both CTAs complete on the first
// one's barriers, where its MMA warp waits for them.
// Every wait is bounded; a timeout records MOE_ERR_TIMEOUT, raises the CTA's
// abort flag so that the other roles stop, and the CTA waits for its own
// copies and MMAs before it returns.
#include "tc.cuh"

namespace moe {

__device__ int g_gemm_error;   // first device-side error of the bf16 products (0: none)

namespace {

using namespace tc;

constexpr int kMaxStages = 12;
constexpr int kStatic = 1024;        // bytes of static shared memory at most
constexpr int kABytes = 128 * 128;   // 128 features x 64 inner indices
constexpr int kStaging = 8 * 4096;

// Steps of 64 summed in one accumulator.  The tensor core adds to its fp32
// accumulator with truncation, so the relative error of a sum grows by about
// 1e-6 for every 1000 inner indices, and by 6e-6 where all terms have one
// sign (6.6e-3 too small at 2^20); partial sums are added up outside it,
// rounded to nearest.  float32 outputs: FWD, DX of 256 inner indices, in
// registers (2.4e-7 off, less than fp32 sums by FMAs from 1000 inner indices
// on; of 512, 4.7e-7 and 0 to 13% faster, 128, 1.5e-7 and 5 to 17% slower;
// adding them to the output took 474 us instead of 208 where a tile has eight
// of them).  DW: of 512 rows, in the output (few experts have several).  bf16
// outputs: of 8192 inner indices, 5e-5 too small at most beside a rounding of
// 2^-9, so that one accumulator holds the sums of most layers.
constexpr int kPartial = 4, kPartialDw = 8, kPartialBf16 = 128;

// Registers a thread of the control warps and of the epilogue's where the
// latter hold 128 float32 sums each: together what the block is launched with,
// 128 * 88 + 256 * 208 = 384 * 168 (72 and 216: DW's control warps spill).
constexpr int kRegs = 168, kControlRegs = 88, kSumRegs = 208;

enum Mode { FWD, DX, DW };

struct Args {
    const int32_t* offsets;
    void* out;
    int64_t ldo;
    int out_f32, accumulate;
    int direct;      // DW: sums added to bf16 ones in registers
    int E, rows;
    int M, N;        // features; DW: columns (`in`)
    int K;           // inner size (DW: ragged)
    int stages;
    int partial;     // steps summed in one accumulator
    int split;       // CTAs of a cluster that share a tile's inner index
    int box;         // smallest height of a copy of the ragged operand (FWD, DX)
    int chunks_a, chunks_b;   // whether one copy brings all 64-column chunks of an MN-major operand
    long long wait;  // limit of every bounded wait, in SM clock cycles
    int withhold;    // testing: CTA 0 leaves its first stage unfilled
};

struct Unit {
    int e, m0, c0, n;   // expert, this CTA's first feature, first column (row of the matrix, or `in` index), columns
    int cb, nb, nh;     // this CTA's share of the columns: first one, how many exist, how many the MMA takes
    int k0, steps;      // DW: first row; steps of 64
    int tail;           // DW: valid rows of the last step
};

// The tiles of a CTA or pair.
template <int MODE, int NB, int CG>
struct Units {
    const Args& a;
    PlanWalk walk;
    const int rank;
    int split, s0, s1;   // CG = 1: the cluster's CTAs that share the inner index, this one's steps

    __device__ Units(const Args& a_, const PlanExpert* tab, const int*, int live, int rank_)
        : a(a_), walk(tab, live, {NB}, (a_.M + 128 * CG - 1) / (128 * CG), blockIdx.x / (CG * a_.split),
                      gridDim.x / (CG * a_.split)),
          rank(CG == 2 ? rank_ : 0), split(a_.split)
    {
        walk.split_steps((a.K + 63) / 64, rank_, split, s0, s1);
    }
    __device__ __forceinline__ bool next(Unit& v)
    {
        PlanTile w;
        if (!walk.next(w)) return false;
        v.e = w.e;
        v.m0 = (w.m * CG + rank) * 128;
        v.c0 = w.r0;
        v.n = w.n;
        v.k0 = 64 * s0;
        v.steps = s1 - s0;
        v.tail = 64;
        v.nh = mma_rows<CG>(v.n) / CG;
        v.cb = v.c0 + v.nh * rank;
        v.nb = max(0, min(v.nh, v.n - v.nh * rank));
        return true;
    }
};

// A weight gradient's tiles: every expert's, an expert's feature tiles
// fastest.  (Pairs of CTAs took 99 us instead of 80 for 128 experts'
// 768 x 2048 with 32 rows each, and 292 instead of 270 for 2048 x 1536 with
// 256: the few steps of a tile do not hide the hand-overs across the pair.)
template <int NB>
struct Units<DW, NB, 1> {
    const Args& a;
    const int* off;   // the offsets, in shared memory
    static constexpr int split = 1;
    const int mt, per;
    long long u, total;

    __device__ Units(const Args& a_, const PlanExpert*, const int* o, int, int)
        : a(a_), off(o), mt((a_.M + 127) / 128), per(mt * ((a_.N + NB - 1) / NB)), u(blockIdx.x),
          total((long long)a_.E * per)
    {
    }
    __device__ __forceinline__ bool next(Unit& v)
    {
        if (u >= total) return false;
        // a 64-bit division takes hundreds of cycles
        v.e = total < 0x7fffffff ? (int)u / per : (int)(u / per);
        const int r = (int)(u - (long long)v.e * per);
        int lo = off[v.e], hi = off[v.e + 1];
        if (lo < 0 || hi < lo || hi > a.rows) lo = hi = 0;
        v.m0 = r % mt * 128;
        v.c0 = r / mt * NB;
        v.n = min(NB, a.N - v.c0);
        v.k0 = lo;
        v.steps = (hi - lo + 63) / 64;
        v.tail = hi - lo - (v.steps - 1) * 64;
        v.nh = mma_rows<1>(v.n);
        v.cb = v.c0;
        v.nb = v.n;
        u += gridDim.x;
        return true;
    }
};

// A warp's 32 features of n columns, ldo elements apart: each store is 32
// adjacent elements of one column.  `mine`: whether the lane's feature exists.
__device__ __forceinline__ void store_cols(uint16_t* p, int64_t ldo, uint32_t src, int n, bool mine)
{
    for (int c = 0; c < n; c += 16) {
        uint32_t d[16];
        tmem_ld16(src + c, d);
        wait_ld(d);
        if (mine) {
#pragma unroll
            for (int j = 0; j < 16; j++) {
                if (c + j < n) *p = f32_to_bf16_bits(__uint_as_float(d[j]));
                p += ldo;
            }
        }
        __syncwarp();   // the warp's next tensor-memory load is a converged one
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi)
{
    return pack_bf16(__uint_as_float(lo), __uint_as_float(hi));
}

// Stores 8 (n < 16) or 16 adjacent elements as bf16, or adds them to what is
// there: fp32 sums, one rounding.
__device__ __forceinline__ void store_row16(uint16_t* p, const uint32_t (&d)[16], int n, bool add)
{
    uint4* o = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int j = 0; j < 2; j++) {
        if (j && n < 16) break;   // `in` is a multiple of 8
        if (!add) {
            o[j] = make_uint4(pack_bf16(d[8 * j], d[8 * j + 1]), pack_bf16(d[8 * j + 2], d[8 * j + 3]),
                              pack_bf16(d[8 * j + 4], d[8 * j + 5]), pack_bf16(d[8 * j + 6], d[8 * j + 7]));
            continue;
        }
        const uint4 b = o[j];
        uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = pack_bf16(__uint_as_float(d[8 * j + 2 * k]) + bf16_bits_to_f32(w[k] & 0xFFFFu),
                             __uint_as_float(d[8 * j + 2 * k + 1]) + bf16_bits_to_f32(w[k] >> 16));
        o[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Adds n columns of an accumulator, a multiple of 16 of them, to a thread's sums.
template <int CW>
__device__ __forceinline__ void add_cols(float (&sum)[CW], uint32_t src, int n)
{
#pragma unroll
    for (int c = 0; c < CW; c += 16) {
        if (c >= n) break;
        uint32_t d[16];
        tmem_ld16(src + c, d);
        wait_ld(d);
#pragma unroll
        for (int j = 0; j < 16; j++) sum[c + j] += __uint_as_float(d[j]);
    }
}

// A warp's 32 rows of dW from row r0 on go out by TMA, 128 bytes of each at a
// time, through swizzled tiles in shared memory; zeros where `none`.  Two
// warps share the rows.  bf16: every other 128 bytes each, through a tile of
// its own (one warp for all, with both tiles, took 194 us instead of 150 for
// 128 experts' 2048 x 1536 with 32 rows each: reading the accumulators and
// packing them was the longest way; with 256 rows each 270 either way).
// float32: the first warp takes all, with both tiles (170 us with both warps,
// 146 so, for 128 experts' 768 x 2048 with 32 rows each).
__device__ __forceinline__ void store_tile(const Args& a, const CUtensorMap& out, const Unit& v, unsigned char* tiles,
                                           int& tile, uint32_t src, int r0, int group, bool none, bool add)
{
    const int lane = threadIdx.x & 31, w = a.out_f32 ? 32 : 64;
    if (a.out_f32 && group) return;
    for (int c = group * w; c < v.n; c += a.out_f32 ? w : 2 * w) {
        uint32_t d[32], e[32];   // 32 float32 values; 64 bf16 ones packed in d
        auto load = [&](int from, uint32_t (&v)[32]) {
            tmem_ld16(src + from, v);
            tmem_ld16(src + from + 16, v + 16);
            wait_ld(v);
            hold16(v + 16);
        };
        if (none) {
#pragma unroll
            for (int j = 0; j < 32; j++) d[j] = 0;
        } else {
            load(c, d);
            if (!a.out_f32) {
                load(c + 32, e);
#pragma unroll
                for (int j = 0; j < 16; j++) d[j] = pack_bf16(d[2 * j], d[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 16; j++) d[16 + j] = pack_bf16(e[2 * j], e[2 * j + 1]);
            }
        }
        if (lane == 0) {   // the tile's previous rows are on their way
            if (a.out_f32) bulk_wait_read<1>();
            else bulk_wait_read<0>();
        }
        __syncwarp();
        unsigned char* row = tiles + 4096 * tile + 128 * lane;
#pragma unroll
        for (int j = 0; j < 8; j++)
            *reinterpret_cast<uint4*>(row + 16 * (j ^ (lane & 7))) =
                make_uint4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if (add) tma_add_3d(&out, smem_u32(tiles + 4096 * tile), v.c0 + c, r0, v.e);
            else tma_store_3d(&out, smem_u32(tiles + 4096 * tile), v.c0 + c, r0, v.e);
            bulk_commit();
        }
        if (a.out_f32) tile ^= 1;   // (the next call goes on from here)
    }
}

// SUMS: row products summed up in the epilogue's registers, for float32 outputs,
// for an inner index split over a cluster and for more steps than an
// accumulator takes.
template <int MODE, int NB, bool SUMS>
struct Epilogue {
    static constexpr int WARPS = MODE == DW || (SUMS && NB > 32) ? 8 : 4;
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr int CW = NB / (WARPS / 4);        // columns of one warp
    // registers moved from the control warps (DW: for bf16 outputs over many rows)
    static constexpr bool SPLIT = (SUMS || MODE == DW) && CW > 64;
};
static_assert(128 * kControlRegs + 256 * kSumRegs <= 384 * kRegs, "a larger split never starts");

template <int MODE, int NB, int CG, bool SUMS>
__global__ void __launch_bounds__(Epilogue<MODE, NB, SUMS>::THREADS, 1)
    gg_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ RowMaps tm_b,
              const __grid_constant__ CUtensorMap tm_out, const Args a)
{
    constexpr int STAGE = kABytes + NB / CG * 128;
    constexpr uint32_t TMEM = 2 * NB;
    constexpr bool PAIR = CG == 2;
    using EPI = Epilogue<MODE, NB, SUMS>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[kMaxStages], ready[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], fin;
    __shared__ uint32_t s_tmem;
    __shared__ CopyPos s_copy[2];
    __shared__ int s_abort, s_live;
    __shared__ long long s_scan[EPI::WARPS];
    unsigned char* ring = smem_raw;
    unsigned char* staging = ring + (size_t)a.stages * STAGE;   // DW: two tiles of 32 rows x 128 bytes per lane quarter
    PlanExpert* tab = reinterpret_cast<PlanExpert*>(staging + (MODE == DW ? kStaging : 0));
    int* off = reinterpret_cast<int*>(tab);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = MODE == DW ? 0 : (int)cluster_rank();   // of a pair, or of a cluster that splits the inner index
    volatile int* abort_v = &s_abort;
    int* err = &g_gemm_error;

    if (smem_u32(ring) & 1023) {   // the swizzle counts on it; static shared memory is padded so
        wait_before();
        if (tid == 0) atomicCAS(err, 0, (int)MOE_ERR_UNSUPPORTED);
        return;
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < a.stages; i++) {
            mbar_init(smem_u32(&full[i]), 2 * CG);   // both copy warps
            mbar_init(smem_u32(&ready[i]), 1);       // DW
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), EPI::WARPS * CG);
        }
        mbar_init(smem_u32(&fin), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tma_prefetch(&tm_a);
    } else if (warp == 2) {
        for (int i = 0; i < kRowMaps && a.box << i <= NB / CG; i++) tma_prefetch(&tm_b.m[i]);
    }
    wait_before();
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(&s_tmem), TMEM);   // (not before: it may wait for what the kernel before holds)
    } else if (warp >= 4) {
        if constexpr (MODE == DW)
            for (int i = tid - 128; i <= a.E; i += 32 * EPI::WARPS) off[i] = a.offsets[i];
        else
            build_plan<32 * EPI::WARPS>(a.offsets, a.E, a.rows, {NB}, tab, s_scan, &s_live);
    }
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the peer's barriers exist
    fence_after();
    const uint32_t tmem = s_tmem;
    Units<MODE, NB, CG> units(a, tab, off, MODE == DW ? 0 : s_live, rank);
    Unit v;
    const uint32_t full0 = PAIR ? peer_addr(smem_u32(full), 0) : smem_u32(full);

    if (warp < 4) {
        if (EPI::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        if (warp == 0) {
            // ============ copies of the features (A)
            if (elect1())
                copy_loop<STAGE, CG>(full0, empty, ring, a.stages, abort_v, a.wait, a.withhold && blockIdx.x == 0, err, &s_copy[0],
                                 [&] { return units.next(v) ? v.steps : -1; },
                                 [&](int s, uint32_t bar, uint32_t sa, int) {
                                     const int k = v.k0 + 64 * s;
                                     mbar_expect_tx<CG>(bar, kABytes);
                                     if (MODE == FWD) {
                                         tma_3d<CG>(sa, &tm_a, k, v.m0, v.e, bar);
                                     } else if (a.chunks_a) {
                                         if (MODE == DX) tma_4d<CG>(sa, &tm_a, 0, k, v.m0 / 64, v.e, bar);
                                         else tma_3d(sa, &tm_a, 0, k, v.m0 / 64, bar);
                                     } else
                                         for (int i = 0; i < 2; i++) {
                                             if (MODE == DX) tma_3d<CG>(sa + 8192 * i, &tm_a, v.m0 + 64 * i, k, v.e, bar);
                                             else tma_2d(sa + 8192 * i, &tm_a, v.m0 + 64 * i, k, bar);
                                         }
                                 });
            __syncwarp();
            start_next();   // (at the kernel's start: the same within 1%, and SMs held for longer)
            if (!PAIR) drain_copies(full, a.stages, s_copy, 0, a.withhold && blockIdx.x == 0, err);
        } else if (warp == 2) {
            // ============ copies of the columns (B)
            if (elect1()) {
                int ub = 0;
                uint32_t bytes = 0;
                copy_loop<STAGE, CG>(full0, empty, ring, a.stages, abort_v, a.wait, a.withhold && blockIdx.x == 0, err, &s_copy[1],
                                 [&] {
                                     if (!units.next(v)) return -1;
                                     ub = MODE == DW ? (a.chunks_b ? NB / 64 : (v.n + 63) / 64) : row_units(v.nb, a.box);
                                     bytes = (uint32_t)(ub * (MODE == DW ? 8192 : a.box * 128));
                                     return v.steps;
                                 },
                                 [&](int s, uint32_t bar, uint32_t sa, int) {
                                     const int k = v.k0 + 64 * s;
                                     const uint32_t sb = sa + kABytes;
                                     mbar_expect_tx<CG>(bar, bytes);   // (none: a pair's second half without columns)
                                     if (MODE != DW)
                                         tma_rows<CG>(sb, tm_b, k, v.cb, ub, a.box, bar);
                                     else if (a.chunks_b)
                                         tma_3d(sb, &tm_b.m[0], 0, k, v.cb / 64, bar);
                                     else
                                         for (int i = 0; i < ub; i++) tma_2d(sb + 8192 * i, &tm_b.m[0], v.cb + 64 * i, k, bar);
                                 });
            }
            __syncwarp();
            if (!PAIR) drain_copies(full, a.stages, s_copy, 1, a.withhold && blockIdx.x == 0, err);
        } else if (warp == 1) {
            // ============ MMAs
            if (!PAIR || rank == 0) {
                if (elect1()) {
                    int st = 0, it = 0;
                    uint32_t ph = 0;
                    bool ok = true;
                    while (ok && units.next(v)) {
                        const uint32_t id = idesc_bf16<CG>(CG * v.nh, MODE != FWD, MODE == DW);
                        uint32_t d = 0;
                        int left = 0;   // steps until the accumulator changes
                        for (int s = 0; s < v.steps; s++) {
                            const bool first = left == 0;
                            if (first) {
                                const int ab = it & 1;
                                if (it >= 2 &&   // the epilogue has read what this accumulator held
                                    !(ok = mbar_wait<CG>(smem_u32(&acc_empty[ab]), ((it >> 1) - 1) & 1, abort_v, a.wait, err)))
                                    break;
                                d = tmem + (uint32_t)(ab * NB);
                                left = min(a.partial, v.steps - s);
                            }
                            const uint32_t bar = smem_u32(MODE == DW ? &ready[st] : &full[st]);
                            if (!(ok = mbar_wait<CG>(bar, ph, abort_v, a.wait, err))) break;
                            fence_after();
                            const uint32_t sa = smem_u32(ring + (size_t)st * STAGE), sb = sa + kABytes;
                            const uint64_t da = MODE == FWD ? desc_k(sa) : desc_mn(sa, 8192);
                            const uint64_t db = MODE == DW ? desc_mn(sb, 8192) : desc_k(sb);
                            // 16 inner indices: 32 bytes along a K-major row, 16 rows MN-major
                            const int kk = MODE == DW && s == v.steps - 1 ? (v.tail + 15) / 16 : 4;
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                if (MODE != DW || k < kk)
                                    mma_bf16<CG>(d, da + k * (MODE == FWD ? 2 : 128), db + k * (MODE == DW ? 128 : 2), id,
                                                 !first || k > 0);
                            commit<CG>(smem_u32(&empty[st]));   // the stage is free once these MMAs have read it
                            if (++st == a.stages) { st = 0; ph ^= 1; }
                            if (--left == 0) {
                                commit<CG>(smem_u32(&acc_full[it & 1]));
                                it++;
                            }
                        }
                    }
                    commit<CG>(smem_u32(&fin));   // every MMA completes before tensor memory is released
                    mbar_drain<CG>(smem_u32(&fin), 0, err);
                }
                __syncwarp();
            }
        } else if (warp == 3) {
            // ============ between copies and MMAs
            if (MODE == DW) {
                int st = 0;
                uint32_t ph = 0;
                bool ok = true;
                while (ok && units.next(v)) {
                    for (int s = 0; s < v.steps; s++) {
                        if (!(ok = mbar_wait_warp(smem_u32(&full[st]), ph, abort_v, a.wait, err))) break;
                        if (s == v.steps - 1 && (v.tail & 15)) {
                            // zero the surplus rows of the last 16-row step in every 64-column chunk of both operands
                            unsigned char* p = ring + (size_t)st * STAGE + 128 * v.tail;
                            const int z = 128 * (16 - (v.tail & 15)), chunks = 2 + (v.nh + 63) / 64;
                            for (int i = 16 * lane; i < z; i += 512)
                                for (int c = 0; c < chunks; c++)
                                    *reinterpret_cast<uint4*>(p + 8192 * c + i) = make_uint4(0, 0, 0, 0);
                            asm volatile("fence.proxy.async;" ::: "memory");
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive(smem_u32(&ready[st]));
                        if (++st == a.stages) { st = 0; ph ^= 1; }
                    }
                }
            }
        }
        if (SUMS && units.split > 1) split_others();
    } else {
        if (EPI::SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // ============ epilogue: lane quarter q = warp % 4, one feature per thread; SUMS: columns
        // from cw on, CW of them
        const int q = warp & 3;
        int it = 0, tile = warp >= 8;   // DW: its staging tile
        bool ok = true, reduced = false;
        while (ok && units.next(v)) {
            const int f = v.m0 + 32 * q + lane;
            const bool mine = f < a.M;
            const bool none = MODE == DW && v.steps == 0;   // an expert without rows: its gradient is zero
            if (none && a.accumulate) continue;
            const int cw = EPI::CW * ((warp - 4) >> 2), c1 = min(v.n, cw + EPI::CW);
            if constexpr (MODE == DW) {
                if (!a.out_f32 && v.steps > a.partial) {   // more rows than a bf16 output's accumulator takes
                    float sum[EPI::CW];
#pragma unroll
                    for (int c = 0; c < EPI::CW; c++) sum[c] = 0.0f;
                    for (int s = 0; s < v.steps; s += a.partial, it++) {
                        const int ab = it & 1;
                        if (!(ok = mbar_wait_warp<CG>(smem_u32(&acc_full[ab]), (it >> 1) & 1, abort_v, a.wait, err))) break;
                        fence_after();
                        add_cols(sum, tmem + (uint32_t)(ab * NB + cw) + ((uint32_t)(32 * q) << 16), v.n - cw);
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&acc_empty[ab]));
                    }
                    if (ok && mine) {
                        uint16_t* o = static_cast<uint16_t*>(a.out) + ((int64_t)v.e * a.M + f) * a.N + v.c0 + cw;
#pragma unroll
                        for (int c = 0; c < EPI::CW; c += 16) {
                            if (cw + c >= v.n) break;
                            uint32_t d[16];
#pragma unroll
                            for (int j = 0; j < 16; j++) d[j] = __float_as_uint(sum[c + j]);
                            store_row16(o + c, d, v.n - cw - c, a.accumulate);
                        }
                    }
                    __syncwarp();
                    continue;
                }
            }
            float sum[SUMS ? EPI::CW : 1];
            if (SUMS) {
#pragma unroll
                for (int c = 0; c < EPI::CW; c++) sum[c] = 0.0f;
            }
            // one accumulator, or the partial sums of every a.partial steps
            for (int s = 0; s == 0 || s < v.steps; s += a.partial) {
                const int ab = it & 1;
                const bool add = s > 0 || (MODE == DW && a.accumulate);   // to what is there
                if (!none) {
                    if (!(ok = mbar_wait_warp<CG>(smem_u32(&acc_full[ab]), (it >> 1) & 1, abort_v, a.wait, err))) break;
                    fence_after();
                }
                const uint32_t src = tmem + (uint32_t)(ab * NB) + ((uint32_t)(32 * q) << 16);
                if constexpr (MODE == DW) {
                    if (a.direct) {
                        // a thread's feature is a row of dW: 16 adjacent columns at a time
                        const int64_t at = ((int64_t)v.e * a.M + f) * a.N + v.c0;
                        for (int c = cw; c < c1; c += 16) {
                            uint32_t d[16];
                            tmem_ld16(src + c, d);
                            wait_ld(d);
                            if (mine) store_row16(static_cast<uint16_t*>(a.out) + at + c, d, v.n - c, true);
                            __syncwarp();   // the warp's next tensor-memory load is a converged one
                        }
                    } else if (v.m0 + 32 * q < a.M) {
                        if (s > 0 && lane == 0) bulk_wait();   // the partial sums before are in place
                        store_tile(a, tm_out, v, staging + 8192 * q, tile, src, v.m0 + 32 * q, (warp - 4) >> 2, none, add);
                    }
                } else if constexpr (SUMS) {
                    add_cols(sum, src + cw, v.n - cw);
                } else {
                    store_cols(static_cast<uint16_t*>(a.out) + (int64_t)v.c0 * a.ldo + f, a.ldo, src, v.n, mine);
                }
                if (none) break;
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(peer_addr(smem_u32(&acc_empty[ab]), 0));
                    else mbar_arrive(smem_u32(&acc_empty[ab]));
                }
                it++;
            }
            if constexpr (SUMS) {
                if (!ok) break;
                if (units.split > 1) {
                    if constexpr (CG == 1) split_reduce(sum, ring, rank, units.split, 32 * q + lane);
                    reduced = true;
                    if (rank) break;
                }
                const int64_t at = (int64_t)(v.c0 + cw) * a.ldo + f;
                const int n = mine ? v.n - cw : 0;
                if (a.out_f32) {
                    float* o = static_cast<float*>(a.out) + at;
#pragma unroll
                    for (int c = 0; c < EPI::CW; c++, o += a.ldo)
                        if (c < n) *o = sum[c];
                } else {
                    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
                    for (int c = 0; c < EPI::CW; c++, o += a.ldo)
                        if (c < n) *o = f32_to_bf16_bits(sum[c]);
                }
                __syncwarp();
            }
        }
        if (SUMS && units.split > 1 && !reduced) split_others();   // no tile, or a wait that ran out
        if (MODE == DW && lane == 0) bulk_wait();   // the staging tiles are read, the stores done
    }
    fence_before();
    __syncthreads();
    if (PAIR) {
        cluster_sync();   // the roles of both CTAs have ended
        if (rank == 0 && tid == 0 && (s_abort || ld_cluster(peer_addr(smem_u32(&s_abort), 1))))
            drain_pair(full, a.stages, s_copy, a.withhold && blockIdx.x == 0, err);
        if (rank == 1 && warp == 1) mbar_drain<CG>(smem_u32(&fin), 0, err);   // the commits' arrivals here
        __syncwarp();
    }
    if (warp == 1) {
        fence_after();
        tmem_dealloc<CG>(tmem, TMEM);
    }
    if (PAIR) cluster_sync();   // nothing of the peer reads or arrives in this CTA's memory any more
}

template <int MODE, int NB, int CG, bool SUMS>
int launch(Args& a, int64_t tiles, int sms, int dev, const CUtensorMap& ta, const RowMaps& tb, const CUtensorMap& to,
           cudaStream_t st)
{
    constexpr int STAGE = kABytes + NB / CG * 128;
    using EPI = Epilogue<MODE, NB, SUMS>;
    static std::atomic<int> smem_set[kMaxDevices];
    auto* kern = gg_kernel<MODE, NB, CG, SUMS>;
    if (int rc = allow_smem(kern, kSmemMax - kStatic, smem_set, dev)) return rc;
    const int fixed = MODE == DW ? kStaging + (int)align_up(4 * (a.E + 1), 128) : plan_bytes(a.E);
    a.stages = (kSmemMax - kStatic - fixed) / STAGE;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const int smem = fixed + a.stages * STAGE;
    if (EPI::SPLIT) {   // the register split counts on what the kernel was compiled to
        static const int regs = [] {
            cudaFuncAttributes at{};
            return cudaFuncGetAttributes(&at, gg_kernel<MODE, NB, CG, SUMS>) == cudaSuccess ? at.numRegs : 0;
        }();
        if (regs != kRegs) return MOE_ERR_UNSUPPORTED;
    }
    ProfScope ps(MOE_PROF_GEMM, st);
    prof_count(MOE_PROF_GEMM, 1);
    MOE_CUDA_TRY(launch_clusters(kern, sms, tiles, CG * a.split, EPI::THREADS, smem, st, ta, tb, to, a));
    return MOE_OK;
}

// An MN-major operand [batch][K][width] (batch 0: no such dimension) in 64
// inner rows by `chunks` 64-column chunks a copy.  Where the width is whole
// chunks, they are a dimension of the map and one copy brings them all;
// otherwise a copy brings one, and *whole is false.
bool map_mn(CUtensorMap* m, int* whole, const void* p, int64_t ld, int width, int K, int chunks, int batch)
{
    *whole = width % 64 == 0;
    if (*whole) {
        const uint64_t dims[4] = {64, (uint64_t)K, (uint64_t)width / 64, (uint64_t)batch};
        const uint64_t strides[3] = {(uint64_t)ld * 2, 128, (uint64_t)ld * K * 2};
        const uint32_t box[4] = {64, 64, (uint32_t)chunks, 1};
        return encode_map(m, E_BF16, batch ? 4 : 3, p, dims, strides, box);
    }
    const uint64_t dims[3] = {(uint64_t)width, (uint64_t)K, (uint64_t)batch};
    const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)ld * K * 2};
    const uint32_t box[3] = {64, 64, 1};
    return encode_map(m, E_BF16, batch ? 3 : 2, p, dims, strides, box);
}

// Products of rows with weights: y = x W^T (FWD) or dx = dy W (DX).
template <int MODE>
int row_product(int E, int in, int out, const uint16_t* x, int64_t ldx, const uint16_t* w, const int32_t* offsets,
                int rows, void* y, int64_t ldy, int y_dtype, void* stream)
{
    Args a{};
    a.offsets = offsets;
    a.out = y;
    a.ldo = ldy;
    a.out_f32 = y_dtype == MOE_DT_F32;
    a.partial = a.out_f32 ? kPartial : kPartialBf16;
    a.E = E;
    a.rows = rows;
    a.M = MODE == FWD ? out : in;
    a.K = MODE == FWD ? in : out;
    a.wait = test_wait_cycles(kWaitCycles);
    a.withhold = test_withhold();
    CUtensorMap ta;
    RowMaps tb;
    if (MODE == FWD) {
        const uint64_t dims[3] = {(uint64_t)in, (uint64_t)out, (uint64_t)E};
        const uint64_t strides[2] = {(uint64_t)in * 2, (uint64_t)in * out * 2};
        const uint32_t box[3] = {64, 128, 1};
        if (!encode_map(&ta, E_BF16, 3, w, dims, strides, box)) return MOE_ERR_CUDA;
    } else if (!map_mn(&ta, &a.chunks_a, w, in, in, out, 2, E)) {
        return MOE_ERR_CUDA;
    }
    int sms = 0, dev = 0;
    if (int rc = device_sms(&sms, &dev)) return rc;
    // Tiles of 32 rows where the experts have few (each tile streams its
    // weights whatever its rows: 243 us against 265 with tiles of 256 for 16
    // tokens x 6 of 256 experts), or where so many still fit the SMs at once;
    // pairs of CTAs and 256 rows else (4096 tokens: 1.5 ms against 4).
    const int64_t small_tiles = most_tiles(E, rows, 32, (a.M + 127) / 128);
    const bool small = rows <= 16 * (int64_t)E || small_tiles <= sms;
    a.box = small ? 16 : 32;
    if (!encode_rows(&tb, E_BF16, x, ldx, a.K, rows, a.box, small ? 32 : 128)) return MOE_ERR_CUDA;
    const int steps = (a.K + 63) / 64;
    a.split = small ? split_of(small_tiles, steps, sms) : 1;
    const bool sums = a.out_f32 || a.split > 1 || steps > a.partial;
    cudaStream_t st = as_stream(stream);
    if (small)
        return sums ? launch<MODE, 32, 1, true>(a, small_tiles, sms, dev, ta, tb, ta, st)
                    : launch<MODE, 32, 1, false>(a, small_tiles, sms, dev, ta, tb, ta, st);
    const int64_t tiles = most_tiles(E, rows, 256, (a.M + 255) / 256);
    return sums ? launch<MODE, 256, 2, true>(a, tiles, sms, dev, ta, tb, ta, st)
                : launch<MODE, 256, 2, false>(a, tiles, sms, dev, ta, tb, ta, st);
}

}  // namespace

int gemm_device_error(int clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof v) != cudaSuccess) return MOE_ERR_CUDA;
    if (clear && v) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_gemm_error, &z, sizeof z) != cudaSuccess) return MOE_ERR_CUDA;
    }
    return v;
}

namespace tc {

bool encode_map(CUtensorMap* m, Elem type, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const CUtensorMapDataType t = type == E_U8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : type == E_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(m, t, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(RowMaps* r, Elem type, const void* p, int64_t ld, int width, int rows, int box, int most)
{
    const int size = type == E_U8 ? 1 : 2;
    const uint64_t dims[2] = {(uint64_t)width, (uint64_t)rows}, strides[1] = {(uint64_t)ld * size};
    for (int i = 0; i < kRowMaps && box << i <= most; i++) {
        const uint32_t b[2] = {128u / size, (uint32_t)(box << i)};
        if (!encode_map(&r->m[i], type, 2, p, dims, strides, b)) return false;
    }
    return true;
}

}  // namespace tc
}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm(int32_t experts, int32_t in, int32_t out, const uint16_t* d_x, int64_t ldx,
                                const uint16_t* d_w, const int32_t* d_offsets, int32_t rows, void* d_y, int64_t ldy,
                                int32_t y_dtype, void* stream)
{
    if (int rc = check_gemm_sizes(experts, in, out, rows, 8)) return rc;
    if (!out_dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!words_ok(d_offsets) || !rows_ok(d_x, ldx, in, 2) || !rows_ok(d_w, in, in, 2) || !rows_ok(d_y, ldy, out, dtype_size(y_dtype)))
        return MOE_ERR_INVALID_ARG;
    return row_product<FWD>(experts, in, out, d_x, ldx, d_w, d_offsets, rows, d_y, ldy, y_dtype, stream);
}

extern "C" int moe_grouped_gemm_dx(int32_t experts, int32_t in, int32_t out, const uint16_t* d_dy, int64_t lddy,
                                   const uint16_t* d_w, const int32_t* d_offsets, int32_t rows, void* d_dx,
                                   int64_t lddx, int32_t dx_dtype, void* stream)
{
    if (int rc = check_gemm_sizes(experts, in, out, rows, 8)) return rc;
    if (!out_dtype_ok(dx_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!words_ok(d_offsets) || !rows_ok(d_dy, lddy, out, 2) || !rows_ok(d_w, in, in, 2) ||
        !rows_ok(d_dx, lddx, in, dtype_size(dx_dtype)))
        return MOE_ERR_INVALID_ARG;
    return row_product<DX>(experts, in, out, d_dy, lddy, d_w, d_offsets, rows, d_dx, lddx, dx_dtype, stream);
}

extern "C" int moe_grouped_gemm_dw(int32_t experts, int32_t in, int32_t out, const uint16_t* d_dy, int64_t lddy,
                                   const uint16_t* d_x, int64_t ldx, const int32_t* d_offsets, int32_t rows,
                                   void* d_dw, int32_t dw_dtype, int32_t accumulate, void* stream)
{
    if (int rc = check_gemm_sizes(experts, in, out, rows, 8)) return rc;
    if (!out_dtype_ok(dw_dtype) || !words_ok(d_offsets) || !rows_ok(d_dw, in, in, dtype_size(dw_dtype))) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!rows_ok(d_dy, lddy, out, 2) || !rows_ok(d_x, ldx, in, 2))) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {
        if (!accumulate)
            MOE_CUDA_TRY(cudaMemsetAsync(d_dw, 0, (size_t)experts * out * in * dtype_size(dw_dtype), st));
        return MOE_OK;
    }
    Args a{};
    a.offsets = d_offsets;
    a.out = d_dw;
    a.ldo = in;
    a.out_f32 = dw_dtype == MOE_DT_F32;
    a.accumulate = accumulate ? 1 : 0;
    a.partial = a.out_f32 ? kPartialDw : kPartialBf16;
    a.E = experts;
    a.rows = rows;
    a.M = out;
    a.N = in;
    a.wait = test_wait_cycles(kWaitCycles);
    a.withhold = test_withhold();
    a.direct = a.accumulate && !a.out_f32;
    CUtensorMap ta, to;
    RowMaps tb;
    const uint64_t dims[3] = {(uint64_t)in, (uint64_t)out, (uint64_t)experts};
    const int size = dtype_size(dw_dtype);
    const uint64_t strides[2] = {(uint64_t)in * size, (uint64_t)in * out * size};
    const uint32_t box[3] = {128u / size, 32, 1};
    if (!map_mn(&ta, &a.chunks_a, d_dy, lddy, out, rows, 2, 0) || !map_mn(&tb.m[0], &a.chunks_b, d_x, ldx, in, rows, 4, 0) ||
        !encode_map(&to, a.out_f32 ? E_F32 : E_BF16, 3, d_dw, dims, strides, box))
        return MOE_ERR_CUDA;
    a.box = 256;   // one map of the columns
    a.split = 1;
    int sms = 0, dev = 0;
    if (int rc = device_sms(&sms, &dev)) return rc;
    const int64_t tiles = (int64_t)experts * ((out + 127) / 128) * ((in + 255) / 256);
    return launch<DW, 256, 1, false>(a, tiles, sms, dev, ta, tb, to, st);
}
