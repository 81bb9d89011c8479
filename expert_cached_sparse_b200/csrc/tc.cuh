// Tensor-core (tcgen05), TMA and mbarrier wrappers of the expert matrix
// products (grouped_gemm.cu, grouped_gemm_fp8.cu).  Copies, MMAs and commits
// are issued by one thread, the one elect1() picks in its warp, which walks
// its role's loop alone: against a warp-wide loop with an election per
// instruction four MMAs take 61 cycles to issue instead of 163.
#pragma once

#include <atomic>

#include <cuda.h>

#include "common.cuh"
#include "overlap.cuh"

namespace moe {
namespace tc {

constexpr long long kWaitCycles = 4000000000ll;   // ~2 s: drains, and waits unless a test sets a limit

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// True for one lane of a converged warp.
__device__ __forceinline__ bool elect1()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The cluster address of `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// One arrival by the calling lane on a barrier anywhere in the cluster: what it
// and the lanes of its warp did before is done for whoever waits there with an
// acquire at cluster scope (mbar_try<2>).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ long long ld_cluster64(uint32_t addr)
{
    long long v;
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ------------------------------------------------------------------ inner index split over a cluster
// Calls whose tiles leave most SMs without work give each tile to a cluster of
// a.split CTAs, a share of the inner index each (at most one tile a cluster).
// Their sums meet in the first CTA's shared memory, where the ring was, and
// are added there in the CTAs' order: the same bits every time.
// Called by the warps that hold the sums, `index` the thread's place among
// 128; every other warp of the CTA calls split_others once its work is done.
template <int N>
__device__ __forceinline__ void split_reduce(float (&sum)[N], unsigned char* ring, int rank, int split, int index)
{
    cluster_sync();   // no CTA's copies or MMAs use the rings any more
    if (rank > 0) {
        const uint32_t to = peer_addr(smem_u32(ring) + (uint32_t)(((rank - 1) * N * 128 + index) * 4), 0);
#pragma unroll
        for (int c = 0; c < N; c++) st_cluster(to + 512 * c, sum[c]);
    }
    cluster_sync();
    if (rank == 0)
        for (int r = 1; r < split; r++) {
            const float* from = reinterpret_cast<const float*>(ring) + (r - 1) * N * 128 + index;
#pragma unroll
            for (int c = 0; c < N; c++) sum[c] += from[128 * c];
        }
}
__device__ __forceinline__ void split_others()
{
    __syncwarp();
    cluster_sync();
    cluster_sync();
}

// ------------------------------------------------------------------ mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// An arrival that announces `bytes` of copies.  CG = 2: on a barrier of the
// pair's first CTA, from either.  It publishes nothing itself, so it is a
// relaxed one: the copies' own completion on the barrier is a release at
// cluster scope.
template <int CG = 1>
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    if (CG == 1)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
    else
        asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                     : "memory");
}
// One arrival by the calling lane.
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// CG = 2: a barrier of this CTA on which the pair's other CTA, or work issued
// there, arrives too, so the acquire is one at cluster scope.
template <int CG = 1>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    if (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
    return ok != 0;
}
// Bounded wait: false when another role raised the CTA's abort flag, or after
// `limit` cycles, in which case it raises the flag itself and records
// MOE_ERR_TIMEOUT in *error.
template <int CG = 1>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, long long limit,
                                          int* error)
{
    if (mbar_try<CG>(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try<CG>(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            *abort_flag = 1;
            atomicCAS(error, 0, (int)MOE_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The same for a converged warp: every lane gets the same answer.
template <int CG = 1>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, long long limit,
                                               int* error)
{
    return __all_sync(0xffffffffu, mbar_wait<CG>(bar, parity, abort_flag, limit, error));
}
// Drain wait for this CTA's own copies or MMAs before it exits: bounded by
// time only.
template <int CG = 1>
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity, int* error)
{
    const long long t0 = clock64();
    while (!mbar_try<CG>(bar, parity))
        if (clock64() - t0 > kWaitCycles) {
            atomicCAS(error, 0, (int)MOE_ERR_TIMEOUT);
            return;
        }
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// Copies into this CTA's shared memory.  CG = 2: their barrier may be the
// other CTA's of the pair (`bar` a cluster address).
#define MOE_TC_LOAD(dim, coords, ...)                                                                             \
    do {                                                                                                          \
        if (CG == 1)                                                                                              \
            asm volatile("cp.async.bulk.tensor." dim ".shared::cluster.global.tile.mbarrier::complete_tx::bytes " \
                         "[%0], [%1, " coords "], [%2];" ::"r"(dst), "l"(m), "r"(bar), __VA_ARGS__ : "memory");   \
        else                                                                                                      \
            asm volatile("cp.async.bulk.tensor." dim ".shared::cluster.global.tile.mbarrier::complete_tx::bytes"  \
                         ".cta_group::2 "                                                                         \
                         "[%0], [%1, " coords "], [%2];" ::"r"(dst), "l"(m), "r"(bar), __VA_ARGS__ : "memory");   \
    } while (0)
template <int CG = 1>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar)
{
    MOE_TC_LOAD("2d", "{%3, %4}", "r"(x), "r"(y));
}
template <int CG = 1>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar)
{
    MOE_TC_LOAD("3d", "{%3, %4, %5}", "r"(x), "r"(y), "r"(z));
}
template <int CG = 1>
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w, uint32_t bar)
{
    MOE_TC_LOAD("4d", "{%3, %4, %5, %6}", "r"(x), "r"(y), "r"(z), "r"(w));
}
#undef MOE_TC_LOAD
// Stores of a converged warp's own tiles: ordered by one lane's bulk groups,
// so commit and wait run on lane 0, which issues.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>   // all but the newest N groups have read their source
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Where a copy warp stands: copies issued, next stage, its phase bit.
struct CopyPos {
    long long issued;
    int st;
    uint32_t ph;
};
// A copy warp's loop over the stages of its tiles, walked by one thread:
// next() gives the steps of the next tile or -1, issue(s, bar, address, stage)
// starts the copies of step s and announces their bytes on the stage's barrier
// (`full`: the address of the first one; CG = 2: in the pair's first CTA).
// `withheld`: the first stage is never filled (a test's doing).
template <int STAGE, int CG, class NEXT, class ISSUE>
__device__ __forceinline__ void copy_loop(uint32_t full, uint64_t* empty, unsigned char* ring, int stages,
                                          volatile int* abort_flag, long long limit, bool withheld, int* error,
                                          volatile CopyPos* end, NEXT next, ISSUE issue)
{
    int st = 0, steps;
    uint32_t ph = 0;
    long long issued = 0;
    bool ok = true;
    while (ok && (steps = next()) >= 0)
        for (int s = 0; s < steps; s++) {
            if (!(ok = mbar_wait<CG>(smem_u32(&empty[st]), ph ^ 1, abort_flag, limit, error))) break;
            if (withheld) withheld = false;
            else issue(s, full + 8 * st, smem_u32(ring) + (uint32_t)(st * STAGE), st);
            issued++;
            if (++st == stages) { st = 0; ph ^= 1; }
        }
    end->issued = issued;
    end->st = st;
    end->ph = ph;
}
// End of the two copy warps of a CTA (converged): every issued copy lands
// before the CTA exits.  After an abort one warp may be ahead; the other
// arrives for the stages it did not fill, so that their phases complete with
// the copies in flight.  No divisions: this is on every call's way out.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, volatile CopyPos* end, int mine, bool withheld,
                                             int* error)
{
    asm volatile("bar.sync 1, 64;" ::: "memory");
    int st = end[mine].st, behind = (int)max(0ll, end[!mine].issued - end[mine].issued);
    uint32_t ph = end[mine].ph;
    const long long most = end[mine].issued + behind;
    for (; behind > 0; behind--) {
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&full[st]));
        if (++st == stages) { st = 0; ph ^= 1; }
    }
    if (mine == 0)   // stage i was last filled in this pass over the ring if i < st, else in the previous one
        for (int i = 0; i < stages && i < most; i++)
            if (!(withheld && i == 0)) mbar_drain(smem_u32(&full[i]), i < st ? ph : (ph ^ 1), error);
}

// The same for a pair of CTAs whose copies all complete on the first one's
// barriers: called by one thread there when the copy warps and the MMAs of both
// have ended and one of them gave up (otherwise the MMAs have waited for every
// copy), before either CTA exits.
__device__ __forceinline__ void drain_pair(uint64_t* full, int stages, CopyPos* end, bool withheld, int* error)
{
    long long n[4], most = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        n[i] = ld_cluster64(peer_addr(smem_u32(&end[i & 1].issued), i >> 1));
        most = max(most, n[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (withheld && i < 2 && n[i] > 0) mbar_arrive(smem_u32(&full[0]));
        for (long long k = n[i]; k < most; k++) mbar_arrive(smem_u32(&full[k % stages]));
    }
    for (long long k = max(0ll, most - stages); k < most; k++)
        mbar_drain<2>(smem_u32(&full[k % stages]), (uint32_t)(k / stages) & 1, error);
}

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One arrival on `bar` once every MMA issued so far has finished; for a pair
// (CG = 2) on the barrier at that address in both CTAs.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
                         "r"(bar), "h"((uint16_t)3)
                     : "memory");
}
// `cols` (a power of two >= 32) tensor-memory columns, in both CTAs of a
// pair; the address lands in *slot.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols)
{
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// Shared-memory descriptors in the 128-byte swizzle.  K-major: rows of 128
// bytes (one row per M or N index), 8-row groups 1024 bytes apart.  MN-major:
// rows of 128 bytes (64 16-bit M or N indices) per K index, 8-row groups 1024
// bytes apart, the next 64 M or N indices `chunk` bytes on.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t chunk)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(chunk >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor, fp32 accumulators, M = 128 (128 CG), N = n (a
// multiple of 16 CG): bf16 operands (kind::f16) with either operand MN-major,
// or e4m3 (kind::f8f6f4, K-major, every format field 0).
template <int CG>
__device__ __forceinline__ uint32_t idesc_bf16(int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | (8u * CG << 24);
}
__device__ __forceinline__ uint32_t idesc_e4m3(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }

// D[tmem] (+)= A[smem] B[smem], K = 16 bf16 or 32 e4m3 columns.  A pair's MMA
// is issued by its first CTA: each CTA holds 128 rows of A, half of B's N rows
// and the accumulator of its own 128 rows, all at the same addresses.
#define MOE_TC_MMA(name, kind)                                                                                    \
    template <int CG>                                                                                             \
    __device__ __forceinline__ void name(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)        \
    {                                                                                                             \
        if (CG == 1)                                                                                              \
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                       \
                         "tcgen05.mma.cta_group::1.kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),            \
                         "l"(a), "l"(b), "r"(idesc), "r"(acc));                                                   \
        else                                                                                                      \
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                       \
                         "tcgen05.mma.cta_group::2.kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),            \
                         "l"(a), "l"(b), "r"(idesc), "r"(acc));                                                   \
    }
MOE_TC_MMA(mma_bf16, "f16")
MOE_TC_MMA(mma_e4m3, "f8f6f4")
#undef MOE_TC_MMA

// 16 consecutive columns of the warp's 32 lanes (32 * (warp % 4) on).  The
// registers hold them only after wait_ld, which takes the registers through
// itself so that no use is moved ahead of it.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
                 "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void hold16(uint32_t* v)
{
    asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                      "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                      "+r"(v[15]));
}
__device__ __forceinline__ void wait_ld(uint32_t* v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    hold16(v);
}

// ------------------------------------------------------------------ host: tensor maps
// A tensor of `rank` dimensions (dims[0] innermost), strides in bytes of dims
// 1.., copied in boxes whose inner extent is 128 bytes and that lie in shared
// memory in the 128-byte swizzle.  Reads outside the tensor give zeros,
// writes there nothing.  False when the driver refuses it.
enum Elem { E_BF16, E_F32, E_U8 };
bool encode_map(CUtensorMap* m, Elem type, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box);

// The copies that bring n rows (n <= 256) of a row matrix, 128 bytes of each,
// into shared memory: one map per box height box << i, as few copies as two
// heights allow (the surplus rows cost L2 reads, but a copy's issue costs
// more: see grouped_gemm.cu).
constexpr int kRowMaps = 4;
struct RowMaps {
    CUtensorMap m[kRowMaps];
};
__device__ __forceinline__ int row_units(int n, int box)   // in boxes of the smallest height
{
    int u = (n + box - 1) / box;
    while (__popc(u) > 2) u += u & -u;
    return u;
}
template <int CG = 1>
__device__ __forceinline__ void tma_rows(uint32_t dst, const RowMaps& maps, int x, int row, int units, int box,
                                         uint32_t bar)
{
    for (int i = kRowMaps - 1; i >= 0; i--)
        if (units >> i & 1) {
            tma_2d<CG>(dst, &maps.m[i], x, row, bar);
            dst += (uint32_t)(128 * box << i);
            row += box << i;
        }
}
// Maps of a row matrix with heights box, 2 box, ... up to `most`.
bool encode_rows(RowMaps* r, Elem type, const void* p, int64_t ld, int width, int rows, int box, int most);

}  // namespace tc

// ------------------------------------------------------------------ the plan of a call
// A call's tiles run through its experts, an expert's feature tiles, and
// fastest the blocks of rows of a feature tile.  CTA (or cluster) c of G takes
// tiles c, c + G, c + 2 G, ..., so that what runs at one time is neighbours,
// which share weights and rows in L2.  (Equal contiguous runs of tiles, one a
// CTA, took 1.4 to 1.8 times as long on 4096 tokens: each expert's rows were
// read again for every feature tile.  The largest experts first, for even
// rounds, took up to 1.25 times as long: tiles bound by their weights no longer
// ran beside those bound by MMAs.)
struct PlanExpert {
    int pre;       // blocks of the experts before
    int e, r0, r1; // expert and its rows
};

// How an expert's rows are cut into blocks.
struct RowBlocks {
    int size;   // most rows of a block, a multiple of 32
    __device__ __forceinline__ int blocks(int rows) const { return (rows + size - 1) / size; }
    // rows of a block: equal shares, in 32s
    __device__ __forceinline__ int share(int rows) const
    {
        const int n = blocks(rows);
        return n == 1 ? size : ((rows + n - 1) / n + 31) & ~31;
    }
};

// Rows of expert e; none for a range that no offsets of moe_permute hold.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int rows, int& lo, int& hi)
{
    lo = offsets[e];
    hi = offsets[e + 1];
    if (lo < 0 || hi < lo || hi > rows) lo = hi = 0;
}

// Bytes of a plan's table in shared memory.
__host__ __device__ static inline int plan_bytes(int E) { return (int)align_up(sizeof(PlanExpert) * (E + 1), 128); }

// Builds the table in shared memory: the experts with rows in ascending order,
// then a closing entry {blocks in all}, and their number in *live.  Called by
// the last NT threads of the CTA, beside what the first ones set up; a barrier
// of the CTA has to follow.  Ranges that overlap so often that the blocks pass
// 2^31 void the call.
template <int NT>
__device__ __forceinline__ void build_plan(const int32_t* offsets, int E, int rows, const RowBlocks& B,
                                           PlanExpert* tab, long long* scratch, int* live)
{
    const int tid = threadIdx.x - (blockDim.x - NT), lane = tid & 31, warp = tid >> 5, nt = NT;
    const int per = (E + nt - 1) / nt, e0 = min(E, tid * per), e1 = min(E, e0 + per);
    // experts in the low 13 bits, blocks above: one sum for both
    long long sum = 0;
    for (int e = e0; e < e1; e++) {
        int lo, hi;
        expert_rows(offsets, e, rows, lo, hi);
        if (hi > lo) sum += ((long long)B.blocks(hi - lo) << 13) + 1;
    }
    long long in = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += x;
    }
    if (lane == 31) scratch[warp] = in;
    asm volatile("bar.sync 2, %0;" ::"n"(NT) : "memory");
    long long base = in - sum, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w++) {
        if (w < warp) base += scratch[w];
        total += scratch[w];
    }
    const bool voided = total >> 13 > 0x7fffffff;
    const int n = voided ? 0 : (int)(total & 8191);
    if (!voided)
        for (int e = e0; e < e1; e++) {
            int lo, hi;
            expert_rows(offsets, e, rows, lo, hi);
            if (hi == lo) continue;
            tab[base & 8191] = {(int)(base >> 13), e, lo, hi};
            base += ((long long)B.blocks(hi - lo) << 13) + 1;
        }
    if (tid == 0) {
        tab[n] = {voided ? 0 : (int)(total >> 13), 0, 0, 0};
        *live = n;
    }
}

// A tile: the m-th feature tile of expert e, n rows from r0 on.
struct PlanTile {
    int e, m, r0, n;
};

// Walks a CTA's tiles: number `part` of `parts`, mt feature tiles an expert.
struct PlanWalk {
    const PlanExpert* tab;
    const RowBlocks B;
    int live, mt, i, parts, span;
    long long u, total;

    __device__ PlanWalk(const PlanExpert* t, int live_, const RowBlocks& b, int mt_, int part, int parts_)
        : tab(t), B(b), live(live_), mt(mt_), i(0), parts(parts_), span(parts_ / mt_ + 1), u(part), total((long long)t[live_].pre * mt_)
    {
    }
    // This CTA's share [lo, hi) of `steps` steps of the inner index, with the index split over
    // a cluster.  Offsets that no call of moe_permute writes (ranges that overlap) can make
    // more tiles than clusters: the first CTA of each then does them alone.
    __device__ __forceinline__ void split_steps(int steps, int rank, int& split, int& lo, int& hi)
    {
        if (split > 1 && total > parts) {
            if (rank) total = 0;
            split = 1;
        }
        lo = split > 1 ? steps * rank / split : 0;
        hi = split > 1 ? steps * (rank + 1) / split : steps;
    }
    __device__ __forceinline__ bool next(PlanTile& v)
    {
        if (u >= total) return false;
        int hi = min(live - 1, i + span);   // every expert has mt tiles at least
        while (i < hi) {                     // the last expert whose first tile is at most u
            const int mid = (i + hi + 1) >> 1;
            if ((long long)tab[mid].pre * mt <= u) i = mid;
            else hi = mid - 1;
        }
        const PlanExpert x = tab[i];
        const long long r = u - (long long)x.pre * mt;
        u += parts;
        const int n = x.r1 - x.r0, nt = B.blocks(n);
        if (nt == 1) {   // no divisions: a small tile is not much longer than they take
            v = {x.e, (int)r, x.r0, n};
            return true;
        }
        int m, t;
        if (r < 0x7fffffff) {   // a 64-bit division takes hundreds of cycles
            m = (int)r / nt;
            t = (int)r - m * nt;
        } else {
            m = (int)(r / nt);
            t = (int)(r % nt);
        }
        const int share = B.share(n), r0 = x.r0 + t * share;
        v = {x.e, m, r0, min(share, x.r1 - r0)};
        return true;
    }
};

// Rows that the MMAs of a tile of n rows take: a multiple of 16 for each CTA.
template <int CG>
__device__ __forceinline__ int mma_rows(int n)
{
    return (n + 16 * CG - 1) / (16 * CG) * (16 * CG);
}

// Most tiles that `rows` rows of E experts can make: blocks of `size` rows by mt feature tiles.
static inline int64_t most_tiles(int E, int rows, int size, int64_t mt)
{
    const int64_t live = E < rows ? E : rows, blocks = rows / size + live;
    return mt * (blocks < rows ? blocks : rows);
}
// CTAs to split the inner index over, given the most tiles (of few rows) and
// the steps of a tile: as many as leave every tile its cluster on three
// quarters of the SMs (clusters do not pack them all) and four steps a CTA.
static inline int split_of(int64_t tiles, int steps, int sms)
{
    int split = 1;
    while (split < 8 && tiles * split * 2 <= sms * 3 / 4 && steps >= 8 * split) split *= 2;
    return split;
}

// CTAs in clusters of CG: one CTA an SM, but no more clusters than tiles.
template <class... P, class... A>
static inline cudaError_t launch_clusters(void (*kern)(P...), int sms, int64_t tiles, int CG, int threads, int smem,
                                          cudaStream_t st, const A&... args)
{
    return launch_overlapped(kern, (int)(tiles < sms / CG ? tiles : sms / CG) * CG, CG, threads, smem, st, args...);
}

// ------------------------------------------------------------------ host: checks common to the products
constexpr int64_t kMaxGemmDim = 1 << 20;
constexpr int kSmemMax = 227 * 1024;

static inline int check_gemm_sizes(int experts, int in, int out, int rows, int in_multiple)
{
    if (experts <= 0 || in <= 0 || in % in_multiple || out <= 0 || out % 8 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (experts > kMaxExperts || in > kMaxGemmDim || out > kMaxGemmDim || rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
// A matrix of 16-byte aligned rows of `width` elements of `size` bytes.
static inline bool rows_ok(const void* p, int64_t ld, int64_t width, int size)
{
    return p && !((uintptr_t)p & 15) && ld >= width && ld < ((int64_t)1 << 36) && (ld * size) % 16 == 0;
}
// int32 or float32 values.
static inline bool words_ok(const void* p) { return p && !((uintptr_t)p & 3); }
static inline bool out_dtype_ok(int t) { return t == MOE_DT_F32 || t == MOE_DT_BF16; }
static inline int dtype_size(int t) { return t == MOE_DT_F32 ? 4 : 2; }

// SMs of the current device, and its number.
static inline int device_sms(int* sms, int* dev)
{
    static std::atomic<int> count[kMaxDevices];
    MOE_CUDA_TRY(cudaGetDevice(dev));
    if (*dev < 0 || *dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
    if (!(*sms = count[*dev].load(std::memory_order_relaxed))) {
        MOE_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev));
        count[*dev].store(*sms, std::memory_order_relaxed);
    }
    return MOE_OK;
}
// Lets a kernel use `most` bytes of dynamic shared memory, once a device (`set`: a flag each).
template <class K>
static inline int allow_smem(K* kern, int most, std::atomic<int>* set, int dev)
{
    if (!set[dev].load(std::memory_order_relaxed)) {
        MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        set[dev].store(1, std::memory_order_relaxed);
    }
    return MOE_OK;
}

}  // namespace moe
