// Window attention over a paged cache, head_dim 512, on pairs of SMs (tcgen05 with cta_group::2).
//
// Formulation.  Every query row of a sequence (token x head) attends to rows that its neighbours attend to
// too, so a task is 128 query rows: consecutive (token, head) rows of one sequence (two tokens of 64 heads,
// one of 128, eight of 16).  A pair of SMs shares the task, 64 rows each:
//   S[128 x 128] = Q[128 x 512] . K^T      a tile: four blocks of 32 positions; each SM holds 64 rows of Q and
//                                          the 512-wide rows of two of the blocks
//   O[128 x 512] += P[128 x 128] . V       each SM holds its 64 rows of P and all four blocks' rows in its half
//                                          of d
// Both are M = 128 products of the pair: an SM's 64 rows fill its 128 TMEM lanes, lanes 0-63 with the first
// half of the columns and 64-127 with the second.  One SM alone would have O of 128 rows x 512 in all of its
// TMEM, and M = 64 products run at half the rate (64 rows x N 256 x K 16 take 64 cycles a SM here, measured).
// TMEM: O in 256 columns, three S buffers of 64, and the softmax's running maxima and sums.
//
// Blocks, not rows, are loaded: 32 positions lie in one page (a page is a multiple of 32 rows), so a block is a TMA
// box and there is no gather.  K (stages of 64 rows x 128 of d, 16 KB) and V (of a block x 256 of d) go through a ring
// of four stages each, a tile's worth: the two rows of one position that a SM needs for K and for V are other halves,
// and are fetched from L2 separately.  The softmax of a tile runs behind the next two tiles' logits.
//
// Masked positions.  A block is loaded whole, so rows that some or all of the task's tokens do not see come
// with it, and they may hold anything.  Their p is set to zero, but 0 x NaN is NaN: a logit that is not finite in
// a column that not every token sees makes the softmax warps look at that row of V (in their half of d) before the
// product, and clear what is not finite in it.  A row that is not finite gives every query row such a logit, those behind
// the task's last among them (they find it where a CTA has none of the task's own); a query row that is not finite
// gives one to every position, whose rows are not touched then.  Rows that see a bad row have a NaN there anyway.
//
// Roles (each CTA of the pair, 22 warps): warps 0 and 21 issue the pair's logits and P.V (rank 0; rank 1's warp 21
// passes on that its V has landed); warp 1 turns units into tasks, up to four ahead; warp 2 loads K, warp 20 V,
// warp 3 Q; warps 4-7 and 8-11 softmax, every second tile each; warps 12-15 and 16-19 epilogue, half of d each.
// Rows of codes (32 warps) are widened to bf16 in the same stages: warp 2 describes the tiles and pulls their rows
// into L2, warps 16-23 widen K and 24-31 V, warps 12-15 are the epilogue, warp 1 loads Q too and warp 3 issues P.V.
// Every wait is bounded; one that gives up raises the timeout bit and every role unwinds.
//
// What it measured (a call among others, the range over several GPUs; b sequences of one token but for the prompts): 128
// heads, window 4096 + 128 first, b = 256: 258-272 us, 4.3-4.6 TB/s of cache; 64 heads, window 128, a prompt of 4095
// with the rotation: 139-143 us, 3.8 TB/s of q and o (over e4m3 rows 204, e2m1 202); 128 heads, window 2048, prompts of
// 4096 tokens in all: 1.62-1.67 ms, 1.4 PFLOP/s; e4m3 rows, 64 heads, window 1024, b = 64: 39 us; e2m1 rows, 16 heads,
// window 512, 240 tokens of 48 sequences: 23 us.  Long windows of bf16 rows are bound by L2, out of which each row comes
// twice (pulled into L2 ahead they take longer), prompts of short windows by a task's chain (Q, logits, softmax, P.V, O
// out: O has one buffer), codes by the widening's instructions.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "sa_fp4.cuh"
#include "sa_fp8.cuh"
#include "sa_internal.cuh"
#include "sa_paged.cuh"
#include "sa_tc.cuh"

namespace sa {
namespace {

using namespace tc;

constexpr int kD = 512;
constexpr int kM = 128;            // query rows of a task
constexpr int kBlock = 32;         // positions of a block
constexpr int kTileBlocks = 4;     // blocks of a tile
constexpr int kKStages = 4, kVStages = 4;  // of the two rings
constexpr int kInfos = 8, kTasks = 4;  // tiles and tasks described ahead
// Warps: the first four, softmax and the first epilogue group are the same for every format
constexpr bool codes_of(int fmt) { return fmt != SA_KV_BF16; }
constexpr int epilogue_groups(int fmt) { return codes_of(fmt) ? 1 : 2; }
constexpr int kWarpEpilogue = 12;
constexpr int kWarpWiden = 16;                                            // codes: eight warps of K, eight of V
constexpr int warp_v(int fmt) { return codes_of(fmt) ? -1 : 20; }         // bf16: V's loads
constexpr int warp_q(int fmt) { return codes_of(fmt) ? 1 : 3; }           // (codes: the tasks' warp loads Q too)
constexpr int warp_pv(int fmt) { return codes_of(fmt) ? 3 : 21; }
constexpr int warps_of(int fmt) { return codes_of(fmt) ? 32 : 22; }
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// TMEM columns: O, three S buffers, a row's running maximum after the last two tiles, and the softmax groups' final
// maxima and sums
constexpr uint32_t kColO = 0, kColS = 256, kColM = 448, kColT = 452;

constexpr uint32_t kStageBytes = 16384;
constexpr uint32_t kQBytes = 65536;  // [8 blocks of 64 d][64 rows][128 B]
constexpr uint32_t kPBytes = 16384;  // [2 halves of the columns][64 rows][128 B], two buffers
constexpr uint32_t kOffK = 0;
constexpr uint32_t kOffV = kOffK + kKStages * kStageBytes;
constexpr uint32_t kOffQ = kOffV + kVStages * kStageBytes;
constexpr uint32_t kOffP = kOffQ + kQBytes;
constexpr uint32_t kOffMisc = kOffP + 2 * kPBytes;

struct Task {
    int row0, rows;   // its first row among all of q's, and how many are its own
    int tok0, off0;   // that row's token and head
    int pos0;         // that token's position
    int pmax;         // its last token's
    int seq, split;
    int k0, nb;       // the unit's blocks: k0 .. k0 + nb - 1 of the task's
    int fb, wb;       // block k of the task is k < fb ? k : k - fb + wb of the sequence
    int more;         // 0: no further task
};

struct Misc {
    // full: of K and Q both CTAs' parts have landed (rank 0's); of V this CTA's, in rank 0 the other's too, which
    // passes it on
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t q_full[4], q_empty[4];          // (a quarter of Q)
    uint64_t s_full[3], s_empty[3];          // (s_empty, p_full, o_empty: rank 0's, both CTAs arrive)
    uint64_t p_full[2], p_empty[2], o_full, o_empty;
    uint64_t info_full[kInfos], info_empty[kInfos];  // (info_empty: codes)
    uint64_t task_full[kTasks], task_empty[kTasks];
    uint64_t stats_full, stats_empty;
    uint64_t pair_bar[2][2], mx_empty[2][2], m_full[4], sum_full[2], sum_empty[2], done;
    uint32_t tmem_base;
    int abort;
    int base[kInfos][kTileBlocks];    // first position of a tile's blocks: -1 no page, -2 no block
    int rows[kInfos][kTileBlocks];    // codes: their first rows in the pool
    int whole[kInfos];                // every token of the task sees every position of the tile's blocks
    Task task[kTasks];
    float mx[2][128];
    float sum[128];
};
constexpr uint32_t kSmem = kOffMisc + sizeof(Misc);
static_assert(kSmem <= 232448, "shared memory budget");

struct Params {
    paged::Batch a;
    const uint8_t* kv8;       // codes and their scales
    const uint8_t* kv_scale;
    const float* sink;
    __nv_bfloat16* o;
    float* lse;
    float* part_ml;
    float* part_o;
    uint32_t* status;
    const float* rope;
    int64_t npos;
    int rope_dim;
    float scale_log2;
    int n;               // tokens
    int h;
    int window, first;
    int n_splits;
    int units;           // no more than these
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An address of this CTA's shared memory in rank 0's.
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// An arrival at a barrier of either CTA.  What it announces is in shared memory or TMEM, for the tensor core to read
// (behind a proxy or tcgen05 fence) or to overwrite, so that the default scope does: arrivals and waits of
// cluster scope wait for a thread's global writes too, and made a tile take 10 k cycles.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A wait by a converged warp, with a warp-uniform result.  The hardware suspends the warp until the phase completes or
// a millisecond has passed (a poll that returns at once takes issue slots from the warps that work); bounded to
// some two seconds, and left as soon as another role has given up.  (Out of line: see the note on code below.)
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
    for (int i = 0; i < 2000; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity & 1), "r"(1000000u)
            : "memory");
        if (__all_sync(0xffffffffu, ok != 0)) return true;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
    }
    *abort = 1;
    return false;
}
static __device__ __noinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
    return wait_here(bar, parity, abort);
}
__device__ __forceinline__ bool wait(uint64_t& bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, wait_for(smem_addr(&bar), parity, abort));
}
// The same for a phase that has most likely completed long ago: looked at in line first.
__device__ __forceinline__ bool wait_done(uint64_t& bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_test_wait(smem_addr(&bar), parity & 1)) || wait(bar, parity, abort);
}
// One arrival for a converged warp, after what every lane did.
__device__ __forceinline__ void warp_arrive(uint64_t& bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&bar));
}
__device__ __forceinline__ void warp_arrive_leader(uint64_t& bar, int lane) {
    __syncwarp();
    if (lane == 0) arrive_at(at_leader(smem_addr(&bar)));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The same, and (cta_group::2) into this CTA with the barrier in either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(
            dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// The pair's product, from the words of its descriptors (the same in both CTAs); one elected lane issues.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .b64 da, db;\n .reg .pred p, e;\n mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
        " setp.ne.b32 p, %6, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at a barrier in both CTAs once every product issued so far has completed.
__device__ __forceinline__ void commit_pair(uint64_t& bar) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b16 m;\n mov.b16 m, 3;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(
            smem_addr(&bar))
        : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// One, two and four 32-bit words of a thread's own TMEM lane.
__device__ __forceinline__ float tmem_ld_x1(uint32_t at) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
    tmem_wait_ld();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_ld_x4(uint32_t at, float& a, float& b, float& c, float& d) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
    tmem_wait_ld();
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
    c = __uint_as_float(r[2]);
    d = __uint_as_float(r[3]);
}
__device__ __forceinline__ void tmem_st_x1(uint32_t at, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(__float_as_uint(v)) : "memory");
    tmem_wait_st();
}
__device__ __forceinline__ void tmem_st_x2(uint32_t at, float a, float b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at), "r"(__float_as_uint(a)),
                 "r"(__float_as_uint(b))
                 : "memory");
    tmem_wait_st();
}
// Whether one of eight bf16 in shared memory is an infinity or a NaN.
__device__ __forceinline__ bool any_not_finite(uint32_t at) {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
    bool any = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        any |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
    return any;
}
// 32 bytes at a 32-byte aligned address
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Bits lo .. hi of a word (none where hi < lo).
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 31);
    return hi < lo ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}
// The positions base .. base + 31 that every token from position p0 to p1 sees.
static __device__ __noinline__ uint32_t seen(int window, int first, int base, int p0, int p1) {
    return base < 0 ? 0u : bits(p1 - window + 1 - base, p0 - base) | bits(0, min(first - 1, p0) - base);
}

// Walks the sequences, 32 at a time, to the one that a tile of 128 rows is in; the tiles asked for rise.  (The whole warp.)
struct Walk {
    int seq0 = -32;
    uint32_t before = 0, total = 0;         // the sequences at hand are from seq0 on, with the tiles before and in them
    int q0 = 0, q1 = 0, len = 0;            // lane l: sequence seq0 + l's tokens and length
    uint32_t upto = 0;                      // and its and its forerunners' tiles

    // Sequence and tile in it, or false: there are no more.
    __device__ __forceinline__ bool find(const Params& p, uint32_t tile, int lane, int& seq, int& at, int& from, int& to,
                                         int& length) {
        while (tile >= before + total) {
            before += total;
            seq0 += 32;
            if (seq0 < 0 || seq0 >= p.a.b) return false;  // (2^31 - 1 sequences: seq0 wraps)
            const int64_t s = (int64_t)seq0 + lane;
            q0 = q1 = len = 0;
            if (s < p.a.b) {
                len = __ldg(p.a.kv_len + s);
                q0 = min(max(__ldg(p.a.q_start + s), 0), p.n);
                q1 = min(max(__ldg(p.a.q_start + s + 1), q0), p.n);
            }
            upto = ((uint32_t)(q1 - q0) * (uint32_t)p.h + kM - 1) / kM;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            total = __shfl_sync(0xffffffffu, upto, 31);
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, upto > tile - before)) - 1;
        const uint32_t prev = __shfl_sync(0xffffffffu, upto, who == 0 ? 0 : who - 1);
        seq = seq0 + who;
        at = (int)(tile - before - (who == 0 ? 0 : prev));
        from = __shfl_sync(0xffffffffu, q0, who);
        to = __shfl_sync(0xffffffffu, q1, who);
        length = __shfl_sync(0xffffffffu, len, who);
        return true;
    }
};

// Unit u -> its task (the whole warp calls, with rising u); false: there are no more.
__device__ __forceinline__ bool task_of(const Params& p, int u, int lane, Walk& walk, Task& t) {
    const int tile = u / p.n_splits;
    int seq, at, q0, q1, len;
    if (!walk.find(p, tile, lane, seq, at, q0, q1, len)) return false;
    const int r0 = at * kM, rows = (q1 - q0) * p.h - r0;
    t.seq = seq;
    t.split = u - tile * p.n_splits;
    t.rows = min(rows, kM);
    const int tok = r0 / p.h;
    t.off0 = r0 - tok * p.h;
    t.tok0 = q0 + tok;
    t.row0 = q0 * p.h + r0;
    // (lengths far outside the table's range, which are errors, are held where 32 bits do)
    const int64_t pos = (int64_t)len - (q1 - q0) + tok;
    t.pos0 = (int)min(max(pos, -(int64_t(1) << 30)), (int64_t(1) << 31) - 1 - kM);
    t.pmax = t.pos0 + (t.off0 + t.rows - 1) / p.h;
    // blocks: the first positions' and the window's, those of both once; none past the table's last page
    const int last = (int)min((int64_t)t.pmax, p.a.max_pages * p.a.page - 1);
    if (last < t.pmax) atomicOr(p.status, kStatusBadIndex);
    t.fb = t.wb = t.k0 = t.nb = 0;
    if (last >= 0) {
        t.fb = (int)((uint32_t)(min(p.first, last + 1) + kBlock - 1) / kBlock);
        t.wb = max((int)((uint32_t)max(0, t.pos0 - p.window + 1) / kBlock), t.fb);
        const int n = t.fb + max(0, (int)((uint32_t)last / kBlock) - t.wb + 1);
        const int per = (n + kTileBlocks * p.n_splits - 1) / (kTileBlocks * p.n_splits) * kTileBlocks;
        t.k0 = min(t.split * per, n);
        t.nb = min(n, t.k0 + per) - t.k0;
    }
    return true;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Rows of codes widened into the stages, in place: a warp copies its share of a stage's codes, `kLoads` pieces of 16 bytes
// a lane, and their scales into the part of the stage that its bf16 rows will fill, ahead of the one that it reads back
// and writes widened.  (Through registers, a warp waited for its loads, and every scoreboard that they share.)
template <int kFmt>
struct Widen {
    static constexpr int kLoads = kFmt == SA_KV_FP8_E4M3 ? 4 : 2;
    static constexpr int kRowBytes = kFmt == SA_KV_FP8_E4M3 ? kD : kD / 2;
    uint4 code[kLoads];
    uint32_t scale[kLoads];

    // `own` is the warp's part of the stage, which goes on every `hop` bytes; a lane's codes start at `src`, the pieces
    // `step` rows apart, and a word of scales for every one of 16 lanes at `sc`.
    static __device__ __forceinline__ void copy(uint32_t own, int hop, const uint8_t* src, int step, const uint8_t* sc,
                                                int lane) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x)
            copy16(own + (x >> 1) * hop + (x & 1) * 512 + 16 * lane, src + x * step * kRowBytes);
        if (lane < 16) copy4(own + 2 * hop + 4 * lane, sc);
    }
    // Back: a lane's own pieces, and its rows' scales (`at`, and `by` bytes from piece to piece).
    __device__ __forceinline__ void read(uint32_t own, int hop, int at, int by, int lane) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(code[x].x), "=r"(code[x].y), "=r"(code[x].z), "=r"(code[x].w)
                         : "r"(own + (x >> 1) * hop + (x & 1) * 512 + 16 * lane)
                         : "memory");
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(scale[x]) : "r"(own + 2 * hop + at + x * by) : "memory");
        }
    }
    // Into a stage whose groups of eight rows are `group` bytes apart and whose blocks of 64 d `block`; the rows in the
    // stage start at `first`.  (Lanes of a row that hold the same place of different blocks, which are the same
    // banks, store their 16-byte units in different orders.)
    __device__ __forceinline__ void store(uint32_t stage, int first, int lanes, int group, int block, int lane) const {
        const int ul = lane & (lanes - 1), step = 32 / lanes, r0 = first + lane / lanes;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            const int r = r0 + step * x;
            const uint32_t row = stage + (uint32_t)((r >> 3) * group + (r & 7) * 128);
            if constexpr (kFmt == SA_KV_FP8_E4M3) {
                uint4 lo, hi;
                fp8::dequant16(code[x], fp8::e8m0_to_f32(scale[x]), lo, hi);
                const int u = 2 * ul, turn = (ul >> 2) & 1;
                const uint32_t at = row + (uint32_t)((u >> 3) * block) + (uint32_t)((((u & 7) | turn) ^ (r & 7)) << 4);
                const uint4 a = turn ? hi : lo, b = turn ? lo : hi;
                st_shared_v4(at, a.x, a.y, a.z, a.w);
                st_shared_v4(at ^ 16u, b.x, b.y, b.z, b.w);
            } else {
                const int u = 4 * ul, turn = lanes == 8 ? (ul >> 1) & 3 : ul & 2;
                const uint32_t at = row + (uint32_t)((u >> 3) * block) + (uint32_t)(((u & 7) ^ (r & 7)) << 4);
                const float sc = fp4::scale_f32(scale[x]);
                uint32_t w[4] = {code[x].x, code[x].y, code[x].z, code[x].w};
                if (turn & 1) {
                    uint32_t v = w[0];
                    w[0] = w[1];
                    w[1] = v;
                    v = w[2];
                    w[2] = w[3];
                    w[3] = v;
                }
                if (turn & 2) {
                    uint32_t v = w[0];
                    w[0] = w[2];
                    w[2] = v;
                    v = w[1];
                    w[1] = w[3];
                    w[3] = v;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 v = fp4::dequant8(w[k], sc);
                    st_shared_v4(at ^ (uint32_t)((k ^ turn) << 4), v.x, v.y, v.z, v.w);
                }
            }
        }
    }
};

template <int kFmt, bool kRope>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * warps_of(kFmt), 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ Params p) {
    constexpr bool kCodes = codes_of(kFmt);
    constexpr int kEpilogues = epilogue_groups(kFmt), kWarpV = warp_v(kFmt), kWarpPv = warp_pv(kFmt);
    extern __shared__ __align__(1024) uint8_t smem[];
    Misc& M = *reinterpret_cast<Misc*>(smem + kOffMisc);
    const uint32_t s_k = smem_addr(smem + kOffK), s_v = smem_addr(smem + kOffV), s_q = smem_addr(smem + kOffQ),
                   s_p = smem_addr(smem + kOffP);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = __shfl_sync(0xffffffffu, cta_rank(), 0);  // (warp-uniform for the compiler too)
    volatile int* abort = &M.abort;
    pdl_trigger();
    if (smem_addr(smem) & 1023u) {  // (the swizzle's alignment, which leaves no room to be rounded to)
        if (tid == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(smem_addr(&M.k_full[s]), kCodes ? 8 : 2);  // (both CTAs' loading warp, or widening warps)
            mbar_init(smem_addr(&M.k_empty[s]), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(smem_addr(&M.v_full[s]), (kCodes ? 4 : 1) * (rank == 0 ? 2 : 1));
            mbar_init(smem_addr(&M.v_empty[s]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&M.q_full[i]), 1);
            mbar_init(smem_addr(&M.q_empty[i]), 1);
        }
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(smem_addr(&M.info_full[i]), 1);
            mbar_init(smem_addr(&M.info_empty[i]), 20);  // (codes: the widening warps and a softmax group)
        }
        for (int i = 0; i < kTasks; ++i) {
            mbar_init(smem_addr(&M.task_full[i]), 1);
            mbar_init(smem_addr(&M.task_empty[i]), warps_of(kFmt) - 1);  // all but the one that fills it
        }
        for (int b = 0; b < 3; ++b) {
            mbar_init(smem_addr(&M.s_full[b]), 1);
            mbar_init(smem_addr(&M.s_empty[b]), 8);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&M.pair_bar[b][0]), 2);
            mbar_init(smem_addr(&M.pair_bar[b][1]), 2);
            mbar_init(smem_addr(&M.mx_empty[b][0]), 2);
            mbar_init(smem_addr(&M.mx_empty[b][1]), 2);
            mbar_init(smem_addr(&M.sum_full[b]), 2 * kEpilogues);
            mbar_init(smem_addr(&M.sum_empty[b]), 2 * kEpilogues);
            mbar_init(smem_addr(&M.p_full[b]), 8);
            mbar_init(smem_addr(&M.p_empty[b]), 1);
        }
        mbar_init(smem_addr(&M.o_full), 1);
        mbar_init(smem_addr(&M.o_empty), 8 * kEpilogues);
        for (int w = 0; w < 4; ++w) mbar_init(smem_addr(&M.m_full[w]), 1);
        mbar_init(smem_addr(&M.stats_full), 8);
        mbar_init(smem_addr(&M.stats_empty), 4 * kEpilogues);
        mbar_init(smem_addr(&M.done), 2);
        M.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&M.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (!kCodes && warp == 2 && lane == 0) {
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (warp == warp_q(kFmt) && lane == 0) tma_prefetch_desc(&q_map);
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // the other CTA's barriers and TMEM are there
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, M.tmem_base, 0);
    // the set-up above touches no global memory; everything below may read what the work queued before this launch
    // writes
    pdl_wait();

    // The tasks, in turn: fetch(t) waits for the next one's description; false: none is left (or a wait gave up).
    uint32_t nth = 0;
    bool ok = true;
    auto fetch = [&](Task& t) {
        const uint32_t i = nth % kTasks;
        ok = ok && wait(M.task_full[i], nth / kTasks, abort);
        if (!ok) return false;
        t = M.task[i];
        warp_arrive(M.task_empty[i], lane);
        ++nth;
        // (uniform for the compiler too, so that the loops over them are)
        t.nb = __shfl_sync(0xffffffffu, t.nb, 0);
        return __shfl_sync(0xffffffffu, t.more, 0) != 0;
    };

    uint32_t q_tasks = 0, q_sent = 0;
    auto load_q = [&](int row0) {
        for (int q = 0; q < 4 && ok; ++q) {
            if (!(ok = wait(M.q_empty[q], q_tasks ^ 1u, abort))) break;
            if (lane == 0) {
                const uint32_t bar = smem_addr(&M.q_full[q]);
                if (rank == 0) mbar_arrive_expect_tx(bar, 2 * 16384);
                tma_load_3d_pair(s_q + q * 16384, &q_map, 0, row0 + 64 * (int)rank, 2 * q, at_leader(bar));
            }
            ++q_sent;
        }
        ++q_tasks;
    };
    auto drain_q = [&] {
        if (!ok && lane == 0 && rank == 0)
            for (uint32_t k = q_sent > 4 ? q_sent - 4 : 0; k < q_sent; ++k)
                mbar_drain(smem_addr(&M.q_full[k % 4]), (k / 4) & 1);
    };

    if (warp == 1) {
        // ------------------------------------------------------------------ tasks
        const int pairs = gridDim.x >> 1;
        Walk walk;
        for (int u = blockIdx.x >> 1; ok; u += pairs) {
            Task t = {};
            const bool more = u < p.units && task_of(p, u, lane, walk, t);
            t.more = more;
            const uint32_t i = nth % kTasks;
            if (!(ok = wait(M.task_empty[i], (nth / kTasks) ^ 1u, abort))) break;
            if (lane == 0) M.task[i] = t;
            warp_arrive(M.task_full[i], lane);
            ++nth;
            if (!more) break;
            if (kCodes && t.nb) load_q(t.row0);
        }
        if (kCodes) drain_q();
    } else if (warp == 0 || warp == kWarpPv) {
        // ------------------------------------------------------------------ the pair's products
        // Warp 0 issues the logits, another one P.V (of bf16 rows, rank 1's passes on that its V has landed).  One warp for
        // both spent 600 cycles a stage of 256 cycles of products (a wait for a barrier that has long completed takes
        // 130, a commit 75, and the tensor pipe holds too few products to bridge them); of two, one's products run
        // behind the other's barriers.
        constexpr uint32_t id_s = idesc_bf16_f32(kM, 128, false, false);
        constexpr uint32_t id_o = idesc_bf16_f32(kM, 256, false, true);
        const uint64_t a_s = smem_desc_sw128(s_q, 16, 1024), b_s = smem_desc_sw128(s_k, 16, 2048);
        const uint64_t a_o = smem_desc_sw128(s_p, 16, 1024), b_o = smem_desc_sw128(s_v, 4096, 1024);
        const bool leader = rank == 0;
        uint32_t st = 0, st_use = 0, g = 0, c = 0;
        bool landed = false;  // stage st has: its barrier was looked at while the stage before it was issued
        auto stage_in = [&](uint64_t* full) {
            if (!landed) ok = ok && wait(full[st], st_use, abort);
            return ok;
        };
        auto peek = [&](uint64_t* full, uint32_t stages) {
            const uint32_t n = st + 1 == stages ? 0 : st + 1;
            return mbar_test_wait(smem_addr(&full[n]), (st_use + (n == 0)) & 1);
        };
        auto stage_out = [&](uint64_t* empty, uint32_t stages, bool next) {
            if (leader) {
                commit_pair(empty[st]);
                landed = __all_sync(0xffffffffu, next);
            }
            if (++st == stages) {
                st = 0;
                ++st_use;
            }
        };
        Task t;
        if (warp == 0 && !leader) {
            while (fetch(t)) {
            }
        } else if (warp == 0) {
            while (fetch(t)) {
                if (t.nb == 0) continue;
                const int nt = (t.nb + kTileBlocks - 1) / kTileBlocks;
                for (int i = 0; i < nt && ok; ++i, ++g) {
                    const uint32_t b = g % 3;
                    ok = wait(M.s_empty[b], (g / 3) ^ 1u, abort);
                    for (int q = 0; q < 4 && ok; ++q) {
                        if (i == 0) {
                            ok = wait(M.q_full[q], c, abort);
                        }
                        if (!ok || !stage_in(M.k_full)) break;
                        tc_fence_after();
                        const bool next = peek(M.k_full, kKStages);
                        const uint32_t alo = (uint32_t)a_s + q * (16384 >> 4);
                        const uint32_t blo = (uint32_t)b_s + st * (kStageBytes >> 4);
#pragma unroll 4
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t at = (k & 3) * (32 >> 4);
                            mma_pair(tmem + kColS + 64 * b, alo + (k >> 2) * (8192 >> 4) + at, (uint32_t)(a_s >> 32),
                                     blo + (k >> 2) * (1024 >> 4) + at, (uint32_t)(b_s >> 32), id_s, (q | k) != 0);
                        }
                        if (i == nt - 1) commit_pair(M.q_empty[q]);
                        stage_out(M.k_empty, kKStages, next);
                    }
                    if (ok) commit_pair(M.s_full[b]);
                }
                ++c;
            }
        } else if (kCodes && !leader) {
            while (fetch(t)) {
            }
        } else {
            while (fetch(t)) {
                if (t.nb == 0) continue;
                for (int i = 0; 4 * i < t.nb && ok; ++i, ++g) {
                    if (leader) {
                        ok = wait(M.p_full[g & 1], g >> 1, abort);
                        if (i == 0) ok = ok && wait(M.o_empty, c ^ 1u, abort);
                        tc_fence_after();
                    }
                    const int nb = min(kTileBlocks, t.nb - kTileBlocks * i);
                    for (int j = 0; j < nb && ok; ++j) {
                        if (!stage_in(M.v_full)) break;
                        if (!kCodes && !leader) warp_arrive_leader(M.v_full[st], lane);
                        bool next = false;
                        if (leader) {
                            tc_fence_after();
                            next = peek(M.v_full, kVStages);
                            const uint32_t alo =
                                (uint32_t)a_o + (g & 1) * (kPBytes >> 4) + (j & 1) * (8192 >> 4) + (j >> 1) * (64 >> 4);
                            const uint32_t blo = (uint32_t)b_o + st * (kStageBytes >> 4);
#pragma unroll
                            for (int dh = 0; dh < 2; ++dh)
#pragma unroll
                                for (int ks = 0; ks < 2; ++ks)
                                    mma_pair(tmem + kColO + 128 * dh, alo + ks * (32 >> 4), (uint32_t)(a_o >> 32),
                                             blo + ks * (2048 >> 4) + dh * (8192 >> 4), (uint32_t)(b_o >> 32), id_o,
                                             (i | j | ks) != 0);
                        }
                        stage_out(M.v_empty, kVStages, next);
                    }
                    if (leader && ok) {
                        commit_pair(M.p_empty[g & 1]);
                        if (kTileBlocks * (i + 1) >= t.nb) commit_pair(M.o_full);
                    }
                }
                ++c;
            }
        }
        // every product has completed, and every arrival at either CTA's barriers, before the accumulators are
        // released (an abandoned one too)
        if (leader) commit_pair(M.done);
        wait(M.done, 0, abort);
    } else if (warp == 2 || warp == kWarpV) {
        // ------------------------------------------------------------------ K (warp 2) and V
        // (codes: warp 2 describes the tiles, up to eight ahead, and pulls their rows into L2)
        const bool is_v = warp == kWarpV;
        const uint32_t stages = is_v ? kVStages : kKStages, ring = is_v ? s_v : s_k;
        uint64_t* const full = is_v ? M.v_full : M.k_full;
        uint64_t* const empty = is_v ? M.v_empty : M.k_empty;
        uint32_t st = 0, st_use = 0, g = 0;
        // (V's copies complete at this CTA's barrier, K's of both CTAs at rank 0's, which expects them all.  Rank 1's warp
        // arrives there as well, also for a tile of one block, of which it copies nothing: else the products would go
        // on without it, and its wait for a stage would come more than a phase too late to tell that it is free.)
        auto load = [&](uint32_t bytes, auto issue) {
            if (!(ok = ok && wait(empty[st], st_use ^ 1u, abort))) return;
            if (lane == 0) {
                const uint32_t bar = smem_addr(&full[st]);
                if (is_v || rank == 0) mbar_arrive_expect_tx(bar, bytes);
                issue(ring + st * kStageBytes, is_v ? bar : at_leader(bar));
                if (!is_v && rank != 0) arrive_at(at_leader(bar));
            }
            if (++st == stages) {
                st = 0;
                ++st_use;
            }
        };
        Task t;
        while (fetch(t)) {
            int rows32 = 0, base32 = -2;  // lane l: the blocks 32 at a time
            for (int i = 0; 4 * i < t.nb && ok; ++i, ++g) {
                if ((i & 7) == 0) {
                    const int k = t.k0 + 4 * i + lane;
                    base32 = -2;
                    rows32 = 0;
                    if (4 * i + lane < t.nb) {
                        const int blk = k < t.fb ? k : k - t.fb + t.wb;
                        const int64_t row = paged::row_of(p.a, t.seq, (uint32_t)blk * kBlock);
                        // (a block without a page: some rows that are there, which no token sees)
                        base32 = row < 0 ? -1 : blk * kBlock;
                        rows32 = row < 0 ? 0 : (int)row;
                        if (row < 0 && !is_v && rank == 0) atomicOr(p.status, kStatusBadIndex);
                    }
                }
                const int src = 4 * (i & 7) + (lane & 3);
                const int row = __shfl_sync(0xffffffffu, rows32, src), base = __shfl_sync(0xffffffffu, base32, src);
                const int nb = min(kTileBlocks, t.nb - 4 * i);
                if (is_v) {
                    for (int j = 0; j < nb && ok; ++j) {
                        const int at = __shfl_sync(0xffffffffu, row, j);
                        load(kStageBytes, [&](uint32_t dst, uint32_t bar) {
                            tma_load_3d(dst, &v_map, 0, at, 4 * (int)rank, bar);
                        });
                    }
                    continue;
                }
                if (kCodes && !(ok = wait(M.info_empty[g % kInfos], (g / kInfos) ^ 1u, abort))) break;
                const bool all = lane < nb && seen(p.window, p.first, base, t.pos0, t.pmax) == 0xffffffffu;
                const bool whole = __all_sync(0xffffffffu, lane >= kTileBlocks || all);
                if (lane < kTileBlocks) M.base[g % kInfos][lane] = lane < nb ? base : -2;
                if (lane == 0) M.whole[g % kInfos] = whole;
                if constexpr (kCodes) {
                    constexpr int kBytes = Widen<kFmt>::kRowBytes;
                    if (lane < kTileBlocks) M.rows[g % kInfos][lane] = row;
                    if (lane < nb && (lane & 1) == (int)rank) {
                        prefetch_l2(p.kv8 + (int64_t)row * kBytes, kBlock * kBytes);
                        prefetch_l2(p.kv_scale + (int64_t)row * (kD / 32), kBlock * (kD / 32));
                    }
                    warp_arrive(M.info_full[g % kInfos], lane);
                    continue;
                }
                warp_arrive(M.info_full[g % kInfos], lane);
                const int own = (nb - (int)rank + 1) / 2;  // this CTA's blocks: rank, rank + 2
                const int g0 = __shfl_sync(0xffffffffu, row, (int)rank) >> 3,
                          g1 = __shfl_sync(0xffffffffu, row, (int)rank + 2) >> 3;
                for (int q = 0; q < 4 && ok; ++q)
                    load((uint32_t)nb * 8192u, [&](uint32_t dst, uint32_t bar) {
                        if (own > 0) tma_load_4d_pair(dst, &k_map, 0, 0, 2 * q, g0, bar);
                        if (own > 1) tma_load_4d_pair(dst + 8192, &k_map, 0, 0, 2 * q, g1, bar);
                    });
            }
        }
        // after a failed wait, the copies under way land before the CTA exits (K's: rank 0 sees those of both, and
        // rank 1 gives its own the time)
        if (!kCodes && !ok && lane == 0 && !is_v && rank != 0)
            for (int i = 0; i < 100; ++i) __nanosleep(1000);
        if (!kCodes && !ok && lane == 0 && (is_v || rank == 0)) {
            const uint32_t n = st_use * stages + st;
            for (uint32_t k = n > stages ? n - stages : 0; k < n; ++k)
                mbar_drain(smem_addr(&full[k % stages]), (k / stages) & 1);
        }
    } else if (!kCodes && warp == warp_q(kFmt)) {
        // ------------------------------------------------------------------ Q
        Task t;
        while (fetch(t))
            if (t.nb) load_q(t.row0);
        drain_q();
    } else if (kCodes && warp >= kWarpWiden && warp < kWarpWiden + 16) {
        // ------------------------------------------------------------------ rows of codes: K (eight warps) and V (eight)
        // Four warps of either take the even stages of the ring, four the odd, whichever task they belong to: a warp has a
        // stage's every use, so that the use before has been let go when it waits for this one's turn.  (By stages of a
        // task, the odd four had none of a task of one block, ran up to four tasks ahead, and took a stage whose last
        // use but one was still to come for free: a wait tells a phase from the next, not from the one after.)
        if constexpr (kCodes) {
            constexpr bool k8 = kFmt == SA_KV_FP8_E4M3;
            const bool is_v = warp >= kWarpWiden + 8;
            const int w = warp & 3, turn = (warp >> 2) & 1;
            uint64_t* const full = is_v ? M.v_full : M.k_full;
            uint64_t* const empty = is_v ? M.v_empty : M.k_empty;
            const uint32_t ring = is_v ? s_v : s_k;
            // K: a stage is 64 rows x 128 d, warps 0 and 1 those of block `rank`, 2 and 3 of rank + 2; V: 32 rows x this
            // CTA's 256 d
            const int lanes = (is_v ? 16 : 8) / (k8 ? 1 : 2), first = is_v ? 8 * w : 16 * w;
            const int group = is_v ? 1024 : 2048, block = is_v ? 4096 : 1024;
            // (the warp's part of a stage, and a lane's place in its rows' codes and scales: see Widen)
            using W = Widen<kFmt>;
            constexpr uint32_t kRing = 4;
            static_assert(kKStages == kRing && kVStages == kRing, "one ring's arithmetic for both");
            const uint32_t own = ring + (is_v ? 1024 : 4096) * w;
            const int hop = is_v ? 4096 : 1024, ul = lane & (lanes - 1), rl = lane / lanes, step = 32 / lanes;
            const uint8_t* const src = p.kv8 + ((first & 31) + rl) * W::kRowBytes + 16 * ul +
                                       (is_v ? W::kRowBytes / 2 * (int)rank : 0);
            const uint8_t* const sc = p.kv_scale + (is_v ? (first + (lane >> 1)) * (kD / 32) + 8 * (int)rank + 4 * (lane & 1)
                                                         : ((first & 31) + lane) * (kD / 32));
            const int sc_by = (is_v ? 8 : 4) * step, sc_at = (is_v ? 8 : 4) * rl + (k8 ? ul >> 1 : ul);
            uint32_t seq = 0, g = 0;  // stages before the task's, tiles before them
            Task t;
            while (fetch(t)) {
                const int nt = (t.nb + kTileBlocks - 1) / kTileBlocks, stages = is_v ? t.nb : 4 * nt;
                const int j_k = (int)rank + 2 * (w >> 1);
                // Stage `put`'s copies go out before `n`, the last but one, is widened, but with a stage to be widened
                // they do not wait for their place: the product that frees it may need that stage (where rows of V
                // are cleared, all of a tile's before its first is used).
                const int n0 = (turn ^ (int)seq) & 1;
                int put = n0;
#pragma unroll 1
                for (int n = n0; n < stages; n += 2) {
                    while (put < stages && put <= n + 2) {
                        const uint32_t gi = (g + (put >> 2)) % kInfos, m = seq + put, e = smem_addr(&empty[m % kRing]);
                        if (put > n && !__all_sync(0xffffffffu, mbar_test_wait(e, ((m / kRing) ^ 1u) & 1u))) break;
                        if ((put & 2) == 0)
                            ok = ok && wait_here(smem_addr(&M.info_full[gi]), (g + (put >> 2)) / kInfos, abort);
                        ok = ok && wait_here(e, (m / kRing) ^ 1u, abort);
                        if (!ok) break;
                        if (is_v || (put & ~3) + j_k < t.nb) {
                            const int64_t row = M.rows[gi][is_v ? put & 3 : j_k];
                            W::copy(own + (m % kRing) * kStageBytes, hop,
                                    src + row * W::kRowBytes + (is_v ? 0 : W::kRowBytes / 4 * (put & 3)), step,
                                    sc + row * (kD / 32) + (is_v ? 0 : 4 * (put & 3)), lane);
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        // (the last of a tile's stages of this warp lets its description go)
                        if ((put & 2) || put + 2 >= stages) warp_arrive(M.info_empty[gi], lane);
                        put += 2;
                    }
                    if (!ok) break;
                    const uint32_t st = (seq + n) % kRing;
                    if (put > n + 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                    if (is_v || (n & ~3) + j_k < t.nb) {
                        W x;
                        x.read(own + st * kStageBytes, hop, sc_at, sc_by, lane);
                        __syncwarp();
                        x.store(ring + st * kStageBytes, first, lanes, group, block, lane);
                    }
                    fence_proxy_async_smem();
                    if (is_v && rank != 0) warp_arrive(full[st], lane);
                    warp_arrive_leader(full[st], lane);
                }
                if (is_v && n0 && (stages & 3) == 1 && ok) {  // (a last tile of one block has no second stage)
                    const uint32_t last = g + nt - 1, gi = last % kInfos;
                    ok = wait_here(smem_addr(&M.info_full[gi]), last / kInfos, abort);
                    warp_arrive(M.info_empty[gi], lane);
                }
                seq += stages;
                g += nt;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp >= 4 && warp < kWarpEpilogue) {
        // ------------------------------------------------------------------ softmax
        // A thread has one row of the CTA's 64 and half of a tile's columns (64: blocks `half` and half + 2); the
        // thread 64 further has the other half, and the two trade their maxima.  Two groups of four warps take the
        // tiles in turn: a tile's chain of steps is longer than its products, and of two tiles' chains only the
        // running maximum is passed from one to the next (through TMEM, which the same lanes of either group read).
        // Each group sums its own tiles' p.  A block's logits are read from TMEM
        // twice, for the maximum and for p, by loops: with both blocks in registers and the loops unrolled, the
        // warps of a SM waited for instructions (4.2 warps at every issue, over a sliding window's prefill).
        const int w = warp & 3, half = w >> 1, row = 32 * (w & 1) + lane, me = 32 * w + lane;
        const uint32_t lane_base = (uint32_t)(32 * w) << 16;
        const uint32_t prow = s_p + half * 8192 + (uint32_t)row * 128;
        const float sc = p.scale_log2;
        const uint32_t grp = (uint32_t)(warp - 4) >> 2;
        uint32_t g = 0, c = 0, v_seq = 0;
        Task t;
        while (fetch(t)) {
            // (a row that is not the task's own has the last one's mask; it is not stored)
            const int pos = t.pos0 + (t.off0 + min(64 * (int)rank + row, t.rows - 1)) / p.h;
            float m = -INFINITY, l = 0.f;  // of this group's tiles: the maximum that l is relative to
            for (int i = 0; kTileBlocks * i < t.nb && ok; ++i, ++g) {
                const uint32_t v_at = v_seq;
                v_seq += min(kTileBlocks, t.nb - kTileBlocks * i);
                if ((g & 1) != grp) continue;
                // (S's buffers go round in threes, from one group to the other: the use before this one had completed when
                // that group passed its maximum on, a tile ago)
                const uint32_t b = g & 1, sb = g % 3, gi = g % kInfos;
                const bool first = i == 0;
                ok = wait(M.info_full[gi], g / kInfos, abort) && wait(M.s_full[sb], g / 3, abort);
                if (!ok) break;
                const bool whole = __shfl_sync(0xffffffffu, M.whole[gi], 0) != 0;
                const uint32_t sa = tmem + lane_base + kColS + 64 * sb;
                tc_fence_after();
                uint32_t v0 = 0xffffffffu, v1 = 0xffffffffu, bad0 = 0, bad1 = 0;  // by block: seen, and to be cleared
                if (!whole) {
                    v0 = seen(p.window, p.first, M.base[gi][half], pos, pos);
                    v1 = seen(p.window, p.first, M.base[gi][half + 2], pos, pos);
                }
                float mt = -INFINITY;
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(sa + 16 * k, r);
                    tmem_wait_ld();
                    if (!whole) {
                        // A logit that is not finite makes the sum of their products with zero a NaN
                        uint64_t z = f2(0.f, 0.f);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            z = ffma2(f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), f2(0.f, 0.f), z);
                        float z0, z1;
                        f2_split(z, z0, z1);
                        if (!(z0 + z1 == 0.f)) {
                            uint32_t odd = 0;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                odd |= (uint32_t)!(fabsf(__uint_as_float(r[j])) < INFINITY) << j;
                            (k & 2 ? bad1 : bad0) |= odd << (16 * (k & 1));
                        }
                        const uint32_t v = (k & 2 ? v1 : v0) >> (16 * (k & 1));
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r[j] = v & (1u << j) ? __float_as_uint(__uint_as_float(r[j]) * sc) : 0xff800000u;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float x0, x1;
                            const uint64_t s2 = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                            f2_split(fmul2(s2, f2(sc, sc)), x0, x1);
                            r[2 * j] = __float_as_uint(x0);
                            r[2 * j + 1] = __float_as_uint(x1);
                        }
                    }
                    float x[5];
#pragma unroll
                    for (int j = 0; j < 5; ++j)
                        x[j] = max3f(__uint_as_float(r[3 * j]), __uint_as_float(r[3 * j + 1]), __uint_as_float(r[3 * j + 2]));
                    mt = max3f(max3f(mt, __uint_as_float(r[15]), x[0]), x[1], max3f(x[2], x[3], x[4]));
                }
                if (bad0 | bad1) {  // in columns that not every row sees (a block that is not there has no V)
                    const int base0 = M.base[gi][half], base1 = M.base[gi][half + 2];
                    bad0 = base0 == -2 ? 0u : bad0 & ~seen(p.window, p.first, base0, t.pos0, t.pmax);
                    bad1 = base1 == -2 ? 0u : bad1 & ~seen(p.window, p.first, base1, t.pos0, t.pmax);
                }
                if constexpr (kCodes) warp_arrive(M.info_empty[gi], lane);
                // (the partner may be a tile behind, and still has to read this warp's last maxima)
                if (!(ok = wait_done(M.mx_empty[grp][w & 1], (g >> 1) ^ 1u, abort))) break;
                M.mx[b][me] = mt;
                warp_arrive(M.pair_bar[grp][w & 1], lane);
                if (!(ok = wait(M.pair_bar[grp][w & 1], g >> 1, abort))) break;
                mt = fmaxf(mt, M.mx[b][me ^ 64]);
                warp_arrive(M.mx_empty[grp][w & 1], lane);
                // P's buffer is free once the P.V two tiles back has completed
                if (!(ok = wait(M.p_empty[b], (g >> 1) ^ 1u, abort))) break;
                // the running maximum before this tile, and after it: raised only where a logit exceeds it by more
                // than the threshold
                if (g > 0 && !(ok = wait(M.m_full[w], g - 1, abort))) break;
                float before = -INFINITY, mn = mt;
                if (!first) {
                    tc_fence_after();
                    before = tmem_ld_x1(tmem + lane_base + kColM + (b ^ 1));
                    mn = mt > before + kRescaleThreshold ? mt : before;
                }
                tmem_st_x1(tmem + lane_base + kColM + b, mn);
                tc_fence_before();
                warp_arrive(M.m_full[w], lane);
                const bool corr = !first && mn != before;
                const float mu = mn == -INFINITY ? 0.f : mn;
                uint64_t acc = f2(0.f, 0.f);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(sa + 16 * k, r);
                    tmem_wait_ld();
                    if (k == 3) {
                        tc_fence_before();
                        warp_arrive_leader(M.s_empty[sb], lane);
                    }
                    const uint32_t v = (k & 2 ? v1 : v0) >> (16 * (k & 1));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t pk[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = 8 * u + 2 * j;
                            float x0, x1;
                            const uint64_t s2 = f2(__uint_as_float(r[at]), __uint_as_float(r[at + 1]));
                            f2_split(ffma2(s2, f2(sc, sc), f2(-mu, -mu)), x0, x1);
                            if (!whole) {
                                x0 = v & (1u << at) ? x0 : -INFINITY;
                                x1 = v & (2u << at) ? x1 : -INFINITY;
                            }
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            acc = fadd2(acc, f2(p0, p1));
                            pk[j] = pack_bf16(p0, p1);
                        }
                        st_shared_v4(prow + b * kPBytes + (((uint32_t)(2 * k + u) ^ ((uint32_t)row & 7)) << 4), pk[0], pk[1],
                                     pk[2], pk[3]);
                    }
                }
                float a0, a1;
                f2_split(acc, a0, a1);
                l = fmaf(mn == m ? 1.f : fast_exp2(m - mn), l, a0 + a1);  // (0 l where nothing was summed yet)
                m = mn;
                if (__any_sync(0xffffffffu, corr || (bad0 | bad1) != 0)) {
                    // O is whole, and V's stages have been left, once the previous tile's P.V has completed
                    // (the other group's barrier: the phase before had completed when that group passed its maximum on)
                    if (g > 0 && !(ok = wait(M.p_empty[b ^ 1], (g - 1) >> 1, abort))) break;
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, corr)) {
                        const float al = corr ? fast_exp2(before - mn) : 1.f;
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
                            uint32_t o[32];
                            const uint32_t ta = tmem + lane_base + kColO + 32 * k;
                            tmem_ld_32x32b_x32(ta, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
                            tmem_st_32x32b_x32(ta, o);
                        }
                        tmem_wait_st();
                    }
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {  // rows of V to clear
                        uint32_t rows = __reduce_or_sync(0xffffffffu, k ? bad1 : bad0);
                        if (!rows) continue;
                        const uint32_t vs = v_at + half + 2 * k;
                        if (!(ok = wait(M.v_full[vs % kVStages], vs / kVStages, abort))) break;
                        // (4 pieces of 128 bytes: a lane 16 of them.  The logit may be a bad q's, and other rows of the
                        // task see this one of V: only what is not finite itself is cleared, 0 times the rest is 0)
                        const uint32_t at = s_v + (vs % kVStages) * kStageBytes + (lane >> 3) * 4096 + (lane & 7) * 16;
                        for (; rows; rows &= rows - 1) {
                            const uint32_t to = at + (__ffs(rows) - 1) * 128;
                            if (any_not_finite(to)) st_shared_v4(to, 0u, 0u, 0u, 0u);
                        }
                    }
                    if (!ok) break;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive_leader(M.p_full[b], lane);
            }
            if (!ok) break;
            if (!(ok = wait(M.stats_empty, c ^ 1u, abort))) break;
            tmem_st_x2(tmem + lane_base + kColT + 2 * grp, m, l);
            tc_fence_before();
            warp_arrive(M.stats_full, lane);
            ++c;
        }
    } else {
        // ------------------------------------------------------------------ epilogue
        // A thread has one row and 128 of its d (256, where there is one group of four warps): of the half that its
        // lane holds, every second 32, so that the groups share the turned ones (all of them in one group's half
        // made it 40 us of a prompt's 175: O is free for the next task when the last warp has read it).
        const int w = warp & 3, grp = (warp - kWarpEpilogue) >> 2, half = w >> 1, row = 32 * (w & 1) + lane;
        const uint32_t lane_base = (uint32_t)(32 * w) << 16;
        const bool split = p.n_splits > 1;
        uint32_t c = 0, c_o = 0;
        Task t;
        while (fetch(t)) {
            const int r = 64 * (int)rank + row;
            const bool mine = r < t.rows;
            const int tok = (t.off0 + r) / p.h, head = t.off0 + r - tok * p.h;
            const float2* turn = nullptr;
            if constexpr (kRope) {
                int64_t pos = t.pos0 + min(tok, t.pmax - t.pos0);
                if (pos >= p.npos) {
                    if (mine && half + grp == 0) atomicOr(p.status, kStatusBadIndex);
                    pos = p.npos - 1;
                }
                turn = reinterpret_cast<const float2*>(p.rope) + max(pos, (int64_t)0) * (p.rope_dim >> 1);
                // (on its way while the products run: one token's epilogue would wait a microsecond for it)
                if (half)
                    for (int x = 0; x < p.rope_dim >> 1; x += 16)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(turn + x));
            }
            const float sink = __ldg(p.sink + head);
            ok = wait(M.stats_full, c, abort);
            if (ok && t.nb) ok = wait(M.o_full, c_o, abort);
            if (!ok) break;
            tc_fence_after();
            // the two groups' sums, relative to the larger maximum (the last tile's), then the two halves'
            float m0, l0, m1, l1;
            tmem_ld_x4(tmem + lane_base + kColT, m0, l0, m1, l1);
            tc_fence_before();
            warp_arrive(M.stats_empty, lane);
            const float top = fmaxf(m0, m1), mu = top == -INFINITY ? 0.f : top;
            const float mine_l = l0 * fast_exp2(m0 - mu) + l1 * fast_exp2(m1 - mu);
            if (!(ok = wait(M.sum_empty[w & 1], c ^ 1u, abort))) break;  // (the last task's have been read)
            M.sum[32 * w + lane] = mine_l;  // (the same from either group)
            warp_arrive(M.sum_full[w & 1], lane);
            if (!(ok = wait(M.sum_full[w & 1], c, abort))) break;
            const float l = mine_l + M.sum[(32 * w + lane) ^ 64];
            warp_arrive(M.sum_empty[w & 1], lane);
            ++c;
            const int64_t flat = (int64_t)t.row0 + r;
            const int64_t part = ((int64_t)(t.tok0 + tok) * p.n_splits + t.split) * p.h + head;
            float inv = 0.f;
            if (!split) {
                if (l > 0.f) inv = 1.f / (l + fast_exp2(sink * kLog2e - mu));
                if (p.lse && mine && half + grp == 0) p.lse[flat] = log_sum_exp(l, mu, sink);
            } else if (mine && half + grp == 0) {
                *reinterpret_cast<float2*>(p.part_ml + 2 * part) = make_float2(mu, l);
            }
            if (t.nb == 0 && split) continue;  // (its sum is 0: O is not looked at)
            // Lanes 2 i and 2 i + 1 trade 32-byte pieces of their rows, so that each store writes 64 bytes of 16 rows (32
            // of 32, a lane's own, take twice the time: a store's time is its pieces')
            const bool odd = lane & 1;
            const int at_row = mine ? (split ? (int)part : (int)flat) : -1;
            const int even_row = __shfl_sync(0xffffffffu, at_row, lane & 30);
            const int odd_row = __shfl_sync(0xffffffffu, at_row, lane | 1);
#pragma unroll 1
            for (int k = grp; k < 8; k += kEpilogues) {  // 32 d at a time
                const int d0 = 256 * half + 32 * k;
                uint32_t o[32];
                __syncwarp();
                if (t.nb) {
                    tmem_ld_32x32b_x32(tmem + lane_base + kColO + 32 * k, o);
                    tmem_wait_ld();
                    if (k + kEpilogues >= 8) {
                        tc_fence_before();
                        warp_arrive_leader(M.o_empty, lane);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0u;
                }
                if constexpr (kRope) {
                    // (a + i b)(c - i s), on the f32 sums (partials too: the merge is linear)
                    const int e0 = d0 - (kD - p.rope_dim);
                    if (e0 + 32 > 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int e = e0 + 2 * j;
                            if (e < 0) continue;
                            const float2 cs = __ldg(turn + (e >> 1));
                            const float a = __uint_as_float(o[2 * j]), b = __uint_as_float(o[2 * j + 1]);
                            o[2 * j] = __float_as_uint(fmaf(a, cs.x, b * cs.y));
                            o[2 * j + 1] = __float_as_uint(fmaf(b, cs.x, -a * cs.y));
                        }
                    }
                }
                // two pieces, of even and odd lanes, into x[0..7] (the even row's) and x[8..15] (the odd row's)
                auto trade_and_store = [&](uint32_t (&x)[16], char* base, int row_bytes, int at) {
                    uint32_t e[8], f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? x[j] : x[8 + j], 1);
                        e[j] = odd ? got : x[j];
                        f[j] = odd ? x[8 + j] : got;
                    }
                    if (even_row >= 0) store32(base + (int64_t)even_row * row_bytes + at + 32 * odd, e);
                    if (odd_row >= 0) store32(base + (int64_t)odd_row * row_bytes + at + 32 * odd, f);
                };
                uint32_t x[16];
                if (split) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = o[16 * q + j];
                        trade_and_store(x, reinterpret_cast<char*>(p.part_o), 4 * kD, 4 * (d0 + 16 * q));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        x[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    trade_and_store(x, reinterpret_cast<char*>(p.o), 2 * kD, 2 * d0);
                }
            }
            if (t.nb) ++c_o;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && M.abort) atomicOr(p.status, kStatusTimeout);
    __syncwarp();
    cluster_barrier();  // nobody reads this CTA's shared memory, or arrives at its barriers, any more
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// How many parts a task's blocks are cut into: more than one only where the tasks (about: a token's tile or the
// rows' tiles, whichever are more) leave pairs of SMs without work, and only of four tiles and more: a part a tile.  (One
// token of 64 heads, whole / in parts of two tiles / of one, the merge's launch among them: window 256, 3 tiles, 12.8 / - /
// 13.1 us; 384, 4 tiles, 14.6 / 14.4 / 13.2; 1024, 9 tiles, 21.7 / 15.7 / 13.9.  30 such tokens of window 4096: 61 whole, 44
// in two parts.)
int window_splits(int64_t n, int64_t b, int h, int64_t window, int64_t first, int sms) {
    const int64_t tiles = std::max<int64_t>(std::max<int64_t>((n * h + kM - 1) / kM, std::min(b, n)), 1);
    const int64_t keys = first + kBlock + window + kM / h + 2 * kBlock;
    const int64_t key_tiles = (keys + kBlock * kTileBlocks - 1) / (kBlock * kTileBlocks);
    const int64_t most = key_tiles > 3 ? key_tiles : 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(sms / 2 / tiles, most), 64));
}

}  // namespace

// (Other pages, and other d, go by index table through the families that gather by row: pages of 16 rows take 509 us where
// pages of 64 take 258-272 (256 tokens of 128 heads, window 4096), and 197 where they take 139-143 (a prompt of 4095).)
bool window_tc_supports(int d, int kv_format, int page) {
    (void)kv_format;
    return d == kD && page % kBlock == 0;
}

size_t window_tc_scratch_bytes(int64_t n, int64_t b, int h, int64_t window, int64_t first) {
    const size_t s = window_splits(n, b, h, window, first, kMaxSmCount);
    return s == 1 ? 0 : align_up((size_t)n * s * h * 2 * sizeof(float), 256) + (size_t)n * s * h * kD * sizeof(float);
}

size_t window_tc_scratch_bound(int64_t n, int h, int64_t window, int64_t first) {
    // (of one sequence, which has the fewest tiles: as many parts only from as few tiles, and of those the most tokens)
    size_t most = 0;
    for (int s = 2; s <= 64 && 2 * s <= kMaxSmCount; ++s)
        most = std::max(most, window_tc_scratch_bytes(std::min<int64_t>(n, kMaxSmCount / 2 / s * kM / h), 1, h, window, first));
    return most;
}

cudaError_t window_tc_launch(const WindowCall& c) {
    const int sms = device_sm_count();
    // Q: 64 rows x two blocks of 64 d, block by block.  V: 32 rows x four blocks of 64 d, block by block.  K: 32
    // rows x two blocks of 64 d, eight rows of one block behind those of the other (so that a stage's 64 rows,
    // two boxes, are 2 KB a step of eight in either block).
    CUtensorMap q_map, k_map, v_map;
    const int64_t rows = c.a.n_pages * c.a.page;
    const bool codes = c.kv_format != SA_KV_BF16;
    if (!encode_blocks_map(q_map, c.q, kD, c.n * c.h, 64, 2)) return cudaErrorInvalidValue;
    if (codes) {
        k_map = v_map = q_map;  // (not looked at)
    } else if (!encode_blocks_map(v_map, c.kv, kD, rows, kBlock, 4) || !encode_groups_map(k_map, c.kv, kD, rows, kBlock, 2))
        return cudaErrorInvalidValue;
    Params p = {};
    p.a = c.a;
    p.kv8 = codes ? reinterpret_cast<const uint8_t*>(c.kv) : nullptr;
    p.kv_scale = c.kv_scale;
    p.sink = c.sink;
    p.o = reinterpret_cast<__nv_bfloat16*>(c.o);
    p.lse = c.lse;
    p.status = c.status;
    p.rope = c.rope;
    p.npos = c.npos;
    p.rope_dim = c.rope_dim;
    p.scale_log2 = c.softmax_scale * kLog2e;
    p.n = (int)c.n;
    p.h = c.h;
    p.window = (int)c.window;
    p.first = (int)c.first;
    // (no more parts than the table's positions make)
    const Reach seen = reach_of(c.window, c.first, c.a.max_pages, c.a.page);
    p.n_splits = window_splits(c.n, c.a.b, c.h, seen.window, seen.first, sms);
    const int64_t units = (c.n * c.h / kM + c.a.b) * p.n_splits;
    if (units > INT32_MAX - kMaxSmCount) return cudaErrorInvalidConfiguration;  // (the kernel counts units in 32 bits)
    p.units = (int)units;
    if (p.n_splits > 1) {
        p.part_ml = reinterpret_cast<float*>(c.scratch);
        p.part_o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(c.scratch) +
                                            align_up((size_t)c.n * p.n_splits * c.h * 2 * sizeof(float), 256));
    }
    using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Params);
    static const Kernel kernels[3][2] = {
        {window_tc_kernel<SA_KV_BF16, false>, window_tc_kernel<SA_KV_BF16, true>},
        {window_tc_kernel<SA_KV_FP8_E4M3, false>, window_tc_kernel<SA_KV_FP8_E4M3, true>},
        {window_tc_kernel<SA_KV_FP4_E2M1, false>, window_tc_kernel<SA_KV_FP4_E2M1, true>}};
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        for (auto& by_rope : kernels)
            for (auto fn : by_rope) {
                e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
                if (e != cudaSuccess) return e;
            }
        if (dev < 64) configured[dev] = true;
    }
    const Kernel kernel = kernels[c.kv_format][c.rope ? 1 : 0];
    const int threads = 32 * (codes ? warps_of(SA_KV_FP8_E4M3) : warps_of(SA_KV_BF16));
    int64_t pairs = sms / 2;
    if (pairs > units) pairs = units;
    e = launch_pdl(kernel, dim3((unsigned)(2 * pairs)), dim3(threads), kSmem, c.stream, q_map, k_map, v_map, p);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    return attn_combine_launch(p.part_ml, p.part_o, c.sink, c.o, c.lse, c.n, c.h, kD, p.n_splits,
                               c.a.q_start + c.a.b, c.stream);
}

}  // namespace sa
