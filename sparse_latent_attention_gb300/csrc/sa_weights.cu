// The attention weight each cache row received, and its C ABI entry (include/cache/sa_evict.h):
//   w(token, entry) = sum over heads of e^(scale q.k - lse),  acc[row of the entry] += round(w 2^32)
//
// Formulation.  With the softmax's log-sum-exp given, a weight needs no second pass and no maximum: one
// product S^T[128 entries x heads] = KV_tile[128 x d] . Q^T and a sum of exponentials along the heads.
// The rows of a tile are the product's M dimension, so an accumulator lane is an entry: a thread reads its
// entry's logits from TMEM, adds up the heads in registers and issues one integer addition to the row's
// accumulator.  Entries are independent of one another: empty ones are not copied (their lane holds
// whatever was there) and not added, and (token, tile) units may run anywhere, so the units are cut evenly
// over the SMs whatever the batch.  The accumulators are integers, so the order of the additions does
// not matter.
//
// The product's d is cut into two ranges with an accumulator each, added up in the epilogue in f32.  One
// accumulator over all of d = 512, cut by the tensor core after every 16 products, came to a relative error of
// 1.9e-6 in the weights of bf16 rows (0.7e-6 to 1.04e-6 with two).  Up to 64 heads each range has an issuing
// warp too: a stage's products take about as long as the wait and the commits around them, which two warps pass
// behind each other's products (214 us against 257 for the prefill below).
//
// What bounds it: that prefill's 4096 queries have 2.09 M entries (80 % of their columns) and copy 2.1 GB of rows
// out of L2 in 214 us, 10 TB/s or 32 bytes a cycle and SM (the products of all columns alone would take 90 us, at
// the measured bf16 rate; units without an entry are computed like the others); the long decode, 144 MB of
// codes and scales once (38 us at the measured copy rate), is held up by the widening.
//
// Roles (persistent CTAs, 19 or 27 warps; every wait is bounded, as in the attention kernel).  A stage is
// 128 d of a tile [two 64-d blocks of 128 rows x 128 bytes].  What one warp does for a stage or a tile is a chain of
// short latencies (a copy phase ~270 cycles, a hand-over ~250, a tile's epilogue ~3500), longer than the
// product itself takes, so two groups of warps take turns at the stages and two at the tiles:
//   warp 0 (and the last, up to 64 heads)  MMA issue (one elected lane): per stage eight MMAs of
//                128 x kN x 16
//   warp 1       Q by TMA (128-byte swizzle), 128 d at a time: that part of the next token's Q is loaded as
//                soon as the last tile's product has passed it
//   warps 2-9    epilogue: exponentials, sum over heads, accumulation; four warps a tile
//   warps 10-    gather, four or eight warps a stage: bf16 rows with 16-byte cp.async; rows of codes
//                are loaded a turn ahead into registers and widened into the stage (exact: see
//                sa_fp8.cuh, sa_fp4.cuh)

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache/sa_evict.h"
#include "sa_fp4.cuh"
#include "sa_internal.cuh"
#include "sa_tc.cuh"

namespace sa {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnits = 4294967296.f;  // 2^32 units of the accumulator to a weight of 1

constexpr int kTile = 128;              // entries per tile (M)
constexpr int kWarpEpilogue = 2, kWarpGather = 10;
constexpr int kMaxSteps = 4;            // 128-d stages of a row: d <= 512
constexpr uint32_t kBlockBytes = kTile * 128;        // 64 d of a tile
constexpr uint32_t kStageBytes = 2 * kBlockBytes;

// By the kv format: the warps of a gather group, and the rows of a stage that each fills.  Copying takes few
// instructions, and fewer warps leave the others quicker (a prefill's 4096 queries x 640 bf16 rows, 64 heads:
// 214 us with four, 249 with eight); widening takes many (a long decode's 256 x 2176 4-bit rows, 128 heads:
// 108 us with eight, 120 with four).
template <int kFmt>
struct Gather {
    static constexpr int kWarps = kFmt == SA_KV_BF16 ? 4 : 8;
    static constexpr int kRows = kTile / kWarps;
    static constexpr int kWarpMma2 = kWarpGather + 2 * kWarps;  // the second MMA issuer
    static constexpr int kThreads = 32 * (kWarpMma2 + 1);
};

// By the heads a product covers (kN = 64 or 128): the stages that fit beside Q.
template <int kN>
struct Shape {
    static constexpr uint32_t kQBlockBytes = kN * 128;  // 64 d of Q
    static constexpr uint32_t kQBytes = 2 * kMaxSteps * kQBlockBytes;
    static constexpr int kStages = kN == 64 ? 5 : 3;
    // Two issuing warps release the stages out of order, one range's later stage before the other's earlier
    // one.  A gather warp that waits for stage n (n - kStages released) must not do so while the use before
    // (n - 2 kStages) is still in progress: the barrier's parity would answer for the wrong use.  It has seen
    // n - 9 and n - 7 released when it comes to n with five stages, one of which the warp that issued n - 10
    // released after it.  With three stages it has only seen n - 5 and n - 7, both of which can precede
    // n - 6: those have one issuing warp.
    static constexpr bool kTwoIssuers = kStages == 5;
    static constexpr uint32_t kOffQ = kStages * kStageBytes;
    static constexpr uint32_t kOffMisc = kOffQ + kQBytes;
};

struct Misc {
    uint64_t kv_full[5], kv_empty[5];
    uint64_t q_full[kMaxSteps], q_empty[kMaxSteps];
    uint64_t s_full[2], s_empty[2];  // per set of accumulators (TMEM)
    uint64_t lse_bar[2], done;
    uint32_t tmem_base;
    int abort;
    alignas(16) float nlse[2][128];  // -lse log2(e) of a token's heads, a table per epilogue group
};

template <int kN>
constexpr uint32_t smem_bytes() {
    return Shape<kN>::kOffMisc + (uint32_t)sizeof(Misc) + 1024u;  // + alignment slack
}
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory budget");

struct Params {
    const uint8_t* q;   // for the L2 prefetch; q_row bytes a head
    int64_t q_row;
    const uint8_t* kv;
    const uint8_t* kv_scale;
    const float* lse;
    const int32_t* idx;
    unsigned long long* acc;
    uint32_t* status;
    float scale_log2;
    int64_t s_len;
    int h, steps;   // 128-d stages of a row; the last is half of one when d is not a multiple of 128
    bool half;
    int64_t rows;
    int topk, n_tiles;
    int64_t n_units;  // (token, tile)
};

// A CTA's units: an even share of all, in order, so that a token's tiles mostly meet the same Q.
struct Range {
    int64_t begin, end;
};
__device__ __forceinline__ Range unit_range(const Params& p) {
    const int64_t g = gridDim.x, i = blockIdx.x, base = p.n_units / g, rem = p.n_units % g;
    Range r;
    r.begin = i * base + (i < rem ? i : rem);
    r.end = r.begin + base + (i < rem ? 1 : 0);
    return r;
}

// Walks the units in order.
struct Unit {
    int64_t token, seq, pos;
    int tile;
    __device__ __forceinline__ Unit(const Params& p, int64_t u) {
        token = u / p.n_tiles;
        tile = (int)(u - token * p.n_tiles);
        seq = token / p.s_len;
        pos = token - seq * p.s_len;
    }
    __device__ __forceinline__ void step(const Params& p) {
        if (++tile == p.n_tiles) {
            tile = 0;
            ++token;
            if (++pos == p.s_len) {
                pos = 0;
                ++seq;
            }
        }
    }
};

// The entry in row r of a unit's tile as it stands in idx (-1 past the columns).  It is loaded a tile
// ahead, so it must not be looked at before it is needed: valid() then makes it a cache row or -1.
__device__ __forceinline__ int entry_of(const Params& p, const Unit& u, int r) {
    const int col = u.tile * kTile + r;
    return col < p.topk ? __ldg(p.idx + u.token * (int64_t)p.topk + col) : -1;
}
__device__ __forceinline__ int valid(const Params& p, int j, bool& any_bad) {
    asm volatile("" : "+r"(j));  // (no test of it moves up to the load)
    const bool bad = j < -1 || j >= p.rows;
    any_bad |= bad;
    return bad ? -1 : j;
}

// A gather group's place in the sequence of stages: it takes every other one.
struct Cursor {
    Unit u;
    int64_t i;  // the unit, from the CTA's first
    int c;      // the stage in it
    __device__ __forceinline__ Cursor(const Params& p, int64_t begin, int group) : u(p, begin), i(0), c(0) {
        if (group) advance(p, 1);
    }
    __device__ __forceinline__ void advance(const Params& p, int by) {
        c += by;
        while (c >= p.steps) {
            c -= p.steps;
            ++i;
            u.step(p);
        }
    }
    // the next unit that the group has a stage of (with one stage a unit, every other unit)
    __device__ __forceinline__ Unit next_unit(const Params& p, int64_t& at) const {
        Unit n = u;
        n.step(p);
        if (p.steps == 1) n.step(p);
        at = i + (p.steps == 1 ? 2 : 1);
        return n;
    }
};

// The 32 codes of a scale's block, on their way from memory to a stage.
template <int kFmt>
struct Codes {
    uint32_t w[kFmt == SA_KV_FP4_E2M1 ? 4 : 8];
};

// A bf16 gather warp's copies of a stage: 16 bytes of each of a lane's kPer rows from kOff bytes into it.
// Row i's place is 1024 bytes (eight rows) on from row i - 4's.
template <int kOff, int kPer, int kI = 0>
__device__ __forceinline__ void copy_rows(const uint32_t (&dst)[4], const uint8_t* const (&src)[kPer],
                                          uint32_t there) {
    if constexpr (kI < kPer) {
        if (there >> kI & 1) cp_async16_at<(kI / 4) * 1024, kOff>(dst[kI % 4], src[kI]);
        copy_rows<kOff, kPer, kI + 1>(dst, src, there);
    }
}

template <int kFmt, int kN>
__global__ void __launch_bounds__(Gather<kFmt>::kThreads, 1)
    row_weights_kernel(const __grid_constant__ CUtensorMap q_map, Params p) {
    using Sh = Shape<kN>;
    constexpr int kStages = Sh::kStages, kGroupWarps = Gather<kFmt>::kWarps, kWarpRows = Gather<kFmt>::kRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    Misc& M = *reinterpret_cast<Misc*>(smem + Sh::kOffMisc);
    const uint32_t s_kv = smem_addr(smem), s_q = smem_addr(smem + Sh::kOffQ);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &M.abort;
    pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&M.kv_full[i]), kGroupWarps);
            mbar_init(smem_addr(&M.kv_empty[i]), 1);
        }
        for (int i = 0; i < kMaxSteps; ++i) {
            mbar_init(smem_addr(&M.q_full[i]), 1);
            mbar_init(smem_addr(&M.q_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&M.s_full[i]), Sh::kTwoIssuers && p.steps > 2 ? 2 : 1);
            mbar_init(smem_addr(&M.s_empty[i]), 4);
            mbar_init(smem_addr(&M.lse_bar[i]), 128);
        }
        mbar_init(smem_addr(&M.done), 2);
        M.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tmem_alloc(smem_addr(&M.tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 1 && lane == 0) tma_prefetch_desc(&q_map);
    pdl_wait();  // the set-up above touches no global memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M.tmem_base;
    const Range range = unit_range(p);

    if (warp == 0 || warp == Gather<kFmt>::kWarpMma2) {
        // ------------------------------------------------------------------ MMA issue
        // A tile's stages 0 and 1 go into the first accumulator, 2 and 3 into the second.  With two issuers
        // warp 0 takes the former and the other warp the latter.
        constexpr uint32_t id = idesc_bf16_f32(kTile, kN, false, false);
        const uint64_t a0 = smem_desc_sw128(s_kv, 16, 1024);  // tile rows, K-major
        const uint64_t b0 = smem_desc_sw128(s_q, 16, 1024);   // heads, K-major
        const uint32_t ahi = (uint32_t)(a0 >> 32), bhi = (uint32_t)(b0 >> 32);
        const int c0 = warp == 0 ? 0 : Sh::kTwoIssuers ? 2 : p.steps;
        const int c1 = Sh::kTwoIssuers ? min(p.steps, c0 + 2) : p.steps;
        bool ok = true;
        int st = c0 % kStages;
        uint32_t ph = 0, k = 0, qph = 0;
        auto skip = [&](int n) {  // the stages that the other warp issues
            st += n;
            if (st >= kStages) {
                st -= kStages;
                ph ^= 1;
            }
        };
        Unit u(p, range.begin);
        for (int64_t i = range.begin; i < range.end && ok && c0 < c1; ++i, ++k) {
            const bool first = i == range.begin || u.tile == 0;
            const bool last = i == range.end - 1 || u.tile == p.n_tiles - 1;
            const uint32_t b = k & 1;
            if (!(ok = warp_wait(smem_addr(&M.s_empty[b]), ((k >> 1) & 1) ^ 1, abort))) break;
            for (int c = c0; c < c1; ++c) {
                ok = (!first || warp_wait(smem_addr(&M.q_full[c]), qph, abort)) &&
                     warp_wait(smem_addr(&M.kv_full[st]), ph, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t col = tmem + 256 * b + kN * (c >> 1);
                uint32_t alo = (uint32_t)a0 + st * (kStageBytes >> 4);
                uint32_t blo = (uint32_t)b0 + 2 * c * (Sh::kQBlockBytes >> 4);
                const int blocks = c == p.steps - 1 && p.half ? 1 : 2;
#pragma unroll
                for (int k64 = 0; k64 < 2; ++k64) {
                    if (k64 == blocks) break;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_lohi_elect(col, alo + 2 * q, ahi, blo + 2 * q, bhi, id,
                                       (uint32_t)(c & 1) | (uint32_t)k64 | (uint32_t)q);
                    alo += kBlockBytes >> 4;
                    blo += Sh::kQBlockBytes >> 4;
                }
                mma_commit_elect(smem_addr(&M.kv_empty[st]));
                if (last) mma_commit_elect(smem_addr(&M.q_empty[c]));
                skip(1);
            }
            if (!ok) break;
            mma_commit_elect(smem_addr(&M.s_full[b]));
            if (last) qph ^= 1;
            skip(p.steps - (c1 - c0));
            u.step(p);
        }
        // let every issued MMA finish before the accumulators are released
        mma_commit_elect(smem_addr(&M.done));
        warp_wait(smem_addr(&M.done), 0, abort);
    } else if (warp == 1) {
        // ------------------------------------------------------------------ Q loads (TMA)
        if (lane == 0) {
            bool ok = true;
            uint32_t n = 0;  // tokens begun
            int loaded = 0;  // parts of the last of them that were asked for
            Unit u(p, range.begin);
            const int64_t last_token = (range.end - 1) / p.n_tiles;
            for (int64_t token = u.token; token <= last_token && ok; ++token) {
                ++n;
                loaded = 0;
                for (int c = 0; c < p.steps; ++c) {
                    if (!(ok = mbar_wait(smem_addr(&M.q_empty[c]), n & 1, abort))) break;
                    const int blocks = c == p.steps - 1 && p.half ? 1 : 2;
                    const uint32_t bar = smem_addr(&M.q_full[c]);
                    mbar_arrive_expect_tx(bar, blocks * Sh::kQBlockBytes);
                    for (int k64 = 0; k64 < blocks; ++k64)
                        tma_load_2d(s_q + (2 * c + k64) * Sh::kQBlockBytes, &q_map, 128 * c + 64 * k64,
                                    (int32_t)(token * p.h), bar);
                    ++loaded;
                }
                // the next token's heads into L2 meanwhile
                if (token < last_token)
                    for (int i = 0; i < p.h; i += 8)
                        prefetch_l2(p.q + ((token + 1) * p.h + i) * p.q_row,
                                    (uint32_t)(min(8, p.h - i) * p.q_row));
            }
            // after a failed wait, let the loads under way land before the CTA exits
            if (*abort)
                for (int c = 0; c < p.steps; ++c) {
                    const uint32_t uses = n - (c < loaded ? 0u : 1u);  // times part c was asked for
                    if (uses > 0) mbar_drain(smem_addr(&M.q_full[c]), (uses - 1) & 1);
                }
        }
        __syncwarp();
    } else if (warp < kWarpGather) {
        // ------------------------------------------------------------------ epilogue
        const int group = (warp - kWarpEpilogue) >> 2;  // takes the CTA's units group, group + 2, ...
        const int q4 = warp & 3;  // the TMEM lanes this warp may read: 32 q4 .. 32 q4 + 31
        const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
        const int et = 32 * q4 + lane;  // 0 .. 127: its entry of the tile, and the head whose lse it brings
        const bool two = p.steps > 2;  // both accumulators are used
        const uint32_t s_at = tmem + lane_base + 256 * group;
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        float* table = M.nlse[group];
        bool ok = true, bad = false;
        uint32_t n = 0, lse_phase = 0;
        int64_t token = -1;  // whose lse the table holds
        const int64_t count = range.end - range.begin;
        Unit u(p, range.begin), un = u;  // un: the group's next unit, whose entry is loaded meanwhile
        if (group) un.step(p);
        int jn = group < count ? entry_of(p, un, et) : -1;
        float ln = group < count && et < p.h ? __ldg(p.lse + un.token * p.h + et) : 0.f;
        for (int64_t i = group; i < count && ok; i += 2, ++n) {
            u = un;
            const int j = valid(p, jn, bad);
            if (u.token != token) {
                token = u.token;
                // every warp of the group has read the old table; the new one is there
                if (!(ok = wg_sync(smem_addr(&M.lse_bar[group]), lse_phase, abort))) break;
                table[et] = -ln * kLog2e;
                if (!(ok = wg_sync(smem_addr(&M.lse_bar[group]), lse_phase, abort))) break;
            }
            un.step(p);
            un.step(p);
            if (i + 2 < count) {
                jn = entry_of(p, un, et);
                if (un.token != token && et < p.h) ln = __ldg(p.lse + un.token * p.h + et);
            }
            if (!(ok = warp_wait(smem_addr(&M.s_full[group]), n & 1, abort))) break;
            tc_fence_after();
            uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
            // 16 heads at a time: their partial products from both accumulators, added up
#pragma unroll 1
            for (int q = 0; q < kN / 16; ++q) {
                uint32_t r[16], v[16];
                tmem_ld_32x32b_x16(s_at + 16 * q, r);
                if (two) tmem_ld_32x32b_x16(s_at + kN + 16 * q, v);
                tmem_wait_ld();
                if (q == kN / 16 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&M.s_empty[group]));
                }
                const int heads = p.h - 16 * q;  // of these 16
                if (heads <= 0) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 n4 = *reinterpret_cast<const float4*>(&table[16 * q + 4 * c]);
                    uint64_t v0 = f2(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1]));
                    uint64_t v1 = f2(__uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3]));
                    if (two) {
                        v0 = fadd2(v0, f2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])));
                        v1 = fadd2(v1, f2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])));
                    }
                    float x[4], e[4];
                    f2_split(ffma2(v0, sc2, f2(n4.x, n4.y)), x[0], x[1]);
                    f2_split(ffma2(v1, sc2, f2(n4.z, n4.w)), x[2], x[3]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) e[y] = fast_exp2(x[y]);
                    if (heads < 16) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (4 * c + y >= heads) e[y] = 0.f;
                    }
                    sum[0] = fadd2(sum[0], f2(e[0], e[1]));
                    sum[1] = fadd2(sum[1], f2(e[2], e[3]));
                }
            }
            float w0, w1;
            f2_split(fadd2(sum[0], sum[1]), w0, w1);
            const float w = fminf(fmaxf(w0 + w1, 0.f), (float)p.h);  // (a NaN becomes 0)
            if (j >= 0) atomicAdd(p.acc + u.seq * p.rows + j, __float2ull_rn(w * kUnits));
        }
    } else if constexpr (kFmt == SA_KV_BF16) {
        // ------------------------------------------------------------------ gather, bf16
        // Lane l copies 16-byte unit l % 16 (of a stage's 256 bytes) of rows l / 16, l / 16 + 2, ... of the
        // warp's 32: two rows' 256 bytes an instruction.
        constexpr int kPer = kWarpRows / 2;
        const int group = (warp - kWarpGather) / kGroupWarps, unit = lane & 15;
        const int r0 = kWarpRows * ((warp - kWarpGather) % kGroupWarps) + (lane >> 4);  // row r0 + 2 i
        uint32_t d[4];  // where the unit of rows r0 + 2 i, i % 4, goes, from row r0 + 2 i (i % 4 = 0) on
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = s_kv + (uint32_t)(unit >> 3) * kBlockBytes + (r0 + 2 * i) * 128 +
                   ((uint32_t)((unit ^ (r0 + 2 * i)) & 7) << 4);
        const uint32_t row_bytes = (uint32_t)p.steps * 256 - (p.half ? 128 : 0);
        const int64_t count = range.end - range.begin;
        bool ok = true, any_bad = false;
        int st = group, under_way = -1;  // the stage to fill; the one filled but not handed over
        uint32_t ph = 1;
        auto hand_over = [&] {
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&M.kv_full[under_way]));
        };
        Cursor cur(p, range.begin, group);
        const uint8_t* src[kPer];
        uint32_t there = 0;  // bit i: row r0 + 2 i has an entry
        // each lane brings the entry of one of the warp's rows
        const int my_row = kWarpRows * ((warp - kWarpGather) % kGroupWarps) + lane % kWarpRows;
        int jn = cur.i < count ? entry_of(p, cur.u, my_row) : -1;
        int64_t unit_at = -1;  // the unit that src points into
        while (cur.i < count) {
            if (cur.i != unit_at) {
                unit_at = cur.i;
                const uint8_t* base = p.kv + cur.u.seq * p.rows * row_bytes + unit * 16;
                const int j = valid(p, jn, any_bad);
                there = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int ji = __shfl_sync(0xFFFFFFFFu, j, (lane >> 4) + 2 * i);
                    there |= ji >= 0 ? 1u << i : 0u;
                    src[i] = base + (uint64_t)(uint32_t)ji * row_bytes;
                }
                int64_t at;
                const Unit nu = cur.next_unit(p, at);
                if (at < count) jn = entry_of(p, nu, my_row);
            }
            // the stage of the group's last turn is handed over before the wait for a free one, so that
            // the product has work while this warp waits for it
            if (under_way >= 0) hand_over();
            under_way = -1;
            if (!(ok = warp_wait(smem_addr(&M.kv_empty[st]), ph, abort))) break;
            if (!(cur.c == p.steps - 1 && p.half && unit >= 8)) {
                const uint32_t at = st * kStageBytes;
                const uint32_t dd[4] = {d[0] + at, d[1] + at, d[2] + at, d[3] + at};
                switch (cur.c) {
                    case 0: copy_rows<0, kPer>(dd, src, there); break;
                    case 1: copy_rows<256, kPer>(dd, src, there); break;
                    case 2: copy_rows<512, kPer>(dd, src, there); break;
                    default: copy_rows<768, kPer>(dd, src, there); break;
                }
            }
            cp_async_commit();
            under_way = st;
            if ((st += 2) >= kStages) {
                st -= kStages;
                ph ^= 1;
            }
            cur.advance(p, 2);
        }
        if (ok && under_way >= 0) hand_over();
        cp_async_wait<0>();
        if (any_bad) atomicOr(p.status, kStatusBadIndex);
    } else {
        // ------------------------------------------------------------------ gather, rows of codes
        // Lane l widens a scale's block, codes 32 (l / 8) .. + 31 of a 128-d stage, of rows l % 8,
        // l % 8 + 8, ... of the warp's (a store instruction's eight lanes meet eight rows: no bank conflict).
        // The codes of the group's next stage are loaded before it waits for that stage.
        constexpr int kLaneBytes = kFmt == SA_KV_FP4_E2M1 ? 16 : 32, kPer = kWarpRows / 8;
        const int group = (warp - kWarpGather) / kGroupWarps, part = lane >> 3;
        const int r0 = kWarpRows * ((warp - kWarpGather) % kGroupWarps) + (lane & 7);  // row r0 + 8 y
        // the lane's 16-byte units 4 (part % 2) .. + 3 of 64-d block part / 2; row r0 + 8 is 1024 bytes on
        const uint32_t dst = s_kv + (uint32_t)(part >> 1) * kBlockBytes + r0 * 128 +
                             ((uint32_t)((4 * (part & 1)) ^ (r0 & 7)) << 4);
        const uint32_t row_bytes = (uint32_t)p.steps * (4 * kLaneBytes) - (p.half ? 2 * kLaneBytes : 0);
        const uint32_t row_scales = 4 * p.steps - (p.half ? 2 : 0);
        const int64_t count = range.end - range.begin;
        bool ok = true, any_bad = false;
        Cursor cur(p, range.begin, group);  // the stage to load next
        const uint8_t* codes[kPer];
        // the scales of stage `part` of each row: a row's four lanes hold all of them (a byte load for every
        // lane and stage filled the few lines that the L1 has beside the stages)
        uint32_t scales[kPer];
        uint32_t there = 0;  // bit y: row r0 + 8 y has an entry
        int at_c = 0;        // the stage whose codes x holds
        int jn[kPer];
        int64_t unit_at = -1;  // the unit that codes points into
#pragma unroll
        for (int y = 0; y < kPer; ++y) jn[y] = cur.i < count ? entry_of(p, cur.u, r0 + 8 * y) : -1;
        Codes<kFmt> x[kPer];
        auto load = [&] {
            if (cur.i >= count) return;
            if (cur.i != unit_at) {
                unit_at = cur.i;
                const int64_t first = cur.u.seq * p.rows;
                there = 0;
                const uint8_t* cb = p.kv + first * row_bytes + part * kLaneBytes;
                const uint8_t* sb = p.kv_scale + first * row_scales + 4 * part;
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    const int j = valid(p, jn[y], any_bad);
                    there |= j >= 0 ? 1u << y : 0u;
                    codes[y] = cb + (uint64_t)(uint32_t)j * row_bytes;
                    scales[y] = 0;
                    const uint8_t* sc = sb + (uint64_t)(uint32_t)j * row_scales;
                    if (j >= 0 && part < p.steps) {
                        if (!p.half) {
                            scales[y] = __ldg(reinterpret_cast<const uint32_t*>(sc));
                        } else {  // rows of an odd number of halfwords
                            scales[y] = __ldg(reinterpret_cast<const uint16_t*>(sc));
                            if (part < p.steps - 1)
                                scales[y] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(sc + 2)) << 16;
                        }
                    }
                }
                int64_t at;
                const Unit nu = cur.next_unit(p, at);
                if (at < count) {
#pragma unroll
                    for (int y = 0; y < kPer; ++y) jn[y] = entry_of(p, nu, r0 + 8 * y);
                }
            }
            at_c = cur.c;
            const bool inside = !(cur.c == p.steps - 1 && p.half && part >= 2);
#pragma unroll
            for (int y = 0; y < kPer; ++y) {
                if ((there >> y & 1) && inside) {
                    const uint4* at = reinterpret_cast<const uint4*>(codes[y] + cur.c * (4 * kLaneBytes));
#pragma unroll
                    for (int i = 0; i < kLaneBytes / 16; ++i) {
                        const uint4 v = __ldg(at + i);
                        x[y].w[4 * i] = v.x;
                        x[y].w[4 * i + 1] = v.y;
                        x[y].w[4 * i + 2] = v.z;
                        x[y].w[4 * i + 3] = v.w;
                    }
                }
            }
            cur.advance(p, 2);
        };
        const int64_t n_stages = count * p.steps;
        load();
        int st = group;
        uint32_t ph = 1;
        for (int64_t s = group; s < n_stages; s += 2) {
            if (!(ok = warp_wait(smem_addr(&M.kv_empty[st]), ph, abort))) break;
#pragma unroll
            for (int y = 0; y < kPer; ++y) {
                const uint32_t se = __shfl_sync(0xFFFFFFFFu, scales[y], 8 * at_c + (lane & 7)) >> (8 * part) & 255u;
                if (!(there >> y & 1) || (at_c == p.steps - 1 && p.half && part >= 2)) continue;
                const uint32_t at = dst + st * kStageBytes + 1024 * y;
                const float sc = kFmt == SA_KV_FP4_E2M1 ? fp4::scale_f32(se) : fp8::e8m0_to_f32(se);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t(&w)[kLaneBytes / 4] = x[y].w;
                    uint4 lo, hi;
                    if constexpr (kFmt == SA_KV_FP4_E2M1)
                        fp4::dequant16(make_uint2(w[2 * i], w[2 * i + 1]), sc, lo, hi);
                    else
                        fp8::dequant16(make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]), sc,
                                       lo, hi);
                    st_shared_v4(at ^ (32u * i), lo.x, lo.y, lo.z, lo.w);
                    st_shared_v4(at ^ (32u * i + 16u), hi.x, hi.y, hi.z, hi.w);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&M.kv_full[st]));
            if ((st += 2) >= kStages) {
                st -= kStages;
                ph ^= 1;
            }
            load();
        }
        if (any_bad) atomicOr(p.status, kStatusBadIndex);
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && M.abort) atomicOr(p.status, kStatusTimeout);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int kFmt, int kN>
cudaError_t launch(const CUtensorMap& map, const Params& p, cudaStream_t stream) {
    static bool configured[64] = {};  // per instance and device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(row_weights_kernel<kFmt, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<kN>());
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    const int64_t sms = device_sm_count();
    const dim3 grid((unsigned)(p.n_units < sms ? p.n_units : sms));
    return launch_pdl(row_weights_kernel<kFmt, kN>, grid, dim3(Gather<kFmt>::kThreads), smem_bytes<kN>(), stream, map, p);
}

template <int kN>
cudaError_t launch_fmt(int fmt, const CUtensorMap& map, const Params& p, cudaStream_t stream) {
    return fmt == SA_KV_BF16       ? launch<SA_KV_BF16, kN>(map, p, stream)
           : fmt == SA_KV_FP8_E4M3 ? launch<SA_KV_FP8_E4M3, kN>(map, p, stream)
                                   : launch<SA_KV_FP4_E2M1, kN>(map, p, stream);
}

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_row_weights(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format,
                                    const float* lse, const int32_t* idx, float softmax_scale, int64_t b,
                                    int64_t s, int h, int d, int64_t rows, int topk, int64_t* acc,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace sa;
    if (!kv_format_known(kv_format)) return SA_ERR_INVALID_ARG;
    if (b < 0 || s < 0 || h < 1 || d < 1 || rows < 0 || topk < 0) return SA_ERR_INVALID_ARG;
    // (the shapes sparse_attn takes)
    if (sa_sparse_attn_workspace_size(b, s, h, d, rows, topk, kv_format) == 0) return SA_ERR_UNSUPPORTED;
    if (topk > INT32_MAX - kTile) return SA_ERR_UNSUPPORTED;  // a tile's last column is a 32-bit number
    if (kv_format == SA_KV_BF16 && kv_scale) return SA_ERR_INVALID_ARG;
    if (b * s == 0 || topk == 0) return SA_OK;
    if (!q || !lse || !idx || (rows > 0 && (!kv || !acc))) return SA_ERR_INVALID_ARG;
    if (kv_format != SA_KV_BF16 && rows > 0 && !kv_scale) return SA_ERR_INVALID_ARG;
    // the kernel reads a row's scales in words (halfwords where a row is an odd number of them); at d = 512,
    // as sparse_attn does
    const uintptr_t scale_align = d == 512 ? 16 : d % 128 == 0 ? 4 : 2;
    if (!is_aligned(q, 16) || !is_aligned(kv, 16) || !is_aligned(kv_scale, scale_align) || !is_aligned(lse, 4) ||
        !is_aligned(idx, 4) || !is_aligned(acc, 8))
        return SA_ERR_INVALID_ARG;
    const size_t n_tok = (size_t)(b * s), acc_bytes = (size_t)(b * rows) * 8;
    if (overlap(acc, acc_bytes, q, n_tok * h * (size_t)d * 2) ||
        overlap(acc, acc_bytes, kv, (size_t)(b * rows) * kv_row_bytes(kv_format, d)) ||
        overlap(acc, acc_bytes, kv_scale, (size_t)(b * rows) * (d / 32)) ||
        overlap(acc, acc_bytes, lse, n_tok * h * 4) || overlap(acc, acc_bytes, idx, n_tok * topk * 4))
        return SA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < SA_STATUS_BYTES) return SA_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256) || overlap(acc, acc_bytes, workspace, workspace_bytes))
        return SA_ERR_INVALID_ARG;
    const int n = h <= 64 ? 64 : 128;  // heads a product covers
    CUtensorMap map;
    if (!encode_rows_map(map, q, d, (int64_t)n_tok * h, n)) return SA_ERR_CUDA;
    Params p;
    p.q = reinterpret_cast<const uint8_t*>(q);
    p.q_row = 2 * (int64_t)d;
    p.kv = reinterpret_cast<const uint8_t*>(kv);
    p.kv_scale = kv_scale;
    p.lse = lse;
    p.idx = idx;
    p.acc = reinterpret_cast<unsigned long long*>(acc);
    p.status = reinterpret_cast<uint32_t*>(workspace);
    p.scale_log2 = softmax_scale * kLog2e;
    p.s_len = s;
    p.h = h;
    p.steps = (d + 127) / 128;
    p.half = d % 128 != 0;
    p.rows = rows;
    p.topk = topk;
    p.n_tiles = (topk + kTile - 1) / kTile;
    p.n_units = b * s * (int64_t)p.n_tiles;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = n == 64 ? launch_fmt<64>(kv_format, map, p, st) : launch_fmt<128>(kv_format, map, p, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
