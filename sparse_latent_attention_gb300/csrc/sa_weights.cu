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
// Roles (persistent CTAs, 22 warps; every wait is bounded, as in the attention kernel):
//   warp 0      MMA issue (one elected lane): per 64-d chunk of a tile four MMAs of 128 x kN x 16
//   warp 1      Q by TMA (128-byte swizzle), chunk by chunk: a chunk of the next token's Q is loaded as
//               soon as the last tile's product has passed it
//   warps 2-5   epilogue: exponentials, sum over heads, accumulation
//   warps 6-21  gather, eight rows of the tile each, one 64-d chunk [128 rows x 128 bytes] a stage: bf16
//               rows with 16-byte cp.async; rows of codes are loaded eight chunks ahead into registers and
//               widened into the stage (exact: see sa_fp8.cuh, sa_fp4.cuh)

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
constexpr int kWarpEpilogue = 2, kWarpGather = 6, kGatherWarps = 16;
constexpr int kThreads = 32 * (kWarpGather + kGatherWarps);
constexpr int kMaxChunks = 8;           // 64-d chunks of a row: d <= 512
constexpr uint32_t kStageBytes = kTile * 128;
constexpr int kMaxStages = 9;

// By the heads a product covers (kN = 64 or 128): the stages that fit beside Q, and how many stages a
// bf16 gather warp keeps in flight before it waits for the oldest (at most stages - 1).
template <int kN>
struct Shape {
    static constexpr uint32_t kQChunkBytes = kN * 128;
    static constexpr uint32_t kQBytes = kMaxChunks * kQChunkBytes;
    static constexpr int kStages = kN == 64 ? 9 : 5;
    static constexpr int kLag = kN == 64 ? 5 : 3;
    static constexpr uint32_t kOffQ = kStages * kStageBytes;
    static constexpr uint32_t kOffMisc = kOffQ + kQBytes;
};

struct Misc {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t q_full[kMaxChunks], q_empty[kMaxChunks];
    uint64_t s_full[2], s_empty[2];  // per accumulator (TMEM)
    uint64_t done;
    uint32_t tmem_base;
    int abort;
    alignas(16) float nlse[4][128];  // -lse log2(e) of the token's heads, a table per epilogue warp
};

template <int kN>
constexpr uint32_t smem_bytes() {
    return Shape<kN>::kOffMisc + (uint32_t)sizeof(Misc) + 1024u;  // + alignment slack
}
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory budget");

struct Params {
    const uint8_t* kv;
    const uint8_t* kv_scale;
    const float* lse;
    const int32_t* idx;
    unsigned long long* acc;
    uint32_t* status;
    float scale_log2;
    int64_t s_len;
    int h, chunks;
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

// The entry in row r of a unit's tile: its cache row, or -1 (empty, past the columns, or out of range).
__device__ __forceinline__ int entry_of(const Params& p, const Unit& u, int r, bool& bad) {
    const int col = u.tile * kTile + r;
    int j = col < p.topk ? __ldg(p.idx + u.token * (int64_t)p.topk + col) : -1;
    bad = j < -1 || j >= p.rows;
    return bad ? -1 : j;
}

// Sixteen codes of a row and their scale, on their way from memory to a stage.
template <int kFmt>
struct Codes {
    uint32_t w[kFmt == SA_KV_FP4_E2M1 ? 2 : 4];
    uint32_t scale;  // the e8m0 byte; kNone: no row
};
constexpr uint32_t kNone = 0xFFFFFFFFu;

template <int kFmt, int kN>
__global__ void __launch_bounds__(kThreads, 1)
    row_weights_kernel(const __grid_constant__ CUtensorMap q_map, Params p) {
    using Sh = Shape<kN>;
    constexpr int kStages = Sh::kStages;
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
            mbar_init(smem_addr(&M.kv_full[i]), kGatherWarps);
            mbar_init(smem_addr(&M.kv_empty[i]), 1);
        }
        for (int i = 0; i < kMaxChunks; ++i) {
            mbar_init(smem_addr(&M.q_full[i]), 1);
            mbar_init(smem_addr(&M.q_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&M.s_full[i]), 1);
            mbar_init(smem_addr(&M.s_empty[i]), 4);
        }
        mbar_init(smem_addr(&M.done), 1);
        M.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        tmem_alloc(smem_addr(&M.tmem_base), 256);
        tmem_relinquish();
    }
    if (warp == 1 && lane == 0) tma_prefetch_desc(&q_map);
    pdl_wait();  // the set-up above touches no global memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M.tmem_base;
    const Range range = unit_range(p);

    if (warp == 0) {
        // ------------------------------------------------------------------ MMA issue
        constexpr uint32_t id = idesc_bf16_f32(kTile, kN, false, false);
        const uint64_t a0 = smem_desc_sw128(s_kv, 16, 1024);  // tile rows, K-major
        const uint64_t b0 = smem_desc_sw128(s_q, 16, 1024);   // heads, K-major
        const uint32_t ahi = (uint32_t)(a0 >> 32), bhi = (uint32_t)(b0 >> 32);
        bool ok = true;
        int st = 0;
        uint32_t ph = 0, k = 0, qph = 0;
        Unit u(p, range.begin);
        for (int64_t i = range.begin; i < range.end && ok; ++i, ++k) {
            const bool first = i == range.begin || u.tile == 0;
            const bool last = i == range.end - 1 || u.tile == p.n_tiles - 1;
            const uint32_t b = k & 1;
            if (!(ok = warp_wait(smem_addr(&M.s_empty[b]), ((k >> 1) & 1) ^ 1, abort))) break;
            const uint32_t col = tmem + 128 * b;
            for (int c = 0; c < p.chunks; ++c) {
                ok = (!first || warp_wait(smem_addr(&M.q_full[c]), qph, abort)) &&
                     warp_wait(smem_addr(&M.kv_full[st]), ph, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t alo = (uint32_t)a0 + st * (kStageBytes >> 4);
                const uint32_t blo = (uint32_t)b0 + c * (Sh::kQChunkBytes >> 4);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mma_lohi_elect(col, alo + 2 * q, ahi, blo + 2 * q, bhi, id, (c | q) != 0);
                mma_commit_elect(smem_addr(&M.kv_empty[st]));
                if (last) mma_commit_elect(smem_addr(&M.q_empty[c]));
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
            mma_commit_elect(smem_addr(&M.s_full[b]));
            if (last) qph ^= 1;
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
            int loaded = 0;  // chunks of the last of them that were asked for
            Unit u(p, range.begin);
            const int64_t last_token = range.end > range.begin ? (range.end - 1) / p.n_tiles : -1;
            for (int64_t token = u.token; token <= last_token && ok; ++token) {
                ++n;
                loaded = 0;
                for (int c = 0; c < p.chunks; ++c) {
                    if (!(ok = mbar_wait(smem_addr(&M.q_empty[c]), n & 1, abort))) break;
                    mbar_arrive_expect_tx(smem_addr(&M.q_full[c]), Sh::kQChunkBytes);
                    tma_load_2d(s_q + c * Sh::kQChunkBytes, &q_map, 64 * c, (int32_t)(token * p.h),
                                smem_addr(&M.q_full[c]));
                    ++loaded;
                }
            }
            // after a failed wait, let the loads under way land before the CTA exits
            if (*abort)
                for (int c = 0; c < p.chunks; ++c) {
                    const uint32_t uses = n - (c < loaded ? 0u : 1u);  // times chunk c was asked for
                    if (uses > 0) mbar_drain(smem_addr(&M.q_full[c]), (uses - 1) & 1);
                }
        }
        __syncwarp();
    } else if (warp < kWarpGather) {
        // ------------------------------------------------------------------ epilogue
        const int q4 = warp & 3;  // the TMEM lanes this warp may read: 32 q4 .. 32 q4 + 31
        const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
        float* table = M.nlse[q4];
        bool ok = true, bad;
        uint32_t k = 0;
        Unit u(p, range.begin), un = u;  // un: a unit ahead, whose entry is loaded meanwhile
        int jn = -1;
        float ln[kN / 32];  // the next token's lse, heads lane + 32 i
        auto load_lse = [&](int64_t token) {
#pragma unroll
            for (int i = 0; i < kN / 32; ++i)
                ln[i] = lane + 32 * i < p.h ? __ldg(p.lse + token * p.h + lane + 32 * i) : 0.f;
        };
        if (range.begin < range.end) {
            jn = entry_of(p, u, 32 * q4 + lane, bad);
            load_lse(u.token);
        }
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        for (int64_t i = range.begin; i < range.end && ok; ++i, ++k) {
            const uint32_t b = k & 1;
            const int j = jn;
            if (i == range.begin || u.tile == 0) {
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kN / 32; ++q) table[lane + 32 * q] = -ln[q] * kLog2e;
                __syncwarp();
                if (range.end - i > p.n_tiles - u.tile) load_lse(u.token + 1);
            }
            un.step(p);
            if (i + 1 < range.end) jn = entry_of(p, un, 32 * q4 + lane, bad);
            if (!(ok = warp_wait(smem_addr(&M.s_full[b]), (k >> 1) & 1, abort))) break;
            tc_fence_after();
            uint64_t sum[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
            for (int q = 0; q < kN / 32; ++q) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem + lane_base + 128 * b + 32 * q, r);
                tmem_wait_ld();
                if (q == kN / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&M.s_empty[b]));
                }
                if (32 * q >= p.h) continue;
                const int heads = p.h - 32 * q;  // of these 32
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 n4 = *reinterpret_cast<const float4*>(&table[32 * q + 4 * c]);
                    float x[4];
                    f2_split(ffma2(f2(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1])), sc2,
                                   f2(n4.x, n4.y)), x[0], x[1]);
                    f2_split(ffma2(f2(__uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3])), sc2,
                                   f2(n4.z, n4.w)), x[2], x[3]);
                    float e[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) e[y] = fast_exp2(x[y]);
                    if (heads < 32) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (4 * c + y >= heads) e[y] = 0.f;
                    }
                    sum[2 * (c & 1)] = fadd2(sum[2 * (c & 1)], f2(e[0], e[1]));
                    sum[2 * (c & 1) + 1] = fadd2(sum[2 * (c & 1) + 1], f2(e[2], e[3]));
                }
            }
            float w0, w1;
            f2_split(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), w0, w1);
            const float w = fminf(fmaxf(w0 + w1, 0.f), (float)p.h);  // (a NaN becomes 0)
            if (j >= 0) atomicAdd(p.acc + u.seq * p.rows + j, __float2ull_rn(w * kUnits));
            u = un;
        }
    } else if constexpr (kFmt == SA_KV_BF16) {
        // ------------------------------------------------------------------ gather, bf16
        // Lane l copies 16-byte unit l % 8 of rows l / 8 and l / 8 + 4 of the warp's eight.
        const int gw = warp - kWarpGather, unit = lane & 7;
        const int r0 = 8 * gw + (lane >> 3), r1 = r0 + 4;
        const uint32_t d0 = s_kv + r0 * 128 + ((uint32_t)(unit ^ (r0 & 7)) << 4);
        const uint32_t d1 = s_kv + r1 * 128 + ((uint32_t)(unit ^ (r1 & 7)) << 4);
        const int64_t row_bytes = (int64_t)p.chunks * 128;
        bool ok = true, bad0, bad1;
        int st = 0, st_full = 0;  // the stage to fill next, and the oldest one still under way
        uint32_t ph = 1, under_way = 0;
        Unit u(p, range.begin);
        int j0 = -1, j1 = -1;
        for (int64_t i = range.begin; i < range.end && ok; ++i) {
            if (i == range.begin) {
                j0 = entry_of(p, u, r0, bad0);
                j1 = entry_of(p, u, r1, bad1);
                if (bad0 || bad1) atomicOr(p.status, kStatusBadIndex);
            }
            const uint8_t* base = p.kv + u.seq * p.rows * row_bytes + unit * 16;
            const uint8_t* g0 = base + j0 * row_bytes;
            const uint8_t* g1 = base + j1 * row_bytes;
            const bool v0 = j0 >= 0, v1 = j1 >= 0;
            u.step(p);
            if (i + 1 < range.end) {  // the next unit's entries
                j0 = entry_of(p, u, r0, bad0);
                j1 = entry_of(p, u, r1, bad1);
                if (bad0 || bad1) atomicOr(p.status, kStatusBadIndex);
            }
            for (int c = 0; c < p.chunks; ++c) {
                if (!(ok = warp_wait(smem_addr(&M.kv_empty[st]), ph, abort))) break;
                if (v0) cp_async16(d0 + st * kStageBytes, g0 + c * 128, 16u);
                if (v1) cp_async16(d1 + st * kStageBytes, g1 + c * 128, 16u);
                cp_async_commit();
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
                if (++under_way > (uint32_t)Sh::kLag) {
                    cp_async_wait<Sh::kLag>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&M.kv_full[st_full]));
                    if (++st_full == kStages) st_full = 0;
                    --under_way;
                }
            }
        }
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        for (; ok && under_way > 0; --under_way) {
            if (lane == 0) mbar_arrive(smem_addr(&M.kv_full[st_full]));
            if (++st_full == kStages) st_full = 0;
        }
    } else {
        // ------------------------------------------------------------------ gather, rows of codes
        // Four lanes a row: lane l widens codes 16 (l % 4) .. + 15 of each 64-d chunk of row l / 4 of the
        // warp's eight.  The loads run kAhead chunks before the widening, over the ends of tiles.
        constexpr int kAhead = 8;
        constexpr int kLaneBytes = kFmt == SA_KV_FP4_E2M1 ? 8 : 16;
        const int gw = warp - kWarpGather, sub = lane & 3;
        const int r = 8 * gw + (lane >> 2);
        const uint32_t dst = s_kv + r * 128 + ((uint32_t)((2 * sub) ^ (r & 7)) << 4);
        const int64_t row_bytes = (int64_t)p.chunks * (4 * kLaneBytes);
        const int64_t n_steps = (range.end - range.begin) * p.chunks;
        // the chunk to load next
        Unit u(p, range.begin);
        const uint8_t *codes = nullptr, *scales = nullptr;
        int64_t left = range.end - range.begin;  // tiles not yet begun
        int c = 0, jn = -1;
        bool there = false, bad;
        if (left > 0) {
            jn = entry_of(p, u, r, bad);
            if (bad) atomicOr(p.status, kStatusBadIndex);
        }
        auto load = [&](Codes<kFmt>& x) {
            if (c == 0) {
                there = left > 0 && jn >= 0;
                if (there) {
                    const int64_t row = u.seq * p.rows + jn;
                    codes = p.kv + row * row_bytes + sub * kLaneBytes;
                    scales = p.kv_scale + row * (2 * p.chunks) + (sub >> 1);
                }
                u.step(p);
                if (--left > 0) {
                    jn = entry_of(p, u, r, bad);
                    if (bad) atomicOr(p.status, kStatusBadIndex);
                }
            }
            x.scale = kNone;
            if (there) {
                if constexpr (kFmt == SA_KV_FP4_E2M1) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes + c * 32));
                    x.w[0] = v.x;
                    x.w[1] = v.y;
                } else {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(codes + c * 64));
                    x.w[0] = v.x;
                    x.w[1] = v.y;
                    x.w[2] = v.z;
                    x.w[3] = v.w;
                }
                x.scale = __ldg(scales + 2 * c);
            }
            if (++c == p.chunks) c = 0;
        };
        Codes<kFmt> ring[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(ring[i]);
        bool ok = true;
        int st = 0;
        uint32_t ph = 1;
        for (int64_t s = 0; s < n_steps && ok; s += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (s + i >= n_steps) break;
                if (!(ok = warp_wait(smem_addr(&M.kv_empty[st]), ph, abort))) break;
                if (ring[i].scale != kNone) {
                    uint4 lo, hi;
                    if constexpr (kFmt == SA_KV_FP4_E2M1)
                        fp4::dequant16(make_uint2(ring[i].w[0], ring[i].w[1]),
                                       fp4::scale_f32(ring[i].scale), lo, hi);
                    else
                        fp8::dequant16(make_uint4(ring[i].w[0], ring[i].w[1], ring[i].w[2], ring[i].w[3]),
                                       fp8::e8m0_to_f32(ring[i].scale), lo, hi);
                    const uint32_t at = dst + st * kStageBytes;
                    st_shared_v4(at, lo.x, lo.y, lo.z, lo.w);
                    st_shared_v4(at ^ 16u, hi.x, hi.y, hi.z, hi.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&M.kv_full[st]));
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
                load(ring[i]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && M.abort) atomicOr(p.status, kStatusTimeout);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
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
    return launch_pdl(row_weights_kernel<kFmt, kN>, grid, dim3(kThreads), smem_bytes<kN>(), stream, map, p);
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
    if (kv_format == SA_KV_BF16 && kv_scale) return SA_ERR_INVALID_ARG;
    if (b * s == 0 || topk == 0) return SA_OK;
    if (!q || !lse || !idx || (rows > 0 && (!kv || !acc))) return SA_ERR_INVALID_ARG;
    if (kv_format != SA_KV_BF16 && rows > 0 && !kv_scale) return SA_ERR_INVALID_ARG;
    if (!is_aligned(q, 16) || !is_aligned(kv, 16) || !is_aligned(kv_scale, 16) || !is_aligned(lse, 4) ||
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
    p.kv = reinterpret_cast<const uint8_t*>(kv);
    p.kv_scale = kv_scale;
    p.lse = lse;
    p.idx = idx;
    p.acc = reinterpret_cast<unsigned long long*>(acc);
    p.status = reinterpret_cast<uint32_t*>(workspace);
    p.scale_log2 = softmax_scale * kLog2e;
    p.s_len = s;
    p.h = h;
    p.chunks = d / 64;
    p.rows = rows;
    p.topk = topk;
    p.n_tiles = (topk + kTile - 1) / kTile;
    p.n_units = b * s * (int64_t)p.n_tiles;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = n == 64 ? launch_fmt<64>(kv_format, map, p, st) : launch_fmt<128>(kv_format, map, p, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
