// The paged latent cache's write side, and the window attention over it: argument checks, and the index table
// for the kernel families that gather by row (include/serve/sa_paged.h).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "sa_internal.cuh"
#include "sa_paged.cuh"
#include "sa_rows.cuh"
#include "serve/sa_paged.h"

namespace sa {
namespace {

using namespace rows;
using paged::Batch;

// ---------------------------------------------------------------------------------------------
// page_write
// ---------------------------------------------------------------------------------------------

struct Write {
    const __nv_bfloat16* x;
    int64_t xs, n;
    int d;
    Batch a;
    __nv_bfloat16* pages;
    int64_t ps, pp;
    uint8_t* codes;
    int64_t cs, cp;
    uint8_t* scales;
    int64_t ss, sp;
    const float* weight;
    RmsOf of;
    const float* rot;
    int64_t npos;
    int rope_dim;
    uint32_t* status;
};

// A warp a token, eight consecutive elements a lane and chunk (kPer chunks of 256).  kRun tokens one behind the
// other a warp: their rows are under way before the first one's sequence and page are known, and the sequence is
// looked for once.  Bound by arithmetic whose steps wait for one another, at few warps: some 650 instructions a row of
// 512 with norm, rotation and 4-bit codes (a third are the norm's products and what they lose, a third the codes and
// their round trip, a sixth what makes the codes exact), 96 registers, so that 29 % of the warps are there; 59 % of
// the issue slots are used, and the first stall is the wait for the instruction before.  65536 such rows take 74 us with
// two tokens a warp and five blocks a SM (seven, whose registers spill, take 1 us more), 61 where codes next to a border
// may fall to its other side.
template <int kQuant, int kPer, int kRun, bool kVec>
__global__ void __launch_bounds__(128, kPer == 4 ? 3 : 5) page_write_kernel(const __grid_constant__ Write p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, chunks = p.d >> 3;
    const int64_t t0 = (blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5)) * kRun;
    uint4 in[kRun][kPer];
#pragma unroll
    for (int r = 0; r < kRun; ++r)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = lane + 32 * i;
            in[r][i] = c < chunks && t0 + r < p.n ? load8<kVec>(p.x + (t0 + r) * p.xs + 8 * c)
                                                  : make_uint4(0u, 0u, 0u, 0u);
        }
    // the weights of this lane's columns, for all of its tokens
    uint64_t w[kPer][4];
    if (p.weight) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = lane + 32 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[i][j] = c < chunks ? tc::f2(__ldg(p.weight + 8 * c + 2 * j), __ldg(p.weight + 8 * c + 2 * j + 1)) : 0ull;
        }
    }
    paged::Token k = {0, 0, -1};
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
        const int64_t t = t0 + r;
        if (t >= p.n) break;
        if (r > 0 && t < k.end) {
            ++k.pos;
        } else {
            k = paged::token_of(p.a, t);
        }
        if (k.pos < 0) continue;
        uint32_t page, off;
        if (!paged::place_of(p.a, k.seq, (uint32_t)k.pos, page, off) || (p.rot && k.pos >= p.npos)) {
            if (p.status && lane == 0) atomicOr(p.status, kStatusBadIndex);
            continue;
        }
        uint64_t v[kPer][4];  // elements 2 j and 2 j + 1
        uint32_t large = 0u;
        if (p.weight) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                large = largest_pair(largest_pair(large, largest_pair(in[r][i].x, in[r][i].y)),
                                     largest_pair(in[r][i].z, in[r][i].w));
            large = largest_pair(large, large << 16);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float e[8];
            unpacked8(in[r][i], e);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = tc::f2(e[2 * j], e[2 * j + 1]);
        }
        Two f = {1.f, 0.f};
        float scale = 1.f;
        if (p.weight) {
            auto squares = [&](float largest) {
                Squares<4 * kPer> sum(largest);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum.add(v[i][j]);
                return warp_sum(sum.total());
            };
            f = add(squares(__uint_as_float(large)), p.of.shift);
            if (leaves_range(f)) {
                scale = rescaling(f);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], tc::f2(scale, scale));
                f = add_scaled(squares(__uint_as_float(large & 0x7FFFFFFFu) * scale), p.of.shift, scale);
            }
            f = inverse_rms(f, p.of);
        }
        const uint64_t fh = tc::f2(f.h, f.h), fn = tc::f2(-f.h, -f.h), fl = tc::f2(f.l, f.l);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = lane + 32 * i;
            if (32 * i >= chunks) break;
            const bool mine = c < chunks;
            float h[8], l[8], out[8];  // y in two parts, and rounded
            if (p.weight) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // x f as p + e + x fl, that times w: each product's rounding from the product again with the
                    // rounded one, which the negative factor gives, taken away
                    const uint64_t x = v[i][j], pr = mul2(x, fh), np = mul2(x, fn);
                    const uint64_t pl = fma2(x, fl, fma2(x, fh, np));
                    const uint64_t q = mul2(pr, w[i][j]), ql = fma2(pl, w[i][j], fma2(pr, w[i][j], mul2(np, w[i][j])));
                    tc::f2_split(q, h[2 * j], h[2 * j + 1]);
                    tc::f2_split(ql, l[2 * j], l[2 * j + 1]);
                    tc::f2_split(add2(q, ql), out[2 * j], out[2 * j + 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) tc::f2_split(v[i][j], h[2 * j], h[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    l[j] = 0.f;
                    out[j] = h[j];
                }
            }
            const int first = p.d - p.rope_dim;
            const bool turned = p.rot && mine && 8 * c + 8 > first;
            if (turned) {
                const float2* turn = reinterpret_cast<const float2*>(p.rot) + k.pos * (p.rope_dim >> 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = 8 * c + 2 * j - first;
                    if (e < 0) continue;
                    // a c - b s: b s rounded to u, what that lost, a c - u in one rounding, and the parts' own
                    const float2 cs = __ldg(turn + (e >> 1));
                    const float a = h[2 * j], b = h[2 * j + 1], al = l[2 * j], bl = l[2 * j + 1];
                    const float u = __fmul_rn(b, cs.y), ul = fmaf(bl, cs.y, fmaf(b, cs.y, -u));
                    const float z = __fmul_rn(b, cs.x), zl = fmaf(bl, cs.x, fmaf(b, cs.x, -z));
                    h[2 * j] = fmaf(a, cs.x, -u);
                    l[2 * j] = fmaf(al, cs.x, -ul);
                    h[2 * j + 1] = fmaf(a, cs.y, z);
                    l[2 * j + 1] = fmaf(al, cs.y, zl);
                    out[2 * j] = h[2 * j] + l[2 * j];
                    out[2 * j + 1] = h[2 * j + 1] + l[2 * j + 1];
                }
            }
            // (for a value on a border, which is seldom: what that one rounding lost, from the row read again)
            auto whole = [&] {
                if (!turned) return;
                const float2* turn = reinterpret_cast<const float2*>(p.rot) + k.pos * (p.rope_dim >> 1);
                float x[8];
                unpacked8(load8<kVec>(p.x + t * p.xs + 8 * c), x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = 8 * c + 2 * j - first;
                    if (e < 0) continue;
                    float a = x[2 * j], b = x[2 * j + 1];
                    if (p.weight) {
                        a = __fmul_rn(__fmul_rn(a * scale, f.h), __ldg(p.weight + 8 * c + 2 * j));
                        b = __fmul_rn(__fmul_rn(b * scale, f.h), __ldg(p.weight + 8 * c + 2 * j + 1));
                    }
                    auto lost = [&](float m, float y, float sum) {  // a m + y - sum
                        const float q = __fmul_rn(a, m);
                        const Two s = two_sum(q, y);
                        return ((s.h - sum) + s.l) + fmaf(a, m, -q);
                    };
                    const float2 cs = __ldg(turn + (e >> 1));
                    l[2 * j] += lost(cs.x, -__fmul_rn(b, cs.y), h[2 * j]);
                    l[2 * j + 1] += lost(cs.y, __fmul_rn(b, cs.x), h[2 * j + 1]);
                }
            };
            const float top = p.weight || p.rot ? settle8(h, l, out, whole) : largest8(out);
            uint4 values;
            if constexpr (kQuant == SA_KV_BF16) {
                values = packed8(out);
            } else {
                constexpr bool kFp4 = kQuant == SA_KV_FP4_E2M1;
                uint2 codes;
                uint32_t se;
                quantise8<kFp4>(out, top, codes, se);
                values = values8<kFp4>(codes, se);
                if (p.codes && mine) {
                    store_codes8<kVec, kFp4>(p.codes + page * p.cp + off * p.cs + (kFp4 ? 4 : 8) * c, codes);
                    if ((c & 3) == 0) p.scales[page * p.sp + off * p.ss + (c >> 2)] = (uint8_t)se;
                }
            }
            if (p.pages && mine) store8<kVec>(p.pages + page * p.pp + off * p.ps + 8 * c, values);
        }
    }
}

template <int kQuant, int kPer, bool kVec>
cudaError_t write_run(const Write& p, cudaStream_t st) {
    // two waves of a token a warp hold 40 a SM; beyond, two tokens a warp (one / two: 64 rows 4.3 / 5.0 us, 4096 rows 7.6 /
    // 8.5, 8192 rows 12.1 / 11.9, 65536 rows 72.0 / 64.5)
    const bool few = p.n <= 40 * (int64_t)device_sm_count();
    const int64_t per = few ? 4 : 8, grid = (p.n + per - 1) / per;
    return few ? launch_pdl(page_write_kernel<kQuant, kPer, 1, kVec>, dim3((unsigned)grid), dim3(128), 0, st, p)
               : launch_pdl(page_write_kernel<kQuant, kPer, 2, kVec>, dim3((unsigned)grid), dim3(128), 0, st, p);
}

template <int kQuant>
cudaError_t write_launch(const Write& p, bool vec, cudaStream_t st) {
    if (!vec) return write_run<kQuant, 4, false>(p, st);
    if (p.d <= 256) return write_run<kQuant, 1, true>(p, st);
    if (p.d <= 512) return write_run<kQuant, 2, true>(p, st);
    return write_run<kQuant, 4, true>(p, st);
}

// ---------------------------------------------------------------------------------------------
// window_attn by an index table
// ---------------------------------------------------------------------------------------------

// The pool's row of each position that a token may see, -1 where there is none: entry c < lead of a token's row is
// position c, entry lead + c position p - window + 1 + c where that is not below lead.  (lead is `first`, or where the
// table holds fewer positions than a token may see all of those, and no entry follows.)  pos: each token's position in the
// rotation's table.  A block a token and 128 entries at a time.
__global__ void __launch_bounds__(128) window_rows_kernel(Batch a, int64_t n, int window, int first, int lead, int topk,
                                                          int32_t* idx, int32_t* pos, int64_t npos,
                                                          uint32_t* status) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const paged::Token k = paged::token_of(a, t);
    bool bad = k.pos >= a.max_pages * a.page;
    if (pos && blockIdx.y == 0 && threadIdx.x == 0) {
        bad |= k.pos >= npos;
        pos[t] = (int32_t)(k.pos < 0 ? 0 : k.pos >= npos ? npos - 1 : k.pos);
    }
    for (int c = (int)(blockIdx.y * blockDim.x + threadIdx.x); c < topk; c += (int)(gridDim.y * blockDim.x)) {
        int32_t row = -1;
        const int64_t j = c < lead ? c : k.pos - window + 1 + (c - lead);
        if (j >= 0 && j <= k.pos && (c < lead ? j < first || j > k.pos - window : j >= lead)) {
            row = (int32_t)paged::row_of(a, k.seq, (uint32_t)j);
            bad |= row < 0;
        }
        idx[t * topk + c] = row;
    }
    if (bad) atomicOr(status, kStatusBadIndex);
}

// A pool of rows: their bytes, and how far apart rows and pages are.
struct Pool {
    const void* at;
    int64_t width, row, page;
};

// Whether two pools share a byte.  Pages, or rows, equally far apart may lie between one another (codes and
// scales side by side in a row, or in a page); of others the whole spans count.
bool pools_overlap(const Pool& a, const Pool& b, int64_t n_pages, int64_t rows) {
    const int64_t as = (rows - 1) * a.row + a.width, bs = (rows - 1) * b.row + b.width;
    if (!overlap(a.at, (n_pages - 1) * a.page + as, b.at, (n_pages - 1) * b.page + bs)) return false;
    if (n_pages > 1 && a.page != b.page) return true;
    if (n_pages > 1 && apart(a.at, as, b.at, bs, a.page)) return false;
    return !(rows > 1 && a.row == b.row && (n_pages == 1 || a.page % a.row == 0) &&
             apart(a.at, a.width, b.at, b.width, a.row));
}

constexpr int64_t k31 = int64_t(1) << 31;

// What count * stride elements span has to be an address's distance.
bool spans(int64_t count, int64_t stride) { return (double)count * (double)stride < 72057594037927936.0; }

bool window_shape(int64_t n, int64_t b, int h, int d, int64_t window, int64_t first, int page) {
    return n >= 0 && b >= 0 && h >= 1 && d >= 1 && window >= 1 && first >= 0 && page >= 1 &&
           window < (int64_t(1) << 30) && first < (int64_t(1) << 30) && first + window < (int64_t(1) << 30);
}

bool window_supported(int64_t n, int h, int d) {
    return h <= 128 && d >= 64 && d <= 512 && d % 64 == 0 && n < k31 && n * (int64_t)h < k31;
}

// The workspace of a call: the status word and the scratch of the kernels that the call is routed to, then, of those that
// gather by row, the index table and positions.
struct Parts {
    int topk;  // entries of the index table
    size_t idx, pos, all;
};

Parts parts_of(int64_t n, int64_t b, int h, int d, Reach seen, int page, int kv_format) {
    if (window_tc_supports(d, kv_format, page)) {
        const size_t all = SA_STATUS_BYTES + align_up(window_tc_scratch_bytes(n, b, h, seen.window, seen.first), 256);
        return {0, all, all, all};
    }
    const int topk = (int)(seen.first + seen.window);
    const int fam = routed_family(SA_FAMILY_AUTO, h, d, kv_format, 1, 0);
    Parts s;
    s.topk = topk;
    s.idx = align_up(routed_workspace_bytes(fam, 1, n, h, d, 0, topk), 256);
    s.pos = s.idx + align_up((size_t)n * topk * sizeof(int32_t), 256);
    s.all = s.pos + align_up((size_t)n * sizeof(int32_t), 256);
    return s;
}

}  // namespace
}  // namespace sa

extern "C" sa_status sa_page_write(const void* x, int64_t n, int d, int64_t x_stride, const int32_t* page_table,
                                   int64_t max_pages, int64_t table_stride, const int32_t* q_start,
                                   const int32_t* kv_len, int64_t b, int64_t n_pages, int page, int quant,
                                   void* pages, int64_t pages_stride, int64_t pages_page_stride, uint8_t* codes,
                                   int64_t codes_stride, int64_t codes_page_stride, uint8_t* scales,
                                   int64_t scales_stride, int64_t scales_page_stride, const float* weight,
                                   float eps, const float* rot, int64_t npos, int rope_dim, void* status,
                                   void* stream) {
    using namespace sa;
    if (n < 0 || d < 32 || d % 32 != 0 || b < 0 || n_pages < 0 || page < 1 || max_pages < 0) return SA_ERR_INVALID_ARG;
    if (!kv_format_known(quant) || (!pages && !codes) || !codes != !scales) return SA_ERR_INVALID_ARG;
    if (codes && quant == SA_KV_BF16) return SA_ERR_INVALID_ARG;
    if (rot && (rope_dim < 2 || rope_dim % 2 != 0 || rope_dim > d || npos < 0)) return SA_ERR_INVALID_ARG;
    if (weight && !(eps >= 0.f)) return SA_ERR_INVALID_ARG;
    if (d > 1024 || n >= k31 || n_pages >= k31 || n_pages * (int64_t)page >= (int64_t(1) << 40) || max_pages >= k31 ||
        b >= k31)
        return SA_ERR_UNSUPPORTED;
    if (n == 0 || b == 0) return SA_OK;
    if (n_pages < 1) return SA_ERR_INVALID_ARG;
    if (!x || !aligned(x, 2) || x_stride < d) return SA_ERR_INVALID_ARG;
    if (!q_start || !aligned(q_start, 4) || !kv_len || !aligned(kv_len, 4)) return SA_ERR_INVALID_ARG;
    if ((max_pages > 0 && !page_table) || !aligned(page_table, 4) || (b > 1 && table_stride < max_pages))
        return SA_ERR_INVALID_ARG;
    if (!aligned(weight, 4) || !aligned(rot, 8) || !aligned(status, 4)) return SA_ERR_INVALID_ARG;
    if (!spans(n, x_stride) || !spans(b, table_stride) || !spans(npos, rot ? rope_dim : 0) ||
        (pages && (!spans(page, pages_stride) || !spans(n_pages, pages_page_stride))) ||
        (codes && (!spans(page, codes_stride) || !spans(n_pages, codes_page_stride) || !spans(page, scales_stride) ||
                   !spans(n_pages, scales_page_stride))))
        return SA_ERR_INVALID_ARG;
    const int64_t cw = quant == SA_KV_FP4_E2M1 ? d / 2 : d, sw = d / 32, r1 = page - 1, g1 = n_pages - 1;
    const int64_t p1 = r1 * pages_stride + d, c1 = r1 * codes_stride + cw, s1 = r1 * scales_stride + sw;  // a page's
    if (pages && (!aligned(pages, 2) || pages_stride < d || (n_pages > 1 && pages_page_stride < p1)))
        return SA_ERR_INVALID_ARG;
    if (codes && (codes_stride < cw || (n_pages > 1 && codes_page_stride < c1) || scales_stride < sw ||
                  (n_pages > 1 && scales_page_stride < s1)))
        return SA_ERR_INVALID_ARG;
    const struct {
        const void* at;
        int64_t bytes;
        bool written;
    } t[] = {{pages, 2 * (g1 * pages_page_stride + p1), true},
             {codes, g1 * codes_page_stride + c1, true},
             {scales, g1 * scales_page_stride + s1, true},
             {status, 4, true},
             {x, 2 * ((n - 1) * x_stride + d), false},
             {weight, 4 * (int64_t)d, false},
             {rot, 4 * npos * rope_dim, false},
             {q_start, 4 * (b + 1), false},
             {kv_len, 4 * b, false},
             {page_table, 4 * ((b - 1) * table_stride + max_pages), false}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 10; ++j)
            if (j >= 3 && overlap(t[i].at, t[i].bytes, t[j].at, t[j].bytes)) return SA_ERR_INVALID_ARG;
    const Pool pools[] = {{pages, 2 * (int64_t)d, 2 * pages_stride, 2 * pages_page_stride},
                          {codes, cw, codes_stride, codes_page_stride},
                          {scales, sw, scales_stride, scales_page_stride}};
    if (pools_overlap(pools[0], pools[1], n_pages, page) || pools_overlap(pools[0], pools[2], n_pages, page) ||
        pools_overlap(pools[1], pools[2], n_pages, page))
        return SA_ERR_INVALID_ARG;
    Write p = {};
    p.x = reinterpret_cast<const __nv_bfloat16*>(x);
    p.xs = x_stride;
    p.n = n;
    p.d = d;
    p.a = {page_table, max_pages, table_stride, b, n_pages, q_start, kv_len, page};
    p.pages = reinterpret_cast<__nv_bfloat16*>(pages);
    p.ps = pages_stride;
    p.pp = pages_page_stride;
    p.codes = codes;
    p.cs = codes_stride;
    p.cp = codes_page_stride;
    p.scales = scales;
    p.ss = scales_stride;
    p.sp = scales_page_stride;
    p.weight = weight;
    if (weight) p.of = rms_of(d, eps);
    p.rot = rot;
    p.npos = npos;
    p.rope_dim = rot ? rope_dim : 0;
    p.status = reinterpret_cast<uint32_t*>(status);
    const int ca = quant == SA_KV_FP4_E2M1 ? 4 : 8;
    const bool vec = aligned(x, 16) && x_stride % 8 == 0 &&
                     (!pages || (aligned(pages, 16) && pages_stride % 8 == 0 && pages_page_stride % 8 == 0)) &&
                     (!codes || (aligned(codes, ca) && codes_stride % ca == 0 && codes_page_stride % ca == 0));
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = quant == SA_KV_BF16       ? write_launch<SA_KV_BF16>(p, vec, st)
                          : quant == SA_KV_FP8_E4M3 ? write_launch<SA_KV_FP8_E4M3>(p, vec, st)
                                                    : write_launch<SA_KV_FP4_E2M1>(p, vec, st);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

extern "C" size_t sa_window_attn_workspace_size(int64_t n, int64_t b, int h, int d, int64_t window, int64_t first,
                                                int page, int kv_format) {
    using namespace sa;
    if (!kv_format_known(kv_format) || !window_shape(n, b, h, d, window, first, page) || !window_supported(n, h, d))
        return 0;
    if (n < 1) n = 1;
    if (window_tc_supports(d, kv_format, page))
        return SA_STATUS_BYTES + align_up(window_tc_scratch_bound(n, h, window, first), 256);
    const int topk = (int)(first + window);
    const size_t scratch = routed_family(SA_FAMILY_AUTO, h, d, kv_format, 1, 0) == SA_FAMILY_TCGEN05
                               ? attn_tc_scratch_bound(n, h, topk)
                               : attn_mma_scratch_bound(n, h, d, topk);
    return align_up(SA_STATUS_BYTES + align_up(scratch, 256), 256) + align_up((size_t)n * topk * sizeof(int32_t), 256) +
           align_up((size_t)n * sizeof(int32_t), 256);
}

extern "C" sa_status sa_window_attn(const void* q, const void* kv, const uint8_t* kv_scale, int kv_format,
                                    const float* sink, const int32_t* page_table, int64_t max_pages,
                                    int64_t table_stride, const int32_t* q_start, const int32_t* kv_len,
                                    float softmax_scale, int64_t n, int64_t b, int h, int d, int64_t n_pages,
                                    int page, int64_t window, int64_t first, void* o, float* lse, const float* rot,
                                    int64_t npos, int rope_dim, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    using namespace sa;
    if (!kv_format_known(kv_format) || !window_shape(n, b, h, d, window, first, page) || n_pages < 0 || max_pages < 0)
        return SA_ERR_INVALID_ARG;
    if (!window_supported(n, h, d) || n_pages >= k31 || n_pages * page >= k31 || max_pages >= k31 || b >= k31)
        return SA_ERR_UNSUPPORTED;
    if (kv_format == SA_KV_BF16 && kv_scale) return SA_ERR_INVALID_ARG;
    if (rot && (rope_dim < 2 || rope_dim % 2 != 0 || rope_dim > d || npos < 1)) return SA_ERR_INVALID_ARG;
    const bool tc = attn_tc_supports(h, d, kv_format, 1, 0);
    if (rot && !tc) return SA_ERR_UNSUPPORTED;
    // (the pair kernel's roles wait at most some two seconds for one another, for a task's positions too: 2^24 of them
    // take half of one)
    if (window_tc_supports(d, kv_format, page) && std::min(first + window, max_pages * page) > (int64_t(1) << 24))
        return SA_ERR_UNSUPPORTED;
    if (n == 0 || b == 0) return SA_OK;
    const bool codes = kv_format != SA_KV_BF16;
    if (!q || !sink || !o || !q_start || !kv_len || (max_pages > 0 && !page_table)) return SA_ERR_INVALID_ARG;
    if (n_pages < 1 || !kv || (codes && !kv_scale)) return SA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(o, 16) || !aligned(sink, 4) || !aligned(lse, 4) ||
        !aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(rot, 8) ||
        !aligned(kv_scale, tc ? 16 : 4) || (window_tc_supports(d, kv_format, page) && !aligned(o, 32)) ||
        (b > 1 && table_stride < max_pages) || !spans(b, table_stride) || !spans(npos, rot ? rope_dim : 0))
        return SA_ERR_INVALID_ARG;
    const Parts parts = parts_of(n, b, h, d, reach_of(window, first, max_pages, page), page, kv_format);
    const int64_t ob = 2 * n * h * d, rows = n_pages * page;
    const struct {
        const void* at;
        int64_t bytes;
    } t[] = {{o, ob},
             {lse, 4 * n * h},
             {workspace, (int64_t)parts.all},
             {q, ob},
             {kv, rows * kv_row_bytes(kv_format, d)},
             {kv_scale, rows * (d / 32)},
             {sink, 4 * (int64_t)h},
             {rot, 4 * npos * rope_dim},
             {q_start, 4 * (b + 1)},
             {kv_len, 4 * b},
             {page_table, 4 * ((b - 1) * table_stride + max_pages)}};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 11; ++j)
            if (j != 2 && overlap(t[i].at, t[i].bytes, t[j].at, t[j].bytes)) return SA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < parts.all) return SA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SA_ERR_INVALID_ARG;
    for (int j = 0; j < 11; ++j)
        if (j != 2 && overlap(t[2].at, t[2].bytes, t[j].at, t[j].bytes)) return SA_ERR_INVALID_ARG;

    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    const Batch a = {page_table, max_pages, table_stride, b, n_pages, q_start, kv_len, page};
    if (window_tc_supports(d, kv_format, page)) {
        WindowCall c;
        c.q = q;
        c.kv = kv;
        c.kv_scale = kv_scale;
        c.kv_format = kv_format;
        c.sink = sink;
        c.a = a;
        c.softmax_scale = softmax_scale;
        c.n = n;
        c.h = h;
        c.window = window;
        c.first = first;
        c.o = o;
        c.lse = lse;
        c.rope = rot;
        c.npos = npos;
        c.rope_dim = rope_dim;
        c.status = reinterpret_cast<uint32_t*>(ws);
        c.scratch = ws + SA_STATUS_BYTES;
        c.stream = st;
        return window_tc_launch(c) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
    }
    int32_t* idx = reinterpret_cast<int32_t*>(ws + parts.idx);
    int32_t* pos = rot ? reinterpret_cast<int32_t*>(ws + parts.pos) : nullptr;
    // no more entries than the table has positions: 116 tokens of 100 heads over some 60 e4m3 rows of 256 take 38 us, 158 with
    // all entries of a window of 1133
    const int topk = parts.topk, lead = topk < first + window ? topk : (int)first;
    const int cols = (topk + 511) / 512 < 64 ? (topk + 511) / 512 : 64;
    cudaError_t e = launch_pdl(window_rows_kernel, dim3((unsigned)n, cols), dim3(128), 0, st, a, n, (int)window,
                               (int)first, lead, topk, idx, pos, npos, reinterpret_cast<uint32_t*>(ws));
    if (e != cudaSuccess) return SA_ERR_CUDA;
    AttnCall c;
    c.q = q;
    c.kv = kv;
    c.kv_scale = kv_scale;
    c.kv_format = kv_format;
    c.sink = sink;
    c.idx = idx;
    c.softmax_scale = softmax_scale;
    c.b = 1;
    c.s = n;
    c.h = h;
    c.d = d;
    c.rows = rows;
    c.topk = topk;
    c.o = o;
    c.status = reinterpret_cast<uint32_t*>(ws);
    c.scratch = ws + SA_STATUS_BYTES;
    c.scratch_bytes = parts.idx - SA_STATUS_BYTES;
    c.stream = st;
    c.rope = rot;
    c.rope_dim = rot ? rope_dim : 0;
    c.rope_at = pos;
    c.n_live = q_start + b;
    c.lse = lse;
    e = tc ? attn_tc_launch(c) : attn_mma_launch(c);
    return e == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
