// skv_pages.hip -- gfx950 kernels of the paged cache's bookkeeping and copies.
//
//   page_plan   a step's block tables, slot maps and positions from request
//               lengths, in one launch
//   page_rows   rows into pages and pages into rows, with or without a change
//               of type
#include <algorithm>

#include "skv_pages.h"

namespace skv {
namespace {

constexpr uint32_t kThreads = 256;

// ------------------------------------------------------------------ plan
// Exclusive sums of new tokens and pages over up to 4096 requests, then one
// binary search per packed row.  Every workgroup computes the sums for
// itself (they are a few KB of reads that stay in L2) and keeps them in LDS,
// so the call is one launch with no exchange between workgroups: a
// workgroup's rows that fall into freshly taken blocks find their page in the
// free list itself, not in the table entry another workgroup writes.

constexpr uint32_t kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;

// The sum saturates at 2^31 - 1; sums of valid requests never get there
// without passing `tokens`, which is flagged.
__device__ __forceinline__ uint32_t cap31(uint64_t x) { return x > 0x7fffffffull ? 0x7fffffffu : uint32_t(x); }

__device__ __forceinline__ PlanRequest request_at(const PlanLaunch& a, uint32_t b) {
    return plan_request(a.lens[b], a.fresh[b], a.width, a.page_shift);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan(PlanLaunch a) {
    extern __shared__ uint32_t lds[];
    uint32_t* s_row = lds;                        // [requests + 1] first packed row of each request
    uint32_t* s_page = lds + a.requests + 1;      // [requests + 1] first taken page
    __shared__ uint64_t s_sum[2][kPlanWaves];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t P = 1u << a.page_shift;
    uint32_t flags = 0;
    uint64_t row0 = 0, page0 = 0;
    for (uint32_t base = 0; base < a.requests; base += kPlanThreads) {
        const uint32_t b = base + tid;
        uint32_t rows = 0, pages = 0;
        if (b < a.requests) {
            const PlanRequest r = request_at(a, b);
            if (r.bad) flags |= SKV_PAGES_LENGTH;
            rows = r.len - r.old;
            if (a.free_list) pages = pages_for(r.len, a.page_shift) - pages_for(r.old, a.page_shift);
        }
        uint64_t x = rows, y = pages;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint64_t u = __shfl_up(x, d), v = __shfl_up(y, d);
            if (lane >= d) {
                x += u;
                y += v;
            }
        }
        if (lane == 63) {
            s_sum[0][wave] = x;
            s_sum[1][wave] = y;
        }
        __syncthreads();
        uint64_t xa = row0, ya = page0;
        for (uint32_t w = 0; w < kPlanWaves; ++w) {
            if (w < wave) {
                xa += s_sum[0][w];
                ya += s_sum[1][w];
            }
            row0 += s_sum[0][w];
            page0 += s_sum[1][w];
        }
        if (b < a.requests) {
            s_row[b] = cap31(xa + x - rows);
            s_page[b] = cap31(ya + y - pages);
        }
        __syncthreads();
    }
    if (tid == 0) {
        s_row[a.requests] = cap31(row0);
        s_page[a.requests] = cap31(page0);
        if (row0 > a.tokens) flags |= SKV_PAGES_ROWS;
        if (a.free_list && page0 > a.free_pages) flags |= SKV_PAGES_FREE;
    }
    __syncthreads();

    const uint32_t g = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
    for (uint32_t b = g; b <= a.requests; b += stride) {
        a.starts[b] = int32_t(min(s_row[b], a.tokens));
        a.taken[b] = int32_t(s_page[b]);
    }
    // the last request whose first entry is at or before e (the ones after it start later)
    auto owner = [&](const uint32_t* first, uint32_t e) {
        uint32_t lo = 0, hi = a.requests;
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) >> 1;
            if (first[mid] <= e) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const uint32_t n_pages = s_page[a.requests];
    for (uint64_t e = g; e < n_pages; e += stride) {
        const uint32_t b = owner(s_page, uint32_t(e));
        const PlanRequest r = request_at(a, b);
        const uint32_t block = pages_for(r.old, a.page_shift) + uint32_t(e) - s_page[b];
        a.table[int64_t(b) * a.table_stride + block] = e < a.free_pages ? a.free_list[e] : -1;
    }
    const uint32_t n_rows = s_row[a.requests];
    for (uint64_t t = g; t < a.tokens; t += stride) {
        int32_t slot = -1, position = -1;
        if (t < n_rows) {
            const uint32_t b = owner(s_row, uint32_t(t));
            const PlanRequest r = request_at(a, b);
            const uint32_t pos = r.old + uint32_t(t) - s_row[b], block = pos >> a.page_shift;
            const uint32_t have = a.free_list ? pages_for(r.old, a.page_shift) : a.width;
            position = int32_t(pos);
            int32_t page;
            bool ended = false;
            if (block >= have) {
                const uint32_t e = s_page[b] + block - have;
                ended = e >= a.free_pages;            // flagged above
                page = ended ? -1 : a.free_list[e];
            } else {
                page = a.table[int64_t(b) * a.table_stride + block];
            }
            slot = slot_of(page, pos & (P - 1), a.page_shift);
            if (slot < 0 && !ended) flags |= SKV_PAGES_PAGE;
        }
        a.slots[t] = slot;
        a.positions[t] = position;
    }
    if (flags && a.status) atomicOr(a.status, flags);
}

// ------------------------------------------------------------------ rows
__device__ __forceinline__ uint32_t bf16_round(float x) {       // to nearest, ties to even; NaN stays one
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// Four values to e4m3 codes: the hardware rounds to nearest even; values
// past +-448 are clamped first, NaN passes through to the NaN code.
__device__ __forceinline__ uint32_t e4m3_pack(float a, float b, float c, float d) {
    auto sat = [](float x) { return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f); };
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), v, true);
    return uint32_t(v);
}

// x / scale, correctly rounded, from the correctly rounded reciprocal r of a
// scale within 2^+-60: one step of x - q scale in exact arithmetic (Markstein),
// three instructions against eleven of a division.  Where the step is not a
// number (x is infinite or NaN) or has lost a zero's sign, the product already
// is what the quotient is.
__device__ __forceinline__ float divided(float x, float scale, float r) {
    const float q = x * r, y = fmaf(fmaf(-q, scale, x), r, q);
    return fabsf(y) > 0.0f ? y : q;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// An item is 16 bytes of a copy, or 16 values where the type changes (32
// bytes of bf16, 16 of e4m3).  x: items of a token's heads, y: layer and K|V.
// Bound by memory.  One item a thread, as many workgroups as it takes: 1.2 GB
// of e4m3 rows out of their pages in 194 us, 6.2 TB/s (four items a thread,
// one after another 222 us, requested together 219); a prompt's 32768 rows of
// 8 heads into e4m3 pages, 0.2 GB, in 34 us (44 where the rows come from
// memory; both 46 with stores that stay in the caches; an attention that reads
// the pages right after takes the same either way).  Rows that keep their type
// are stored the ordinary way: past the caches 32768 of them take 48 us for
// 59, but then the attention after them loses more (8 prompts of 2048 tokens,
// both together, 348 for 344).
struct RowsGeo {
    uint32_t items;              // per token
    uint32_t per_head;           // items per head
    uint32_t magic_items, magic_head;   // ceil(2^32 / d): exact quotients below 2^16
    uint32_t tokens_per_block;
};

__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t d, uint32_t magic) {
    return d == 1 ? n : uint32_t((uint64_t(n) * magic) >> 32);
}

template <bool kToPages, bool kConvert>
__global__ void __launch_bounds__(kThreads) page_rows(RowsLaunch a, RowsGeo g) {
    const uint32_t layer = blockIdx.y >> 1, which = blockIdx.y & 1;
    const uint32_t eb_rows = a.rows_dtype == SKV_E4M3 ? 1 : 2, eb_pages = a.pages_dtype == SKV_E4M3 ? 1 : 2;
    const uint32_t values = kConvert ? 16 : 16 / eb_rows;
    uint8_t* pages = static_cast<uint8_t*>(which ? a.v_pages : a.k_pages) + int64_t(layer) * a.page_layer * eb_pages;
    uint8_t* rows = static_cast<uint8_t*>(which ? a.v : a.k) + int64_t(layer) * a.row_layer * eb_rows;
    const float* scales = which ? a.v_scale : a.k_scale;
    const uint32_t t0 = blockIdx.x * g.tokens_per_block;
    const uint32_t nt = min(g.tokens_per_block, a.tokens - t0);
    const uint32_t P1 = (1u << a.page_shift) - 1;
    uint32_t flags = 0;
    for (uint32_t i = threadIdx.x; i < nt * g.items; i += kThreads) {       // once, but for over 256 items a token
        const uint32_t dt = div_by(i, g.items, g.magic_items), c = i - dt * g.items;
        const uint32_t head = div_by(c, g.per_head, g.magic_head), off = (c - head * g.per_head) * values;
        const uint32_t t = t0 + dt;
        const int32_t slot = a.slots[t];
        const bool fits = uint32_t(slot) < a.n_slots;
        if (slot >= 0 && !fits) flags |= SKV_PAGES_SLOT;
        if (kToPages && !fits) continue;
        const uint32_t in = fits ? uint32_t(slot) : 0;
        uint4* row = reinterpret_cast<uint4*>(rows + (int64_t(t) * a.row_token + int64_t(head) * a.row_head + off) * eb_rows);
        uint4* at = reinterpret_cast<uint4*>(pages + (int64_t(in >> a.page_shift) * a.page_page +
                                                      int64_t(in & P1) * a.page_token + int64_t(head) * a.page_head + off) *
                                                         eb_pages);
        if (!kConvert) {
            uint4 x = kToPages ? *row : *at;          // (slot 0 stands in for none)
            if (!fits) x = uint4{0, 0, 0, 0};
            *(kToPages ? at : row) = x;
        } else if (kToPages) {
            const uint4 lo = row[0], hi = row[1];
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            const float scale = scales ? scales[head] : 1.0f, inv = 1.0f / scale, mag = fabsf(scale);
            uint32_t r[4];
            if (mag > 0x1p-60f && mag < 0x1p60f) {
                for (int e = 0; e < 4; ++e)
                    r[e] = e4m3_pack(divided(bf16_lo(w[2 * e]), scale, inv), divided(bf16_hi(w[2 * e]), scale, inv),
                                     divided(bf16_lo(w[2 * e + 1]), scale, inv), divided(bf16_hi(w[2 * e + 1]), scale, inv));
            } else {
                for (int e = 0; e < 4; ++e)
                    r[e] = e4m3_pack(bf16_lo(w[2 * e]) / scale, bf16_hi(w[2 * e]) / scale, bf16_lo(w[2 * e + 1]) / scale,
                                     bf16_hi(w[2 * e + 1]) / scale);
            }
            using u32x4 = __attribute__((__vector_size__(16))) uint32_t;
            __builtin_nontemporal_store(u32x4{r[0], r[1], r[2], r[3]}, reinterpret_cast<u32x4*>(at));
        } else {
            uint4 x = *at;
            if (!fits) x = uint4{0, 0, 0, 0};
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            const float scale = scales && fits ? scales[head] : 1.0f;          // zeros stay +0 whatever the scale
            uint32_t r[8];
            for (int e = 0; e < 4; ++e) {
                const float f0 = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 0), f1 = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 1);
                const float f2 = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 2), f3 = __builtin_amdgcn_cvt_f32_fp8(int(w[e]), 3);
                r[2 * e] = bf16_round(f0 * scale) | bf16_round(f1 * scale) << 16;
                r[2 * e + 1] = bf16_round(f2 * scale) | bf16_round(f3 * scale) << 16;
            }
            row[0] = uint4{r[0], r[1], r[2], r[3]};
            row[1] = uint4{r[4], r[5], r[6], r[7]};
        }
    }
    if (flags && a.status) atomicOr(a.status, flags);
}

uint32_t magic(uint32_t d) { return uint32_t(((1ull << 32) + d - 1) / d); }

}  // namespace

hipError_t launch_plan(const PlanLaunch& a, hipStream_t stream) {
    const uint64_t work = std::max<uint64_t>({a.tokens, a.requests, a.free_pages ? a.requests : 0});
    const uint32_t blocks = uint32_t(std::min<uint64_t>(std::max<uint64_t>((work + kPlanThreads - 1) / kPlanThreads, 1), 512));
    page_plan<<<blocks, kPlanThreads, 8 * (a.requests + 1), stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_rows(const RowsLaunch& a, hipStream_t stream) {
    const bool convert = a.rows_dtype != a.pages_dtype;
    const uint32_t values = convert ? 16 : 16 / elem_bytes(a.rows_dtype);
    RowsGeo g;
    g.per_head = a.head_dim / values;
    g.items = a.heads * g.per_head;
    g.magic_items = magic(g.items);
    g.magic_head = magic(g.per_head);
    // (2^16 / 8 items at most in a token's row: quotients stay below 2^16)
    g.tokens_per_block = std::max(1u, kThreads / g.items);
    const dim3 grid((a.tokens + g.tokens_per_block - 1) / g.tokens_per_block, 2 * a.layers);
    if (a.to_pages) {
        if (convert) page_rows<true, true><<<grid, kThreads, 0, stream>>>(a, g);
        else page_rows<true, false><<<grid, kThreads, 0, stream>>>(a, g);
    } else {
        if (convert) page_rows<false, true><<<grid, kThreads, 0, stream>>>(a, g);
        else page_rows<false, false><<<grid, kThreads, 0, stream>>>(a, g);
    }
    return hipGetLastError();
}

}  // namespace skv
