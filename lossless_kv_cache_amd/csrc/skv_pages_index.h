// skv_pages_index.h -- what the paged-cache kernels do with lengths, starts,
// table entries and slots before they follow any of them.  Plain integer
// functions, compiled for the kernels and, by the tests, for the host.
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#define SKV_HD __host__ __device__ __forceinline__
#else
#define SKV_HD inline
#endif

namespace skv {

// A request of a plan: tokens before and after the step; 0, 0 and bad where
// the lengths make no sense (new < 0, len < new, or past the table's width).
struct PlanRequest {
    uint32_t old, len;
    bool bad;
};

SKV_HD PlanRequest plan_request(int32_t len, int32_t fresh, uint32_t width, uint32_t page_shift) {
    if (fresh < 0 || len < fresh || int64_t(len) > (int64_t(width) << page_shift)) return PlanRequest{0, 0, true};
    return PlanRequest{uint32_t(len) - uint32_t(fresh), uint32_t(len), false};
}

// Pages a request takes from the free list: ceil(len / P) - ceil(old / P).
SKV_HD uint32_t pages_for(uint32_t tokens, uint32_t page_shift) {
    return uint32_t((uint64_t(tokens) + (1u << page_shift) - 1) >> page_shift);
}

// Slot of offset `in` of a page, or -1 where the page is no id (negative) or
// the slot would pass 2^31 - 1.
SKV_HD int32_t slot_of(int32_t page, uint32_t in, uint32_t page_shift) {
    if (page < 0 || page > int32_t(0x7fffffffu >> page_shift) - 1) return -1;
    return int32_t((uint32_t(page) << page_shift) | in);
}

// A request's queries: packed rows [row, row + n) of the batch's `tokens`,
// and its length; n = 0 where lengths or starts make no sense.
struct Span {
    uint32_t row, n, len;
};

enum SpanFault { kSpanFine = 0, kSpanLength = 1, kSpanRows = 2 };

SKV_HD SpanFault make_span(int32_t len, int64_t r0, int64_t r1, uint32_t tokens, uint32_t width, uint32_t page_shift,
                           uint32_t max_new, Span* s) {
    *s = Span{0, 0, 0};
    if (len < 0 || int64_t(len) > (int64_t(width) << page_shift) || r0 < 0 || r1 < r0 || r1 > int64_t(tokens))
        return kSpanLength;
    if (r1 - r0 > int64_t(max_new)) return kSpanRows;
    *s = Span{uint32_t(r0), uint32_t(r1 - r0), uint32_t(len)};
    return kSpanFine;
}

// The page a table entry names; page 0 (and *bad) where it names none.
SKV_HD uint32_t page_or_zero(int32_t entry, uint32_t pages, bool* bad) {
    if (uint32_t(entry) < pages) return uint32_t(entry);
    *bad = true;
    return 0;
}

}  // namespace skv
