/* The index functions of the paged-cache kernels, for calls from Python. */
#include "../../lossless_kv_cache_amd/csrc/skv_pages_index.h"

using namespace skv;

extern "C" {
int plan(int32_t len, int32_t fresh, uint32_t width, uint32_t shift, uint32_t* old, uint32_t* now) {
    const PlanRequest r = plan_request(len, fresh, width, shift);
    *old = r.old;
    *now = r.len;
    return r.bad;
}
uint32_t pages(uint32_t tokens, uint32_t shift) { return pages_for(tokens, shift); }
int32_t slot(int32_t page, uint32_t in, uint32_t shift) { return slot_of(page, in, shift); }
int span(int32_t len, int64_t r0, int64_t r1, uint32_t tokens, uint32_t width, uint32_t shift, uint32_t max_new,
         uint32_t out[3]) {
    Span s;
    const int f = make_span(len, r0, r1, tokens, width, shift, max_new, &s);
    out[0] = s.row;
    out[1] = s.n;
    out[2] = s.len;
    return f;
}
int page(int32_t entry, uint32_t count, uint32_t* out) {
    bool bad = false;
    *out = page_or_zero(entry, count, &bad);
    return bad;
}
}
