// skv_pages.cpp -- the paged-cache part of the C ABI declared in include/skv.h.
//
// Host side: argument checks (everything that depends on sizes, strides and
// alignment is settled here, so a launch never finds an array smaller than
// its indexes; what depends on device data is checked by the kernels) and the
// launches on the caller's stream.  Nothing here allocates or throws.
#include "skv_pages.h"

namespace {

constexpr uint64_t kMaxSlots = 0x7fffffffull;
constexpr uint64_t kMaxLength = 1ull << 30;      // of a request in attention: key indexes keep room above it
constexpr uint32_t kMaxPlanRequests = 4096;
constexpr uint32_t kMaxRequests = 65535;
constexpr uint32_t kMaxGroup = 64;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// A stride keeps 16-byte alignment; that of a dimension of one element is never used.
bool stride16(int64_t elements, uint32_t eb, uint32_t size) { return size <= 1 || (elements * int64_t(eb)) % 16 == 0; }

int shift_of(uint32_t page_tokens) {
    if (page_tokens < 8 || page_tokens > 1024 || (page_tokens & (page_tokens - 1))) return -1;
    return __builtin_ctz(page_tokens);
}

// The pool's description: sizes, then strides and alignment.
int check_pages(const skv_pages* pg, const void* k, const void* v) {
    if (!pg || !k || !v) return SKV_ERR_ARG;
    if (pg->abi_version != SKV_ABI_VERSION || (pg->dtype != SKV_BF16 && pg->dtype != SKV_E4M3) ||
        shift_of(pg->page_tokens) < 0 || pg->layers == 0 || pg->layers > 4096 || pg->pages == 0 || pg->heads == 0 ||
        pg->head_dim == 0 || pg->head_dim % 16 != 0 || uint64_t(pg->heads) * pg->head_dim > 65536 ||
        uint64_t(pg->pages) * pg->page_tokens > kMaxSlots)
        return SKV_ERR_SHAPE;
    const uint32_t eb = skv::elem_bytes(pg->dtype);
    if (!aligned16(k) || !aligned16(v) || !stride16(pg->page_stride, eb, pg->pages) ||
        !stride16(pg->token_stride, eb, pg->page_tokens) || !stride16(pg->head_stride, eb, pg->heads) ||
        !stride16(pg->layer_stride, eb, pg->layers))
        return SKV_ERR_ARG;
    return SKV_OK;
}

int page_rows(const skv_pages* pg, void* k_pages, void* v_pages, const skv_rows* rows, void* k, void* v,
              const int32_t* slots, const float* k_scale, const float* v_scale, uint32_t* status, hipStream_t stream,
              bool to_pages) {
    const int rc = check_pages(pg, k_pages, v_pages);
    if (rc != SKV_OK) return rc;
    if (!rows) return SKV_ERR_ARG;
    // copies, or bf16 rows of a scaled e4m3 pool
    if (rows->dtype != pg->dtype && !(rows->dtype == SKV_BF16 && pg->dtype == SKV_E4M3)) return SKV_ERR_SHAPE;
    if (rows->tokens > kMaxSlots) return SKV_ERR_SHAPE;
    if (rows->dtype == pg->dtype && (k_scale || v_scale)) return SKV_ERR_ARG;
    if (rows->tokens == 0) return SKV_OK;
    if (!k || !v || !slots) return SKV_ERR_ARG;
    const uint32_t eb = skv::elem_bytes(rows->dtype);
    if (!aligned16(k) || !aligned16(v) || !stride16(rows->token_stride, eb, rows->tokens) ||
        !stride16(rows->head_stride, eb, pg->heads) || !stride16(rows->layer_stride, eb, pg->layers))
        return SKV_ERR_ARG;
    skv::RowsLaunch a{};
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k = k;
    a.v = v;
    a.slots = slots;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.status = status;
    a.page_layer = pg->layer_stride;
    a.page_page = pg->page_stride;
    a.page_token = pg->token_stride;
    a.page_head = pg->head_stride;
    a.row_layer = rows->layer_stride;
    a.row_token = rows->token_stride;
    a.row_head = rows->head_stride;
    a.layers = pg->layers;
    a.tokens = rows->tokens;
    a.heads = pg->heads;
    a.head_dim = pg->head_dim;
    a.page_shift = uint32_t(shift_of(pg->page_tokens));
    a.n_slots = pg->pages * pg->page_tokens;
    a.rows_dtype = rows->dtype;
    a.pages_dtype = pg->dtype;
    a.to_pages = to_pages;
    return skv::launch_rows(a, stream) == hipSuccess ? SKV_OK : SKV_ERR_DEVICE;
}

}  // namespace

extern "C" {

int skv_page_plan(const int32_t* d_lens, const int32_t* d_new, uint32_t requests, int32_t* d_table, uint32_t width,
                  int64_t table_stride, const int32_t* d_free, uint32_t free_pages, uint32_t page_tokens,
                  uint32_t tokens, int32_t* d_slots, int32_t* d_positions, int32_t* d_starts, int32_t* d_taken,
                  uint32_t* d_status, hipStream_t stream) {
    if (!d_lens || !d_new || !d_table || !d_starts || !d_taken) return SKV_ERR_ARG;
    if (tokens && (!d_slots || !d_positions)) return SKV_ERR_ARG;
    const int shift = shift_of(page_tokens);
    if (shift < 0 || requests == 0 || requests > kMaxPlanRequests || width == 0 ||
        uint64_t(width) * page_tokens > kMaxSlots || tokens > kMaxSlots || free_pages > kMaxSlots)
        return SKV_ERR_SHAPE;
    if (requests > 1 && table_stride < int64_t(width)) return SKV_ERR_ARG;
    skv::PlanLaunch a{};
    a.lens = d_lens;
    a.fresh = d_new;
    a.table = d_table;
    a.free_list = d_free;
    a.slots = d_slots;
    a.positions = d_positions;
    a.starts = d_starts;
    a.taken = d_taken;
    a.status = d_status;
    a.table_stride = table_stride;
    a.requests = requests;
    a.width = width;
    a.free_pages = d_free ? free_pages : 0;
    a.page_shift = uint32_t(shift);
    a.tokens = tokens;
    return skv::launch_plan(a, stream) == hipSuccess ? SKV_OK : SKV_ERR_DEVICE;
}

int skv_page_write(const skv_pages* pages, void* d_k_pages, void* d_v_pages, const skv_rows* rows, const void* d_k,
                   const void* d_v, const int32_t* d_slots, const float* d_k_scale, const float* d_v_scale,
                   uint32_t* d_status, hipStream_t stream) {
    return page_rows(pages, d_k_pages, d_v_pages, rows, const_cast<void*>(d_k), const_cast<void*>(d_v), d_slots,
                     d_k_scale, d_v_scale, d_status, stream, true);
}

int skv_page_read(const skv_pages* pages, const void* d_k_pages, const void* d_v_pages, const skv_rows* rows,
                  void* d_k, void* d_v, const int32_t* d_slots, const float* d_k_scale, const float* d_v_scale,
                  uint32_t* d_status, hipStream_t stream) {
    return page_rows(pages, const_cast<void*>(d_k_pages), const_cast<void*>(d_v_pages), rows, d_k, d_v, d_slots,
                     d_k_scale, d_v_scale, d_status, stream, false);
}

int skv_page_attention(const skv_pages* pages, const skv_attention* a, void* d_work, size_t* work_bytes,
                       hipStream_t stream) {
    if (!a || !work_bytes) return SKV_ERR_ARG;
    int rc = check_pages(pages, a->k_pages, a->v_pages);
    if (rc != SKV_OK) return rc;
    if (a->abi_version != SKV_ABI_VERSION || pages->layers != 1 ||
        (pages->head_dim != 64 && pages->head_dim != 128 && pages->head_dim != 256))
        return SKV_ERR_SHAPE;
    if (a->requests == 0 || a->requests > kMaxRequests || a->width == 0 || a->q_heads == 0 ||
        a->q_heads % pages->heads != 0 || a->q_heads / pages->heads > kMaxGroup ||
        uint64_t(a->tokens) * a->q_heads > kMaxSlots || uint64_t(a->width) * pages->page_tokens > kMaxLength)
        return SKV_ERR_SHAPE;
    if (a->causal > 1 || !(a->scale == a->scale)) return SKV_ERR_ARG;
    if (!a->starts && a->tokens != a->requests) return SKV_ERR_ARG;
    if (pages->dtype == SKV_BF16 && (a->k_scale || a->v_scale)) return SKV_ERR_ARG;
    if (a->requests > 1 && a->table_stride < int64_t(a->width)) return SKV_ERR_ARG;
    if (!a->table || !a->lens) return SKV_ERR_ARG;
    if (a->tokens && (!a->q || !a->out)) return SKV_ERR_ARG;
    if (!aligned16(a->q) || !aligned16(a->out) || !stride16(a->q_token_stride, 2, a->tokens) ||
        !stride16(a->q_head_stride, 2, a->q_heads) || !stride16(a->out_token_stride, 2, a->tokens) ||
        !stride16(a->out_head_stride, 2, a->q_heads))
        return SKV_ERR_ARG;
    const uint32_t eb = skv::elem_bytes(pages->dtype);
    skv::AttentionLaunch l{};
    l.q = static_cast<const uint16_t*>(a->q);
    l.k_pages = static_cast<const uint8_t*>(a->k_pages);
    l.v_pages = static_cast<const uint8_t*>(a->v_pages);
    l.table = a->table;
    l.lens = a->lens;
    l.starts = a->starts;
    l.k_scale = a->k_scale;
    l.v_scale = a->v_scale;
    l.out = static_cast<uint16_t*>(a->out);
    l.lse = a->lse;
    l.status = a->status;
    l.page_stride = pages->page_stride * eb;
    l.token_stride = pages->token_stride * eb;
    l.head_stride = pages->head_stride * eb;
    l.table_stride = a->table_stride;
    l.q_token = a->q_token_stride;
    l.q_head = a->q_head_stride;
    l.out_token = a->out_token_stride;
    l.out_head = a->out_head_stride;
    l.requests = a->requests;
    l.tokens = a->tokens;
    l.heads = pages->heads;
    l.group = a->q_heads / pages->heads;
    l.width = a->width;
    l.pages = pages->pages;
    l.page_shift = uint32_t(shift_of(pages->page_tokens));
    l.max_new = a->starts ? a->max_new : 1;
    if (l.max_new > a->tokens) l.max_new = a->tokens;
    l.causal = a->causal;
    l.scale = a->scale;
    const bool few = skv::attention_few_rows(l);
    const uint64_t need = few ? skv::split_work_bytes(pages->head_dim) : skv::tiles_work_bytes(l, pages->head_dim);
    if (!d_work) {
        *work_bytes = need;
        return SKV_OK;
    }
    if (*work_bytes < need) {
        *work_bytes = need;
        return SKV_ERR_CAPACITY;
    }
    if (!aligned16(d_work)) return SKV_ERR_ARG;
    if (a->tokens == 0) return SKV_OK;
    const hipError_t e = few ? skv::launch_split(l, pages->head_dim, pages->dtype, d_work, stream)
                             : skv::launch_tiles(l, pages->head_dim, pages->dtype, d_work, stream);
    return e == hipSuccess ? SKV_OK : SKV_ERR_DEVICE;
}

int skv_page_check(const uint32_t* d_status, uint32_t* flags, hipStream_t stream) {
    if (!d_status) return SKV_ERR_ARG;
    uint32_t word = 0;
    if (hipMemcpyAsync(&word, d_status, sizeof word, hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
        return SKV_ERR_DEVICE;
    if (flags) *flags = word;
    return word ? SKV_ERR_PAGES : SKV_OK;
}

}  // extern "C"
