// skv_attention.hip -- attention of new tokens over a paged cache (gfx950).
//
// s_j = scale q.k_j over the keys a query sees, m = max s, l = sum exp(s - m),
// out = sum exp(s - m) v / l, lse = m + log l; in one pass over the keys with
// a running m and l, o and l rescaled by exp(m_old - m_new) when m grows.
#include "skv_pages.h"

namespace skv {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float bf16_f32(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ uint32_t bf16_of(float x) {       // to nearest, ties to even; NaN stays one
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ Span span_of(const AttentionLaunch& a, uint32_t b, uint32_t& flags) {
    Span s;
    const SpanFault f = make_span(a.lens[b], a.starts ? a.starts[b] : int64_t(b),
                                  a.starts ? a.starts[b + 1] : int64_t(b) + 1, a.tokens, a.width, a.page_shift,
                                  a.max_new, &s);
    if (f) flags |= f == kSpanLength ? SKV_PAGES_LENGTH : SKV_PAGES_ROWS;
    return s;
}

// Byte offset of token j of request b in the pool (its first head).
__device__ __forceinline__ int64_t token_at(const AttentionLaunch& a, uint32_t b, uint32_t j, uint32_t& flags) {
    bool bad = false;
    const uint32_t page = page_or_zero(a.table[int64_t(b) * a.table_stride + (j >> a.page_shift)], a.pages, &bad);
    if (bad) flags |= SKV_PAGES_PAGE;
    return int64_t(page) * a.page_stride + int64_t(j & ((1u << a.page_shift) - 1)) * a.token_stride;
}

// One query row by one wavefront, key after key, D / 64 of the head's values
// in each lane: the definition in 32 bits.
template <int D, bool kE4m3>
__device__ __forceinline__ void row_plain(const AttentionLaunch& a, uint32_t b, const Span& s, uint32_t i,
                                          uint32_t head, uint32_t& flags) {
    constexpr int V = D / 64;
    const uint32_t lane = threadIdx.x & 63, kv = head / a.group;
    const int64_t qo = int64_t(s.row + i) * a.q_token + int64_t(head) * a.q_head + lane * V;
    float q[V], o[V];
    for (int e = 0; e < V; ++e) {
        q[e] = bf16_f32(a.q[qo + e]);
        o[e] = 0.0f;
    }
    const float ks = a.scale * (a.k_scale ? a.k_scale[kv] : 1.0f), vs = a.v_scale ? a.v_scale[kv] : 1.0f;
    const int64_t last = a.causal ? int64_t(s.len) - s.n + i : int64_t(s.len) - 1;
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j <= last; ++j) {
        const int64_t at = token_at(a, b, uint32_t(j), flags) + int64_t(kv) * a.head_stride + lane * V * (kE4m3 ? 1 : 2);
        float k[V], v[V], dot = 0.0f;
        for (int e = 0; e < V; ++e) {
            if (kE4m3) {
                k[e] = __builtin_amdgcn_cvt_f32_fp8(a.k_pages[at + e], 0);
                v[e] = __builtin_amdgcn_cvt_f32_fp8(a.v_pages[at + e], 0);
            } else {
                k[e] = bf16_f32(reinterpret_cast<const uint16_t*>(a.k_pages + at)[e]);
                v[e] = bf16_f32(reinterpret_cast<const uint16_t*>(a.v_pages + at)[e]);
            }
            dot += q[e] * k[e];
        }
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
        const float x = dot * ks, top = fmaxf(m, x);
        // -infinity stands for "nothing yet": it must not meet itself in a difference
        const float ref = top == -INFINITY ? 0.0f : top;
        const float keep = __builtin_amdgcn_exp2f((m - ref) * kLog2e);
        const float p = x != x ? x : __builtin_amdgcn_exp2f((x - ref) * kLog2e);
        l = l * keep + p;
        for (int e = 0; e < V; ++e) o[e] = o[e] * keep + p * v[e];
        m = top;
    }
    const int64_t oo = int64_t(s.row + i) * a.out_token + int64_t(head) * a.out_head + lane * V;
    for (int e = 0; e < V; ++e) a.out[oo + e] = uint16_t(bf16_of(last < 0 ? 0.0f : o[e] / l * vs));
    if (a.lse && lane == 0) a.lse[uint64_t(s.row + i) * a.heads * a.group + head] = last < 0 ? -INFINITY : m + __logf(l);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) attention_rows(AttentionLaunch a) {
    const uint32_t head = blockIdx.y, b = blockIdx.z, i = blockIdx.x * 4 + (threadIdx.x >> 6);
    uint32_t flags = 0;
    const Span s = span_of(a, b, flags);
    if (i < s.n) row_plain<D, kE4m3>(a, b, s, i, head, flags);
    if (flags && a.status) atomicOr(a.status, flags);
}

template <int D, bool kE4m3>
hipError_t launch_rows_kernel(const AttentionLaunch& a, hipStream_t stream) {
    const dim3 grid((a.max_new + 3) / 4, a.heads * a.group, a.requests);
    attention_rows<D, kE4m3><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

uint64_t attention_work_bytes(const AttentionLaunch&, uint32_t) { return 256; }

hipError_t launch_attention(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void*, hipStream_t stream) {
    const bool e4m3 = dtype == SKV_E4M3;
    switch (head_dim) {
        case 64: return e4m3 ? launch_rows_kernel<64, true>(a, stream) : launch_rows_kernel<64, false>(a, stream);
        case 128: return e4m3 ? launch_rows_kernel<128, true>(a, stream) : launch_rows_kernel<128, false>(a, stream);
        default: return e4m3 ? launch_rows_kernel<256, true>(a, stream) : launch_rows_kernel<256, false>(a, stream);
    }
}

}  // namespace skv
