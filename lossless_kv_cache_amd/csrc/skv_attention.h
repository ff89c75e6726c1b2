// skv_attention.h -- what the attention kernels share (gfx950 device code).
//
// s_j = scale q.k_j over the keys a query sees, m = max s, l = sum exp(s - m),
// out = sum exp(s - m) v / l, lse = m + log l; in one pass over the keys with
// a running m and l, o and l rescaled by exp(m_old - m_new) when m grows.
#pragma once

#include <algorithm>

#include "skv_pages.h"

namespace skv {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

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

// ------------------------------------------------------------------ tiles
// Products run on 32x32x16 bf16 MFMA.  Scores are computed transposed, S^T =
// K Q^T: A = 32 keys x 16 dims, B = 16 dims x 32 query rows, so each lane
// owns one query row (lane % 32) and 16 of a tile's 32 keys, keys
//   8 (r / 4) + 4 (lane / 32) + r % 4        (accumulator register r)
// and row maxima and sums need one exchange between the two half-waves.  The
// probabilities then are, in place, the B operand of O^T = V^T P^T when V's
// keys are taken in the same order: the lane's 8 keys of k-step s are
// registers 8 (s % 2) .. of tile s / 2.  V^T comes from the row-major tile in
// LDS through the transposing LDS reads.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

#define SKV_LDS(T) __attribute__((address_space(3))) T*

// Geometry of tiles of head_dim D in LDS: rows of kRow bytes, 16-byte chunk c
// of row r kept at chunk c ^ swizzle(r), so that the lanes that read LDS in
// one cycle (16 of 16 bytes for K, 32 of 8 bytes for V) meet different banks.
template <int D, bool kE4m3>
struct Tile {
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);        // bytes
    static constexpr int kChunks = kRow / 16;
    static constexpr int kPer256 = kRow >= 256 ? 1 : 256 / kRow;
    static constexpr int kRowsPerLoad = 1024 / kRow;        // rows that a wave's 16-byte load covers
    __device__ static uint32_t swizzle_k(uint32_t r) { return (r / kPer256) & (kChunks < 16 ? kChunks - 1 : 15); }
    __device__ static uint32_t swizzle_v(uint32_t r) {
        if (!kE4m3) return kRow >= 256 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
        if (kRow >= 256) return (r & 3) << 1 | (r & 8);
        if (kRow == 128) return ((r >> 1) & 1) << 1 | ((r >> 1) & 4);
        return (r >> 2) & 2;
    }
};

// A value that is the same in every lane, where the compiler can see that it is.
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return uint64_t(__builtin_amdgcn_readfirstlane(uint32_t(x >> 32))) << 32 |
           uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(x)));
}

// Quotients of 64-bit numbers that mostly fit 32 bits, where a division is a third as long.
__device__ __forceinline__ uint64_t quotient(uint64_t x, uint64_t y) {
    return (x | y) >> 32 ? x / y : uint32_t(x) / uint32_t(y);
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((SKV_LDS(const void))p));
}

// 16 bytes per lane from global memory to LDS at `lds` + 16 * lane, without
// passing through registers.  The wave waits for it itself (wait_loads).
// Written as assembly because the compiler would make every later LDS read
// wait for every such load; no register is written, so nothing can be reused
// too early.
//
// kOnce: what is read once and by one workgroup goes past the caches'
// replacement (nt), which one that several workgroups read must not.
template <bool kOnce = false>
__device__ __forceinline__ void load_lds16(const uint8_t* g, uint32_t lds) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds);
    if constexpr (kOnce)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(to), "v"(g) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(g) : "memory");
}
// The same from a base that is the same for the wave and a byte offset per lane.
template <bool kOnce = false>
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t offset, uint32_t lds) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds);
    if constexpr (kOnce)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(to), "v"(offset), "s"(base)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base)
                     : "memory");
}
// Every load above has landed and every LDS read before has its data.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

// Eight e4m3 codes to bf16 (exact: 4 significant bits into 8).
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return u.v;
}

// LDS addresses of a lane's operands.  A swizzled chunk index is an exclusive
// or, and the row offsets used (multiples of 16 and 32) do not change the
// swizzle, so one base per lane and exclusive ors with constants give every
// address, with tile, row and stage as constant offsets.
//
// K's A operand for k-steps 2p, 2p + 1 of 32 keys.  bf16: two 16-byte reads,
// the lane's half h holds dims 16s + 8h..; e4m3: one 16-byte read, dims 32p +
// 16h .. + 15, the first 8 for step 2p (Q is loaded to match, see load_q).
template <int D, bool kE4m3>
__device__ __forceinline__ uint32_t base_k(uint32_t lane) {
    using T = Tile<D, kE4m3>;
    const uint32_t r = lane & 31, h = lane >> 5;
    return r * T::kRow + ((h ^ T::swizzle_k(r)) << 4);
}

template <int D, bool kE4m3>
__device__ __forceinline__ void read_k(uint32_t base, uint32_t offset, int p, bf16x8 (&k)[2]) {
    if constexpr (!kE4m3) {
        for (int i = 0; i < 2; ++i)
            k[i] = *reinterpret_cast<SKV_LDS(const bf16x8)>((base ^ uint32_t(64 * p + 32 * i)) + offset);
    } else {
        const u32x4 x = *reinterpret_cast<SKV_LDS(const u32x4)>((base ^ uint32_t(32 * p)) + offset);
        k[0] = widen(x[0], x[1]);
        k[1] = widen(x[2], x[3]);
    }
}

// V^T's A operand: dims 32 dt + lane % 32, the 8 keys of the lane's half of
// 16 keys (see above for their order).  The transposing reads give 16 lanes
// the columns of a matrix of 4 rows x 16 (16-bit) or 8 x 16 (8-bit) whose
// rows 4 or 2 neighbouring lanes address.
template <int D, bool kE4m3>
__device__ __forceinline__ uint32_t base_v(uint32_t lane) {
    using T = Tile<D, kE4m3>;
    const uint32_t h = lane >> 5, side = (lane >> 4) & 1, i = lane & 15;
    if constexpr (!kE4m3) {
        const uint32_t r = 4 * h + (i >> 2);
        return r * T::kRow + (((2 * side + ((i & 3) >> 1)) ^ T::swizzle_v(r)) << 4) + 8 * (i & 1);
    } else {
        const uint32_t j = i >> 1, r = 4 * h + (j & 3) + 2 * (j & 4);
        return r * T::kRow + ((side ^ T::swizzle_v(r)) << 4) + 8 * (i & 1);
    }
}

template <int D, bool kE4m3>
__device__ __forceinline__ bf16x8 read_v(uint32_t base, uint32_t offset, int dt) {
    if constexpr (!kE4m3) {
        union {
            s16x4 q[2];
            bf16x8 v;
        } u;
        for (int e = 0; e < 2; ++e)
            u.q[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<SKV_LDS(s16x4)>(
                (base ^ uint32_t(64 * dt)) + offset + 8 * e * Tile<D, kE4m3>::kRow));
        return u.v;
    } else {
        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            reinterpret_cast<SKV_LDS(i32x2)>((base ^ uint32_t(32 * dt)) + offset));
        return widen(uint32_t(x[0]), uint32_t(x[1]));
    }
}

// Q^T's B operand for one query row per lane; zero where there is none.  A
// negative scale is folded into Q's sign (exact), a zero one into Q itself,
// so the kernels see a positive factor.
template <int D, bool kE4m3>
__device__ __forceinline__ void load_q(const uint16_t* row, bool have, float factor, uint32_t lane, bf16x8 (&q)[D / 16]) {
    const uint32_t h = lane >> 5, flip = factor < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        union {
            u32x4 w;
            bf16x8 v;
        } u;
        u.w = u32x4{0, 0, 0, 0};
        const uint32_t dim = kE4m3 ? 32 * (s >> 1) + 16 * h + 8 * (s & 1) : 16 * s + 8 * h;
        if (have && factor != 0.0f) u.w = *reinterpret_cast<const u32x4*>(row + dim);
        u.w ^= flip;
        q[s] = u.v;
    }
}

__device__ __forceinline__ float half_max(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// A wave's running state for 32 query rows: m in units of the raw scores.
template <int D>
struct Rows {
    f32x16 o[D / 32];
    float m, l;
    __device__ void clear() {
        for (auto& t : o)
            for (int r = 0; r < 16; ++r) t[r] = 0.0f;
        m = -INFINITY;
        l = 0.0f;
    }
};

__device__ __forceinline__ float exp2_diff(float m, float top) {      // exp2(m - top), 0 for "nothing"
    return m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
}

// Four values of a finished row to memory; true if one is NaN.
__device__ __forceinline__ bool store_out(const AttentionLaunch& a, uint64_t row, uint32_t head, uint32_t dim, f32x4 x) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x2 w;
    w[0] = bf16_of(x[0]) | bf16_of(x[1]) << 16;
    w[1] = bf16_of(x[2]) | bf16_of(x[3]) << 16;
    *reinterpret_cast<u32x2*>(a.out + int64_t(row) * a.out_token + int64_t(head) * a.out_head + dim) = w;
    return x[0] != x[0] || x[1] != x[1] || x[2] != x[2] || x[3] != x[3];
}

__device__ __forceinline__ void store_lse(const AttentionLaunch& a, uint64_t row, uint32_t head, float m, float l) {
    if (a.lse) a.lse[row * (uint64_t(a.heads) * a.group) + head] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Partial sums (m in base-2 units, l, o), joined in order.
struct Joined {
    float m, l;
    f32x4 o;
};

// The next at most N of them: their loads are in flight together.
template <uint32_t N, int D, class Slot>
__device__ __forceinline__ void join_some(Joined& j, uint32_t p, uint32_t to, uint32_t rows, uint32_t r, uint32_t f,
                                          Slot slot_of) {
    float m[N], l[N];
    f32x4 o[N];
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const float* slot = slot_of(min(p + i, to - 1));
        m[i] = slot[rows * D + r];
        l[i] = slot[rows * (D + 1) + r];
        o[i] = *reinterpret_cast<const f32x4*>(slot + r * D + 4 * f);
    }
    float top = j.m;
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        if (p + i >= to) m[i] = -INFINITY;
        top = fmaxf(top, m[i]);
    }
    const float keep = exp2_diff(j.m, top);
    j.l *= keep;
    j.o *= keep;
    j.m = top;
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const float k = exp2_diff(m[i], top);
        j.l += k * l[i];
        if (m[i] != -INFINITY) j.o += k * o[i];    // else all its keys were hidden, and o may be 0 * NaN
    }
}

// Sixteen at a time, and fewer where few are left, since a place that stands
// for none is loaded too: 9 new tokens over each of 64 caches of 1024 tokens,
// in pieces of 4 tiles, take 38.2 us that way and 43.8 with sixteen throughout
// (one cache of 65536 takes 49.0 and 47.6).
template <int D, class Slot>
__device__ __forceinline__ Joined join_parts(uint32_t from, uint32_t to, uint32_t rows, uint32_t r, uint32_t f, Slot slot_of) {
    Joined j{-INFINITY, 0.0f, f32x4{0, 0, 0, 0}};
    for (uint32_t p = from; p < to;) {
        if (to - p > 8) {
            join_some<16, D>(j, p, to, rows, r, f, slot_of);
            p += 16;
        } else if (to - p > 4) {
            join_some<8, D>(j, p, to, rows, r, f, slot_of);
            p += 8;
        } else {
            join_some<4, D>(j, p, to, rows, r, f, slot_of);
            p += 4;
        }
    }
    return j;
}

}  // namespace
}  // namespace skv
