// skv_attention.hip -- attention of new tokens over a paged cache (gfx950).
//
// s_j = scale q.k_j over the keys a query sees, m = max s, l = sum exp(s - m),
// out = sum exp(s - m) v / l, lse = m + log l; in one pass over the keys with
// a running m and l, o and l rescaled by exp(m_old - m_new) when m grows.
//
//   attention_split    requests with at most 32 query rows (new tokens x the
//                      heads of a KV head): bound by reading the cache, so
//                      the keys are dealt out evenly over the chip
//   attention_combine  joins the parts of a request whose keys fell to more
//                      than one workgroup
//   attention_tiles    requests with more rows: 128 of them share the keys
//   attention_tile_combine  joins the runs of keys that few tiles are cut into
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

// Geometry of tiles of head_dim D in LDS: rows of RB bytes, 16-byte chunk c
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

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((SKV_LDS(const void))p));
}

// 16 bytes per lane from global memory to LDS at `lds` + 16 * lane, without
// passing through registers.  The wave waits for it itself (wait_loads).
// Written as assembly because the compiler would make every later LDS read
// wait for every such load; no register is written, so nothing can be reused
// too early.
__device__ __forceinline__ void load_lds16(const uint8_t* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
                 "v"(g)
                 : "memory");
}
// The same from a base that is the same for the wave and a byte offset per lane.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
                 "v"(offset), "s"(base)
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

// One tile of 32 * NM keys (kt, vt: the lane's LDS bases in it): scores,
// masked (where `mask`, the same for the wave) past key `limit` of the tile,
// the running maximum, probabilities, and their product with V.  factor > 0:
// scale in base-2 units.
template <int D, bool kE4m3, int NM>
__device__ __forceinline__ void tile_step(uint32_t kt, uint32_t vt, const bf16x8 (&q)[D / 16], float factor, bool mask,
                                          int limit, uint32_t lane, Rows<D>& st) {
    constexpr int kRow = Tile<D, kE4m3>::kRow;
    f32x16 s[NM];
#pragma unroll
    for (int t = 0; t < NM; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
    for (int p = 0; p < D / 32; ++p) {
#pragma unroll
        for (int t = 0; t < NM; ++t) {
            bf16x8 k[2];
            read_k<D, kE4m3>(kt, 32 * t * kRow, p, k);
            s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[0], q[2 * p], s[t], 0, 0, 0);
            s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[1], q[2 * p + 1], s[t], 0, 0, 0);
        }
    }
    if (mask) {
        const int lim = limit - 4 * int(lane >> 5);
#pragma unroll
        for (int t = 0; t < NM; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (32 * t + 8 * (r / 4) + r % 4 > lim) s[t][r] = -INFINITY;
    }
    float top = st.m;
#pragma unroll
    for (int t = 0; t < NM; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
    top = half_max(top);
    // -infinity stands for "nothing yet" and must not meet itself in a difference
    const float ref = top == -INFINITY ? 0.0f : top * factor;
    if (__any(top != st.m)) {
        const float keep = __builtin_amdgcn_exp2f(fmaf(st.m, factor, -ref));
        st.l *= keep;
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) st.o[t][r] *= keep;
        st.m = top;
    }
#pragma unroll
    for (int t = 0; t < NM; ++t) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            union {
                bf16x2 h[4];
                bf16x8 v;
            } p;
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[t][8 * hf + r], factor, -ref));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[t][8 * hf + r + 1], factor, -ref));
                st.l += x + y;
                // rounded to the MFMA's operand type: each probability by at most half a step of bf16, as the
                // result itself is; the sum keeps them in 32 bits
                p.h[r / 2] = bf16x2{__bf16(x), __bf16(y)};
            }
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
                st.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_v<D, kE4m3>(vt, (32 * t + 16 * hf) * kRow, dt), p.v,
                                                                   st.o[dt], 0, 0, 0);
        }
    }
}

// The same in two halves, for a wave that computes the scores of the next
// tile of 64 keys while it turns this one's into probabilities and adds their
// product with V: matrix and vector instructions of one wave then overlap.
// A tile is taken in four steps of 16 keys, each with a quarter of the next
// scores' products.
//
// m need not be the maximum: it is a reference that the sums are relative
// to, moved only when a score passes it by 2^8 (sums and products then stay
// below 2^8 times the number of keys, far from the end of the range, and
// relative roundings are the same), so o is rescaled a few times per row and
// not with every new maximum.
constexpr float kSlack = 8.0f;

template <int D, bool kE4m3>
struct Pipe {
    static constexpr int kRow = Tile<D, kE4m3>::kRow;
    static constexpr int kItems = D / 64;              // (pair of k-steps, half of the keys) per step
    f32x16 s[2];                                       // scores of the tile in hand
    float top;                                         // and their maximum, over the row's two lanes

    __device__ __forceinline__ static void item(int g, int i, int& p, int& t) {
        p = (g * kItems + i) >> 1;
        t = (g * kItems + i) & 1;
    }

    __device__ __forceinline__ static void read_ks(uint32_t kt, int g, bf16x8 (&k)[kItems][2]) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            int p, t;
            item(g, i, p, t);
            read_k<D, kE4m3>(kt, 32 * t * kRow, p, k[i]);
        }
    }

    __device__ __forceinline__ static void scores(int g, const bf16x8 (&k)[kItems][2], const bf16x8 (&q)[D / 16],
                                                  f32x16 (&s)[2]) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            int p, t;
            item(g, i, p, t);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[i][e], q[2 * p + e], s[t], 0, 0, 0);
        }
    }

    __device__ __forceinline__ static void zero(f32x16 (&s)[2]) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[0][r] = s[1][r] = 0.0f;
    }

    __device__ __forceinline__ static float maximum(const f32x16 (&s)[2]) {
        float x = s[0][0], y = s[1][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) {
            x = fmaxf(x, s[0][r]);
            y = fmaxf(y, s[1][r]);
        }
        return half_max(fmaxf(x, y));
    }

    // Scores of the first tile.
    __device__ __forceinline__ void first(uint32_t kt, const bf16x8 (&q)[D / 16]) {
        zero(s);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            bf16x8 k[kItems][2];
            read_ks(kt, g, k);
            scores(g, k, q, s);
        }
        top = maximum(s);
    }

    // Hides keys past `limit` of the tile (the lane's own row's).
    __device__ __forceinline__ void mask(int limit, uint32_t lane) {
        const int lim = limit - 4 * int(lane >> 5);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (32 * t + 8 * (r / 4) + r % 4 > lim) s[t][r] = -INFINITY;
        top = maximum(s);
    }

    // The tile in hand: kNext: also the scores of the next one (its keys at kt), which is then in hand.
    template <bool kNext>
    __device__ __forceinline__ void step(uint32_t kt, uint32_t vt, const bf16x8 (&q)[D / 16], float factor, Rows<D>& st) {
        if (__any((top - st.m) * factor > kSlack)) {               // (not where both are -infinity)
            const float m = fmaxf(st.m, top);
            const float keep = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((st.m - m) * factor);
            st.l *= keep;
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) st.o[t][r] *= keep;
            st.m = m;
        }
        // -infinity stands for "nothing yet" and must not meet itself in a difference
        const float ref = st.m == -INFINITY ? 0.0f : st.m * factor;
        f32x16 n[2];
        bf16x8 k[kItems][2], v[D / 32];
        union Weights {
            bf16x2 h[4];
            bf16x8 v;
        } w;
        if constexpr (kNext) {
            zero(n);
            read_ks(kt, 0, k);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            // the wave with matrix work goes first: the SIMD's other wave has vector work to fill in
            __builtin_amdgcn_s_setprio(1);
            // products: this step's share of the next scores, the last step's probabilities with V
            if constexpr (kNext) scores(g, k, q, n);
            if (g > 0) {
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt)
                    st.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[dt], w.v, st.o[dt], 0, 0, 0);
            }
            if constexpr (kNext) {
                if (g < 3) read_ks(kt, g + 1, k);
            }
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) v[dt] = read_v<D, kE4m3>(vt, 16 * g * kRow, dt);
            Weights x;
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
                const float y = __builtin_amdgcn_exp2f(fmaf(s[g >> 1][8 * (g & 1) + r], factor, -ref));
                const float z = __builtin_amdgcn_exp2f(fmaf(s[g >> 1][8 * (g & 1) + r + 1], factor, -ref));
                st.l += y + z;
                x.h[r / 2] = bf16x2{__bf16(y), __bf16(z)};         // rounded as in tile_step
            }
            w = x;
            // a matrix instruction, then some of the reads that the next step needs and some vector work, in turn
            constexpr int kScores = kNext ? 2 * kItems : 0, kValues = D / 32;
#pragma unroll
            for (int i = 0; i < kScores + (g ? kValues : 0); ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 32 / (kScores + kValues), 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
            st.o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[dt], w.v, st.o[dt], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        if constexpr (kNext) {
            s[0] = n[0];
            s[1] = n[1];
            top = maximum(s);
        }
    }
};

// ------------------------------------------------------------------ few rows
// The keys of every (request, KV head) are cut into units of kWaves * kKeys
// tokens, all units numbered through, and each of kParts workgroups takes an
// equal run of them: the cache is read once and evenly however different the
// lengths are.  A (request, head) counts one unit more than it has keys for,
// about what joining its waves costs.  A workgroup's run covers whole
// (request, head)s, which it finishes, and at most two broken ones (its first
// and last), whose unnormalized sums go to the workspace for
// attention_combine.
//
// A wave keeps two tiles of 16 KB (32 KB for D = 256) in LDS of its own: one
// being used, the other on its way straight from memory, 64 KB in flight per
// CU.  The next (request, head)'s first tile is on its way while the waves
// of the last one are joined.
constexpr uint32_t kSplitRows = 32;

template <int D, bool kE4m3>
struct Split {
    static constexpr int kWaves = D == 256 ? 2 : 4;
    static constexpr int kStage = D == 256 ? 32768 : 16384;                // bytes of K and V per wave
    static constexpr int kKeys = kStage / 2 / Tile<D, kE4m3>::kRow;         // per wave and tile
    static constexpr int kUnit = kWaves * kKeys;
    static_assert(kSplitRows * D * 4 <= kStage, "the join's sums of a wave fit one tile");
};

constexpr uint32_t kParts = 256;      // one workgroup per CU (128 KB of LDS)

struct Units {
    uint64_t total;                   // units of the whole batch
    uint64_t first;                   // of the request looked for
    uint32_t request;
};

// Units of one head of request b: one even where it has no keys, so that rows
// that see none get their zeros.
__device__ __forceinline__ uint32_t units_of(const AttentionLaunch& a, uint32_t b, uint32_t unit, uint32_t& flags) {
    const Span s = span_of(a, b, flags);
    if (s.n == 0 || s.n * a.group > kSplitRows) return 0;
    return 1 + (s.len + unit - 1) / unit;
}

// Sum over the workgroup's threads of x (kThreads of them), to all.
template <int kThreads>
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* s_wave, uint64_t* total) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    uint64_t sum = 0;
    for (uint32_t w = 0; w < kThreads / 64; ++w) {
        if (w < wave) x += s_wave[w];
        sum += s_wave[w];
    }
    *total = sum;
    return x;                          // inclusive
}

// A value that is the same in every lane, where the compiler can see that it is.
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return uint64_t(__builtin_amdgcn_readfirstlane(uint32_t(x >> 32))) << 32 |
           uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(x)));
}

// The batch's units and, with find(total) naming a unit, the request it
// belongs to and that request's first unit.  s_out: LDS for the answer.
template <int kThreads, class Find>
__device__ Units find_units(const AttentionLaunch& a, uint32_t unit, uint32_t& flags, Find find, uint64_t* s_wave,
                            uint64_t* s_out) {
    Units u{0, 0, a.requests};
    uint64_t total, at = 0, before = 0;
    const bool once = a.requests <= kThreads;           // one sum gives the total and every request's place
    if (!once) {
        uint64_t mine = 0;
        for (uint32_t b = threadIdx.x; b < a.requests; b += kThreads) mine += units_of(a, b, unit, flags);
        (void)block_scan<kThreads>(mine, s_wave, &total);
        u.total = total * a.heads;
        at = find(u.total);
    }
    uint32_t ignore = 0;
    for (uint32_t base = 0; base < a.requests; base += kThreads) {
        const uint32_t b = base + threadIdx.x;
        const uint64_t n = b < a.requests ? units_of(a, b, unit, once ? flags : ignore) : 0;
        const uint64_t end = before + block_scan<kThreads>(n, s_wave, &total);
        before += total;
        if (once) {
            u.total = total * a.heads;
            at = find(u.total);
        }
        if (n && at >= (end - n) * a.heads && at < end * a.heads) {
            s_out[0] = (end - n) * a.heads;
            s_out[1] = b;
        }
        if (at < before * a.heads) break;
    }
    __syncthreads();
    u.total = uniform(u.total);
    if (uniform(at) >= u.total) return u;
    u.first = uniform(s_out[0]);
    u.request = uint32_t(uniform(s_out[1]));
    return u;
}

// Workgroups with work: every one of them has at least one unit.
__device__ __forceinline__ uint64_t parts_of(uint64_t total) { return min(total, uint64_t(kParts)); }
__device__ __forceinline__ uint64_t part_begin(uint64_t total, uint32_t part) {
    return part < parts_of(total) ? total * part / parts_of(total) : total;
}

// Workspace: part p's slot: 32 rows of D sums, then 32 maxima (base-2 units)
// and 32 sums of probabilities.
template <int D>
__device__ __forceinline__ float* part_slot(void* work, uint32_t part, uint32_t slot) {
    return static_cast<float*>(work) + (uint64_t(part) * 2 + slot) * kSplitRows * (D + 2);
}

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

template <int D, bool kE4m3>
__global__ void __launch_bounds__((Split<D, kE4m3>::kWaves * 64), 1) attention_split(AttentionLaunch a, void* work) {
    using G = Split<D, kE4m3>;
    using T = Tile<D, kE4m3>;
    constexpr int kThreads = G::kWaves * 64, kLoads = G::kStage / 2 / 1024, kLanes = 64 / T::kRowsPerLoad;
    constexpr int kLook = G::kKeys > 64 ? 2 : 1;         // lane j looks up token j of a tile (and j + 64)
    __shared__ __align__(1024) uint8_t s_tiles[G::kWaves][2][G::kStage];
    __shared__ float s_m[G::kWaves][kSplitRows], s_l[G::kWaves][kSplitRows];
    __shared__ uint64_t s_wave[G::kWaves], s_found[2];
    __shared__ uint32_t s_bad, s_stage[G::kWaves];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t part = blockIdx.x, row = lane & 31;
    uint32_t flags = 0, ignore = 0;
    const Units un = find_units<kThreads>(a, G::kUnit, flags, [&](uint64_t total) { return part_begin(total, part); },
                                          s_wave, s_found);
    if (part == 0 && flags && a.status) atomicOr(a.status, flags);
    flags = 0;
    const uint64_t begin = part_begin(un.total, part), end = part_begin(un.total, part + 1);
    if (begin >= end) return;
    const uint32_t lds0 = lds_address(&s_tiles[wave][0][0]);
    const uint32_t lane_k = lds0 + base_k<D, kE4m3>(lane), lane_v = lds0 + G::kStage / 2 + base_v<D, kE4m3>(lane);

    // the request and head of unit u, the run of its units that is ours, and what its rows need
    uint64_t u = begin, first = un.first;
    uint32_t b = un.request, units = units_of(a, b, G::kUnit, ignore);
    Span sp = span_of(a, b, ignore);
    uint32_t head, run, t0, stop;
    bool whole;
    float raw;
    int first_limit, limit;
    bf16x8 q[D / 16];
    int32_t next[kLook];
    uint32_t stage = 1;
    const uint8_t *kb, *vb;
    auto look_up = [&](uint32_t at, int32_t (&e)[kLook]) __attribute__((always_inline)) {
        for (int i = 0; i < kLook; ++i)
            e[i] = a.table[int64_t(b) * a.table_stride + (min(at + 64 * i + lane, sp.len - 1) >> a.page_shift)];
    };
    auto load_tile = [&](uint32_t at, const int32_t (&e)[kLook], uint32_t to) __attribute__((always_inline)) {
        int64_t off[kLook];
        for (int i = 0; i < kLook; ++i) {
            const uint32_t token = min(at + 64 * i + lane, sp.len - 1);
            bool bad = false;
            const uint32_t page = page_or_zero(e[i], a.pages, &bad);
            if (bad) flags |= SKV_PAGES_PAGE;
            off[i] = int64_t(page) * a.page_stride + int64_t(token & ((1u << a.page_shift) - 1)) * a.token_stride;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t r = i * T::kRowsPerLoad + lane / kLanes, c = lane % kLanes;
            const int64_t o = __shfl(off[(i * T::kRowsPerLoad) / 64], int(r & 63));
            load_lds16(kb + o + ((c ^ T::swizzle_k(r)) << 4), lds0 + to * G::kStage + i * 1024);
            load_lds16(vb + o + ((c ^ T::swizzle_v(r)) << 4), lds0 + to * G::kStage + G::kStage / 2 + i * 1024);
        }
    };
    // Unit u's (request, head): its rows' queries and its first tile, into the stage that is not in use.
    auto open = [&]() __attribute__((always_inline)) -> bool {
        while (units == 0 || u - first >= uint64_t(units) * a.heads) {
            first += uint64_t(units) * a.heads;
            if (++b >= a.requests) return false;
            units = units_of(a, b, G::kUnit, ignore);
            sp = span_of(a, b, ignore);
        }
        head = uint32_t((u - first) / units);
        const uint32_t c0 = uint32_t((u - first) % units), c1 = uint32_t(min(uint64_t(units), c0 + (end - u)));
        run = c1 - c0;
        whole = run == units;
        const uint32_t qi = row / a.group, qg = row - qi * a.group;
        const bool have = row < sp.n * a.group;
        raw = a.scale * (a.k_scale ? a.k_scale[head] : 1.0f);
        first_limit = a.causal ? int(sp.len) - int(sp.n) : int(sp.len) - 1;          // of query 0
        limit = have ? first_limit + (a.causal ? int(qi) : 0) : -1;
        kb = a.k_pages + int64_t(head) * a.head_stride;
        vb = a.v_pages + int64_t(head) * a.head_stride;
        t0 = c0 * G::kUnit + wave * G::kKeys;
        stop = min(c1 * G::kUnit, sp.len);
        if (t0 < stop) {
            int32_t e[kLook];
            look_up(t0, e);
            look_up(t0 + G::kUnit, next);
            load_q<D, kE4m3>(a.q + int64_t(sp.row + qi) * a.q_token + int64_t(head * a.group + qg) * a.q_head, have, raw,
                             lane, q);
            load_tile(t0, e, stage ^ 1);
        }
        return true;
    };

    bool more = open();
    while (more) {
        const float factor = raw == 0.0f ? 1.0f : fabsf(raw) * kLog2e;
        Rows<D> st;
        st.clear();
        for (; t0 < stop; t0 += G::kUnit) {
            stage ^= 1;
            wait_loads();
            if (t0 + G::kUnit < stop) {
                int32_t e[kLook];
                for (int i = 0; i < kLook; ++i) e[i] = next[i];
                look_up(t0 + 2 * G::kUnit, next);
                load_tile(t0 + G::kUnit, e, stage ^ 1);
            }
            tile_step<D, kE4m3, G::kKeys / 32>(lane_k + stage * G::kStage, lane_v + stage * G::kStage, q, factor,
                                               int(t0) + G::kKeys - 1 > first_limit, limit - int(t0), lane, st);
        }
        // what is joined now, before the next one's state takes its place
        const Span was = sp;
        const uint32_t was_b = b, was_head = head, rows = sp.n * a.group, slot_at = u != begin;
        const bool was_whole = whole;
        const int was_limit = first_limit;
        u += run;
        more = u < end && open();
        // the sums of each wave to LDS, into the stage it used last; then every thread takes some of a row's values
        if (row < rows) {
            f32x4* mine = reinterpret_cast<f32x4*>(&s_tiles[wave][stage][0]) + row * (D / 4);
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    mine[(8 * t + 2 * (r / 4) + (lane >> 5)) ^ (row & 7)] =
                        f32x4{st.o[t][r], st.o[t][r + 1], st.o[t][r + 2], st.o[t][r + 3]};
            const float l = half_sum(st.l);
            if (lane < 32) {
                s_m[wave][row] = st.m * factor;
                s_l[wave][row] = l;
            }
        }
        if (lane == 0) s_stage[wave] = stage;
        if (tid == 0) s_bad = 0;
        __syncthreads();
        const float vs = a.v_scale ? a.v_scale[was_head] : 1.0f;
        float* slot = part_slot<D>(work, part, slot_at);
        for (uint32_t i = tid; i < rows * (D / 4); i += kThreads) {
            const uint32_t r = i / (D / 4), f = i % (D / 4);
            float top = s_m[0][r], l = 0.0f;
            for (int w = 1; w < G::kWaves; ++w) top = fmaxf(top, s_m[w][r]);
            f32x4 o{0, 0, 0, 0};
            for (int w = 0; w < G::kWaves; ++w) {
                const float k = exp2_diff(s_m[w][r], top);
                l += k * s_l[w][r];
                if (s_m[w][r] != -INFINITY)        // else all its keys were hidden, and o may be 0 * NaN
                    o += k * reinterpret_cast<const f32x4*>(&s_tiles[w][s_stage[w]][0])[r * (D / 4) + (f ^ (r & 7))];
            }
            if (was_whole) {
                const uint32_t ri = r / a.group, qh = was_head * a.group + r - ri * a.group;
                const bool none = was_limit + (a.causal ? int(ri) : 0) < 0;
                const bool nan = store_out(a, was.row + ri, qh, 4 * f, none ? f32x4{0, 0, 0, 0} : o * (vs / l));
                if (nan && a.causal && was.n > 1) atomicOr(&s_bad, 1u << r);
                if (f == 0) store_lse(a, was.row + ri, qh, none ? -INFINITY : top, none ? 1.0f : l);
            } else {
                *reinterpret_cast<f32x4*>(slot + r * D + 4 * f) = o;
                if (f == 0) {
                    slot[kSplitRows * D + r] = top;
                    slot[kSplitRows * (D + 1) + r] = l;
                }
            }
        }
        __syncthreads();
        // A NaN in a value that only later queries see has reached a row through 0 * NaN in a shared tile: such
        // rows (and those whose NaN is their own) are computed again, key after key.
        if (was_whole && a.causal && was.n > 1) {
            for (uint32_t r = 0, bad = s_bad; r < rows; ++r)
                if ((bad >> r & 1) && r % G::kWaves == wave)
                    row_plain<D, kE4m3>(a, was_b, was, r / a.group, was_head * a.group + r % a.group, flags);
            __syncthreads();
        }
    }
    if (flags && a.status) atomicOr(a.status, flags);
}

// Partial sums (m in base-2 units, l, o) read kAtOnce at a time: their loads are in flight together.
struct Joined {
    float m, l;
    f32x4 o;
};

template <int D, class Slot>
__device__ __forceinline__ Joined join_parts(uint32_t from, uint32_t to, uint32_t rows, uint32_t r, uint32_t f, Slot slot_of) {
    constexpr uint32_t kAtOnce = 8;
    Joined j{-INFINITY, 0.0f, f32x4{0, 0, 0, 0}};
    for (uint32_t p = from; p < to; p += kAtOnce) {
        float m[kAtOnce], l[kAtOnce];
        f32x4 o[kAtOnce];
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) {
            const float* slot = slot_of(min(p + i, to - 1));
            m[i] = slot[rows * D + r];
            l[i] = slot[rows * (D + 1) + r];
            o[i] = *reinterpret_cast<const f32x4*>(slot + r * D + 4 * f);
        }
        float top = j.m;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) {
            if (p + i >= to) m[i] = -INFINITY;
            top = fmaxf(top, m[i]);
        }
        const float keep = exp2_diff(j.m, top);
        j.l *= keep;
        j.o *= keep;
        j.m = top;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) {
            const float k = exp2_diff(m[i], top);
            j.l += k * l[i];
            if (m[i] != -INFINITY) j.o += k * o[i];    // else all its keys were hidden, and o may be 0 * NaN
        }
    }
    return j;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) attention_combine(AttentionLaunch a, const void* work) {
    using G = Split<D, kE4m3>;
    __shared__ uint64_t s_sum[4][2];
    __shared__ uint32_t s_bad;
    const uint32_t head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    uint32_t flags = 0;
    const uint32_t units = units_of(a, b, G::kUnit, flags);
    // the units of the earlier requests, and of all
    uint64_t before = 0, all = 0;
    for (uint32_t i = tid; i < a.requests; i += 256) {
        const uint64_t n = units_of(a, i, G::kUnit, flags);
        all += n;
        if (i < b) before += n;
    }
    for (uint32_t d = 32; d; d >>= 1) {
        before += __shfl_xor(before, d);
        all += __shfl_xor(all, d);
    }
    if ((tid & 63) == 0) {
        s_sum[tid >> 6][0] = before;
        s_sum[tid >> 6][1] = all;
    }
    if (tid == 0) s_bad = 0;
    __syncthreads();
    if (units == 0) return;
    before = all = 0;
    for (int w = 0; w < 4; ++w) {
        before += s_sum[w][0];
        all += s_sum[w][1];
    }
    all *= a.heads;
    const uint64_t u0 = before * a.heads + uint64_t(head) * units, u1 = u0 + units;
    // the part that has unit u: the last p with all * p / parts <= u
    const uint32_t p0 = uint32_t(((u0 + 1) * parts_of(all) - 1) / all), p1 = uint32_t((u1 * parts_of(all) - 1) / all);
    if (p0 == p1) return;              // finished by one workgroup
    const Span sp = span_of(a, b, flags);
    const uint32_t rows = sp.n * a.group, late = part_begin(all, p0) < u0;       // p0's slot: its first or its last
    const int first_limit = a.causal ? int(sp.len) - int(sp.n) : int(sp.len) - 1;
    const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
    for (uint32_t i = tid; i < rows * (D / 4); i += 256) {
        const uint32_t r = i / (D / 4), f = i % (D / 4);
        const Joined j = join_parts<D>(p0, p1 + 1, kSplitRows, r, f, [&](uint32_t p) -> const float* {
            return part_slot<D>(const_cast<void*>(work), p, p == p0 ? late : 0);
        });
        const uint32_t ri = r / a.group, qh = head * a.group + r - ri * a.group;
        const bool none = first_limit + (a.causal ? int(ri) : 0) < 0;
        const bool nan = store_out(a, sp.row + ri, qh, 4 * f, none ? f32x4{0, 0, 0, 0} : j.o * (vs / j.l));
        if (nan && a.causal && sp.n > 1) atomicOr(&s_bad, 1u << r);
        if (f == 0) store_lse(a, sp.row + ri, qh, none ? -INFINITY : j.m, none ? 1.0f : j.l);
    }
    if (!a.causal || sp.n == 1) return;
    __syncthreads();
    for (uint32_t r = 0, bad = s_bad; r < rows; ++r)
        if ((bad >> r & 1) && r % 4 == (tid >> 6))
            row_plain<D, kE4m3>(a, b, sp, r / a.group, head * a.group + r % a.group, flags);
}

// ------------------------------------------------------------------ many rows
// A workgroup takes 128 query rows of one (request, KV head): new tokens x
// the head's query heads, in that order, so all of them share the keys it
// streams through LDS, 64 at a time, two tiles deep.  Each of its four waves
// owns 32 rows.  (64 rows a wave halve the reads of K and V from LDS, but
// the scores then lie in accumulation registers that vector instructions
// reach only through copies: 1.34 ms against 1.05 for 2048 tokens at 32768.)
//
// Work is cut on the device, where the lengths are: a (tile of rows, head)
// with more keys than kTileSlots-th of the whole work is cut into pieces of
// that size, whose unnormalized sums attention_tile_combine joins; the
// others are finished where they are computed.  Requests with the most keys
// come first, and of a request the last rows, which see the most.  The heads
// come fastest: eight consecutive workgroups go to the eight XCDs, so with 8
// KV heads (or a divisor or multiple) each XCD's L2 holds the keys of its own
// heads.
constexpr uint32_t kTileRows = 128, kTileKeys = 64;
constexpr uint32_t kLeastPiece = 4;        // tiles of keys: below, joining costs more than it spreads

// Keys that rows up to `row` of a request see.
__device__ __forceinline__ uint32_t keys_for(const AttentionLaunch& a, const Span& s, uint32_t row) {
    if (!a.causal) return s.len;
    const uint32_t rows = s.n * a.group;
    const int64_t last = int64_t(s.len) - s.n + min(row, rows - 1) / a.group;
    return last < 0 ? 0 : uint32_t(last) + 1;
}

// Workgroups that run at the same time: D = 256 takes all registers of a CU for one.
__host__ __device__ constexpr uint32_t tile_slots(int head_dim) { return head_dim == 256 ? 256 : 512; }

// Upper bound on the tiles of rows of one head, for the host.
uint32_t tile_bound(const AttentionLaunch& a) {
    return uint32_t(uint64_t(a.tokens) * a.group / kTileRows) + std::min(a.requests, a.tokens);
}

struct TileWork {
    uint32_t request;                  // a.requests: none
    uint32_t tiles, pieces;            // tiles of rows of the request; pieces of its longest one
    uint32_t index;                    // among the request's (tile, piece)s, or its tiles for the join
    uint32_t slot;                     // first workspace slot of the request (where pieces > 1)
    uint32_t piece_tiles;              // tiles of keys in a piece
};

struct TileSearch {
    uint64_t sum[4];
    uint32_t key[256], count[256], slots[256], who[256], wave[4][2], found[5];
};

// Where number `index` of the (tile, piece)s of one head is, or for the join
// number `index` of the tiles of requests that are in pieces.  At most
// tile_bound + kSlots / heads of the former, kSlots / heads of the latter, and
// 2 kSlots workspace slots over all heads: a request in pieces has fewer than
// 2 tiles * keys / piece of them.
template <uint32_t kSlots, bool kJoin>
__device__ __forceinline__ TileWork find_work(const AttentionLaunch& a, uint32_t index, uint32_t& flags, TileSearch& s) {
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto measure = [&](uint32_t b, uint32_t& tiles, uint32_t& keys, uint32_t& f) __attribute__((always_inline)) {
        const Span sp = span_of(a, b, f);
        tiles = (sp.n * a.group + kTileRows - 1) / kTileRows;
        keys = tiles ? (keys_for(a, sp, ~0u) + kTileKeys - 1) / kTileKeys : 0;
    };
    uint64_t all = 0;
    uint32_t tiles = 0, keys = 0, ignore = 0;
    for (uint32_t b = tid; b < a.requests; b += 256) {
        measure(b, tiles, keys, flags);
        all += uint64_t(tiles) * keys;
    }
    for (uint32_t d = 32; d; d >>= 1) all += __shfl_xor(all, d);
    if (lane == 0) s.sum[wave] = all;
    if (tid == 0) s.found[0] = a.requests;
    __syncthreads();
    all = (s.sum[0] + s.sum[1] + s.sum[2] + s.sum[3]) * a.heads;
    const uint32_t piece = max(kLeastPiece, uint32_t((all + kSlots - 1) / kSlots));
    uint32_t before = 0, slot0 = 0;
    for (uint32_t base = 0; base < a.requests; base += 256) {
        const uint32_t b = base + tid, n = min(256u, a.requests - base);
        if (b >= a.requests) tiles = keys = 0;
        else if (a.requests > 256) measure(b, tiles, keys, ignore);
        // the longest first
        s.key[tid] = keys;
        __syncthreads();
        uint32_t rank = 0;
        for (uint32_t x = 0; x < n; ++x) rank += s.key[x] > keys || (s.key[x] == keys && x < tid);
        if (tid < n) {
            const uint32_t pieces = max(1u, (keys + piece - 1) / piece);
            s.count[rank] = kJoin ? (pieces > 1 ? tiles : 0) : tiles * pieces;
            s.slots[rank] = pieces > 1 ? tiles * pieces : 0;
            s.who[rank] = tid;
        }
        __syncthreads();
        uint32_t x = tid < n ? s.count[tid] : 0, y = tid < n ? s.slots[tid] : 0;
        const uint32_t own = x, own_slots = y;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint32_t u = __shfl_up(x, d), v = __shfl_up(y, d);
            if (lane >= d) {
                x += u;
                y += v;
            }
        }
        if (lane == 63) {
            s.wave[wave][0] = x;
            s.wave[wave][1] = y;
        }
        __syncthreads();
        uint32_t total = 0, total_slots = 0;
        for (uint32_t w = 0; w < 4; ++w) {
            if (w < wave) {
                x += s.wave[w][0];
                y += s.wave[w][1];
            }
            total += s.wave[w][0];
            total_slots += s.wave[w][1];
        }
        const uint32_t end = before + x;
        if (own && index >= end - own && index < end) {
            s.found[0] = base + s.who[tid];
            s.found[1] = index - (end - own);
            s.found[2] = slot0 + y - own_slots;
        }
        before += total;
        slot0 += total_slots;
        if (index < before) break;
    }
    __syncthreads();
    TileWork t{};
    t.request = __builtin_amdgcn_readfirstlane(s.found[0]);
    if (t.request >= a.requests) return t;
    t.index = __builtin_amdgcn_readfirstlane(s.found[1]);
    t.slot = __builtin_amdgcn_readfirstlane(s.found[2]);
    t.piece_tiles = __builtin_amdgcn_readfirstlane(piece);
    measure(t.request, t.tiles, keys, ignore);
    t.pieces = max(1u, (keys + t.piece_tiles - 1) / t.piece_tiles);
    return t;
}

template <int D>
__device__ __forceinline__ float* tile_slot(void* work, uint64_t id) {
    return static_cast<float*>(work) + id * kTileRows * (D + 2);
}

template <int D, bool kE4m3>
struct TileGeo {
    static constexpr int kStage = 2 * kTileKeys * Tile<D, kE4m3>::kRow;
    static constexpr int kPerCu = tile_slots(D) / 256;               // workgroups a CU holds
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256, (TileGeo<D, kE4m3>::kPerCu)) attention_tiles(AttentionLaunch a, void* work) {
    using T = Tile<D, kE4m3>;
    using G = TileGeo<D, kE4m3>;
    constexpr int kWaveRows = kTileKeys / 4, kLoads = kWaveRows * T::kRow / 1024, kLanes = 64 / T::kRowsPerLoad;
    __shared__ __align__(1024) uint8_t s_tiles[2][G::kStage];
    __shared__ TileSearch s_search;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t head = blockIdx.x % a.heads;
    uint32_t flags = 0;
    const TileWork at = find_work<tile_slots(D), false>(a, blockIdx.x / a.heads, flags, s_search);
    if (blockIdx.x == 0 && flags && a.status) atomicOr(a.status, flags);
    flags = 0;
    if (at.request >= a.requests) return;
    const uint32_t b = at.request, tile = at.tiles - 1 - at.index / at.pieces, piece = at.index % at.pieces;
    const Span sp = span_of(a, b, flags);
    const uint32_t rows = sp.n * a.group, wave_row = tile * kTileRows + 32 * wave;
    const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
    const float raw = a.scale * (a.k_scale ? a.k_scale[head] : 1.0f);
    const float factor = raw == 0.0f ? 1.0f : fabsf(raw) * kLog2e;
    const int first = int(sp.len) - int(sp.n);
    const uint32_t row = wave_row + (lane & 31), qi = row / a.group, qh = head * a.group + row - qi * a.group;
    const bool have = row < rows;
    bf16x8 q[D / 16];
    load_q<D, kE4m3>(a.q + int64_t(sp.row + qi) * a.q_token + int64_t(qh) * a.q_head, have, raw, lane, q);
    const int limit = !have ? -1 : a.causal ? first + int(qi) : int(sp.len) - 1;
    Rows<D> st;
    st.clear();
    // of the wave's rows: the keys that all of them see, and the keys that any of them sees
    const int all_see = wave_row >= rows ? 0 : a.causal ? max(first + int(wave_row / a.group) + 1, 0) : int(sp.len);
    const int any_sees = wave_row >= rows ? 0 : int(keys_for(a, sp, wave_row + 31));
    const uint32_t keys = keys_for(a, sp, tile * kTileRows + kTileRows - 1), span = at.piece_tiles * kTileKeys;
    const bool whole = keys <= span;                   // these rows have one piece
    const uint32_t begin = min(piece * uint64_t(span), uint64_t(keys)), end = min(begin + uint64_t(span), uint64_t(keys));
    if (piece && begin == end) return;                 // earlier rows see fewer keys than the request's last
    const uint8_t* kb = a.k_pages + int64_t(head) * a.head_stride;
    const uint8_t* vb = a.v_pages + int64_t(head) * a.head_stride;
    const uint32_t lds = lds_address(&s_tiles[0][0]), lds0 = lds + wave * kWaveRows * T::kRow;
    const uint32_t lane_k = lds + base_k<D, kE4m3>(lane), lane_v = lds + G::kStage / 2 + base_v<D, kE4m3>(lane);
    // A wave brings in 16 of the 64 keys. Eight of them share a page, so the wave works out two addresses a tile (one
    // and a step where pages are longer), on the scalar unit, and each lane's offsets from them once for all tiles.
    // The last tile of a request, whose rows stop at its last token (what lies behind it may be anything, NaN too),
    // and strides too long for a 32-bit offset take an address per lane.
    const bool shared = a.token_stride >= 0 && a.token_stride < (1 << 26);
    const auto* table = (const __attribute__((address_space(4))) int32_t*)(a.table + int64_t(b) * a.table_stride);
    struct Entries {
        int32_t e[2];
    };
    struct Where {
        int64_t at[2];
    };
    auto look_up = [&](uint32_t at) __attribute__((always_inline)) -> Entries {
        const uint32_t t = at + wave * kWaveRows, last = sp.len - 1;
        return Entries{{table[min(t, last) >> a.page_shift], table[min(t + 8, last) >> a.page_shift]}};
    };
    auto place = [&](uint32_t at, int32_t entry) __attribute__((always_inline)) -> int64_t {
        bool bad = false;
        const uint32_t page = page_or_zero(entry, a.pages, &bad);
        if (bad) flags |= SKV_PAGES_PAGE;
        return int64_t(page) * a.page_stride + int64_t(at & ((1u << a.page_shift) - 1)) * a.token_stride;
    };
    auto find = [&](uint32_t at, const Entries& x) __attribute__((always_inline)) -> Where {
        const uint32_t t = at + wave * kWaveRows;
        Where w;
        w.at[0] = place(t, x.e[0]);
        w.at[1] = a.page_shift > 3 ? w.at[0] + 8 * a.token_stride : place(t + 8, x.e[1]);
        return w;
    };
    auto load_tile = [&](const uint8_t* from, bool v, uint32_t at, const Where& w, uint32_t stage)
                         __attribute__((always_inline)) {
        const uint32_t to = lds0 + stage * G::kStage + (v ? G::kStage / 2 : 0);
        if (shared && at + kTileKeys <= sp.len) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t in = i * T::kRowsPerLoad + lane / kLanes, r = wave * kWaveRows + in, c = lane % kLanes;
                const uint32_t chunk = (c ^ (v ? T::swizzle_v(r) : T::swizzle_k(r))) << 4;
                const uint32_t offset = (in & 7) * uint32_t(a.token_stride) + chunk;
                if constexpr (T::kRowsPerLoad <= 8)
                    load_lds16(from + w.at[(i * T::kRowsPerLoad) >> 3], offset, to + i * 1024);
                else
                    load_lds16(from + (in < 8 ? w.at[0] : w.at[1]) + offset, to + i * 1024);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t r = wave * kWaveRows + i * T::kRowsPerLoad + lane / kLanes, c = lane % kLanes;
                load_lds16(from + token_at(a, b, min(at + r, sp.len - 1), flags) +
                               ((c ^ (v ? T::swizzle_v(r) : T::swizzle_k(r))) << 4),
                           to + i * 1024);
            }
        }
    };
    if (begin < end) {
        // K runs one tile ahead of V: while tile t is finished, the scores of t + 1 are computed and K of t + 2 and V
        // of t + 1 are on their way
        Where now = find(begin, look_up(begin));       // of the tile whose V comes next
        Entries next = look_up(begin + kTileKeys);     // of the tile whose K comes next
        load_tile(kb, false, begin, now, 0);
        load_tile(vb, true, begin, now, 0);
        if (begin + kTileKeys < end) {
            now = find(begin + kTileKeys, next);
            load_tile(kb, false, begin + kTileKeys, now, 1);
            next = look_up(begin + 2 * kTileKeys);
        }
        uint32_t stage = 0, t0 = begin;
        auto advance = [&]() __attribute__((always_inline)) {               // tile t0's V and the next one's K are there
            wait_loads();
            __syncthreads();
            if (t0 + kTileKeys < end) {
                load_tile(vb, true, t0 + kTileKeys, now, stage ^ 1);
                if (t0 + 2 * kTileKeys < end) {
                    now = find(t0 + 2 * kTileKeys, next);
                    load_tile(kb, false, t0 + 2 * kTileKeys, now, stage);
                    next = look_up(t0 + 3 * kTileKeys);
                }
            }
        };
        // the wave's own rows may be done before the workgroup's last ones
        const uint32_t own = min(end, uint32_t(any_sees));
        Pipe<D, kE4m3> pipe;
        auto mask = [&](uint32_t at) __attribute__((always_inline)) {
            if (int(at + kTileKeys) > all_see) pipe.mask(limit - int(at), lane);
        };
        wait_loads();
        __syncthreads();
        if (own > begin) {
            pipe.first(lane_k, q);
            mask(begin);
        }
        for (; t0 + kTileKeys < own; t0 += kTileKeys, stage ^= 1) {
            advance();
            pipe.template step<true>(lane_k + (stage ^ 1) * G::kStage, lane_v + stage * G::kStage, q, factor, st);
            mask(t0 + kTileKeys);
        }
        if (t0 < own) {
            advance();
            pipe.template step<false>(0, lane_v + stage * G::kStage, q, factor, st);
            t0 += kTileKeys;
            stage ^= 1;
        }
        for (; t0 < end; t0 += kTileKeys, stage ^= 1) advance();
    }
    const float l = half_sum(st.l);
    if (!whole) {
        const uint64_t id = uint64_t(at.slot + at.index) * a.heads + head;
        if (id >= a.slots) return;                     // only where requests' rows overlap
        float* slot = tile_slot<D>(work, id);
        const uint32_t r0 = 32 * wave + (lane & 31);
        if (have) {
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<f32x4*>(slot + r0 * D + 32 * t + 2 * r + 4 * (lane >> 5)) =
                        f32x4{st.o[t][r], st.o[t][r + 1], st.o[t][r + 2], st.o[t][r + 3]};
            if (lane < 32) {
                slot[kTileRows * D + r0] = st.m * factor;
                slot[kTileRows * (D + 1) + r0] = l;
            }
        }
    } else {
        bool nan = false;
        if (have) {
            const bool none = limit < 0;
            const float inv = none ? 0.0f : vs / l;
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const f32x4 o{st.o[t][r], st.o[t][r + 1], st.o[t][r + 2], st.o[t][r + 3]};
                    nan |= store_out(a, sp.row + qi, qh, 32 * t + 2 * r + 4 * (lane >> 5), none ? f32x4{0, 0, 0, 0} : o * inv);
                }
            if (lane < 32) store_lse(a, sp.row + qi, qh, none ? -INFINITY : st.m * factor, none ? 1.0f : l);
        }
        const uint64_t any = __ballot(nan && a.causal);
        for (uint32_t bad = uint32_t(any) | uint32_t(any >> 32); bad; bad &= bad - 1) {       // as in attention_split
            const uint32_t r = wave_row + __builtin_ctz(bad);
            row_plain<D, kE4m3>(a, b, sp, r / a.group, head * a.group + r % a.group, flags);
        }
    }
    if (flags && a.status) atomicOr(a.status, flags);
}

// blockIdx.y: 16 of the tile's rows.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) attention_tile_combine(AttentionLaunch a, void* work) {
    __shared__ TileSearch s_search;
    __shared__ uint32_t s_bad;
    const uint32_t tid = threadIdx.x, head = blockIdx.x % a.heads;
    uint32_t flags = 0;
    if (tid == 0) s_bad = 0;
    const TileWork at = find_work<tile_slots(D), true>(a, blockIdx.x / a.heads, flags, s_search);
    if (at.request >= a.requests) return;
    const Span sp = span_of(a, at.request, flags);
    const uint32_t row0 = (at.tiles - 1 - at.index) * kTileRows, from = 16 * blockIdx.y;
    const uint32_t rows = min(kTileRows, sp.n * a.group - row0);
    const uint32_t keys = keys_for(a, sp, row0 + kTileRows - 1), span = at.piece_tiles * kTileKeys;
    if (from >= rows || keys <= span) return;
    const uint32_t pieces = (keys + span - 1) / span, count = min(16u, rows - from);
    const uint64_t slot0 = at.slot + uint64_t(at.index) * at.pieces;
    if ((slot0 + pieces) * a.heads > a.slots) return;
    const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
    for (uint32_t i = tid; i < count * (D / 4); i += 256) {
        const uint32_t r = from + i / (D / 4), f = i % (D / 4);
        const Joined j = join_parts<D>(0, pieces, kTileRows, r, f, [&](uint32_t p) -> const float* {
            return tile_slot<D>(work, (slot0 + p) * a.heads + head);
        });
        const uint32_t row = row0 + r, qi = row / a.group, qh = head * a.group + row - qi * a.group;
        const bool none = keys_for(a, sp, row) == 0;
        const bool nan = store_out(a, sp.row + qi, qh, 4 * f, none ? f32x4{0, 0, 0, 0} : j.o * (vs / j.l));
        if (nan && a.causal) atomicOr(&s_bad, 1u << (r - from));
        if (f == 0) store_lse(a, sp.row + qi, qh, none ? -INFINITY : j.m, none ? 1.0f : j.l);
    }
    if (!a.causal) return;
    __syncthreads();
    for (uint32_t r = 0, bad = s_bad; r < count; ++r)
        if ((bad >> r & 1) && r % 4 == (tid >> 6)) {
            const uint32_t row = row0 + from + r;
            row_plain<D, kE4m3>(a, at.request, sp, row / a.group, head * a.group + row % a.group, flags);
        }
}

// Where no request can have more than 32 rows the split kernel takes the
// batch; else the tile kernel takes all of it, requests with few rows too: of
// their tiles only the waves that have rows compute, and the keys still come
// at the rate of the memory.
bool few_rows(const AttentionLaunch& a) { return a.max_new * uint64_t(a.group) <= kSplitRows; }

// Workspace slots of the tile kernel: as many as find_work gives out, or as the longest table can need.
uint32_t slots_of(const AttentionLaunch& a, int head_dim) {
    const uint64_t keys = ((uint64_t(a.width) << a.page_shift) + kTileKeys - 1) / kTileKeys;
    const uint64_t most = uint64_t(tile_bound(a)) * a.heads * ((keys + kLeastPiece - 1) / kLeastPiece);
    return uint32_t(std::min<uint64_t>(2 * tile_slots(head_dim), most));
}

template <int D, bool kE4m3>
hipError_t launch(AttentionLaunch a, void* work, hipStream_t stream) {
    if (few_rows(a)) {
        attention_split<D, kE4m3><<<kParts, Split<D, kE4m3>::kWaves * 64, 0, stream>>>(a, work);
        attention_combine<D, kE4m3><<<dim3(a.heads, a.requests), 256, 0, stream>>>(a, work);
    } else {
        a.slots = slots_of(a, D);
        const uint32_t extra = tile_slots(D) / a.heads + 1;
        const uint64_t rows = std::min<uint64_t>(kTileRows, uint64_t(a.max_new) * a.group);
        attention_tiles<D, kE4m3><<<(tile_bound(a) + extra) * a.heads, 256, 0, stream>>>(a, work);
        attention_tile_combine<D, kE4m3><<<dim3(extra * a.heads, uint32_t(rows + 15) / 16), 256, 0, stream>>>(a, work);
    }
    return hipGetLastError();
}

}  // namespace

uint64_t attention_work_bytes(const AttentionLaunch& a, uint32_t head_dim) {
    if (few_rows(a)) return uint64_t(kParts) * 2 * kSplitRows * (head_dim + 2) * 4;
    return std::max<uint64_t>(256, uint64_t(slots_of(a, int(head_dim))) * kTileRows * (head_dim + 2) * 4);
}

hipError_t launch_attention(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void* work,
                            hipStream_t stream) {
    const bool e4m3 = dtype == SKV_E4M3;
    switch (head_dim) {
        case 64: return e4m3 ? launch<64, true>(a, work, stream) : launch<64, false>(a, work, stream);
        case 128: return e4m3 ? launch<128, true>(a, work, stream) : launch<128, false>(a, work, stream);
        default: return e4m3 ? launch<256, true>(a, work, stream) : launch<256, false>(a, work, stream);
    }
}

}  // namespace skv
