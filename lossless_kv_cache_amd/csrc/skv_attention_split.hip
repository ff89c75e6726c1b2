// skv_attention_split.hip -- attention of requests with few query rows over a
// paged cache (gfx950): at most 32 rows (new tokens x the heads of a KV head),
// bound by reading the cache, so the keys are dealt out evenly over the chip.
//
//   attention_split    the keys' runs, each by one workgroup
//   attention_combine  joins the parts of a request whose keys fell to more
//                      than one
#include "skv_attention.h"

namespace skv {
namespace {

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

// The keys of every (request, KV head) are cut into units of kWaves * kKeys
// tokens, all units numbered through, and each of kParts workgroups takes an
// equal run of them: the cache is read once and evenly however different the
// lengths are.  A (request, head) counts one unit more than it has keys for,
// about what joining its waves costs.  A workgroup's run covers whole
// (request, head)s, which it finishes, and at most two broken ones (its first
// and last), whose unnormalized sums go to the workspace for
// attention_combine.
//
// A wave keeps two tiles of 16 KB (two waves with 32 KB for bf16 at D = 256)
// in LDS of its own: one being used, the other on its way straight from
// memory, 64 KB in flight per CU.  The next (request, head)'s first tile is on
// its way while the last tile of this one is used and its waves are joined.
//
// Bound by memory: 1.9 GB of four requests at 100000 to 131072 tokens in 306
// us (6.2 TB/s, fetching 1.00 times the cache), 0.74 GB of 64 requests at 100
// to 32768 tokens in e4m3 in 148 us (5.0 TB/s; 249 without the next one's
// early start and the unit for a join).  The loads are marked as read once:
// unmarked, the two take 343 and 163 us, and 2.1 GB in bf16 at D = 256 takes
// 375 for 329.
constexpr uint32_t kSplitRows = 32;

template <int D, bool kE4m3>
struct Split {
    static constexpr int kWaves = Tile<D, kE4m3>::kRow > 256 ? 2 : 4;
    static constexpr int kStage = 65536 / kWaves;                           // bytes of K and V per wave
    static constexpr int kKeys = kStage / 2 / Tile<D, kE4m3>::kRow;         // per wave and tile
    static constexpr int kUnit = kWaves * kKeys;
    // the waves' sums are joined through one tile of LDS each: in one round, or two halves of the values
    static constexpr int kRounds = kSplitRows * D * 4 > kStage ? 2 : 1;
    static_assert(kSplitRows * D * 4 / kRounds <= kStage, "a round's sums of a wave fit one tile");
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

// The batch's units and, with find(total) naming a unit, the request it
// belongs to and that request's first unit.  s_out: LDS for the answer.
template <int kThreads, class Find>
__device__ Units find_units(const AttentionLaunch& a, uint32_t unit, uint32_t& flags, Find find, uint64_t* s_wave,
                            uint64_t* s_out) {
    Units u{0, 0, a.requests};
    if (a.requests <= 64) {            // each wave by itself, a request in each lane
        const uint32_t lane = threadIdx.x & 63;
        const uint32_t n = lane < a.requests ? units_of(a, lane, unit, flags) : 0;         // below 2^24
        uint32_t x = n;
        for (uint32_t d = 1; d < a.requests; d <<= 1) {
            const uint32_t y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        u.total = uint64_t(__builtin_amdgcn_readlane(x, a.requests - 1)) * a.heads;
        const uint64_t at = find(u.total), first = uint64_t(x - n) * a.heads;
        const uint64_t here = __ballot(n && at >= first && at < first + uint64_t(n) * a.heads);
        if (!here) return u;
        u.request = __builtin_ctzll(here);
        u.first = uint64_t(__builtin_amdgcn_readlane(x - n, u.request)) * a.heads;
        return u;
    }
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

// Part p of P = min(total, kParts) begins at floor(total * p / P), so every one of them has at least one unit; no
// division in either case.
static_assert((kParts & (kParts - 1)) == 0, "a power of two");
__device__ __forceinline__ uint64_t part_begin(uint64_t total, uint32_t part) {
    return total < kParts ? min(uint64_t(part), total) : total * min(part, kParts) / kParts;
}
// The part that has unit u: the last p with floor(total * p / P) <= u.
__device__ __forceinline__ uint32_t part_of(uint64_t total, uint64_t u) {
    return total < kParts ? uint32_t(u) : uint32_t(quotient((u + 1) * kParts - 1, total));
}

// Workspace: part p's slot: 32 rows of D sums, then 32 maxima (base-2 units)
// and 32 sums of probabilities.
template <int D>
__device__ __forceinline__ float* part_slot(void* work, uint32_t part, uint32_t slot) {
    return static_cast<float*>(work) + (uint64_t(part) * 2 + slot) * kSplitRows * (D + 2);
}

// How a wave brings a tile of consecutive tokens of one head (the first a
// multiple of 8) from their pages into LDS.  Eight of them share a page, so
// addresses are worked out per eight, on the scalar unit, and a lane adds an
// offset that is the same for every tile.  What lies behind a request's last
// token may be anything, NaN too: there the last token stands in, and (as for
// strides too long for 32 bits) lanes have addresses of their own.
//
// A lane that looks up its own token instead leaves the wave waiting for the
// table within the tile's loads: 256 requests of 1000 tokens in e4m3 take 146
// us that way and 132 this way, 64 of 16384 at D = 256 411 and 375 (both before
// the loads were marked as read once).
template <int D, bool kE4m3>
struct Loader {
    using G = Split<D, kE4m3>;
    using T = Tile<D, kE4m3>;
    static constexpr int kGroups = G::kKeys / 8, kLoads = G::kStage / 2 / 1024, kLanes = 64 / T::kRowsPerLoad;
    static constexpr bool kShared = T::kRowsPerLoad <= 8;        // an instruction's rows share a page
    static_assert(G::kKeys % 16 == 0 && T::kRowsPerLoad <= 16, "an instruction brings rows of at most two eights");

    const __attribute__((address_space(4))) int32_t* table;
    uint32_t last;                       // the request's last token

    __device__ __forceinline__ Loader(const AttentionLaunch& a, uint32_t b, uint32_t len)
        : table((const __attribute__((address_space(4))) int32_t*)(a.table + int64_t(b) * a.table_stride)), last(len - 1) {}

    // The table's entries of the tile from `token` on, which has a token of the request.
    __device__ __forceinline__ void look_up(const AttentionLaunch& a, uint32_t token, int32_t (&e)[kGroups]) const {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) e[g] = table[min(token + 8 * g, last) >> a.page_shift];
    }

    // Bytes from the pool's beginning to the first token of the g-th eight.
    __device__ __forceinline__ int64_t place(const AttentionLaunch& a, uint32_t token, int g, int32_t entry,
                                             uint32_t& flags) const {
        bool bad = false;
        const uint32_t page = page_or_zero(entry, a.pages, &bad);
        if (bad) flags |= SKV_PAGES_PAGE;
        const uint32_t in = min(token + 8 * g, last & ~7u) & ((1u << a.page_shift) - 1);
        return int64_t(page) * a.page_stride + int64_t(in) * a.token_stride;
    }

    __device__ __forceinline__ void load(const AttentionLaunch& a, const uint8_t* kb, const uint8_t* vb, uint32_t token,
                                         const int32_t (&e)[kGroups], uint32_t lds, uint32_t lane, uint32_t& flags) const {
        if (token + G::kKeys <= last + 1 && a.token_stride >= 0 && a.token_stride < (1 << 26)) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int g = i * T::kRowsPerLoad / 8, g1 = kShared ? g : g + 1;
                const int64_t at = place(a, token, g, e[g], flags), at1 = place(a, token, g1, e[g1], flags);
                const uint32_t r = i * T::kRowsPerLoad + lane / kLanes, c = lane % kLanes;
                const uint32_t row = (r & 7) * uint32_t(a.token_stride), to = lds + i * 1024;
                const uint32_t ck = row + ((c ^ T::swizzle_k(r)) << 4), cv = row + ((c ^ T::swizzle_v(r)) << 4);
                if constexpr (kShared) {
                    load_lds16<true>(kb + at, ck, to);
                    load_lds16<true>(vb + at, cv, to + G::kStage / 2);
                } else {
                    load_lds16<true>(kb + (r & 8 ? at1 : at) + ck, to);
                    load_lds16<true>(vb + (r & 8 ? at1 : at) + cv, to + G::kStage / 2);
                }
            }
        } else {
            asm volatile("" : "+v"(lane));           // keeps what is worked out from it here, and registers free
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int g = i * T::kRowsPerLoad / 8, g1 = kShared ? g : g + 1;
                const int64_t at = place(a, token, g, e[g], flags), at1 = place(a, token, g1, e[g1], flags);
                const uint32_t r = i * T::kRowsPerLoad + lane / kLanes, c = lane % kLanes, to = lds + i * 1024;
                const uint32_t row = min(r & 7, last - min(token + (r & ~7u), last & ~7u));
                const int64_t o = (r & 8 && !kShared ? at1 : at) + int64_t(row) * a.token_stride;
                load_lds16<true>(kb + o + ((c ^ T::swizzle_k(r)) << 4), to);
                load_lds16<true>(vb + o + ((c ^ T::swizzle_v(r)) << 4), to + G::kStage / 2);
            }
        }
    }
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__((Split<D, kE4m3>::kWaves * 64), 1) attention_split(AttentionLaunch a, void* work) {
    using G = Split<D, kE4m3>;
    using L = Loader<D, kE4m3>;
    constexpr int kThreads = G::kWaves * 64;
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

    // a run of units of one (request, head): what is ours of it, what its rows need, the wave's tiles
    struct Run {
        Span sp;
        uint32_t b, head, units, t0, stop;
        bool whole;
        float raw;
        int first_limit, limit;          // the last key of query 0, of the lane's row
        const uint8_t *kb, *vb;
    };
    uint64_t u = begin, first = un.first;                          // the next run's first unit; its request's
    uint32_t b = un.request, units = units_of(a, b, G::kUnit, ignore);
    Span sp = span_of(a, b, ignore);
    bf16x8 q[D / 16];
    uint32_t stage = 1;
    auto find = [&](Run& x) __attribute__((always_inline)) -> bool {
        if (u >= end) return false;
        while (units == 0 || u - first >= uint64_t(units) * a.heads) {
            first += uint64_t(units) * a.heads;
            if (++b >= a.requests) return false;
            units = units_of(a, b, G::kUnit, ignore);
            sp = span_of(a, b, ignore);
        }
        x.sp = sp;
        x.b = b;
        x.head = uint32_t(quotient(u - first, units));
        const uint32_t c0 = uint32_t(u - first - uint64_t(x.head) * units);
        const uint32_t c1 = uint32_t(min(uint64_t(units), c0 + (end - u)));
        x.units = c1 - c0;
        x.whole = x.units == units;
        const uint32_t qi = row / a.group;
        x.raw = a.scale * (a.k_scale ? a.k_scale[x.head] : 1.0f);
        x.first_limit = a.causal ? int(sp.len) - int(sp.n) : int(sp.len) - 1;
        x.limit = row < sp.n * a.group ? x.first_limit + (a.causal ? int(qi) : 0) : -1;
        x.kb = a.k_pages + int64_t(x.head) * a.head_stride;
        x.vb = a.v_pages + int64_t(x.head) * a.head_stride;
        x.t0 = c0 * G::kUnit + wave * G::kKeys;
        x.stop = min(c1 * G::kUnit, sp.len);
        u += x.units;
        return true;
    };
    auto look_up = [&](const Run& x, uint32_t at, int32_t (&e)[L::kGroups]) __attribute__((always_inline)) {
        L(a, x.b, x.sp.len).look_up(a, at, e);
    };
    auto load_tile = [&](const Run& x, uint32_t at, const int32_t (&e)[L::kGroups], uint32_t to)
                         __attribute__((always_inline)) {
        L(a, x.b, x.sp.len).load(a, x.kb, x.vb, at, e, lds0 + to * G::kStage, lane, flags);
    };
    auto load_queries = [&](const Run& x) __attribute__((always_inline)) {
        const uint32_t qi = row / a.group, qg = row - qi * a.group;
        load_q<D, kE4m3>(a.q + int64_t(x.sp.row + qi) * a.q_token + int64_t(x.head * a.group + qg) * a.q_head,
                         row < x.sp.n * a.group, x.raw, lane, q);
    };

    Run run, ahead;
    bool more = find(run);
    if (more && run.t0 < run.stop) {
        int32_t e[L::kGroups];
        look_up(run, run.t0, e);
        load_tile(run, run.t0, e, stage ^ 1);
        load_queries(run);
    }
    bool first_run = true;
    while (more) {
        const float factor = run.raw == 0.0f ? 1.0f : fabsf(run.raw) * kLog2e;
        Rows<D> st;
        st.clear();
        // The wave's tiles of this run, each loaded while the one before is used; with the last one in hand, the
        // next run's first is on its way.  A wave without tiles here only does the latter.
        const bool some = run.t0 < run.stop;
        uint32_t t0 = run.t0;
        auto use_tile = [&]() __attribute__((always_inline)) {
            tile_step<D, kE4m3, G::kKeys / 32>(lane_k + stage * G::kStage, lane_v + stage * G::kStage, q, factor,
                                               int(t0) + G::kKeys - 1 > run.first_limit, run.limit - int(t0), lane, st);
        };
        int32_t e[L::kGroups];
        for (; t0 + G::kUnit < run.stop; t0 += G::kUnit) {
            stage ^= 1;
            look_up(run, t0 + G::kUnit, e);
            wait_loads();
            load_tile(run, t0 + G::kUnit, e, stage ^ 1);
            __builtin_amdgcn_sched_barrier(0);         // all loads on their way before the tile is used
            use_tile();
        }
        more = find(ahead);
        const bool coming = more && ahead.t0 < ahead.stop;
        if (coming) look_up(ahead, ahead.t0, e);
        if (some) {
            stage ^= 1;
            wait_loads();
        }
        if (coming) load_tile(ahead, ahead.t0, e, stage ^ 1);
        if (some) use_tile();
        if (coming) load_queries(ahead);
        // what is joined now, before the next one's state takes its place
        const Span was = run.sp;
        const uint32_t was_b = run.b, was_head = run.head, rows = was.n * a.group, slot_at = !first_run;
        const bool was_whole = run.whole;
        const int was_limit = run.first_limit;
        first_run = false;
        run = ahead;
        // the sums of each wave to LDS, into the stage it used last; then every thread takes some of a row's values
        const float vs = a.v_scale ? a.v_scale[was_head] : 1.0f;
        float* slot = part_slot<D>(work, part, slot_at);
        if (row < rows) {
            const float l = half_sum(st.l);
            if (lane < 32) {
                s_m[wave][row] = st.m * factor;
                s_l[wave][row] = l;
            }
        }
        if (lane == 0) s_stage[wave] = stage;
        if (tid == 0) s_bad = 0;
#pragma unroll
        for (int half = 0; half < G::kRounds; ++half) {
            constexpr int kDims = D / G::kRounds, kQuads = kDims / 4;          // of a round
            if (row < rows) {
                f32x4* mine = reinterpret_cast<f32x4*>(&s_tiles[wave][stage][0]) + row * kQuads;
#pragma unroll
                for (int t = 0; t < kDims / 32; ++t)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const f32x16& o = st.o[half * (kDims / 32) + t];
                        mine[(8 * t + 2 * (r / 4) + (lane >> 5)) ^ (row & 7)] = f32x4{o[r], o[r + 1], o[r + 2], o[r + 3]};
                    }
            }
            __syncthreads();
            for (uint32_t i = tid; i < rows * kQuads; i += kThreads) {
                const uint32_t r = i / kQuads, f = i % kQuads, dim = half * kDims + 4 * f;
                float top = s_m[0][r], l = 0.0f;
                for (int w = 1; w < G::kWaves; ++w) top = fmaxf(top, s_m[w][r]);
                f32x4 o{0, 0, 0, 0};
                for (int w = 0; w < G::kWaves; ++w) {
                    const float k = exp2_diff(s_m[w][r], top);
                    l += k * s_l[w][r];
                    if (s_m[w][r] != -INFINITY)        // else all its keys were hidden, and o may be 0 * NaN
                        o += k * reinterpret_cast<const f32x4*>(&s_tiles[w][s_stage[w]][0])[r * kQuads + (f ^ (r & 7))];
                }
                if (was_whole) {
                    const uint32_t ri = r / a.group, qh = was_head * a.group + r - ri * a.group;
                    const bool none = was_limit + (a.causal ? int(ri) : 0) < 0;
                    const bool nan = store_out(a, was.row + ri, qh, dim, none ? f32x4{0, 0, 0, 0} : o * (vs / l));
                    if (nan && a.causal && was.n > 1) atomicOr(&s_bad, 1u << r);
                    if (dim == 0) store_lse(a, was.row + ri, qh, none ? -INFINITY : top, none ? 1.0f : l);
                } else {
                    *reinterpret_cast<f32x4*>(slot + r * D + dim) = o;
                    if (dim == 0) {
                        slot[kSplitRows * D + r] = top;
                        slot[kSplitRows * (D + 1) + r] = l;
                    }
                }
            }
            __syncthreads();
        }
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
    for (uint32_t d = 1; d < 64 && d < a.requests; d <<= 1) {
        before += __shfl_xor(before, d);
        all += __shfl_xor(all, d);
    }
    if ((tid & 63) == 0) {          // (of a power of two of lanes that holds them all)
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
    const uint32_t p0 = part_of(all, u0), p1 = part_of(all, u1 - 1);
    if (p0 == p1) return;              // finished by one workgroup
    const Span sp = span_of(a, b, flags);
    const uint32_t rows = sp.n * a.group, late = part_begin(all, p0) < u0;       // p0's slot: its first or its last
    const int first_limit = a.causal ? int(sp.len) - int(sp.n) : int(sp.len) - 1;
    const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
    // blockIdx.z: 256 of the rows' quads of values
    const uint32_t i = blockIdx.z * 256 + tid;
    if (i < rows * (D / 4)) {
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

template <int D, bool kE4m3>
hipError_t launch(const AttentionLaunch& a, void* work, hipStream_t stream) {
    attention_split<D, kE4m3><<<kParts, Split<D, kE4m3>::kWaves * 64, 0, stream>>>(a, work);
    const uint32_t quads = a.max_new * a.group * (D / 4);
    attention_combine<D, kE4m3><<<dim3(a.heads, a.requests, std::max(1u, (quads + 255) / 256)), 256, 0, stream>>>(a, work);
    return hipGetLastError();
}

}  // namespace

// Where no request can have more than 32 rows this kernel takes the batch;
// else the tile kernel takes all of it, requests with few rows too: of their
// tiles only the waves that have rows compute, which for single tokens still
// reads at 0.6 (e4m3) to 1.0 (long bf16 contexts) of this kernel's rate, and
// saves a batch of chunks a second pair of launches.
bool attention_few_rows(const AttentionLaunch& a) { return a.max_new * uint64_t(a.group) <= kSplitRows; }

uint64_t split_work_bytes(uint32_t head_dim) { return uint64_t(kParts) * 2 * kSplitRows * (head_dim + 2) * 4; }

hipError_t launch_split(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void* work, hipStream_t stream) {
    const bool e4m3 = dtype == SKV_E4M3;
    switch (head_dim) {
        case 64: return e4m3 ? launch<64, true>(a, work, stream) : launch<64, false>(a, work, stream);
        case 128: return e4m3 ? launch<128, true>(a, work, stream) : launch<128, false>(a, work, stream);
        default: return e4m3 ? launch<256, true>(a, work, stream) : launch<256, false>(a, work, stream);
    }
}

}  // namespace skv
