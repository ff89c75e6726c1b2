// skv_attention_tiles.hip -- attention of chunks and prompts over a paged
// cache (gfx950): 128 query rows share the keys.
//
//   attention_tiles         tiles of rows, or pieces of their keys
//   attention_tile_combine  joins the pieces
#include "skv_attention.h"

namespace skv {
namespace {

// A tile of 64 keys, for a wave that computes the scores of the next one
// while it turns this one's into probabilities and adds their product with V:
// matrix and vector instructions of one wave then overlap.  A tile is taken in
// four steps of 16 keys, each with a quarter of the next scores' products.
//
// m need not be the maximum: it is a reference that the sums are relative
// to, moved only when a score passes it by 2^8 (sums and products then stay
// below 2^8 times the number of keys, far from the end of the range), so o is
// rescaled a few times per row and not with every new maximum.  The price: a
// row's largest probability is no longer exactly 1 and is rounded to bf16 like
// the others (results 0.0021 of their 2-norm off in place of 0.0017, of which
// the result's own rounding is 0.0016).
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

// A workgroup takes 128 query rows of one (request, KV head): new tokens x
// the head's query heads, in that order, so all of them share the keys it
// streams through LDS, 64 at a time, two tiles deep.  Each of its four waves
// owns 32 rows.  (64 rows a wave halve the reads of K and V from LDS, but
// the scores then lie in accumulation registers that vector instructions
// reach only through copies: 1.34 ms against 1.05 for 2048 tokens at 32768.)
//
// Work is cut on the device, where the lengths are, so that all of it runs at
// once where it can: with `slots` workgroups at a time and fewer (tile of
// rows, head)s than half of them, into pieces of (whole work) / (slots -
// tiles), which with the tiles' remainders fill the slots; with more, only
// tiles of over twice an even share are cut.  attention_tile_combine joins the
// pieces' unnormalized sums; tiles of one piece are finished where they are
// computed.  Requests with the most keys come first, and of a request the
// last rows, which see the most.  The heads come fastest: eight consecutive
// workgroups go to the eight XCDs, so with 8 KV heads (or a divisor or
// multiple) each XCD's L2 holds the keys of its own heads.
//
// Bound by the matrix units and the power they may draw: 2048 rows x 4 heads
// at 32768 keys in 0.94 to 1.10 ms (1140 to 970 TFLOP/s; the library's bf16
// product of 8192 reaches 1219), matrix units busy 63% of the cycles at 2.0
// GHz; e4m3 pages 1000, head_dim 64 790, 256 910 TFLOP/s.
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
    Span span;                         // its
    uint32_t tiles, pieces;            // tiles of rows of the request; pieces of its longest one
    uint32_t index;                    // among the request's (tile, piece)s, or its tiles for the join
    uint32_t slot;                     // first workspace slot of the request (where pieces > 1)
    uint32_t piece_tiles;              // tiles of keys in a piece
    uint32_t total;                    // all there are to find, where that is known (else the most there can be)
};

struct TileSearch {
    uint64_t sum[8];
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
    auto measure = [&](const Span& sp, uint32_t& tiles, uint32_t& keys) __attribute__((always_inline)) {
        tiles = (sp.n * a.group + kTileRows - 1) / kTileRows;
        keys = tiles ? (keys_for(a, sp, ~0u) + kTileKeys - 1) / kTileKeys : 0;
    };
    auto piece_of = [&](uint64_t all, uint64_t count) __attribute__((always_inline)) -> uint32_t {
        const uint64_t share = count < kSlots / 2 ? kSlots - count : kSlots / 2;
        return max(kLeastPiece, uint32_t(quotient(all + share - 1, share)));
    };
    if (a.requests <= 64) {
        // each wave by itself, a request in each lane: what lies before a request is summed over the others directly
        Span sp{0, 0, 0};
        uint32_t tiles = 0, keys = 0;
        if (lane < a.requests) {
            sp = span_of(a, lane, flags);
            measure(sp, tiles, keys);
        }
        uint64_t all = uint64_t(tiles) * keys;
        uint32_t count = tiles;
        for (uint32_t d = 1; d < 64 && d < a.requests; d <<= 1) {
            all += __shfl_xor(all, d);
            count += __shfl_xor(count, d);
        }
        // (over a power of two of lanes that holds them all)
        all = uniform(all);
        count = __builtin_amdgcn_readfirstlane(count);
        const uint32_t piece = piece_of(all * a.heads, uint64_t(count) * a.heads);
        const uint32_t pieces = max(1u, (keys + piece - 1) / piece);
        const uint32_t slots = pieces > 1 ? tiles * pieces : 0;
        const uint32_t own = kJoin ? (pieces > 1 ? tiles : 0) : tiles * pieces;
        uint32_t begin = 0, slot = 0, total = 0;
        for (uint32_t x = 0; x < a.requests; ++x) {
            const uint32_t k = __builtin_amdgcn_readlane(keys, x), n = __builtin_amdgcn_readlane(own, x);
            const bool first = k > keys || (k == keys && x < lane);         // the longest first
            begin += first ? n : 0;
            slot += first ? __builtin_amdgcn_readlane(slots, x) : 0;
            total += n;
        }
        TileWork t{};
        t.total = total;
        t.request = a.requests;
        const uint64_t here = __ballot(own && index >= begin && index - begin < own);
        if (!here) return t;
        const int at = __builtin_ctzll(here);
        t.request = at;
        t.span = Span{uint32_t(__builtin_amdgcn_readlane(sp.row, at)), uint32_t(__builtin_amdgcn_readlane(sp.n, at)),
                      uint32_t(__builtin_amdgcn_readlane(sp.len, at))};
        t.tiles = __builtin_amdgcn_readlane(tiles, at);
        t.pieces = __builtin_amdgcn_readlane(pieces, at);
        t.index = index - __builtin_amdgcn_readlane(begin, at);
        t.slot = __builtin_amdgcn_readlane(slot, at);
        t.piece_tiles = piece;
        return t;
    }
    uint64_t all = 0, count = 0;
    uint32_t tiles = 0, keys = 0, ignore = 0;
    for (uint32_t b = tid; b < a.requests; b += 256) {
        measure(span_of(a, b, flags), tiles, keys);
        all += uint64_t(tiles) * keys;
        count += tiles;
    }
    for (uint32_t d = 32; d; d >>= 1) {
        all += __shfl_xor(all, d);
        count += __shfl_xor(count, d);
    }
    if (lane == 0) {
        s.sum[wave] = all;
        s.sum[4 + wave] = count;
    }
    if (tid == 0) s.found[0] = a.requests;
    __syncthreads();
    all = (s.sum[0] + s.sum[1] + s.sum[2] + s.sum[3]) * a.heads;
    count = (s.sum[4] + s.sum[5] + s.sum[6] + s.sum[7]) * a.heads;
    const uint32_t piece = piece_of(all, count);
    uint32_t before = 0, slot0 = 0;
    for (uint32_t base = 0; base < a.requests; base += 256) {
        const uint32_t b = base + tid, n = min(256u, a.requests - base);
        if (b >= a.requests) tiles = keys = 0;
        else if (a.requests > 256) measure(span_of(a, b, ignore), tiles, keys);
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
    t.total = a.requests <= 256 ? __builtin_amdgcn_readfirstlane(before) : ~0u;
    t.request = __builtin_amdgcn_readfirstlane(s.found[0]);
    if (t.request >= a.requests) return t;
    t.index = __builtin_amdgcn_readfirstlane(s.found[1]);
    t.slot = __builtin_amdgcn_readfirstlane(s.found[2]);
    t.piece_tiles = __builtin_amdgcn_readfirstlane(piece);
    t.span = span_of(a, t.request, ignore);
    measure(t.span, t.tiles, keys);
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

// kOnce: every request has one tile of rows, so its keys are read by one
// workgroup and marked so: 9 new tokens over each of 64 caches of 16384 in bf16
// take 682 us for 752 at D = 128, 388 for 425 at D = 64, 612 for 625 at D =
// 256.  Keys that tiles share must not be: a chunk of 2048 at 32768 takes 1051
// us with the mark and 1037 without.
template <int D, bool kE4m3, bool kOnce>
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
    const Span sp = at.span;
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
                    load_lds16<kOnce>(from + w.at[(i * T::kRowsPerLoad) >> 3], offset, to + i * 1024);
                else
                    load_lds16<kOnce>(from + (in < 8 ? w.at[0] : w.at[1]) + offset, to + i * 1024);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t r = wave * kWaveRows + i * T::kRowsPerLoad + lane / kLanes, c = lane % kLanes;
                load_lds16<kOnce>(from + token_at(a, b, min(at + r, sp.len - 1), flags) +
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

// An item is kJoinRows rows of a (tile of rows, head) that is in pieces, four
// values a thread; a fixed number of workgroups goes through them, since
// there are mostly few or none (1024 of them look it up in 4 us, one for
// every possible item in 11).
template <int D>
constexpr uint32_t kJoinRows = 1024 / D;

template <int D, bool kE4m3>
__global__ void __launch_bounds__(256) attention_tile_combine(AttentionLaunch a, void* work, uint32_t per_tile) {
    __shared__ TileSearch s_search;
    __shared__ uint32_t s_bad;
    const uint32_t tid = threadIdx.x;
    uint32_t flags = 0;
    uint32_t total = ~0u;              // of tiles in pieces
    for (uint32_t item = blockIdx.x; item / per_tile / a.heads < total; item += gridDim.x) {
        const uint32_t from = kJoinRows<D> * (item % per_tile), head = item / per_tile % a.heads;
        __syncthreads();
        if (tid == 0) s_bad = 0;
        const TileWork at = find_work<tile_slots(D), true>(a, item / per_tile / a.heads, flags, s_search);
        if (at.request >= a.requests) return;
        total = at.total;
        const Span sp = at.span;
        const uint32_t row0 = (at.tiles - 1 - at.index) * kTileRows;
        const uint32_t rows = min(kTileRows, sp.n * a.group - row0);
        const uint32_t keys = keys_for(a, sp, row0 + kTileRows - 1), span = at.piece_tiles * kTileKeys;
        const uint32_t pieces = (keys + span - 1) / span, count = from < rows ? min(kJoinRows<D>, rows - from) : 0;
        const uint64_t slot0 = at.slot + uint64_t(at.index) * at.pieces;
        if (count == 0 || keys <= span || (slot0 + pieces) * a.heads > a.slots) continue;
        const float vs = a.v_scale ? a.v_scale[head] : 1.0f;
        if (tid < count * (D / 4)) {
            const uint32_t r = from + tid / (D / 4), f = tid % (D / 4);
            const Joined j = join_parts<D>(0, pieces, kTileRows, r, f, [&](uint32_t p) -> const float* {
                return tile_slot<D>(work, (slot0 + p) * a.heads + head);
            });
            const uint32_t row = row0 + r, qi = row / a.group, qh = head * a.group + row - qi * a.group;
            const bool none = keys_for(a, sp, row) == 0;
            const bool nan = store_out(a, sp.row + qi, qh, 4 * f, none ? f32x4{0, 0, 0, 0} : j.o * (vs / j.l));
            if (nan && a.causal) atomicOr(&s_bad, 1u << (r - from));
            if (f == 0) store_lse(a, sp.row + qi, qh, none ? -INFINITY : j.m, none ? 1.0f : j.l);
        }
        __syncthreads();
        for (uint32_t r = 0, bad = s_bad; r < count; ++r)
            if ((bad >> r & 1) && r % 4 == (tid >> 6)) {
                const uint32_t row = row0 + from + r;
                row_plain<D, kE4m3>(a, at.request, sp, row / a.group, head * a.group + row % a.group, flags);
            }
    }
}

// Workspace slots of the tile kernel: as many as find_work gives out, or as the longest table can need.
uint32_t slots_of(const AttentionLaunch& a, int head_dim) {
    const uint64_t keys = ((uint64_t(a.width) << a.page_shift) + kTileKeys - 1) / kTileKeys;
    const uint64_t most = uint64_t(tile_bound(a)) * a.heads * ((keys + kLeastPiece - 1) / kLeastPiece);
    return uint32_t(std::min<uint64_t>(2 * tile_slots(head_dim), most));
}

template <int D, bool kE4m3>
hipError_t launch(AttentionLaunch a, void* work, hipStream_t stream) {
    a.slots = slots_of(a, D);
    const uint32_t extra = tile_slots(D) / a.heads + 1;
    const uint64_t rows = uint64_t(a.max_new) * a.group;                       // of a request, at most
    const uint32_t per_tile = uint32_t(std::min<uint64_t>(kTileRows, rows) + kJoinRows<D> - 1) / kJoinRows<D>;
    const uint32_t grid = (tile_bound(a) + extra) * a.heads;
    if (rows <= kTileRows) attention_tiles<D, kE4m3, true><<<grid, 256, 0, stream>>>(a, work);
    else attention_tiles<D, kE4m3, false><<<grid, 256, 0, stream>>>(a, work);
    attention_tile_combine<D, kE4m3><<<std::min(1024u, extra * a.heads * per_tile), 256, 0, stream>>>(a, work, per_tile);
    return hipGetLastError();
}

}  // namespace

uint64_t tiles_work_bytes(const AttentionLaunch& a, uint32_t head_dim) {
    return std::max<uint64_t>(256, uint64_t(slots_of(a, int(head_dim))) * kTileRows * (head_dim + 2) * 4);
}

hipError_t launch_tiles(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void* work, hipStream_t stream) {
    const bool e4m3 = dtype == SKV_E4M3;
    switch (head_dim) {
        case 64: return e4m3 ? launch<64, true>(a, work, stream) : launch<64, false>(a, work, stream);
        case 128: return e4m3 ? launch<128, true>(a, work, stream) : launch<128, false>(a, work, stream);
        default: return e4m3 ? launch<256, true>(a, work, stream) : launch<256, false>(a, work, stream);
    }
}

}  // namespace skv
