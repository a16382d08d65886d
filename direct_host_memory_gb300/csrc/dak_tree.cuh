// The attention of drafted trees (dak_attn_tree): what its two kernels share, dak_tree.cu's for many query
// rows a kv head and dak_tree_few.cu's for few. Work is cut on the device from the lengths, so that a
// captured call follows them: the chunks of all (request, kv head, 256-row tile) lie on one line,
// request-major, each with its cost, and the line is cut into equal ranges, a CTA each. A tile cut by
// no range's end is finished where it is; the others leave partial results (at most two a range, whatever
// the batch) to a merge (dak_tree.cu), which takes those of a tile in order. Where tiles are short they are
// not cut, but belong to the range with their middle. The cuts go by lengths and SM count alone, so that
// results do not depend on the tiers: the host's slabs are the line's beginning, and where its ranges are
// more CTAs than may read the host at once, those take several each.
#pragma once
#include "dak_device.cuh"

namespace dak {

// Cost of a chunk for a tile of one or two 128-row halves.
constexpr unsigned kTreeTwoCost = 3, kTreeOneCost = 2;
constexpr unsigned kTreeSnapRange = 24;  // ranges from here on cut off no tile's first or last chunk alone

struct TreeHead {  // of range r, the partials of the tile that begins in it and ends in a later one
    int b, g, tile, pieces;  // pieces 0: there is no such tile
    int n, len, keys, unused;  // TreeRequest's
};

struct TreeParams {
    const __nv_bfloat16* Q;  // [B][T][Hq][D]
    const int* lens;
    const int* n_new;                // or null
    const unsigned long long* mask;  // or null: a chain
    long long mask_pitch;
    void* O;
    int o_fp32;
    float* o_part;    // [2 * ranges][part_rows][D]: range r's piece of a tile that began before it, then of one that ends after it
    float2* ml_part;  // [2 * ranges][part_rows]: reference (log2 domain), sum
    TreeHead* heads;  // [ranges]
    const uint8_t* kv[2];  // host tier (device-visible), HBM tier
    long long head_bytes;
    int B, T, W, Hq, Hkv, G, L, h_s;  // W: mask words of a token
    int host_requests;  // h_s / Hkv
    int mpt;        // tokens of a 128-row half: 128 / G
    int inv_G, inv_mpt;  // 2^16 / G and 2^16 / mpt rounded up: (r * inv) >> 16 is the quotient for any r here
    int q_tokens;   // tokens that a copy of Q brings: min(mpt, T)
    int part_rows;  // of a tile's partials: half * 128 + row in it, at most
    int wide;       // O is 32-byte aligned
    int ranges, host_ctas, slab_chunks;
    unsigned slack;  // how much longer the longest range may be for whole tiles (tree_plan)
    unsigned tile_cost, min_range;  // of a tile by itself (rows' way in, first chunk's latency, results' way out); of a range, at least
    int in_flight[2];  // copies of a CTA that have not landed, by tier
    float scale_log2;
    DevStatus* st;
};

// A request as the plan sees it.
struct TreeRequest {
    int len, n;                   // cached rows, drafted tokens
    int keys, chunks;             // rows with the drafts, chunks of 64 keys
    int tiles, twos;              // tiles, those of two halves
    unsigned two, one, slab;      // cost of a tile of two halves, of one, of all tiles of a kv head
};

__device__ __forceinline__ TreeRequest tree_request(const TreeParams& p, int len, int n) {
    TreeRequest q;
    q.len = len;
    q.n = n;
    q.keys = min(q.len + n, p.L);
    q.chunks = (q.keys + 63) >> 6;
    const int halves = ((n + p.mpt - 1) * p.inv_mpt) >> 16;
    q.twos = halves >> 1;
    q.tiles = (halves + 1) >> 1;
    q.two = p.tile_cost + kTreeTwoCost * q.chunks;
    q.one = p.tile_cost + kTreeOneCost * q.chunks;
    q.slab = q.twos * q.two + (halves & 1) * q.one;
    return q;
}
__device__ __forceinline__ TreeRequest tree_request(const TreeParams& p, int b) {
    const int n = p.n_new ? p.n_new[b] : p.T;
    return tree_request(p, min(max(p.lens[b], 0), p.L), min(max(n, 0), p.T));
}

// n / d for n below 2^31: the float quotient is off by at most 2^-22 of itself, 2^9; what the remainder says of
// that (off by less than one) is added, and the remainder then puts the last step right. (An integer
// division is dozens of instructions that run for the first time.)
__device__ __forceinline__ unsigned tree_quotient(unsigned n, unsigned d) {
    const float inv = __fdividef(1.f, static_cast<float>(d));
    unsigned q = static_cast<unsigned>(static_cast<float>(n) * inv);
    q += static_cast<int>(static_cast<float>(static_cast<int>(n - q * d)) * inv);
    const int r = static_cast<int>(n - q * d);
    return q + (r >= static_cast<int>(d)) - (r < 0);
}

struct TreePlan {
    unsigned len;                // of a range
    bool whole;                  // ranges take whole tiles, those whose middles lie in them
    int ranges, host_ranges;     // host_ranges: those that touch the host's slabs
    // the first 32 requests, a lane each, which a warp finds without loads:
    TreeRequest own;
    unsigned own_end;            // where its tiles end on the line
};

// By one warp, as are the functions of TreeWalk.
__device__ __forceinline__ TreePlan tree_plan(const TreeParams& p) {
    constexpr unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31, bh = p.host_requests;
    TreePlan x;
    x.own.slab = 0;
    if (lane < p.B) x.own = tree_request(p, lane);
    x.own_end = x.own.slab * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(all, x.own_end, o);
        if (lane >= o) x.own_end += v;
    }
    unsigned total = __shfl_sync(all, x.own_end, 31), host = 0;
    const auto largest = [](const TreeRequest& q) { return q.tiles == 0 ? 0u : q.twos > 0 ? q.two : q.one; };  // of its tiles
    unsigned tile = lane < p.B ? largest(x.own) : 0u;
    const auto host_part = [&](int b, unsigned slab) { return b < bh ? slab * p.Hkv : b == bh ? slab * (p.h_s - bh * p.Hkv) : 0u; };
    if (p.h_s > 0) host = host_part(lane, x.own.slab);
    if (p.B > 32) {
        unsigned more = 0;
#pragma unroll 1
        for (int b = 32 + lane; b < p.B; b += 32) {
            const TreeRequest q = tree_request(p, b);
            more += q.slab * p.Hkv;
            host += host_part(b, q.slab);
            tile = max(tile, largest(q));
        }
        total += __reduce_add_sync(all, more);
    }
    if (p.h_s > 0) host = __reduce_add_sync(all, host);
    tile = max(__reduce_max_sync(all, tile), 1u);
    x.len = max(tree_quotient(total + p.ranges - 1, p.ranges), min(p.min_range, tile));
    x.ranges = static_cast<int>(tree_quotient(total + x.len - 1, x.len));
    // The longest range of whole tiles is about len rounded up to largest ones: where that costs less than what
    // cutting does (a cut tile's second start, its partial results, the merge), no tile is cut.
    unsigned most = tree_quotient(x.len, tile) * tile;
    if (most < x.len) most += tile;
    x.whole = most <= x.len + p.slack;
    x.host_ranges = static_cast<int>(tree_quotient(host + x.len - 1, x.len));
    return x;
}

// A tile on the line, and the part of it that a range takes.
struct TreeWalk {
    int b, g, tile;
    unsigned at;  // where the tile begins
    TreeRequest q;

    __device__ __forceinline__ bool two() const { return tile < q.twos; }
    __device__ __forceinline__ unsigned end() const { return at + (two() ? q.two : q.one); }
    // The tile at position x, which lies on the line.
    __device__ __forceinline__ void find(const TreeParams& p, const TreePlan& plan, unsigned x) {
        constexpr unsigned all = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        unsigned base = 0;  // where the request's tiles begin
        unsigned hit = __ballot_sync(all, x < plan.own_end);
        if (hit) {
            b = __ffs(hit) - 1;
            base = __shfl_sync(all, plan.own_end - plan.own.slab * p.Hkv, b);
        } else {
            base = __shfl_sync(all, plan.own_end, 31);
            b = 32;
#pragma unroll 1
            for (int b0 = 32; b0 < p.B; b0 += 32) {
                const unsigned cost = b0 + lane < p.B ? tree_request(p, b0 + lane).slab * p.Hkv : 0u;
                unsigned incl = cost;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned v = __shfl_up_sync(all, incl, o);
                    if (lane >= o) incl += v;
                }
                hit = __ballot_sync(all, x < base + incl);
                if (hit) {
                    const int l = __ffs(hit) - 1;
                    b = b0 + l;
                    base += __shfl_sync(all, incl - cost, l);
                    break;
                }
                base += __shfl_sync(all, incl, 31);
            }
        }
        load(p, plan);
        g = static_cast<int>(tree_quotient(x - base, q.slab));
        at = base + g * q.slab;
        tile = min(static_cast<int>(tree_quotient(x - at, q.two)), q.twos);
        at += tile * q.two;
    }
    __device__ __forceinline__ void load(const TreeParams& p, const TreePlan& plan) {
        if (b < 32) {
            const int n = __shfl_sync(0xffffffffu, plan.own.n, b);
            q = tree_request(p, __shfl_sync(0xffffffffu, plan.own.len, b), n);
        } else {
            q = tree_request(p, b);
        }
    }
    // The next tile; past the line's end b is B.
    __device__ __forceinline__ void next(const TreeParams& p, const TreePlan& plan) {
        at = end();
        if (++tile < q.tiles) return;
        tile = 0;
        if (++g < p.Hkv) return;
        g = 0;
        while (++b < p.B) {
            load(p, plan);
            if (q.tiles > 0) break;
        }
    }
    // The first chunk that does not belong to the ranges before position x.
    __device__ __forceinline__ int cut(const TreeParams& p, const TreePlan& plan, unsigned x) const {
        if (x <= at) return 0;
        if (x >= end()) return q.chunks;
        if (plan.whole) return 2 * (x - at) <= end() - at ? 0 : q.chunks;
        const unsigned in = max(x - at, p.tile_cost) - p.tile_cost;
        const int t = static_cast<int>(two() ? (in + kTreeTwoCost - 1) / kTreeTwoCost : (in + kTreeOneCost - 1) / kTreeOneCost);
        const int least = plan.len >= kTreeSnapRange ? 2 : 1;
        return t < least ? 0 : q.chunks - t < least ? q.chunks : t;
    }
};

// Draft s of the request is seen by token t, for the 64 keys from key0 on.
__device__ __forceinline__ unsigned long long tree_bits(const TreeParams& p, const TreeRequest& q, int b, int t, int key0) {
    const int d0 = key0 - q.len;  // draft of the first key
    const int n = min(q.keys - q.len, p.mask ? p.T : t + 1);  // drafts that may be seen
    unsigned long long v = ~0ull;
    if (p.mask) {
        const unsigned long long* w = p.mask + b * p.mask_pitch + static_cast<long long>(t) * p.W;
        if (d0 < 0) {
            v = d0 > -64 ? w[0] << -d0 : 0;
        } else {
            const int i = d0 >> 6, sh = d0 & 63;
            v = i < p.W ? w[i] >> sh : 0;
            if (sh && i + 1 < p.W) v |= w[i + 1] << (64 - sh);
        }
    }
    const int valid = n - d0;  // keys before the drafts that may not be seen
    if (valid < 64) v &= valid > 0 ? (1ull << valid) - 1 : 0;
    if (d0 < 0) v |= d0 > -64 ? (1ull << -d0) - 1 : ~0ull;
    return v;
}

// Whether a token sees any row at all.
__device__ __forceinline__ bool tree_sees(const TreeParams& p, const TreeRequest& q, int b, int t) {
    if (q.len > 0) return true;
    unsigned long long any = 0;
    for (int k = 0; k < q.keys; k += 64) any |= tree_bits(p, q, b, t, k);
    return any != 0;
}

// Of a bf16 pair the elements that are infinite or NaN.
__device__ __forceinline__ uint32_t tree_not_finite(uint32_t a) {
    return ((a & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((a & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// Elements 8 c to 8 c + 7 of a row of V.
__device__ __forceinline__ const uint4* tree_v_piece(const TreeParams& p, int b, int g, int D, int key, int c) {
    const long long slab = static_cast<long long>(b) * p.Hkv + g;
    const uint8_t* base = slab < p.h_s ? p.kv[0] + slab * p.head_bytes : p.kv[1] + (slab - p.h_s) * p.head_bytes;
    return reinterpret_cast<const uint4*>(base) + (static_cast<long long>(key >> 6) * 2 * 64 + 64 + (key & 63)) * (D / 8) + (c ^ (key & 7));
}

// What is infinite or NaN in N consecutive bf16 values, added to `to`: the result of an element that a token sees,
// whatever the weights (with infinities of both signs NaN), where its sum with weights would be NaN as soon as one
// of them, or a part of one, is rounded to zero.
template <class Words>
__device__ __forceinline__ void add_not_finite(float* to, const Words* at) {
    const Words v = *at;
    const uint32_t* word = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(Words) / 4); ++k) {
        const uint32_t odd = tree_not_finite(word[k]);
        if (odd & 0xFFFFu) to[2 * k] += bf_lo(word[k]);
        if (odd >> 16) to[2 * k + 1] += bf_hi(word[k]);
    }
}

// The ranges that a CTA takes: the one of its number, unless more ranges touch the host than CTAs may.
struct TreeTurn {
    int first, end, step;
};
__device__ __forceinline__ TreeTurn tree_turn(const TreeParams& p, const TreePlan& plan) {
    const int c = blockIdx.x;
    if (plan.host_ranges <= p.host_ctas) return {c, plan.ranges, p.ranges};
    if (c < p.host_ctas) return {c, plan.host_ranges, p.host_ctas};
    return {plan.host_ranges + c - p.host_ctas, plan.ranges, p.ranges};
}

// What the merge is told of the tile at hand, if it begins in range r and ends in a later one.
__device__ __forceinline__ void tree_head(const TreeParams& p, const TreePlan& plan, const TreeWalk& w, int r, int c0, int c1) {
    if (c0 > 0 || c1 == w.q.chunks) return;
    int last = static_cast<int>(tree_quotient(w.end() - 1, plan.len));  // the range with the tile's last chunk
    while (w.cut(p, plan, last * plan.len) == w.q.chunks) --last;
    p.heads[r] = TreeHead{w.b, w.g, w.tile, last - r + 1, w.q.n, w.q.len, w.q.keys, 0};
}

// Drafted rows that would lie behind the cache, reported once a request.
__device__ __forceinline__ void tree_report(const TreeParams& p, const TreeWalk& w, int c0) {
    if (w.g == 0 && w.tile == 0 && c0 == 0 && w.q.keys - w.q.len < w.q.n) {
        report(p.st, DAK_ERR_BOUNDS, (0x7EEEull << 32) | static_cast<unsigned>(w.b));
    }
}

// Query rows a kv head that tree_few_kernel takes, at most (32 requests over 7K to 8K, 8 kv heads of 128: 16 rows
// 150 us there, 32 rows 149 by tree_kernel; 24 or 32 there 330, their O^T out of registers; one request over 4K,
// heads of 64: 16 rows 10.2 us there, 32 12.2 by tree_kernel).
constexpr int kTreeFewRows = 16;
// Ranges (CTAs) of tree_few_kernel on this device, and its launch; the merge is the caller's.
int tree_few_ctas(int rows);
cudaError_t launch_tree_few(const TreeParams& p, int rows, int D, cudaStream_t s);

}  // namespace dak
