// Decode attention of a tree (or chain) of drafted tokens per request over a placed KV cache,
// dak_attn_tree: o[b,t,h] = softmax(scale q[b,t,h] K^T) V over the rows before the drafts and those
// drafts that the token's mask names. The tokens' query heads of one kv head are the rows of a tile
// (row t * G + h), so that the cache, which dak_attn streams once per token, is streamed once
// for all of them; 64 keys a step on the tcgen05 tensor cores, as in the prefix pass, whose
// comment says how (dak_prefix.cu; what both use: dak_umma_attn.cuh).
//
// Work is cut on the device from the lengths, so that a captured call follows them: the chunks of
// all (request, kv head, 256-row tile) lie on one line, request-major, each with its cost, and
// the line is cut into as many equal ranges as there are SMs, a CTA each. A tile cut by no range's
// end is finished where it is; the others leave partial results (at most two a range, whatever the
// batch) to a second kernel, which merges those of a tile in order. The cuts go by lengths and SM
// count alone, so that results do not depend on the tiers: the host's slabs are the line's beginning,
// and where its ranges are more CTAs than may read the host at once, those take several each.
//
// A range goes through its tiles without the CTA's warps meeting: copies run ahead over the
// tile's end, up to what the ring holds.
#include <algorithm>
#include <cmath>

#include "dak_umma_attn.cuh"

namespace dak {

constexpr int kTreeSoftmax = 2 * 128;             // two streams, a thread a row
constexpr int kTreeThreads = kTreeSoftmax + 3 * 32;  // and copies, each stream's products
constexpr int kTreeRows = 256;                    // of a tile
// Cost of a chunk for a tile of one or two 128-row halves, and of a tile by itself (its rows' way in, the
// first chunk's latency, the results' way out).
constexpr unsigned kTreeTwoCost = 3, kTreeOneCost = 2, kTreeTileCost = 6;
constexpr unsigned kTreeMinRange = 6;             // cost of a range, at least
constexpr unsigned kTreeSnapRange = 24;           // from here on no tile's first or last chunk is cut off alone
constexpr int kTreeHostCtas = 32;
constexpr int kTreeMergeRows = 8;                 // a warp each

struct TreeMaps {
    CUtensorMap tier[2];  // host, HBM
};

struct TreeHead {  // of range r, the partials of the tile that begins in it and ends in a later one
    int b, g, row0, pieces;  // pieces 0: there is no such tile
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
    int inv_G;      // 2^16 / G rounded up: (r * inv_G) >> 16 is r / G for r < 4096
    int part_rows;  // rows of a tile, at most
    int ranges, host_ctas, slab_chunks;
    int in_flight[2];  // copies of a CTA that have not landed, by tier
    float scale_log2;
    DevStatus* st;
};

enum : uint32_t { T_PROD_EMPTY = 0x71, T_PROD_FULL, T_MMA_FULL, T_MMA_P, T_MMA_PV, T_SM_S, T_SM_O, T_DRAIN };

// A request as the plan sees it.
struct TreeRequest {
    int len, keys, rows, chunks;  // cached rows; with the drafts; query rows a kv head; chunks of 64 keys
    int tiles, twos;              // tiles, those of two halves
    unsigned two, one, slab;      // cost of a tile of two halves, of one, of all tiles of a kv head
};

__device__ __forceinline__ TreeRequest tree_request(const TreeParams& p, int b) {
    TreeRequest q;
    const int n = p.n_new ? min(max(p.n_new[b], 0), p.T) : p.T;
    q.len = min(max(p.lens[b], 0), p.L);
    q.keys = min(q.len + n, p.L);
    q.rows = n * p.G;
    q.chunks = (q.keys + 63) >> 6;
    const int halves = (q.rows + 127) >> 7;
    q.twos = halves >> 1;
    q.tiles = (halves + 1) >> 1;
    q.two = kTreeTileCost + kTreeTwoCost * q.chunks;
    q.one = kTreeTileCost + kTreeOneCost * q.chunks;
    q.slab = q.twos * q.two + (halves & 1) * q.one;
    return q;
}

struct TreePlan {
    unsigned len;                // of a range
    int ranges, host_ranges;     // host_ranges: those that touch the host's slabs
};

// By one warp.
__device__ __forceinline__ TreePlan tree_plan(const TreeParams& p) {
    constexpr unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31, bh = p.h_s / p.Hkv;
    unsigned total = 0, host = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const unsigned slab = b < p.B ? tree_request(p, b).slab : 0u;
        total += slab * p.Hkv;
        if (b <= bh) host += slab * (b < bh ? p.Hkv : p.h_s - bh * p.Hkv);
    }
    total = __reduce_add_sync(all, total);
    host = __reduce_add_sync(all, host);
    TreePlan x;
    x.len = max((total + p.ranges - 1) / p.ranges, kTreeMinRange);
    x.ranges = static_cast<int>((total + x.len - 1) / x.len);
    x.host_ranges = static_cast<int>((host + x.len - 1) / x.len);
    return x;
}

// A tile on the line, and the part of it that a range takes.
struct TreeWalk {
    int b, g, tile;
    unsigned at;  // where the tile begins
    TreeRequest q;

    __device__ __forceinline__ bool two() const { return tile < q.twos; }
    __device__ __forceinline__ unsigned end() const { return at + (two() ? q.two : q.one); }
    // The tile at position x, which lies on the line; by one warp.
    __device__ __forceinline__ void find(const TreeParams& p, unsigned x) {
        constexpr unsigned all = 0xffffffffu;
        const int lane = threadIdx.x & 31;
        unsigned base = 0;
        b = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const unsigned cost = b0 + lane < p.B ? tree_request(p, b0 + lane).slab * p.Hkv : 0u;
            unsigned incl = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(all, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(all, x < base + incl);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = b0 + l;
                base += __shfl_sync(all, incl - cost, l);
                break;
            }
            base += __shfl_sync(all, incl, 31);
        }
        q = tree_request(p, b);
        g = static_cast<int>((x - base) / q.slab);
        at = base + g * q.slab;
        tile = min(static_cast<int>((x - at) / q.two), q.twos);
        at += tile * q.two;
    }
    // The next tile; past the line's end b is B.
    __device__ __forceinline__ void next(const TreeParams& p) {
        at = end();
        if (++tile < q.tiles) return;
        tile = 0;
        if (++g < p.Hkv) return;
        g = 0;
        while (++b < p.B) {
            q = tree_request(p, b);
            if (q.tiles > 0) break;
        }
    }
    // The first chunk that does not belong to the ranges before position x.
    __device__ __forceinline__ int cut(unsigned x, unsigned range_len) const {
        if (x <= at) return 0;
        if (x >= end()) return q.chunks;
        const unsigned k = two() ? kTreeTwoCost : kTreeOneCost, in = x - at;
        const int t = in <= kTreeTileCost ? 0 : static_cast<int>((in - kTreeTileCost + k - 1) / k);
        const int least = range_len >= kTreeSnapRange ? 2 : 1;
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

struct KeysUnset {
    uint32_t lo, hi;
    __device__ __forceinline__ bool any() const { return (lo & hi) != 0xffffffffu; }
    __device__ __forceinline__ bool operator()(int k) const { return !((k < 32 ? lo >> k : hi >> (k - 32)) & 1u); }
};

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(const uint4& v) {
    const auto bad = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
    return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}

__device__ __forceinline__ uint4 ld_shared_ordered(const void* p) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)) : "memory");
    return v;
}
__device__ __forceinline__ void clear_shared_ordered(void* p) {
    asm volatile("st.volatile.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(smem_u32(p)), "r"(0) : "memory");
}

template <int D, bool F32>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using C = ChunkCfg<D>;
    constexpr int NS = C::kStages;
    constexpr int SB = F32 ? 1 : 2;  // buffers of S
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    uint8_t* ring = smem + 2 * C::kTileBytes;
    __shared__ uint64_t full[NS], empty[NS], s_full[2][2], p_ready[2][2], pv_done[2][2];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_flag, stop[2];
    __shared__ unsigned bad[DAK_MAX_TREE / 32];  // drafts with infinities or NaN in V, of the tile at work
    volatile int* abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 32) {
        abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        for (int s = 0; s < 2; ++s) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[s][b], 1);
                mbar_init(&p_ready[s][b], 4);
                mbar_init(&pv_done[s][b], 1);
            }
        }
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    grid_dep_wait();  // launched while the previous kernel ends
    grid_dep_launch();
    const TreePlan plan = tree_plan(p);
    // this CTA's ranges: the one of its number, unless more ranges touch the host than CTAs may
    const bool many = plan.host_ranges > p.host_ctas, takes_host = many && static_cast<int>(blockIdx.x) < p.host_ctas;
    const int r0 = !many || takes_host ? blockIdx.x : plan.host_ranges + blockIdx.x - p.host_ctas;
    const int r_end = takes_host ? plan.host_ranges : plan.ranges, r_step = takes_host ? p.host_ctas : p.ranges;
    // TMEM columns: stream s has S at 128 s + 64 b (buffer b) with P over it, and O at 256 + D s

    if (warp == 8) {
        // ---------------------------------------------------------------- copies
        RingPos<NS> pos(0), landed(0);
        int sent = 0, behind = 0;  // copies issued, and of these seen to have landed
        bool ok = true;
        for (int r = r0; r < r_end && ok; r += r_step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            TreeWalk w;
            w.find(p, xs);
            for (; w.b < p.B && w.at < xe && ok; w.next(p)) {
                const int c0 = w.cut(xs, plan.len), c1 = w.cut(xe, plan.len);
                if (lane == 0) {
                    const long long slab = static_cast<long long>(w.b) * p.Hkv + w.g;
                    const int tier = slab < p.h_s ? 0 : 1, window = p.in_flight[tier];
                    const uint64_t policy = w.q.tiles > 1 ? policy_evict_last() : policy_evict_first();
                    const int chunk0 = static_cast<int>((tier ? slab - p.h_s : slab) * p.slab_chunks);
                    for (int c = c0; c < c1; ++c) {
                        if (sent >= NS) ok = wait_phase(&empty[pos.slot], pos.phase ^ 1u, abort, p.st, T_PROD_EMPTY);
                        while (ok && sent - behind >= window) {
                            ok = wait_phase(&full[landed.slot], landed.phase, abort, p.st, T_PROD_FULL);
                            landed.advance(1);
                            ++behind;
                        }
                        if (!ok) break;
                        mbar_arrive_expect_tx(&full[pos.slot], C::kStage);
                        tma_load_chunk(ring + pos.slot * C::kStage, &maps.tier[tier], chunk0 + c, &full[pos.slot], policy);
                        pos.advance(1);
                        ++sent;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
        }
        if (lane == 0) {  // copies in flight land before the CTA may leave
            volatile int dummy = 0;
            for (; behind < sent; ++behind) {
                wait_phase(&full[landed.slot], landed.phase, &dummy, p.st, T_DRAIN);
                landed.advance(1);
            }
        }
        __syncwarp();
    } else if (warp >= 9) {
        // ---------------------------------------------------------------- products, a warp per stream
        const int st = warp - 9;
        const bool leader = elect_one();
        const uint32_t ring_addr = smem_u32(ring);
        const uint32_t s_tmem = tmem + st * 128, o_tmem = tmem + 256 + st * D;
        int n = 0;           // steps of this stream before this tile
        int stage = 0, u = 0;  // stages used and tiles taken before it
        bool ok = true;
        for (int r = r0; r < r_end && ok; r += r_step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            TreeWalk w;
            w.find(p, xs);
            for (; w.b < p.B && w.at < xe; w.next(p)) {
                const int steps = w.cut(xe, plan.len) - w.cut(xs, plan.len);
                if (steps <= 0) continue;
                const bool two = w.two();
                named_bar<2, kTreeSoftmax + 64>();  // Q lies in shared memory
                if (stop[u & 1]) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t q_addr = smem_u32(smem) + (two ? st * C::kTileBytes : 0);
                const int stride = two ? 1 : 2, first = two ? 0 : st, mine = first < steps ? (steps - first + stride - 1) / stride : 0;
                RingPos<NS> kpos(stage + first), vpos(stage + first);
                // S buffer of this stream's step i of the tile, and the parity of its barriers' phase: a
                // wait by parity is right only where the phase before is known to be over and the one after
                // not to be, and steps i and i + SB of a buffer wait for each other.
                const auto buf = [&](int i) { return (n + i) & (SB - 1); };
                const auto par = [&](int i) { return static_cast<uint32_t>((n + i) / SB) & 1u; };
                const auto qk = [&](int i) {
                    if (!wait_phase(&full[kpos.slot], kpos.phase, abort, p.st, T_MMA_FULL)) return false;
                    if (n + i >= SB && !wait_phase(&pv_done[st][buf(i)], par(i) ^ 1u, abort, p.st, T_MMA_PV)) return false;
                    tc_fence_after();
                    if (leader) {
                        issue_qk<D>(s_tmem + buf(i) * 64, q_addr, ring_addr + kpos.slot * C::kStage);
                        umma_commit(&s_full[st][buf(i)]);
                    }
                    __syncwarp();
                    kpos.advance(stride);
                    return true;
                };
                bool go = mine == 0 || qk(0);
                for (int i = 0; i < mine && go; ++i) {
                    if (!F32 && i + 1 < mine && !qk(i + 1)) break;
                    if (!wait_phase(&p_ready[st][buf(i)], par(i), abort, p.st, T_MMA_P)) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t p_tmem = s_tmem + buf(i) * 64, v = ring_addr + vpos.slot * C::kStage + C::kV;
                        if (F32) issue_pv<D, 3>(o_tmem, p_tmem, v, false);
                        else issue_pv<D, 2>(o_tmem, p_tmem, v, i > 0);
                        umma_commit(&pv_done[st][buf(i)]);
                        // a stage is free when both streams have used it, or the one that does has said so twice
                        umma_commit(&empty[vpos.slot]);
                        if (!two) umma_commit(&empty[vpos.slot]);
                    }
                    __syncwarp();
                    vpos.advance(stride);
                    if (F32 && i + 1 < mine) go = qk(i + 1);
                }
                n += mine;
                stage += steps;
                ++u;
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax, a thread a row
        const int st = warp >> 2, quad = warp & 3, r_in = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_addr = tmem + lanes + st * 128, o_addr = tmem + lanes + 256 + st * D;
        int n = 0, stage = 0, u = 0;
        bool go = true;
        for (int r = r0; r < r_end && go; r += r_step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            if (threadIdx.x == 0) p.heads[r].pieces = 0;
            TreeWalk w;
            w.find(p, xs);
            for (; w.b < p.B && w.at < xe; w.next(p)) {
                const int c0 = w.cut(xs, plan.len), c1 = w.cut(xe, plan.len), steps = c1 - c0;
                if (steps <= 0) continue;
                const bool two = w.two();
                const int row0 = w.tile * kTreeRows;
                const auto source = [&](int row) {  // a query row of the request, in Q and O
                    const int t = (row * p.inv_G) >> 16;
                    return ((static_cast<long long>(w.b) * p.T + t) * p.Hq + w.g * p.G + row - t * p.G) * D;
                };
                {   // Q rows into the 128-byte swizzled K-major layout, rows that are none zero
                    constexpr int PIECES = D / 8;  // 16-byte pieces of a row
                    const int count = (two ? 256 : 128) * PIECES;
#pragma unroll 4
                    for (int e = threadIdx.x; e < count; e += kTreeSoftmax) {
                        const int rr = e / PIECES, c = e % PIECES;
                        const bool there = row0 + rr < w.q.rows;
                        cp_async16(smem + (rr >> 7) * C::kTileBytes + (c >> 3) * 16384 + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4),
                                   p.Q + (there ? source(row0 + rr) + c * 8 : 0), there ? 16 : 0);
                    }
                    if (threadIdx.x < DAK_MAX_TREE / 32) bad[threadIdx.x] = 0;
                    if (threadIdx.x == 0) {
                        stop[u & 1] = abort_flag;
                        if (c0 == 0 && c1 < w.q.chunks) {
                            // ranges up to the one with the tile's last chunk
                            int last = static_cast<int>((w.end() - 1) / plan.len);
                            while (w.cut(last * plan.len, plan.len) == w.q.chunks) --last;
                            p.heads[r] = TreeHead{w.b, w.g, row0, last - r + 1};
                        }
                        if (w.g == 0 && w.tile == 0 && c0 == 0 && w.q.keys - w.q.len < (p.n_new ? min(max(p.n_new[w.b], 0), p.T) : p.T)) {
                            report(p.st, DAK_ERR_BOUNDS, (0x7EEEull << 32) | static_cast<unsigned>(w.b));
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    named_bar<2, kTreeSoftmax + 64>();
                    if (stop[u & 1]) {
                        go = false;
                        break;
                    }
                }
                const int row = row0 + (two ? st * 128 : 0) + r_in, t = (row * p.inv_G) >> 16;
                const bool valid_row = row < w.q.rows, warp_has_rows = row - lane < w.q.rows;
                const int stride = two ? 1 : 2;
                const auto buf = [&](int i) { return (n + i) & (SB - 1); };
                const auto par = [&](int i) { return static_cast<uint32_t>((n + i) / SB) & 1u; };
                float m_ref = -INFINITY, l = 0.f;
                // An fp32 output's O is summed here, a step's product at a time: the tensor cores cut off what
                // they add to a sum.
                float sum[F32 ? D / 16 : 1][16] = {};
                const auto add_product = [&] {
#pragma unroll
                    for (int q = 0; q < (F32 ? D / 16 : 0); ++q) {
                        float o[16];
                        tmem_ld16(o_addr + q * 16, o);
                        tmem_wait(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[q][k] += o[k];
                    }
                };
                bool ok = true;
                int i = 0;
                for (int j = two ? 0 : st; j < steps; j += stride, ++i) {
                    const int key0 = (c0 + j) * 64;
                    unsigned long long bits = ~0ull;
                    const bool drafts = key0 + 64 > w.q.len;
                    if (drafts && valid_row) bits = tree_bits(p, w.q, w.b, t, key0);
                    ok = mbar_wait(&s_full[st][buf(i)], par(i), abort, p.st, DAK_ERR_TIMEOUT, T_SM_S);
                    if (!__all_sync(0xffffffffu, ok)) {  // a wait ran out: the whole warp stops
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (drafts) {
                        // Drafted rows' V may hold infinities and NaN, which the probability of zero of a token
                        // that does not see the row would not cancel, and rows behind the drafts anything at all.
                        // Such pieces become zeros for the product; what a token sees of them is added at the end.
                        // Both streams of a step go through them, as either one's product may be first, and a
                        // piece that the other has cleared already is in this one's fence like its own.
                        // (The scores say that the chunk is there.)
                        uint8_t* rows = ring + RingPos<NS>(stage + j).slot * C::kStage + C::kV;
                        const int begin = max(0, w.q.len - key0), end = w.q.keys - key0;
                        for (int e = begin * (D / 8) + r_in; e < 64 * (D / 8); e += 128) {
                            const int kr = e / (D / 8), c = e % (D / 8);
                            uint8_t* piece = rows + (c >> 3) * 16384 + kr * 128 + ((c & 7) << 4);
                            if (kr < end) {
                                if (!not_finite(ld_shared_ordered(piece))) continue;
                                const int s = key0 + kr - w.q.len;
                                atomicOr(&bad[s >> 5], 1u << (s & 31));
                                __threadfence_block();
                            }
                            clear_shared_ordered(piece);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // O so far, its last product done, to the new reference
                    const auto grown = [&](float f) {
                        if (F32) {
#pragma unroll
                            for (int q = 0; q < (F32 ? D / 16 : 0); ++q) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) sum[q][k] *= f;
                            }
                            return;
                        }
                        mbar_wait(&pv_done[st][buf(i - 1)], par(i - 1), abort, p.st, DAK_ERR_TIMEOUT, T_SM_O);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            float o[16];
                            tmem_ld16(o_addr + q * 16, o);
                            tmem_wait(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= f;
                            tmem_st16(o_addr + q * 16, o);
                        }
                    };
                    const uint32_t at_s = s_addr + buf(i) * 64;
                    if (warp_has_rows) {  // lanes without rows share a warp's work, warps without any do none
                        const KeysUnset hidden{static_cast<uint32_t>(bits), static_cast<uint32_t>(bits >> 32)};
                        if (F32 && i > 0) add_product();  // the last step's: its scores' columns are these
                        if (F32) softmax_step<3>(at_s, hidden, p.scale_log2, m_ref, l, i == 0, grown);
                        else softmax_step<2>(at_s, hidden, p.scale_log2, m_ref, l, i == 0, grown);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[st][buf(i)]);
                }
                for (int k = max(0, i - SB); ok && k < i; ++k) {  // one phase of each buffer's
                    ok = mbar_wait(&pv_done[st][buf(k)], par(k), abort, p.st, DAK_ERR_TIMEOUT, T_SM_O);
                }
                __syncwarp();
                if (F32) {  // back to where the results are read from
                    tc_fence_after();
                    if (i > 0) add_product();
#pragma unroll
                    for (int q = 0; q < (F32 ? D / 16 : 0); ++q) tmem_st16(o_addr + q * 16, sum[q]);
                    tmem_wait_st();
                }
                // what tokens see of cleared pieces
#pragma unroll 1
                for (int word = 0; word < DAK_MAX_TREE / 32; ++word) {
                    unsigned set = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile unsigned*>(&bad[word]), 0);
#pragma unroll 1
                    for (; set; set &= set - 1) {
                        const int s = word * 32 + __ffs(set) - 1, key = w.q.len + s, j = (key >> 6) - c0;
                        if (j < 0 || j >= steps || (!two && (j & 1) != st)) continue;
                        const bool sees = valid_row && (tree_bits(p, w.q, w.b, t, key) & 1);
                        if (!__any_sync(0xffffffffu, sees)) continue;
                        const long long slab = static_cast<long long>(w.b) * p.Hkv + w.g;
                        const uint8_t* base = slab < p.h_s ? p.kv[0] + slab * p.head_bytes : p.kv[1] + (slab - p.h_s) * p.head_bytes;
                        const uint4* k_row = reinterpret_cast<const uint4*>(base) + (static_cast<long long>(key >> 6) * 2 * 64 + (key & 63)) * (D / 8);
                        const uint4* v_row = k_row + 64 * (D / 8);
                        const auto products = [](const uint4& a, const uint4& b) {
                            return bf_lo(a.x) * bf_lo(b.x) + bf_hi(a.x) * bf_hi(b.x) + bf_lo(a.y) * bf_lo(b.y) + bf_hi(a.y) * bf_hi(b.y) +
                                   bf_lo(a.z) * bf_lo(b.z) + bf_hi(a.z) * bf_hi(b.z) + bf_lo(a.w) * bf_lo(b.w) + bf_hi(a.w) * bf_hi(b.w);
                        };
                        float x = 0.f;
                        if (sees) {
                            const uint4* q_row = reinterpret_cast<const uint4*>(p.Q + source(row));
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) x += products(q_row[c], k_row[c ^ (key & 7)]);
                        }
                        // a weight that is too small for its type is none the less more than zero
                        const float weight = fmaxf(exp2f(x * p.scale_log2 - (m_ref == -INFINITY ? 0.f : m_ref)), 1e-37f);
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            float o[16];
                            tmem_ld16(o_addr + q * 16, o);
                            tmem_wait(o);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint4 v = v_row[(2 * q + half) ^ (key & 7)];
                                if (!sees || !not_finite(v)) continue;
                                const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    o[half * 8 + 2 * k] += weight * bf_lo(e[k]);
                                    o[half * 8 + 2 * k + 1] += weight * bf_hi(e[k]);
                                }
                            }
                            tmem_st16(o_addr + q * 16, o);
                        }
                        tmem_wait_st();
                    }
                }
                // ---- results
                // Q's memory, no longer read, takes the streams' (m, l) where they share a tile, and then, half
                // a row's columns at a time, the results on their way out.
                constexpr int COLS = D / 2;
                float M = m_ref, total = l, w0 = 1.f, w1 = 0.f;
                const bool both = !two && steps > 1;  // the streams' rows are the same and both had a step
                tc_fence_before();
                if (!two) {
                    float2(*ex)[128] = reinterpret_cast<float2(*)[128]>(smem + C::kTileBytes);
                    ex[st][r_in] = make_float2(m_ref, l);
                    named_bar<3, kTreeSoftmax>();
                    const float2 e0 = ex[0][r_in], e1 = ex[1][r_in];
                    named_bar<3, kTreeSoftmax>();  // ex lies in what is written next
                    M = fmaxf(e0.x, e1.x);
                    const float base = M == -INFINITY ? 0.f : M;
                    w0 = exp2_ftz(e0.x - base);
                    w1 = both ? exp2_ftz(e1.x - base) : 0.f;
                    total = w0 * e0.y + (both ? w1 * e1.y : 0.f);
                }
                tc_fence_after();
                const bool whole = c0 == 0 && c1 == w.q.chunks;
                if (whole && valid_row && !tree_sees(p, w.q, w.b, t)) total = INFINITY;  // O is zero: it becomes zeros
                const float inv = whole ? 1.f / total : 1.f;
                const long long slot = 2ll * r + (c0 == 0);
                if (!whole && valid_row && (two || st == 0)) p.ml_part[slot * p.part_rows + row - row0] = make_float2(M, total);
                float4* staged = reinterpret_cast<float4*>(smem + st * C::kTileBytes + quad * 32 * COLS * 4);
                const int first = row - lane;  // the warp's rows
#pragma unroll 1
                for (int col = two ? 0 : st * COLS; warp_has_rows && col < (two ? D : (st + 1) * COLS); col += COLS) {
#pragma unroll 1
                    for (int q = 0; q < COLS / 16; ++q) {
                        float o[16];
                        tmem_ld16(tmem + lanes + 256 + (two ? st * D : 0) + col + q * 16, o);
                        tmem_wait(o);
                        if (!two) {
                            float b[16];
                            tmem_ld16(tmem + lanes + 256 + D + col + q * 16, b);
                            tmem_wait(b);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = both ? o[k] * w0 + b[k] * w1 : o[k] * w0;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            staged[stage_piece<COLS>(lane, q * 4 + k)] =
                                make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
                        }
                    }
                    __syncwarp();
                    constexpr int PIECES = COLS / 4;
#pragma unroll 4
                    for (int e = lane; e < 32 * PIECES; e += 32) {
                        const int rr = e / PIECES, c = e % PIECES;
                        if (first + rr >= w.q.rows) break;
                        const float4 v = staged[stage_piece<COLS>(rr, c)];
                        if (!whole) {
                            *reinterpret_cast<float4*>(p.o_part + (slot * p.part_rows + first + rr - row0) * D + col + c * 4) = v;
                        } else if (p.o_fp32) {
                            *reinterpret_cast<float4*>(static_cast<float*>(p.O) + source(first + rr) + col + c * 4) = v;
                        } else {
                            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + source(first + rr) + col + c * 4) =
                                make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                        }
                    }
                    __syncwarp();
                }
                n += two ? steps : (steps + 1 - st) / 2;
                stage += steps;
                ++u;
                tc_fence_before();
                named_bar<3, kTreeSoftmax>();  // Q's memory and O are free
                tc_fence_after();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem_sh, 512);
    }
}

// ------------------------------------------------------------------------------------
// merge
// ------------------------------------------------------------------------------------
// Block (r, y): eight rows, a warp each, of the tile that begins in range r and ends in a later one:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over its pieces, in order.
template <int D>
__global__ void __launch_bounds__(32 * kTreeMergeRows) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int LANES = D / 4, AT_ONCE = 32 / LANES;  // pieces that a warp reads at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x;
    grid_dep_wait();
    const TreePlan plan = tree_plan(p);
    if (r >= plan.ranges) return;
    const TreeHead head = p.heads[r];
    const int local = blockIdx.y * kTreeMergeRows + warp;
    // the limits: where a wait ran out, a range's entry may never have been written
    if (head.pieces <= 0 || head.b < 0 || head.b >= p.B || head.g < 0 || head.g >= p.Hkv || head.row0 < 0) return;
    const int n = min(head.pieces, plan.ranges - r);
    const TreeRequest q = tree_request(p, head.b);
    const int row = head.row0 + local;
    if (row >= q.rows || local >= p.part_rows) return;
    const auto slot = [&](int s) { return (2ll * (r + s) + (s == 0)) * p.part_rows + local; };
    const int c = lane % LANES, grp = lane / LANES;
    const auto part = [&](int s) { return *reinterpret_cast<const float4*>(p.o_part + slot(s) * D + c * 4); };
    float4 early[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (grp + k * AT_ONCE < n) early[k] = part(grp + k * AT_ONCE);
    }
    float M = -INFINITY;
    for (int s = lane; s < n; s += 32) M = fmaxf(M, p.ml_part[slot(s)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int s0 = 0; s0 < n; s0 += 32) {
        const float2 v = s0 + lane < n ? p.ml_part[slot(s0 + lane)] : make_float2(-INFINITY, 0.f);
        const float f = exp2f(v.x - base);
        l += f * v.y;
#pragma unroll 4
        for (int k = 0; k < 32; k += AT_ONCE) {
            if (s0 + k >= n) break;
            const float w = __shfl_sync(0xffffffffu, f, k + grp);
            const int s = s0 + k + grp;
            if (s >= n) continue;
            const float4 x = s0 == 0 && k / AT_ONCE < 4 ? early[k / AT_ONCE] : part(s);
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
    }
    if (grp != 0) return;
    const int t = row / p.G;
    if (tree_sees(p, q, head.b, t)) acc.x /= l, acc.y /= l, acc.z /= l, acc.w /= l;
    const long long at = ((static_cast<long long>(head.b) * p.T + t) * p.Hq + head.g * p.G + row - t * p.G) * D + c * 4;
    if (p.o_fp32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = acc;
    } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
struct TreeLayout {
    int ranges, part_rows;
    size_t o_part, ml_part, heads;
    size_t total() const { return o_part + ml_part + heads; }
};

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// As many ranges as SMs; fewer where the cache, full, would not give each the least there may be.
static TreeLayout tree_layout(const dak_placement* KV, int T, int H_q) {
    const int G = H_q / KV->H_kv, rows = T * G;
    const int64_t chunks = (KV->L + 63) / 64, halves = (rows + 127) / 128;
    const int64_t slab = (halves / 2) * (kTreeTileCost + kTreeTwoCost * chunks) + halves % 2 * (kTreeTileCost + kTreeOneCost * chunks);
    const int64_t least = (slab * KV->B * KV->H_kv + kTreeMinRange - 1) / kTreeMinRange;
    TreeLayout x{};
    x.ranges = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), least)));
    x.part_rows = std::min(rows, kTreeRows);
    x.o_part = round256(sizeof(float) * 2 * x.ranges * x.part_rows * KV->D);
    x.ml_part = round256(sizeof(float2) * 2 * x.ranges * x.part_rows);
    x.heads = round256(sizeof(TreeHead) * x.ranges);
    return x;
}

// The whole line's cost, with every cache full, fits an int.
static bool line_fits(const dak_placement* KV, int T, int H_q) {
    const int64_t chunks = (KV->L + 63) / 64, halves = (T * (H_q / KV->H_kv) + 127) / 128;
    return (kTreeTileCost + kTreeOneCost * chunks) * halves * KV->B * KV->H_kv < 0x7FFFFFFF - (1 << 24) &&
           static_cast<int64_t>(KV->B) * KV->H_kv * chunks <= 0x7FFFFFFF;
}

template <int D, bool F32>
static cudaError_t launch_tree(const TreeParams& p, const TreeMaps& maps, cudaStream_t s) {
    auto k = tree_kernel<D, F32>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), ChunkCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = ChunkCfg<D>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k, p, maps);
    if (e != cudaSuccess || p.ranges == 1) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges - 1), static_cast<unsigned>((p.part_rows + kTreeMergeRows - 1) / kTreeMergeRows));
    cfg.blockDim = dim3(32 * kTreeMergeRows);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p);
}

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

static bool off(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace dak

using namespace dak;

extern "C" size_t dak_attn_tree_workspace_bytes(const dak_placement* KV, int T, int H_q) {
    if (!KV || KV->kind != 1 || T < 1 || T > DAK_MAX_TREE || H_q < 1 || H_q % KV->H_kv || H_q / KV->H_kv > 16) return 0;
    return tree_layout(KV, T, H_q).total();
}

extern "C" dak_status dak_attn_tree(const void* Q, const dak_placement* KV, const int* seq_lens, int T, const uint64_t* mask,
                                    int64_t mask_pitch, const int* n_new, int H_q, float scale, void* O, int o_fp32,
                                    void* workspace, size_t ws_bytes, const dak_tuning* tuning, void* stream) {
    if (!KV || KV->kind != 1 || !Q || !O || !seq_lens || T < 1 || H_q < 1 || H_q % KV->H_kv) return DAK_ERR_INVALID;
    const int G = H_q / KV->H_kv, D = KV->D, W = (T + 63) / 64;
    if (T > DAK_MAX_TREE || G > 16 || !line_fits(KV, T, H_q)) return DAK_ERR_UNSUPPORTED;
    if (mask && mask_pitch != 0 && mask_pitch < static_cast<int64_t>(T) * W) return DAK_ERR_INVALID;
    const size_t elems = static_cast<size_t>(KV->B) * T * H_q * D;
    if (overlap(Q, elems * 2, O, elems * (o_fp32 ? 4 : 2))) return DAK_ERR_INVALID;
    if (off(Q, 16) || off(O, 16) || off(workspace, 16) || off(seq_lens, 4) || off(n_new, 4) || off(mask, 8)) return DAK_ERR_ALIGN;
    const TreeLayout x = tree_layout(KV, T, H_q);
    if (!workspace || ws_bytes < x.total()) return DAK_ERR_INVALID;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DAK_ERR_CUDA;
    if (dev != KV->device) return DAK_ERR_INVALID;
    TreeParams p{};
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.lens = seq_lens;
    p.n_new = n_new;
    p.mask = reinterpret_cast<const unsigned long long*>(mask);
    p.mask_pitch = mask_pitch;
    p.O = O;
    p.o_fp32 = o_fp32 ? 1 : 0;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    p.o_part = reinterpret_cast<float*>(w);
    p.ml_part = reinterpret_cast<float2*>(w + x.o_part);
    p.heads = reinterpret_cast<TreeHead*>(w + x.o_part + x.ml_part);
    p.kv[0] = static_cast<const uint8_t*>(KV->host_dev);
    p.kv[1] = static_cast<const uint8_t*>(KV->hbm_ptr);
    p.head_bytes = KV->head_bytes;
    p.B = KV->B;
    p.T = T;
    p.W = W;
    p.Hq = H_q;
    p.Hkv = KV->H_kv;
    p.G = G;
    p.inv_G = (65536 + G - 1) / G;
    p.L = KV->L;
    p.h_s = KV->h_s;
    p.part_rows = x.part_rows;
    p.ranges = x.ranges;
    p.slab_chunks = (KV->L + 63) / 64;
    p.host_ctas = std::min(x.ranges, tuning && tuning->host_ctas > 0 ? tuning->host_ctas : kTreeHostCtas);
    const int window = D == 128 ? ChunkCfg<128>::kInFlight : ChunkCfg<64>::kInFlight;
    const int most = D == 128 ? ChunkCfg<128>::kStages : ChunkCfg<64>::kStages;
    p.in_flight[0] = std::min(most, tuning && tuning->window > 0 ? tuning->window : window);
    p.in_flight[1] = std::min(most, tuning && tuning->hbm_window > 0 ? tuning->hbm_window : window);
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    const int64_t slabs = static_cast<int64_t>(KV->B) * KV->H_kv;
    TreeMaps maps{};
    for (int tier = 0; tier < 2; ++tier) {
        const int64_t n = tier ? slabs - KV->h_s : KV->h_s;
        if (n > 0 && !make_chunk_map(&maps.tier[tier], p.kv[tier], n * p.slab_chunks, D)) return DAK_ERR_CUDA;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(D == 128 ? (o_fp32 ? launch_tree<128, true>(p, maps, s) : launch_tree<128, false>(p, maps, s))
                                : (o_fp32 ? launch_tree<64, true>(p, maps, s) : launch_tree<64, false>(p, maps, s)));
}
