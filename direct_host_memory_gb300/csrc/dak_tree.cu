// Decode attention of a tree (or chain) of drafted tokens per request over a placed KV cache,
// dak_attn_tree: o[b,t,h] = softmax(scale q[b,t,h] K^T) V over the rows before the drafts and those
// drafts that the token's mask names. The tokens' query heads of one kv head are the rows of a tile, as
// many whole tokens as fit in each of its two 128-row halves, so that the cache, which dak_attn streams once
// per token, is streamed once per tile: once for up to 256 rows a kv head, again for every further 256 (by the
// memory that holds it, which for the host's slabs is the link); 64 keys a step on the tcgen05 tensor cores, as in the
// prefix pass, whose comment says how (dak_prefix.cu; what both use: dak_umma_attn.cuh).
// How work is cut: dak_tree.cuh. Up to 16 rows a kv head go to dak_tree_few.cu.
//
// A row is two threads', of a step's keys and of O's columns a half each, so that a sub-partition has four
// softmax warps to cover the latencies of S, exp2 and P. Nothing waits at a tile's end but for what it
// needs: copies run ahead, up to what the ring holds; the next tile's Q is fetched when the last product that
// reads the old one is done, and its first scores are computed while the results, straight from TMEM, are
// on their way out. (48 requests of 64 drafts and 64 heads over 2K 230 us with both, 250 with a thread a row
// and Q, scores and results one after the other.)
//
// What bounds it: with a half tile the cache's bytes (32 requests of 16 drafts and 32/8 heads over 7K to 8K:
// 158 to 161 us, 148 at the copy rate; 32 rows 154, 128 rows 182). With two halves the tensor cores, which P in two
// bf16 parts keeps busy for half as long again: those 48 requests 230 us, of which 13 are the merge, the
// two products 85 at the rate of a large matrix product, 127 with the second part; the pipe is active 60% of
// the time, and the rest is the chain from S to P.V that two streams do not cover. Small calls the start, the
// first chunks and the merge's launch (one request of 8 drafts over 4K: 13.8 us, the merge 4.4 of them). An fp32
// output's sums, in registers, do not fit beside a step's scores: of heads of 128 594 bytes of a thread are spilled and
// 840 read again (of heads of 64 152 and 216), and every step adds a whole product: in that batch 273 us with 32 rows, 311
// with 64, 342 with 128. Host slabs are bound by the link (kTreeHostCtas).
#include <algorithm>
#include <cmath>

#include "dak_tree.cuh"
#include "dak_umma_attn.cuh"

namespace dak {

constexpr int kTreeSoftmax = 2 * 2 * 128;            // two streams, two threads a row
constexpr int kTreeThreads = kTreeSoftmax + 4 * 32;  // and copies, scores, each stream's P.V
// CTAs that read the host's slabs, by dak_attn's number. 32 requests over 7K to 8K, a quarter of the slabs on the host (249
// MB): 4 drafts 1196 us with 16, 32, 64 and 152, 16 drafts 1200, 208 GB/s of the link, where one token by dak_attn takes
// 1190; with 8 CTAs 1243 and 1202. With 3% there 16 drafts take 165, as with 8 to 152. What more rows a step cost shows
// in fewer CTAs: 32 drafts of 8 heads a kv head over 2K 480 us, with 64 451; 64 of them, two tiles and so two passes over the
// link, 942 and 894. Copies under way: two a CTA are enough (windows of 2 to 6 are within 1%, 1 is up to twice as slow).
constexpr int kTreeHostCtas = 32;
constexpr int kTreeMergeRows = 8;                 // a warp each

struct TreeMaps {
    CUtensorMap tier[2];  // host, HBM
    CUtensorMap q;        // (64 elements, head, token, half of a row), 128-byte swizzle
};

enum : uint32_t { T_PROD_EMPTY = 0x71, T_PROD_FULL, T_MMA_FULL, T_MMA_P, T_MMA_PV, T_SM_S, T_SM_O, T_Q_FREE, T_Q_FULL, T_DRAIN };

struct KeysUnset {
    uint32_t bits;
    __device__ __forceinline__ bool any() const { return bits != 0xffffffffu; }
    __device__ __forceinline__ bool operator()(int k) const { return !(bits >> k & 1u); }
};

// OR of a predicate over the two warps that share rows (barrier `id`).
__device__ __forceinline__ bool pair_any(int id, bool mine) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(mine)), "r"(id)
                 : "memory");
    return r != 0;
}

// softmax_step (dak_umma_attn.cuh) for the 32 of a row's 64 scores that begin at column 32 * half of s_addr;
// another warp has the others. (counts: the row is one; what else lies in a tile must not move references.)
// Both go by one reference: where a row outgrows it in either, which pair_any finds, they tell each other
// their maxima (`other`, from its maximum the partner's).
template <int PARTS, class Hidden, class Other, class Grown>
__device__ __forceinline__ void softmax_half(uint32_t s_addr, int half, int pair, const Hidden& hidden, float scale_log2,
                                             float& m_ref, float& l, bool first, bool counts, const Other& other,
                                             const Grown& grown) {
    // with three parts O is in registers too, which leaves none for all scores: they are read twice
    constexpr bool TWICE = PARTS == 3;
    float v[TWICE ? 1 : 2][16];
    const auto mask = [&](int q) {
        if (hidden.any()) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (hidden(q * 16 + k)) v[TWICE ? 0 : q][k] = -INFINITY;
            }
        }
    };
    const auto read_again = [&](int q) {
        tmem_ld16(s_addr + half * 32 + q * 16, v[0]);
        tmem_wait(v[0]);
        mask(q);
    };
    if (!TWICE) {
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld16(s_addr + half * 32 + q * 16, v[TWICE ? 0 : q]);
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_wait(v[TWICE ? 0 : q]);
#pragma unroll
        for (int q = 0; q < 2; ++q) mask(q);
    }
    float mx[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (TWICE) read_again(q);
        const float(&x)[16] = v[TWICE ? 0 : q];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[q][e] = fmaxf(x[8 * e], x[8 * e + 1]);
#pragma unroll
            for (int k = 2; k < 8; k += 2) mx[q][e] = max3(mx[q][e], x[8 * e + k], x[8 * e + k + 1]);
        }
    }
    float m_new = fmaxf(max3(mx[0][0], mx[0][1], mx[1][0]), mx[1][1]) * scale_log2;
    // the reference only moves when a row's maximum outgrows it by 2^8: until then the sums just
    // grow, which fp32 holds
    if (first) {
        m_ref = fmaxf(m_new, other(m_new));
    } else if (pair_any(pair, counts && m_new > m_ref + 8.f)) {
        const float m2 = fmaxf(m_ref, fmaxf(m_new, other(m_new)));
        const float f = m2 == -INFINITY ? 1.f : exp2_ftz(m_ref - m2);
        m_ref = m2;
        l *= f;
        grown(f);
    }
    const float base = m_ref == -INFINITY ? 0.f : m_ref;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 scale2 = make_float2(scale_log2, scale_log2), base2 = make_float2(-base, -base);
    const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t part[PARTS][8];
        if (TWICE) read_again(q);
        const float(&x)[16] = v[TWICE ? 0 : q];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), scale2, base2);
            float2 w = make_float2(exp2_ftz(e.x), exp2_ftz(e.y));
            sum[k & 1] = add2(sum[k & 1], w);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                part[i][k] = pack_bf16(w.x, w.y);
                if (i + 1 < PARTS) w = fma2(make_float2(bf_lo(part[i][k]), bf_hi(part[i][k])), minus, w);
            }
        }
#pragma unroll
        for (int i = 0; i < PARTS; ++i) tmem_st8(s_addr + p_column(2 * half + q, i), part[i]);
    }
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(const uint4& v) {
    const auto bad = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
    return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}
// The values without those.
__device__ __forceinline__ uint4 finite_part(const uint4& v) {
    return make_uint4(v.x & ~tree_not_finite(v.x), v.y & ~tree_not_finite(v.y), v.z & ~tree_not_finite(v.z), v.w & ~tree_not_finite(v.w));
}

__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, int head, int token, int half, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(0), "r"(head), "r"(token), "r"(half), "r"(smem_u32(bar))
        : "memory");
}

// 32 bytes of a thread's own row: a whole sector, where the address allows it in one instruction.
__device__ __forceinline__ void store32(void* to, const uint32_t (&r)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                     "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        static_cast<uint4*>(to)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        static_cast<uint4*>(to)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

__device__ __forceinline__ uint4 ld_shared_ordered(const void* p) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_ordered(void* p, const uint4& v) {
    asm volatile("st.volatile.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(smem_u32(p)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// An infinity or NaN in V of a row before the drafts is in the sum of every token: in a row's stored results (columns col0
// to col0 + cols - 1, fp32 or bf16) it becomes what it is, where a weight in parts (infinity times a part of zero) or a
// factor of zero has made NaN of it. Those of the drafts in `bad`, which the products did not meet, are put in where the
// token sees them. By a warp, whose rows' columns are the same; a row that is none, or whose scores are, stays (sound: false).
template <int D>
__device__ __forceinline__ void odd_values(const TreeParams& p, const TreeRequest& q, int b, int g, int c0, int c1, int t,
                                           bool valid_row, bool sound, const unsigned* bad, int col0, int cols, uint8_t* row, bool as_bf16) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int col = col0; col < col0 + cols; col += 8) {
        float x[8] = {};
        for (int key = c0 * 64 + lane; key < min(c1 * 64, q.len); key += 32) add_not_finite(x, tree_v_piece(p, b, g, D, key, col / 8));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
        }
        if (!valid_row || !sound) continue;
        for (int word = 0; bad && word < DAK_MAX_TREE / 32; ++word) {
            for (unsigned set = bad[word]; set; set &= set - 1) {
                const int key = q.len + word * 32 + __ffs(set) - 1;
                if (tree_bits(p, q, b, t, key) & 1) add_not_finite(x, tree_v_piece(p, b, g, D, key, col / 8));
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (x[k] == 0.f) continue;
            if (as_bf16) reinterpret_cast<__nv_bfloat16*>(row)[col + k] = __float2bfloat16_rn(x[k]);
            else reinterpret_cast<float*>(row)[col + k] = x[k];
        }
    }
}
// Out of line for a bf16 output (32 requests of 64 drafts over 760 rows 53.1 us, 54.4 inlined), inline for fp32, whose
// registers a call disturbs (32 requests of 64 rows over 8K 315 us, 344 with a call).
template <int D>
__device__ __noinline__ void odd_values_apart(const TreeParams& p, TreeRequest q, int b, int g, int c0, int c1, int t,
                                              bool valid_row, bool sound, const unsigned* bad, int col0, int cols, uint8_t* row,
                                              bool as_bf16) {
    odd_values<D>(p, q, b, g, c0, c1, t, valid_row, sound, bad, col0, cols, row, as_bf16);
}

template <int D>
constexpr int kTreeSmem = 2 * ChunkCfg<D>::kTileBytes + ChunkCfg<D>::kStages * ChunkCfg<D>::kStage;

template <int D, bool F32>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using C = ChunkCfg<D>;
    constexpr int NS = C::kStages;
    constexpr int SB = F32 ? 1 : 2;  // buffers of S
    constexpr int kCopies = kTreeSoftmax / 32, kScores = kCopies + 1, kProducts = kScores + 1;  // warps
    extern __shared__ __align__(1024) uint8_t smem[];  // as the swizzle wants it; there is no room for a margin
    uint8_t* ring = smem + 2 * C::kTileBytes;
    __shared__ uint64_t full[NS], empty[NS], s_full[2][2], p_ready[2][2], pv_done[2][2], q_full, q_ready, q_free;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_flag, any_bad;
    __shared__ unsigned bad[DAK_MAX_TREE / 32];  // drafts with infinities or NaN in V, of the tile at work
    __shared__ float maxima[2][2][128];          // by stream, half, row: what threads tell each other
    volatile int* abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 32) {
        abort_flag = 0;
        any_bad = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        for (int s = 0; s < 2; ++s) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[s][b], 1);
                mbar_init(&p_ready[s][b], 8);
                mbar_init(&pv_done[s][b], 1);
            }
        }
        mbar_init(&q_full, 1);
        mbar_init(&q_ready, 1);
        mbar_init(&q_free, 2);
        fence_mbar_init();
    }
    if (threadIdx.x < DAK_MAX_TREE / 32) bad[threadIdx.x] = 0;
    if (warp == kCopies && lane < 2) prefetch_tmap(&maps.tier[lane]);
    if (warp == kProducts) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    grid_dep_wait();  // launched while the previous kernel ends
    grid_dep_launch();
    const TreePlan plan = tree_plan(p);
    if (threadIdx.x == 0 && static_cast<int>(blockIdx.x) >= plan.ranges) p.heads[blockIdx.x].pieces = 0;
    const TreeTurn turn = tree_turn(p, plan);
    TreeWalk w;
    if (turn.first < turn.end) w.find(p, plan, turn.first * plan.len);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    // TMEM columns: stream s has S at 128 s + 64 b (buffer b) with P over it, and O at 256 + D s.
    // S buffer of a stream's n-th step, and the parity of its barriers' phase: a wait by parity is right only
    // where the phase before is known to be over and the one after not to be, and steps n and n + SB of a
    // buffer wait for each other.
    const auto buf = [](int n) { return n & (SB - 1); };
    const auto par = [](int n) { return static_cast<uint32_t>(n / SB) & 1u; };
    // Issuing a product takes a warp some 40 cycles whatever the product's size, and a wait 100. Where the streams
    // share a tile, two steps at once have to keep up with the arrival of two chunks: scores and each stream's P.V
    // have warps of their own (32 chats of 16 drafts over 8K: 172 us with a warp for each stream's scores and P.V,
    // 158 so). With a tile each the products take most of the time, and a warp for both streams' scores
    // holds them up (48 of 64 drafts and 64 heads over 2K: 230 and 242 us).

    if (warp == kCopies) {
        // ---------------------------------------------------------------- copies
        RingPos<NS> pos(0), landed(0);
        int sent = 0, behind = 0;  // copies issued, and of these seen to have landed
        bool ok = true;
        for (int r = turn.first; r < turn.end && ok; r += turn.step) {
            if (lane == 0) p.heads[r].pieces = 0;
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            if (r > turn.first) w.find(p, plan, xs);
            for (; w.b < p.B && w.at < xe && ok; w.next(p, plan)) {
                const int c0 = w.cut(p, plan, xs), c1 = w.cut(p, plan, xe);
                if (lane == 0) {
                    const long long slab = static_cast<long long>(w.b) * p.Hkv + w.g;
                    const int tier = slab < p.h_s ? 0 : 1, window = p.in_flight[tier];
                    // also where another tile reads the chunks again: with evict_last 4 requests of 64 drafts and 64 heads
                    // over 27K took 274 us, 267 so, 32 of heads of 64 over 3.6K 250 and 247, the 48 above 232 and 233
                    const uint64_t policy = policy_evict_first();
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
                    if (c0 < c1) {
                        tree_head(p, plan, w, r, c0, c1);
                        tree_report(p, w, c0);
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
    } else if (warp == kScores) {
        // ---------------------------------------------------------------- Q, and the scores of a tile that both streams share
        const bool leader = elect_one();
        RingPos<NS> pos(0);
        int n[2] = {0, 0};  // steps of the streams so far
        int tiles = 0, twos = 0;  // tiles so far, those of two halves
        bool ok = true, in_flight = false, was_two = false;
        for (int r = turn.first; r < turn.end && ok; r += turn.step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            if (r > turn.first) w.find(p, plan, xs);
            for (; w.b < p.B && w.at < xe && ok; w.next(p, plan)) {
                const int steps = w.cut(p, plan, xe) - w.cut(p, plan, xs);
                if (steps <= 0) continue;
                const bool two = w.two();
                // Q, when the scores that read the last tile's are there: those of a tile of two halves are the
                // streams' own warps' products, whose phases this one has not followed
                if (was_two) {
                    ok = wait_phase(&q_free, static_cast<uint32_t>(twos - 1) & 1u, abort, p.st, T_Q_FREE);
                } else {
                    for (int st = 0; st < 2; ++st) {
                        if (n[st] > 0) ok = ok && wait_phase(&s_full[st][buf(n[st] - 1)], par(n[st] - 1), abort, p.st, T_Q_FREE);
                    }
                }
                if (!ok) break;
                was_two = two;
                if (leader) {
                    const int halves = two ? 2 : 1, bytes = p.q_tokens * p.G * 128;
                    mbar_arrive_expect_tx(&q_full, halves * (D / 64) * bytes);
                    for (int h = 0; h < halves; ++h) {
                        for (int k = 0; k < D / 64; ++k) {
                            tma_load_q(smem + h * C::kTileBytes + k * 16384, &maps.q, w.g * p.G, w.b * p.T + (2 * w.tile + h) * p.mpt, k,
                                       &q_full);
                        }
                    }
                }
                __syncwarp();
                in_flight = !wait_phase(&q_full, static_cast<uint32_t>(tiles) & 1u, abort, p.st, T_Q_FULL);
                ok = !in_flight;
                if (two) {
                    if (ok && leader) mbar_arrive(&q_ready);  // the streams' own warps issue the products
                    __syncwarp();
                    n[0] += steps;
                    n[1] += steps;
                    pos.skip(steps);
                    ++twos;
                }
                for (int j = 0; !two && j < steps && ok; ++j) {
                    const int st = j & 1, i = n[st];
                    ok = wait_phase(&full[pos.slot], pos.phase, abort, p.st, T_MMA_FULL) &&
                         (i < SB || wait_phase(&pv_done[st][buf(i)], par(i) ^ 1u, abort, p.st, T_MMA_PV));  // P in these columns is read
                    tc_fence_after();
                    if (ok && leader) {
                        issue_qk<D>(tmem + st * 128 + buf(i) * 64, smem_u32(smem), smem_u32(ring) + pos.slot * C::kStage);
                        umma_commit(&s_full[st][buf(i)]);
                    }
                    __syncwarp();
                    n[st] += 1;
                    pos.advance(1);
                }
                tiles += ok;
            }
        }
        if (in_flight) {  // Q lands before the CTA may leave
            volatile int dummy = 0;
            wait_phase(&q_full, static_cast<uint32_t>(tiles) & 1u, &dummy, p.st, T_DRAIN);
        }
    } else if (warp >= kProducts) {
        // ---------------------------------------------------------------- P.V, a warp per stream, and its scores if it has a tile of its own
        const int st = warp - kProducts;
        const bool leader = elect_one();
        const uint32_t ring_addr = smem_u32(ring), s_tmem = tmem + st * 128, o_tmem = tmem + 256 + st * D;
        int n = 0, stage = 0;  // steps of this stream and stages used before this tile
        int twos = 0;          // tiles of two halves before it
        bool ok = true;
        for (int r = turn.first; r < turn.end && ok; r += turn.step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            if (r > turn.first) w.find(p, plan, xs);
            for (; w.b < p.B && w.at < xe && ok; w.next(p, plan)) {
                const int steps = w.cut(p, plan, xe) - w.cut(p, plan, xs);
                if (steps <= 0) continue;
                const bool two = w.two();
                const int stride = two ? 1 : 2, first = two ? 0 : st, mine = first < steps ? (steps - first + stride - 1) / stride : 0;
                RingPos<NS> kpos(stage), vpos(stage + first);
                const auto qk = [&](int i) {
                    if (!wait_phase(&full[kpos.slot], kpos.phase, abort, p.st, T_MMA_FULL)) return false;
                    if (n + i >= SB && !wait_phase(&pv_done[st][buf(n + i)], par(n + i) ^ 1u, abort, p.st, T_MMA_PV)) return false;
                    tc_fence_after();
                    if (leader) {
                        issue_qk<D>(s_tmem + buf(n + i) * 64, smem_u32(smem) + st * C::kTileBytes, ring_addr + kpos.slot * C::kStage);
                        umma_commit(&s_full[st][buf(n + i)]);
                        if (i + 1 == mine) umma_commit(&q_free);
                    }
                    __syncwarp();
                    kpos.advance(1);
                    return true;
                };
                if (two) {
                    ok = wait_phase(&q_ready, static_cast<uint32_t>(twos) & 1u, abort, p.st, T_Q_FULL) && qk(0);
                    ++twos;
                }
                for (int i = 0; i < mine && ok; ++i) {
                    const int b = buf(n + i);
                    if (two) ok = F32 || i + 1 >= mine || qk(i + 1);
                    else ok = wait_phase(&full[vpos.slot], vpos.phase, abort, p.st, T_MMA_FULL);
                    ok = ok && wait_phase(&p_ready[st][b], par(n + i), abort, p.st, T_MMA_P);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t p_tmem = s_tmem + b * 64, v = ring_addr + vpos.slot * C::kStage + C::kV;
                        if (F32) issue_pv<D, 3>(o_tmem, p_tmem, v, false);
                        else issue_pv<D, 2>(o_tmem, p_tmem, v, i > 0);
                        umma_commit(&pv_done[st][b]);
                        // a stage is free when both streams have used it, or the one that does has said so twice
                        umma_commit(&empty[vpos.slot]);
                        if (!two) umma_commit(&empty[vpos.slot]);
                    }
                    __syncwarp();
                    vpos.advance(stride);
                    if (F32 && two && i + 1 < mine) ok = qk(i + 1);
                }
                n += mine;
                stage += steps;
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax, two threads a row
        // A wait that ran out ends the waiting, not the loops: the warps go on meeting each other.
        const int st = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, r_in = quad * 32 + lane, pair = 8 + st * 4 + quad;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_addr = tmem + lanes + st * 128;
        constexpr int HALF = D / 2, QUARTER = D / 4;  // columns of O
        const uint32_t o_addr = tmem + lanes + 256 + st * D + half * HALF;  // this thread's
        const auto other = [&](float m) {
            maxima[st][half][r_in] = m;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            return maxima[st][half ^ 1][r_in];
        };
        const int token_in = (r_in * p.inv_G) >> 16, head_in = r_in - token_in * p.G;  // of a half tile
        int n = 0, stage = 0;
        bool failed = false;
        for (int r = turn.first; r < turn.end; r += turn.step) {
            const unsigned xs = r * plan.len, xe = xs + plan.len;
            if (r > turn.first) w.find(p, plan, xs);
            for (; w.b < p.B && w.at < xe; w.next(p, plan)) {
                const int c0 = w.cut(p, plan, xs), c1 = w.cut(p, plan, xe), steps = c1 - c0;
                if (steps <= 0) continue;
                const bool two = w.two();
                const int token0 = (2 * w.tile + (two ? st : 0)) * p.mpt, t = token0 + token_in;
                const bool valid_row = token_in < p.mpt && t < w.q.n;
                const bool warp_has_rows = quad * 32 < min(w.q.n - token0, p.mpt) * p.G;
                const int stride = two ? 1 : 2;
                const auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t where) {
                    if (!failed) failed = !mbar_wait(bar, parity, abort, p.st, DAK_ERR_TIMEOUT, where);
                    __syncwarp();
                    tc_fence_after();
                };
                float m_ref = -INFINITY, l = 0.f;
                // An fp32 output's O is summed here, a step's product at a time: the tensor cores cut off what
                // they add to a sum.
                float sum[F32 ? HALF / 16 : 1][16] = {};
                const auto add_product = [&] {
#pragma unroll
                    for (int q = 0; q < (F32 ? HALF / 16 : 0); ++q) {
                        float o[16];
                        tmem_ld16(o_addr + q * 16, o);
                        tmem_wait(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[q][k] += o[k];
                    }
                };
                int i = 0;
                for (int j = two ? 0 : st; j < steps; j += stride, ++i) {
                    const int key0 = (c0 + j) * 64;
                    uint32_t bits = 0xffffffffu;  // of this thread's keys
                    const bool drafts = key0 + 64 > w.q.len;
                    if (drafts && valid_row) bits = static_cast<uint32_t>(tree_bits(p, w.q, w.b, t, key0) >> (32 * half));
                    wait(&s_full[st][buf(n + i)], par(n + i), T_SM_S);
                    if (drafts) {
                        // Drafted rows' V may hold infinities and NaN, which the probability of zero of a token
                        // that does not see the row would not cancel, and rows behind the drafts anything at all.
                        // They become zeros for the product; what a token sees of them is put in at the end.
                        // Both streams of a step go through them, as either one's product may be first, and a
                        // piece that the other has cleared already is in this one's fence like its own.
                        // (The scores say that the chunk is there.)
                        uint8_t* rows = ring + RingPos<NS>(stage + j).slot * C::kStage + C::kV;
                        const int begin = max(0, w.q.len - key0), end = min(w.q.keys - key0, 64), first = half * 128 + r_in;
                        const auto piece = [&](int e) {
                            const int kr = e / (D / 8), c = e % (D / 8);
                            return rows + (c >> 3) * 16384 + kr * 128 + ((c & 7) << 4);
                        };
                        for (int e = begin * (D / 8) + first; e < end * (D / 8); e += 256) {
                            const uint4 v = ld_shared_ordered(piece(e));
                            if (!not_finite(v)) continue;
                            const int s = key0 + e / (D / 8) - w.q.len;
                            atomicOr(&bad[s >> 5], 1u << (s & 31));
                            any_bad = 1;
                            __threadfence_block();
                            st_shared_ordered(piece(e), finite_part(v));
                        }
                        for (int e = end * (D / 8) + first; e < 64 * (D / 8); e += 256) st_shared_ordered(piece(e), make_uint4(0, 0, 0, 0));
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // O so far, its last product done, to the new reference: this thread's columns
                    const auto grown = [&](float f) {
                        if (F32) {
#pragma unroll
                            for (int q = 0; q < (F32 ? HALF / 16 : 0); ++q) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) sum[q][k] *= f;
                            }
                            return;
                        }
                        wait(&pv_done[st][buf(n + i - 1)], par(n + i - 1), T_SM_O);
#pragma unroll 1
                        for (int q = 0; q < HALF / 16; ++q) {
                            float o[16];
                            tmem_ld16(o_addr + q * 16, o);
                            tmem_wait(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= f;
                            tmem_st16(o_addr + q * 16, o);
                        }
                    };
                    if (warp_has_rows) {  // lanes without rows share a warp's work, warps without any do none
                        if (F32 && i > 0) add_product();  // the last step's: its scores' columns are these
                        softmax_half<F32 ? 3 : 2>(s_addr + buf(n + i) * 64, half, pair, KeysUnset{bits}, p.scale_log2, m_ref, l, i == 0,
                                                  valid_row, other, grown);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[st][buf(n + i)]);
                }
                for (int k = max(0, i - SB); k < i; ++k) wait(&pv_done[st][buf(n + k)], par(n + k), T_SM_O);  // one phase of each buffer's
                if (F32) {  // back to where the results are read from
                    if (i > 0) add_product();
#pragma unroll
                    for (int q = 0; q < (F32 ? HALF / 16 : 0); ++q) tmem_st16(o_addr + q * 16, sum[q]);
                    tmem_wait_st();
                }
                // ---- results: the halves' sums, and where the streams share a tile what the other one has
                const bool both = !two && steps > 1;  // the streams' rows are the same and both had a step
                l += other(l);
                tc_fence_before();
                named_bar<3, kTreeSoftmax>();
                float m_other = -INFINITY, l_other = 0.f;
                if (!two) {
                    maxima[st][half][r_in] = half ? l : m_ref;
                    named_bar<3, kTreeSoftmax>();
                    if (both || st == 1) m_other = maxima[st ^ 1][0][r_in], l_other = maxima[st ^ 1][1][r_in];
                }
                tc_fence_after();
                const float M = fmaxf(m_ref, m_other), base = M == -INFINITY ? 0.f : M;
                const float w_own = both || two || st == 0 ? exp2_ftz(m_ref - base) : 0.f, w_other = exp2_ftz(m_other - base);
                const float total = w_own * l + w_other * l_other;
                const bool whole = c0 == 0 && c1 == w.q.chunks;
                // a token that sees nothing has zeros in O, which stay
                const float inv = !whole || (valid_row && !tree_sees(p, w.q, w.b, t)) ? 1.f : 1.f / total;
                const long long local = (2ll * r + (c0 == 0)) * p.part_rows + (two ? st * 128 : 0) + r_in;  // among the partials
                if (!whole && valid_row && half == 0 && (two || st == 0)) p.ml_part[local] = make_float2(M, total);
                const long long at = ((static_cast<long long>(w.b) * p.T + t) * p.Hq + w.g * p.G + head_in) * D;  // this row in O
                // stream 0's O, or the only one; the other's where both have one
                const uint32_t o0 = tmem + lanes + 256 + (two ? st * D : 0), o1 = tmem + lanes + 256 + D;
                const float w0 = (st == 0 || two ? w_own : w_other) * inv, w1 = (st == 0 ? w_other : w_own) * inv;
                const int col0 = two ? half * HALF : (2 * st + half) * QUARTER, cols = two ? HALF : QUARTER;
                float2 odd[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // NaN where a result is none or infinite
#pragma unroll 1
                for (int col = col0; warp_has_rows && col < col0 + cols; col += 16) {
                    float o[16];
                    tmem_ld16(o0 + col, o);
                    tmem_wait(o);
                    if (both) {
                        float b[16];
                        tmem_ld16(o1 + col, b);
                        tmem_wait(b);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = o[k] * w0 + b[k] * w1;
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] *= w0;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) odd[k & 1] = fma2(make_float2(o[2 * k], o[2 * k + 1]), make_float2(0.f, 0.f), odd[k & 1]);
                    uint32_t out[8];
                    if (valid_row && whole && !F32) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) out[k] = pack_bf16(o[2 * k], o[2 * k + 1]);
                        store32(static_cast<__nv_bfloat16*>(p.O) + at + col, out, p.wide);
                    } else if (valid_row) {
                        float* to = whole ? static_cast<float*>(p.O) + at + col : p.o_part + local * D + col;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) out[k] = __float_as_uint(o[8 * e + k]);
                            store32(to + 8 * e, out, whole ? p.wide : true);
                        }
                    }
                    __syncwarp();
                }
                const bool repair = *reinterpret_cast<volatile int*>(&any_bad) != 0;
                const float none = (odd[0].x + odd[0].y) + (odd[1].x + odd[1].y);
                if (__any_sync(0xffffffffu, valid_row && (repair || (none != 0.f && fabsf(total) < INFINITY)))) {
                    const bool sound = fabsf(total) < INFINITY;  // a row whose own sum is none has scores that are none
                    uint8_t* row = whole ? static_cast<uint8_t*>(p.O) + at * (F32 ? 4 : 2) : reinterpret_cast<uint8_t*>(p.o_part + local * D);
                    const unsigned* drafts = repair ? bad : nullptr;
                    if constexpr (F32) odd_values<D>(p, w.q, w.b, w.g, c0, c1, t, valid_row, sound, drafts, col0, cols, row, false);
                    else odd_values_apart<D>(p, w.q, w.b, w.g, c0, c1, t, valid_row, sound, drafts, col0, cols, row, whole);
                }
                if (repair) {
                    named_bar<3, kTreeSoftmax>();  // all have been through the list
                    if (threadIdx.x < DAK_MAX_TREE / 32) bad[threadIdx.x] = 0;
                    if (threadIdx.x == 32) any_bad = 0;
                }
                n += two ? steps : (steps + 1 - st) / 2;
                stage += steps;
                tc_fence_before();
                named_bar<3, kTreeSoftmax>();  // O is free, and what the threads told each other
                tc_fence_after();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kProducts) {
        tc_fence_after();
        tmem_dealloc(tmem_sh, 512);
    }
}

// ------------------------------------------------------------------------------------
// merge
// ------------------------------------------------------------------------------------
// Block (r, y): eight rows, a warp each, of the tile that begins in range r and ends in a later one:
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over its pieces, in order.
// (No factor is below 1e-37: zero would make NaN of an infinity that V had.)
// What it waits for are loads: the first pieces, which every such tile has, are asked for before it is known
// whether there is one. 4.4 us of one request's 13.5, most of them the launch and two loads one after the
// other; 5 of 157 for 32 rows a kv head of 32 requests, 13 of 224 for 512 rows of 48 (31 MB of partials).
template <int D>
__global__ void __launch_bounds__(32 * kTreeMergeRows) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int LANES = D / 4, AT_ONCE = 32 / LANES;  // pieces that a warp reads at once
    constexpr int EARLY = 2 / AT_ONCE;                  // of a lane's, asked for first
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x;
    const int local = blockIdx.y * kTreeMergeRows + warp, r_in = local & 127, token_in = (r_in * p.inv_G) >> 16;
    if (local >= p.part_rows || token_in >= p.mpt) return;
    const auto slot = [&](int s) { return (2ll * (r + s) + (s == 0)) * p.part_rows + local; };
    const int c = lane % LANES, grp = lane / LANES;
    const auto part = [&](int s) { return *reinterpret_cast<const float4*>(p.o_part + slot(s) * D + c * 4); };
    grid_dep_wait();
    const TreeHead head = p.heads[r];
    float4 early[EARLY];  // range r is not the last
#pragma unroll
    for (int k = 0; k < EARLY; ++k) early[k] = part(grp + k * AT_ONCE);
    float2 first = lane < p.ranges - r ? p.ml_part[slot(lane)] : make_float2(-INFINITY, 0.f);
    // the limits: where a wait ran out, a range's entry may never have been written
    if (head.pieces <= 0 || head.b < 0 || head.b >= p.B || head.g < 0 || head.g >= p.Hkv || head.tile < 0) return;
    const int n = min(head.pieces, p.ranges - r), t = (2 * head.tile + (local >> 7)) * p.mpt + token_in;
    if (t >= min(head.n, p.T)) return;
    if (lane >= n) first = make_float2(-INFINITY, 0.f);
    float M = first.x;
    for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, p.ml_part[slot(s)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](float w, const float4& x) {
        acc.x += w * x.x;
        acc.y += w * x.y;
        acc.z += w * x.z;
        acc.w += w * x.w;
    };
    const auto factor = [&](float m) { return fmaxf(exp2f(m - base), 1e-37f); };
    float f = factor(first.x), l = f * first.y;
#pragma unroll
    for (int k = 0; k < EARLY; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k * AT_ONCE + grp);
        if (grp + k * AT_ONCE < n) add(w, early[k]);
    }
    for (int at = 0; at < n; at += 32) {  // 32 pieces' factors on the lanes
        if (at > 0) {
            const float2 v = at + lane < n ? p.ml_part[slot(at + lane)] : make_float2(-INFINITY, 0.f);
            f = factor(v.x);
            l += f * v.y;
        }
        for (int s0 = at > 0 ? 0 : EARLY * AT_ONCE; s0 < min(32, n - at); s0 += 6 * AT_ONCE) {
            float4 x[6];
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                const int s = s0 + k * AT_ONCE + grp;
                if (s < 32 && at + s < n) x[k] = part(at + s);
            }
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                const int s = s0 + k * AT_ONCE + grp;
                const float w = __shfl_sync(0xffffffffu, f, s & 31);
                if (s < 32 && at + s < n) add(w, x[k]);
            }
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
    TreeRequest q;
    q.len = head.len;
    q.keys = head.keys;
    if (tree_sees(p, q, head.b, t)) acc.x /= l, acc.y /= l, acc.z /= l, acc.w /= l;
    const long long at = ((static_cast<long long>(head.b) * p.T + t) * p.Hq + head.g * p.G + r_in - token_in * p.G) * D + c * 4;
    if (p.o_fp32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = acc;
    } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
// A tile by itself costs about as much as three and two chunks. Short ranges make more partials to merge than
// they save: one chat of 4K, 8 drafts of 32 heads 13.3 us with ranges of 9, 14.9 of 4, 15.3 of 20; four drafts (few)
// 14.0 with 8, 16.9 with 4, 16.3 with 16. 12 chats of up to 2.5K, fp32 heads of 64 (few): 16.5 with a tile's cost of
// 4, 20.4 of 2.
constexpr unsigned kTreeTileCost = 6, kTreeMinRange = 9;        // of tree_kernel
constexpr unsigned kTreeFewTileCost = 4, kTreeFewMinRange = 8;  // of tree_few_kernel
// Tiles that cost no more than this when the cache is full are never cut, and there is no merge (32 drafts of 4
// heads and 4 kv heads, 16 requests over 380 rows: 13.3 us, 19.6 cut; one request of 8 drafts over 380 rows 10.3 and 12.4, over
// 510 11.5 and 11.6; few: one of 4 drafts over 250 rows 10.4 and 12.0, over 380 12.2 and 11.3).
constexpr unsigned kTreeWhole = 24, kTreeFewWhole = 15;
// Larger ones stay whole where that makes the longest range no more than this longer (32 requests of 64 drafts,
// 32/8 heads, 760 rows: 52.9 us, 63.4 cut; few, 64 of 4 over 380 rows 30.8, 33.3 cut).
constexpr unsigned kTreeSlack = 16, kTreeFewSlack = 6;

struct TreeLayout {
    bool few;
    int ranges, part_rows;
    unsigned tile_cost, min_range, slack;
    bool whole;  // no tile is ever cut
    size_t o_part, ml_part, heads;
    size_t total() const { return 16 + o_part + ml_part + heads; }  // the partials begin on 32 bytes
};

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// As many ranges as CTAs run at once; fewer where the cache, full, would not give each the least there may be.
static TreeLayout tree_layout(const dak_placement* KV, int T, int H_q) {
    const int G = H_q / KV->H_kv, mpt = 128 / G;
    TreeLayout x{};
    x.few = T * G <= kTreeFewRows;
    x.tile_cost = x.few ? kTreeFewTileCost : kTreeTileCost;
    x.min_range = x.few ? kTreeFewMinRange : kTreeMinRange;
    const int64_t chunks = (KV->L + 63) / 64, halves = (T + mpt - 1) / mpt;
    x.whole = x.tile_cost + (halves > 1 ? kTreeTwoCost : kTreeOneCost) * chunks <= (x.few ? kTreeFewWhole : kTreeWhole);
    if (x.whole) x.min_range = x.tile_cost + kTreeOneCost;  // of one chunk: a range each
    x.slack = x.whole ? 0x40000000u : x.few ? kTreeFewSlack : kTreeSlack;
    const int64_t slab = (halves / 2) * (x.tile_cost + kTreeTwoCost * chunks) + halves % 2 * (x.tile_cost + kTreeOneCost * chunks);
    const int64_t least = (slab * KV->B * KV->H_kv + x.min_range - 1) / x.min_range;
    const int ctas = x.few ? tree_few_ctas(T * G) : device_sm_count();
    x.ranges = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ctas, least)));
    x.part_rows = T <= mpt ? T * G : std::min(256, 128 + (T - mpt) * G);
    x.o_part = round256(sizeof(float) * 2 * x.ranges * x.part_rows * KV->D);
    x.ml_part = round256(sizeof(float2) * 2 * x.ranges * x.part_rows);
    x.heads = round256(sizeof(TreeHead) * x.ranges);
    return x;
}

// The whole line's cost, with every cache full, fits an int.
static bool line_fits(const dak_placement* KV, int T, int H_q) {
    const int mpt = 128 / (H_q / KV->H_kv);
    const int64_t chunks = (KV->L + 63) / 64, halves = (T + mpt - 1) / mpt;
    return (kTreeTileCost + kTreeOneCost * chunks) * halves * KV->B * KV->H_kv < (1ll << 31) - (1 << 24) &&
           static_cast<int64_t>(KV->B) * KV->H_kv * chunks <= 0x7FFFFFFF && static_cast<int64_t>(KV->B) * T <= 0x7FFFFFFF;
}

// Q's rows as a copy brings them: whole tokens of a kv head's query heads, half a row (64 elements) at a time.
static bool make_query_map(CUtensorMap* map, const void* Q, int64_t tokens, int H_q, int D, int G, int q_tokens) {
    const auto enc = encode_fn();
    if (!enc || fault_due(DAK_FAULT_TENSOR_MAP)) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(tokens), static_cast<cuuint64_t>(D / 64)};
    const cuuint64_t strides[3] = {row, row * H_q, 128};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(q_tokens), 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(Q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F32>
static cudaError_t launch_tree(const TreeParams& p, const TreeMaps& maps, cudaStream_t s) {
    auto k = tree_kernel<D, F32>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), kTreeSmem<D>);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = kTreeSmem<D>;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p, maps);
}

static cudaError_t launch_tree_merge(const TreeParams& p, int D, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges - 1), static_cast<unsigned>((p.part_rows + kTreeMergeRows - 1) / kTreeMergeRows));
    cfg.blockDim = dim3(32 * kTreeMergeRows);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 128 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<128>, p) : cudaLaunchKernelEx(&cfg, tree_merge_kernel<64>, p);
}

}  // namespace dak

using namespace dak;

extern "C" size_t dak_attn_tree_workspace_bytes(const dak_placement* KV, int T, int H_q) {
    if (!KV || KV->kind != 1 || T < 1 || T > DAK_MAX_TREE || H_q < 1 || H_q % KV->H_kv || H_q / KV->H_kv > 16 || !line_fits(KV, T, H_q)) return 0;
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
    if (ranges_overlap(Q, elems * 2, O, elems * (o_fp32 ? 4 : 2))) return DAK_ERR_INVALID;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(workspace, 16) || misaligned(seq_lens, 4) || misaligned(n_new, 4) || misaligned(mask, 8)) return DAK_ERR_ALIGN;
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
    uint8_t* w = static_cast<uint8_t*>(workspace) + (misaligned(workspace, 32) ? 16 : 0);
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
    p.mpt = 128 / G;
    p.inv_G = (65536 + G - 1) / G;
    p.inv_mpt = (65536 + p.mpt - 1) / p.mpt;
    p.q_tokens = std::min(p.mpt, T);
    p.wide = !misaligned(O, 32);
    p.L = KV->L;
    p.h_s = KV->h_s;
    p.host_requests = KV->h_s / KV->H_kv;
    p.part_rows = x.part_rows;
    p.ranges = x.ranges;
    p.tile_cost = x.tile_cost;
    p.min_range = x.min_range;
    p.slack = x.slack;
    p.slab_chunks = (KV->L + 63) / 64;
    p.host_ctas = std::min(x.ranges, tuning && tuning->host_ctas > 0 ? tuning->host_ctas : kTreeHostCtas);
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x.few) {
        p.in_flight[0] = tuning ? tuning->window : 0;
        p.in_flight[1] = tuning ? tuning->hbm_window : 0;
        e = launch_tree_few(p, T * G, D, s);
    } else {
        const int window = D == 128 ? ChunkCfg<128>::kInFlight : ChunkCfg<64>::kInFlight;
        const int most = D == 128 ? ChunkCfg<128>::kStages : ChunkCfg<64>::kStages;
        p.in_flight[0] = std::min(most, tuning && tuning->window > 0 ? tuning->window : window);
        p.in_flight[1] = std::min(most, tuning && tuning->hbm_window > 0 ? tuning->hbm_window : window);
        const int64_t slabs = static_cast<int64_t>(KV->B) * KV->H_kv;
        TreeMaps maps{};
        for (int tier = 0; tier < 2; ++tier) {
            const int64_t n = tier ? slabs - KV->h_s : KV->h_s;
            if (n > 0 && !make_chunk_map(&maps.tier[tier], p.kv[tier], n * p.slab_chunks, D)) return DAK_ERR_CUDA;
        }
        if (!make_query_map(&maps.q, Q, static_cast<int64_t>(KV->B) * T, H_q, D, G, p.q_tokens)) return DAK_ERR_CUDA;
        e = D == 128 ? (o_fp32 ? launch_tree<128, true>(p, maps, s) : launch_tree<128, false>(p, maps, s))
                     : (o_fp32 ? launch_tree<64, true>(p, maps, s) : launch_tree<64, false>(p, maps, s));
    }
    if (x.whole || x.ranges == 1) return cuda_status(e);
    return cuda_status(e == cudaSuccess ? launch_tree_merge(p, D, s) : e);
}
