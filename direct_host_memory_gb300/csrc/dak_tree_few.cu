// The attention of drafted trees for few query rows a kv head (up to kTreeFewRows tokens x heads), where
// a 128-row tile of the tensor cores would be mostly empty: warp MMAs with the rows on their narrow side, as
// in the pass over the own caches of dak_serve.cu,
//   S^T (16 tokens x rows) = K (16 x D) . Q^T (D x rows)
//   O^T (D x rows)        += V^T (D x 16 tokens) . P^T (16 tokens x rows)
// in NB blocks of 8 rows. A producer thread streams 64-token chunks into a ring, four warps take 16 tokens
// each and are merged at a tile's (or a range's) end. How work is cut: dak_tree.cuh.
//
// What bounds it: the cache's bytes (32 requests of 4 drafts and 32/8 heads of 128 over 7K to 8K 150 us, 145 at
// the copy rate; heads of 64 81 us, 73). Small calls the latency of the start, the first chunks, the warps' merge
// and the pieces': one request over 4K 14 us, over 5 rows 7, 12 of 16/16 heads of 64 over up to 2.5K, fp32 output, 17 us (8.6). Five
// warps and two CTAs an SM leave 168 registers a thread, of which 9 to 16 rows of heads of 128 spill a little (about 105
// bytes; 152 us in that batch, fp32 output 165; heads of 64 do not, 81 and 94) and more rows O^T and Q: 24 rows of heads of
// 64 102 us and 13.5 for one request (121 and 12.2 by tree_kernel), 32 rows 157 and 17.6.
#include <algorithm>
#include <atomic>

#include "dak_tree.cuh"

namespace dak {

constexpr int kFewConsumers = 4;
constexpr int kFewThreads = 32 * (1 + kFewConsumers);
constexpr int kFewMaxStages = 6;

enum : uint32_t { W_PROD_EMPTY = 0x81, W_CONS_FULL, W_DRAIN };

template <int D>
constexpr int few_stage_bytes() { return 2 * 64 * D * 2; }

// CTAs an SM by registers: O^T and Q of more rows leave room for two.
constexpr int few_ctas_per_sm(int NB) { return NB == 1 ? 3 : 2; }

template <int D, int NB>
constexpr int few_fixed_bytes() {  // the four warps' merge
    return 2 * 8 * NB * (D + 2) * 4;
}
template <int D, int NB>
constexpr int few_stages() {  // as many as the CTAs of an SM have room for
    const int room = (228 * 1024 / few_ctas_per_sm(NB) - 1024 - 192 - few_fixed_bytes<D, NB>()) / few_stage_bytes<D>();
    return room < kFewMaxStages ? room : kFewMaxStages;
}

template <int D, int NB, int PARTS>
__global__ void __launch_bounds__(kFewThreads, few_ctas_per_sm(NB)) tree_few_kernel(const __grid_constant__ TreeParams p) {
    constexpr int KS = D / 16;                // k-steps of the scores, row tiles of O^T
    constexpr int CHUNK_BYTES = 64 * D * 2;   // K (or V) of a chunk
    constexpr int STAGE = 2 * CHUNK_BYTES, W = few_stages<D, NB>();
    constexpr int ROWS = 8 * NB;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[W], empty[W];
    __shared__ int abort_flag, any_left_out;  // of the tile at work's drafts, of the product
    volatile int* abort = &abort_flag;
    float* comb = reinterpret_cast<float*>(smem + W * STAGE);  // [2][ROWS][D + 2]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        abort_flag = any_left_out = 0;
        for (int s = 0; s < W; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kFewConsumers);
        }
        fence_mbar_init();
    }
    grid_dep_wait();  // launched while the previous kernel ends
    grid_dep_launch();
    const TreePlan plan = tree_plan(p);
    if (threadIdx.x == 32 && static_cast<int>(blockIdx.x) >= plan.ranges) p.heads[blockIdx.x].pieces = 0;
    const TreeTurn turn = tree_turn(p, plan);
    TreeWalk w;
    if (turn.first < turn.end) w.find(p, plan, turn.first * plan.len);
    __syncthreads();

    if (warp == 0) {
        const uint64_t policy = policy_evict_first();
        int s = 0, i = 0, landed = 0;  // copies issued, and of these seen to have landed
        uint32_t phase = 0;
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
                    const uint8_t* base = tier ? p.kv[1] + (slab - p.h_s) * p.head_bytes : p.kv[0] + slab * p.head_bytes;
                    for (int c = c0; c < c1; ++c, ++i) {
                        if (i >= W) ok = mbar_wait(&empty[s], phase ^ 1u, abort, p.st, DAK_ERR_TIMEOUT, W_PROD_EMPTY);
                        for (; ok && i - landed >= window; ++landed) {
                            ok = mbar_wait(&full[landed % W], static_cast<uint32_t>(landed / W) & 1u, abort, p.st, DAK_ERR_TIMEOUT, W_PROD_EMPTY);
                        }
                        if (!ok) break;
                        mbar_arrive_expect_tx(&full[s], STAGE);
                        bulk_g2s(smem + s * STAGE, base + static_cast<long long>(c) * STAGE, STAGE, &full[s], policy);
                        if (++s == W) s = 0, phase ^= 1u;
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
            for (landed = max(landed, i - W); landed < i; ++landed) {
                mbar_wait(&full[landed % W], static_cast<uint32_t>(landed / W) & 1u, &dummy, p.st, DAK_ERR_TIMEOUT, W_DRAIN);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int wk = warp - 1;
    const int q4 = lane & 3, ra = lane >> 2;  // MMA fragments: columns 2 q4, 2 q4 + 1; rows ra, ra + 8
    const int mi = lane >> 3, rr = lane & 7;  // ldmatrix: matrix, row in it
    const auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewConsumers) : "memory"); };
    int s = 0;
    uint32_t phase = 0;
    bool failed = false;  // a wait ran out: skip the work but keep meeting the named barriers
    for (int r = turn.first; r < turn.end; r += turn.step) {
        const unsigned xs = r * plan.len, xe = xs + plan.len;
        if (r > turn.first) w.find(p, plan, xs);
        for (; w.b < p.B && w.at < xe; w.next(p, plan)) {
            const int c0 = w.cut(p, plan, xs), c1 = w.cut(p, plan, xe), rows = w.q.n * p.G;
            if (c0 >= c1) continue;
            // row r of this kv head: token r / G, head r % G of the request
            const auto row_at = [&](int row) {
                const int t = (row * p.inv_G) >> 16;
                return ((static_cast<long long>(w.b) * p.T + t) * p.Hq + w.g * p.G + row - t * p.G) * D;
            };
            uint32_t q[NB][KS][2];  // rows nb * 8 + ra, elements ks * 16 + 2 q4 (+ 8)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int row = nb * 8 + ra;
                const __nv_bfloat16* from = p.Q + (row < rows ? row_at(row) : 0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        q[nb][ks][j] = row < rows ? *reinterpret_cast<const uint32_t*>(from + ks * 16 + 2 * q4 + 8 * j) : 0u;
                    }
                }
            }
            float o[KS][NB][4];  // elements 16 t + ra (+ 8), rows nb * 8 + 2 q4 (+ 1)
#pragma unroll
            for (int t = 0; t < KS; ++t) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) o[t][nb][0] = o[t][nb][1] = o[t][nb][2] = o[t][nb][3] = 0.f;
            }
            float m[NB][2], l[NB][2];  // reference and this lane's sum of rows nb * 8 + 2 q4 (+ 1)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.f;

            for (int c = c0; c < c1; ++c) {
                const int key0 = c * 64 + 16 * wk;  // of this warp's 16
                const int valid = w.q.keys - key0;
                uint32_t seen[NB][2];  // of the 16, by row
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) seen[nb][0] = seen[nb][1] = 0xFFFFu;
                const bool drafts = key0 + 16 > w.q.len;
                if (drafts) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = nb * 8 + 2 * q4 + e;
                            if (row < rows) seen[nb][e] = static_cast<uint32_t>(tree_bits(p, w.q, w.b, (row * p.inv_G) >> 16, key0)) & 0xFFFFu;
                        }
                    }
                }
                if (!failed && !mbar_wait(&full[s], phase, abort, p.st, DAK_ERR_TIMEOUT, W_CONS_FULL)) failed = true;
                if (!__any_sync(0xffffffffu, failed) && valid > 0) {
                    const uint32_t ks_base = smem_u32(smem + s * STAGE), vs_base = ks_base + CHUNK_BYTES;
                    float sc[NB][4];  // tokens ra (0, 1) and ra + 8 (2, 3), rows nb * 8 + 2 q4 (+ 1)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
                    {
                        const int tok = 16 * wk + (mi & 1) * 8 + rr;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            const int cc = ks * 2 + (mi >> 1);
                            uint32_t a0, a1, a2, a3;
                            ldsm_x4(ks_base + static_cast<uint32_t>(tok * D * 2 + ((cc ^ (tok & 7)) << 4)), a0, a1, a2, a3);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(sc[nb], a0, a1, a2, a3, q[nb][ks][0], q[nb][ks][1]);
                        }
                    }
                    bool grown = false;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sc[nb][e] = seen[nb][e & 1] >> (e < 2 ? ra : ra + 8) & 1u ? sc[nb][e] * p.scale_log2 : -INFINITY;
                        }
                        grown |= fmaxf(sc[nb][0], sc[nb][2]) > m[nb][0] + 8.f;
                        grown |= fmaxf(sc[nb][1], sc[nb][3]) > m[nb][1] + 8.f;
                    }
                    // a row's reference moves only when one of its scores outgrows it by 2^8
                    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float mx = fmaxf(sc[nb][e], sc[nb][2 + e]);
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                                mx = fmaxf(mx, m[nb][e]);
                                const float f = mx == -INFINITY ? 1.f : exp2_ftz(m[nb][e] - mx);
                                m[nb][e] = mx;
                                l[nb][e] *= f;
#pragma unroll
                                for (int tt = 0; tt < KS; ++tt) {
                                    o[tt][nb][e] *= f;
                                    o[tt][nb][2 + e] *= f;
                                }
                            }
                        }
                    }
                    uint32_t pb[NB][PARTS][2];  // P^T as the B operand: tokens 0..7 and 8..15
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float base = m[nb][e & 1] == -INFINITY ? 0.f : m[nb][e & 1];
                            x[e] = sc[nb][e] = exp2_ftz(sc[nb][e] - base);
                            l[nb][e & 1] += x[e];
                        }
#pragma unroll
                        for (int k = 0; k < PARTS; ++k) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t v = pack_bf16(x[2 * h], x[2 * h + 1]);
                                pb[nb][k][h] = movmatrix(v);
                                x[2 * h] -= bf_lo(v);
                                x[2 * h + 1] -= bf_hi(v);
                            }
                        }
                    }
                    // Rows behind the last may hold anything, also infinities and NaN, which a probability of zero
                    // would not cancel; drafted rows likewise for a row that does not see them: their infinities and
                    // NaN are left out of the product and put in at the end where they are seen.
                    const int tok = 16 * wk + (mi >> 1) * 8 + rr;
                    const uint32_t lo = pair_mask(valid - 2 * q4), hi = pair_mask(valid - 8 - 2 * q4);
                    const uint32_t committed_lo = pair_mask(w.q.len - key0 - 2 * q4), committed_hi = pair_mask(w.q.len - key0 - 8 - 2 * q4);
                    uint32_t left_out = 0;
#pragma unroll
                    for (int tt = 0; tt < KS; ++tt) {
                        const int cc = tt * 2 + (mi & 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4_t(vs_base + static_cast<uint32_t>(tok * D * 2 + ((cc ^ (tok & 7)) << 4)), a0, a1, a2, a3);
                        if (drafts) {
                            const uint32_t x0 = tree_not_finite(a0) & ~committed_lo & lo, x1 = tree_not_finite(a1) & ~committed_lo & lo;
                            const uint32_t x2 = tree_not_finite(a2) & ~committed_hi & hi, x3 = tree_not_finite(a3) & ~committed_hi & hi;
                            left_out |= x0 | x1 | x2 | x3;
                            a0 &= lo & ~x0;
                            a1 &= lo & ~x1;
                            a2 &= hi & ~x2;
                            a3 &= hi & ~x3;
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            // for an fp32 output the chunk's product apart: the tensor cores cut off what they add to a sum
                            float apart[4] = {0.f, 0.f, 0.f, 0.f};
                            float(&to)[4] = PARTS == 3 ? apart : o[tt][nb];
#pragma unroll
                            for (int k = 0; k < PARTS; ++k) mma_bf16_16816(to, a0, a1, a2, a3, pb[nb][k][0], pb[nb][k][1]);
                            if (PARTS == 3) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[tt][nb][e] += apart[e];
                            }
                        }
                    }
                    if (left_out) any_left_out = 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                if (++s == W) s = 0, phase ^= 1u;
            }

            // ---- merge the four warps (2 and 3 into 0 and 1, then those two)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 4);
                    l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 8);
                    l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 16);
                }
            }
            float* mine = comb + (wk & 1) * ROWS * (D + 2);
            const auto put = [&] {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = nb * 8 + 2 * q4 + e;
                        if (h >= rows) continue;
#pragma unroll
                        for (int tt = 0; tt < KS; ++tt) {
                            mine[h * (D + 2) + tt * 16 + ra] = o[tt][nb][e];
                            mine[h * (D + 2) + tt * 16 + ra + 8] = o[tt][nb][2 + e];
                        }
                        if (ra == 0) {
                            mine[h * (D + 2) + D] = m[nb][e];
                            mine[h * (D + 2) + D + 1] = l[nb][e];
                        }
                    }
                }
            };
            if (wk >= 2) put();
            bar();
            if (wk < 2) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = nb * 8 + 2 * q4 + e;
                        if (h >= rows) continue;
                        const float* row = mine + h * (D + 2);
                        const float m2 = row[D], M = fmaxf(m[nb][e], m2), base = M == -INFINITY ? 0.f : M;
                        const float fa = exp2_ftz(m[nb][e] - base), fb = exp2_ftz(m2 - base);
                        m[nb][e] = M;
                        l[nb][e] = l[nb][e] * fa + row[D + 1] * fb;
#pragma unroll
                        for (int tt = 0; tt < KS; ++tt) {
                            o[tt][nb][e] = o[tt][nb][e] * fa + row[tt * 16 + ra] * fb;
                            o[tt][nb][2 + e] = o[tt][nb][2 + e] * fa + row[tt * 16 + ra + 8] * fb;
                        }
                    }
                }
                __syncwarp();  // a row is read whole before it is written
                put();
            }
            bar();
            const bool whole = c0 == 0 && c1 == w.q.chunks, repair = *reinterpret_cast<volatile int*>(&any_left_out) != 0;
            bool odd = false;
            const auto combined = [&](int h, int d, float(&v)[4]) {  // of two warps each
                const float* ca = comb + h * (D + 2);
                const float* cb = ca + ROWS * (D + 2);
                const float M = fmaxf(ca[D], cb[D]), base = M == -INFINITY ? 0.f : M;
                const float fa = exp2_ftz(ca[D] - base), fb = exp2_ftz(cb[D] - base);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = fa * ca[d + k] + fb * cb[d + k];
                return make_float2(M, fa * ca[D + 1] + fb * cb[D + 1]);
            };
            const auto store = [&](int h, int d, const float2& ml, float(&v)[4]) {
                if (!whole) {
                    const long long at = (2ll * r + (c0 == 0)) * p.part_rows + h;
                    *reinterpret_cast<float4*>(p.o_part + at * D + d) = make_float4(v[0], v[1], v[2], v[3]);
                    if (d == 0) p.ml_part[at] = ml;
                    return;
                }
                // a token that sees nothing has zeros, which stay
                if (tree_sees(p, w.q, w.b, (h * p.inv_G) >> 16)) v[0] /= ml.y, v[1] /= ml.y, v[2] /= ml.y, v[3] /= ml.y;
                const long long at = row_at(h) + d;
                if (PARTS == 3) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = make_float4(v[0], v[1], v[2], v[3]);
                else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            };
            for (int e = threadIdx.x - 32; e < rows * (D / 4); e += 32 * kFewConsumers) {
                const int h = e / (D / 4), d = e % (D / 4) * 4;
                float v[4];
                const float2 ml = combined(h, d, v);
                // (a row whose own sum is none has scores that are none)
                odd |= fmaf(v[0], 0.f, v[1] * 0.f) + fmaf(v[2], 0.f, v[3] * 0.f) != 0.f && fabsf(ml.y) < INFINITY;
                store(h, d, ml, v);
            }
            // An infinity or NaN in V of a row before the drafts is in the sum of every token: here it becomes what it
            // is, where a weight in parts (infinity times a part of zero) or a factor of zero has made NaN of it. Those of
            // the drafts, which the products did not meet, are put in where the token sees them.
            if (odd || repair) {
                const int d = (threadIdx.x - 32) % (D / 4) * 4;  // the same in all of a thread's rows
                const auto v_at = [&](int key) {
                    return reinterpret_cast<const uint2*>(tree_v_piece(p, w.b, w.g, D, key, d >> 3)) + (d >> 2 & 1);
                };
                float cached[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int key = c0 * 64; key < min(c1 * 64, w.q.len); ++key) add_not_finite(cached, v_at(key));
#pragma unroll 1
                for (int h = (threadIdx.x - 32) / (D / 4); h < rows; h += 32 * kFewConsumers / (D / 4)) {
                    float v[4], x[4] = {cached[0], cached[1], cached[2], cached[3]};
                    const float2 ml = combined(h, d, v);
#pragma unroll 1
                    for (int key = max(c0 * 64, w.q.len); key < min(c1 * 64, w.q.keys); ++key) {
                        if (tree_bits(p, w.q, w.b, (h * p.inv_G) >> 16, key) & 1) add_not_finite(x, v_at(key));
                    }
                    if (!(fabsf(ml.y) < INFINITY)) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (x[k] != 0.f) v[k] = x[k];
                    }
                    store(h, d, ml, v);
                }
            }
            if (repair) {
                bar();  // all have read it
                if (threadIdx.x == 32) any_left_out = 0;
            }
            bar();  // comb is rewritten by the next tile
        }
    }
}

template <int D, int NB, int PARTS>
static cudaError_t launch_few(const TreeParams& given, cudaStream_t s) {
    constexpr int W = few_stages<D, NB>(), kSmem = W * few_stage_bytes<D>() + few_fixed_bytes<D, NB>();
    TreeParams p = given;
    for (int& n : p.in_flight) n = n > 0 ? std::min(n, W) : W;
    auto k = tree_few_kernel<D, NB, PARTS>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p);
}

template <int D>
static cudaError_t launch_few_d(const TreeParams& p, int rows, cudaStream_t s) {
    if (rows <= 8) return p.o_fp32 ? launch_few<D, 1, 3>(p, s) : launch_few<D, 1, 2>(p, s);
    return p.o_fp32 ? launch_few<D, 2, 3>(p, s) : launch_few<D, 2, 2>(p, s);
}

int tree_few_ctas(int rows) { return few_ctas_per_sm(rows <= 8 ? 1 : 2) * device_sm_count(); }

cudaError_t launch_tree_few(const TreeParams& p, int rows, int D, cudaStream_t s) {
    return D == 128 ? launch_few_d<128>(p, rows, s) : launch_few_d<64>(p, rows, s);
}

}  // namespace dak
