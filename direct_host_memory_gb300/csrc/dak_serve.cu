// Decode attention for serving long chats: dak_attn_acc (which also accumulates every position's
// attention weight) and dak_attn_prefix (whose requests share prefixes). Up to three launches:
//   the prefix pass (dak_prefix.cu), partials per row and key range;
//   the own pass (serve_kernel), partials per row and context split, and the scores if weights are
//     accumulated;
//   the merge (serve_merge_kernel) of both into O, and the weights from the scores.
// The own pass reads a cache as dak_attn does (layout and tiers: dak_attn.cu): a producer thread
// streams 64-token chunks into a shared-memory ring, four consumer warps take 16 tokens each.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "dak_device.cuh"

namespace dak {

struct ServeParams {
    const __nv_bfloat16* Q;  // [B][Hq][D]
    const uint8_t* kv[2];    // host tier (device-visible), HBM tier
    const int* seq_lens;
    float* o_part;    // [B][Hq][n_split][D], unnormalised
    float2* ml_part;  // [B][Hq][n_split]: reference (log2 domain), sum
    float* scores;    // [B * Hkv][score_pitch][G rounded up to even], log2 domain, or null
    int score_pitch;
    int B, Hq, Hkv, G, L, h_s, n_split, split_len;
    float scale_log2;
    long long head_bytes;
    int n_host_ctas, n_hbm_ctas, host_window, hbm_window;
    unsigned host_units, hbm_units;
    int wait_newest;  // as in dak_attn (tuning pdl 2)
    int wait_first;   // without programmatic launch asked for: the previous kernel may write anything
    int wait_late;    // the previous kernel is the call's prefix pass: only this grid's end waits for it
    DevStatus* st;
    unsigned* link;
    unsigned link_after;
};

constexpr int kChunk = 64;
constexpr int kConsumers = 4;
constexpr int kServeThreads = 32 * (1 + kConsumers);
// Chunks in flight of a CTA, by D: three CTAs an SM keep 192 or 144 KiB on their way. More queue in the
// memory system (32 requests over 8K, D 128: 2 or 3 169 us, 4 185 us), fewer leave it idle (12 requests of
// 16 kv heads over up to 2.5K, D 64: 18.8 us with 2, 17.2 with 3).
constexpr int serve_stages(int D) { return D == 128 ? 2 : 3; }
constexpr int kServeMaxStages = 5;

enum : uint32_t { V_PROD_EMPTY = 0x61, V_CONS_FULL, V_DRAIN };

struct ServeUnit {
    int b, g, s;
    int t0, t1;  // tokens; none: t0 >= t1
    int len;     // tokens of the request
    const uint8_t* base;
};

// Unit u of a tier: by split and then by slab, so that CTAs that take every n-th unit share ragged
// lengths evenly (short requests have none of the later splits).
__device__ __forceinline__ ServeUnit serve_unit(const ServeParams& p, unsigned u, int tier) {
    const unsigned slabs = tier ? static_cast<unsigned>(p.B) * p.Hkv - p.h_s : p.h_s;
    const unsigned local = u % slabs, slab = local + (tier ? p.h_s : 0);
    ServeUnit x;
    x.s = static_cast<int>(u / slabs);
    x.b = static_cast<int>(slab / p.Hkv);
    x.g = static_cast<int>(slab % p.Hkv);
    x.len = p.seq_lens ? min(max(p.seq_lens[x.b], 0), p.L) : p.L;
    x.t0 = x.s * p.split_len;
    x.t1 = min(x.len, x.t0 + p.split_len);
    x.base = p.kv[tier] + static_cast<long long>(local) * p.head_bytes;
    return x;
}

// The query heads of a kv head are the narrow side of both products, so that they are the 8-wide N
// of the warp MMAs (NB blocks of 8 heads) and tokens or head elements the 16-high M:
//   S^T (16 tokens x heads) = K (16 x D) . Q^T (D x heads)
//   O^T (D x heads)        += V^T (D x 16 tokens) . P^T (16 tokens x heads)
// Against the other way round (heads in 16 rows) that is half the MMAs and half the registers of O
// and Q for up to 8 heads, and three CTAs an SM instead of two; with them the pass is bound by
// memory where that way the work per chunk held it up (32 requests over 7K to 8.2K, 32 query and 8 kv
// heads, D 128, with the weights' scores: 155 us, 6.5 TB/s; the whole call 168 us instead of 189).
// Sums, references and scores stay in fp32. P^T moves from the accumulators' layout into
// the second product's by a transpose of 8x8 blocks, in PARTS bf16 parts (two keep the rounding of
// the weights far below a bf16 output's, three below an fp32 one's). The reference of a head's
// exponents moves only when a score outgrows it by 2^8, which a vote finds.
template <int D, int NB, int PARTS>
__global__ void __launch_bounds__(kServeThreads, NB == 1 ? 3 : 2) serve_kernel(const ServeParams p) {
    constexpr int KS = D / 16;                  // k-steps of the scores, row tiles of O^T
    constexpr int CHUNK_BYTES = kChunk * D * 2;  // K (or V) of a chunk
    constexpr int STAGE = 2 * CHUNK_BYTES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[8], empty[8];
    __shared__ int abort_flag;
    volatile int* abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool host = static_cast<int>(blockIdx.x) < p.n_host_ctas;
    const int tier = host ? 0 : 1, W = host ? p.host_window : p.hbm_window;
    const unsigned u0 = host ? blockIdx.x : blockIdx.x - p.n_host_ctas, step = host ? p.n_host_ctas : p.n_hbm_ctas;
    const unsigned units = host ? p.host_units : p.hbm_units;
    float* comb = reinterpret_cast<float*>(smem + static_cast<size_t>(W) * STAGE);  // [2][G][D + 2]

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < W; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        fence_mbar_init();
    }
    __syncthreads();
    if (p.wait_first) grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            const bool link = host && p.link;
            if (link) link_wait(p.link, p.link_after, p.st);
            int s = 0, i = 0;
            uint32_t phase = 0;
            bool waited = false;
            for (unsigned u = u0; u < units && !*abort; u += step) {
                const ServeUnit x = serve_unit(p, u, tier);
                for (int t = x.t0; t < x.t1; t += kChunk, ++i) {
                    if (p.wait_newest && !waited && t + kChunk >= x.len) {
                        grid_dep_wait();  // this chunk holds the newest token, which the previous kernel writes
                        waited = true;
                    }
                    if (i >= W && !mbar_wait(&empty[s], phase ^ 1u, abort, p.st, DAK_ERR_TIMEOUT, V_PROD_EMPTY)) goto done;
                    mbar_arrive_expect_tx(&full[s], STAGE);
                    bulk_g2s(smem + static_cast<size_t>(s) * STAGE, x.base + static_cast<long long>(t / kChunk) * STAGE, STAGE,
                             &full[s], pol);
                    if (++s == W) s = 0, phase ^= 1u;
                }
            }
        done:
            if (link) link_signal(p.link);
            volatile int dummy = 0;
            for (int k = 0; k < W && k < i; ++k) {
                const int last = ((i - 1 - k) / W) * W + k;
                mbar_wait(&full[k], static_cast<uint32_t>((last / W) & 1), &dummy, p.st, DAK_ERR_TIMEOUT, V_DRAIN);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    if (!p.wait_late) grid_dep_wait();
    const int w = warp - 1;
    const int q4 = lane & 3, ra = lane >> 2;  // MMA fragments: columns 2 q4, 2 q4 + 1; rows ra, ra + 8
    const int mi = lane >> 3, rr = lane & 7;  // ldmatrix: matrix, row in it
    const int Gp = (p.G + 1) & ~1;
    int s = 0;
    uint32_t phase = 0;
    bool failed = false;  // a wait ran out: skip the work but keep meeting the named barriers
    // Q of a unit as the B operand: heads nb * 8 + ra, elements ks * 16 + 2 q4 (+ 8)
    const auto load_q = [&](const ServeUnit& x, uint32_t(&q)[NB][KS][2]) {
        const __nv_bfloat16* qb = p.Q + (static_cast<long long>(x.b) * p.Hq + static_cast<long long>(x.g) * p.G) * D;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int h = nb * 8 + ra;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    q[nb][ks][j] = h < p.G ? *reinterpret_cast<const uint32_t*>(qb + h * D + ks * 16 + 2 * q4 + 8 * j) : 0u;
                }
            }
        }
    };
    for (unsigned u = u0; u < units; u += step) {
        const ServeUnit x = serve_unit(p, u, tier);
        if (x.t0 >= x.t1) continue;
        uint32_t q[NB][KS][2];
        load_q(x, q);
        float o[KS][NB][4];  // rows 16 t + ra (+ 8), heads nb * 8 + 2 q4 (+ 1)
#pragma unroll
        for (int t = 0; t < KS; ++t) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) o[t][nb][0] = o[t][nb][1] = o[t][nb][2] = o[t][nb][3] = 0.f;
        }
        float m[NB][2], l[NB][2];  // reference and this lane's sum of heads nb * 8 + 2 q4 (+ 1)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.f;

        for (int t = x.t0; t < x.t1; t += kChunk) {
            if (!failed && !mbar_wait(&full[s], phase, abort, p.st, DAK_ERR_TIMEOUT, V_CONS_FULL)) failed = true;
            const int valid = min(kChunk, x.t1 - t) - 16 * w;  // tokens of this warp's 16 that are real
            if (!failed && valid > 0) {
                const uint32_t ks_base = smem_u32(smem + static_cast<size_t>(s) * STAGE);
                const uint32_t vs_base = ks_base + CHUNK_BYTES;
                float sc[NB][4];  // tokens ra (0, 1) and ra + 8 (2, 3), heads nb * 8 + 2 q4 (+ 1)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
                {
                    const int tok = 16 * w + (mi & 1) * 8 + rr;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int c = ks * 2 + (mi >> 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4(ks_base + static_cast<uint32_t>(tok * D * 2 + ((c ^ (tok & 7)) << 4)), a0, a1, a2, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(sc[nb], a0, a1, a2, a3, q[nb][ks][0], q[nb][ks][1]);
                    }
                }
                bool grown = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[nb][e] = (e < 2 ? ra : ra + 8) < valid ? sc[nb][e] * p.scale_log2 : -INFINITY;
                    }
                    grown |= fmaxf(sc[nb][0], sc[nb][2]) > m[nb][0] + 8.f;
                    grown |= fmaxf(sc[nb][1], sc[nb][3]) > m[nb][1] + 8.f;
                }
                if (p.scores) {
                    // rows past the valid ones lie inside the padded slab
                    float* at = p.scores + ((static_cast<long long>(x.b) * p.Hkv + x.g) * p.score_pitch + t + 16 * w + ra) * Gp;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const int h = nb * 8 + 2 * q4;
                        if (h < Gp) {
                            *reinterpret_cast<float2*>(at + h) = make_float2(sc[nb][0], sc[nb][1]);
                            *reinterpret_cast<float2*>(at + 8 * Gp + h) = make_float2(sc[nb][2], sc[nb][3]);
                        }
                    }
                }
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
                    float r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float base = m[nb][e & 1] == -INFINITY ? 0.f : m[nb][e & 1];
                        r[e] = exp2_ftz(sc[nb][e] - base);
                        l[nb][e & 1] += r[e];
                    }
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t v = pack_bf16(r[2 * h], r[2 * h + 1]);
                            pb[nb][k][h] = movmatrix(v);
                            r[2 * h] -= bf_lo(v);
                            r[2 * h + 1] -= bf_hi(v);
                        }
                    }
                }
                {
                    const int tok = 16 * w + (mi >> 1) * 8 + rr;
                    // rows past the valid tokens may hold anything, also infinities and NaN, which a
                    // probability of zero would not cancel
                    const uint32_t lo = pair_mask(valid - 2 * q4), hi = pair_mask(valid - 8 - 2 * q4);
#pragma unroll
                    for (int tt = 0; tt < KS; ++tt) {
                        const int c = tt * 2 + (mi & 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4_t(vs_base + static_cast<uint32_t>(tok * D * 2 + ((c ^ (tok & 7)) << 4)), a0, a1, a2, a3);
                        if (valid < 16) {
                            a0 &= lo;
                            a1 &= lo;
                            a2 &= hi;
                            a3 &= hi;
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            // for an fp32 output the chunk's product apart: the tensor cores cut off what
                            // they add to a sum (30 requests over 7K: 5.7e-7 with the sum there, 2.7e-7
                            // so, in the same time)
                            float apart[4] = {0.f, 0.f, 0.f, 0.f};
                            float(&to)[4] = PARTS == 3 ? apart : o[tt][nb];
#pragma unroll
                            for (int k = 0; k < PARTS; ++k) {
                                mma_bf16_16816(to, a0, a1, a2, a3, pb[nb][k][0], pb[nb][k][1]);
                            }
                            if (PARTS == 3) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[tt][nb][e] += apart[e];
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == W) s = 0, phase ^= 1u;
        }

        // ---- merge the four warps (2 and 3 into 0 and 1, then those two), write the partial
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 4);
                l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 8);
                l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], 16);
            }
        }
        const auto bar = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory"); };
        const auto put = [&] {
            float* row = comb + static_cast<size_t>(w & 1) * p.G * (D + 2);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = nb * 8 + 2 * q4 + e;
                    if (h >= p.G) continue;
#pragma unroll
                    for (int tt = 0; tt < KS; ++tt) {
                        row[h * (D + 2) + tt * 16 + ra] = o[tt][nb][e];
                        row[h * (D + 2) + tt * 16 + ra + 8] = o[tt][nb][2 + e];
                    }
                    if (ra == 0) {
                        row[h * (D + 2) + D] = m[nb][e];
                        row[h * (D + 2) + D + 1] = l[nb][e];
                    }
                }
            }
        };
        if (w >= 2) put();
        bar();
        if (w < 2) {
            const float* row = comb + static_cast<size_t>(w) * p.G * (D + 2);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = nb * 8 + 2 * q4 + e;
                    if (h >= p.G) continue;
                    const float m2 = row[h * (D + 2) + D], M = fmaxf(m[nb][e], m2), base = M == -INFINITY ? 0.f : M;
                    const float fa = exp2_ftz(m[nb][e] - base), fb = exp2_ftz(m2 - base);
                    m[nb][e] = M;
                    l[nb][e] = l[nb][e] * fa + row[h * (D + 2) + D + 1] * fb;
#pragma unroll
                    for (int tt = 0; tt < KS; ++tt) {
                        o[tt][nb][e] = o[tt][nb][e] * fa + row[h * (D + 2) + tt * 16 + ra] * fb;
                        o[tt][nb][2 + e] = o[tt][nb][2 + e] * fa + row[h * (D + 2) + tt * 16 + ra + 8] * fb;
                    }
                }
            }
            __syncwarp();  // a row is read whole before it is written
            put();
        }
        bar();
        const long long row0 = static_cast<long long>(x.b) * p.Hq + static_cast<long long>(x.g) * p.G;
        for (int e = threadIdx.x - 32; e < p.G * (D / 2); e += 32 * kConsumers) {
            const int h = e / (D / 2), d = e % (D / 2) * 2;
            const float* ca = comb + h * (D + 2);
            const float* cb = ca + p.G * (D + 2);
            const float M = fmaxf(ca[D], cb[D]), base = M == -INFINITY ? 0.f : M;
            const float fa = exp2_ftz(ca[D] - base), fb = exp2_ftz(cb[D] - base);
            const long long at = (row0 + h) * p.n_split + x.s;
            *reinterpret_cast<float2*>(p.o_part + at * D + d) =
                make_float2(fa * ca[d] + fb * cb[d], fa * ca[d + 1] + fb * cb[d + 1]);
            if (d == 0) p.ml_part[at] = make_float2(M, fa * ca[D + 1] + fb * cb[D + 1]);
        }
        bar();  // comb is rewritten by the next unit
    }
    // this grid's end stands for the prefix pass's too
    if (p.wait_late) grid_dep_wait();
}

// ------------------------------------------------------------------------------------
// merge
// ------------------------------------------------------------------------------------
// Block (b, g) x y: the first row_blocks merge query heads,
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the own cache's splits and then the
//   prefix's ranges. A block merges one head, each group of its threads taking every GROUPS-th partial,
//   the groups' sums in order; or (WARPS) each of its warps does, with a partial's reference and sum on
//   a lane each, where heads are many and their partials few: no barriers and a quarter of the blocks
//   (8192 heads of about five partials behind the passes of a wide batch: 78.4 -> 68.0 us for the whole
//   call; 1024 heads: 35.4 -> 37.0, so that few heads keep the blocks). Later blocks take
//   kMergePositions positions of the slab each,
//   acc_out = acc_in + sum_r 2^(score_r - M_r) / l_r.
// A request without any token has zeros; scores of NaN, or of infinity throughout, have NaN as their
// softmax, in O and in the weights.
// What a block waits for are loads, so that the partials or scores it will need are asked for before
// the maxima they are taken against are known. Splits behind a request's tokens have no partials.
struct MergeParams {
    const float* own_o;
    const float2* own_ml;
    int n_own, split_len;
    const float* pre_o;  // prefix pass (launch_prefix); n_pre 0: none
    const float2* pre_ml;
    const int* n_ranges;
    const int* prefix_of;
    const int* prefix_lens;
    int n_pre, n_prefix, prefix_L;
    void* O;
    int o_fp32;
    const float* scores;
    int score_pitch;
    const float* acc_in;
    float* acc_out;
    const int* seq_lens;
    int Hq, Hkv, G, L;
    int row_blocks;  // of a (b, g): G, or with WARPS a quarter of that
};
constexpr int kMergeThreads = 128;
constexpr int kMergePositions = 512;  // 32 requests over 8K: 169.1 us a call; with 256 171.5, with 1024 170.3
constexpr int kMaxSplits = 1024;
constexpr int kWarpMergeRows = 16;  // heads an SM from which on warps merge, of at most 32 partials each
constexpr int kMaxRanges = 256;  // of a prefix; at most the SM count

template <int D, bool WARPS>
__global__ void __launch_bounds__(kMergeThreads) serve_merge_kernel(const MergeParams p) {
    constexpr int LANES = D / 4, GROUPS = kMergeThreads / LANES;
    constexpr int PER = kMergePositions / kMergeThreads;
    __shared__ float fs[WARPS ? 1 : kMaxSplits + kMaxRanges];
    __shared__ __align__(16) float red[WARPS ? 1 : GROUPS][D];
    __shared__ float2 wred[kMergeThreads / 32];
    __shared__ float2 rows[16];  // reference, 1 / sum
    const int b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = p.seq_lens ? min(max(p.seq_lens[b], 0), p.L) : p.L;
    const int j0 = (static_cast<int>(blockIdx.y) - p.row_blocks) * kMergePositions;
    if (j0 >= L) return;
    bool prefixed = false;
    if (p.n_pre > 0) {
        const int f = p.prefix_of ? p.prefix_of[b] : 0;
        prefixed = f >= 0 && f < p.n_prefix && (p.prefix_lens ? p.prefix_lens[f] : p.prefix_L) > 0;
    }
    const int n_own = (L + p.split_len - 1) / p.split_len;
    grid_dep_wait();
    // the limits: where a wait of the prefix pass ran out, its later units' counts were never written
    const int n = n_own + (prefixed ? min(max(p.n_ranges[b], 0), p.n_pre) : 0);
    const long long row0 = static_cast<long long>(b) * p.Hq + static_cast<long long>(g) * p.G;
    const auto ml = [&](long long row, int s) {
        return s < n_own ? p.own_ml[row * p.n_own + s] : p.pre_ml[row * p.n_pre + s - n_own];
    };
    if (WARPS && static_cast<int>(blockIdx.y) < p.row_blocks) {
        constexpr int PER_WARP = 32 / LANES;  // partials that a warp reads at once
        const int h = blockIdx.y * (kMergeThreads / 32) + warp;
        if (h >= p.G) return;
        const long long row = row0 + h;
        const int c = lane % LANES, grp = lane / LANES;
        const auto part = [&](int s) {
            const float* o = s < n_own ? p.own_o + (row * p.n_own + s) * D : p.pre_o + (row * p.n_pre + s - n_own) * D;
            return *reinterpret_cast<const float4*>(o + c * 4);
        };
        float4 first[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (grp + k * PER_WARP < n) first[k] = part(grp + k * PER_WARP);
        }
        const float2 v = lane < n ? ml(row, lane) : make_float2(-INFINITY, 0.f);
        float M = v.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float f = exp2f(v.x - (M == -INFINITY ? 0.f : M));
        float l = f * v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const auto add = [&](float w, const float4& x) {
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        };
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float w = __shfl_sync(0xffffffffu, f, (grp + k * PER_WARP) & 31);
            if (grp + k * PER_WARP < n) add(w, first[k]);
        }
#pragma unroll 4
        for (int s0 = 4 * PER_WARP; s0 < n; s0 += PER_WARP) {
            const float w = __shfl_sync(0xffffffffu, f, (s0 + grp) & 31);
            if (s0 + grp < n) add(w, part(s0 + grp));
        }
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
        if (grp == 0) {
            if (n > 0) acc.x /= l, acc.y /= l, acc.z /= l, acc.w /= l;  // no tokens at all: zeros
            if (p.o_fp32) {
                *reinterpret_cast<float4*>(static_cast<float*>(p.O) + row * D + c * 4) = acc;
            } else {
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + row * D + c * 4) =
                    make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
            }
        }
        return;
    }
    if (!WARPS && static_cast<int>(blockIdx.y) < p.row_blocks) {
        const long long row = row0 + blockIdx.y;
        const int c = tid % LANES, grp = tid / LANES;
        const auto part = [&](int s) {
            const float* o = s < n_own ? p.own_o + (row * p.n_own + s) * D : p.pre_o + (row * p.n_pre + s - n_own) * D;
            return *reinterpret_cast<const float4*>(o + c * 4);
        };
        float4 first[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (grp + k * GROUPS < n) first[k] = part(grp + k * GROUPS);
        }
        float M = -INFINITY;
        for (int s = tid; s < n; s += kMergeThreads) {
            const float2 v = ml(row, s);
            M = fmaxf(M, v.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) wred[warp].x = M;
        __syncthreads();
        M = fmaxf(fmaxf(wred[0].x, wred[1].x), fmaxf(wred[2].x, wred[3].x));
        const float base = M == -INFINITY ? 0.f : M;
        float l = 0.f;
        for (int s = tid; s < n; s += kMergeThreads) {
            const float2 v = ml(row, s);
            const float f = exp2f(v.x - base);
            fs[s] = f;
            l += f * v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) wred[warp].y = l;
        __syncthreads();
        l = (wred[0].y + wred[1].y) + (wred[2].y + wred[3].y);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const auto add = [&](int s, const float4& v) {
            const float f = fs[s];
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        };
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (grp + k * GROUPS < n) add(grp + k * GROUPS, first[k]);
        }
#pragma unroll 4
        for (int s = grp + 4 * GROUPS; s < n; s += GROUPS) add(s, part(s));
        *reinterpret_cast<float4*>(&red[grp][c * 4]) = acc;
        __syncthreads();
        if (tid < D) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) v += red[k][tid];
            v = n > 0 ? v / l : 0.f;  // no tokens at all: zeros
            if (p.o_fp32) static_cast<float*>(p.O)[row * D + tid] = v;
            else static_cast<__nv_bfloat16*>(p.O)[row * D + tid] = __float2bfloat16_rn(v);
        }
        return;
    }
    const long long slab = blockIdx.x;
    const int Gp = (p.G + 1) & ~1;
    const float* sc = p.scores + (slab * p.score_pitch + j0 + tid) * Gp;  // position j0 + tid + k * 128
    float2 early[PER][2];  // the first four heads' scores
    float w[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int j = j0 + tid + k * kMergeThreads;
        w[k] = p.acc_in && j < L ? p.acc_in[slab * p.L + j] : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (j < L && 2 * h < Gp) {
                early[k][h] = *reinterpret_cast<const float2*>(sc + static_cast<long long>(k) * kMergeThreads * Gp + 2 * h);
            }
        }
    }
    for (int r = warp; r < p.G; r += kMergeThreads / 32) {
        float M = -INFINITY, l = 0.f;
        for (int s = lane; s < n; s += 32) M = fmaxf(M, ml(row0 + r, s).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float base = M == -INFINITY ? 0.f : M;
        for (int s = lane; s < n; s += 32) {
            const float2 v = ml(row0 + r, s);
            l += exp2f(v.x - base) * v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) rows[r] = make_float2(base, 1.f / l);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int j = j0 + tid + k * kMergeThreads;
        if (j >= L) break;
        float add = 0.f;
        const auto count = [&](int h, const float2& v) {  // heads 2 h and 2 h + 1
            add += exp2f(v.x - rows[2 * h].x) * rows[2 * h].y;
            if (2 * h + 1 < p.G) add += exp2f(v.y - rows[2 * h + 1].x) * rows[2 * h + 1].y;
        };
        count(0, early[k][0]);
        if (Gp > 2) count(1, early[k][1]);
        for (int h = 2; 2 * h < Gp; ++h) {
            count(h, *reinterpret_cast<const float2*>(sc + static_cast<long long>(k) * kMergeThreads * Gp + 2 * h));
        }
        p.acc_out[slab * p.L + j] = w[k] + add;
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
constexpr int kServeHostCtas = 32, kServeHostWindow = 4;

// Splits of a cache: at most 512 tokens each, so that requests of different lengths fill the SMs
// alike and their tails are short; 256 where that leaves the CTAs fewer than about four units each
// (own caches of up to 1024 tokens behind a prefix, 32 requests: 34.5 -> 32.4 us for the whole call,
// and 128 tokens 34.5 again); and more where dak_attn's rule fills the SMs better.
constexpr int kServeSplitTokens = 512;
static int serve_default_split(const dak_placement* KV) {
    const int64_t units = static_cast<int64_t>(KV->B) * KV->H_kv * ((KV->L + kServeSplitTokens - 1) / kServeSplitTokens);
    const int tokens = units < 4ll * 3 * device_sm_count() ? kServeSplitTokens / 2 : kServeSplitTokens;
    return std::min(kMaxSplits, std::max(dak_attn_default_split(KV), (KV->L + tokens - 1) / tokens));
}

static int split_tokens(int L, int n_split) { return ((L + n_split - 1) / n_split + kChunk - 1) / kChunk * kChunk; }

template <int D>
static int serve_smem_bytes(int W, int G) {
    return W * 2 * kChunk * D * 2 + 2 * G * (D + 2) * 4;
}

template <int D, int NB, int PARTS>
static cudaError_t launch_serve(const ServeParams& p, int W, cudaStream_t s) {
    static SmemLimit limit;
    auto k = serve_kernel<D, NB, PARTS>;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), serve_smem_bytes<D>(kServeMaxStages, 8 * NB));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.n_host_ctas + p.n_hbm_ctas));
    cfg.blockDim = dim3(kServeThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(serve_smem_bytes<D>(W, p.G));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p);
}

// CTAs of the own pass that an SM holds, by ring depth and query heads (asked once).
template <int D>
static int serve_ctas_per_sm(int W, int G) {
    static std::atomic<int> known[kServeMaxStages + 1][17];
    int n = known[W][G].load(std::memory_order_relaxed);
    if (n) return n;
    const int smem = serve_smem_bytes<D>(W, G);
    const cudaError_t e =
        G <= 8 ? cudaFuncSetAttribute(serve_kernel<D, 1, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      serve_smem_bytes<D>(kServeMaxStages, 8))
               : cudaFuncSetAttribute(serve_kernel<D, 2, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      serve_smem_bytes<D>(kServeMaxStages, 16));
    if (e != cudaSuccess ||
        (G <= 8 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, serve_kernel<D, 1, 2>, kServeThreads, smem)
                : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, serve_kernel<D, 2, 2>, kServeThreads, smem)) !=
            cudaSuccess) {
        cudaGetLastError();
        return 1;
    }
    n = std::max(1, n);
    known[W][G].store(n, std::memory_order_relaxed);
    return n;
}

// Workspace: the own pass's partials (o, then references and sums), the prefix pass's (likewise, then
// the ranges' counts) and the scores, each rounded up to 256 bytes.
struct ServeLayout {
    int n_own, n_pre, score_pitch;
    size_t own_o, own_ml, pre_o, pre_ml, ranges, scores;
    size_t total() const { return own_o + own_ml + pre_o + pre_ml + ranges + scores; }
};

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

static ServeLayout serve_layout(const dak_placement* KV, const dak_placement* P, int H_q, int n_split, bool with_acc) {
    ServeLayout x{};
    const size_t rows = static_cast<size_t>(KV->B) * H_q, slabs = static_cast<size_t>(KV->B) * KV->H_kv;
    const int G = H_q / KV->H_kv;
    x.n_own = n_split > 0 ? n_split : serve_default_split(KV);
    x.n_pre = P ? prefix_max_ranges(P, static_cast<int64_t>(rows)) : 0;
    x.own_o = round256(rows * x.n_own * KV->D * sizeof(float));
    x.own_ml = round256(rows * x.n_own * sizeof(float2));
    x.pre_o = round256(rows * x.n_pre * KV->D * sizeof(float));
    x.pre_ml = round256(rows * x.n_pre * sizeof(float2));
    x.ranges = P ? round256(static_cast<size_t>(KV->B) * sizeof(int)) : 0;
    x.score_pitch = (KV->L + kChunk - 1) / kChunk * kChunk;
    x.scores = with_acc ? round256(slabs * x.score_pitch * ((G + 1) & ~1) * sizeof(float)) : 0;
    return x;
}

// Partial overlap of two arrays (the same array twice is none).
static bool partly_overlaps(const void* a, const void* b, size_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x != y && x < y + bytes && y < x + bytes;
}

static dak_status serve_attention(const void* Q, const dak_placement* KV, const int* seq_lens, const dak_placement* P,
                                  const int* prefix_lens, const int* prefix_of, int H_q, float scale, void* O,
                                  int o_fp32, const float* acc_in, float* acc_out, void* ws, size_t ws_bytes,
                                  const dak_tuning* t, cudaStream_t stream, const LinkHandoff* link) {
    if (!KV || KV->kind != 1 || !Q || !O || H_q <= 0 || H_q % KV->H_kv) return DAK_ERR_INVALID;
    const int G = H_q / KV->H_kv, D = KV->D;
    if (G > 16) return DAK_ERR_UNSUPPORTED;
    if (P && (P->kind != 1 || P->D != D || P->H_kv != KV->H_kv || P->device != KV->device)) return DAK_ERR_INVALID;
    if (P && P->B > kMaxPrefixes) return DAK_ERR_UNSUPPORTED;
    if (t && t->n_split > kMaxSplits) return DAK_ERR_INVALID;
    if (acc_out && G + (KV->L + kMergePositions - 1ll) / kMergePositions > 65535) return DAK_ERR_UNSUPPORTED;  // the merge's grid
    const int64_t slabs = static_cast<int64_t>(KV->B) * KV->H_kv;
    if (acc_out && acc_in && partly_overlaps(acc_in, acc_out, static_cast<size_t>(slabs) * KV->L * sizeof(float))) {
        return DAK_ERR_INVALID;
    }
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(ws, 16) || misaligned(acc_in, 4) || misaligned(acc_out, 4) ||
        misaligned(seq_lens, 4) || misaligned(prefix_lens, 4) || misaligned(prefix_of, 4)) {
        return DAK_ERR_ALIGN;
    }
    const ServeLayout x = serve_layout(KV, P, H_q, t ? t->n_split : 0, acc_out != nullptr);
    if (!ws || ws_bytes < x.total() || slabs * x.n_own > 0x7FFFFFFF) return DAK_ERR_INVALID;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DAK_ERR_CUDA;
    if (dev != KV->device) return DAK_ERR_INVALID;

    uint8_t* w = static_cast<uint8_t*>(ws);
    const auto take = [&](size_t bytes) {
        uint8_t* at = w;
        w += bytes;
        return at;
    };
    MergeParams m{};
    ServeParams p{};
    p.o_part = reinterpret_cast<float*>(take(x.own_o));
    p.ml_part = reinterpret_cast<float2*>(take(x.own_ml));
    float* pre_o = reinterpret_cast<float*>(take(x.pre_o));
    float* pre_ml = reinterpret_cast<float*>(take(x.pre_ml));
    int* n_ranges = reinterpret_cast<int*>(take(x.ranges));
    p.scores = acc_out ? reinterpret_cast<float*>(w) : nullptr;
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
    if (P) {
        const dak_status r =
            launch_prefix(Q, P, prefix_lens, prefix_of, KV->B, H_q, p.scale_log2, o_fp32, pre_o, pre_ml, n_ranges, stream);
        if (r != DAK_OK) return r;
        m.pre_o = pre_o;
        m.pre_ml = reinterpret_cast<const float2*>(pre_ml);
        m.n_ranges = n_ranges;
        m.prefix_of = prefix_of;
        m.prefix_lens = prefix_lens;
        m.n_pre = x.n_pre;
        m.n_prefix = P->B;
        m.prefix_L = P->L;
    }
    // ---- own pass
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.kv[0] = static_cast<const uint8_t*>(KV->host_dev);
    p.kv[1] = static_cast<const uint8_t*>(KV->hbm_ptr);
    p.seq_lens = seq_lens;
    p.score_pitch = x.score_pitch;
    p.B = KV->B;
    p.Hq = H_q;
    p.Hkv = KV->H_kv;
    p.G = G;
    p.L = KV->L;
    p.h_s = KV->h_s;
    p.n_split = x.n_own;
    p.split_len = split_tokens(KV->L, x.n_own);
    p.head_bytes = KV->head_bytes;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    p.host_units = static_cast<unsigned>(static_cast<int64_t>(KV->h_s) * x.n_own);
    p.hbm_units = static_cast<unsigned>((slabs - KV->h_s) * x.n_own);
    int W = (t && t->hbm_window > 0) ? std::min(t->hbm_window, kServeMaxStages) : serve_stages(D);
    if (!(t && t->hbm_window > 0) && slabs * x.n_own <= device_sm_count()) {
        W = std::max(W, std::min(p.split_len / kChunk, kServeMaxStages));  // a unit's chunks in flight at once
    }
    if (t && t->window > 0) W = std::max(W, std::min(t->window, kServeMaxStages));
    const int per_sm = D == 128 ? serve_ctas_per_sm<128>(W, G) : serve_ctas_per_sm<64>(W, G);
    dak_tuning tun = t ? *t : dak_tuning{};
    tun.no_wave_align = 1;  // units differ in length: no grid is a whole number of waves of them
    const Sched sc = schedule(static_cast<int>(p.host_units), static_cast<int>(p.hbm_units), device_sm_count() * per_sm, &tun,
                              kServeHostCtas, std::min(kServeHostWindow, W), W, W);
    p.n_host_ctas = sc.n_host_ctas;
    p.n_hbm_ctas = sc.n_hbm_ctas;
    p.host_window = sc.host_window;
    p.hbm_window = sc.hbm_window;
    p.wait_first = !P && !(t && t->pdl > 0);
    p.wait_newest = !P && t && t->pdl == 2;
    p.wait_late = P != nullptr;
    if (link && link->ctr) {
        p.link = link->ctr;
        p.link_after = link->after;
    }
    const int Wl = std::max(p.host_window, p.hbm_window);
    cudaError_t e;
    if (D == 128) {
        e = G <= 8 ? (o_fp32 ? launch_serve<128, 1, 3>(p, Wl, stream) : launch_serve<128, 1, 2>(p, Wl, stream))
                   : (o_fp32 ? launch_serve<128, 2, 3>(p, Wl, stream) : launch_serve<128, 2, 2>(p, Wl, stream));
    } else {
        e = G <= 8 ? (o_fp32 ? launch_serve<64, 1, 3>(p, Wl, stream) : launch_serve<64, 1, 2>(p, Wl, stream))
                   : (o_fp32 ? launch_serve<64, 2, 3>(p, Wl, stream) : launch_serve<64, 2, 2>(p, Wl, stream));
    }
    if (e != cudaSuccess) return cuda_status(e);
    if (link && link->signals && p.link) *link->signals = p.n_host_ctas;
    // ---- merge
    m.own_o = p.o_part;
    m.own_ml = p.ml_part;
    m.n_own = x.n_own;
    m.split_len = p.split_len;
    m.O = O;
    m.o_fp32 = o_fp32 ? 1 : 0;
    m.scores = p.scores;
    m.score_pitch = x.score_pitch;
    m.acc_in = acc_in;
    m.acc_out = acc_out;
    m.seq_lens = seq_lens;
    m.Hq = H_q;
    m.Hkv = KV->H_kv;
    m.G = G;
    m.L = KV->L;
    const bool warps = x.n_own + x.n_pre <= 32 && slabs * G >= kWarpMergeRows * device_sm_count();
    m.row_blocks = warps ? (G + kMergeThreads / 32 - 1) / (kMergeThreads / 32) : G;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(slabs),
                       static_cast<unsigned>(m.row_blocks + (acc_out ? (KV->L + kMergePositions - 1) / kMergePositions : 0)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (D == 128) {
        e = warps ? cudaLaunchKernelEx(&cfg, serve_merge_kernel<128, true>, m) : cudaLaunchKernelEx(&cfg, serve_merge_kernel<128, false>, m);
    } else {
        e = warps ? cudaLaunchKernelEx(&cfg, serve_merge_kernel<64, true>, m) : cudaLaunchKernelEx(&cfg, serve_merge_kernel<64, false>, m);
    }
    return cuda_status(e);
}

static bool serve_shape(const dak_placement* KV, int H_q, int n_split) {
    return KV && KV->kind == 1 && H_q > 0 && H_q % KV->H_kv == 0 && n_split <= kMaxSplits;
}

}  // namespace dak

extern "C" size_t dak_attn_acc_workspace_bytes(const dak_placement* KV, int H_q, int n_split) {
    return dak::serve_shape(KV, H_q, n_split) ? dak::serve_layout(KV, nullptr, H_q, n_split, true).total() : 0;
}

extern "C" dak_status dak_attn_acc(const void* Q, const dak_placement* KV, const int* seq_lens, int H_q, float scale,
                                   void* O, int o_fp32, const float* acc_in, float* acc_out, void* workspace,
                                   size_t ws_bytes, const dak_tuning* tuning, void* stream) {
    if (!acc_out) return DAK_ERR_INVALID;
    dak::LinkHandoff lk;
    int signals = 0;
    const bool joined = dak::link_join(tuning, &lk);
    if (joined) lk.signals = &signals;
    const dak_status r =
        dak::serve_attention(Q, KV, seq_lens, nullptr, nullptr, nullptr, H_q, scale, O, o_fp32, acc_in, acc_out,
                             workspace, ws_bytes, tuning, static_cast<cudaStream_t>(stream), joined ? &lk : nullptr);
    if (joined && r == DAK_OK) dak::link_commit(tuning, signals);
    return r;
}

extern "C" size_t dak_attn_prefix_workspace_bytes(const dak_placement* KV, const dak_placement* P, int H_q,
                                                  int n_split, int with_acc) {
    if (!P || P->kind != 1 || !dak::serve_shape(KV, H_q, n_split)) return 0;
    return dak::serve_layout(KV, P, H_q, n_split, with_acc != 0).total();
}

extern "C" dak_status dak_attn_prefix(const void* Q, const dak_placement* KV, const int* seq_lens,
                                      const dak_placement* P, const int* prefix_lens, const int* prefix_of, int H_q,
                                      float scale, void* O, int o_fp32, const float* acc_in, float* acc_out,
                                      void* workspace, size_t ws_bytes, const dak_tuning* tuning, void* stream) {
    if (!P) return DAK_ERR_INVALID;
    return dak::serve_attention(Q, KV, seq_lens, P, prefix_lens, prefix_of, H_q, scale, O, o_fp32, acc_in, acc_out,
                                workspace, ws_bytes, tuning, static_cast<cudaStream_t>(stream), nullptr);
}
