// The prefix pass of dak_attn_prefix: attention of all requests that share a prefix over the
// prefix's rows, each (prefix, kv head) slab streamed once for up to 256 query rows (a row = one
// request's query head). Partial results go to the merge of dak_attn.cu.
//
// The contraction is GEMM-shaped (rows x keys x D twice), so it runs on the tcgen05 tensor cores
// as the usual two products with an online softmax between them:
//   S  = Q (128 rows x D, shared memory) . K^T (D x 128 keys, shared memory) -> TMEM, fp32
//   P  = 2^(S * scale log2 e - m), written back into S's TMEM columns as bf16
//   O += P (TMEM) . V (128 keys x D, shared memory) -> TMEM, fp32
// A CTA has two streams, each a warpgroup of 128 threads (thread = row) with its own S, P and O
// in TMEM, so that one stream's softmax runs under the other's products. With more than 128
// rows the streams hold two row tiles and both go through every key; with fewer they hold the
// same rows and take the 128-key steps in turn, and their results are merged in the CTA.
//
// The cache stores piece c of token t at c ^ (t & 7), which is the tensor cores' 128-byte swizzle
// once a row's two 128-byte halves lie apart; a 5-D tensor map (64 elements, 64 tokens, K or V,
// chunk, half) brings a step's K or V so in one copy. K is then a K-major operand; V, whose rows
// are keys, an MN-major one.
//
// Which CTA works on what is planned on the device from the prefixes' lengths and the requests'
// map, so that a captured call follows them: units (prefix, kv head, 256-row tile, key range),
// every prefix cut into ranges of at most T chunks, T the smallest for which the units still fit
// the CTAs at once.
#include <algorithm>

#include <cudaTypedefs.h>

#include "dak_device.cuh"

namespace dak {

constexpr int kPrefixThreads = 10 * 32;  // two softmax warpgroups, copies, MMAs
constexpr int kPrefixMinChunks = 2;      // chunks of 64 keys in a range, at least

struct PrefixMaps {
    CUtensorMap step[2];  // [host, HBM]: a whole step (KEYS keys)
    CUtensorMap tail[2];  // one chunk of 64 keys
};

struct PrefixParams {
    const __nv_bfloat16* Q;
    const int* lens;   // [n_prefix] or null
    const int* of;     // [B] or null
    float* o_part;     // [B * Hq][n_pre][D]
    float2* ml_part;   // [B * Hq][n_pre]: m (log2 domain), l
    int* n_ranges;     // [n_prefix]: key ranges of a prefix that has members and rows
    int B, Hq, Hkv, G, L, n_prefix, n_pre, h_s, slab_chunks;
    float scale_log2;
    DevStatus* st;
};

enum : uint32_t { X_PROD_EMPTY = 0x51, X_MMA_FULL, X_MMA_P, X_MMA_PV, X_SM_S, X_SM_V, X_SM_O, X_DRAIN };

// What a CTA works on.
struct PrefixUnit {
    int f, g, s;       // prefix, kv head, key range
    int c0, c1;        // its chunks
    int len;           // rows of the prefix
    int members;       // requests of this tile
    int two;           // the members fill more than one 128-row tile
    int units;         // units of the whole launch
};

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int kv, int chunk, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4, "
        "%2}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(kv), "r"(chunk), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int ID, int THREADS>
__device__ __forceinline__ void prefix_bar() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

__device__ __forceinline__ int prefix_chunks(const PrefixParams& p, int f) {
    const int n = p.lens ? min(max(p.lens[f], 0), p.L) : p.L;
    return (n + 63) >> 6;
}

// Unit u of the launch into *unit (units == 0: none at all) and its members' requests. All threads
// call it; scratch: n_prefix int2 of shared memory, free until the next barrier.
__device__ __forceinline__ void plan_unit(const PrefixParams& p, int u, int2* scratch, PrefixUnit* unit, int* member) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int mpt = 128 / p.G;  // members of a 128-row tile
    for (int f = tid; f < p.n_prefix; f += kPrefixThreads) scratch[f] = make_int2(p.of ? 0 : f == 0 ? p.B : 0, 0);
    __syncthreads();
    if (p.of) {
        for (int b = tid; b < p.B; b += kPrefixThreads) {
            const int e = p.of[b];
            if (e >= 0 && e < p.n_prefix) atomicAdd(&scratch[e].x, 1);
            if (e >= p.n_prefix && blockIdx.x == 0) report(p.st, DAK_ERR_BOUNDS, (0x9F1Full << 32) | static_cast<unsigned>(b));
        }
        __syncthreads();
    }
    if (tid < 32) {
        const unsigned all = 0xffffffffu;
        int cmax = 1;
        for (int f = lane; f < p.n_prefix; f += 32) {
            const int c = prefix_chunks(p, f);
            const int tiles = c > 0 ? (scratch[f].x + 2 * mpt - 1) / (2 * mpt) : 0;
            scratch[f].y = tiles;
            if (tiles) cmax = max(cmax, c);
        }
        __syncwarp();
        cmax = __reduce_max_sync(all, cmax);
        const auto ranges = [&](int c, int T) { return min((c + T - 1) / T, p.n_pre); };
        const auto total = [&](int T) {
            int n = 0;
            for (int f = lane; f < p.n_prefix; f += 32) {
                if (scratch[f].y) n += scratch[f].y * ranges(prefix_chunks(p, f), T);
            }
            return __reduce_add_sync(all, n) * p.Hkv;
        };
        int lo = min(kPrefixMinChunks, cmax), hi = cmax;
        if (total(hi) < static_cast<int>(gridDim.x)) {
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (total(mid) <= static_cast<int>(gridDim.x)) hi = mid;
                else lo = mid + 1;
            }
        }
        const int T = hi;
        int base = 0, f = -1, start = 0;
        for (int f0 = 0; f0 < p.n_prefix; f0 += 32) {
            const int ff = f0 + lane;
            int n = 0;
            if (ff < p.n_prefix && scratch[ff].y) n = scratch[ff].y * ranges(prefix_chunks(p, ff), T) * p.Hkv;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(all, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(all, u < base + incl);
            if (f < 0 && hit) {
                const int l = __ffs(hit) - 1;
                f = f0 + l;
                start = base + __shfl_sync(all, incl - n, l);
            }
            base += __shfl_sync(all, incl, 31);
        }
        if (f < 0) {
            if (lane == 0) unit->units = 0;
        } else {
            const int c = prefix_chunks(p, f), n = ranges(c, T), tiles = scratch[f].y, cnt = scratch[f].x;
            const int rem = u - start;
            const int g = rem / (tiles * n), t = rem / n % tiles, s = rem % n;
            const int r0 = t * 2 * mpt, here = min(2 * mpt, cnt - r0);
            if (lane == 0) {
                unit->f = f;
                unit->g = g;
                unit->s = s;
                unit->c0 = static_cast<int>(static_cast<long long>(c) * s / n);
                unit->c1 = static_cast<int>(static_cast<long long>(c) * (s + 1) / n);
                unit->len = p.lens ? min(max(p.lens[f], 0), p.L) : p.L;
                unit->members = here;
                unit->two = here > mpt;
                unit->units = base;
                if (g == 0 && t == 0 && s == 0) p.n_ranges[f] = n;
            }
            if (!p.of) {
                for (int i = lane; i < here; i += 32) member[i] = r0 + i;
            } else {
                int seen = 0;
                for (int b0 = 0; b0 < p.B && seen < r0 + here; b0 += 32) {
                    const bool mine = b0 + lane < p.B && p.of[b0 + lane] == f;
                    const unsigned m = __ballot_sync(all, mine);
                    const int rank = seen + __popc(m & ((1u << lane) - 1)) - r0;
                    if (mine && rank >= 0 && rank < here) member[rank] = b0 + lane;
                    seen += __popc(m);
                }
            }
        }
    }
    __syncthreads();
}

// KEYS: keys of a step, 128 (bf16 output, P in two bf16 parts) or 64 (fp32 output, three).
template <int D, int KEYS>
struct PrefixCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = 128 * D * 2;  // one Q tile
    static constexpr int kStage = KEYS * D * 2;     // K or V of a step
    static constexpr int kStages = std::min(12, (224 * 1024 - 2 * kTileBytes) / kStage);
    static constexpr int kSmem = 2 * kTileBytes + kStages * kStage + 1024;
};

template <int D, int KEYS>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ PrefixMaps maps) {
    using C = PrefixCfg<D, KEYS>;
    constexpr int NS = C::kStages;
    constexpr int SMAX = KEYS / 64;  // chunks of a whole step
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    uint8_t* ring = smem + 2 * C::kTileBytes;
    __shared__ uint64_t full[NS], empty[NS], s_full[2], p_ready[2], pv_done[2];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_flag;
    __shared__ PrefixUnit unit;
    __shared__ int member[256];
    // (m, l) of a row in each stream, where the streams share one Q tile: in the other's memory
    float2(*ex)[128] = reinterpret_cast<float2(*)[128]>(smem + C::kTileBytes);
    volatile int* abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 4);
            mbar_init(&pv_done[s], 1);
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
    // TMEM columns: S (and P over it) of the two streams at 0 and 128, O at 256 and 256 + D
    long long it0 = 0;        // K and V stages used by earlier units
    int used[2] = {0, 0};     // steps each stream did in earlier units
    for (int u = blockIdx.x;; u += gridDim.x) {
        plan_unit(p, u, reinterpret_cast<int2*>(smem), &unit, member);
        const PrefixUnit x = unit;
        if (x.units == 0) break;
        const int steps = (x.c1 - x.c0 + SMAX - 1) / SMAX;
        const int items = x.two ? 2 * steps : steps;  // item i: stream i & 1, step i / 2 or i
        constexpr int parts = KEYS == 64 ? 3 : 2;
        const long long slab = static_cast<long long>(x.f) * p.Hkv + x.g;
        const int tier = slab < p.h_s ? 0 : 1;
        const int step_of_shift = x.two ? 1 : 0;
        __syncthreads();  // the scratch that the plan used is Q's memory

        if (warp == 8) {
            // ------------------------------------------------------------ copies
            if (lane == 0) {
                const int chunk0 = static_cast<int>((tier ? slab - p.h_s : slab) * p.slab_chunks);
                long long it = it0;
                for (int j = 0; j < steps; ++j) {
                    const int c = x.c0 + j * SMAX, nk = min(SMAX, x.c1 - c);
                    const CUtensorMap* map = nk == SMAX ? &maps.step[tier] : &maps.tail[tier];
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int s = static_cast<int>(it % NS);
                        if (it >= NS && !mbar_wait(&empty[s], static_cast<uint32_t>((it / NS - 1) & 1), abort, p.st,
                                                   DAK_ERR_TIMEOUT, X_PROD_EMPTY)) {
                            goto copies_done;
                        }
                        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nk * 64 * D * 2));
                        tma_load_5d(ring + static_cast<size_t>(s) * C::kStage, map, kv, chunk0 + c, &full[s]);
                    }
                }
            copies_done:
                if (*abort) {  // copies in flight land before the CTA may leave
                    volatile int dummy = 0;
                    for (int s = 0; s < NS && s < it; ++s) {
                        const long long last = ((it - 1 - s) / NS) * NS + s;
                        mbar_wait(&full[s], static_cast<uint32_t>((last / NS) & 1), &dummy, p.st, DAK_ERR_TIMEOUT, X_DRAIN);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ------------------------------------------------------------ products
            prefix_bar<2, 288>();  // Q lies in shared memory
            tc_fence_after();
            if (lane == 0) {
                const uint32_t q_addr = smem_u32(smem), ring_addr = smem_u32(ring);
                const auto stage_at = [&](int j, int kv) { return static_cast<int>((it0 + 2 * j + kv) % NS); };
                const auto wait_full = [&](int j, int kv) {
                    const long long it = it0 + 2 * j + kv;
                    return mbar_wait(&full[it % NS], static_cast<uint32_t>((it / NS) & 1), abort, p.st, DAK_ERR_TIMEOUT,
                                     X_MMA_FULL);
                };
                const auto qk = [&](int i) {
                    const int st = i & 1, j = i >> step_of_shift;
                    const int nk = min(SMAX, x.c1 - x.c0 - j * SMAX);
                    if (!wait_full(j, 0)) return false;
                    // S's columns still hold the P that the stream's last product reads
                    if (i >= 2 && !mbar_wait(&pv_done[st], static_cast<uint32_t>((used[st] + (i >> 1) - 1) & 1), abort,
                                             p.st, DAK_ERR_TIMEOUT, X_MMA_PV)) {
                        return false;
                    }
                    tc_fence_after();
                    const uint32_t a = q_addr + (x.two ? st * C::kTileBytes : 0);
                    const uint32_t b = ring_addr + stage_at(j, 0) * C::kStage;
                    const uint32_t idesc = idesc_bf16_f32(128, static_cast<uint32_t>(64 * nk));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t h = k >> 2, in = (k & 3) * 32;
                        umma_bf16(tmem + st * 128, smem_desc(a + h * 16384 + in, 16, 1024, 2),
                                  smem_desc(b + h * (8192 * nk) + in, 16, 1024, 2), idesc, k > 0);
                    }
                    umma_commit(&s_full[st]);
                    if (!x.two || st == 1) umma_commit(&empty[stage_at(j, 0)]);
                    return true;
                };
                const auto pv = [&](int i) {
                    const int st = i & 1, j = i >> step_of_shift;
                    const int nk = min(SMAX, x.c1 - x.c0 - j * SMAX);
                    if (!wait_full(j, 1) || !mbar_wait(&p_ready[st], static_cast<uint32_t>((used[st] + (i >> 1)) & 1),
                                                       abort, p.st, DAK_ERR_TIMEOUT, X_MMA_P)) {
                        return false;
                    }
                    tc_fence_after();
                    const uint32_t v = ring_addr + stage_at(j, 1) * C::kStage;
                    // V: N = D along a row's halves (8192 nk bytes apart), K = the keys, in groups of
                    // eight 1024 bytes apart; bit 16: B is MN-major
                    const uint32_t idesc = idesc_bf16_f32(128, D) | (1u << 16);
                    for (int q = 0; q < parts; ++q) {
                        for (int k = 0; k < 4 * nk; ++k) {
                            umma_bf16_ts(tmem + 256 + st * D, tmem + st * 128 + q * (KEYS / 2) + k * 8,
                                         smem_desc(v + k * 2048, 8192 * nk, 1024, 2), idesc, i >= 2 || q > 0 || k > 0);
                        }
                    }
                    umma_commit(&pv_done[st]);
                    if (!x.two || st == 1) umma_commit(&empty[stage_at(j, 1)]);
                    return true;
                };
                bool ok = qk(0) && (items < 2 || qk(1));
                for (int i = 0; i < items && ok; ++i) ok = pv(i) && (i + 2 >= items || qk(i + 2));
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ softmax, one row a thread
            const int st = warp >> 2, r = (warp & 3) * 32 + lane;
            const int mpt = 128 / p.G;
            {   // Q rows into the 128-byte swizzled K-major layout, rows without a member zero
                const int n_rows = x.two ? 256 : 128;
                for (int e = threadIdx.x; e < n_rows * (D / 8); e += 256) {
                    const int row = e / (D / 8), c = e % (D / 8);
                    const int tile = row >> 7, rr = row & 127, m = rr / p.G;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (m < mpt && tile * mpt + m < x.members) {
                        const long long qrow = static_cast<long long>(member[tile * mpt + m]) * p.Hq + x.g * p.G + rr - m * p.G;
                        v = *reinterpret_cast<const uint4*>(p.Q + qrow * D + c * 8);
                    }
                    *reinterpret_cast<uint4*>(smem + tile * C::kTileBytes + (c >> 3) * 16384 + rr * 128 +
                                              (((c & 7) ^ (rr & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                prefix_bar<2, 288>();
            }
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t s_addr = tmem + lanes + st * 128, o_addr = tmem + lanes + 256 + st * D;
            float m_ref = -INFINITY, l = 0.f;
            bool ok = true;
            int mine = 0;
            for (int i = st; i < items; i += 2, ++mine) {
                const int j = i >> step_of_shift;
                const int k0 = (x.c0 + j * SMAX) * 64;  // first key of the step
                const int nk = min(SMAX, x.c1 - x.c0 - j * SMAX), valid = min(64 * nk, x.len - k0);
                ok = mbar_wait(&s_full[st], static_cast<uint32_t>((used[st] + mine) & 1), abort, p.st, DAK_ERR_TIMEOUT,
                               X_SM_S);
                if (!__all_sync(0xffffffffu, ok)) {  // a wait ran out: the whole warp stops
                    ok = false;
                    break;
                }
                tc_fence_after();
                float s[KEYS];
#pragma unroll
                for (int q = 0; q < KEYS / 32; ++q) {
                    if (q < 2 * nk) tmem_ld32(s_addr + q * 32, s + q * 32);
                }
                tmem_wait_ld();
                if (valid < KEYS) {
                    if (!x.two || st == 0) {
                        // rows of V past the prefix may hold anything, also infinities and NaN,
                        // which a probability of zero would not cancel
                        const long long vit = it0 + 2 * j + 1;
                        mbar_wait(&full[vit % NS], static_cast<uint32_t>((vit / NS) & 1), abort, p.st, DAK_ERR_TIMEOUT,
                                  X_SM_V);
                        uint8_t* v = ring + static_cast<size_t>(vit % NS) * C::kStage;
                        for (int e = (warp & 3) * 32 + lane; e < (64 * nk - valid) * (D / 8); e += 128) {
                            const int row = valid + e / (D / 8), c = e % (D / 8);
                            *reinterpret_cast<uint4*>(v + (c >> 3) * (8192 * nk) + row * 128 + ((c & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
#pragma unroll
                    for (int k = 0; k < KEYS; ++k) {
                        if (k >= valid) s[k] = -INFINITY;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < KEYS; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k]);
                const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                // the reference only moves when a row's maximum outgrows it by 2^8: until then the
                // sums just grow, which fp32 holds
                if (mine == 0) {
                    m_ref = m_new;
                } else if (__any_sync(0xffffffffu, m_new > m_ref + 8.f)) {
                    const float m2 = fmaxf(m_ref, m_new);
                    const float f = m2 == -INFINITY ? 1.f : exp2_ftz(m_ref - m2);
                    m_ref = m2;
                    l *= f;
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        float o[32];
                        tmem_ld32(o_addr + q * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f;
                        tmem_st32(o_addr + q * 32, o);
                    }
                }
                const float base = m_ref == -INFINITY ? 0.f : m_ref;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < KEYS / 32; ++q) {
                    if (q < 2 * nk) {
                        uint32_t hi[16], lo[16], th[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float a = exp2_ftz(fmaf(s[q * 32 + 2 * k], p.scale_log2, -base));
                            const float b = exp2_ftz(fmaf(s[q * 32 + 2 * k + 1], p.scale_log2, -base));
                            sum[(2 * k) & 3] += a;
                            sum[(2 * k + 1) & 3] += b;
                            hi[k] = pack_bf16(a, b);
                            const float ra = a - bf_lo(hi[k]), rb = b - bf_hi(hi[k]);
                            lo[k] = pack_bf16(ra, rb);
                            if (KEYS == 64) th[k] = pack_bf16(ra - bf_lo(lo[k]), rb - bf_hi(lo[k]));
                        }
                        tmem_st16(s_addr + q * 16, hi);
                        if (parts > 1) tmem_st16(s_addr + KEYS / 2 + q * 16, lo);
                        if (KEYS == 64) tmem_st16(s_addr + KEYS + q * 16, th);
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[st]);
            }
            if (ok && mine > 0) {
                mbar_wait(&pv_done[st], static_cast<uint32_t>((used[st] + mine - 1) & 1), abort, p.st, DAK_ERR_TIMEOUT,
                          X_SM_O);
            }
            __syncwarp();
            // ---- results: row r of this stream's tile, or of the tile that the streams share
            const int tile = x.two ? st : 0, m = r / p.G;
            const bool valid_row = m < mpt && tile * mpt + m < x.members;
            long long at = 0;
            if (valid_row) {
                at = (static_cast<long long>(member[tile * mpt + m]) * p.Hq + x.g * p.G + r - m * p.G) * p.n_pre + x.s;
            }
            if (x.two) {
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    float o[32];
                    tmem_ld32(o_addr + q * 32, o);
                    tmem_wait_ld();
                    if (valid_row) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            *reinterpret_cast<float4*>(p.o_part + at * D + q * 32 + k) =
                                make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                    }
                }
                if (valid_row) p.ml_part[at] = make_float2(m_ref, l);
            } else {
                ex[st][r] = make_float2(m_ref, l);
                tc_fence_before();
                prefix_bar<3, 256>();
                tc_fence_after();
                const float2 e0 = ex[0][r], e1 = ex[1][r];
                const float M = fmaxf(e0.x, e1.x), base = M == -INFINITY ? 0.f : M;
                const float f0 = exp2_ftz(e0.x - base), f1 = exp2_ftz(e1.x - base);
                const bool both = items > 1;  // the second stream had a step
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    const int col = st * (D / 2) + q * 32;
                    float a[32], b[32];
                    tmem_ld32(tmem + lanes + 256 + col, a);
                    tmem_ld32(tmem + lanes + 256 + D + col, b);
                    tmem_wait_ld();
                    if (valid_row) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) a[k] = both ? a[k] * f0 + b[k] * f1 : a[k] * f0;
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            *reinterpret_cast<float4*>(p.o_part + at * D + col + k) =
                                make_float4(a[k], a[k + 1], a[k + 2], a[k + 3]);
                        }
                    }
                }
                if (valid_row && st == 0) p.ml_part[at] = make_float2(M, e0.y * f0 + (both ? e1.y * f1 : 0.f));
            }
        }
        it0 += 2 * steps;
        used[0] += (items + 1) / 2;
        used[1] += items / 2;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (abort_flag || u + static_cast<int>(gridDim.x) >= x.units) break;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The prefix's chunks of one tier as the kernel copies them, nk chunks at a time.
static bool make_prefix_map(CUtensorMap* map, const void* base, int64_t chunks, int D, int nk) {
    const auto enc = encode_fn();
    if (!enc || fault_due(DAK_FAULT_TENSOR_MAP)) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[5] = {64, 64, 2, static_cast<cuuint64_t>(chunks), static_cast<cuuint64_t>(D / 64)};
    const cuuint64_t strides[4] = {row, 64 * row, 128 * row, 128};
    const cuuint32_t box[5] = {64, 64, 1, static_cast<cuuint32_t>(nk), static_cast<cuuint32_t>(D / 64)};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int prefix_max_ranges(const dak_placement* P) {
    const int chunks = (P->L + 63) / 64;
    return std::max(1, std::min(device_sm_count() / P->H_kv, (chunks + kPrefixMinChunks - 1) / kPrefixMinChunks));
}

template <int D, int KEYS>
static cudaError_t launch_prefix_d(const PrefixParams& p, const PrefixMaps& maps, int grid, cudaStream_t s) {
    auto k = prefix_kernel<D, KEYS>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PrefixCfg<D, KEYS>::kSmem);
    if (e != cudaSuccess) return e;
    k<<<grid, kPrefixThreads, PrefixCfg<D, KEYS>::kSmem, s>>>(p, maps);
    return cudaGetLastError();
}

dak_status launch_prefix(const void* Q, const dak_placement* P, const int* lens, const int* of, int B, int H_q,
                         float scale_log2, int o_fp32, float* o_part, float* ml_part, int* n_ranges, cudaStream_t s) {
    const int D = P->D, keys = o_fp32 ? 64 : 128;
    PrefixParams p{};
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.lens = lens;
    p.of = of;
    p.o_part = o_part;
    p.ml_part = reinterpret_cast<float2*>(ml_part);
    p.n_ranges = n_ranges;
    p.B = B;
    p.Hq = H_q;
    p.Hkv = P->H_kv;
    p.G = H_q / P->H_kv;
    p.L = P->L;
    p.n_prefix = P->B;
    p.n_pre = prefix_max_ranges(P);
    p.h_s = P->h_s;
    p.slab_chunks = (P->L + 63) / 64;
    p.scale_log2 = scale_log2;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    const int64_t slabs = static_cast<int64_t>(P->B) * P->H_kv;
    PrefixMaps maps{};
    for (int tier = 0; tier < 2; ++tier) {
        const int64_t n = tier ? slabs - P->h_s : P->h_s;
        const void* base = tier ? P->hbm_ptr : P->host_dev;
        if (n == 0) continue;
        if (!make_prefix_map(&maps.step[tier], base, n * p.slab_chunks, D, keys / 64) ||
            !make_prefix_map(&maps.tail[tier], base, n * p.slab_chunks, D, 1)) {
            return DAK_ERR_CUDA;
        }
    }
    // no more CTAs than units can come out: every tile with members in every range
    const int per_tile = 2 * (128 / p.G);
    const int64_t tiles = std::min<int64_t>(B, P->B + static_cast<int64_t>(B) / per_tile);
    const int grid = static_cast<int>(std::min<int64_t>(device_sm_count(), tiles * p.Hkv * p.n_pre));
    cudaError_t e;
    if (D == 128) {
        e = o_fp32 ? launch_prefix_d<128, 64>(p, maps, grid, s) : launch_prefix_d<128, 128>(p, maps, grid, s);
    } else {
        e = o_fp32 ? launch_prefix_d<64, 64>(p, maps, grid, s) : launch_prefix_d<64, 128>(p, maps, grid, s);
    }
    return cuda_status(e);
}

}  // namespace dak
