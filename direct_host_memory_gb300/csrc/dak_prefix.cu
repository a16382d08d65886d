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

constexpr int kPrefixThreads = 11 * 32;  // two softmax warpgroups, copies, each stream's products
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
    int* n_ranges;     // [B]: key ranges that a request's rows have partials of (not written without any)
    int B, Hq, Hkv, G, L, n_prefix, n_pre, h_s, slab_chunks;
    int mpt;  // members of a 128-row tile: 128 / G
    float scale_log2;
    DevStatus* st;
};

enum : uint32_t { X_PROD_EMPTY = 0x51, X_PROD_FULL, X_MMA_FULL, X_MMA_P, X_MMA_PV, X_MMA_GO, X_SM_S, X_SM_V, X_SM_O, X_DRAIN };

// What a CTA works on.
struct PrefixUnit {
    int f, g, s;       // prefix, kv head, key range
    int c0, c1;        // its chunks
    int len;           // rows of the prefix
    int members;       // requests of this tile
    int two;           // the members fill more than one 128-row tile
    int units;         // units of the whole launch
};

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int kv, int chunk, uint64_t* bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%2, %3, %4, %2}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(kv), "r"(chunk), "r"(smem_u32(bar)), "l"(policy)
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

// 16 columns of this thread's lane; the values are there after tmem_wait(v).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
// Waits for every load of this thread; the registers pass through so that no use of them moves up.
__device__ __forceinline__ void tmem_wait(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 bytes global -> shared, `bytes` (16 or 0) of them from src and zeros for the rest.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int ID, int THREADS>
__device__ __forceinline__ void prefix_bar() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

__device__ __forceinline__ void report_prefix(const PrefixParams& p, int b) {
    report(p.st, DAK_ERR_BOUNDS, (0x9F1Full << 32) | static_cast<unsigned>(b));
}

// Unit u of the launch into *unit (units == 0: none at all) and its members' requests, by one warp.
// Every CTA waits for this before its first copy, so it is built for latency: the map and the
// lengths are loaded side by side (the first 128 requests' map stays in registers), counting and
// searching run in shared memory, scratch[f] (n_prefix int4, free until the next barrier): requests,
// halves (see below), chunks, rows; divisions are 32-bit.
__device__ __forceinline__ void plan_unit(const PrefixParams& p, int u, int4* scratch, PrefixUnit* unit, int* member) {
    constexpr unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int per_tile = 2 * p.mpt;  // members of a 256-row tile
    const int ctas = static_cast<int>(gridDim.x);
    int map[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) map[k] = p.of && k * 32 + lane < p.B ? p.of[k * 32 + lane] : -1;
    const auto map_of = [&](int b0) {  // the map of requests b0 + lane, in steps of 32 from 0
        return b0 == 0 ? map[0] : b0 == 32 ? map[1] : b0 == 64 ? map[2] : b0 == 96 ? map[3]
               : b0 + lane < p.B ? p.of[b0 + lane] : -1;
    };
    // Requests' rows make full tiles of two 128-row halves and one more of one or two. A half over a
    // chunk is a unit of work, so that a tile of two is cut into twice the ranges; `halves` holds
    // both kinds: tiles of two in its upper bits, one of one in bit 0.
    const auto halves_of = [&](int cnt) {
        const int full = cnt / per_tile, rest = cnt - full * per_tile;
        return rest > p.mpt ? 2 * full + 2 : 2 * full + (rest > 0);
    };
    const auto ranges = [&](int work, int c, int T) {
        return max(1, min(min((work + T - 1) / T, p.n_pre), c / kPrefixMinChunks));
    };
    const auto units_of = [&](int halves, int c, int T) {  // per kv head
        return halves == 0 || c == 0 ? 0 : (halves >> 1) * ranges(2 * c, c, T) + (halves & 1) * ranges(c, c, T);
    };
    int f = -1, start = 0, base = 0, T = 1;
    int4 e;
    if (p.n_prefix == 1) {
        const int len = p.lens ? min(max(p.lens[0], 0), p.L) : p.L;
        int cnt = p.B;
        if (p.of) {
            cnt = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int v = map_of(b0);
                if (v > 0 && blockIdx.x == 0) report_prefix(p, b0 + lane);
                cnt += __popc(__ballot_sync(all, v == 0));
            }
        }
        e = make_int4(cnt, halves_of(cnt), (len + 63) >> 6, len);
        const int tiles = ((e.y + 1) >> 1) * p.Hkv;
        if (tiles > 0 && e.z > 0) {
            T = 2 * e.z;
            if (tiles < ctas) {
                if (e.y == 1 || (e.y & 1) == 0) {  // tiles of one kind: each the same share of the CTAs
                    const int each = ctas / tiles, work = e.y == 1 ? e.z : 2 * e.z;
                    T = (work + each - 1) / each;
                } else {
                    int lo = 1;
                    while (lo < T) {
                        const int mid = (lo + T) >> 1;
                        if (units_of(e.y, e.z, mid) * p.Hkv <= ctas) T = mid;
                        else lo = mid + 1;
                    }
                }
            }
            base = units_of(e.y, e.z, T) * p.Hkv;
            if (u < base) f = 0;
        }
    } else {
        for (int i = lane; i < p.n_prefix; i += 32) {
            const int len = p.lens ? min(max(p.lens[i], 0), p.L) : p.L;
            scratch[i] = make_int4(p.of || i > 0 ? 0 : p.B, 0, (len + 63) >> 6, len);
        }
        __syncwarp();
        if (p.of) {
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int v = map_of(b0);
                const bool in = v >= 0 && v < p.n_prefix;
                if (v >= p.n_prefix && blockIdx.x == 0) report_prefix(p, b0 + lane);
                const unsigned same = __match_any_sync(all, in ? v : -1);
                if (in && lane == __ffs(same) - 1) scratch[v].x += __popc(same);
                __syncwarp();
            }
        }
        int cmax = 1, n_tiles = 0;
        float work = 0.f;
        for (int i = lane; i < p.n_prefix; i += 32) {
            const int4 q = scratch[i];
            const int halves = q.z > 0 ? halves_of(q.x) : 0;
            scratch[i].y = halves;
            n_tiles += (halves + 1) >> 1;
            work += static_cast<float>(halves) * static_cast<float>(q.z);
            if (halves) cmax = max(cmax, q.z);
        }
        __syncwarp();
        cmax = __reduce_max_sync(all, cmax);
        n_tiles = __reduce_add_sync(all, n_tiles) * p.Hkv;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(all, work, o);
        work *= static_cast<float>(p.Hkv);
        T = 2 * cmax;
        if (n_tiles < ctas) {
            // the units lie between work / T and work / T + n_tiles
            const auto total = [&](int t) {
                int k = 0;
                for (int i = lane; i < p.n_prefix; i += 32) k += units_of(scratch[i].y, scratch[i].z, t);
                return __reduce_add_sync(all, k) * p.Hkv;
            };
            int lo = min(T, max(1, static_cast<int>(min(work / static_cast<float>(ctas), 1e9f)) - 1));
            T = max(lo, min(T, static_cast<int>(min(work / static_cast<float>(ctas - n_tiles), 1e9f)) + 2));
            while (lo < T) {
                const int mid = (lo + T) >> 1;
                if (total(mid) <= ctas) T = mid;
                else lo = mid + 1;
            }
        }
        for (int f0 = 0; f0 < p.n_prefix; f0 += 32) {
            const int ff = f0 + lane;
            const int k = ff < p.n_prefix ? units_of(scratch[ff].y, scratch[ff].z, T) * p.Hkv : 0;
            int incl = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(all, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(all, u < base + incl);
            if (f < 0 && hit) {
                const int l = __ffs(hit) - 1;
                f = f0 + l;
                start = base + __shfl_sync(all, incl - k, l);
            }
            base += __shfl_sync(all, incl, 31);
        }
        if (f >= 0) e = scratch[f];
    }
    if (f < 0) {
        if (lane == 0) unit->units = 0;
        return;
    }
    // units of a prefix: by kv head, in it the tiles of two and then the one of one, by range
    const int c = e.z, twos = e.y >> 1, r2 = ranges(2 * c, c, T), per_g = units_of(e.y, c, T);
    const int rem = u - start, g = rem / per_g, rg = rem - g * per_g;
    const bool two = rg < twos * r2;
    const int n = two ? r2 : ranges(c, c, T), t = two ? rg / r2 : twos, s = rg - t * r2;
    const int r0 = t * per_tile, here = min(per_tile, e.x - r0);
    if (lane == 0) {
        const int each = c / n, more = c - each * n;  // the first `more` ranges get a chunk more
        unit->f = f;
        unit->g = g;
        unit->s = s;
        unit->c0 = s * each + min(s, more);
        unit->c1 = unit->c0 + each + (s < more);
        unit->len = e.w;
        unit->members = here;
        unit->two = two;
        unit->units = base;
    }
    if (!p.of) {
        for (int i = lane; i < here; i += 32) member[i] = r0 + i;
    } else {
        int seen = 0;
        for (int b0 = 0; b0 < p.B && seen < r0 + here; b0 += 32) {
            const int v = map_of(b0);
            const unsigned m = __ballot_sync(all, v == f);
            const int rank = seen + __popc(m & ((1u << lane) - 1)) - r0;
            if (v == f && rank >= 0 && rank < here) member[rank] = b0 + lane;
            seen += __popc(m);
        }
    }
    __syncwarp();
    if (g == 0 && s == 0) {
        for (int i = lane; i < here; i += 32) p.n_ranges[member[i]] = n;
    }
}

// The products of a step of nk chunks of 64 keys, one thread. Descriptors differ in their start
// address alone, which is the low word's. This and all code that a CTA runs only a few times is kept
// small: a first run fetches its instructions through the memory system that K and V saturate, at 10
// cycles an instruction and more, which set the time of short prefixes.
//
// S (128 rows x 64 nk keys) = Q . K^T: both K-major, 128-byte rows in 8-row groups 1024 bytes apart,
// 32 bytes further per 16 columns and a half further per 64.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr, int nk) {
    const uint32_t idesc = idesc_bf16_f32(128, static_cast<uint32_t>(64 * nk));
    uint64_t qd = smem_desc(q_addr, 16, 1024, 2), kd = smem_desc(k_addr, 16, 1024, 2);
#pragma unroll 1
    for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_bf16(d_tmem, qd + k * 2, kd + k * 2, idesc, h > 0 || k > 0);
        qd += 16384 >> 4;
        kd += static_cast<uint64_t>(8192 * nk) >> 4;
    }
}

// O (128 rows x D) += P . V: P from TMEM in `parts` bf16 parts, two keys a column, where the softmax
// put them; V MN-major (idesc bit 16): N = D along a row's halves, 8192 nk bytes apart, K = the
// keys in groups of eight, 1024 bytes apart.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_addr, int nk, int parts, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, D) | (1u << 16);
    uint64_t vd = smem_desc(v_addr, static_cast<uint32_t>(8192 * nk), 1024, 2);
    uint32_t acc = accumulate;
#pragma unroll 1
    for (int k = 0; k < 4 * nk; ++k) {  // 16 keys: columns 16 k + 8 q of P's part q, the third at 64 + 8 k
        for (int q = 0; q < parts; ++q) {
            umma_bf16_ts(d_tmem, p_tmem + (q < 2 ? k * 16 + q * 8 : 64 + k * 8), vd, idesc, acc);
            acc = 1;
        }
        vd += 2048 >> 4;
    }
}

// One step of a row: S (nk chunks of 64 keys, the first `valid` of them real) into P over it in TMEM,
// with the running maximum (of the reference, log2 domain) and sum. S is read twice, once for the
// maximum and once for the exponentials, 32 columns a turn.
template <int D, int PARTS>
__device__ __forceinline__ void softmax_step(uint32_t s_addr, uint32_t o_addr, int nk, int valid, float scale_log2,
                                             float& m_ref, float& l, bool first) {
    const auto load = [&](int q, float(&v)[2][16]) {
        tmem_ld16(s_addr + q * 32, v[0]);
        tmem_ld16(s_addr + q * 32 + 16, v[1]);
        tmem_wait(v[0]);
        tmem_wait(v[1]);
        if (valid < 32 * q + 32) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                if (32 * q + k >= valid) v[k >> 4][k & 15] = -INFINITY;
            }
        }
    };
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int q = 0; q < 2 * nk; ++q) {
        float v[2][16];
        load(q, v);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            mx[0] = max3(mx[0], v[0][k], v[0][k + 1]);
            mx[1] = max3(mx[1], v[1][k], v[1][k + 1]);
        }
    }
    const float m_new = fmaxf(mx[0], mx[1]) * scale_log2;
    // the reference only moves when a row's maximum outgrows it by 2^8: until then the sums just
    // grow, which fp32 holds
    if (first) {
        m_ref = m_new;
    } else if (__any_sync(0xffffffffu, m_new > m_ref + 8.f)) {
        const float m2 = fmaxf(m_ref, m_new);
        const float f = m2 == -INFINITY ? 1.f : exp2_ftz(m_ref - m2);
        m_ref = m2;
        l *= f;
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
            float o[16];
            tmem_ld16(o_addr + q * 16, o);
            tmem_wait(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= f;
            tmem_st16(o_addr + q * 16, o);
        }
    }
    const float base = m_ref == -INFINITY ? 0.f : m_ref;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 scale2 = make_float2(scale_log2, scale_log2), base2 = make_float2(-base, -base);
    const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll 1
    for (int q = 0; q < 2 * nk; ++q) {
        float v[2][16];
        load(q, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi[8], lo[8], th[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 e = fma2(make_float2(v[h][2 * k], v[h][2 * k + 1]), scale2, base2);
                const float2 w = make_float2(exp2_ftz(e.x), exp2_ftz(e.y));
                sum[k & 1] = add2(sum[k & 1], w);
                hi[k] = pack_bf16(w.x, w.y);
                if (PARTS == 1) continue;
                float2 r = fma2(make_float2(bf_lo(hi[k]), bf_hi(hi[k])), minus, w);
                lo[k] = pack_bf16(r.x, r.y);
                if (PARTS == 3) {
                    r = fma2(make_float2(bf_lo(lo[k]), bf_hi(lo[k])), minus, r);
                    th[k] = pack_bf16(r.x, r.y);
                }
            }
            // P goes over the 16 scores that it was made from, part by part; the third part has the
            // columns behind a step of 64
            tmem_st8(s_addr + q * 32 + h * 16, hi);
            if (PARTS >= 2) tmem_st8(s_addr + q * 32 + h * 16 + 8, lo);
            if (PARTS == 3) tmem_st8(s_addr + 64 + q * 16 + h * 8, th);
        }
    }
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The 32 rows of HALF columns that a warp put into `stage` (piece c of row r at c ^ (r & 7)) to rows
// `at` of each lane (negative: none) of out, `pitch` apart; neighbouring lanes on neighbouring
// addresses (each thread storing its own row took 4 us for a tile).
template <int HALF>
__device__ __forceinline__ void store_rows(const uint8_t* stage, float* out, int pitch, long long at) {
    constexpr int HP = HALF / 4;
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < 32 * HP; e += 32) {
        const int row = e / HP, c = e % HP;
        const long long to = __shfl_sync(0xffffffffu, at, row);
        const float4 v = *reinterpret_cast<const float4*>(stage + row * (HALF * 4) + ((c ^ (row & 7)) << 4));
        if (to >= 0) *reinterpret_cast<float4*>(out + to * pitch + c * 4) = v;
    }
    __syncwarp();
}

// Where a count of K and V stages lies in the ring.
template <int NS>
struct RingPos {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ explicit RingPos(int n) : slot(n % NS), phase(static_cast<uint32_t>(n / NS) & 1u) {}
    __device__ __forceinline__ void advance(int by) {  // by < NS
        slot += by;
        if (slot >= NS) {
            slot -= NS;
            phase ^= 1u;
        }
    }
};

// KEYS: keys of a step, 128 (bf16 output, P in one or two bf16 parts) or 64 (fp32 output, three).
template <int D, int KEYS>
struct PrefixCfg {
    static constexpr int kTileBytes = 128 * D * 2;  // one Q tile
    static constexpr int kStage = KEYS * D * 2;     // K or V of a step
    static constexpr int kStages = std::min(12, (224 * 1024 - 2 * kTileBytes) / kStage);
    // copies of a CTA that have not landed yet: enough for the memory system's latency; more only
    // queue in it and hold up everything else that comes that way
    static constexpr int kInFlight = std::min(kStages, 96 * 1024 / kStage);
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
    __shared__ uint64_t full[NS], empty[NS], s_full[2], p_ready[2], pv_done[2], go;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_flag;
    __shared__ PrefixUnit unit;
    __shared__ int member[256];
    // (m, l) of a row in each stream, where the streams share one Q tile: in the other's memory
    float2(*ex)[128] = reinterpret_cast<float2(*)[128]>(smem + C::kTileBytes);
    volatile int* abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();  // the pass over the own caches fills SMs as they become free

    if (threadIdx.x == 32) {
        abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        mbar_init(&go, 1);
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
    // warp 0 goes straight to the plan and meets the others after it
    tc_fence_before();
    if (warp == 0) asm volatile("bar.arrive 5, %0;" ::"n"(kPrefixThreads) : "memory");
    else prefix_bar<5, kPrefixThreads>();
    tc_fence_after();
    // TMEM columns: S (and P over it) of the two streams at 0 and 128, O at 256 and 256 + D
    int it0 = 0;              // K and V stages used by earlier units
    int used[2] = {0, 0};     // steps each stream did in earlier units
    int paired = 0;           // earlier units with two row tiles
    for (int u = blockIdx.x;; u += gridDim.x) {
        if (warp == 0) plan_unit(p, u, reinterpret_cast<int4*>(smem), &unit, member);
        __syncthreads();
        tc_fence_after();
        const uint32_t tmem = tmem_sh;
        const PrefixUnit x = unit;
        if (x.units == 0) break;
        const int steps = (x.c1 - x.c0 + SMAX - 1) / SMAX;
        // bf16 parts of P. With two row tiles the products and the softmax set the pace, not K and V:
        // one part, as in dak_attn (its rounding stays below that of a bf16 output); with one the
        // second part's products are free.
        const int parts = KEYS == 64 ? 3 : x.two ? 1 : 2;
        const int items = x.two ? 2 * steps : steps;  // item i: stream i & 1, step i / 2 or i
        const long long slab = static_cast<long long>(x.f) * p.Hkv + x.g;
        const int tier = slab < p.h_s ? 0 : 1;
        const int step_of_shift = x.two ? 1 : 0;
        if (warp == 8) {
            // ------------------------------------------------------------ copies
            prefix_bar<4, 288>();  // Q's loads are on their way, ahead of the stream of K and V
            if (lane == 0) {
                const uint64_t policy = policy_evict_first();
                const auto wait_landed = [&](int i) {
                    return mbar_wait(&full[i % NS], static_cast<uint32_t>((i / NS) & 1), abort, p.st, DAK_ERR_TIMEOUT,
                                     X_PROD_FULL);
                };
                const int chunk0 = static_cast<int>((tier ? slab - p.h_s : slab) * p.slab_chunks);
                int it = it0;
                for (int j = 0; j < steps; ++j) {
                    const int c = x.c0 + j * SMAX, nk = min(SMAX, x.c1 - c);
                    const CUtensorMap* map = nk == SMAX ? &maps.step[tier] : &maps.tail[tier];
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int s = it % NS;
                        if (it >= NS && !mbar_wait(&empty[s], static_cast<uint32_t>((it / NS - 1) & 1), abort, p.st,
                                                   DAK_ERR_TIMEOUT, X_PROD_EMPTY)) {
                            goto copies_done;
                        }
                        if (it >= it0 + C::kInFlight && !wait_landed(it - C::kInFlight)) goto copies_done;
                        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nk * 64 * D * 2));
                        tma_load_5d(ring + static_cast<size_t>(s) * C::kStage, map, kv, chunk0 + c, &full[s], policy);
                    }
                }
            copies_done:
                if (*abort) {  // copies in flight land before the CTA may leave
                    volatile int dummy = 0;
                    for (int s = 0; s < NS && s < it; ++s) {
                        const int last = ((it - 1 - s) / NS) * NS + s;
                        mbar_wait(&full[s], static_cast<uint32_t>((last / NS) & 1), &dummy, p.st, DAK_ERR_TIMEOUT, X_DRAIN);
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 9) {
            // ------------------------------------------------------------ products, a warp per stream
            // The whole warp runs the loop, so that its state and the descriptors stay warp-uniform;
            // one elected lane issues. With one warp for both streams, what lies between the products
            // (waits, address arithmetic) added up: 2.6k cycles a step of both at 1.5k of products.
            const int st = warp - 9, stride = x.two ? 1 : 2;
            prefix_bar<2, 320>();  // Q lies in shared memory
            tc_fence_after();
            const bool leader = elect_one();
            const uint32_t q_addr = smem_u32(smem) + (x.two ? st * C::kTileBytes : 0), ring_addr = smem_u32(ring);
            const uint32_t s_tmem = tmem + st * 128, o_tmem = tmem + 256 + st * D;
            int j = x.two ? 0 : st, n = used[st];
            RingPos<NS> pos(it0 + 2 * j);  // K of step j; V follows
            const auto wait_full = [&](RingPos<NS> r) {
                return mbar_wait(&full[r.slot], r.phase, abort, p.st, DAK_ERR_TIMEOUT, X_MMA_FULL);
            };
            // a stage is free when both streams have used it, or the one that does has said so twice
            const auto release = [&](int slot) {
                umma_commit(&empty[slot]);
                if (!x.two) umma_commit(&empty[slot]);
            };
            const auto qk = [&]() {
                tc_fence_after();
                if (leader) {
                    const uint32_t b = ring_addr + pos.slot * C::kStage;
                    issue_qk<D>(s_tmem, q_addr, b, min(SMAX, x.c1 - x.c0 - j * SMAX));
                    umma_commit(&s_full[st]);
                    release(pos.slot);
                }
                __syncwarp();
            };
            // Two row tiles: the second stream starts once the first one's softmax is done, so that from
            // then on each one's softmax runs under the other's products (in step they waited for the
            // tensor cores together and then left them idle together).
            bool ok = j < steps && wait_full(pos);
            if (ok && x.two && st == 1) ok = mbar_wait(&go, paired & 1, abort, p.st, DAK_ERR_TIMEOUT, X_MMA_GO);
            if (ok) qk();
            for (bool first = true; ok; first = false, ++n) {
                RingPos<NS> v = pos;
                v.advance(1);
                ok = wait_full(v) && mbar_wait(&p_ready[st], n & 1, abort, p.st, DAK_ERR_TIMEOUT, X_MMA_P);
                if (!ok) break;
                if (first && x.two && st == 0 && lane == 0) mbar_arrive(&go);
                tc_fence_after();
                if (leader) {
                    const uint32_t b = ring_addr + v.slot * C::kStage;
                    issue_pv<D>(o_tmem, s_tmem, b, min(SMAX, x.c1 - x.c0 - j * SMAX), parts, !first);
                    umma_commit(&pv_done[st]);
                    release(v.slot);
                }
                __syncwarp();
                j += stride;
                if (j >= steps) break;
                pos.advance(2 * stride);
                // S's columns hold the P that the product just issued reads: it finishes first
                ok = wait_full(pos) && mbar_wait(&pv_done[st], n & 1, abort, p.st, DAK_ERR_TIMEOUT, X_MMA_PV);
                if (ok) qk();
            }
            __syncwarp();
        } else if (warp < 8) {
            // ------------------------------------------------------------ softmax, one row a thread
            const int st = warp >> 2, r = (warp & 3) * 32 + lane;
            const int mpt = p.mpt;
            {   // Q rows into the 128-byte swizzled K-major layout, rows without a member zero
                constexpr int PIECES = D / 8;  // 16-byte pieces of a row
                const int n = (x.two ? 256 : 128) * PIECES;
#pragma unroll 1
                for (int e = threadIdx.x; e < n; e += 256) {
                    const int rr = (e / PIECES) & 127, tile = e / (128 * PIECES), c = e % PIECES, m = rr / p.G;
                    const bool there = m < mpt && tile * mpt + m < x.members;
                    const __nv_bfloat16* src = p.Q + c * 8;
                    if (there) src += (static_cast<long long>(member[tile * mpt + m]) * p.Hq + x.g * p.G + rr - m * p.G) * D;
                    cp_async16(smem + tile * C::kTileBytes + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), src,
                               there ? 16 : 0);
                }
                asm volatile("bar.arrive 4, 288;" ::: "memory");  // K and V may start behind these copies
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                prefix_bar<2, 320>();
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
                if (valid < 64 * nk && (!x.two || st == 0)) {
                    // rows of V past the prefix may hold anything, also infinities and NaN, which a
                    // probability of zero would not cancel
                    const int vit = it0 + 2 * j + 1;
                    mbar_wait(&full[vit % NS], static_cast<uint32_t>((vit / NS) & 1), abort, p.st, DAK_ERR_TIMEOUT, X_SM_V);
                    uint8_t* v = ring + static_cast<size_t>(vit % NS) * C::kStage;
                    for (int e = r; e < (64 * nk - valid) * (D / 8); e += 128) {
                        const int row = valid + e / (D / 8), c = e % (D / 8);
                        *reinterpret_cast<uint4*>(v + (c >> 3) * (8192 * nk) + row * 128 + ((c & 7) << 4)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (KEYS == 64) softmax_step<D, 3>(s_addr, o_addr, nk, valid, p.scale_log2, m_ref, l, mine == 0);
                else if (x.two) softmax_step<D, 1>(s_addr, o_addr, nk, valid, p.scale_log2, m_ref, l, mine == 0);
                else softmax_step<D, 2>(s_addr, o_addr, nk, valid, p.scale_log2, m_ref, l, mine == 0);
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
            // half a row's columns at a time go through this stream's Q tile, which is free now
            constexpr int HALF = D / 2;
            uint8_t* stage = smem + st * C::kTileBytes + (warp & 3) * 32 * HALF * 4;
            const auto put = [&](const float(&o)[16], int q) {  // 16 columns from q * 16 of the half
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    *reinterpret_cast<float4*>(stage + lane * (HALF * 4) + (((q * 4 + k) ^ (lane & 7)) << 4)) =
                        make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            };
            const auto flush = [&](int col) { store_rows<HALF>(stage, p.o_part + col, D, valid_row ? at : -1ll); };
            if (x.two) {
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                    for (int q = 0; q < HALF / 16; ++q) {
                        float o[16];
                        tmem_ld16(o_addr + h * HALF + q * 16, o);
                        tmem_wait(o);
                        put(o, q);
                    }
                    flush(h * HALF);
                }
                if (valid_row) p.ml_part[at] = make_float2(m_ref, l);
            } else {
                ex[st][r] = make_float2(m_ref, l);
                tc_fence_before();
                prefix_bar<3, 256>();
                tc_fence_after();
                const float2 e0 = ex[0][r], e1 = ex[1][r];
                prefix_bar<3, 256>();  // ex lies in what is written next
                const float M = fmaxf(e0.x, e1.x), base = M == -INFINITY ? 0.f : M;
                const float f0 = exp2_ftz(e0.x - base), f1 = exp2_ftz(e1.x - base);
                const bool both = items > 1;  // the second stream had a step
#pragma unroll 1
                for (int q = 0; q < HALF / 16; ++q) {  // stream 0 the first half of the columns
                    float a[16], b[16];
                    tmem_ld16(tmem + lanes + 256 + st * HALF + q * 16, a);
                    tmem_ld16(tmem + lanes + 256 + D + st * HALF + q * 16, b);
                    tmem_wait(a);
                    tmem_wait(b);
#pragma unroll
                    for (int k = 0; k < 16; ++k) a[k] = both ? a[k] * f0 + b[k] * f1 : a[k] * f0;
                    put(a, q);
                }
                flush(st * HALF);
                if (valid_row && st == 0) p.ml_part[at] = make_float2(M, e0.y * f0 + (both ? e1.y * f1 : 0.f));
            }
        }
        it0 += 2 * steps;
        used[0] += (items + 1) / 2;
        used[1] += items / 2;
        paired += x.two;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (abort_flag || u + static_cast<int>(gridDim.x) >= x.units) break;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem_sh, 512);
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
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), PrefixCfg<D, KEYS>::kSmem);
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
    p.mpt = 128 / p.G;
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
