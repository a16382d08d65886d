// The prefix pass of dak_attn_prefix: attention of all requests that share a prefix over the
// prefix's rows, each (prefix, kv head) slab streamed once for up to 256 query rows (a row = one
// request's query head). Partial results go to the merge of dak_serve.cu.
//
// The contraction is GEMM-shaped (rows x keys x D twice), so it runs on the tcgen05 tensor cores
// as the usual two products with an online softmax between them, 64 keys a step:
//   S  = Q (128 rows x D, shared memory) . K^T (D x 64 keys, shared memory) -> TMEM, fp32
//   P  = 2^(S * scale log2 e - m), written to TMEM in two bf16 parts (three for an fp32 output)
//   O += P (TMEM) . V (64 keys x D, shared memory) -> TMEM, fp32
// A CTA has two streams, each 128 threads (thread = row) and a warp that issues its products, with S
// and O in TMEM and P written over the S that it comes from. S has two buffers, so that the next
// step's scores are there when a step's softmax ends.
// With more than 128 rows the streams hold two row tiles and both go through every key; with fewer
// they hold the same rows and take the steps in turn, and their results are merged in the CTA.
//
// The cache stores piece c of token t at c ^ (t & 7), which is the tensor cores' 128-byte swizzle
// once a row's two 128-byte halves lie apart; a 5-D tensor map (64 elements, 64 tokens, K and V,
// chunk, half) brings a chunk so in one copy of up to 32 KiB (issuing a copy takes its thread 0.3 us
// whatever its size, which held K and V apart to 20 bytes a cycle and SM). K is then a K-major
// operand; V, whose rows are keys, an MN-major one.
//
// What bounds it: with two row tiles a step's chain from S through the softmax to P and P.V, 2310 cycles
// (1640 with P in one part, half a bit of the output for speed, which is not taken). No pipe is full: the
// tensor cores are active 40% of the time, instructions issue in 29% of the cycles, exp2 and conversions 13%;
// a sub-partition has two softmax warps, one of each stream, to cover their latencies, and registers for no
// more. With one the arrival of K and V, 23 bytes a cycle and SM, about what L2 delivers to all SMs at
// once; short prefixes the start (plan, Q, first chunks: 5 to 12 thousand cycles, most of them code that
// runs for the first time). 128 requests of 64 query and 8 kv heads, D 128, over 16K, 9K and 130 rows and
// up to 256 own ones: 76.3 us for the whole call; 32 of 32 heads over 8K and up to 1024 own ones: 31.7 us.
//
// Which CTA works on what is planned on the device from the prefixes' lengths and the requests'
// map, so that a captured call follows them: units (prefix, kv head, 256-row tile, key range),
// every prefix cut into ranges of at most T chunks, T the smallest for which the units still fit
// the CTAs at once.
#include <algorithm>

#include <cudaTypedefs.h>

#include "dak_device.cuh"

namespace dak {

constexpr int kSoftmaxThreads = 2 * 128;  // two streams, a thread a row
constexpr int kPrefixThreads = kSoftmaxThreads + 3 * 32;  // and copies, each stream's products
constexpr int kPrefixTwoCost = 3, kPrefixOneCost = 2;  // of a chunk, by a tile's 128-row halves
constexpr int kPrefixMinChunks = 2;      // chunks of 64 keys in a range, at least
constexpr int64_t kPrefixPartialBytes = 64ll << 20;  // of partials in the workspace (prefix_max_ranges)

struct PrefixMaps {
    CUtensorMap tier[2];  // host, HBM: chunks of 64 keys
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
    int inv_G;  // 2^16 / G rounded up: (r * inv_G) >> 16 is r / G for any row r of a tile
    float scale_log2;
    DevStatus* st;
};

enum : uint32_t { X_PROD_EMPTY = 0x51, X_PROD_FULL, X_MMA_FULL, X_MMA_P, X_MMA_PV, X_SM_S, X_SM_O, X_DRAIN };

// What a CTA works on.
struct PrefixUnit {
    int f, g, s;       // prefix, kv head, key range
    int c0, c1;        // its chunks
    int len;           // rows of the prefix
    int members;       // requests of this tile
    int two;           // the members fill more than one 128-row tile
    int units;         // units of the whole launch
    int shared;        // other tiles read the same chunks
};

__device__ __forceinline__ void tma_load_chunk(void* dst, const CUtensorMap* map, int chunk, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%2, %2, %3, %2}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(chunk), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// mbar_wait with a plain test first: where the phase is long over, as it mostly is for the warps that
// issue products, the suspending form takes twice the time.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort, DevStatus* st, uint32_t where) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok || mbar_wait(bar, parity, abort, st, DAK_ERR_TIMEOUT, where);
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

// n / d for n >= 0 and quotients below 2^21 (the float quotient is off by less than one, which the
// remainder puts right), a few instructions where the integer division is dozens.
__device__ __forceinline__ int quotient(int n, int d) {
    const int q = static_cast<int>(static_cast<float>(n) * __fdividef(1.f, static_cast<float>(d))), r = n - q * d;
    return q + (r >= d) - (r < 0);
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
    // Requests' rows make full tiles of two 128-row halves and one more of one or two; `halves` holds
    // both kinds: tiles of two in its upper bits, one of one in bit 0. The ranges are cut as if a chunk
    // cost a tile of two 1.5 times what it costs one of one (2310 cycles to about 1450 of its bytes' arrival;
    // 128 requests over 16K, 9K and 130 rows, from a cold L2: 81 us so, 85 by 5 to 4 or 8 to 7, 86 by 4 to 3;
    // one prefix alone takes the same time by all of them).
    const auto halves_of = [&](int cnt) {
        const int full = quotient(cnt, per_tile), rest = cnt - full * per_tile;
        return rest > p.mpt ? 2 * full + 2 : 2 * full + (rest > 0);
    };
    // Ranges of a tile: its work over T, rounded up. (Any number from 1 to the limits is a valid cut;
    // what it takes is the same one everywhere, so a reciprocal does.)
    const auto ranges = [&](int cost, int c, float inv) {
        return max(1, min(min(__float2int_ru(static_cast<float>(cost * c) * inv - 1e-3f), p.n_pre), c / kPrefixMinChunks));
    };
    const auto units_of = [&](int halves, int c, float inv) {  // per kv head
        return halves == 0 || c == 0 ? 0 : (halves >> 1) * ranges(kPrefixTwoCost, c, inv) + (halves & 1) * ranges(kPrefixOneCost, c, inv);
    };
    const auto inverse = [](int t) { return __fdividef(1.f, static_cast<float>(t)); };
    int f = -1, start = 0, base = 0, T = 1;
    int4 e;
    if (p.n_prefix == 1) {
        const int len = p.lens ? min(max(p.lens[0], 0), p.L) : p.L;
        int cnt = p.B;
        if (p.of) {
            cnt = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int v = map_of(b0);
                if (v > 0 && blockIdx.x == 0) report_prefix(p, b0 + lane);
                cnt += __popc(__ballot_sync(all, v == 0));
            }
        }
        e = make_int4(cnt, halves_of(cnt), (len + 63) >> 6, len);
        const int tiles = ((e.y + 1) >> 1) * p.Hkv;
        if (tiles > 0 && e.z > 0) {
            T = kPrefixTwoCost * e.z;
            if (tiles < ctas) {
                if (e.y == 1 || (e.y & 1) == 0) {  // tiles of one kind: each the same share of the CTAs
                    const int each = quotient(ctas, tiles), work = (e.y == 1 ? kPrefixOneCost : kPrefixTwoCost) * e.z;
                    T = quotient(work + each - 1, each);
                } else {
                    int lo = 1;
#pragma unroll 1
                    while (lo < T) {
                        const int mid = (lo + T) >> 1;
                        if (units_of(e.y, e.z, inverse(mid)) * p.Hkv <= ctas) T = mid;
                        else lo = mid + 1;
                    }
                }
            }
            base = units_of(e.y, e.z, inverse(T)) * p.Hkv;
            if (u < base) f = 0;
        }
    } else {
#pragma unroll 1
        for (int i = lane; i < p.n_prefix; i += 32) {
            const int len = p.lens ? min(max(p.lens[i], 0), p.L) : p.L;
            scratch[i] = make_int4(p.of || i > 0 ? 0 : p.B, 0, (len + 63) >> 6, len);
        }
        __syncwarp();
        if (p.of) {
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int v = map_of(b0);
                const bool in = v >= 0 && v < p.n_prefix;
                if (v >= p.n_prefix && blockIdx.x == 0) report_prefix(p, b0 + lane);
                if (in) atomicAdd(&scratch[v].x, 1);
            }
            __syncwarp();
        }
        int cmax = 1, n_tiles = 0;
        float work = 0.f;
#pragma unroll 1
        for (int i = lane; i < p.n_prefix; i += 32) {
            const int4 q = scratch[i];
            const int halves = q.z > 0 ? halves_of(q.x) : 0;
            scratch[i].y = halves;
            n_tiles += (halves + 1) >> 1;
            work += static_cast<float>((halves >> 1) * kPrefixTwoCost + (halves & 1) * kPrefixOneCost) * static_cast<float>(q.z);
            if (halves) cmax = max(cmax, q.z);
        }
        __syncwarp();
        cmax = __reduce_max_sync(all, cmax);
        n_tiles = __reduce_add_sync(all, n_tiles) * p.Hkv;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(all, work, o);
        work *= static_cast<float>(p.Hkv);
        T = kPrefixTwoCost * cmax;
        if (n_tiles < ctas) {
            // the units lie between work / T and work / T + n_tiles
            const auto sum_on_lanes = [&](int t) {
                int k = 0;
                const float inv = inverse(t);
#pragma unroll 1
                for (int i = lane; i < p.n_prefix; i += 32) k += units_of(scratch[i].y, scratch[i].z, inv);
                return __reduce_add_sync(all, k) * p.Hkv;
            };
            int lo = min(T, max(1, static_cast<int>(min(work / static_cast<float>(ctas), 1e9f)) - 1));
            T = max(lo, min(T, static_cast<int>(min(work / static_cast<float>(ctas - n_tiles), 1e9f)) + 2));
            if (p.n_prefix <= 32) {  // a lane a candidate
#pragma unroll 1
                while (lo < T) {
                    const int step = (T - lo + 30) / 31, t = min(T, lo + lane * step);
                    const float inv = inverse(t);
                    int k = 0;
#pragma unroll 1
                    for (int i = 0; i < p.n_prefix; ++i) k += units_of(scratch[i].y, scratch[i].z, inv);
                    // the lowest that fits (T does, or is the most there is); all below do not
                    const int at = __ffs(__ballot_sync(all, k * p.Hkv <= ctas || t == T)) - 1;
                    T = min(T, lo + at * step);
                    lo = at > 0 ? min(T, lo + (at - 1) * step + 1) : T;
                }
            } else {
#pragma unroll 1
                while (lo < T) {
                    const int mid = (lo + T) >> 1;
                    if (sum_on_lanes(mid) <= ctas) T = mid;
                    else lo = mid + 1;
                }
            }
        }
        const float inv = inverse(T);
#pragma unroll 1
        for (int f0 = 0; f0 < p.n_prefix; f0 += 32) {
            const int ff = f0 + lane;
            const int k = ff < p.n_prefix ? units_of(scratch[ff].y, scratch[ff].z, inv) * p.Hkv : 0;
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
    const float inv = inverse(T);
    const int c = e.z, twos = e.y >> 1, r2 = ranges(kPrefixTwoCost, c, inv), per_g = units_of(e.y, c, inv);
    const int rem = u - start, g = quotient(rem, per_g), rg = rem - g * per_g;
    const bool two = rg < twos * r2;
    const int n = two ? r2 : ranges(kPrefixOneCost, c, inv), t = two ? quotient(rg, r2) : twos, s = rg - t * r2;
    const int r0 = t * per_tile, here = min(per_tile, e.x - r0);
    if (lane == 0) {
        const int each = quotient(c, n), more = c - each * n;  // the first `more` ranges get a chunk more
        unit->f = f;
        unit->g = g;
        unit->s = s;
        unit->c0 = s * each + min(s, more);
        unit->c1 = unit->c0 + each + (s < more);
        unit->len = e.w;
        unit->members = here;
        unit->two = two;
        unit->units = base;
        unit->shared = e.y > 2;
    }
    if (!p.of) {
#pragma unroll 1
        for (int i = lane; i < here; i += 32) member[i] = r0 + i;
    } else {
        int seen = 0;
#pragma unroll 1
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
#pragma unroll 1
        for (int i = lane; i < here; i += 32) p.n_ranges[member[i]] = n;
    }
}

// The products of a step, one thread. Descriptors differ in their start address alone, which is the
// low word's. This and all code that a CTA runs only a few times is kept small: a first run fetches
// its instructions through the memory system that K and V saturate, at 10 cycles an instruction and
// more, which set the time of short prefixes.
//
// S (128 rows x 64 keys) = Q . K^T: both K-major, 128-byte rows in 8-row groups 1024 bytes apart, 32
// bytes further per 16 columns and a half further per 64.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_addr, uint32_t k_addr) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 64);
    const uint64_t qd = smem_desc(q_addr, 16, 1024, 2), kd = smem_desc(k_addr, 16, 1024, 2);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        umma_bf16(d_tmem, qd + (k >> 2) * (16384 >> 4) + (k & 3) * 2, kd + (k >> 2) * (16384 >> 4) + (k & 3) * 2, idesc, k > 0);
    }
}

// Columns of the 16 keys k of part q of P, from where its S begins: a third part lies beyond it.
__device__ __forceinline__ constexpr uint32_t p_column(int k, int q) { return q < 2 ? k * 16 + q * 8 : 64 + k * 8; }

// O (128 rows x D) += P . V: P from TMEM in PARTS bf16 parts, two keys a column, where the softmax
// put them; V MN-major (idesc bit 16): N = D along a row's halves, 16384 bytes apart, K = the keys in
// groups of eight, 1024 bytes apart.
template <int D, int PARTS>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_addr, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, D) | (1u << 16);
    const uint64_t vd = smem_desc(v_addr, 16384, 1024, 2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 16 keys: 8 columns of each part (p_column)
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            umma_bf16_ts(d_tmem, p_tmem + p_column(k, q), vd + k * (2048 >> 4), idesc,
                         k > 0 || q > 0 ? 1u : static_cast<uint32_t>(accumulate));
        }
    }
}

// One step of a row: its 64 scores (from `valid` on not real) into P in PARTS bf16 parts, over them, with
// the row's running sum and the reference that its exponents are taken against (log2 domain). `grown`
// is called when a row of the warp outgrows its reference, with the factor for O.
template <int PARTS, class Grown>
__device__ __forceinline__ void softmax_step(uint32_t s_addr, int valid, float scale_log2, float& m_ref, float& l, bool first,
                                             const Grown& grown) {
    // with three parts O is in registers too, which leaves none for all scores: they are read twice
    constexpr bool TWICE = PARTS == 3;
    float v[TWICE ? 1 : 4][16];
    const auto mask = [&](int q) {
        if (valid < 64) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (q * 16 + k >= valid) v[TWICE ? 0 : q][k] = -INFINITY;
            }
        }
    };
    const auto read_again = [&](int q) {
        tmem_ld16(s_addr + q * 16, v[0]);
        tmem_wait(v[0]);
        mask(q);
    };
    if (!TWICE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld16(s_addr + q * 16, v[TWICE ? 0 : q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_wait(v[TWICE ? 0 : q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) mask(q);
    }
    float mx[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (TWICE) read_again(q);
        const float(&x)[16] = v[TWICE ? 0 : q];
        mx[q] = fmaxf(x[0], x[1]);
#pragma unroll
        for (int k = 2; k < 16; k += 2) mx[q] = max3(mx[q], x[k], x[k + 1]);
    }
    const float m_new = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale_log2;
    // the reference only moves when a row's maximum outgrows it by 2^8: until then the sums just
    // grow, which fp32 holds
    if (first) {
        m_ref = m_new;
    } else if (__any_sync(0xffffffffu, m_new > m_ref + 8.f)) {
        const float m2 = fmaxf(m_ref, m_new);
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
    for (int q = 0; q < 4; ++q) {
        uint32_t hi[8], lo[8], th[8];
        if (TWICE) read_again(q);
        const float(&x)[16] = v[TWICE ? 0 : q];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), scale2, base2);
            const float2 w = make_float2(exp2_ftz(e.x), exp2_ftz(e.y));
            sum[k & 1] = add2(sum[k & 1], w);
            hi[k] = pack_bf16(w.x, w.y);
            float2 r = fma2(make_float2(bf_lo(hi[k]), bf_hi(hi[k])), minus, w);
            lo[k] = pack_bf16(r.x, r.y);
            if (PARTS == 3) {
                r = fma2(make_float2(bf_lo(lo[k]), bf_hi(lo[k])), minus, r);
                th[k] = pack_bf16(r.x, r.y);
            }
        }
        tmem_st8(s_addr + p_column(q, 0), hi);
        tmem_st8(s_addr + p_column(q, 1), lo);
        if (PARTS == 3) tmem_st8(s_addr + p_column(q, 2), th);
    }
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The 32 rows of COLS columns that a warp put into `stage` (piece c of row r at stage_piece) to rows
// `at` of each lane (negative: none) of out, `pitch` apart; neighbouring lanes on neighbouring
// addresses (each thread storing its own row took 4 us for a tile).
template <int COLS>
__device__ __forceinline__ int stage_piece(int row, int c) {
    return row * (COLS / 4) + (c ^ (row & (COLS / 4 - 1)));
}

template <int COLS>
__device__ __forceinline__ void store_rows(const float4* stage, float* out, int pitch, long long at) {
    constexpr int PIECES = COLS / 4;
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < 32 * PIECES; e += 32) {
        const int row = e / PIECES, c = e % PIECES;
        const long long to = __shfl_sync(0xffffffffu, at, row);
        const float4 v = stage[stage_piece<COLS>(row, c)];
        if (to >= 0) *reinterpret_cast<float4*>(out + to * pitch + c * 4) = v;
    }
    __syncwarp();
}

// Where a count of stages (chunks) lies in the ring.
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

template <int D>
struct PrefixCfg {
    static constexpr int kTileBytes = 128 * D * 2;  // one Q tile
    static constexpr int kStage = 2 * 64 * D * 2;   // a chunk: per half row, K's 64 rows and then V's
    static constexpr int kV = 64 * 128;             // V behind K
    static constexpr int kStages = (224 * 1024 - 2 * kTileBytes) / kStage;
    // copies of a CTA that have not landed yet: enough for the memory system's latency; more only
    // queue in it and hold up everything else that comes that way
    static constexpr int kInFlight = 96 * 1024 / kStage;
    static constexpr int kSmem = 2 * kTileBytes + kStages * kStage + 1024;
};

// F32: fp32 output, P in three bf16 parts, which leave no room for a second S.
template <int D, bool F32>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ PrefixMaps maps) {
    using C = PrefixCfg<D>;
    constexpr int NS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    uint8_t* ring = smem + 2 * C::kTileBytes;
    __shared__ uint64_t full[NS], empty[NS], s_full[2][2], p_ready[2][2], pv_done[2][2];
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_flag;
    __shared__ PrefixUnit unit;
    // the tile's requests: not in the ring, where copies by another proxy would follow these writes
    __shared__ int member[256];
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
    // warp 0 goes straight to the plan and meets the others after it
    tc_fence_before();
    if (warp == 0) asm volatile("bar.arrive 5, %0;" ::"n"(kPrefixThreads) : "memory");
    else prefix_bar<5, kPrefixThreads>();
    tc_fence_after();
    grid_dep_wait();  // launched while the previous kernel ends
    grid_dep_launch();  // the pass over the own caches fills SMs as they become free
    // TMEM columns: stream s has S at 128 s + 64 b (buffer b) with P over it, and O at 256 + D s
    constexpr int SB = F32 ? 1 : 2;  // buffers of S
    int it0 = 0;  // stages used by earlier units
    int filled[2][2] = {{0, 0}, {0, 0}};  // steps of each stream by its S buffers
    for (int u = blockIdx.x;; u += gridDim.x) {
        if (warp == 0) plan_unit(p, u, reinterpret_cast<int4*>(smem), &unit, member);
        __syncthreads();
        tc_fence_after();
        const uint32_t tmem = tmem_sh;
        const PrefixUnit x = unit;
        if (x.units == 0) break;
        // Steps are chunks. Two row tiles: both streams take every step; one: they take turns.
        // P has two bf16 parts (2^-16), whatever the number of rows, so that a request's error does not
        // depend on how many others share its prefix: of one part (2^-8) alone the error would be as large
        // as the output's rounding. An fp32 output takes three (2^-24).
        const int steps = x.c1 - x.c0;
        const int stride = x.two ? 1 : 2;
        // S buffer of a stream's step i of this unit, and the parity of its barriers' phase. Each buffer
        // has barriers of its own: a wait by parity is right only where the phase before is known to be
        // over and the one after not to be, and steps i and i + 2 of a buffer wait for each other.
        const auto buf = [&](int i) { return i & (SB - 1); };
        const auto par = [&](int f0, int f1, int i) { return static_cast<uint32_t>((buf(i) ? f1 : f0) + i / SB) & 1u; };
        const long long slab = static_cast<long long>(x.f) * p.Hkv + x.g;
        const int tier = slab < p.h_s ? 0 : 1;

        if (warp == 8) {
            // ------------------------------------------------------------ copies
            prefix_bar<4, kSoftmaxThreads + 32>();  // Q's loads are on their way, ahead of the stream of K and V
            if (lane == 0) {
                const uint64_t policy = x.shared ? policy_evict_last() : policy_evict_first();
                const int chunk0 = static_cast<int>((tier ? slab - p.h_s : slab) * p.slab_chunks) + x.c0;
                RingPos<NS> pos(it0), landed(it0);
                int i = 0;
                bool ok = true;
                for (; i < steps; ++i) {
                    if (it0 + i >= NS) ok = wait_phase(&empty[pos.slot], pos.phase ^ 1u, abort, p.st, X_PROD_EMPTY);
                    if (ok && i >= C::kInFlight) {
                        ok = wait_phase(&full[landed.slot], landed.phase, abort, p.st, X_PROD_FULL);
                        landed.advance(1);
                    }
                    if (!ok) break;
                    mbar_arrive_expect_tx(&full[pos.slot], C::kStage);
                    tma_load_chunk(ring + pos.slot * C::kStage, &maps.tier[tier], chunk0 + i, &full[pos.slot], policy);
                    pos.advance(1);
                }
                if (!ok) {  // copies in flight land before the CTA may leave
                    volatile int dummy = 0;
                    for (int k = max(0, i - C::kInFlight); k < i; ++k) {
                        const RingPos<NS> r(it0 + k);
                        wait_phase(&full[r.slot], r.phase, &dummy, p.st, X_DRAIN);
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 9) {
            // ------------------------------------------------------------ products, a warp per stream
            // The whole warp runs the loop, so that its state and the descriptors stay warp-uniform;
            // one elected lane issues.
            const int st = warp - 9;
            prefix_bar<2, kSoftmaxThreads + 64>();  // Q lies in shared memory
            tc_fence_after();
            const bool leader = elect_one();
            const uint32_t q_addr = smem_u32(smem) + (x.two ? st * C::kTileBytes : 0), ring_addr = smem_u32(ring);
            const uint32_t s_tmem = tmem + st * 128, o_tmem = tmem + 256 + st * D;
            const int first = x.two ? 0 : st, mine = first < steps ? (steps - first + stride - 1) / stride : 0;
            const int f0 = filled[st][0], f1 = filled[st][1];
            RingPos<NS> kpos(it0 + first), vpos(it0 + first);
            const auto qk = [&](int i) {  // S of this stream's step i
                if (!wait_phase(&full[kpos.slot], kpos.phase, abort, p.st, X_MMA_FULL)) return false;
                // the product that read P in these columns is done
                if (i >= SB && !wait_phase(&pv_done[st][buf(i)], par(f0, f1, i - SB), abort, p.st, X_MMA_PV)) return false;
                tc_fence_after();
                if (leader) {
                    issue_qk<D>(s_tmem + buf(i) * 64, q_addr, ring_addr + kpos.slot * C::kStage);
                    umma_commit(&s_full[st][buf(i)]);
                }
                __syncwarp();
                kpos.advance(stride);
                return true;
            };
            bool ok = mine == 0 || qk(0);
            for (int i = 0; i < mine && ok; ++i) {
                if (!F32 && i + 1 < mine && !qk(i + 1)) break;
                if (!wait_phase(&p_ready[st][buf(i)], par(f0, f1, i), abort, p.st, X_MMA_P)) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t p_tmem = s_tmem + buf(i) * 64, v = ring_addr + vpos.slot * C::kStage + C::kV;
                    if (F32) issue_pv<D, 3>(o_tmem, p_tmem, v, false);
                    else issue_pv<D, 2>(o_tmem, p_tmem, v, i > 0);
                    umma_commit(&pv_done[st][buf(i)]);
                    // a stage is free when both streams have used it, or the one that does has said so twice
                    umma_commit(&empty[vpos.slot]);
                    if (!x.two) umma_commit(&empty[vpos.slot]);
                }
                __syncwarp();
                vpos.advance(stride);
                if (F32 && i + 1 < mine) ok = qk(i + 1);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ softmax, a thread a row
            const int st = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
            const int mpt = p.mpt;
            // where row r of this stream's tile, or of the tile that the streams share, has its results
            const int tile = x.two ? st : 0, m = (r * p.inv_G) >> 16;
            const bool valid_row = m < mpt && tile * mpt + m < x.members;
            long long at = 0;
            if (valid_row) {
                at = (static_cast<long long>(member[tile * mpt + m]) * p.Hq + x.g * p.G + r - m * p.G) * p.n_pre + x.s;
            }
            {   // Q rows into the 128-byte swizzled K-major layout, rows without a member zero
                constexpr int PIECES = D / 8;  // 16-byte pieces of a row
                const int n = (x.two ? 256 : 128) * PIECES;
#pragma unroll 4
                for (int e = threadIdx.x; e < n; e += kSoftmaxThreads) {
                    const int rr = (e / PIECES) & 127, t = e / (128 * PIECES), c = e % PIECES, mm = (rr * p.inv_G) >> 16;
                    const bool there = mm < mpt && t * mpt + mm < x.members;
                    const __nv_bfloat16* src = p.Q + c * 8;
                    if (there) src += (static_cast<long long>(member[t * mpt + mm]) * p.Hq + x.g * p.G + rr - mm * p.G) * D;
                    cp_async16(smem + t * C::kTileBytes + (c >> 3) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), src,
                               there ? 16 : 0);
                }
                asm volatile("bar.arrive 4, %0;" ::"n"(kSoftmaxThreads + 32) : "memory");  // K and V may start behind these copies
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                prefix_bar<2, kSoftmaxThreads + 64>();
            }
            const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
            const uint32_t s_addr = tmem + lanes + st * 128, o_addr = tmem + lanes + 256 + st * D;
            const int f0 = filled[st][0], f1 = filled[st][1];
            float m_ref = -INFINITY, l = 0.f;
            // An fp32 output's O is summed here, a step's product at a time: the tensor cores cut off what
            // they add to a sum, about 2^-26 of it an instruction, twelve a step and always towards zero
            // (100 requests of 64 query heads over 8000 rows: relative error 5.4e-6 so and 75 us, 4.0e-7
            // and 92 us with the sums here).
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
            for (int j = x.two ? 0 : st; j < steps; j += stride, ++i) {
                const int valid = min(64, x.len - (x.c0 + j) * 64);
                ok = mbar_wait(&s_full[st][buf(i)], par(f0, f1, i), abort, p.st, DAK_ERR_TIMEOUT, X_SM_S);
                if (!__all_sync(0xffffffffu, ok)) {  // a wait ran out: the whole warp stops
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (valid < 64) {
                    // Rows of V past the prefix may hold anything, also infinities and NaN, which a
                    // probability of zero would not cancel. Both streams of a step clear them, as either
                    // one's product may be first.
                    // (The scores say that the chunk is there.)
                    uint8_t* rows = ring + RingPos<NS>(it0 + j).slot * C::kStage + C::kV;
                    for (int e = r; e < (64 - valid) * (D / 8); e += 128) {
                        const int row = valid + e / (D / 8), c = e % (D / 8);
                        *reinterpret_cast<uint4*>(rows + (c >> 3) * 16384 + row * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
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
                    mbar_wait(&pv_done[st][buf(i - 1)], par(f0, f1, i - 1), abort, p.st, DAK_ERR_TIMEOUT, X_SM_O);
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
                if (F32 && i > 0) add_product();  // the last step's: its scores' columns are these
                if (F32) softmax_step<3>(at_s, valid, p.scale_log2, m_ref, l, i == 0, grown);
                else softmax_step<2>(at_s, valid, p.scale_log2, m_ref, l, i == 0, grown);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[st][buf(i)]);
            }
            for (int k = max(0, i - SB); ok && k < i; ++k) {  // one phase of each buffer's
                ok = mbar_wait(&pv_done[st][buf(k)], par(f0, f1, k), abort, p.st, DAK_ERR_TIMEOUT, X_SM_O);
            }
            __syncwarp();
            if (F32) {  // back to where the results are read from
                tc_fence_after();
                if (i > 0) add_product();
#pragma unroll
                for (int q = 0; q < (F32 ? D / 16 : 0); ++q) tmem_st16(o_addr + q * 16, sum[q]);
                tmem_wait_st();
            }
            // ---- results
            // Q's memory, no longer read, takes the streams' (m, l) where they share a tile, and then, half
            // a row's columns at a time, the results on their way out.
            constexpr int COLS = D / 2;
            float M = m_ref, total = l, w0 = 1.f, w1 = 0.f;
            const bool both = !x.two && steps > 1;  // the streams' rows are the same and both had a step
            tc_fence_before();
            if (!x.two) {
                float2(*ex)[128] = reinterpret_cast<float2(*)[128]>(smem + C::kTileBytes);
                ex[st][r] = make_float2(m_ref, l);
                prefix_bar<3, kSoftmaxThreads>();
                const float2 e0 = ex[0][r], e1 = ex[1][r];
                prefix_bar<3, kSoftmaxThreads>();  // ex lies in what is written next
                M = fmaxf(e0.x, e1.x);
                const float base = M == -INFINITY ? 0.f : M;
                w0 = exp2_ftz(e0.x - base);
                w1 = both ? exp2_ftz(e1.x - base) : 0.f;
                total = w0 * e0.y + (both ? w1 * e1.y : 0.f);
            }
            tc_fence_after();
            float4* stage = reinterpret_cast<float4*>(smem + st * C::kTileBytes + quad * 32 * COLS * 4);
#pragma unroll 1
            for (int col = x.two ? 0 : st * COLS; col < (x.two ? D : (st + 1) * COLS); col += COLS) {
#pragma unroll 1
                for (int q = 0; q < COLS / 16; ++q) {
                    float o[16];
                    tmem_ld16(tmem + lanes + 256 + (x.two ? st * D : 0) + col + q * 16, o);
                    tmem_wait(o);
                    if (!x.two) {
                        float b[16];
                        tmem_ld16(tmem + lanes + 256 + D + col + q * 16, b);
                        tmem_wait(b);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = both ? o[k] * w0 + b[k] * w1 : o[k] * w0;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        stage[stage_piece<COLS>(lane, q * 4 + k)] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
                store_rows<COLS>(stage, p.o_part + col, D, valid_row ? at : -1ll);
            }
            if (valid_row && (x.two || st == 0)) p.ml_part[at] = make_float2(M, total);
        }
        it0 += steps;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int n = x.two ? steps : (steps + 1 - st) / 2;
            filled[st][0] += (n + SB - 1) / SB;
            filled[st][1] += SB == 2 ? n / 2 : 0;
        }
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

// The prefix's chunks of one tier as the kernel copies them: (64 elements, 64 tokens, K and V, chunk,
// half of a row).
static bool make_prefix_map(CUtensorMap* map, const void* base, int64_t chunks, int D) {
    const auto enc = encode_fn();
    if (!enc || fault_due(DAK_FAULT_TENSOR_MAP)) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
    const cuuint64_t dims[5] = {64, 64, 2, static_cast<cuuint64_t>(chunks), static_cast<cuuint64_t>(D / 64)};
    const cuuint64_t strides[4] = {row, 64 * row, 128 * row, 128};
    const cuuint32_t box[5] = {64, 64, 2, 1, static_cast<cuuint32_t>(D / 64)};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every row has a place in the workspace for each range that its prefix may be cut into. As many ranges as a
// kv head has SMs, so that one request alone fills them, are 545 MB for 512 requests of 16 query heads on one
// kv head, whose prefix is cut into a few: past kPrefixPartialBytes there are fewer. Those 512 over 16K rows
// 105.6 us so, 116.9 without the limit (fewer partials are merged by warps); one of them alone over
// 16K 42 us, 51 without, 38 with 128 MiB, 54 with 32; one of 256 requests of 32 and 8 heads 52, 51, 49, 60.
int prefix_max_ranges(const dak_placement* P, int64_t rows) {
    const int chunks = (P->L + 63) / 64;
    const int most = std::min(std::min(device_sm_count(), 256) / P->H_kv, (chunks + kPrefixMinChunks - 1) / kPrefixMinChunks);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, kPrefixPartialBytes / (rows * (P->D + 2) * 4))));
}

template <int D, bool F32>
static cudaError_t launch_prefix_d(const PrefixParams& p, const PrefixMaps& maps, int grid, cudaStream_t s) {
    auto k = prefix_kernel<D, F32>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(k), PrefixCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kPrefixThreads);
    cfg.dynamicSmemBytes = PrefixCfg<D>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p, maps);
}

dak_status launch_prefix(const void* Q, const dak_placement* P, const int* lens, const int* of, int B, int H_q,
                         float scale_log2, int o_fp32, float* o_part, float* ml_part, int* n_ranges, cudaStream_t s) {
    const int D = P->D;
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
    p.inv_G = (65536 + p.G - 1) / p.G;
    p.L = P->L;
    p.n_prefix = P->B;
    p.n_pre = prefix_max_ranges(P, static_cast<int64_t>(B) * H_q);
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
        if (!make_prefix_map(&maps.tier[tier], base, n * p.slab_chunks, D)) return DAK_ERR_CUDA;
    }
    // no more CTAs than units can come out: every tile with members in every range
    const int per_tile = 2 * (128 / p.G);
    const int64_t tiles = std::min<int64_t>(B, P->B + static_cast<int64_t>(B) / per_tile);
    const int grid = static_cast<int>(std::min<int64_t>(device_sm_count(), tiles * p.Hkv * p.n_pre));
    cudaError_t e;
    if (D == 128) {
        e = o_fp32 ? launch_prefix_d<128, true>(p, maps, grid, s) : launch_prefix_d<128, false>(p, maps, grid, s);
    } else {
        e = o_fp32 ? launch_prefix_d<64, true>(p, maps, grid, s) : launch_prefix_d<64, false>(p, maps, grid, s);
    }
    return cuda_status(e);
}

}  // namespace dak
