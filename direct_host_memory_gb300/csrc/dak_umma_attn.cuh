// Attention on the tcgen05 tensor cores over chunks of a placed KV cache, the parts that the prefix
// pass (dak_prefix.cu) and the attention of drafted trees (dak_tree.cu) share: chunks by tensor map into
// shared memory, the two products of a 64-key step, the softmax between them, results on their way out.
#pragma once
#include <cudaTypedefs.h>

#include "dak_device.cuh"

namespace dak {

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
__device__ __forceinline__ void named_bar() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// n / d for n >= 0 and quotients below 2^21 (the float quotient is off by less than one, which the
// remainder puts right), a few instructions where the integer division is dozens.
__device__ __forceinline__ int quotient(int n, int d) {
    const int q = static_cast<int>(static_cast<float>(n) * __fdividef(1.f, static_cast<float>(d))), r = n - q * d;
    return q + (r >= d) - (r < 0);
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

// The keys of a step from n on.
struct KeysFrom {
    int n;
    __device__ __forceinline__ bool any() const { return n < 64; }
    __device__ __forceinline__ bool operator()(int k) const { return k >= n; }
};

// One step of a row: its 64 scores (those of `hidden` keys do not count) into P in PARTS bf16 parts, over them, with
// the row's running sum and the reference that its exponents are taken against (log2 domain). `grown`
// is called when a row of the warp outgrows its reference, with the factor for O.
template <int PARTS, class Hidden, class Grown>
__device__ __forceinline__ void softmax_step(uint32_t s_addr, const Hidden& hidden, float scale_log2, float& m_ref, float& l, bool first,
                                             const Grown& grown) {
    // with three parts O is in registers too, which leaves none for all scores: they are read twice
    constexpr bool TWICE = PARTS == 3;
    float v[TWICE ? 1 : 4][16];
    const auto mask = [&](int q) {
        if (hidden.any()) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (hidden(q * 16 + k)) v[TWICE ? 0 : q][k] = -INFINITY;
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
    __device__ __forceinline__ void skip(int by) {
        const int to = slot + by;
        phase ^= static_cast<uint32_t>(to / NS) & 1u;
        slot = to % NS;
    }
    __device__ __forceinline__ void advance(int by) {  // by < NS
        slot += by;
        if (slot >= NS) {
            slot -= NS;
            phase ^= 1u;
        }
    }
};

template <int D>
struct ChunkCfg {
    static constexpr int kTileBytes = 128 * D * 2;  // one Q tile
    static constexpr int kStage = 2 * 64 * D * 2;   // a chunk: per half row, K's 64 rows and then V's
    static constexpr int kV = 64 * 128;             // V behind K
    static constexpr int kStages = (224 * 1024 - 2 * kTileBytes) / kStage;
    // copies of a CTA that have not landed yet: enough for the memory system's latency; more only
    // queue in it and hold up everything else that comes that way
    static constexpr int kInFlight = 96 * 1024 / kStage;
    static constexpr int kSmem = 2 * kTileBytes + kStages * kStage + 1024;
};

// The chunks of one tier as the kernels copy them: (64 elements, 64 tokens, K and V, chunk, half of a
// row).
inline bool make_chunk_map(CUtensorMap* map, const void* base, int64_t chunks, int D) {
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

}  // namespace dak
