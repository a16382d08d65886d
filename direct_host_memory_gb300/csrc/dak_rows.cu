// Rows of a placed KV cache moved as a whole: the accepted path of a tree of drafted tokens
// (dak_kv_commit) and requests that take over the rows of others (dak_kv_fork). Layout and tiers:
// dak_attn.cu.
#include <algorithm>
#include <climits>

#include "dak_device.cuh"

namespace dak {

// A slab's address in whichever tier holds it.
struct Tiers {
    uint8_t* host;
    uint8_t* hbm;
    long long head_bytes;
    int h_s;
    __device__ __forceinline__ uint8_t* slab(long long s) const {
        return s < h_s ? host + s * head_bytes : hbm + (s - h_s) * head_bytes;
    }
};

static Tiers tiers_of(const dak_placement* p) {
    return {static_cast<uint8_t*>(p->host_dev), static_cast<uint8_t*>(p->hbm_ptr), p->head_bytes, p->h_s};
}

// ------------------------------------------------------------------------------------
// commit
// ------------------------------------------------------------------------------------
struct CommitParams {
    Tiers kv;
    const int* lens;
    const int* n_new;
    const int* path;
    const int* n_path;
    int* lens_out;
    int* slot_pos;
    float* acc;
    int T, P, Hkv, L;
    DevStatus* st;
};


// One block per slab, a thread per 16-byte piece of up to eight rows of K or V. A path ascends, so that
// path[i] >= i: no row is written before the rows after it in the path have been read, if every
// group of rows is read whole before it is written, and groups are taken in order. What a block waits
// for are loads one after the other, the path and then the rows, which more slabs at once cover: with 64
// threads 18 blocks fit an SM (256 requests of 8 kv heads, up to 48 of 64 drafts, tables: 12.1 us, 55 MB
// of rows read and written in 8.2 at the copy rate; 13.3 with 128 threads, 17.4 with 256 and the tables behind
// the rows; four rows a thread 13.4). Where slabs are few enough for blocks of 256 to be there at once, and
// paths long, those have fewer groups to take one after the other (up to 83 of 88 drafts of one request and 2 kv
// heads 3.1 us, 7.9 with 64 threads).
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) commit_kernel(const CommitParams p) {
    constexpr int PIECES = 2 * (D / 8);                // of a row's K and V
    constexpr int LANES = THREADS / PIECES;     // rows side by side
    constexpr int PER = 8;
    constexpr int MORE = (DAK_MAX_TREE + THREADS - 1) / THREADS;  // drafts of a thread
    __shared__ int path[DAK_MAX_TREE];
    const int tid = threadIdx.x, b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv;
    const long long slab = blockIdx.x;
    grid_dep_wait();  // launched while the previous kernel ends
    const int* in = p.path + static_cast<long long>(b) * p.P;
    int v[MORE], before[MORE];
#pragma unroll
    for (int k = 0; k < MORE; ++k) {
        const int i = tid + k * THREADS;
        v[k] = i < p.P ? in[i] : 0;
        before[k] = i > 0 && i < p.P ? in[i - 1] : -1;
    }
    const int base = min(max(p.lens[b], 0), p.L), n_new = p.n_new ? min(max(p.n_new[b], 0), p.T) : p.T;
    const int drafts = min(n_new, p.L - base);
    int n = min(max(p.n_path[b], 0), p.P);
    bool good = true;
#pragma unroll
    for (int k = 0; k < MORE; ++k) {
        const int i = tid + k * THREADS;
        if (i >= n) continue;
        path[i] = v[k];
        good = good && v[k] >= 0 && v[k] > before[k] && v[k] < drafts;
    }
    if (!__syncthreads_and(good)) {
        if (g == 0 && tid == 0) report(p.st, DAK_ERR_BOUNDS, (0xC0113ull << 32) | static_cast<unsigned>(b));
        n = 0;
    }
    if (g == 0 && tid == 0) p.lens_out[b] = base + n;
    int* pos = p.slot_pos ? p.slot_pos + slab * p.L + base : nullptr;
    float* acc = p.acc ? p.acc + slab * p.L + base : nullptr;
    int pv[MORE];
    float av[MORE];
#pragma unroll
    for (int k = 0; k < MORE; ++k) {
        const int i = tid + k * THREADS;
        pv[k] = pos && i < n ? pos[path[i]] : -1;
        av[k] = acc && i < n ? acc[path[i]] : 0.f;
    }
    uint4* rows = reinterpret_cast<uint4*>(p.kv.slab(slab));
    const int piece = tid % PIECES, kv = piece / (D / 8), c = piece % (D / 8), r0 = tid / PIECES;
    const auto at = [&](int j) -> uint4& {
        return rows[(static_cast<long long>(j >> 6) * 2 + kv) * (8 * D) + (j & 63) * (D / 8) + (c ^ (j & 7))];
    };
    for (int i0 = 0; i0 < n; i0 += LANES * PER) {
        uint4 x[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * LANES + r0;
            if (i < n && path[i] != i) x[k] = at(base + path[i]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * LANES + r0;
            if (i < n && path[i] != i) at(base + i) = x[k];
        }
    }
    if (!pos && !acc) return;
    __syncthreads();  // entries are all read
#pragma unroll
    for (int k = 0; k < MORE; ++k) {
        const int i = tid + k * THREADS;
        if (i >= drafts) continue;
        if (pos) pos[i] = pv[k];
        if (acc) acc[i] = av[k];
    }
}

// ------------------------------------------------------------------------------------
// fork
// ------------------------------------------------------------------------------------
struct ForkParams {
    Tiers to, from;
    const int* src_of;
    const int* lens;
    const int* first;
    int* lens_out;
    const int* src_pos;
    int* pos;
    const float* src_acc;
    float* acc;
    int B, L, src_B, src_L, Hkv;
    int same;   // src is KV
    int stage;  // bytes of one of the two staging buffers
    DevStatus* st;
};

constexpr int kForkThreads = 256;
constexpr int kForkMax = DAK_MAX_FORK;

__device__ __forceinline__ void copy_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A unit's stretch in one request: where it begins, which of its 16-byte pieces are wanted, and (of a
// taker) where in the staging buffer its source's stretch lies.
struct __align__(16) ForkStretch {
    uint8_t* at;
    int pieces;  // first | end << 16
    int from;
};

// Every request that others go on from is a source, with a place in the staging buffers. A unit is the
// same stretch of bytes (a power of two, at most 64 rows of K or V, as many as fit in a buffer
// for all sources) of one chunk and kv head: it is read from every source, and once all have arrived
// written to every taker. No other unit reads or writes these bytes of any request, so that any map can
// be taken in place, and a source is read once however many take from it. Two buffers: a unit's bytes
// are on their way while the one before is written. What bounds it: bytes (16 samples of two prompts over 7K:
// 560 MB, 92.5 us, 81 at the copy rate); with many requests of many lengths the lists (about 4 us) and
// units of few pieces (any of 61 over up to 3000 tracked rows 34.8 us, 22 at the copy rate, 3 of them for
// the tables; all of 3001 rows 57.5, 45); a few beams the lists, one unit's way in and out: 7.5 us.
template <int D>
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int n_src, n_take, lowest, highest;
    uint8_t* buffer = smem;
    ForkStretch* read_at = reinterpret_cast<ForkStretch*>(smem + 2 * p.stage);  // of each source, of the next unit
    ForkStretch* write_at = read_at + p.src_B;                                  // of each taker, of this unit
    int* slot_of = reinterpret_cast<int*>(write_at + p.B);
    int* src_f = slot_of + p.src_B;    // of each source: request, rows wanted
    int* src_lo = src_f + p.src_B;
    int* src_n = src_lo + p.src_B;
    int* take_b = src_n + p.src_B;     // of each taker: request, its source's place, first row
    int* take_slot = take_b + p.B;
    int* take_lo = take_slot + p.B;
    const int tid = threadIdx.x;
    if (tid == 0) n_src = n_take = 0, lowest = INT_MAX, highest = 0;
    for (int f = tid; f < p.src_B; f += kForkThreads) src_lo[f] = INT_MAX;  // for now by request
    grid_dep_wait();  // launched while the previous kernel ends
    __syncthreads();
    for (int b = tid; b < p.B; b += kForkThreads) {
        const int f = p.src_of[b];
        const bool known = f >= 0 && f < p.src_B, takes = known && !(p.same && f == b);
        int n = 0, lo = 0;
        if (known) {
            n = min(max(p.lens[f], 0), p.src_L);
            if (n > p.L) {
                if (blockIdx.x == 0) report(p.st, DAK_ERR_BOUNDS, (0xF02Cull << 32) | static_cast<unsigned>(b));
                n = p.L;
            }
            lo = p.first ? min(max(p.first[b], 0), n) : 0;
        } else if (f >= p.src_B && blockIdx.x == 0) {
            report(p.st, DAK_ERR_BOUNDS, (0xF02Dull << 32) | static_cast<unsigned>(b));
        }
        if (blockIdx.x == 0) {
            if (takes) p.lens_out[b] = n;
            else if (p.same) p.lens_out[b] = min(max(p.lens[b], 0), p.L);
        }
        if (takes && lo < n) {
            const int k = atomicAdd(&n_take, 1);
            take_b[k] = b;
            take_slot[k] = f;  // for now the request
            take_lo[k] = lo;
            atomicMin(&src_lo[f], lo);
            atomicMin(&lowest, lo);
            atomicMax(&highest, n);
        }
    }
    __syncthreads();
    const int takers = n_take;
    if (takers == 0) return;
    for (int f = tid; f < p.src_B; f += kForkThreads) {
        slot_of[f] = src_lo[f] < INT_MAX ? atomicAdd(&n_src, 1) : -1;
    }
    __syncthreads();
    const int sources = n_src;
    // the lists by place; src_lo is read by request before it is written by place
    for (int f0 = 0; f0 < p.src_B; f0 += kForkThreads) {
        const int f = f0 + tid;
        const bool in = f < p.src_B && slot_of[f] >= 0;
        if (in) {
            src_f[slot_of[f]] = f;
            src_n[slot_of[f]] = min(min(max(p.lens[f], 0), p.src_L), p.L);
        }
    }
    for (int k = tid; k < takers; k += kForkThreads) take_slot[k] = slot_of[take_slot[k]];
    __syncthreads();
    for (int s = tid; s < sources; s += kForkThreads) slot_of[s] = src_lo[src_f[s]];
    __syncthreads();
    const int* lo_of = slot_of;  // by place from here on

    constexpr int kRow = 2 * D;          // bytes of a row of K or V
    constexpr int kHalf = 64 * kRow;     // of a chunk's K or V
    int unit = kHalf;
    while (unit > 16 && unit * sources > p.stage) unit >>= 1;
    const long long halves = (((highest + 63) >> 6) - (lowest >> 6)) * 2ll * p.Hkv;
    // smaller ones where the SMs would not all have one (62 requests from one of 560 rows, 2 kv heads: 9.6 us, 24.2)
    while (unit > 512 && halves * (kHalf / unit) < gridDim.x) unit >>= 1;
    const int shift = 31 - __clz(unit >> 4);  // pieces of 16 bytes of a unit: 1 << shift
    const int subs = kHalf / unit, sub_shift = 31 - __clz(subs), c0 = lowest >> 6;
    const long long n_units = halves << sub_shift;
    // Unit x, stretches of one slab side by side: kv head, offset in the slab, and the rows lo .. n - 1 of
    // one request as pieces of it.
    const auto stretch = [&](long long x, const Tiers& tiers, int request, int lo, int n, int from) {
        const int in_half = static_cast<int>(x & (subs - 1)) * unit, kv = static_cast<int>(x >> sub_shift) & 1;
        const int y = static_cast<int>(x >> (sub_shift + 1)), c = y / p.Hkv, g = y - c * p.Hkv, row0 = (c0 + c) * 64;
        // of the half's pieces, and of this stretch's
        const int first = max(min(max(lo - row0, 0) * (kRow / 16) - in_half / 16, 1 << shift), 0);
        const int end = max(min(min(n - row0, 64) * (kRow / 16) - in_half / 16, 1 << shift), 0);
        ForkStretch at;
        at.at = tiers.slab(static_cast<long long>(request) * p.Hkv + g) + (static_cast<long long>(c0 + c) * 2 + kv) * kHalf + in_half;
        at.pieces = first | end << 16;
        at.from = from;
        return at;
    };
    const auto sources_of = [&](long long x) {
        for (int s = tid; s < sources; s += kForkThreads) read_at[s] = stretch(x, p.from, src_f[s], lo_of[s], src_n[s], s * unit);
    };
    const auto read = [&](uint8_t* to) {
        for (int e = tid; e < sources << shift; e += kForkThreads) {
            const ForkStretch from = read_at[e >> shift];
            const int k = e & ((1 << shift) - 1);
            if (k >= (from.pieces & 0xFFFF) && k < from.pieces >> 16) copy_async16(to + from.from + (k << 4), from.at + (k << 4));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    long long x = blockIdx.x;
    if (x < n_units) sources_of(x);
    __syncthreads();
    if (x < n_units) read(buffer);
    __syncthreads();
    if (x + gridDim.x < n_units) sources_of(x + gridDim.x);
    for (int k = 0; x < n_units; x += gridDim.x, k ^= 1) {
        __syncthreads();  // the other buffer is free, the next stretches are known
        if (x + gridDim.x < n_units) read(buffer + (k ^ 1) * p.stage);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        for (int t = tid; t < takers; t += kForkThreads) {
            write_at[t] = stretch(x, p.to, take_b[t], take_lo[t], src_n[take_slot[t]], take_slot[t] * unit);
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const uint8_t* from = buffer + k * p.stage;
#pragma unroll 4
        for (int e = tid; e < takers << shift; e += kForkThreads) {
            const ForkStretch to = write_at[e >> shift];
            const int i = e & ((1 << shift) - 1);
            if (i >= (to.pieces & 0xFFFF) && i < to.pieces >> 16) {
                *reinterpret_cast<uint4*>(to.at + (i << 4)) = *reinterpret_cast<const uint4*>(from + to.from + (i << 4));
            }
        }
        if (x + 2ll * gridDim.x < n_units) sources_of(x + 2ll * gridDim.x);
    }
    __syncthreads();
    if (!p.pos && !p.acc) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the tables likewise, a word of each a row; short stretches, so that every CTA has some
    int rows = 256;
    while (rows > 32 && (rows * sources * 8 > 2 * p.stage || (highest - lowest) / rows * p.Hkv < static_cast<int>(gridDim.x))) rows >>= 1;
    while (rows > 1 && rows * sources * 8 > 2 * p.stage) rows >>= 1;
    const int lg = 31 - __clz(rows), blocks = (highest - lowest + rows - 1) / rows;
    int* hold_pos = reinterpret_cast<int*>(buffer);
    float* hold_acc = reinterpret_cast<float*>(hold_pos + rows * sources);
    const long long from_x = (blockIdx.x + gridDim.x - n_units % gridDim.x) % gridDim.x;  // on where the units ended
    for (long long y = from_x; y < static_cast<long long>(blocks) * p.Hkv; y += gridDim.x) {
        const int g = static_cast<int>(y % p.Hkv), j0 = lowest + static_cast<int>(y / p.Hkv) * rows;
        for (int e = tid; e < sources << lg; e += kForkThreads) {
            const int s = e >> lg, j = j0 + (e & (rows - 1));
            if (j < lo_of[s] || j >= src_n[s]) continue;
            const long long at = (static_cast<long long>(src_f[s]) * p.Hkv + g) * p.src_L + j;
            if (p.pos) copy_async4(&hold_pos[e], &p.src_pos[at]);
            if (p.acc) copy_async4(&hold_acc[e], &p.src_acc[at]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll 4
        for (int e = tid; e < takers << lg; e += kForkThreads) {
            const int t = e >> lg, r = e & (rows - 1), j = j0 + r, s = take_slot[t];
            if (j < take_lo[t] || j >= src_n[s]) continue;
            const long long at = (static_cast<long long>(take_b[t]) * p.Hkv + g) * p.L + j;
            if (p.pos) p.pos[at] = hold_pos[(s << lg) + r];
            if (p.acc) p.acc[at] = hold_acc[(s << lg) + r];
        }
        __syncthreads();
    }
}

static int fork_plan_bytes(int B, int src_B) {
    return (src_B + B) * static_cast<int>(sizeof(ForkStretch)) + (4 * src_B + 3 * B) * static_cast<int>(sizeof(int));
}

template <int D>
static cudaError_t launch_fork(ForkParams& p, cudaStream_t s) {
    // Three CTAs an SM, or two or one where the lists take more room (16 beams of 8 kv heads over 850 rows 7.5 us with
    // three, 8.6 with two; 16 samples of two prompts over 7K 91, 95, with four 98; any of 61 requests over up
    // to 3000 tracked rows 34.8, 35.5, 34.5).
    constexpr int kMost = 3, kRoom[kMost] = {220 * 1024, 110 * 1024, 73 * 1024};  // by CTAs an SM, from one on
    const int plan = fork_plan_bytes(p.B, p.src_B);
    const int least = std::max(16 * 1024, 16 * p.src_B);
    int per_sm = kMost;
    while (per_sm > 1 && plan + 2 * least > kRoom[per_sm - 1]) --per_sm;
    p.stage = (kRoom[per_sm - 1] - plan) / 2 / 128 * 128;
    const int smem = 2 * p.stage + plan;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(fork_kernel<D>), kRoom[0]);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(per_sm * device_sm_count()));
    cfg.blockDim = dim3(kForkThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fork_kernel<D>, p);
}

}  // namespace dak

using namespace dak;

extern "C" dak_status dak_kv_commit(const dak_placement* KV, const int* seq_lens, int T, const int* n_new, const int* path,
                                    int P, const int* n_path, int* lens_out, int* slot_pos, float* acc, void* stream) {
    if (!KV || KV->kind != 1 || !seq_lens || !path || !n_path || !lens_out || T < 1 || P < 1 || P > T) return DAK_ERR_INVALID;
    if (T > DAK_MAX_TREE) return DAK_ERR_UNSUPPORTED;
    if (misaligned(seq_lens, 4) || misaligned(n_new, 4) || misaligned(path, 4) || misaligned(n_path, 4) || misaligned(lens_out, 4) || misaligned(slot_pos, 4) || misaligned(acc, 4)) {
        return DAK_ERR_ALIGN;
    }
    const size_t lens = static_cast<size_t>(KV->B) * 4;
    if (ranges_overlap(lens_out, lens, seq_lens, lens) || ranges_overlap(lens_out, lens, n_new, lens) || ranges_overlap(lens_out, lens, n_path, lens) ||
        ranges_overlap(lens_out, lens, path, lens * P)) {
        return DAK_ERR_INVALID;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DAK_ERR_CUDA;
    if (dev != KV->device) return DAK_ERR_INVALID;
    CommitParams p{};
    p.kv = tiers_of(KV);
    p.lens = seq_lens;
    p.n_new = n_new;
    p.path = path;
    p.n_path = n_path;
    p.lens_out = lens_out;
    p.slot_pos = slot_pos;
    p.acc = acc;
    p.T = T;
    p.P = P;
    p.Hkv = KV->H_kv;
    p.L = KV->L;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    const int64_t slabs = static_cast<int64_t>(KV->B) * KV->H_kv;
    const bool wide = P > 16 && slabs <= 4 * device_sm_count();  // wide blocks of all slabs are there at once
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(slabs));
    cfg.blockDim = dim3(wide ? 256 : 64);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (wide) {
        return cuda_status(KV->D == 128 ? cudaLaunchKernelEx(&cfg, commit_kernel<128, 256>, p)
                                        : cudaLaunchKernelEx(&cfg, commit_kernel<64, 256>, p));
    }
    return cuda_status(KV->D == 128 ? cudaLaunchKernelEx(&cfg, commit_kernel<128, 64>, p)
                                    : cudaLaunchKernelEx(&cfg, commit_kernel<64, 64>, p));
}

extern "C" dak_status dak_kv_fork(const dak_placement* KV, const dak_placement* src, const int* src_of, const int* seq_lens,
                                  const int* first, int* lens_out, const int* src_slot_pos, int* slot_pos,
                                  const float* src_acc, float* acc, void* stream) {
    if (!KV || KV->kind != 1 || !src || src->kind != 1 || !src_of || !seq_lens || !lens_out) return DAK_ERR_INVALID;
    if (src->H_kv != KV->H_kv || src->D != KV->D || src->device != KV->device) return DAK_ERR_INVALID;
    if (KV->B > kForkMax || src->B > kForkMax) return DAK_ERR_UNSUPPORTED;
    if (!slot_pos != !src_slot_pos || !acc != !src_acc) return DAK_ERR_INVALID;
    if (misaligned(src_of, 4) || misaligned(seq_lens, 4) || misaligned(first, 4) || misaligned(lens_out, 4) || misaligned(src_slot_pos, 4) || misaligned(slot_pos, 4) ||
        misaligned(src_acc, 4) || misaligned(acc, 4)) {
        return DAK_ERR_ALIGN;
    }
    const size_t lens = static_cast<size_t>(KV->B) * 4, src_lens = static_cast<size_t>(src->B) * 4;
    if (ranges_overlap(lens_out, lens, src_of, lens) || ranges_overlap(lens_out, lens, first, lens) || ranges_overlap(lens_out, lens, seq_lens, src_lens)) {
        return DAK_ERR_INVALID;
    }
    if (src == KV) {
        if (slot_pos != src_slot_pos || acc != src_acc) return DAK_ERR_INVALID;
    } else {
        const size_t to = lens * KV->H_kv * KV->L, from = src_lens * src->H_kv * src->L;
        if (ranges_overlap(slot_pos, to, src_slot_pos, from) || ranges_overlap(acc, to, src_acc, from)) return DAK_ERR_INVALID;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DAK_ERR_CUDA;
    if (dev != KV->device) return DAK_ERR_INVALID;
    ForkParams p{};
    p.to = tiers_of(KV);
    p.from = tiers_of(src);
    p.src_of = src_of;
    p.lens = seq_lens;
    p.first = first;
    p.lens_out = lens_out;
    p.src_pos = src_slot_pos;
    p.pos = slot_pos;
    p.src_acc = src_acc;
    p.acc = acc;
    p.B = KV->B;
    p.L = KV->L;
    p.src_B = src->B;
    p.src_L = src->L;
    p.Hkv = KV->H_kv;
    p.same = src == KV;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(KV->D == 128 ? launch_fork<128>(p, s) : launch_fork<64>(p, s));
}
