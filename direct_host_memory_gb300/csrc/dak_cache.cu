// What changes the contents of a placed KV cache between attention calls: new tokens rotated
// and appended (dak_kv_append_rope), and the least attended tokens evicted (dak_kv_evict).
// The cache layout is the one of dak_attn.cu: a (request, kv head) slab is ceil(L/64) chunks
// [K 64 x D][V 64 x D] bf16, the 16-byte piece c of token t's row stored at c ^ (t & 7).
#include <algorithm>
#include <climits>
#include <cmath>

#include "dak_device.cuh"

namespace dak {

// ------------------------------------------------------------------------------------
// rotation and append
// ------------------------------------------------------------------------------------
struct RopeParams {
    dak_rope_plan rope;
    const void* q;
    const void* k;
    const void* v;
    long long q_pitch, k_pitch, v_pitch;  // elements from token to token
    const int* slots;
    const int* positions;
    const int* n_new;
    __nv_bfloat16* q_out;
    int* slot_pos;
    float* acc;
    uint8_t* host;
    uint8_t* hbm;
    long long head_bytes;
    int T, Hq, Hkv, L, h_s;
    DevStatus* st;
};

constexpr int kRopeThreads = 128;

template <bool F32>
__device__ __forceinline__ float load_elem(const void* p, long long i) {
    if (F32) return static_cast<const float*>(p)[i];
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Eight consecutive elements at i as they lie in memory (16-byte aligned), and as fp32.
template <bool F32>
struct Piece;
template <>
struct Piece<false> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p, long long i) {
        v = ld_nc_v4(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
        x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
    }
};
template <>
struct Piece<true> {
    uint4 v[2];
    __device__ __forceinline__ void load(const void* p, long long i) {
        v[0] = ld_nc_v4(static_cast<const float*>(p) + i);
        v[1] = ld_nc_v4(static_cast<const float*>(p) + i + 4);
    }
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            x[4 * k] = __uint_as_float(v[k].x), x[4 * k + 1] = __uint_as_float(v[k].y);
            x[4 * k + 2] = __uint_as_float(v[k].z), x[4 * k + 3] = __uint_as_float(v[k].w);
        }
    }
};

__device__ __forceinline__ uint4 pack8(const float* y) {
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}

// One block per token (or a share of its heads, where tokens are few). A thread's unit is a pair of
// 16-byte output pieces: of a query or key head the two that hold the same pairs' halves, or where
// pairs do not lie so (interleaved, a share of pieces that turn, halves not of whole pieces) and in
// value heads two pieces side by side. Its inputs are asked for first; the position, its angles and
// the table of cos and sin come under those loads. Position x turns modulo 2^64 is the angle as a
// binary fraction of a turn, without a rounding (turns itself is good to f_i * 2^-55, so the angle to
// 2^-35 turns at position 10^6 and 2^-24 at 2^31); its upper 32 bits, signed, are half-turns * 2^-31. Products and sums in fp32, one rounding to bf16 at the store. Memory bound: every element is
// read and written once (8192 tokens of 32 query and 8 kv heads, D 128, bf16: 33.7 us, 5.4 TB/s; with a
// thread a piece, and its pair's other half by a load of its own, 48 us); a few tokens are bound by the
// launch (1 token 2.9 us, 256 tokens fp32 4.5 us).
enum { kRopeSplit = 0, kRopeInterleaved = 1, kRopePart = 2 };  // PART: halves of a part of the head

template <int D, bool F32, int KIND>
__global__ void __launch_bounds__(kRopeThreads, F32 ? 6 : 8) append_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int PAIRS = D / 16;  // units of a head
    constexpr int PER = 3;         // units in flight per thread (a token of the 8B shape: all of them)
    __shared__ float2 cs[D / 2];
    const int b = blockIdx.x / p.T, t = blockIdx.x - b * p.T;
    const long long token = blockIdx.x;
    const int R = p.rope.rot_dim, half = R / 2;
    const int heads = p.Hq + 2 * p.Hkv, n_units = heads * PAIRS, stride = gridDim.y * kRopeThreads;
    grid_dep_wait();  // launched while the previous kernel ends
    const int n_new = p.n_new ? p.n_new[b] : p.T, slot = p.slots[b], first = p.positions ? p.positions[b] : slot;
    bool ready = false, in_range = false;
    long long row = 0, pos = 0;
    for (int u0 = blockIdx.y * kRopeThreads + threadIdx.x; u0 - static_cast<int>(threadIdx.x) < n_units; u0 += PER * stride) {
        Piece<F32> raw[PER][2];
        // unit u: its head, where its pieces begin in it
        const auto place = [&](int u, int& h, int& e0, int& e1, bool& is_q, bool& is_v, int& g) {
            h = u / PAIRS;
            is_q = h < p.Hq;
            is_v = h >= p.Hq + p.Hkv;
            g = is_q ? h : is_v ? h - p.Hq - p.Hkv : h - p.Hq;
            const int c = u - h * PAIRS;
            const bool apart = KIND == kRopeSplit && !is_v;
            e0 = apart ? c * 8 : c * 16;
            e1 = apart ? e0 + D / 2 : e0 + 8;
        };
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int u = u0 + k * stride;
            if (u >= n_units) continue;
            int h, e0, e1, g;
            bool is_q, is_v;
            place(u, h, e0, e1, is_q, is_v, g);
            const void* src = is_q ? p.q : is_v ? p.v : p.k;
            const long long at = token * (is_q ? p.q_pitch : is_v ? p.v_pitch : p.k_pitch) + static_cast<long long>(g) * D;
            raw[k][0].load(src, at + e0);
            raw[k][1].load(src, at + e1);
        }
        if (!ready) {
            if (t >= n_new) return;
            row = static_cast<long long>(slot) + t;
            pos = static_cast<long long>(first) + t;
            in_range = row >= 0 && row < p.L;
            if (static_cast<int>(threadIdx.x) < half) {
                const uint64_t turn = static_cast<uint64_t>(pos) * p.rope.turns[threadIdx.x];
                const float a = static_cast<float>(static_cast<int>(static_cast<uint32_t>(turn >> 32))) * 0x1p-31f;
                float s, c;
                sincospif(a, &s, &c);
                cs[threadIdx.x] = make_float2(c * p.rope.scale, s * p.rope.scale);
            }
            if (!in_range && blockIdx.y == 0 && threadIdx.x == 0) {
                report(p.st, DAK_ERR_BOUNDS, 0xA9901000ull << 32 | static_cast<unsigned>(b));
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int u = u0 + k * stride;
            if (u >= n_units) continue;
            int h, e0, e1, g;
            bool is_q, is_v;
            place(u, h, e0, e1, is_q, is_v, g);
            if (!is_q && !in_range) continue;
            float x[16];
            raw[k][0].get(x);
            raw[k][1].get(x + 8);
            if (!is_v) {
                if (KIND == kRopeSplit) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = cs[e0 + i];
                        const float a = x[i], c = x[8 + i];
                        x[i] = a * f.x - c * f.y;
                        x[8 + i] = c * f.x + a * f.y;
                    }
                } else if (KIND == kRopeInterleaved) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        if (e0 + i >= R) continue;
                        const float2 f = cs[(e0 + i) >> 1];
                        const float a = x[i], c = x[i + 1];
                        x[i] = a * f.x - c * f.y;
                        x[i + 1] = c * f.x + a * f.y;
                    }
                } else {  // a pair's other half by a load of its own
                    const void* src = is_q ? p.q : p.k;
                    const long long at = token * (is_q ? p.q_pitch : p.k_pitch) + static_cast<long long>(g) * D;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = e0 + i;
                        if (e >= R) continue;
                        const float2 f = cs[e < half ? e : e - half];
                        const float o = load_elem<F32>(src, at + (e < half ? e + half : e - half));
                        x[i] = x[i] * f.x + (e < half ? -o : o) * f.y;
                    }
                }
            }
            const uint4 y0 = pack8(x), y1 = pack8(x + 8);
            if (is_q) {
                __nv_bfloat16* out = p.q_out + (token * p.Hq + h) * D;
                *reinterpret_cast<uint4*>(out + e0) = y0;
                *reinterpret_cast<uint4*>(out + e1) = y1;
            } else {
                const long long slab = static_cast<long long>(b) * p.Hkv + g;
                uint4* base =
                    reinterpret_cast<uint4*>(slab < p.h_s ? p.host + slab * p.head_bytes : p.hbm + (slab - p.h_s) * p.head_bytes);
                base += (row >> 6) * (16 * D) + (is_v ? 8 * D : 0) + (row & 63) * (D / 8);
                base[(e0 >> 3) ^ (row & 7)] = y0;
                base[(e1 >> 3) ^ (row & 7)] = y1;
                if (!is_v && e0 == 0) {
                    if (p.slot_pos) p.slot_pos[slab * p.L + row] = static_cast<int>(pos);
                    if (p.acc) p.acc[slab * p.L + row] = 0.f;
                }
            }
        }
    }
}

template <int D, bool F32>
static cudaError_t launch_append_rope(const RopeParams& p, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.rope.interleaved) return cudaLaunchKernelEx(&cfg, append_rope_kernel<D, F32, kRopeInterleaved>, p);
    if (p.rope.rot_dim == D) return cudaLaunchKernelEx(&cfg, append_rope_kernel<D, F32, kRopeSplit>, p);
    return cudaLaunchKernelEx(&cfg, append_rope_kernel<D, F32, kRopePart>, p);
}

// ------------------------------------------------------------------------------------
// eviction
// ------------------------------------------------------------------------------------
struct EvictParams {
    const int* seq_lens;
    const float* acc;
    float* acc_out;
    const int* pos;
    int* pos_out;
    int* lens_out;
    int* src_out;
    int* moves;   // [slabs][2][list]: the holes and the movers of each slab, in ascending order
    int* n_moves; // [slabs]
    int list;     // longest list: min(n_keep, L - n_keep)
    int Hkv, L, n_keep, n_recent;
    uint8_t* host;
    uint8_t* hbm;
    long long head_bytes;
    int h_s;
};

constexpr int kEvictThreads = 512;
constexpr int kMoveThreads = 256;

// Order of eviction as an unsigned key: protected slots highest, then the weight, NaN lowest;
// -0 equals +0.
__device__ __forceinline__ uint32_t evict_key(float w, bool newest) {
    if (newest) return 0xFFFFFFFFu;
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

// Caches longer than a cluster's registers hold (kEvictMaxSlots): one block per slab that reads the
// tables again for every pass (8 slabs of 131K slots so: 1.14 ms; by clusters: 78 us). The n_keep-th largest key by a radix select over bytes, then one
// pass over the slots in order that gives every slot its fate and every hole and mover its rank.
__global__ void __launch_bounds__(kEvictThreads) evict_select_long_kernel(const EvictParams p) {
    constexpr int NW = kEvictThreads / 32;
    __shared__ int hist[256];
    __shared__ int red[NW];
    __shared__ int sh_a, sh_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long slab = blockIdx.x;
    const int b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv;
    const int n = min(max(p.seq_lens[b], 0), p.L), keep = p.n_keep;
    const float* acc = p.acc + slab * p.L;
    const int* pos = p.pos + slab * p.L;
    float* acc_out = p.acc_out + slab * p.L;
    int* pos_out = p.pos_out + slab * p.L;
    int* src = p.src_out ? p.src_out + slab * keep : nullptr;
    const bool copy = p.acc_out != p.acc, copy_pos = p.pos_out != p.pos;
    if (g == 0 && tid == 0) p.lens_out[b] = min(n, keep);
    if (n <= keep) {
        for (int i = tid; i < n; i += kEvictThreads) {
            if (copy) acc_out[i] = acc[i];
            if (copy_pos) pos_out[i] = pos[i];
        }
        if (src) {
            for (int i = tid; i < keep; i += kEvictThreads) src[i] = i < n ? i : -1;
        }
        if (tid == 0) p.n_moves[slab] = 0;
        return;
    }
    // newest position
    int m = INT_MIN;
    for (int i = tid; i < n; i += kEvictThreads) m = max(m, pos[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = red[0];
    for (int w = 1; w < NW; ++w) m = max(m, red[w]);
    const long long oldest = static_cast<long long>(m) - p.n_recent;  // newer than this: protected
    // the keep-th largest key, a byte at a time from the top: prefix = its leading bytes,
    // want = how many of the keys that share them are kept
    uint32_t prefix = 0;
    int want = keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kEvictThreads) {
            const uint32_t k = evict_key(acc[i], pos[i] > oldest);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = want, d = 255;
            while (d > 0 && hist[d] < left) left -= hist[d--];
            sh_a = d;
            sh_b = left;
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sh_a) << shift;
        want = sh_b;
        __syncthreads();
    }
    // slots in order: above the threshold kept, at it the first `want`
    int eq_seen = 0, n_holes = 0, n_movers = 0;
    int* holes = p.moves + slab * 2 * p.list;
    int* movers = holes + p.list;
    const uint32_t below = (1u << lane) - 1;
    // a block-wide exclusive rank of `mine`, and the tile's count added to `total`
    const auto rank_of = [&](bool mine, int& total) {
        const uint32_t bal = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) red[warp] = __popc(bal);
        __syncthreads();
        int before = total + __popc(bal & below), all = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += red[w];
            all += red[w];
        }
        total += all;
        __syncthreads();
        return before;
    };
    for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < n ? evict_key(acc[i], pos[i] > oldest) : 0u;
        const bool eq = i < n && k == prefix;
        const int at = rank_of(eq, eq_seen);
        const bool kept = i < n && (k > prefix || (eq && at < want));
        const bool hole = i < keep && !kept, mover = i >= keep && kept;
        const int hr = rank_of(hole, n_holes), mr = rank_of(mover, n_movers);
        if (hole) holes[hr] = i;
        if (mover) movers[mr] = i;
        if (kept && i < keep) {
            if (copy) acc_out[i] = acc[i];
            if (copy_pos) pos_out[i] = pos[i];
            if (src) src[i] = i;
        }
    }
    __syncthreads();
    const int cnt = n_holes;  // as many holes as movers
    if (tid == 0) p.n_moves[slab] = cnt;
    for (int r = tid; r < cnt; r += kEvictThreads) {
        const int to = holes[r], from = movers[r];
        acc_out[to] = acc[from];
        pos_out[to] = pos[from];
        if (src) src[to] = from;
    }
    __syncthreads();
    for (int i = keep + tid; i < n; i += kEvictThreads) {
        acc_out[i] = 0.f;
        pos_out[i] = -1;
    }
}

// The moved rows of a slab, K and V, from slots movers[r] to holes[r], by `threads` threads of which
// this is `self`. Every thread has four 16-byte pieces in flight; a row's pieces lie on
// neighbouring threads.
template <int D>
__device__ __forceinline__ void move_rows(const EvictParams& p, long long slab, const int* holes, const int* movers, int cnt,
                                          int self, int threads) {
    constexpr int PIECES = D / 8, PER_ROW = 2 * PIECES;
    uint4* base =
        reinterpret_cast<uint4*>(slab < p.h_s ? p.host + slab * p.head_bytes : p.hbm + (slab - p.h_s) * p.head_bytes);
    const auto piece_of = [](int row, int v, int c) {
        return static_cast<long long>(row >> 6) * (128 * PIECES) + v * 64 * PIECES + (row & 63) * PIECES + (c ^ (row & 7));
    };
    const int q = self % PER_ROW, c = q % PIECES, v = q / PIECES;  // the same piece of every row it takes
    const int step = threads / PER_ROW;
    for (int r0 = self / PER_ROW; r0 < cnt; r0 += 4 * step) {
        uint4 x[4];
        int to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = r0 + k * step;
            to[k] = -1;
            if (r < cnt) {
                to[k] = holes[r];
                x[k] = base[piece_of(movers[r], v, c)];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (to[k] >= 0) base[piece_of(to[k], v, c)] = x[k];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    grid_dep_wait();
    const long long slab = blockIdx.x;
    const int* holes = p.moves + slab * 2 * p.list;
    move_rows<D>(p, slab, holes, holes + p.list, p.n_moves[slab], blockIdx.y * kMoveThreads + threadIdx.x,
                 gridDim.y * kMoveThreads);
}

// The eviction of one slab by a cluster of 1 to 8 CTAs, the slots' keys in registers: CTA c holds slots
// [c, c + 1) * 1024 R, thread t the slots r * 1024 + t of them. Reading the tables costs one pass;
// everything after is counting:
//   newest position -> key of every slot (evict_key) -> the n_keep-th largest key by a radix select
//   (11, 11 and 10 bits, histograms in shared memory, of the whole cluster added up by every CTA) ->
//   kept slots (at the threshold key the lowest ones) -> ranks of holes and movers -> lists, tables,
//   and with MOVE the rows themselves.
// Ranks in slot order: ballots per (r, warp), whose counts are scanned in that order, offset by the
// cluster's earlier CTAs. What one CTA needs of each other one, the lanes of a warp read at once.
// Weights are compared and moved as they are, nothing is rounded. 128 slabs from up to 8192 slots to
// 4096: 55.7 us, of which the rows, D 128, take 38 us (7 TB/s read and written) and what comes before
// them 10 us of latencies; 8 slabs from 131K to 65K: 78 us, the counting 26 us on 64 SMs (their 8 MB of
// tables alone 5 us) and then the rows on all; 128 slabs that each lose a few rows: 7 us, all latency.
constexpr int kClusterThreads = 1024;
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictMaxSlots = kEvictMaxCluster * kClusterThreads * 16;
constexpr int kBins = 2048;

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ int2 ld_cluster2(const int* p, uint32_t rank) {
    int2 v;
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(mapa_shared(smem_u32(p), rank))
                 : "memory");
    return v;
}

template <int D, int R, bool CLUSTER, bool MOVE>
__global__ void __launch_bounds__(kClusterThreads, 1) evict_kernel(const EvictParams p, const int n_cluster) {
    constexpr int NW = kClusterThreads / 32;
    constexpr int ENTRIES = R * NW;  // (r, warp) pairs
    __shared__ __align__(8) int hist[3][kBins];
    __shared__ int cnt[ENTRIES];
    __shared__ int wsum[NW];
    __shared__ int share[4];  // read by the cluster: newest position, equals, holes and movers
    __shared__ int coarse[3][NW];  // read by the cluster: sums of 64 bins, from the top
    __shared__ int pick[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cluster = CLUSTER ? n_cluster : 1, rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
    const long long slab = blockIdx.x / cluster;
    const int b = static_cast<int>(slab / p.Hkv), g = static_cast<int>(slab - static_cast<long long>(b) * p.Hkv);
    grid_dep_wait();  // launched while the previous kernel ends
    const int n = min(max(p.seq_lens[b], 0), p.L), keep = p.n_keep;
    const float* acc = p.acc + slab * p.L;
    const int* pos = p.pos + slab * p.L;
    float* acc_out = p.acc_out + slab * p.L;
    int* pos_out = p.pos_out + slab * p.L;
    int* src = p.src_out ? p.src_out + slab * keep : nullptr;
    const bool copy = p.acc_out != p.acc, copy_pos = p.pos_out != p.pos;
    const int s0 = rank * R * kClusterThreads + tid;  // slot of r: s0 + r * 1024
    const auto sync = [] {
        if (CLUSTER) cluster_sync_all();
        else __syncthreads();
    };
    // the `what` of every CTA of the cluster, CTA c's on lane c
    const auto of_cluster = [&](const int* what, int none) { return lane < cluster ? ld_cluster(what, lane) : none; };
    if (!MOVE) grid_dep_launch();
    if (g == 0 && rank == 0 && tid == 0) p.lens_out[b] = min(n, keep);
    if (n <= keep) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = s0 + r * kClusterThreads;
            if (copy && i < n) acc_out[i] = acc[i];
            if (copy_pos && i < n) pos_out[i] = pos[i];
            if (src && i < keep) src[i] = i < n ? i : -1;
        }
        if (rank == 0 && tid == 0) p.n_moves[slab] = 0;
        return;
    }
    uint32_t key[R];
    {
        float w[R];
        int q[R];
        int newest = INT_MIN;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = s0 + r * kClusterThreads;
            w[r] = i < n ? acc[i] : 0.f;
            q[r] = i < n ? pos[i] : INT_MIN;
            newest = max(newest, q[r]);
        }
        for (int i = tid; i < 3 * kBins; i += kClusterThreads) {
            (&hist[0][0])[i] = 0;
        }
        newest = __reduce_max_sync(0xffffffffu, newest);
        if (lane == 0) wsum[warp] = newest;
        __syncthreads();
        newest = __reduce_max_sync(0xffffffffu, wsum[lane]);
        if (CLUSTER) {
            if (tid == 0) share[0] = newest;
            sync();
            newest = __reduce_max_sync(0xffffffffu, of_cluster(&share[0], INT_MIN));
        }
        // protected: a position above newest - n_recent (which may lie below every int32)
        const bool every = static_cast<long long>(newest) - p.n_recent < INT_MIN;
        const int oldest = every ? INT_MIN : newest - p.n_recent;
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = evict_key(w[r], every || q[r] > oldest);
    }
    uint32_t prefix = 0;  // leading bits of the threshold key
    int want = keep;      // how many of the keys that share them are kept
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (s0 + r * kClusterThreads < n && (pass == 0 || (key[r] >> above) == (prefix >> above))) {
                atomicAdd(&hist[pass][(key[r] >> shift) & digits], 1);
            }
        }
        // thread t: bins 2047 - 2t and 2046 - 2t, so that a scan by thread runs from the top
        __syncthreads();
        const int hi = kBins - 1 - 2 * tid;
        const int c1 = hist[pass][hi], c0 = hist[pass][hi - 1];
        if (CLUSTER) {
            // the warp of bins that the threshold lies in by the cluster's coarse sums, then its bins: all
            // CTAs' 2048 bins by every CTA were three quarters of a pass's time
            const int sum = __reduce_add_sync(0xffffffffu, c1 + c0);
            if (lane == 0) coarse[pass][warp] = sum;
            sync();
            if (warp == 0) {
                const auto scan_from_top = [&](int v) {  // inclusive
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int u = __shfl_up_sync(0xffffffffu, v, o);
                        if (lane >= o) v += u;
                    }
                    return v;
                };
                int v[kEvictMaxCluster], all = 0;
#pragma unroll
                for (int c = 0; c < kEvictMaxCluster; ++c) v[c] = c < cluster ? ld_cluster(&coarse[pass][lane], c) : 0;
#pragma unroll
                for (int c = 0; c < kEvictMaxCluster; ++c) all += v[c];
                const int upto = scan_from_top(all);
                const int at = __ffs(__ballot_sync(0xffffffffu, upto >= want)) - 1;  // its warp
                const int above_it = __shfl_sync(0xffffffffu, upto - all, at);
                const int top = kBins - 1 - 2 * (at * 32 + lane);
                int2 w[kEvictMaxCluster];
#pragma unroll
                for (int c = 0; c < kEvictMaxCluster; ++c) {
                    w[c] = c < cluster ? ld_cluster2(&hist[pass][top - 1], c) : make_int2(0, 0);
                }
                int d1 = 0, d0 = 0;
#pragma unroll
                for (int c = 0; c < kEvictMaxCluster; ++c) {
                    d0 += w[c].x;
                    d1 += w[c].y;
                }
                const int before = above_it + scan_from_top(d1 + d0) - d1 - d0;
                if (before < want && want <= before + d1) {
                    pick[0] = top;
                    pick[1] = want - before;
                    pick[2] = d1;
                } else if (before + d1 < want && want <= before + d1 + d0) {
                    pick[0] = top - 1;
                    pick[1] = want - before - d1;
                    pick[2] = d0;
                }
            }
        } else {
            int incl = c1 + c0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            int before = lane < warp ? wsum[lane] : 0;
            before = __reduce_add_sync(0xffffffffu, before) + incl - c1 - c0;  // keys above this thread's bins
            if (before < want && want <= before + c1) {
                pick[0] = hi;
                pick[1] = want - before;
                pick[2] = c1;
            } else if (before + c1 < want && want <= before + c1 + c0) {
                pick[0] = hi - 1;
                pick[1] = want - before - c1;
                pick[2] = c0;
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(pick[0]) << shift;
        want = pick[1];
    }
    // exclusive scan of cnt over its entries in order; returns the sum
    const auto scan = [&]() {
        int v = tid < ENTRIES ? cnt[tid] : 0, incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        const int mine = wsum[lane];
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
        const int all = __reduce_add_sync(0xffffffffu, mine);
        if (tid < ENTRIES) cnt[tid] = before + incl - v;
        __syncthreads();
        return all;
    };
    const uint32_t below = (1u << lane) - 1;
    uint32_t kept = 0;  // bit r
    if (pick[2] == want) {  // every key at the threshold is kept, as where it is no other's
#pragma unroll
        for (int r = 0; r < R; ++r) {
            kept |= static_cast<uint32_t>(s0 + r * kClusterThreads < n && key[r] >= prefix) << r;
        }
    } else {  // the lowest `want` of them
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t bal = __ballot_sync(0xffffffffu, s0 + r * kClusterThreads < n && key[r] == prefix);
            if (lane == 0) cnt[r * NW + warp] = __popc(bal);
        }
        __syncthreads();
        const int all = scan();
        int eq_before = 0;
        if (CLUSTER) {
            if (tid == 0) share[1] = all;
            sync();
            const int v = of_cluster(&share[1], 0);
            eq_before = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = s0 + r * kClusterThreads < n, eq = in && key[r] == prefix;
            const uint32_t bal = __ballot_sync(0xffffffffu, eq);
            bool k = in && key[r] > prefix;
            if (bal && eq) k = eq_before + cnt[r * NW + warp] + __popc(bal & below) < want;
            kept |= static_cast<uint32_t>(k) << r;
        }
    }
    __syncthreads();
    // holes (low half of a count) and movers (high half); both fit: a CTA has at most 16384 slots
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = s0 + r * kClusterThreads;
        const bool k = kept >> r & 1u;
        const uint32_t bh = __ballot_sync(0xffffffffu, i < keep && !k), bm = __ballot_sync(0xffffffffu, i >= keep && k);
        if (lane == 0) cnt[r * NW + warp] = __popc(bh) | (__popc(bm) << 16);
    }
    __syncthreads();
    const int all = scan();
    int h_before = 0, m_before = 0, total = all & 0xFFFF;
    if (CLUSTER) {
        if (tid == 0) share[2] = all;
        sync();
        const int v = of_cluster(&share[2], 0), mine = lane < rank ? v : 0;
        h_before = __reduce_add_sync(0xffffffffu, mine & 0xFFFF);
        m_before = __reduce_add_sync(0xffffffffu, mine >> 16);
        total = __reduce_add_sync(0xffffffffu, v & 0xFFFF);
    }
    int* holes = p.moves + slab * 2 * p.list;
    int* movers = holes + p.list;
    // The tables' entries are read again, in a cluster four slots at a time before any of them is written:
    // the compiler keeps each load behind the stores before it, and of a long cache's 16 slots a thread
    // one latency after the other was a third of the selection's time (81 -> 77 us for 131K slots; of the
    // few slots of a single CTA's threads the registers cost more, 55.6 -> 57.1 us).
    constexpr int BATCH = CLUSTER ? 4 : 1;
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += BATCH) {
        float w[BATCH];
        int q[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = s0 + (r0 + k) * kClusterThreads;
            const bool stays = (kept >> (r0 + k) & 1u) && i < keep;
            if (stays && copy) w[k] = acc[i];
            if (stays && copy_pos) q[k] = pos[i];
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int r = r0 + k, i = s0 + r * kClusterThreads;
            const bool is_kept = kept >> r & 1u, hole = i < keep && !is_kept, mover = i >= keep && is_kept;
            const uint32_t bh = __ballot_sync(0xffffffffu, hole), bm = __ballot_sync(0xffffffffu, mover);
            if (bh | bm) {
                const int at = cnt[r * NW + warp];
                if (hole) holes[h_before + (at & 0xFFFF) + __popc(bh & below)] = i;
                if (mover) movers[m_before + (at >> 16) + __popc(bm & below)] = i;
            }
            if (is_kept && i < keep) {
                if (copy) acc_out[i] = w[k];
                if (copy_pos) pos_out[i] = q[k];
                if (src) src[i] = i;
            }
        }
    }
    sync();  // the lists are whole
    // A mover's entries go to its hole's slot, below n_keep, where nothing is read any more; the
    // tables behind n_keep are read and then cleared by the thread that has the slot.
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += BATCH) {
        int to[BATCH], q[BATCH];
        float w[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int r = r0 + k, i = s0 + r * kClusterThreads;
            to[k] = -1;
            if (i - lane + 32 <= keep) continue;  // the whole warp
            const bool mover = i >= keep && (kept >> r & 1u);
            const uint32_t bm = __ballot_sync(0xffffffffu, mover);
            if (mover) {
                to[k] = holes[m_before + (cnt[r * NW + warp] >> 16) + __popc(bm & below)];
                w[k] = acc[i];
                q[k] = pos[i];
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = s0 + (r0 + k) * kClusterThreads;
            if (i - lane + 32 <= keep) continue;
            if (to[k] >= 0) {
                acc_out[to[k]] = w[k];
                pos_out[to[k]] = q[k];
                if (src) src[to[k]] = i;
            }
            if (i >= keep && i < n) {
                acc_out[i] = 0.f;
                pos_out[i] = -1;
            }
        }
    }
    if (rank == 0 && tid == 0) p.n_moves[slab] = total;
    if (MOVE) move_rows<D>(p, slab, holes, movers, total, rank * kClusterThreads + tid, cluster * kClusterThreads);
}

template <int D, int R>
static cudaError_t launch_evict(const EvictParams& p, unsigned slabs, int cluster, bool move, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(slabs * static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster == 1) {
        return move ? cudaLaunchKernelEx(&cfg, evict_kernel<D, R, false, true>, p, 1)
                    : cudaLaunchKernelEx(&cfg, evict_kernel<D, R, false, false>, p, 1);
    }
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return move ? cudaLaunchKernelEx(&cfg, evict_kernel<D, R, true, true>, p, cluster)
                : cudaLaunchKernelEx(&cfg, evict_kernel<D, R, true, false>, p, cluster);
}

template <int D>
static cudaError_t launch_evict_d(const EvictParams& p, unsigned slabs, cudaStream_t s) {
    const int sms = device_sm_count();
    cudaError_t e;
    bool move = false;
    if (p.L > kEvictMaxSlots) {
        evict_select_long_kernel<<<slabs, kEvictThreads, 0, s>>>(p);
        e = cudaGetLastError();
    } else {
        // as few CTAs as hold a slab; more while SMs are idle and each keeps a few thousand slots (32
        // slabs of 16K: 44.0 us with two CTAs each, 36.8 with four; 8 of 8K: 14.1 with one, 15.7 with two)
        int cluster = 1;
        while (cluster * kClusterThreads * 16 < p.L) cluster *= 2;
        while (cluster < kEvictMaxCluster && static_cast<int64_t>(slabs) * cluster * 2 <= sms && p.L > cluster * kClusterThreads * 4) {
            cluster *= 2;
        }
        // few slabs leave SMs without a CTA: a second launch moves their rows with all of them (8 slabs
        // of 131K: 90.5 us in one launch, 80.3 in two; 8 of 8K: 24.1 and 15.7; but 128 of 8K: 57.8 and
        // 63.4, and 128 of 4K: 31.4 and 34.1)
        move = static_cast<int64_t>(slabs) * cluster * 4 >= 3ll * sms || p.list <= 256;
        const int per_thread = (p.L + cluster * kClusterThreads - 1) / (cluster * kClusterThreads);
        e = per_thread <= 4   ? launch_evict<D, 4>(p, slabs, cluster, move, s)
            : per_thread <= 8 ? launch_evict<D, 8>(p, slabs, cluster, move, s)
                              : launch_evict<D, 16>(p, slabs, cluster, move, s);
    }
    if (e != cudaSuccess || move || p.list == 0) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(slabs, static_cast<unsigned>(std::max<int64_t>(1, 8ll * sms / slabs)));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<D>, p);
}

static bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

static bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

static dak_status device_matches(const dak_placement* p) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DAK_ERR_CUDA;
    return dev == p->device ? DAK_OK : DAK_ERR_INVALID;
}

}  // namespace dak

using namespace dak;

extern "C" dak_status dak_placement_data(const dak_placement* p, void** host, void** hbm) {
    if (!p) return DAK_ERR_INVALID;
    if (host) *host = p->host_ptr;
    if (hbm) *hbm = p->hbm_ptr;
    return DAK_OK;
}

extern "C" dak_status dak_rope_from_freqs(int head_dim, const double* inv_freq, int n_pairs, int interleaved,
                                          double attn_scale, dak_rope_plan* out) {
    if (!inv_freq || !out) return DAK_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return DAK_ERR_UNSUPPORTED;
    if (n_pairs < 1 || n_pairs > head_dim / 2 || !std::isfinite(attn_scale) || attn_scale > 1e30) return DAK_ERR_INVALID;
    dak_rope_plan r{};
    r.head_dim = head_dim;
    r.rot_dim = 2 * n_pairs;
    r.interleaved = interleaved ? 1 : 0;
    r.scale = attn_scale > 0 ? static_cast<float>(attn_scale) : 1.0f;
    for (int i = 0; i < n_pairs; ++i) {
        if (!std::isfinite(inv_freq[i])) return DAK_ERR_INVALID;
        // the division (and 2 pi as a double) is off by less than 2^-52 relative; fmod is exact, sign kept
        const double t = std::fmod(inv_freq[i] / 6.283185307179586476925, 1.0);
        const double f = std::floor(std::ldexp(std::fabs(t), 64) + 0.5);
        const uint64_t u = f >= 0x1p64 ? 0 : static_cast<uint64_t>(f);
        r.turns[i] = t < 0 ? 0 - u : u;  // a turn backwards is its complement
    }
    *out = r;
    return DAK_OK;
}

extern "C" dak_status dak_rope_make(int head_dim, const dak_rope_config* cfg, dak_rope_plan* out) {
    if (!cfg || !out) return DAK_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return DAK_ERR_UNSUPPORTED;
    const int R = cfg->rot_dim > 0 ? cfg->rot_dim : head_dim;
    const double theta = cfg->theta > 0 ? cfg->theta : 500000.0;
    const double s = cfg->factor > 0 ? cfg->factor : 1.0;
    double low = cfg->low_turns, high = cfg->high_turns;
    if (low <= 0 && high <= 0) low = 1.0, high = 32.0;
    if (R % 2 || R > head_dim || !std::isfinite(theta) || !std::isfinite(s) || std::isnan(cfg->theta) ||
        std::isnan(cfg->factor)) {
        return DAK_ERR_INVALID;
    }
    double inv[64];
    for (int i = 0; i < R / 2; ++i) {
        const double e = -2.0 * i / R;
        const double f = std::pow(theta, e);
        switch (cfg->scaling) {
            case DAK_ROPE_PLAIN:
                inv[i] = f;
                break;
            case DAK_ROPE_LINEAR:
                inv[i] = f / s;
                break;
            case DAK_ROPE_NTK:
                inv[i] = R > 2 ? std::pow(theta * std::pow(s, static_cast<double>(R) / (R - 2)), e) : f;
                break;
            case DAK_ROPE_BY_PARTS: {
                if (!(cfg->orig_len > 0) || !std::isfinite(cfg->orig_len) || !(low >= 0) || !(high > low) ||
                    !std::isfinite(high)) {
                    return DAK_ERR_INVALID;
                }
                const double turns = cfg->orig_len * f / 6.283185307179586476925;
                const double mix = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
                inv[i] = f / s * (1 - mix) + f * mix;
                break;
            }
            default:
                return DAK_ERR_INVALID;
        }
    }
    return dak_rope_from_freqs(head_dim, inv, R / 2, cfg->interleaved, cfg->attn_scale, out);
}

extern "C" dak_status dak_kv_append_rope_acc(const dak_placement* KV, const dak_rope_plan* rope, const void* q,
                                             const void* k, const void* v, int in_fp32, int T, int H_q, int64_t q_pitch,
                                             int64_t k_pitch, int64_t v_pitch, const int* slots, const int* positions,
                                             const int* n_new, void* q_out, int* slot_pos, float* acc, void* stream) {
    if (!KV || KV->kind != 1 || !rope || !k || !v || !slots || T < 1 || H_q < 0) return DAK_ERR_INVALID;
    if (H_q > 0 && (!q || !q_out)) return DAK_ERR_INVALID;
    const int D = KV->D;
    if (rope->head_dim != D || rope->rot_dim < 2 || rope->rot_dim > D || rope->rot_dim % 2) return DAK_ERR_INVALID;
    const int64_t kv_row = static_cast<int64_t>(KV->H_kv) * D, q_row = static_cast<int64_t>(H_q) * D;
    if (k_pitch < kv_row || v_pitch < kv_row || (H_q > 0 && q_pitch < q_row)) return DAK_ERR_INVALID;
    const int64_t tokens = static_cast<int64_t>(KV->B) * T;
    if (tokens > 0x7FFFFFFF || static_cast<int64_t>(H_q) + 2ll * KV->H_kv > (1 << 24)) return DAK_ERR_INVALID;
    const int size = in_fp32 ? 4 : 2, per16 = 16 / size;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_out, 16) || misaligned(slots, 4) ||
        misaligned(positions, 4) || misaligned(n_new, 4) || misaligned(slot_pos, 4) || misaligned(acc, 4) ||
        k_pitch % per16 || v_pitch % per16 || (H_q > 0 && q_pitch % per16)) {
        return DAK_ERR_ALIGN;
    }
    if (H_q > 0) {
        const size_t out_bytes = static_cast<size_t>(tokens) * q_row * 2;
        const auto span = [&](int64_t pitch, int64_t row) { return static_cast<size_t>((tokens - 1) * pitch + row) * size; };
        if (ranges_overlap(q_out, out_bytes, q, span(q_pitch, q_row)) ||
            ranges_overlap(q_out, out_bytes, k, span(k_pitch, kv_row)) ||
            ranges_overlap(q_out, out_bytes, v, span(v_pitch, kv_row))) {
            return DAK_ERR_INVALID;
        }
    }
    const dak_status m = device_matches(KV);
    if (m != DAK_OK) return m;
    RopeParams p{};
    p.rope = *rope;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_pitch = q_pitch;
    p.k_pitch = k_pitch;
    p.v_pitch = v_pitch;
    p.slots = slots;
    p.positions = positions;
    p.n_new = n_new;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.slot_pos = slot_pos;
    p.acc = acc;
    p.host = static_cast<uint8_t*>(KV->host_dev);
    p.hbm = static_cast<uint8_t*>(KV->hbm_ptr);
    p.head_bytes = KV->head_bytes;
    p.T = T;
    p.Hq = H_q;
    p.Hkv = KV->H_kv;
    p.L = KV->L;
    p.h_s = KV->h_s;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    // few tokens: their heads over several blocks, up to eight blocks an SM
    const int units = (H_q + 2 * KV->H_kv) * (D / 16), blocks = (units + kRopeThreads - 1) / kRopeThreads;
    const int64_t room = std::max<int64_t>(1, 8ll * device_sm_count() / tokens);
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(std::min<int64_t>(std::min(blocks, 16), room)));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(D == 128 ? (in_fp32 ? launch_append_rope<128, true>(p, grid, s) : launch_append_rope<128, false>(p, grid, s))
                                : (in_fp32 ? launch_append_rope<64, true>(p, grid, s) : launch_append_rope<64, false>(p, grid, s)));
}

extern "C" dak_status dak_kv_append_rope(const dak_placement* KV, const dak_rope_plan* rope, const void* q,
                                         const void* k, const void* v, int in_fp32, int T, int H_q, int64_t q_pitch,
                                         int64_t k_pitch, int64_t v_pitch, const int* slots, const int* positions,
                                         const int* n_new, void* q_out, int* slot_pos, void* stream) {
    return dak_kv_append_rope_acc(KV, rope, q, k, v, in_fp32, T, H_q, q_pitch, k_pitch, v_pitch, slots, positions,
                                  n_new, q_out, slot_pos, nullptr, stream);
}

// Workspace: per slab a count and the holes and movers, of which there are at most
// min(n_keep, L - n_keep) <= L / 2 each.
extern "C" size_t dak_kv_evict_workspace_bytes(const dak_placement* KV) {
    if (!KV || KV->kind != 1) return 0;
    const size_t slabs = static_cast<size_t>(KV->B) * KV->H_kv;
    return (slabs * (1 + 2 * static_cast<size_t>(KV->L / 2)) * sizeof(int) + 15) / 16 * 16;
}

extern "C" dak_status dak_kv_evict(const dak_placement* KV, const int* seq_lens, int n_keep, int n_recent,
                                   const float* acc, float* acc_out, const int* slot_pos, int* slot_pos_out,
                                   int* lens_out, int* src_out, void* workspace, size_t ws_bytes, void* stream) {
    if (!KV || KV->kind != 1 || !seq_lens || !acc || !acc_out || !slot_pos || !slot_pos_out || !lens_out || !workspace) {
        return DAK_ERR_INVALID;
    }
    if (n_keep < 1 || n_keep > KV->L || n_recent < 0 || n_recent > n_keep) return DAK_ERR_INVALID;
    if (misaligned(seq_lens, 4) || misaligned(acc, 4) || misaligned(acc_out, 4) || misaligned(slot_pos, 4) ||
        misaligned(slot_pos_out, 4) || misaligned(lens_out, 4) || misaligned(src_out, 4) || misaligned(workspace, 16)) {
        return DAK_ERR_ALIGN;
    }
    if (ws_bytes < dak_kv_evict_workspace_bytes(KV)) return DAK_ERR_INVALID;
    const size_t slabs = static_cast<size_t>(KV->B) * KV->H_kv;
    const size_t table = slabs * KV->L * 4, lens = static_cast<size_t>(KV->B) * 4;
    if ((acc_out != acc && ranges_overlap(acc_out, table, acc, table)) ||
        (slot_pos_out != slot_pos && ranges_overlap(slot_pos_out, table, slot_pos, table)) ||
        ranges_overlap(lens_out, lens, seq_lens, lens)) {
        return DAK_ERR_INVALID;
    }
    const dak_status m = device_matches(KV);
    if (m != DAK_OK) return m;
    EvictParams p{};
    p.seq_lens = seq_lens;
    p.acc = acc;
    p.acc_out = acc_out;
    p.pos = slot_pos;
    p.pos_out = slot_pos_out;
    p.lens_out = lens_out;
    p.src_out = src_out;
    p.n_moves = static_cast<int*>(workspace);
    p.moves = p.n_moves + slabs;
    p.list = n_keep < KV->L - n_keep ? n_keep : KV->L - n_keep;
    p.Hkv = KV->H_kv;
    p.L = KV->L;
    p.n_keep = n_keep;
    p.n_recent = n_recent;
    p.host = static_cast<uint8_t*>(KV->host_dev);
    p.hbm = static_cast<uint8_t*>(KV->hbm_ptr);
    p.head_bytes = KV->head_bytes;
    p.h_s = KV->h_s;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = KV->D == 128 ? launch_evict_d<128>(p, static_cast<unsigned>(slabs), s)
                                       : launch_evict_d<64>(p, static_cast<unsigned>(slabs), s);
    return cuda_status(e);
}
