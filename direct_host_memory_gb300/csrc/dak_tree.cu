// Decode attention of a tree (or chain) of drafted tokens per request over a placed KV cache,
// dak_attn_tree. The cache layout is the one of dak_attn.cu.
#include <algorithm>
#include <cmath>

#include "dak_device.cuh"

namespace dak {

struct TreeParams {
    const __nv_bfloat16* Q;  // [B][T][Hq][D]
    const int* lens;
    const int* n_new;               // or null
    const unsigned long long* mask;  // or null: a chain
    long long mask_pitch;
    void* O;
    int o_fp32;
    const uint8_t* kv[2];  // host tier (device-visible), HBM tier
    long long head_bytes;
    int B, T, W, Hq, Hkv, G, L, h_s;  // W: mask words of a token
    float scale_log2;
    DevStatus* st;
};

// A warp per (token, query head).
template <int D>
__global__ void __launch_bounds__(128) tree_kernel(const TreeParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.T * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq), t = static_cast<int>(row / p.Hq % p.T), b = static_cast<int>(row / p.Hq / p.T);
    const int n_new = p.n_new ? min(max(p.n_new[b], 0), p.T) : p.T;
    if (t >= n_new) return;
    const int len = min(max(p.lens[b], 0), p.L), drafts = min(n_new, p.L - len), g = h / p.G;
    if (drafts < n_new && t == 0 && h == 0 && lane == 0) report(p.st, DAK_ERR_BOUNDS, (0x7EEEull << 32) | static_cast<unsigned>(b));
    const long long slab = static_cast<long long>(b) * p.Hkv + g;
    const uint8_t* base = slab < p.h_s ? p.kv[0] + slab * p.head_bytes : p.kv[1] + (slab - p.h_s) * p.head_bytes;
    const auto elem = [&](int j, int kv, int d) {
        const __nv_bfloat16* c = reinterpret_cast<const __nv_bfloat16*>(base) + ((static_cast<long long>(j >> 6) * 2 + kv) * 64 + (j & 63)) * D;
        return __bfloat162float(c[((d >> 3) ^ (j & 7)) * 8 + (d & 7)]);
    };
    float q[E], o[E];
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(p.Q[row * D + e * 32 + lane]), o[e] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool any = false;
    for (int j = 0; j < len + drafts; ++j) {
        const int s = j - len;
        if (s >= 0) {
            const bool sees = p.mask ? p.mask[b * p.mask_pitch + static_cast<long long>(t) * p.W + (s >> 6)] >> (s & 63) & 1 : s <= t;
            if (!sees) continue;
        }
        any = true;
        float x = 0.f;
        for (int e = 0; e < E; ++e) x += q[e] * elem(j, 0, e * 32 + lane);
        for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        x *= p.scale_log2;
        const float m2 = fmaxf(m, x), ref = m2 == -INFINITY ? 0.f : m2, f = exp2f(m - ref), w = exp2f(x - ref);
        m = m2;
        l = l * f + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * elem(j, 1, e * 32 + lane);
    }
    for (int e = 0; e < E; ++e) {
        const float v = any ? o[e] / l : 0.f;
        if (p.o_fp32) static_cast<float*>(p.O)[row * D + e * 32 + lane] = v;
        else static_cast<__nv_bfloat16*>(p.O)[row * D + e * 32 + lane] = __float2bfloat16_rn(v);
    }
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
    return 256;
}

extern "C" dak_status dak_attn_tree(const void* Q, const dak_placement* KV, const int* seq_lens, int T, const uint64_t* mask,
                                    int64_t mask_pitch, const int* n_new, int H_q, float scale, void* O, int o_fp32,
                                    void* workspace, size_t ws_bytes, const dak_tuning* tuning, void* stream) {
    (void)tuning;
    if (!KV || KV->kind != 1 || !Q || !O || !seq_lens || T < 1 || H_q < 1 || H_q % KV->H_kv) return DAK_ERR_INVALID;
    const int G = H_q / KV->H_kv, D = KV->D, W = (T + 63) / 64;
    if (T > DAK_MAX_TREE || G > 16) return DAK_ERR_UNSUPPORTED;
    if (mask && mask_pitch != 0 && mask_pitch < static_cast<int64_t>(T) * W) return DAK_ERR_INVALID;
    const size_t elems = static_cast<size_t>(KV->B) * T * H_q * D;
    if (overlap(Q, elems * 2, O, elems * (o_fp32 ? 4 : 2))) return DAK_ERR_INVALID;
    if (off(Q, 16) || off(O, 16) || off(workspace, 16) || off(seq_lens, 4) || off(n_new, 4) || off(mask, 8)) return DAK_ERR_ALIGN;
    if (!workspace || ws_bytes < dak_attn_tree_workspace_bytes(KV, T, H_q)) return DAK_ERR_INVALID;
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
    p.kv[0] = static_cast<const uint8_t*>(KV->host_dev);
    p.kv[1] = static_cast<const uint8_t*>(KV->hbm_ptr);
    p.head_bytes = KV->head_bytes;
    p.B = KV->B;
    p.T = T;
    p.W = W;
    p.Hq = H_q;
    p.Hkv = KV->H_kv;
    p.G = G;
    p.L = KV->L;
    p.h_s = KV->h_s;
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
    p.st = status_ptr();
    if (!p.st) return DAK_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(KV->B) * T * H_q, blocks = (rows + 3) / 4;
    if (blocks > 0x7FFFFFFF) return DAK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D == 128) tree_kernel<128><<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
    else tree_kernel<64><<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}
