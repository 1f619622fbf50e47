// Attention of a tree of drafted tokens over the paged bf16 cache: a node sees the cached keys, itself and its ancestors.
#include <algorithm>

#include "tree.cuh"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

struct TreeArgs {
    const void* q;
    const bf16 *k, *v;
    long long q_stride, kv_stride;
    const int32_t *parents, *n_nodes, *seqs, *kv_lens;
    int N, max_len;
    void* out;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// grid (N, 8, B), 128 threads: a node's two heads. Warp w takes keys w, w + 4, ...; a lane holds 4 of the 128 dims.
template <typename T>
__global__ void __launch_bounds__(128) k_tree_attn(Pages c, TreeArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int par[MAX_NODES];
    __shared__ float sm[4][2], sl[4][2], so[4][2][HD];
    const int i = blockIdx.x, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = row_of(c, a.seqs, b), n = a.n_nodes ? a.n_nodes[b] : a.N, len = a.kv_lens[b];
    const bool report = i == 0 && g == 0 && tid == 0;
    if (row == -1) return;
    if (row < 0 || n < 0 || n > a.N || len < 0 || len > a.max_len) {
        if (report) set_err(c.err, TTS_BB_TREE_ERR_RANGE);
        return;
    }
    bool bad = false;
    if (tid < n) {
        par[tid] = a.parents[(size_t)b * a.N + tid];
        bad = par[tid] < -1 || par[tid] >= tid;
    }
    if (__syncthreads_or(bad)) {
        if (report) set_err(c.err, TTS_BB_TREE_ERR_TREE);
        return;
    }
    if (i >= n) return;
    const size_t node = (size_t)b * a.N + i;
    float4 q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) q[h] = load4(static_cast<const T*>(a.q) + node * a.q_stride + (2 * g + h) * HD + lane * 4);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 o[2] = {};
    const float scale = 0.08838834764831845f;
    auto take = [&](const bf16* kp, const bf16* vp) {
        const float4 k = load4(kp + lane * 4), v = load4(vp + lane * 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float s = warp_sum(q[h].x * k.x + q[h].y * k.y + q[h].z * k.z + q[h].w * k.w) * scale;
            const float m1 = fmaxf(m[h], s), base = m1 == -INFINITY ? 0.f : m1;
            const float f = expf(m[h] - base), p = expf(s - base);
            m[h] = m1;
            l[h] = l[h] * f + p;
            o[h].x = o[h].x * f + p * v.x;
            o[h].y = o[h].y * f + p * v.y;
            o[h].z = o[h].z * f + p * v.z;
            o[h].w = o[h].w * f + p * v.w;
        }
    };
    for (int j = warp; j < len; j += 4) {
        const int page = page_of(c, row, j);
        if (page < 0) {
            if (report || (i == 0 && g == 0 && lane == 0)) set_err(c.err, TTS_BB_TREE_ERR_PAGE);
            continue;
        }
        const bf16* const t = c.pool + page * KV_BLOCK + (size_t)g * (KVB * HD) + (size_t)(j % KVB) * HD;
        take(t, t + KV_BLOCK / 2);
    }
    int step = 0;
    for (int j = i; j >= 0; j = par[j], ++step) {
        if ((step & 3) != warp) continue;
        const size_t at = ((size_t)b * a.N + j) * a.kv_stride + g * HD;
        take(a.k + at, a.v + at);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float4*>(&so[warp][h][lane * 4]) = o[h];
        if (lane == 0) { sm[warp][h] = m[h]; sl[warp][h] = l[h]; }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w][h]);
        const float base = M == -INFINITY ? 0.f : M;
        for (int w = 0; w < 4; ++w) {
            const float f = expf(sm[w][h] - base);
            L += f * sl[w][h];
            O += f * so[w][h][tid];
        }
        static_cast<T*>(a.out)[(node * NQ + 2 * g + h) * HD + tid] = (T)(L == 0.f ? 0.f : O / L);
    }
}

}  // namespace

TTS_API size_t tts_bb_tree_attention_workspace(int B, int N, int max_len) {
    if (!tree_ok(B, N) || max_len < 0 || max_len > (1 << 30)) return 0;
    return 0;
}

TTS_API tts_bb_status tts_bb_tree_attention(const tts_bb_kv_cache* cache, int layer, int B, int N, const void* q, int type,
                                            int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                            const int32_t* parents, const int32_t* n_nodes, const int32_t* seqs,
                                            const int32_t* kv_lens, int max_len, void* out, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    if (!cache_ok(cache) || layer < 0 || layer >= cache->n_layers || !tree_ok(B, N) || !q || !k || !v || !parents || !kv_lens || !out ||
        (type != TTS_BB_T_F32 && type != TTS_BB_T_BF16) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        q_stride < NQ * HD || q_stride % (type == TTS_BB_T_F32 ? 4 : 8) || kv_stride < NKV * HD || kv_stride % 8 || max_len < 0 ||
        max_len > (1 << 30) || (long long)max_len > (long long)cache->blocks_per_seq * KVB || (!seqs && B > cache->n_seqs) ||
        !words_aligned(parents, n_nodes, seqs, kv_lens))
        return TTS_BB_E_INVALID;
    const size_t need = tts_bb_tree_attention_workspace(B, N, max_len);
    if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const TreeArgs a{q, static_cast<const bf16*>(k), static_cast<const bf16*>(v), q_stride, kv_stride, parents, n_nodes, seqs, kv_lens,
                     N, max_len, out};
    const dim3 grid(N, NKV, B);
    if (type == TTS_BB_T_F32) launch_pdl(k_tree_attn<float>, grid, 128, 0, static_cast<cudaStream_t>(stream), pages_of(cache, layer), a);
    else launch_pdl(k_tree_attn<bf16>, grid, 128, 0, static_cast<cudaStream_t>(stream), pages_of(cache, layer), a);
    return launched();
}
