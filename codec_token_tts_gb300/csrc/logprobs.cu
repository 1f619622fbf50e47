// Log probabilities of given tokens, entropy, log-sum-exp and the most probable tokens of logits rows.
//
// With m the row's largest logit at its lowest id i*, r = sum over the other ids of exp(z - m) and t = sum over
// them of exp(z - m) (z - m):
//   lse = m + log1p(r),  log p(i) = (z_i - m) - log1p(r),  H = log1p(r) - t / (1 + r)
// (the largest term, exactly 1, stays out of the sum, so a row sure of its answer keeps its digits).
// Order of the alternatives: the float's bits made monotone in the high word, the complement of the id in the low
// one: no two keys are equal, and the larger key is the larger logit or, among equals, the lower id.
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "../../include/tts_bb.h"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

typedef unsigned long long u64;
constexpr float NEG_INF = -INFINITY;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ u64 key_of(float z, int i) { return pack_argmax(z + 0.f, i); }  // -0 + 0 = +0
__device__ __forceinline__ int id_of(u64 k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
__device__ __forceinline__ float value_of(u64 k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ u64 warp_max_key(u64 k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) { const u64 w = __shfl_xor_sync(0xffffffffu, k, o); k = w > k ? w : k; }
    return k;
}

struct Args {
    int R, V, n_top;
    long long stride, allowed_stride;
    const int32_t* targets;
    const uint32_t* allowed;
    float *logprob, *entropy, *lse;
    int32_t* top_ids;
    float* top_lp;
};

__device__ __forceinline__ bool is_allowed(const uint32_t* a, int i) { return !a || (a[i >> 5] >> (i & 31) & 1u); }

constexpr int THREADS = 256;

template <typename T>
__device__ __forceinline__ T block_sum(T v, T* sm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
    for (int w = 1; w < THREADS / 32; ++w) v += sm[w];
    return v;
}
__device__ __forceinline__ u64 block_max_key(u64 k, u64* sm) {
    k = warp_max_key(k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = k;
    __syncthreads();
    k = sm[0];
    for (int w = 1; w < THREADS / 32; ++w) k = sm[w] > k ? sm[w] : k;
    return k;
}

// grid R, THREADS threads: one row each; a pass for the maximum, one for the sums, one for each alternative.
template <typename T>
__global__ void __launch_bounds__(THREADS) k_logprobs(const T* __restrict__ logits, Args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ u64 smk[THREADS / 32];
    __shared__ float smf[THREADS / 32];
    const int row = blockIdx.x, tid = threadIdx.x;
    const T* z = logits + (size_t)row * a.stride;
    const uint32_t* ok = a.allowed ? a.allowed + (size_t)row * a.allowed_stride : nullptr;
    u64 best = 0;
    int bad = 0;
    for (int i = tid; i < a.V; i += THREADS) {
        const float v = to_f(z[i]);
        if (!is_allowed(ok, i)) continue;
        if (!(v < INFINITY)) bad = 1;
        else if (v > NEG_INF) { const u64 k = key_of(v, i); best = k > best ? k : best; }
    }
    bad = __syncthreads_or(bad);
    best = block_max_key(best, smk);
    const int top = best ? id_of(best) : -1;
    const float m = best ? value_of(best) : 0.f;
    float r = 0.f, t = 0.f;
    for (int i = tid; i < a.V; i += THREADS) {
        if (i == top || !is_allowed(ok, i)) continue;
        const float d = to_f(z[i]) - m, e = expf(d);
        r += e;
        if (e > 0.f) t += e * d;
    }
    r = block_sum(r, smf);
    t = block_sum(t, smf);
    const float nan = __int_as_float(0x7FC00000), log_s = log1pf(r);
    if (tid == 0) {
        if (a.targets && a.logprob) {
            const int i = a.targets[row];
            const float v = i >= 0 && i < a.V && is_allowed(ok, i) ? to_f(z[i]) : NEG_INF;
            a.logprob[row] = bad ? nan : best ? (v - m) - log_s : NEG_INF;
        }
        if (a.entropy) a.entropy[row] = bad ? nan : best ? log_s - t / (1.f + r) : 0.f;
        if (a.lse) a.lse[row] = bad ? nan : best ? m + log_s : NEG_INF;
    }
    u64 last = ~0ull;
    for (int j = 0; j < a.n_top; ++j) {
        if (last && !bad) {
            u64 k = 0;
            for (int i = tid; i < a.V; i += THREADS) {
                const float v = to_f(z[i]);
                if (!is_allowed(ok, i) || !(v > NEG_INF)) continue;
                const u64 c = key_of(v, i);
                if (c < last && c > k) k = c;
            }
            last = block_max_key(k, smk);
        }
        if (tid == 0) {
            a.top_ids[(size_t)row * a.n_top + j] = last && !bad ? id_of(last) : -1;
            a.top_lp[(size_t)row * a.n_top + j] = bad ? nan : last ? (value_of(last) - m) - log_s : NEG_INF;
        }
    }
}

}  // namespace

TTS_API size_t tts_bb_token_logprobs_workspace(int, int, int) { return 0; }

TTS_API tts_bb_status tts_bb_token_logprobs(int R, int V, const void* logits, int type, int64_t row_stride,
                                            const int32_t* targets, const uint32_t* allowed, int64_t allowed_stride,
                                            int n_top, float* logprob, float* entropy, float* lse, int32_t* top_ids,
                                            float* top_logprobs, void* workspace, size_t workspace_bytes, void* stream) {
    if (R < 1 || V < 1 || !logits || row_stride < V || n_top < 0 || n_top > TTS_BB_LOGPROBS_MAX_TOP ||
        type < TTS_BB_T_F32 || type > TTS_BB_T_F16 || (uintptr_t)logits % (type == TTS_BB_T_F32 ? 4 : 2) ||
        (targets && !logprob) || (n_top && (!top_ids || !top_logprobs)) ||
        (allowed && allowed_stride != 0 && allowed_stride < ((int64_t)V + 31) / 32))
        return TTS_BB_E_INVALID;
    const size_t need = tts_bb_token_logprobs_workspace(R, V, n_top);
    if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 16)) return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Args a{R, V, n_top, row_stride, allowed_stride, targets, allowed, logprob, entropy, lse, top_ids, top_logprobs};
    if (type == TTS_BB_T_F32) launch_pdl(k_logprobs<float>, R, THREADS, 0, st, static_cast<const float*>(logits), a);
    else if (type == TTS_BB_T_BF16) launch_pdl(k_logprobs<bf16>, R, THREADS, 0, st, static_cast<const bf16*>(logits), a);
    else launch_pdl(k_logprobs<__half>, R, THREADS, 0, st, static_cast<const __half*>(logits), a);
    return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA;
}
