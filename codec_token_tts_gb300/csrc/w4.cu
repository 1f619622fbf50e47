// Products with 4-bit weights and group scales, y = x W^T for a few rows of x, on the caller's buffers.
//
// W[n][k] = scale[n][k / G] (code - zero). The tensor cores take the whole number code - zero, which is exact
// in bf16: 128 + code is one logical operation on a nibble (0x4300 | code), and adding -(128 + zero) is exact.
// An fp32 row of x enters as three bf16 parts (8 + 8 + 8 bits by truncation, together x itself), each in
// a column of its own, so every product is exact, sums are fp32, and a scale multiplies each group's sum.
//
// Layout (tts_bb_w4_pack): for 16 rows (one m16n8k16 tile high) and one group, a record of G * 8 bytes of
// codes and 16 parameter words. Lane (r = lane / 4, q = lane % 4) of a warp finds its codes of the group in
// 16-byte pieces, one coalesced load each (G = 32: 8 bytes). Word i is the A operand of step i: nibble j the
// low, nibble j + 4 the high half of register j: rows r (j even) and r + 8 (j odd), columns q G / 4 + 4 i + {0, 1}
// (j < 2) and + {2, 3}; the columns of a group may stand in any order as long as x's do too, and this one gives a
// lane contiguous x. Parameter word: bf16 -(128 + zero) in the low, bf16 scale in the high half.
#include <algorithm>

#include "common.cuh"
#include "../../include/tts_bb.h"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

constexpr int WARPS = 8;

__host__ __device__ constexpr int record_bytes(int G) { return G * 8 + 64; }

// grid (K / G, ceil(N / 16)), 32 threads
__global__ void k_w4_pack(int N, int K, int G, const uint8_t* __restrict__ codes, const bf16* __restrict__ scales,
                          const uint8_t* __restrict__ zeros, uint8_t* __restrict__ packed) {
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.x, tile = blockIdx.y, lane = threadIdx.x, r = lane >> 2, q = lane & 3;
    const int groups = K / G, words = G / 16;  // words of a lane
    uint8_t* rec = packed + ((size_t)tile * groups + g) * record_bytes(G);
    for (int i = 0; i < words; ++i) {
        uint32_t w = 0;
        for (int j = 0; j < 8; ++j) {
            const int n = tile * 16 + r + (j & 1) * 8, k = g * G + q * (G / 4) + 4 * i + (j & 2) + (j >> 2);
            const uint32_t b = n < N ? codes[((size_t)n * K + k) >> 1] : 0u;
            w |= (k & 1 ? b >> 4 : b & 15u) << (4 * j);
        }
        // pieces of 4 words (G = 32: of 2)
        const int per = words < 4 ? words : 4;
        reinterpret_cast<uint32_t*>(rec)[((i / per) * 32 + lane) * per + i % per] = w;
    }
    if (lane < 16) {
        const int n = tile * 16 + lane;
        const size_t at = (size_t)n * groups + g;
        const uint32_t s = n < N ? __bfloat16_as_ushort(scales[at]) : 0u;
        const float z = n < N && zeros ? (float)(zeros[at] & 15) : 8.f;
        reinterpret_cast<uint32_t*>(rec + G * 8)[lane] = s << 16 | __bfloat16_as_ushort(__float2bfloat16_rn(-(128.f + z)));
    }
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// one word of codes -> the A registers of a step; z0, z1: -(128 + zero) of rows r, r + 8, twice each
__device__ __forceinline__ void dequant(uint32_t w, uint32_t z0, uint32_t z1, uint32_t* a) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = add_bf16x2((w >> (4 * j) & 0x000F000Fu) | 0x43004300u, j & 1 ? z1 : z0);
}
// part (0, 1, 2) of an fp32 value: 8 significant bits each, by truncation; m1, m2: all ones above bit 15 where part >= 1, 2
__device__ __forceinline__ float part_of(float x, uint32_t m1, uint32_t m2) {
    x -= __uint_as_float(__float_as_uint(x) & m1);
    return x - __uint_as_float(__float_as_uint(x) & m2);
}

template <typename T> constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;

// grid (ceil(N / 16), chunks of x rows), WARPS * 32 threads: one 16-row tile, its groups dealt to the warps; NT tiles
// of 8 columns, a column being one part of one row of x. The warps' sums are added in their order.
template <typename T, int G, int NT>
__global__ void __launch_bounds__(WARPS * 32) k_w4_linear(int T_, int N, int K, const T* __restrict__ x, long long stride,
                                                          const uint8_t* __restrict__ packed, T* __restrict__ y, int per) {
    pdl_wait();
    pdl_trigger();
    constexpr int P = PARTS<T>, WORDS = G / 16;
    const int tile = blockIdx.x, t0 = blockIdx.y * per, nt_tok = min(per, T_ - t0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
    const int groups = K / G;
    float acc[NT][4] = {};
    for (int g = warp; g < groups; g += WARPS) {
        const uint8_t* rec = packed + ((size_t)tile * groups + g) * record_bytes(G);
        uint32_t w[WORDS];
        if constexpr (WORDS == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(rec + lane * 8);
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(rec + (i * 32 + lane) * 16);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        }
        const uint32_t p0 = reinterpret_cast<const uint32_t*>(rec + G * 8)[r];
        const uint32_t p1 = reinterpret_cast<const uint32_t*>(rec + G * 8)[r + 8];
        const uint32_t z0 = __byte_perm(p0, p0, 0x1010), z1 = __byte_perm(p1, p1, 0x1010);
        float d[NT][4] = {};
        uint32_t a[WORDS][4];
#pragma unroll
        for (int i = 0; i < WORDS; ++i) dequant(w[i], z0, z1, a[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = nt * 8 + r, tok = c / P;
            const bool on = tok < nt_tok;
            const T* src = x + (size_t)(t0 + (on ? tok : 0)) * stride + g * G + q * (G / 4);
            uint32_t b[2 * WORDS];
            if constexpr (P == 1) {
#pragma unroll
                for (int i = 0; i < WORDS / 2; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
                    b[4 * i] = v.x; b[4 * i + 1] = v.y; b[4 * i + 2] = v.z; b[4 * i + 3] = v.w;
                }
            } else {
                const int part = c - tok * P;
                const uint32_t m1 = part >= 1 ? 0xFFFF0000u : 0u, m2 = part >= 2 ? 0xFFFF0000u : 0u;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(src + 4 * i);
                    b[2 * i] = __byte_perm(__float_as_uint(part_of(v.x, m1, m2)), __float_as_uint(part_of(v.y, m1, m2)), 0x7632);
                    b[2 * i + 1] = __byte_perm(__float_as_uint(part_of(v.z, m1, m2)), __float_as_uint(part_of(v.w, m1, m2)), 0x7632);
                }
            }
#pragma unroll
            for (int i = 0; i < WORDS; ++i) mma(d[nt], a[i], on ? b[2 * i] : 0u, on ? b[2 * i + 1] : 0u);
        }
        const float s0 = __uint_as_float(p0 & 0xFFFF0000u), s1 = __uint_as_float(p1 & 0xFFFF0000u);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] += s0 * d[nt][0]; acc[nt][1] += s0 * d[nt][1];
            acc[nt][2] += s1 * d[nt][2]; acc[nt][3] += s1 * d[nt][3];
        }
    }
    __shared__ float red[WARPS][NT * 8][17];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[warp][nt * 8 + 2 * q + (e & 1)][r + (e >> 1) * 8] = acc[nt][e];
    __syncthreads();
    for (int i = threadIdx.x; i < nt_tok * 16; i += WARPS * 32) {
        const int tok = i >> 4, n = i & 15;
        float v = 0.f;
#pragma unroll
        for (int p = P - 1; p >= 0; --p)  // the small parts first
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += red[w][tok * P + p][n];
        if (tile * 16 + n < N) y[(size_t)(t0 + tok) * N + tile * 16 + n] = (T)v;
    }
}

template <typename T, int G>
void launch(int T_, int N, int K, const void* x, int64_t stride, const void* packed, void* y, cudaStream_t st) {
    constexpr int P = PARTS<T>;
    const int per = std::min(T_, 64 / P), nt = (per * P + 7) / 8;
    const dim3 grid((N + 15) / 16, (T_ + per - 1) / per);
    auto go = [&](auto k) {
        launch_pdl(k, grid, WARPS * 32, 0, st, T_, N, K, static_cast<const T*>(x), (long long)stride,
                   static_cast<const uint8_t*>(packed), static_cast<T*>(y), per);
    };
    if (nt <= 1) go(k_w4_linear<T, G, 1>);
    else if (nt <= 2) go(k_w4_linear<T, G, 2>);
    else if (nt <= 4) go(k_w4_linear<T, G, 4>);
    else go(k_w4_linear<T, G, 8>);
}

bool sizes_ok(int N, int K, int G) {
    return N >= 1 && N <= (1 << 20) && (G == 32 || G == 64 || G == 128) && K >= G && K % G == 0 && K <= (1 << 20);
}

}  // namespace

TTS_API size_t tts_bb_w4_packed_bytes(int N, int K, int group) {
    return sizes_ok(N, K, group) ? (size_t)((N + 15) / 16) * (K / group) * record_bytes(group) : 0;
}

TTS_API tts_bb_status tts_bb_w4_pack(int N, int K, int group, const void* codes, const void* scales, const void* zeros,
                                     void* packed, void* stream) {
    if (!sizes_ok(N, K, group) || !codes || !scales || !packed || (uintptr_t)packed % 16 || (uintptr_t)scales % 2)
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    launch_pdl(k_w4_pack, dim3(K / group, (N + 15) / 16), 32, 0, static_cast<cudaStream_t>(stream), N, K, group,
               static_cast<const uint8_t*>(codes), static_cast<const bf16*>(scales), static_cast<const uint8_t*>(zeros),
               static_cast<uint8_t*>(packed));
    return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA;
}

TTS_API tts_bb_status tts_bb_w4_linear(int T, int N, int K, int group, const void* x, int type, int64_t x_stride,
                                       const void* packed, void* y, void* stream) {
    const int es = type == TTS_BB_T_F32 ? 4 : 2;
    if (!sizes_ok(N, K, group) || T < 1 || T > TTS_BB_W4_MAX_TOKENS || !x || !packed || !y || x_stride < K ||
        (type != TTS_BB_T_F32 && type != TTS_BB_T_BF16) || (uintptr_t)x % 16 || (x_stride * es) % 16 ||
        (uintptr_t)packed % 16 || (uintptr_t)y % es)
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto t) {
        typedef decltype(t) E;
        if (group == 32) launch<E, 32>(T, N, K, x, x_stride, packed, y, st);
        else if (group == 64) launch<E, 64>(T, N, K, x, x_stride, packed, y, st);
        else launch<E, 128>(T, N, K, x, x_stride, packed, y, st);
    };
    if (type == TTS_BB_T_F32) go(float{});
    else go(bf16{});
    return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA;
}
