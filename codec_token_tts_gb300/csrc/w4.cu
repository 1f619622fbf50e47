// Products with 4-bit weights and group scales, y = x W^T for a few rows of x, on the caller's buffers.
//
// W[n][k] = scale[n][k / G] (code - zero). Bound by the codes' bytes where the matrix is large, by one launch's latency where
// it is small; what comes next are the integer instructions that take nibbles apart (two a cycle and SM).
//
// Main kernel (k_w4_staged): the half word 000c is the fp16 number c 2^-24, 00c0 is 16 c 2^-24 (subnormals and the first
// binade are evenly spaced), so a word of 8 codes is a step's operand of m16n8k16 after one shift, four masks and four
// multiply-adds to (code - zero) 2^-9, exact in fp16. (The subnormal numbers themselves as operands lose up to 5 bits of the
// products' sum, measured; and zeros by the sums of x, scale (sum x code - zero sum x), lose the digits of a small sum
// beside one large x whose weight is 0.) Each row of x is scaled by a power of two to a largest magnitude in [2^14, 2^15)
// and stands in shared memory as fp16: bf16 rows exactly (down to 2^-29 of the row's largest), fp32 rows as two parts, to
// within one fp32 step together (twice 11 bits and a sign), each part a column of its own. So products are exact and sums fp32.
//
// Layout (tts_bb_w4_pack): for 16 rows of W (one m16n8k16 tile high) and one group, a record of G * 8 bytes of
// codes and 16 parameter words. Lane (r = lane / 4, q = lane % 4) of a warp finds its codes of the group in
// 16-byte pieces, one coalesced load each (G = 32: 8 bytes). Word i is the A operand of step i: nibble j the
// low, nibble j + 4 the high half of register j: rows r (j even) and r + 8 (j odd), columns q G / 4 + 4 i + {0, 1}
// (j < 2) and + {2, 3}; the columns of a group may stand in any order as long as x's do too, and this one gives a
// lane contiguous x. Parameter word: fp16 -zero 2^-9 in the low, bf16 scale in the high half.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "../../include/tts_bb.h"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

constexpr int WARPS = 8;

__host__ __device__ constexpr int record_bytes(int G) { return G * 8 + 64; }

// grid (ceil(N / 16), K / G), 32 threads: up to 65536 tiles, which only a grid's first dimension may have
__global__ void k_w4_pack(int N, int K, int G, const uint8_t* __restrict__ codes, const bf16* __restrict__ scales,
                          const uint8_t* __restrict__ zeros, uint8_t* __restrict__ packed) {
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.y, tile = blockIdx.x, lane = threadIdx.x, r = lane >> 2, q = lane & 3;
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
        reinterpret_cast<uint32_t*>(rec + G * 8)[lane] = s << 16 | __half_as_ushort(__float2half_rn(-z * 0x1p-9f));
    }
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// loads by 32-bit addresses of shared memory (1 x 16384 x 16384 bf16 35.2 us, by pointers 36.3)
__device__ __forceinline__ uint4 shared4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 shared2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t shared1(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), v); }

__device__ __forceinline__ float peer(const float* p, int rank) {  // *p in the shared memory of a block of the cluster
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T> constexpr int COLS = sizeof(T) == 4 ? 2 : 1;  // fp16 parts, columns, of a row of x
constexpr int RED_ROW = 17, STAGES = 3;
constexpr int MOST_COLS = 32;
// tiles of 8 columns that a kernel is built for
constexpr int tiles_for(int cols) { return cols <= 8 ? 1 : cols <= 16 ? 2 : 4; }
constexpr size_t staged_bytes(int cols, int K, int G) {
    return (size_t)cols * K * 2 + (size_t)2 * WARPS * tiles_for(cols) * 8 * RED_ROW * 4 + (size_t)WARPS * STAGES * record_bytes(G);
}

// grid (blocks, chunks of x rows), WARPS * 32 threads. A block stages its rows of x once and walks the 16-row tiles of W
// with the stride of the grid; a tile's groups are dealt to the warps, whose records come by cp.async through a ring of each
// warp's own, two on their way while one is multiplied.
// Shared memory: x as B registers, 16 bytes (two steps) a lane and piece: [group][G / 32 pieces][columns][4 lanes]; the warps'
// sums of a tile, twice: one barrier a tile; the rings. Sums are added in the warps' order.
// With SPLIT a cluster of blocks has K in slices of `slice` columns, a block each (the last may have fewer, or none), and a
// warp a tile of its own. After a round of WARPS tiles the blocks lay down their sums, arrive at the cluster's barrier, go
// on with the next round, and only then wait and add up a share of the tiles each. A block scales its slices of the rows by
// itself.
template <typename T, int G, int NT, bool SPLIT>
__global__ void __launch_bounds__(WARPS * 32, NT <= 2 ? 3 : 2)
    k_w4_staged(int T_, int N, int K_all, const T* __restrict__ x, long long stride, const uint8_t* __restrict__ packed,
                T* __restrict__ y, int per, int slice, int n_split) {
    constexpr int P = COLS<T>, WORDS = G / 16, PIECES = G / 32, C8 = NT * 8;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t largest[TTS_BB_W4_MAX_TOKENS];
    const int t0 = blockIdx.y * per, rows = min(per, T_ - t0), cols = rows * P, groups = K_all / G, tiles = (N + 15) / 16;
    const int rank = SPLIT ? blockIdx.x % n_split : 0, team = SPLIT ? blockIdx.x / n_split : blockIdx.x;
    const int teams = SPLIT ? gridDim.x / n_split : gridDim.x;
    const int k0 = SPLIT ? min(rank * slice, K_all) : 0, K = SPLIT ? min(slice, K_all - k0) : K_all;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
    uint4* const xs = reinterpret_cast<uint4*>(smem);
    float* const red = reinterpret_cast<float*>(smem + (size_t)cols * (SPLIT ? slice : K) * 2);
    if (tid < TTS_BB_W4_MAX_TOKENS) largest[tid] = 0u;
    pdl_wait();  // the weights too: the launch before may be the one that packs them
    pdl_trigger();
    constexpr int REC = record_bytes(G);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(red + 2 * WARPS * C8 * RED_ROW) + warp * STAGES * REC;
    // what comes next: its address, the records of the tile from it on, the tile; and its place in the ring
    constexpr int STEP = SPLIT ? 1 : WARPS, TILE_STEP = SPLIT ? WARPS : 1;
    const int first = team * TILE_STEP + (SPLIT ? warp : 0), group0 = SPLIT ? k0 / G : warp;
    const int each = SPLIT ? K / G : (groups - warp + WARPS - 1) / WARPS;  // records of a tile that are this warp's
    int ahead_tile = each > 0 ? first : tiles, left = each;
    const uint8_t* src = packed + ((size_t)first * groups + group0) * REC + lane * 16;
    const long long jump = ((long long)teams * TILE_STEP * groups - (long long)each * STEP) * REC;
    const uint32_t dst0 = ring_at + lane * 16;
    const auto fetch = [&](uint32_t place) {
        const uint32_t dst = dst0 + place;
        if (ahead_tile < tiles) {
#pragma unroll
            for (int i = 0; i < REC; i += 512)
                if (i + 512 <= REC || lane * 16 < REC - i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i), "l"(src + i) : "memory");
            src += STEP * REC;
            if (--left == 0) { left = each; ahead_tile += teams * TILE_STEP; src += jump; }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i * REC);
    __syncthreads();
    const int chunks = K / 8;  // 8 values each
    for (int u0 = 0; u0 < rows * chunks; u0 += WARPS * 32) {
        const int u = u0 + tid, row = min(u / chunks, rows - 1);
        uint32_t b = 0u;  // the bits of magnitudes order them, infinities and NaN above all
        if (u < rows * chunks) {
            float v[8];
            load8(x + (size_t)(t0 + row) * stride + k0 + (u - row * chunks) * 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) b = max(b, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
        // a warp's 32 chunks mostly lie in one row
        if (__all_sync(0xffffffffu, row == __shfl_sync(0xffffffffu, row, 0))) {
            b = __reduce_max_sync(0xffffffffu, b);
            if (lane == 0) atomicMax(&largest[row], b);
        } else {
            atomicMax(&largest[row], b);
        }
    }
    __syncthreads();
    // 2^(14 - exponent of the largest), the largest taken as at least 2^-113: 2^127 is the largest power of two, and brings
    // what is smaller to whole multiples of fp16's least number, so that no digit is lost there either
    const auto up_of = [&](int row) { return __uint_as_float((268u - min(max(largest[row] >> 23, 14u), 254u)) << 23); };
    for (int u = tid; u < rows * chunks; u += WARPS * 32) {
        const int row = u / chunks, chunk = u - row * chunks;
        float v[8];
        load8(x + (size_t)(t0 + row) * stride + k0 + chunk * 8, v);
        const float up = up_of(row);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= up;
        const int g = chunk / (G / 8), sub = chunk % (G / 8), lane_q = sub / PIECES, piece = sub % PIECES;
#pragma unroll
        for (int part = 0; part < P; ++part) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 w = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                const float2 f = __half22float2(w);
                v[2 * e] -= f.x;
                v[2 * e + 1] -= f.y;
                h[e] = *reinterpret_cast<const uint32_t*>(&w);
            }
            xs[((g * PIECES + piece) * cols + row * P + part) * 4 + lane_q] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    __shared__ float down[TTS_BB_W4_MAX_TOKENS];  // what takes a row's scaling back; an infinity or a NaN in the row: NaN
    if (tid < rows) down[tid] = largest[tid] < 0x7F800000u ? 0x1p9f / up_of(tid) : __int_as_float(0x7FC00000);
    __syncthreads();

    uint32_t at[NT];  // this lane's column of each tile of 8; behind the last one, that one again: nobody reads its sums
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) at[nt] = (uint32_t)(min(nt * 8 + r, cols - 1) * 4 + q) * 16;
    const uint32_t x_at = (uint32_t)__cvta_generic_to_shared(xs), piece = cols * 64;  // bytes of a piece
    const uint32_t code_at = ring_at + lane * (WORDS == 2 ? 8 : 16), par_at = ring_at + G * 8 + r * 4;
    // waits for the cluster's sums of a round, adds up this block's share of it
    const auto add_up = [&](int tile, int turn) {
        cluster_wait();
        const auto go = [&](auto split) {
            constexpr int S = decltype(split)::value;
            for (int i = rank * (WARPS * 32) + tid; i < WARPS * rows * 16; i += S * WARPS * 32) {
                const int n = i & 15, row = (i >> 4) % rows, w = (i >> 4) / rows;
                float part[P][S];
#pragma unroll
                for (int j = 0; j < P; ++j)
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        part[j][s] = peer(red + ((size_t)(turn * WARPS + w) * C8 + row * P + j) * RED_ROW + n, s);
                float v = 0.f;
#pragma unroll
                for (int j = P - 1; j >= 0; --j)  // the small part first
#pragma unroll
                    for (int s = 0; s < S; ++s) v += part[j][s];
                if ((tile + w) * 16 + n < N) y[(size_t)(t0 + row) * N + (tile + w) * 16 + n] = (T)v;
            }
        };
        if (n_split == 2) go(std::integral_constant<int, 2>{});
        else if (n_split == 4) go(std::integral_constant<int, 4>{});
        else go(std::integral_constant<int, 8>{});
    };
    int last = 0, last_turn = 0;
    uint32_t rec = 0, before = (STAGES - 1) * REC;  // the places of the record at hand, and of the one before it
    for (int tile = team * TILE_STEP, turn = 0; tile < tiles; tile += teams * TILE_STEP, turn ^= 1) {
        float acc[NT][4] = {};
        uint32_t xg = x_at + (SPLIT ? 0 : warp) * PIECES * piece;
        const int n_rec = !SPLIT || tile + warp < tiles ? each : 0;
        for (int g = 0; g < n_rec; ++g, xg += STEP * PIECES * piece) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncwarp();
            fetch(before);  // which every lane has read
            uint32_t cw[WORDS];
            if constexpr (WORDS == 2) {
                const uint2 v = shared2(code_at + rec);
                cw[0] = v.x; cw[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i) {
                    const uint4 v = shared4(code_at + rec + i * 512);
                    cw[4 * i] = v.x; cw[4 * i + 1] = v.y; cw[4 * i + 2] = v.z; cw[4 * i + 3] = v.w;
                }
            }
            const uint32_t p0 = shared1(par_at + rec), p1 = shared1(par_at + rec + 32);
            const uint32_t z0 = __byte_perm(p0, 0u, 0x1010), z1 = __byte_perm(p1, 0u, 0x1010);
            // times 2^15 and 2^11
            const auto take = [&](uint32_t w, uint32_t (&a)[4]) {
                const uint32_t h = w >> 8;
                a[0] = fma_f16x2(w & 0x000F000Fu, 0x78007800u, z0);
                a[1] = fma_f16x2(w & 0x00F000F0u, 0x68006800u, z1);
                a[2] = fma_f16x2(h & 0x000F000Fu, 0x78007800u, z0);
                a[3] = fma_f16x2(h & 0x00F000F0u, 0x68006800u, z1);
            };
            const float s0 = __uint_as_float(p0 & 0xFFFF0000u), s1 = __uint_as_float(p1 & 0xFFFF0000u);
            float d[NT][4] = {};
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                uint32_t a[2][4];
                take(cw[2 * i], a[0]);
                take(cw[2 * i + 1], a[1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 b = shared4(xg + at[nt] + i * piece);
                    mma_f16(d[nt], a[0], b.x, b.y);
                    mma_f16(d[nt], a[1], b.z, b.w);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] += s0 * d[nt][0];
                acc[nt][1] += s0 * d[nt][1];
                acc[nt][2] += s1 * d[nt][2];
                acc[nt][3] += s1 * d[nt][3];
            }
            before = rec;
            rec = rec == (STAGES - 1) * REC ? 0u : rec + REC;
        }
        float* const mine = red + (size_t)(turn * WARPS + warp) * C8 * RED_ROW;
        if constexpr (SPLIT) {
            if (tile != team * TILE_STEP) add_up(tile - teams * TILE_STEP, turn ^ 1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = nt * 8 + 2 * q + (e & 1);
                float v = acc[nt][e];
                if constexpr (SPLIT) v *= down[min(col, cols - 1) / P];
                mine[col * RED_ROW + r + (e >> 1) * 8] = v;
            }
        if constexpr (SPLIT) {
            cluster_arrive();
            last = tile;
            last_turn = turn;
        } else {
            __syncthreads();
            for (int i = tid; i < rows * 16; i += WARPS * 32) {
                const int row = i >> 4, n = i & 15;
                float v = 0.f;
#pragma unroll
                for (int part = P - 1; part >= 0; --part)  // the small part first
#pragma unroll
                    for (int w = 0; w < WARPS; ++w) v += red[((size_t)(turn * WARPS + w) * C8 + row * P + part) * RED_ROW + n];
                if (tile * 16 + n < N) y[(size_t)(t0 + row) * N + tile * 16 + n] = (T)(v * down[row]);
            }
        }
    }
    if constexpr (SPLIT) {
        add_up(last, last_turn);
        cluster_arrive();  // no block leaves while another reads its sums
        cluster_wait();
    }
}

// Blocks or clusters of a kernel that run at a time on the current device, asked once for a count of blocks an SM: sizes of shared
// memory with the same count share the answer of the first, which sets the grid, not the results.
struct Resident {
    std::atomic<int> n[64];
};
template <typename K>
int clusters_at_a_time(Resident& s, K* kernel, const cudaLaunchConfig_t& cfg) {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    std::atomic<int>& kept = s.n[dev & 63];
    if ((n = kept.load(std::memory_order_relaxed)) > 0) return n;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 1;
    kept.store(n, std::memory_order_relaxed);
    return n;
}

// Room of two blocks an SM, of one, of three.
constexpr size_t STAGED_MOST = 112 * 1024, STAGED_ONE = 220 * 1024, STAGED_THREE = 74 * 1024;

int blocks_an_sm(size_t smem, int nt) { return smem > STAGED_MOST ? 1 : nt <= 2 && smem <= STAGED_THREE ? 3 : 2; }

template <typename T, int G, bool SPLIT>
void launch_staged(int T_, int N, int K, const T* x, int64_t stride, const uint8_t* w, T* y, int per, int n_split,
                   cudaStream_t st) {
    constexpr int P = COLS<T>;
    const int tiles = (N + 15) / 16, groups = K / G, slice = (groups + n_split - 1) / n_split * G;
    const int nt = tiles_for(per * P), chunks = (T_ + per - 1) / per;
    const size_t smem = staged_bytes(per * P, slice, G);
    const int fit = blocks_an_sm(smem, nt);
    auto go = [&](auto k, int which) {
        static SmemState state[3];
        if (smem > 48 * 1024 - 512) allow_smem(state[which], k, STAGED_ONE);
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = n_split;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n_split, chunks);
        cfg.blockDim = WARPS * 32;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = at;
        cfg.numAttrs = SPLIT ? 2 : 1;
        if constexpr (SPLIT) {
            // as many clusters as run at a time: with 19 of 8 blocks asked for and fewer resident, the last would wait for
            // the first to end
            static Resident resident[3][3][3];
            const int at_a_time = clusters_at_a_time(resident[which][n_split == 2 ? 0 : n_split == 4 ? 1 : 2][fit - 1], k, cfg);
            cfg.gridDim.x = n_split * std::min((tiles + WARPS - 1) / WARPS, std::max(1, at_a_time / chunks));
        } else {
            cfg.gridDim.x = std::min(tiles, std::max(1, 152 * fit / chunks));
        }
        cudaLaunchKernelEx(&cfg, k, T_, N, K, x, (long long)stride, w, y, per, slice, n_split);
    };
    if (nt == 1) go(k_w4_staged<T, G, 1, SPLIT>, 0);
    else if (nt == 2) go(k_w4_staged<T, G, 2, SPLIT>, 1);
    else go(k_w4_staged<T, G, 4, SPLIT>, 2);
}

// At most 32 columns at a time (64 in one pass over the weights spill or leave one block an SM: 64 rows x 4096 x 4096 fp32
// 41 us, bf16 30; by 32 columns 26 and 19). Whether K is split:
// - No, where a block has little to stage for each of its tiles: 1 x 4096 x 1024 3.1 us (split in 4: 3.6), 1 x 16384 x 4096
//   10.5 (11.6).
// - Else over as few blocks as give nearly every SM one, or more than two (between one and two, some SMs have twice the
//   work of others): fp32 4 x 4096 x 4096 9.9 -> 6.2 us by 4, 8 x 1024 x 4096 13.0 -> 5.8 by 8, 8 x 8192 x 2048 11.0 -> 8.0
//   by 2 (9.2 by 4), 4 x 16384 x 16384 56 by 2 -> 40 by 4. A single row of few tiles stays whole: 1 x 2048 x 8192 6.7 us,
//   7.4 by 8; and one of many: 1 x 16384 x 16384 bf16 by 4 took 1.05 times as
//   long (in a stream of launches; in a captured graph both the same).
// - As many as two blocks an SM have room for, at most 8; in chunks of fewer rows where a slice is too long even then.
template <typename T, int G>
void launch(int T_, int N, int K, const void* x, int64_t stride, const void* packed, void* y, cudaStream_t st) {
    constexpr int P = COLS<T>;
    const auto bytes = [&](int per, int n) { return staged_bytes(per * P, (K / G + n - 1) / n * G, G); };
    int per = std::min(T_, MOST_COLS / P), n = 1;
    const int tiles = (N + 15) / 16, rounds = (tiles + WARPS - 1) / WARPS, chunks = (T_ + per - 1) / per;
    const int blocks = std::min(tiles, std::max(1, 152 * blocks_an_sm(bytes(per, 1), tiles_for(per * P)) / chunks));
    const long long stage_a_tile = (long long)per * K * blocks / tiles;
    if (stage_a_tile >= 4500 && (T_ > 1 || (rounds >= 32 && tiles < 2 * blocks))) {
        const auto uneven = [&](long long b) { return b < 128 || (b > 152 && b <= 304); };
        for (n = 2; n < 8 && 2 * n <= K / G && uneven((long long)rounds * n * chunks);) n *= 2;
    }
    while (n < 8 && bytes(per, n) > STAGED_MOST) n *= 2;
    while (per > 1 && bytes(per, n) > STAGED_ONE) per = (per + 1) / 2;
    const T* const xt = static_cast<const T*>(x);
    const uint8_t* const w = static_cast<const uint8_t*>(packed);
    if (n == 1) launch_staged<T, G, false>(T_, N, K, xt, stride, w, static_cast<T*>(y), per, n, st);
    else launch_staged<T, G, true>(T_, N, K, xt, stride, w, static_cast<T*>(y), per, n, st);
}

bool sizes_ok(int N, int K, int G) {
    return N >= 1 && N <= (1 << 20) && (G == 32 || G == 64 || G == 128) && K >= G && K % G == 0 && K <= (1 << 18);
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
    launch_pdl(k_w4_pack, dim3((N + 15) / 16, K / group), 32, 0, static_cast<cudaStream_t>(stream), N, K, group,
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
