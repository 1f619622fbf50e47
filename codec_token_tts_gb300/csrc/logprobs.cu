// Log probabilities of given tokens, entropy, log-sum-exp and the most probable tokens of logits rows.
//
// With m the row's largest logit at its lowest id i*, r = sum over the other ids of exp(z - m) and t = sum over
// them of exp(z - m) (z - m):
//   lse = m + log1p(r),  log p(i) = (z_i - m) - log1p(r),  H = log1p(r) - t / (1 + r)
// (the largest term, exactly 1, stays out of the sum, so a row sure of its answer keeps its digits).
// Order of the alternatives: the float's bits made monotone in the high word, the complement of the id in the low
// one: no two keys are equal, and the larger key is the larger logit or, among equals, the lower id.
#include <cuda_fp16.h>

#include <algorithm>
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

constexpr float LOG2E = 1.4426950408889634f;
constexpr unsigned ALL = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a part of a row amounts to: its largest logit m (NONE: nothing with probability), r and t as above, less the one
// term of m itself. Two parts are joined exactly so: with delta = the smaller m less the larger,
//   r = r1 + e^delta (1 + r2),  t = t1 + e^delta (t2 + delta (1 + r2))
constexpr float NONE = -INFINITY;
struct Part {
    float m, r, t;
    int bad;
};
__device__ __forceinline__ Part join(const Part& x, const Part& y) {
    const bool xy = x.m >= y.m;
    const Part &a = xy ? x : y, &b = xy ? y : x;
    Part o = {a.m, a.r, a.t, x.bad | y.bad};
    if (b.m > NONE) {
        const float d = b.m - a.m, e = ex2(d * LOG2E);
        if (e > 0.f) {  // else d may be so large (the type's lowest value) that its product overflows: 0 times an infinity
            o.r += e * (1.f + b.r);
            o.t += e * (b.t + d * (1.f + b.r));
        }
    }
    return o;
}
// the row's numbers; log_s: log1p(r), z: the target's logit
__device__ __forceinline__ void finish(const Args& a, int row, const Part& p, float log_s, bool wanted, float z) {
    const float nan = __int_as_float(0x7FC00000);
    const bool some = p.m > NONE;
    if (a.targets && a.logprob) a.logprob[row] = p.bad ? nan : some && wanted ? (z - p.m) - log_s : NEG_INF;
    if (a.entropy) a.entropy[row] = p.bad ? nan : some ? log_s - p.t / (1.f + p.r) : 0.f;
    if (a.lse) a.lse[row] = p.bad ? nan : some ? p.m + log_s : NEG_INF;
}
__device__ __forceinline__ void write_top(const Args& a, int row, int j, u64 key, const Part& p, float log_s) {
    const float nan = __int_as_float(0x7FC00000);
    a.top_ids[(size_t)row * a.n_top + j] = key && !p.bad ? id_of(key) : -1;
    a.top_lp[(size_t)row * a.n_top + j] = p.bad ? nan : key ? (value_of(key) - p.m) - log_s : NEG_INF;
}
template <typename T>
__device__ __forceinline__ bool target_of(const Args& a, const T* z, const uint32_t* ok, int row, float& v) {
    v = 0.f;
    if (!a.targets) return false;
    const int i = a.targets[row];
    if (i < 0 || i >= a.V || !is_allowed(ok, i)) return false;
    v = to_f(z[i]);
    return true;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
// two floats an instruction
typedef u64 f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void halves(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mulp(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 addp(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fmap(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// ---------------------------------------------------------------- one warp a row
// Rows of up to 32 * NV logits (NV even), held in registers: lane l has ids l, l + 32, .... One pass for the maximum, one for the
// sums, one that marks the alternatives: ids whose logit reaches the n_top-th largest of the 32 lanes' maxima (a bound below
// the n_top-th largest of all), usually a few more than n_top, ranked by counting. Near the least of the 32 maxima that bound
// gets loose (all 32 of 1025 ids: about 130 candidates): more than 12 alternatives start at place 0.7 n_top and halve their
// way to one that at least n_top and at most CAP ids reach (49152 x 1025, 32 alternatives: 75 us, 98 from the last place
// on; 20: 57 and 62).
// What bounds it are the instructions of these passes (49152 x 1025 fp32 with a mask and 5 alternatives: 47 us, 4.3 TB/s), so
// a pass is kept to what most rows need; and their number, since code that does not fit the instruction cache stalls: what
// few rows need is a loop over memory. These are rows with an allowed logit that is not within 1e30 (a NaN, an infinity, the
// type's lowest value: 49152 x 1025 with -inf in every row 444 us) and rows with more equal candidates than CAP.
constexpr int ROW_WARPS = 4, CAP = 96;
constexpr float OUT = -1e30f;  // stands for a masked logit

__device__ __forceinline__ float row_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
// One row by a warp, in loops over memory: any values.
template <typename T>
__device__ __noinline__ Part sums_of(const T* z, const uint32_t* ok, int V, int lane) {
    Part p = {NEG_INF, 0.f, 0.f, 0};
    bool bad = false;
    for (int i = lane; i < V; i += 32) {
        const float v = is_allowed(ok, i) ? to_f(z[i]) : NEG_INF;
        bad |= !(v < INFINITY);
        p.m = fmaxf(p.m, v);
    }
    p.m = warp_max(p.m);
    p.bad = __any_sync(ALL, bad);
    int same = 0;
    for (int i = lane; i < V; i += 32) {
        const float v = is_allowed(ok, i) ? to_f(z[i]) : NEG_INF, d = fmaxf(v - (p.m > NONE ? p.m : 0.f), -1e4f), e = ex2(d * LOG2E);
        p.t += e * d;
        if (d == 0.f) ++same;
        else p.r += e;
    }
    p.r = warp_sum(p.r) + (float)(__reduce_add_sync(ALL, same) - 1);
    p.t = warp_sum(p.t);
    return p;
}
// The n largest keys of a row, one after the other.
template <typename T>
__device__ __noinline__ void tops_of(const T* z, const uint32_t* ok, const Args& a, int row, const Part& p, int lane) {
    const float log_s = log1pf(p.r);
    u64 last = ~0ull;
    for (int j = 0; j < a.n_top; ++j) {
        if (last && !p.bad) {
            u64 k = 0;
            for (int i = lane; i < a.V; i += 32) {
                const float v = is_allowed(ok, i) ? to_f(z[i]) : NEG_INF;
                const u64 c = v > NEG_INF ? key_of(v, i) : 0ull;
                if (c < last && c > k) k = c;
            }
            last = warp_max_key(k);
        }
        if (lane == 0) write_top(a, row, j, last, p, log_s);
    }
}

template <typename T, int NV>
__global__ void __launch_bounds__(ROW_WARPS * 32) k_logprobs_warp(const T* __restrict__ logits, Args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ u64 found[ROW_WARPS][CAP];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int WORDS = (NV + 31) / 32;
    uint32_t mask[WORDS];  // this lane's ids of the row that are not masked: bit i of id 32 i + lane
    for (int row = blockIdx.x * ROW_WARPS + warp, turn = 0; row < a.R; row += gridDim.x * ROW_WARPS, ++turn) {
        const T* z = logits + (size_t)row * a.stride;
        const uint32_t* ok = a.allowed ? a.allowed + (size_t)row * a.allowed_stride : nullptr;
        if (turn == 0 || a.allowed_stride) {  // once for all rows
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                const int n = a.V - lane - 1024 * w;  // of the ids from 1024 w + lane on, in steps of 32
                mask[w] = n >= 993 ? 0xFFFFFFFFu : n > 0 ? (1u << ((n + 31) >> 5)) - 1u : 0u;
                if (ok) {
                    uint32_t bits = 0u;
#pragma unroll 8
                    for (int i = 32 * w; i < NV && i < 32 * w + 32; ++i)
                        if (i * 32 < a.V) bits |= (ok[i] >> lane & 1u) << (i & 31);
                    mask[w] &= bits;
                }
            }
        }
        float v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = mask[i / 32] >> (i & 31) & 1u ? to_f(z[i * 32 + lane]) : OUT;
        float tz;
        const bool wanted = target_of(a, z, ok, row, tz);
        float mine = v[0], most = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i += 2) {
            mine = max3(mine, v[i], v[i + 1]);
            most = max3_nan(most, fabsf(v[i]), fabsf(v[i + 1]));
        }
        const bool odd = !(most <= 1e30f);
        Part p = {row_max(mine), 0.f, 0.f, 0};
        if (__any_sync(ALL, odd) || p.m == OUT) {
            p = sums_of(z, ok, a.V, lane);
            if (lane == 0) finish(a, row, p, log1pf(p.r), wanted, tz);
            tops_of(z, ok, a, row, p, lane);
            continue;
        }
        f2 r2 = 0, t2 = 0;  // two zeros each
        const f2 m2 = pair(-p.m, -p.m), l2e = pair(LOG2E, LOG2E);
#pragma unroll
        for (int i = 0; i < NV; i += 2) {
            const f2 d = addp(pair(v[i], v[i + 1]), m2);
            float x0, x1;
            halves(mulp(d, l2e), x0, x1);
            const f2 e = pair(ex2(x0), ex2(x1));
            r2 = addp(r2, e);
            t2 = fmap(e, d, t2);
        }
        float r0, r1, t0, t1;
        halves(r2, r0, r1);
        halves(t2, t0, t1);
        p.r = warp_sum(r0 + r1) - 1.f;
        p.t = warp_sum(t0 + t1);
        if (p.r < 1.f) {  // the digits behind the 1: lost only in the lanes that hold m, whose logits the warp sums again without it
            const bool owner = mine == p.m;
            float rest = 0.f;
            int same = 0;
            for (unsigned b = __ballot_sync(ALL, owner); b; b &= b - 1)
                for (int i = lane * 32 + __ffs(b) - 1; i < a.V; i += 32 * 32) {
                    const float d = (is_allowed(ok, i) ? to_f(z[i]) : OUT) - p.m;
                    if (d == 0.f) ++same;
                    else rest += ex2(d * LOG2E);
                }
            p.r = warp_sum((owner ? 0.f : r0 + r1) + rest) + (float)(__reduce_add_sync(ALL, same) - 1);
        }
        const float log_s = log1pf(p.r);
        if (lane == 0) finish(a, row, p, log_s, wanted, tz);
        if (a.n_top == 0) continue;
        float bound = p.m, s = mine;
        int k = a.n_top - 1, few = -1, enough = k;  // places among the lanes' maxima; few: fewer than n_top reach it
        if (a.n_top <= 8) {  // the largest of the lanes' maxima taken out n_top - 1 times, equal ones together
            for (int j = 1; j < a.n_top; ++j) {
                if (s == bound) s = NEG_INF;
                bound = row_max(s);
            }
        } else {  // the lanes' maxima in falling order
#pragma unroll
            for (int m = 2; m <= 32; m <<= 1)
#pragma unroll
                for (int j = m >> 1; j; j >>= 1) {
                    const float o = __shfl_xor_sync(ALL, s, j);
                    s = ((lane & m) == 0) == ((lane & j) == 0) ? fmaxf(s, o) : fminf(s, o);
                }
            if (a.n_top > 12 && a.V > CAP) k = a.n_top * 7 / 10;
            bound = __shfl_sync(ALL, s, k);
        }
        uint32_t in[(NV + 31) / 32];
        int count, n;
        while (true) {
            bound = fmaxf(bound, OUT);
            count = 0;
#pragma unroll
            for (int w = 0; w < (NV + 31) / 32; ++w) {
                in[w] = 0u;
#pragma unroll
                for (int i = 32 * w; i < NV && i < 32 * w + 32; ++i)
                    if (v[i] >= bound) in[w] |= 1u << (i & 31);
                in[w] &= mask[w];  // an id that counts may be as low as OUT
                count += __popc(in[w]);
            }
            n = __reduce_add_sync(ALL, count);
            if (n < a.n_top && k < a.n_top - 1 && bound > OUT) {
                few = k;
                k = (k + enough + 1) / 2;
            } else if (n > CAP && a.n_top > 8 && k - few > 1) {
                enough = k;
                k = (few + k) / 2;
            } else {
                break;
            }
            bound = __shfl_sync(ALL, s, k);
        }
        if (n > CAP) {
            tops_of(z, ok, a, row, p, lane);
            continue;
        }
        int at = count;  // places of the lanes before this one, and of this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(ALL, at, o);
            if (lane >= o) at += u;
        }
        at -= count;
#pragma unroll
        for (int w = 0; w < (NV + 31) / 32; ++w)
            for (uint32_t b = in[w]; b; b &= b - 1) {
                const int i = (w * 32 + __ffs(b) - 1) * 32 + lane;
                found[warp][at++] = key_of(to_f(z[i]), i);
            }
        __syncwarp();
        for (int x = lane; x < n; x += 32) {
            const u64 k = found[warp][x];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += found[warp][j] > k;
            if (rank < a.n_top) write_top(a, row, rank, k, p, log_s);
        }
        for (int j = min(n, a.n_top) + lane; j < a.n_top; j += 32) write_top(a, row, j, 0ull, p, log_s);
        __syncwarp();  // before the next row's candidates
    }
}

// ---------------------------------------------------------------- a cluster a row
// A row cut into the slices of 1, 2, 4 or 8 blocks, each slice staged in shared memory (16-byte pieces where the row's alignment
// has them; the places before and behind it hold -inf, so that all of it is read in 16-byte pieces) and read three times
// there: maximum (masked ids become -inf in it), then sums and the candidates: logits that reach a bound below the n_top-th
// largest, at most LIST of them (with more equal ones, or where the only logits above -inf lie in few of the warps' places, one
// alternative after the other is looked for: 64 x 151676 with 1500 ids side by side, 20 alternatives 158 us). Block 0
// joins the slices. A few long rows are bound by the passes' latency (64 x 151676 bf16, 20 alternatives: 16 us, of which
// memory would take 3), many by the passes' instructions (2000 x 25000 fp32: 77 us, 2.6 TB/s).
constexpr int LIST = 1024, MAX_TOP = TTS_BB_LOGPROBS_MAX_TOP;
// A slice of SLICE_BYTES leaves room for two blocks an SM (2000 x 25000 fp32 in one slice 77 us, in slices of 48 KB 103). Threads of
// a block, by its slice: 128 up to SMALL_SLICE (16000 x 3100 fp32 77 us, by 256 threads 128; 64 x 100000 fp32 25 us by 128,
// 20 by 256), 512 beyond MEDIUM_SLICE, where fewer blocks share an SM (2000 x 25000 fp32 77 us, by 256 threads 88; 800 x 60000
// in slices of 60 KB 117 by 512, 95 by 256).
constexpr int SLICE_BYTES = 100 * 1024, MAX_SLICE_BYTES = 192 * 1024, SMALL_SLICE = 16 * 1024, MEDIUM_SLICE = 80 * 1024;

template <typename T> constexpr int EACH = 16 / sizeof(T);  // logits of a 16-byte piece
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[4], float) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8], bf16) { unpack8(u, v); }
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8], __half) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <int THREADS> struct Block {
    float f[THREADS / 32];
    float g[THREADS / 32];
    int count;
    u64 list[LIST];
    u64 top[MAX_TOP];
    Part part, parts[8];
};
template <int THREADS>
__device__ __forceinline__ u64 block_max_key(u64 k, u64* sm) {
    k = warp_max_key(k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = k;
    __syncthreads();
    k = sm[0];
    for (int w = 1; w < THREADS / 32; ++w) k = sm[w] > k ? sm[w] : k;
    return k;
}
template <typename V>
__device__ __forceinline__ V peer(const V* p, int rank) {  // *p in the shared memory of a block of the cluster
    static_assert(sizeof(V) == 4 || sizeof(V) == 8, "one word or two");
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    V v;
    if constexpr (sizeof(V) == 8) {
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(*reinterpret_cast<u64*>(&v)) : "r"(at) : "memory");
    } else {
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(*reinterpret_cast<uint32_t*>(&v)) : "r"(at) : "memory");
    }
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// grid R * n_parts; slice: a multiple of 32 logits
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_logprobs_block(const T* __restrict__ logits, Args a, int n_parts, int slice) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ Block<THREADS> sm;
    constexpr int E = EACH<T>;
    const int row = blockIdx.x / n_parts, part = blockIdx.x - row * n_parts, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* z = logits + (size_t)row * a.stride;
    const uint32_t* ok = a.allowed ? a.allowed + (size_t)row * a.allowed_stride : nullptr;
    const int i0 = part * slice, n = max(0, min(slice, a.V - i0));
    const T* src = z + i0;
    const int mis = (int)((uintptr_t)src % 16 / sizeof(T));  // the slice's first logit in its 16-byte piece
    const int pieces = n ? (mis + n + E - 1) / E : 0;
    T* const st = reinterpret_cast<T*>(stage);
    const T low = (T)NEG_INF;
    float tz = 0.f;
    const bool wanted = part == 0 && tid == 0 && target_of(a, z, ok, row, tz);
    if (tid == 0) sm.count = 0;
    // Staging, and the maximum on the way. Piece q holds the slice's logits q E - mis ..; the first and the last may be cut. A
    // thread later reads the pieces that it wrote.
    float mine = NEG_INF;
    const auto take = [&](int q, uint4 u) {
        float v[E];
        unpack(u, v, T{});
        if (ok) {
            const int i = i0 + q * E - mis, w = max(i, 0) >> 5;
            const uint32_t lo = ok[w], hi = (w + 1) * 32 < a.V ? ok[w + 1] : 0u;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int b = i + e - w * 32;  // 0 .. 38
                if (b >= 0 && !((b < 32 ? lo >> b : hi >> (b - 32)) & 1u)) {
                    v[e] = NEG_INF;
                    reinterpret_cast<T*>(&u)[e] = low;
                }
            }
        }
        *reinterpret_cast<uint4*>(st + q * E) = u;
#pragma unroll
        for (int e = 0; e < E; e += 2) mine = max3_nan(mine, v[e], v[e + 1]);
    };
    const int q0 = mis ? 1 : 0, q1 = (mis + n) / E;  // whole pieces
    int q = q0 + tid;
    for (; q + 3 * THREADS < q1; q += 4 * THREADS) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = ldg_nc_v4(src + (q + k * THREADS) * E - mis);
#pragma unroll
        for (int k = 0; k < 4; ++k) take(q + k * THREADS, u[k]);
    }
    for (; q < q1; q += THREADS) take(q, ldg_nc_v4(src + q * E - mis));
    // the cut ones: by the threads that the later passes give them to
    for (int c = 0; c < 2; ++c) {
        const int p = c ? q1 : 0;
        if ((c ? q1 >= pieces || (q1 == 0 && q0) : !q0) || (p + THREADS - q0) % THREADS != tid || !pieces) continue;
        uint4 u;
        T* const to = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = p * E - mis + e;
            to[e] = i >= 0 && i < n ? src[i] : low;
        }
        take(p, u);
    }
    const bool odd = !(mine < INFINITY);  // a NaN stays one
    const float wm = warp_max(mine);
    // the j-th largest of a warp's 32 maxima, j = n_top / warps rounded up: so many logits of each warp are that large, and
    // the least of these bounds is one for n_top of the slice. Of the warps whose lanes all have a piece (or the first).
    const int full = min(max(pieces / 32, 1), THREADS / 32);
    float bv = NEG_INF;
    if (a.n_top) {
        float s = mine;
#pragma unroll
        for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
            for (int j = k >> 1; j; j >>= 1) {
                const float o = __shfl_xor_sync(ALL, s, j);
                s = ((lane & k) == 0) == ((lane & j) == 0) ? fmaxf(s, o) : fminf(s, o);
            }
        bv = __shfl_sync(ALL, s, min((a.n_top - 1) / full, 31));
    }
    if (lane == 0) { sm.f[warp] = wm; sm.g[warp] = warp < full ? bv : INFINITY; }
    const int bad = __syncthreads_or(odd);
    Part p = {NEG_INF, 0.f, 0.f, bad};
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) p.m = fmaxf(p.m, sm.f[w]);
    bv = sm.g[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) bv = fminf(bv, sm.g[w]);
    const bool some = p.m > NONE, seek = a.n_top && some;
    bv = fmaxf(bv, -3.4028235e38f);  // -inf is no alternative
    // sums and candidates
    const float m = some ? p.m : 0.f;
    const int mine0 = (tid + q0) % THREADS;  // this thread's pieces: those of the staging
    f2 r2 = 0, t2 = 0;                       // two zeros each
    const f2 m2 = pair(-m, -m), l2e = pair(LOG2E, LOG2E);
    const bool look = seek && mine >= bv;
    for (int q = mine0; q < pieces; q += THREADS) {
        float v[E];
        unpack(*reinterpret_cast<const uint4*>(st + q * E), v, T{});
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float d0, d1, x0, x1;
            halves(addp(pair(v[e], v[e + 1]), m2), d0, d1);
            const f2 d = pair(fmaxf(d0, -1e30f), fmaxf(d1, -1e30f));  // not -inf: 0 times it
            halves(mulp(d, l2e), x0, x1);
            const f2 x = pair(ex2(x0), ex2(x1));
            r2 = addp(r2, x);
            t2 = fmap(x, d, t2);
        }
        if (look) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (v[e] >= bv) {
                    const int at = atomicAdd(&sm.count, 1);
                    if (at < LIST) sm.list[at] = key_of(v[e], i0 + q * E - mis + e);
                }
        }
    }
    const auto sum_up = [&](float x, float y, float& sx, float& sy) {
        x = warp_sum(x);
        y = warp_sum(y);
        __syncthreads();
        if (lane == 0) { sm.f[warp] = x; sm.g[warp] = y; }
        __syncthreads();
        sx = sy = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) { sx += sm.f[w]; sy += sm.g[w]; }
    };
    {
        float a0, a1, b0, b1;
        halves(r2, a0, a1);
        halves(t2, b0, b1);
        sum_up(a0 + a1, b0 + b1, p.r, p.t);
        p.r -= 1.f;
    }
    if (p.r < 1.f) {  // the digits behind the 1: once more without the largest
        float x = 0.f, same = 0.f;
        for (int q = mine0; q < pieces; q += THREADS) {
            float v[E];
            unpack(*reinterpret_cast<const uint4*>(st + q * E), v, T{});
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = fmaxf(v[e] - m, -1e30f);
                if (d == 0.f) same += 1.f;
                else x += ex2(d * LOG2E);
            }
        }
        float rest;
        sum_up(x, same, rest, p.r);
        p.r = rest + (p.r - 1.f);
    }
    // the slice's alternatives, in order
    if (a.n_top) {
        for (int j = tid; j < MAX_TOP; j += THREADS) sm.top[j] = 0ull;
        __syncthreads();
        const int found = seek ? sm.count : 0;
        if (found <= LIST) {
            for (int x = tid; x < found; x += THREADS) {
                const u64 k = sm.list[x];
                int rank = 0;
#pragma unroll 16
                for (int j = 0; j < found; ++j) rank += sm.list[j] > k;
                if (rank < a.n_top) sm.top[rank] = k;
            }
        } else {
            u64 last = ~0ull;
            for (int j = 0; j < a.n_top && last; ++j) {
                u64 k = 0;
                for (int q = mine0; q < pieces; q += THREADS) {
                    float v[E];
                    unpack(*reinterpret_cast<const uint4*>(st + q * E), v, T{});
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const u64 c = v[e] > NEG_INF ? key_of(v[e], i0 + q * E - mis + e) : 0ull;
                        if (c < last && c > k) k = c;
                    }
                }
                last = block_max_key<THREADS>(k, sm.list);
                if (tid == 0) sm.top[j] = last;
            }
        }
    }
    if (tid == 0) sm.part = p;
    if (n_parts == 1) {
        __syncthreads();
        const float log_s = log1pf(p.r);
        if (tid == 0) finish(a, row, p, log_s, wanted, tz);
        for (int j = tid; j < a.n_top; j += THREADS) write_top(a, row, j, sm.top[j], p, log_s);
        return;
    }
    cluster_sync();
    if (part == 0) {
        // all that is elsewhere at once
        const int total = n_parts * a.n_top;  // at most 256
        for (int x = tid; x < total; x += THREADS) sm.list[x] = peer(&sm.top[x % a.n_top], x / a.n_top);
        if (tid < n_parts) sm.parts[tid] = Part{peer(&sm.part.m, tid), peer(&sm.part.r, tid), peer(&sm.part.t, tid), peer(&sm.part.bad, tid)};
        __syncthreads();
        p = sm.parts[0];
        for (int s = 1; s < n_parts; ++s) p = join(p, sm.parts[s]);
        const float log_s = log1pf(p.r);
        if (tid == 0) finish(a, row, p, log_s, wanted, tz);
        if (a.n_top) {
            for (int j = tid; j < a.n_top; j += THREADS) write_top(a, row, j, 0ull, p, log_s);
            __syncthreads();
            for (int x = tid; x < total; x += THREADS) {
                const u64 k = sm.list[x];
                if (!k) continue;
                int rank = 0;
#pragma unroll 16
                for (int j = 0; j < total; ++j) rank += sm.list[j] > k;
                if (rank < a.n_top) write_top(a, row, rank, k, p, log_s);
            }
        }
    }
    cluster_sync();  // no block leaves while another reads its slice's results
}

// ---------------------------------------------------------------- rows longer than 8 slices of shared memory
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

// grid R, THREADS threads: one row each; a pass for the maximum, one for the sums, one for each alternative.
template <typename T>
__global__ void __launch_bounds__(THREADS) k_logprobs_long(const T* __restrict__ logits, Args a) {
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
    best = block_max_key<THREADS>(best, smk);
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
    const Part p = {best ? m : NONE, r, t, bad};
    const float log_s = log1pf(r);
    if (tid == 0) {
        float tz;
        const bool wanted = target_of(a, z, ok, row, tz);
        finish(a, row, p, log_s, wanted, tz);
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
            last = block_max_key<THREADS>(k, smk);
        }
        if (tid == 0) write_top(a, row, j, last, p, log_s);
    }
}

// launch_pdl with clusters of n blocks, and shared memory beyond the default
template <typename T, int TH>
void launch_block(const T* logits, const Args& a, int n, int slice, cudaStream_t st) {
    const size_t smem = (size_t)slice * sizeof(T) + 16;
    static SmemState state;
    if (smem + sizeof(Block<TH>) > 48 * 1024) allow_smem(state, k_logprobs_block<T, TH>, MAX_SLICE_BYTES + 16);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = n;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.R * n));
    cfg.blockDim = TH;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = n > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, k_logprobs_block<T, TH>, logits, a, n, slice);
}

// Many rows of up to 96 logits a lane: a warp each (below 4 warps an SM a row's latency counts, and a block's threads
// share it: 600 x 2048 bf16, masked, 5 alternatives 5.7 us, by warps 6.8). Else a block a row, or a cluster: slices of at most
// SLICE_BYTES, and more, shorter ones while the rows alone leave SMs idle.
template <typename T>
void launch(const T* logits, const Args& a, cudaStream_t st) {
    // as many blocks as fit at a time: a warp goes on with further rows, and takes the mask apart once
    const auto warps = [&](auto k, int fit) {
        launch_pdl(k, std::min((a.R + ROW_WARPS - 1) / ROW_WARPS, fit * 152), ROW_WARPS * 32, 0, st, logits, a);
    };
    if (a.R >= 4 * 152 || a.V <= 256) {
        if (a.V <= 8 * 32) return warps(k_logprobs_warp<T, 8>, 10);
        if (a.V <= 34 * 32) return warps(k_logprobs_warp<T, 34>, 8);
        if (a.V <= 64 * 32) return warps(k_logprobs_warp<T, 64>, 4);
        if (a.V <= 96 * 32) return warps(k_logprobs_warp<T, 96>, 3);
    }
    const long long bytes = (long long)a.V * sizeof(T);
    int n = 1;
    while (n < 8 && (bytes > (long long)n * SLICE_BYTES || (a.R * n < 2 * 152 && bytes > n * 8192))) n *= 2;
    const int slice = ((a.V + n - 1) / n + 31) / 32 * 32;
    if ((long long)slice * sizeof(T) > MAX_SLICE_BYTES)
        launch_pdl(k_logprobs_long<T>, a.R, THREADS, 0, st, logits, a);
    else if ((long long)slice * sizeof(T) <= SMALL_SLICE)
        launch_block<T, 128>(logits, a, n, slice, st);
    else if ((long long)slice * sizeof(T) <= MEDIUM_SLICE)
        launch_block<T, 256>(logits, a, n, slice, st);
    else
        launch_block<T, 512>(logits, a, n, slice, st);
}

}  // namespace

TTS_API size_t tts_bb_token_logprobs_workspace(int, int, int) { return 0; }  // no sizes need any

TTS_API tts_bb_status tts_bb_token_logprobs(int R, int V, const void* logits, int type, int64_t row_stride,
                                            const int32_t* targets, const uint32_t* allowed, int64_t allowed_stride,
                                            int n_top, float* logprob, float* entropy, float* lse, int32_t* top_ids,
                                            float* top_logprobs, void* /*workspace*/, size_t /*workspace_bytes*/, void* stream) {
    if (R < 1 || R > (1 << 27) || V < 1 || V > (1 << 30) || !logits || row_stride < V || n_top < 0 || n_top > TTS_BB_LOGPROBS_MAX_TOP ||
        type < TTS_BB_T_F32 || type > TTS_BB_T_F16 || (uintptr_t)logits % (type == TTS_BB_T_F32 ? 4 : 2) ||
        (targets && !logprob) || (n_top && (!top_ids || !top_logprobs)) ||
        (allowed && allowed_stride != 0 && allowed_stride < ((int64_t)V + 31) / 32) ||
        !words_aligned(targets, allowed, logprob, entropy, lse, top_ids, top_logprobs))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Args a{R, V, n_top, row_stride, allowed_stride, targets, allowed, logprob, entropy, lse, top_ids, top_logprobs};
    if (type == TTS_BB_T_F32) launch(static_cast<const float*>(logits), a, st);
    else if (type == TTS_BB_T_BF16) launch(static_cast<const bf16*>(logits), a, st);
    else launch(static_cast<const __half*>(logits), a, st);
    return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA;
}
