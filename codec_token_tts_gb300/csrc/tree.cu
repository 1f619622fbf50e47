// Verification of a tree of drafted tokens against the target's probabilities, and the accepted path's keys and
// values into the caches of all layers.
//
// Verification. With r_0 = p and Z_0 = 1, a rejected child leaves r_{k+1} = (r_k - Z_k q)^+. Since Z_k q >= 0 and r_k is
// either 0 or p - c_k q, this is r_{k+1} = (p - c_{k+1} q)^+ with the one number c_{k+1} = c_k + Z_k: no array is kept
// between rejections, and each costs one pass over the rows p and q that sums r. Children's indices lie above their
// parent's, so one walk over the nodes in their order meets each accepted node's children in turn.
//
// Sums decide which whole number is the answer, so they have to hold far more bits than a float. A thread adds its ids' rests in pairs of
// floats (the sum, and what its roundings left; two ids an instruction: 2^-48 of the sum and less, of the tens of ids that a thread has of
// 151676); between threads they are whole numbers of 2^-60, whose order does not matter. Up to 16384 threads' halves are cut off there,
// so a sum is off by 2^-46 of the row's 1 at most, however little is left, and c by that for each rejection. The ids around the answer are
// then gone through in whole numbers of 2^-60 alone: exact for probabilities from 2^-37 up (24 bits above 2^-60), cut off at 2^-60 below that.
#include <algorithm>

#include "tree.cuh"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

typedef unsigned long long u64;

constexpr int MAX_CLUSTER = 16, THREADS_SM = 1024;
// Ids that one block takes; below that it has fewer threads, whose barriers cost less and of which more sequences' are at work at a time
// (64 x 2048, chosen drafts, 25 nodes: 7.2 us, by 512 threads 7.9; 1000 x 2048, drawn, 6 nodes: 16.3 and 25.7; 700 x 30000: 61 and 55).
constexpr int BLOCK_IDS = 4096, THREADS = 512, THREADS_SMALL = 256;

// a probability's bits, within 0 .. 1 (a NaN counts as 1, or as 0 where its sign is set)
__device__ __forceinline__ uint32_t prob_bits(float x) { return (uint32_t)min(max(__float_as_int(x), 0), 0x3F800000); }
// in units of 2^-60: the mantissa of 1 has its bit 60, that of others stands 127 - exponent lower
__device__ __forceinline__ u64 fix60(float x) {
    const uint32_t b = prob_bits(x), s = 127 - (b >> 23);
    const u64 m = (u64)((b << 5 & 0x0FFFFFFFu) | 0x10000000u) << 32;
    return s < 64 ? m >> s : 0ull;
}
// a * b / 2^s
__device__ __forceinline__ u64 mul_shift(u64 a, u64 b, int s) { return (__umul64hi(a, b) << (64 - s)) | (a * b >> s); }
// what c (in 2^-58) times q leaves of p: nothing where the product is 16 or more, which is beyond 64 bits (c grows by up to 1 with each of
// up to 63 rejections, and q may be 1)
__device__ __forceinline__ u64 rest60(u64 p, u64 c, u64 q) {
    if (__umul64hi(c, q) >> 58) return 0ull;
    const u64 t = mul_shift(c, q, 58);
    return p > t ? p - t : 0ull;
}

// a pair of floats in units of 2^-60 (0 below 0 or where it is not a number, 8 at most)
__device__ __forceinline__ u64 pair60(float s, float rest) {
    const auto fix = [](float x) {  // 0 <= x < 16
        const uint32_t b = __float_as_uint(x), e = b >> 23;
        const u64 m = (b & 0x7FFFFFu) | 0x800000u;
        return e >= 90 ? m << (e - 90) : e > 66 ? m >> (90 - e) : 0ull;
    };
    // s may be 0 beside a rest, or below it
    const float t = s + rest, z = t - s, y = (s - (t - z)) + (rest - z);
    if (!(t > 0.f)) return 0ull;
    const u64 a = fix(fminf(t, 8.f)), d = fix(fminf(fabsf(y), 1.f));
    return y < 0.f ? (a > d ? a - d : 0ull) : a + d;
}
// two floats an instruction
__device__ __forceinline__ u64 both(float a, float b) {
    u64 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void halves(u64 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ u64 sub2(u64 a, u64 b) { return fma2(b, both(-1.f, -1.f), a); }
// (s, rest) += x and the small y: the rounding of s + x goes to rest (Knuth's two-sum)
__device__ __forceinline__ void gather2(u64& s, u64& rest, u64 x, u64 y) {
    const u64 t = add2(s, x), z = sub2(t, s);
    rest = add2(rest, add2(add2(sub2(s, sub2(t, z)), sub2(x, z)), y));
    s = t;
}
// p - q of two ids where that is above 0: what rounds off p - min(p, q) is exact too
__device__ __forceinline__ void rest2(u64& s, u64& rest, float p0, float p1, float q0, float q1) {
    const u64 p = both(p0, p1), q = both(fminf(p0, q0), fminf(p1, q1)), d = sub2(p, q);
    gather2(s, rest, d, sub2(sub2(p, d), q));
}
// p - c q where that is above 0, c = (hi, lo): the sign is that of the sum, since c q may lie to either side of what it rounds to
__device__ __forceinline__ void rest2(u64& s, u64& rest, float p0, float p1, float q0, float q1, u64 hi, u64 lo) {
    const u64 p = both(p0, p1), q = both(q0, q1), h = mul2(hi, q);
    const u64 l = fma2(lo, q, fma2(hi, q, mul2(h, both(-1.f, -1.f))));  // what h rounded off, and lo q
    const u64 d = sub2(p, h), e = sub2(sub2(sub2(p, d), h), l);
    float t0, t1, d0, d1, e0, e1;
    halves(add2(d, e), t0, t1);
    halves(d, d0, d1);
    halves(e, e0, e1);
    if (t0 <= 0.f) d0 = e0 = 0.f;
    if (t1 <= 0.f) d1 = e1 = 0.f;
    gather2(s, rest, both(d0, d1), both(e0, e1));
}
// ids x .. x + 3 of a row of V, 0 for those outside
__device__ __forceinline__ float4 four(const float* row, int x, int V) {
    return make_float4(x >= 0 && x < V ? row[x] : 0.f, x >= -1 && x < V - 1 ? row[x + 1] : 0.f, x >= -2 && x < V - 2 ? row[x + 2] : 0.f,
                       x < V - 3 ? row[x + 3] : 0.f);
}
// f(x, p[x .. x + 3], q[x .. x + 3]) for a lane's ids of first .. last - 1, whole and aligned where `vec` (q may be null)
template <typename F>
__device__ __forceinline__ void for_ids(const float* p, const float* q, int first, int last, int V, int lane, bool vec, F f) {
    int x = first + lane * 4;
    const auto guarded = [&] { f(x, four(p, x, V), q ? four(q, x, V) : make_float4(0.f, 0.f, 0.f, 0.f)); };
    if (vec) {
        if (first < 0) {
            guarded();
            x += 128;
        }
        const int end = min(last, V) - 4;
#pragma unroll 4
        for (; x <= end; x += 128)
            f(x, *reinterpret_cast<const float4*>(p + x), q ? *reinterpret_cast<const float4*>(q + x) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
#pragma unroll 1
    for (; x < last && x < V; x += 128) guarded();
}
// a whole number of 2^-s as a pair of floats
__device__ __forceinline__ void pair_of(u64 v, float unit, float& hi, float& lo) {
    hi = __ull2float_rn(v);
    lo = (float)(long long)(v - __float2ull_rz(hi)) * unit;
    hi *= unit;
}
// Whether u q Z < p - c q, for pairs of floats Z and c (48 bits; exact where Z is 1 and c is 0).
__device__ __forceinline__ bool accepts(float u, float q, float zh, float zl, float p, float ch, float cl) {
    const float a = u * q, a1 = fmaf(u, q, -a), b = a * zh, b1 = fmaf(a, zh, -b) + fmaf(a, zl, a1 * zh);
    const float h = ch * q, l = fmaf(ch, q, -h) + cl * q;
    const float t = p - h, z = t - p, e = (p - (t - z)) - (h + z) - l;  // t + e = p - c q
    return (b - t) + (b1 - e) < 0.f;
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_peer(u64* p, int rank, u64 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

struct VerifyArgs {
    const int32_t *tokens, *parents, *n_nodes;
    const float *target, *draft, *u, *u_next;
    long long p_stride, q_stride;
    int32_t *n_accepted, *path, *next, *err;
    int N, V, ctas, seg;  // blocks of a cluster, ids of a warp
};

// The nodes of sequence b, 0 where it is padding or out of order (by one warp, lanes hold nodes l and l + 32).
__device__ __forceinline__ int tree_nodes(const int32_t* n_nodes, int b, int N, int lane, const int (&par)[2], int32_t* err, bool report) {
    const int n = n_nodes ? n_nodes[b] : N;
    if (n < 0 || n > N) {
        if (report && lane == 0) set_err(err, TTS_BB_TREE_ERR_RANGE);
        return 0;
    }
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) bad |= lane + 32 * h < n && (par[h] < -1 || par[h] >= lane + 32 * h);
    if (__any_sync(0xffffffffu, bad)) {
        if (report && lane == 0) set_err(err, TTS_BB_TREE_ERR_TREE);
        return 0;
    }
    return n;
}
// Count and nodes of the chosen path, by one warp.
__device__ __forceinline__ void write_path(u64 chosen, int b, int N, int lane, int32_t* n_accepted, int32_t* path) {
    const int count = __popcll(chosen);
    if (lane == 0) n_accepted[b] = count;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        const u64 below = (1ull << j) - 1;
        if (j >= N) continue;
        if (chosen >> j & 1) path[(size_t)b * N + __popcll(chosen & below)] = j;
        if (j >= count) path[(size_t)b * N + j] = -1;
    }
}

enum { WALK_PASS, WALK_LAST };

struct VerifyShared {
    int par[MAX_NODES], tok[MAX_NODES];
    float p[MAX_NODES], q[MAX_NODES], u[MAX_NODES];
    u64 wsum[THREADS / 32];
    u64 tot[2][MAX_CLUSTER];  // the blocks' sums of a pass, by its parity
    u64 chosen, gone;         // accepted nodes; rejected children of the current node (drafts that were not drawn)
    u64 c;                    // 2^-58
    float hi, lo;             // c
    int found;                // the last id that is left where the whole numbers end before the sum does
    int n, cur, event;
};

// grid (ctas, B), a cluster of ctas blocks for each sequence. Block r of a cluster owns the ids
// [r, r + 1) * NWARPS * seg, warp w of it seg of them.
template <bool DRAWN, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS_SM / THREADS) k_tree_verify(VerifyArgs a) {
    constexpr int NWARPS = THREADS / 32;
    __shared__ VerifyShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y, rank = blockIdx.x;
    const bool many = a.ctas > 1;
    if (many) cluster_arrive();  // waited for before the first word goes to a peer
    pdl_wait();
    pdl_trigger();
    const float u_next = a.u_next[b];
    if (warp == 0) {
        int par[2], tok[2];
        float u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // one wait for all
            const int j = lane + 32 * h;
            const size_t at = (size_t)b * a.N + j;
            par[h] = j < a.N ? a.parents[at] : -1;
            tok[h] = j < a.N ? a.tokens[at] : -1;
            u[h] = j < a.N ? a.u[at] : 0.f;
        }
        const int n = tree_nodes(a.n_nodes, b, a.N, lane, par, a.err, rank == 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            if (j >= n) continue;
            // what the target and the draft of its parent give the node's token
            const int x = tok[h];
            const bool real = x >= 0 && x < a.V && par[h] >= 0;
            const size_t row = (size_t)b * a.N + max(par[h], 0);
            sh.par[j] = par[h];
            sh.tok[j] = real ? x : -1;
            sh.u[j] = u[h];
            sh.p[j] = real ? __uint_as_float(prob_bits(a.target[row * a.p_stride + x])) : 0.f;
            if (DRAWN) sh.q[j] = real ? __uint_as_float(prob_bits(a.draft[row * a.q_stride + x])) : 0.f;
        }
        if (lane == 0) {
            if (rank == 0) a.next[b] = n ? 0 : -1;  // some id, whatever the numbers are
            sh.n = n;
        }
    }
    __syncthreads();
    if (many) cluster_wait();
    const int n = sh.n;
    if (n == 0) {  // for all blocks of the cluster
        if (rank == 0 && warp == 0) write_path(0, b, a.N, lane, a.n_accepted, a.path);
        return;
    }
    const int at0 = (rank * NWARPS + warp) * a.seg;  // ids of this warp, but for the row's alignment
    u64 Z = 0;
    int parity = 0;
    // the walk's state, in warp 0: the nodes that have not been looked at, the children among them that may be accepted
    u64 chosen = 1, gone = 0, ahead = ~1ull, c58 = 0;
    int cur = 0;
    bool summed = false;  // the block's sums are those of node cur's rest as it stands
    const bool able[2] = {lane < n && sh.tok[lane] >= 0, lane + 32 < n && sh.tok[lane + 32] >= 0};
    const int parent[2] = {lane < n ? sh.par[lane] : -1, lane + 32 < n ? sh.par[lane + 32] : -1};
    for (;;) {
        if (warp == 0) {
            // the mass that the next child is measured by: Z of the pass before, 1 less the rejected ones, or 1
            float zh = 1.f, zl = 0.f, ch = 0.f, cl = 0.f;
            if (DRAWN && c58) {
                pair_of(Z, 0x1p-60f, zh, zl);
                pair_of(c58, 0x1p-58f, ch, cl);
            }
            int event = WALK_LAST;
            u64 mass = 1ull << 60;
            for (;;) {
                u64 kids = (u64)__ballot_sync(0xffffffffu, able[1] && parent[1] == cur) << 32 | __ballot_sync(0xffffffffu, able[0] && parent[0] == cur);
                kids &= ahead;
                if (!kids) break;
                const int j = __ffsll(kids) - 1;
                ahead = ~0ull << j << 1;
                const float p = sh.p[j];
                bool again = false;  // a token that was rejected here before
                if (!DRAWN) {
#pragma unroll 1
                    for (u64 g = gone; g; g &= g - 1) again |= sh.tok[__ffsll(g) - 1] == sh.tok[j];
                }
                if (!again && accepts(sh.u[j], DRAWN ? sh.q[j] : 1.f, zh, zl, p, ch, cl)) {
                    chosen |= 1ull << j;
                    cur = j;
                    c58 = gone = 0;
                    mass = 1ull << 60;
                    zh = 1.f;
                    zl = ch = cl = 0.f;
                    summed = false;
                } else if (DRAWN) {
                    const u64 more = c58 ? Z >> 2 : 1ull << 58;
                    c58 = c58 + more < c58 ? ~0ull : c58 + more;
                    event = WALK_PASS;
                    break;
                } else if (!again) {
                    gone |= 1ull << j;
                    mass -= min(mass, fix60(p));
                    pair_of(mass, 0x1p-60f, zh, zl);
                }
            }
            // the path's end: the sums are there where the last pass was of this node's rest
            if (event == WALK_LAST && summed) event = WALK_LAST + 1;
            summed = true;
            if (lane == 0) {
                pair_of(c58, 0x1p-58f, sh.hi, sh.lo);
                sh.c = c58;
                sh.chosen = chosen;
                sh.gone = gone;
                sh.cur = cur;
                sh.event = event;
            }
        }
        __syncthreads();
        const int event = sh.event;
        if (event > WALK_LAST) break;
        // sums of the rest of node cur
        const u64 c = sh.c;
        const size_t row = (size_t)b * a.N + sh.cur;
        const float* const p = a.target + row * a.p_stride;
        const float* const q = DRAWN ? a.draft + row * a.q_stride : nullptr;
        // ids from a whole 16 bytes of both rows on
        const bool vec = !DRAWN || (((uintptr_t)p ^ (uintptr_t)q) & 15) == 0;
        const int first = at0 - (vec ? (int)((uintptr_t)p >> 2 & 3) : 0), last = first + a.seg;
        u64 s = 0, rest = 0;
        if (!DRAWN || c == 0) {
            for_ids(p, nullptr, first, last, a.V, lane, vec, [&](int, float4 f, float4) {
                gather2(s, rest, both(f.x, f.y), 0ull);
                gather2(s, rest, both(f.z, f.w), 0ull);
            });
        } else if (c == 1ull << 58) {
            for_ids(p, q, first, last, a.V, lane, vec, [&](int, float4 f, float4 g) {
                rest2(s, rest, f.x, f.y, g.x, g.y);
                rest2(s, rest, f.z, f.w, g.z, g.w);
            });
        } else {
            const u64 hi = both(sh.hi, sh.hi), lo = both(sh.lo, sh.lo);
            for_ids(p, q, first, last, a.V, lane, vec, [&](int, float4 f, float4 g) {
                rest2(s, rest, f.x, f.y, g.x, g.y, hi, lo);
                rest2(s, rest, f.z, f.w, g.z, g.w, hi, lo);
            });
        }
        float s0, s1, r0, r1;
        halves(s, s0, s1);
        halves(rest, r0, r1);
        u64 sum = pair60(s0, r0) + pair60(s1, r1);
        sum = warp_sum64(sum);
        if (!DRAWN && lane == 0) {  // less the rejected tokens, each once
            for (u64 g = sh.gone; g; g &= g - 1) {
                const int j = __ffsll(g) - 1, x = sh.tok[j];
                if (x >= first && x < last) sum -= min(sum, fix60(sh.p[j]));
            }
        }
        if (lane == 0) sh.wsum[warp] = sum;
        __syncthreads();
        u64 block = lane < NWARPS ? sh.wsum[lane] : 0ull;
        block = warp_sum64(block);
        if (many) {
            if (tid < a.ctas) store_peer(&sh.tot[parity][rank], tid, block);
            cluster_arrive();
            cluster_wait();
            Z = 0;
            for (int i = 0; i < a.ctas; ++i) Z += sh.tot[parity][i];
        } else {
            if (tid == 0) sh.tot[parity][0] = block;
            Z = block;
            __syncthreads();
        }
        parity ^= 1;
        if (event == WALK_LAST) break;
    }
    // the next token
    parity ^= 1;
    const u64 c = sh.c;
    const size_t row = (size_t)b * a.N + sh.cur;
    const float* const p = a.target + row * a.p_stride;
    const float* const q = DRAWN ? a.draft + row * a.q_stride : nullptr;
    if (rank == 0 && warp == 0) write_path(sh.chosen, b, a.N, lane, a.n_accepted, a.path);
    if (Z) {
        u64 t = mul_shift(fix60(u_next), Z, 60);
        if (t >= Z) t = Z - 1;  // u_next of 1
        for (int i = 0; i < rank; ++i) {
            if (t < sh.tot[parity][i]) return;  // in a block before this one
            t -= sh.tot[parity][i];
        }
        // in this block: the warp whose ids it lies among, which all warps search together, 4 ids a thread at a time
        u64 upto = lane < NWARPS ? sh.wsum[lane] : 0ull;
        const u64 own = upto;
#pragma unroll
        for (int o = 1; o < NWARPS; o <<= 1) {
            const u64 w = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += w;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, lane < NWARPS && upto > t);
        if (!over) return;  // in a block behind this one
        const bool vec = !DRAWN || (((uintptr_t)p ^ (uintptr_t)q) & 15) == 0;
        const int in = __ffs(over) - 1, from = (rank * NWARPS + in) * a.seg - (vec ? (int)((uintptr_t)p >> 2 & 3) : 0), to = min(a.V, from + a.seg);
        t -= __shfl_sync(0xffffffffu, upto - own, in);
        int seen = max(from, 0);  // of this thread's ids the last one that is left
        for (int x0 = from; x0 < to; x0 += THREADS * 4) {
            u64 r[4], mine = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = x0 + tid * 4 + i;
                r[i] = x >= 0 && x < to ? fix60(p[x]) : 0ull;
                if (DRAWN) {
                    if (c && x >= 0 && x < to) r[i] = rest60(r[i], c, fix60(q[x]));
                } else {
                    for (u64 g = sh.gone; g; g &= g - 1)
                        if (sh.tok[__ffsll(g) - 1] == x) r[i] = 0;
                }
                if (r[i]) seen = x;
                mine += r[i];
            }
            u64 incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 w = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += w;
            }
            __syncthreads();
            if (lane == 31) sh.wsum[warp] = incl;
            __syncthreads();
            u64 all = lane < NWARPS ? sh.wsum[lane] : 0ull;
            const u64 before_me = all;
#pragma unroll
            for (int o = 1; o < NWARPS; o <<= 1) {
                const u64 w = __shfl_up_sync(0xffffffffu, all, o);
                if (lane >= o) all += w;
            }
            u64 at = __shfl_sync(0xffffffffu, all - before_me, warp) + incl - mine;
            const u64 total = __shfl_sync(0xffffffffu, all, NWARPS - 1);
            if (t >= at && t < at + mine) {
                int i = 0;
                while (t >= at + r[i]) at += r[i++];
                a.next[b] = x0 + tid * 4 + i;
            }
            if (t < total) return;
            t -= total;
        }
        // the floats' sum ends 2^-46 behind the whole numbers': the last id
        if (tid == 0) sh.found = 0;
        __syncthreads();
        atomicMax(&sh.found, seen);
        __syncthreads();
        if (tid == 0) a.next[b] = sh.found;
        return;
    }
    // nothing is left: the most probable token of p. Keys order by value, then by the lowest id
    u64 best = 0;
    for (int x = at0 + lane; x < min(a.V, at0 + a.seg); x += 32) best = max(best, (u64)prob_bits(p[x]) << 32 | (uint32_t)~x);
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) sh.wsum[warp] = best;
    __syncthreads();
    best = lane < NWARPS ? sh.wsum[lane] : 0ull;
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (many) {
        parity ^= 1;
        if (tid == 0) store_peer(&sh.tot[parity][rank], 0, best);
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        for (int i = 0; i < a.ctas; ++i) best = max(best, sh.tot[parity][i]);
    }
    if (rank == 0 && tid == 0) a.next[b] = (int)~(uint32_t)best;
}

// a warp a sequence
constexpr int GREEDY_WARPS = 4;
__global__ void __launch_bounds__(GREEDY_WARPS * 32) k_tree_greedy(VerifyArgs a, const int32_t* __restrict__ ids, int B) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x * GREEDY_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= B) return;
    int par[2], tok[2], id[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        const size_t at = (size_t)b * a.N + j;
        par[h] = j < a.N ? a.parents[at] : -1;
        tok[h] = j < a.N ? a.tokens[at] : 0;
        id[h] = j < a.N ? ids[at] : 0;
    }
    const int n = tree_nodes(a.n_nodes, b, a.N, lane, par, a.err, true);
    u64 chosen = n ? 1 : 0;
    int cur = 0, want = __shfl_sync(0xffffffffu, id[0], 0);
    for (int step = 0; step < n; ++step) {  // a path is no longer than the tree
        uint32_t hit[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) hit[h] = __ballot_sync(0xffffffffu, lane + 32 * h < n && par[h] == cur && tok[h] == want);
        if (!(hit[0] | hit[1])) break;
        cur = hit[0] ? __ffs(hit[0]) - 1 : 31 + __ffs(hit[1]);
        chosen |= 1ull << cur;
        want = __shfl_sync(0xffffffffu, cur < 32 ? id[0] : id[1], cur & 31);
    }
    write_path(chosen, b, a.N, lane, a.n_accepted, a.path);
    if (lane == 0) a.next[b] = n ? want : -1;
}

struct CommitArgs {
    const bf16 *k, *v;
    long long row_stride, layer_stride;
    const int32_t *path, *n_accepted, *seqs, *kv_lens;
    int N;
};
// grid (layers, B), 128 threads: 16 bytes of K and of V each, COMMIT tokens at a time, whose nodes, pages and values are each asked for
// at once (three waits). Bound by memory: 28 layers x 64 sequences, 288 tokens, each a row of K and V of 2 KB that is read whole and
// written as 256 bytes a head: 13.7 us, 4.8 TB/s read and written (2 tokens 13.9, 8 15.1; a row by 256 threads, token by token, 15.9)
constexpr int COMMIT = 4;
__global__ void __launch_bounds__(128) k_tree_commit(Pages c, CommitArgs a) {
    pdl_wait();
    pdl_trigger();
    const int l = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int row = row_of(c, a.seqs, b), n = a.n_accepted[b], len = a.kv_lens[b];
    const bool report = l == 0 && tid == 0;
    if (row == -1) return;
    if (row < 0 || n < 0 || n > a.N || len < 0) {
        if (report) set_err(c.err, TTS_BB_TREE_ERR_RANGE);
        return;
    }
    const long long from = l * a.layer_stride + tid * 8;
    bf16* const to = c.pool + l * c.layer_stride + (size_t)(tid >> 4) * (KVB * HD) + (tid & 15) * 8;
    const long long room = (long long)c.bps * KVB;
    for (int j0 = 0; j0 < n; j0 += COMMIT) {
        int node[COMMIT], page[COMMIT];
        uint4 x[COMMIT][2];
#pragma unroll
        for (int i = 0; i < COMMIT; ++i) {
            const long long pos = (long long)len + j0 + i;
            const bool in = j0 + i < n && pos < room;
            node[i] = in ? a.path[(size_t)b * a.N + j0 + i] : -1;
            page[i] = in ? c.table[(size_t)row * c.bps + pos / KVB] : -1;
            if (report && j0 + i < n && pos >= room) set_err(c.err, TTS_BB_TREE_ERR_RANGE);
        }
#pragma unroll
        for (int i = 0; i < COMMIT; ++i) {
            const bool in = j0 + i < n && (long long)len + j0 + i < room, known = node[i] >= 0 && node[i] < a.N, there = page[i] >= 0 && page[i] < c.n_blocks;
            if (report && in && !(known && there)) set_err(c.err, known ? TTS_BB_TREE_ERR_PAGE : TTS_BB_TREE_ERR_TREE);
            if (!known || !there) {
                page[i] = -1;
                continue;
            }
            const long long at = from + ((long long)b * a.N + node[i]) * a.row_stride;
            x[i][0] = *reinterpret_cast<const uint4*>(a.k + at);
            x[i][1] = *reinterpret_cast<const uint4*>(a.v + at);
        }
#pragma unroll
        for (int i = 0; i < COMMIT; ++i) {
            if (page[i] < 0) continue;
            bf16* const at = to + page[i] * KV_BLOCK + (size_t)(((unsigned)len + j0 + i) % KVB) * HD;
            *reinterpret_cast<uint4*>(at) = x[i][0];
            *reinterpret_cast<uint4*>(at + KV_BLOCK / 2) = x[i][1];
        }
    }
}

// Blocks of a sequence's cluster: one for each BLOCK_IDS, while all sequences' blocks run in two turns, so that what a walk's end leaves free
// is taken. Drawn drafts of 151676 ids, 64 x 12 nodes: 39.7 us, in one turn (4 blocks a sequence) 44.7, in four (16) 54.9; 128 x 6 nodes 55,
// 71 and 61. Walks of a pass or two, and shorter rows, would rather have one turn: chosen drafts, 64 x 12 nodes 23.1 us, 17.1 and 39.4;
// drawn, 32 x 12 nodes 32.2, 28.2 and 32.1; 64 x 12 nodes of 30000 ids 23.4, 17.9 and 23.4.
int verify_ctas(int B, int V) {
    int n = 1;
    while (n < MAX_CLUSTER && n * BLOCK_IDS < V && 2 * n * B <= 2 * (THREADS_SM / THREADS) * 152) n *= 2;
    return n;
}

}  // namespace

TTS_API tts_bb_status tts_bb_tree_verify(int B, int N, int V, const int32_t* tokens, const int32_t* parents, const int32_t* n_nodes,
                                         const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                                         const float* u, const float* u_next, int32_t* n_accepted, int32_t* path,
                                         int32_t* next_token, int32_t* err, void* stream) {
    if (!tree_ok(B, N) || V < 1 || V > (1 << 30) || !tokens || !parents || !target || target_stride < V ||
        (draft && draft_stride < V) || !u || !u_next || !n_accepted || !path || !next_token ||
        !words_aligned(tokens, parents, n_nodes, u, u_next, n_accepted, path, next_token, err, target, draft))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const int ctas = verify_ctas(B, V);
    const bool large = V > BLOCK_IDS;
    const int threads = large ? THREADS : THREADS_SMALL, turn = ctas * threads * 4;  // ids at a time
    const int seg = (int)((V + 3ll + turn - 1) / turn) * 128;  // and 3 ids that alignment skips
    const VerifyArgs a{tokens, parents, n_nodes, target, draft, u, u_next, target_stride, draft_stride, n_accepted, path, next_token, err,
                       N, V, ctas, seg};
    const auto go = [&](auto kernel, SmemState& state) {
        allow_smem(state, kernel, 0, true);
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = ctas;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas, B);
        cfg.blockDim = dim3(threads);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cfg.attrs = at;
        cfg.numAttrs = ctas > 1 ? 2 : 1;
        cudaLaunchKernelEx(&cfg, kernel, a);
    };
    static SmemState states[4];
    if (large) draft ? go(k_tree_verify<true, THREADS>, states[0]) : go(k_tree_verify<false, THREADS>, states[1]);
    else draft ? go(k_tree_verify<true, THREADS_SMALL>, states[2]) : go(k_tree_verify<false, THREADS_SMALL>, states[3]);
    return launched();
}

TTS_API tts_bb_status tts_bb_tree_verify_greedy(int B, int N, const int32_t* tokens, const int32_t* parents, const int32_t* n_nodes,
                                                const int32_t* target_ids, int32_t* n_accepted, int32_t* path, int32_t* next_token,
                                                int32_t* err, void* stream) {
    if (!tree_ok(B, N) || !tokens || !parents || !target_ids || !n_accepted || !path || !next_token ||
        !words_aligned(tokens, parents, n_nodes, target_ids, n_accepted, path, next_token, err))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    VerifyArgs a{};
    a.tokens = tokens;
    a.parents = parents;
    a.n_nodes = n_nodes;
    a.n_accepted = n_accepted;
    a.path = path;
    a.next = next_token;
    a.err = err;
    a.N = N;
    launch_pdl(k_tree_greedy, (B + GREEDY_WARPS - 1) / GREEDY_WARPS, GREEDY_WARPS * 32, 0, static_cast<cudaStream_t>(stream), a, target_ids, B);
    return launched();
}

TTS_API tts_bb_status tts_bb_tree_commit(const tts_bb_kv_cache* cache, int B, int N, const void* k, const void* v, int64_t row_stride,
                                         int64_t layer_stride, const int32_t* path, const int32_t* n_accepted, const int32_t* seqs,
                                         const int32_t* kv_lens, void* stream) {
    if (!cache_ok(cache) || !tree_ok(B, N) || !k || !v || !aligned16(k) || !aligned16(v) || row_stride < NKV * HD || row_stride % 8 ||
        (cache->n_layers > 1 && (layer_stride < 0 || layer_stride % 8)) || cache->n_layers > 65535 || !path || !n_accepted || !kv_lens ||
        (!seqs && B > cache->n_seqs) || !words_aligned(path, n_accepted, seqs, kv_lens))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const CommitArgs a{static_cast<const bf16*>(k), static_cast<const bf16*>(v), row_stride, cache->n_layers > 1 ? layer_stride : 0, path, n_accepted,
                       seqs, kv_lens, N};
    launch_pdl(k_tree_commit, dim3(cache->n_layers, B), 128, 0, static_cast<cudaStream_t>(stream), pages_of(cache, 0), a);
    return launched();
}
