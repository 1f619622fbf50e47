// Attention of a tree of drafted tokens over the paged bf16 cache: a node sees the cached keys, itself and its ancestors.
//
// The two query heads of a KV head and up to 64 nodes are the 128 rows of a tile of the tensor cores: row 2 i + h is node i's
// head 2 g + h. A sequence's keys are its cache pages of 64 and, behind them, one page of the tree's own keys, masked by
// each node's ancestors. Sums: out = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m), c = log2 e / sqrt 128, with the running
// maximum m of the tiles so far.
#include <algorithm>
#include <type_traits>

#include "tcgen05.cuh"
#include "tree.cuh"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

typedef unsigned long long u64;

struct TreeArgs {
    const void* q;
    const bf16* v;
    long long q_stride, kv_stride;
    const int32_t *parents, *n_nodes, *seqs, *kv_lens;
    int B, N, max_len;
    void* out;
    int4* meta;   // [shares]: the first piece of each
    float* part;  // [shares][2][2 N][PART]
};

constexpr int PAGE_BYTES = KVB * HD * 2;  // K or V of a page and head
constexpr int PART = HD + 4;              // 128 sums, the reference and the weight, 16-byte rows
constexpr int SHARES = 152;               // a block an SM

// A share's work: a piece of the tiles of one (sequence, KV head), the pages 0 .. pages - 1 of which the last is the tree.
struct Piece {
    int b, g, row, len, n;  // b < 0: no more
    int t0, t1, pages;
    int ok;                 // the tree is in order (known where the piece holds the tree's page)
    int whole, first;
    uint32_t bad[2];        // nodes whose values are not all finite
    u64 seen[MAX_NODES];    // ancestors and self
};

// bf16: tiles of two pages, queries as they are, weights in two bf16 parts. fp32: tiles of one page, queries and
// weights in three parts each, which is all of their bits.
template <bool F32>
struct Lay {
    static constexpr int KT = F32 ? 64 : 128, PAGES = KT / KVB, QPARTS = F32 ? 3 : 1, PPARTS = F32 ? 3 : 2;
    static constexpr int SLOT = KT * HD * 2, SLOTS = F32 ? 7 : 5;
    static constexpr int Q_BYTES = 128 * HD * 2;
    static constexpr int RING_OFF = QPARTS * Q_BYTES, END = RING_OFF + SLOTS * SLOT;
};
constexpr int SOFT_WARPS = 4, SUM_WARPS = 4, W_LOAD = 8, W_MMA = 9, W_SCHED = 10, WARPS = 11, NT = WARPS * 32;
constexpr int PIECES = 3;      // descriptors in flight
constexpr int RING = 4;        // tiles whose factors are kept
constexpr int TMEM_COLS = 512; // scores / weights of tile t at 128 (t & 1), its sums at 256 + 128 (t & 1)

struct Shared {
    u64 full[8], empty[8];      // ring slots
    u64 s_full[2], p_full[2];   // scores there (and the word of `there`), weights there (4 warps)
    u64 o_full[2], o_empty[2];  // a tile's sums and factors there (1 + 4), taken (4)
    u64 q_full, piece_full[PIECES], piece_empty[PIECES], fin;
    u64 sums[WARPS];
    uint32_t tmem;
    int abort;
    int start[2];
    int there[8];  // of tile t, at t % 8: a bit for each of its pages that was there
    Piece piece[PIECES];
    float alpha[RING][128], m[RING][128], l[RING][128];
};
template <bool F32>
constexpr int SMEM = Lay<F32>::END + (int)sizeof(Shared);
static_assert(SMEM<false> <= 232448 && SMEM<true> <= 232448, "shared memory of a block");

__device__ __forceinline__ void arrive(u64* bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s_addr(bar)) : "memory"); }
__device__ __forceinline__ void arrive_tx(u64* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D += A B with A (bf16 pairs, a column a pair) in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(bd), "r"(idesc), "r"(acc));
}
// two floats an instruction
__device__ __forceinline__ u64 pair(float a, float b) {
    u64 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void halves(u64 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// Whether sequence b has work; its cache row, keys and nodes.
__device__ __forceinline__ bool sequence(const Pages& c, const TreeArgs& a, int b, bool report, int& row, int& len, int& n) {
    row = row_of(c, a.seqs, b);
    n = a.n_nodes ? a.n_nodes[b] : a.N;
    len = a.kv_lens[b];
    if (row == -1) return false;
    if (row < 0 || n < 0 || n > a.N || len < 0 || len > a.max_len) {
        if (report) set_err(c.err, TTS_BB_TREE_ERR_RANGE);
        return false;
    }
    return n > 0;
}
__host__ __device__ constexpr int tiles_of(int len, int pages_a_tile) { return ((len + KVB - 1) / KVB + pages_a_tile) / pages_a_tile; }

// A warp finds what each node sees; lanes hold nodes l and l + 32. By doubling: what is seen within 2^k steps, and the node
// 2^k steps up. False where a parent is out of order (taken as -1 then).
__device__ __forceinline__ bool ancestors(const int32_t* parents, int n, int lane, u64 (&seen)[2]) {
    int up[2];
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        up[h] = j < n ? parents[j] : -1;
        if (up[h] < -1 || up[h] >= j) {
            bad = true;
            up[h] = -1;
        }
        seen[h] = 1ull << j;
    }
    while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
        int next[2];
        u64 more[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = up[h] & 31;
            const u64 m0 = __shfl_sync(0xffffffffu, seen[0], at), m1 = __shfl_sync(0xffffffffu, seen[1], at);
            const int u0 = __shfl_sync(0xffffffffu, up[0], at), u1 = __shfl_sync(0xffffffffu, up[1], at);
            more[h] = up[h] < 0 ? 0 : up[h] < 32 ? m0 : m1;
            next[h] = up[h] < 0 ? -1 : up[h] < 32 ? u0 : u1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            seen[h] |= more[h];
            up[h] = next[h];
        }
    }
    return !__any_sync(0xffffffffu, bad);
}

__device__ __forceinline__ bool finite16(uint32_t half) { return (half & 0x7F80u) != 0x7F80u; }

// a row's 128 numbers to out
__device__ __forceinline__ void store_row(float* to, const float* x, float f) {
#pragma unroll
    for (int d = 0; d < HD; d += 4) *reinterpret_cast<float4*>(to + d) = make_float4(x[d] * f, x[d + 1] * f, x[d + 2] * f, x[d + 3] * f);
}
__device__ __forceinline__ void store_row(bf16* to, const float* x, float f) {
#pragma unroll
    for (int d = 0; d < HD; d += 8)
        *reinterpret_cast<uint4*>(to + d) = make_uint4(bf16_pair(x[d] * f, x[d + 1] * f), bf16_pair(x[d + 2] * f, x[d + 3] * f),
                                                       bf16_pair(x[d + 4] * f, x[d + 5] * f), bf16_pair(x[d + 6] * f, x[d + 7] * f));
}

// grid: the shares, 352 threads. All tiles of all (sequence, KV head) are one line, cut into equal shares. A warp deals the
// pieces of its share, one loads pages by TMA into a ring of K and V slots (in the order in which the products take them),
// one issues the products: S = Q K^T of tile t + 1, then O = P V of tile t. Four warps (a thread a row) turn scores into weights,
// which replace them in TMEM as the A operand of P V; four more add each tile's sums to those in their registers. Every wait is bounded.
template <bool F32>
__global__ void __launch_bounds__(NT, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap pool_map, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                Pages c, TreeArgs a) {
    typedef Lay<F32> L;
    typedef std::conditional_t<F32, float, bf16> T;
    extern __shared__ __align__(1024) unsigned char smem[];
    if (s_addr(smem) & 1023u) {  // the swizzled tiles need a 1 KB-aligned base
        if (threadIdx.x == 0) {
            set_err(c.err, TTS_BB_TREE_ERR_TIMEOUT);
            pdl_wait();
            a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        return;
    }
    Shared& sh = *reinterpret_cast<Shared*>(smem + L::END);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = blockIdx.x;
    volatile int* const stop = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            tc_mbar_init((uint64_t*)sh.full + i, 1);
            tc_mbar_init((uint64_t*)sh.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc_mbar_init((uint64_t*)sh.s_full + i, 2);
            tc_mbar_init((uint64_t*)sh.p_full + i, SOFT_WARPS);
            tc_mbar_init((uint64_t*)sh.o_full + i, 1 + SOFT_WARPS);
            tc_mbar_init((uint64_t*)sh.o_empty + i, SUM_WARPS);
        }
        tc_mbar_init((uint64_t*)&sh.q_full, SOFT_WARPS);
        for (int i = 0; i < PIECES; ++i) {
            tc_mbar_init((uint64_t*)sh.piece_full + i, 1);
            tc_mbar_init((uint64_t*)sh.piece_empty + i, 2 + SOFT_WARPS + SUM_WARPS);
        }
        tc_mbar_init((uint64_t*)&sh.fin, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s_addr(&sh.tmem)), "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    // where the share begins: the sequences' tiles, one a thread at a time; the sum of all first, where one turn is not enough
    long long total = 0, before = 0, first = 0, units = 0;
    long long share = 0;
    const auto count = [&](int b, bool report) {
        int row, len, n;
        return b < a.B && sequence(c, a, b, report, row, len, n) ? tiles_of(len, L::PAGES) : 0;
    };
    const auto deal = [&](long long tiles) {
        units = tiles * NKV;
        share = (units + gridDim.x - 1) / gridDim.x;
        first = me * share;
    };
    const bool one_turn = a.B <= NT;
    if (!one_turn) {
        for (int i = tid; i < a.B; i += NT) total += count(i, me == 0);
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) sh.sums[warp] = total;
        __syncthreads();
        total = 0;
        for (int w = 0; w < WARPS; ++w) total += sh.sums[w];
        deal(total);
    }
    for (int i = tid; i - tid < a.B && before * NKV <= first; i += NT) {
        const int n = count(i, one_turn && me == 0);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += w;
        }
        __syncthreads();
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        long long mine = before + incl - n;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) mine += sh.sums[w];
            before += sh.sums[w];
        }
        if (one_turn) deal(before);
        if (first >= mine * NKV && first < (mine + n) * NKV) {
            sh.start[0] = i;
            sh.start[1] = (int)(first - mine * NKV);
        }
    }
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;
    const bool any = first < units;
    bool ok = true;
    const auto wait = [&](u64* bar, uint32_t parity) {  // by whole warps
        if (ok) ok = __all_sync(0xffffffffu, tc_wait((uint64_t*)bar, parity, stop));
        if (!ok && lane == 0) *stop = 1;
        return ok;
    };
    const auto wait1 = [&](u64* bar, uint32_t parity) {  // by one lane
        if (ok) ok = tc_wait((uint64_t*)bar, parity, stop);
        if (!ok) *stop = 1;
        return ok;
    };

    if (warp == W_SCHED) {
        int b = sh.start[0], at = sh.start[1], known = -1;
        long long left = any ? min(share, units - first) : 0;
        u64 seen[2] = {0, 0};
        bool tree_ok = true, head = true;
        int row = 0, len = 0, n = 0;
        if (left > 0) sequence(c, a, b, false, row, len, n);
        if (!any && lane == 0) a.meta[me] = make_int4(-1, 0, 0, 0);
        for (int k = 0;; ++k) {
            const int slot = k % PIECES;
            if (k >= PIECES && !wait(&sh.piece_empty[slot], (k / PIECES - 1) & 1)) break;
            Piece& p = sh.piece[slot];
            if (left <= 0) {
                if (lane == 0) {
                    p.b = -1;
                    arrive(&sh.piece_full[slot]);
                }
                break;
            }
            const int nt = tiles_of(len, L::PAGES), g = at / nt, t0 = at - g * nt, t1 = (int)min((long long)nt, t0 + left);
            if (t1 == nt) {
                if (known != b) {
                    tree_ok = ancestors(a.parents + (size_t)b * a.N, n, lane, seen);
                    known = b;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) p.seen[lane + 32 * h] = seen[h];
                if (!tree_ok && lane == 0) set_err(c.err, TTS_BB_TREE_ERR_TREE);
            }
            if (lane == 0) {
                p.b = b;
                p.g = g;
                p.row = row;
                p.len = len;
                p.n = n;
                p.t0 = t0;
                p.t1 = t1;
                p.pages = (len + KVB - 1) / KVB + 1;
                p.ok = t1 < nt || tree_ok;
                p.whole = t0 == 0 && t1 == nt;
                p.first = head;
                p.bad[0] = p.bad[1] = 0;
                // of the share's first piece: its (sequence, head), nodes, and whether it begins and ends that one; bit 2: in order
                if (head) a.meta[me] = make_int4(b * NKV + g, n, (t0 > 0) | (t1 == nt) << 1 | p.ok << 2, 0);
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.piece_full[slot]);
            head = false;
            left -= t1 - t0;
            at += t1 - t0;
            if (at == nt * NKV && left > 0) {
                at = 0;
                do ++b; while (b < a.B && !sequence(c, a, b, false, row, len, n));
                if (b >= a.B) left = 0;
            }
        }
    } else if (warp == W_LOAD) {
        if (lane == 0) {
            int slot_at = 0, tile = 0;  // loads so far; the block's tiles whose keys were loaded
            // which 0: K, 1: V of tile t
            const auto load = [&](const Piece& p, int t, int which) {
                const int s = slot_at % L::SLOTS;
                if (slot_at >= L::SLOTS && !wait1(&sh.empty[s], (slot_at / L::SLOTS - 1) & 1)) return false;
                int rows[L::PAGES], there = 0;
#pragma unroll
                for (int i = 0; i < L::PAGES; ++i) {
                    const int page = t * L::PAGES + i;
                    rows[i] = -1;
                    if (page < p.pages - 1) {
                        const int at = page_of(c, p.row, page * KVB);
                        if (at < 0) set_err(c.err, TTS_BB_TREE_ERR_PAGE);
                        else rows[i] = ((at * 2 + which) * NKV + p.g) * KVB;
                    } else if (page == p.pages - 1) {
                        rows[i] = p.b * a.N;
                    }
                    there |= (rows[i] >= 0) << i;
                }
                if (!which) sh.there[tile++ % 8] = there;  // fewer than 8 tiles are in flight: each takes two slots
                arrive_tx(&sh.full[s], (uint32_t)__popc(there) * PAGE_BYTES);
                unsigned char* const to = smem + L::RING_OFF + s * L::SLOT;
#pragma unroll
                for (int i = 0; i < L::PAGES; ++i) {
                    if (rows[i] < 0) continue;
                    const bool tree = t * L::PAGES + i == p.pages - 1;
                    const CUtensorMap* map = !tree ? &pool_map : which ? &v_map : &k_map;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // K: [64 dims of h][keys]; V: [page][64 dims of h][64 keys]
                        const int off = which ? i * PAGE_BYTES + h * (PAGE_BYTES / 2) : h * (L::SLOT / 2) + i * (PAGE_BYTES / 2);
                        tma_load_2d(to + off, map, (tree ? p.g * HD : 0) + h * 64, rows[i], (uint64_t*)&sh.full[s]);
                    }
                }
                ++slot_at;
                return true;
            };
            for (int k = 0; ok; ++k) {
                const int slot = k % PIECES;
                if (!wait1(&sh.piece_full[slot], (k / PIECES) & 1)) break;
                const Piece& p = sh.piece[slot];
                if (p.b < 0) break;
                load(p, p.t0, 0);
                for (int t = p.t0; ok && t < p.t1; ++t) {
                    if (t + 1 < p.t1 && !load(p, t + 1, 0)) break;
                    load(p, t, 1);
                }
                arrive(&sh.piece_empty[slot]);
            }
            if (*stop)  // copies in flight land before the block ends
                for (int j = max(0, slot_at - L::SLOTS); j < slot_at; ++j) {
                    const unsigned long long t0 = g_time();
                    while (!tc_mbar_try((uint64_t*)&sh.full[j % L::SLOTS], (j / L::SLOTS) & 1) && g_time() - t0 < TC_TIMEOUT_NS) {
                    }
                }
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
            constexpr uint32_t IDESC_S = IDESC | ((uint32_t)(L::KT >> 3) << 17), IDESC_PV = IDESC | ((uint32_t)(HD >> 3) << 17) | (1u << 16);
            const uint32_t q0 = s_addr(smem), ring = s_addr(smem + L::RING_OFF);
            int slot_at = 0, tile = 0;
            const auto scores = [&](int j) {  // of the block's tile j
                const int s = slot_at % L::SLOTS;
                if (!wait1(&sh.full[s], (slot_at / L::SLOTS) & 1)) return;
                // the weights of tile j - 2, which the scores replace, were taken by its product
                if (j >= 2 && !wait1(&sh.o_full[j & 1], ((j - 2) >> 1) & 1)) return;
                tc_after();
                const uint32_t k0 = ring + (uint32_t)(s * L::SLOT), d = tmem + (uint32_t)((j & 1) * 128);
#pragma unroll
                for (int part = L::QPARTS - 1; part >= 0; --part)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        at_mma(d, sw128_desc(q0 + (uint32_t)(part * L::Q_BYTES + (kk >> 2) * (L::Q_BYTES / 2) + (kk & 3) * 32)),
                               sw128_desc(k0 + (uint32_t)((kk >> 2) * (L::SLOT / 2) + (kk & 3) * 32)), IDESC_S, part < L::QPARTS - 1 || kk ? 1u : 0u);
                arrive(&sh.s_full[j & 1]);
                at_commit((uint64_t*)&sh.s_full[j & 1]);
                at_commit((uint64_t*)&sh.empty[s]);
                ++slot_at;
            };
            for (int k = 0; ok; ++k) {
                const int slot = k % PIECES;
                if (!wait1(&sh.piece_full[slot], (k / PIECES) & 1)) break;
                const int nt = sh.piece[slot].b < 0 ? 0 : sh.piece[slot].t1 - sh.piece[slot].t0;
                if (nt == 0) break;
                if (!wait1(&sh.q_full, k & 1)) break;
                scores(tile);
                for (int t = 0; ok && t < nt; ++t, ++tile) {
                    if (t + 1 < nt) scores(tile + 1);
                    if (!ok || !wait1(&sh.p_full[tile & 1], (tile >> 1) & 1)) break;
                    const int s = slot_at % L::SLOTS;
                    if (!wait1(&sh.full[s], (slot_at / L::SLOTS) & 1)) break;
                    if (tile >= 2 && !wait1(&sh.o_empty[tile & 1], ((tile >> 1) - 1) & 1)) break;
                    tc_after();
                    const uint32_t v0 = ring + (uint32_t)(s * L::SLOT), w = tmem + (uint32_t)((tile & 1) * 128), d = tmem + 256 + (uint32_t)((tile & 1) * 128);
#pragma unroll
                    for (int part = L::PPARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int kk = 0; kk < L::KT / 16; ++kk)  // 16 keys a step: 8 columns of weights
                            mma_ts(d, w + (uint32_t)(part * (L::KT / 2) + kk * 8),
                                   sw128_desc_mn(v0 + (uint32_t)((kk >> 2) * PAGE_BYTES + (kk & 3) * 2048), PAGE_BYTES / 2, 1024), IDESC_PV,
                                   part < L::PPARTS - 1 || kk ? 1u : 0u);
                    at_commit((uint64_t*)&sh.o_full[tile & 1]);
                    at_commit((uint64_t*)&sh.empty[s]);
                    ++slot_at;
                }
                arrive(&sh.piece_empty[slot]);
            }
            if (!ok) *stop = 1;
            at_commit((uint64_t*)&sh.fin);  // every product has ended
            const unsigned long long t0 = g_time();
            while (!tc_mbar_try((uint64_t*)&sh.fin, 0) && g_time() - t0 < TC_TIMEOUT_NS) {
            }
        }
    } else if (warp < SOFT_WARPS) {
        // ---------------- scores to weights: thread = row
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const int r = tid;
        const float cs = 0.08838834764831845f * 1.4426950408889634f;
        int slot_at = 0, tile = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k % PIECES;
            if (!wait(&sh.piece_full[slot], (k / PIECES) & 1)) break;
            Piece& p = sh.piece[slot];
            if (p.b < 0) break;
            const int nt = p.t1 - p.t0, rows = 2 * p.n;
            const bool mine = warp * 32 < rows;
            if (mine) {
                // queries of this warp's rows; those of the piece before were read by products that have ended
                const T* const q = static_cast<const T*>(a.q) + (size_t)p.b * a.N * a.q_stride + 2 * p.g * HD;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    constexpr int V = F32 ? 2 : 1;
                    uint4 x[8][V];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = (half * 8 + i) * 32 + lane, qr = warp * 32 + (e >> 4), pc = e & 15;
#pragma unroll
                        for (int v = 0; v < V; ++v) x[i][v] = make_uint4(0u, 0u, 0u, 0u);
                        if (qr < rows) {
                            const uint4* const src = reinterpret_cast<const uint4*>(q + (qr >> 1) * a.q_stride + (qr & 1) * HD + pc * 8);
#pragma unroll
                            for (int v = 0; v < V; ++v) x[i][v] = src[v];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = (half * 8 + i) * 32 + lane, qr = warp * 32 + (e >> 4), pc = e & 15;
                        unsigned char* const to = smem + (pc >> 3) * (L::Q_BYTES / 2) + sw128_off(qr, pc & 7);
                        if constexpr (F32) {
                            float f[8];
                            uint32_t w[4];
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                f[4 * v] = __uint_as_float(x[i][v].x);
                                f[4 * v + 1] = __uint_as_float(x[i][v].y);
                                f[4 * v + 2] = __uint_as_float(x[i][v].z);
                                f[4 * v + 3] = __uint_as_float(x[i][v].w);
                            }
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    w[u] = bf16_pair(f[2 * u], f[2 * u + 1]);
                                    f[2 * u] -= __uint_as_float(w[u] << 16);
                                    f[2 * u + 1] -= __uint_as_float(w[u] & 0xFFFF0000u);
                                }
                                *reinterpret_cast<uint4*>(to + part * L::Q_BYTES) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
                            *reinterpret_cast<uint4*>(to) = x[i][0];
                        }
                    }
                }
                fence_async();
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.q_full);
            float m = -INFINITY, mc = -INFINITY, l = 0.f;  // the largest score, that times cs, the sum of weights
            for (int t = 0; t < nt; ++t, ++tile) {
                const int vi = slot_at + (t + 1 < nt ? 2 * t + 2 : 2 * t + 1), vs = vi % L::SLOTS;
                if (!wait(&sh.s_full[tile & 1], (tile >> 1) & 1)) break;
                tc_after();
                // the keys that count, a bit each, and the pages whose values have to be made safe
                u64 keys[L::PAGES];
                bool partial = false;
                const int there = sh.there[tile % 8];
#pragma unroll
                for (int i = 0; i < L::PAGES; ++i) {
                    const int page = (p.t0 + t) * L::PAGES + i, valid = p.len - page * KVB;
                    keys[i] = !(there >> i & 1) ? 0ull : page == p.pages - 1 ? (r < rows ? p.seen[r >> 1] : 0ull) : valid >= KVB ? ~0ull : (1ull << valid) - 1;
                    partial |= page >= p.pages - 1 || valid < KVB || !(there >> i & 1);
                }
                if (partial) {
                    // rows of V that do not count are zeroed, and what is not finite among the tree's (it is added to the rows that see it at
                    // the end): 0 times it would be NaN. Warp w: keys 16 w .. 16 w + 15 of each page
                    if (!wait(&sh.full[vs], (vi / L::SLOTS) & 1)) break;
                    unsigned char* const v0 = smem + L::RING_OFF + vs * L::SLOT;
#pragma unroll
                    for (int i = 0; i < L::PAGES; ++i) {
                        const int page = (p.t0 + t) * L::PAGES + i;
                        const bool tree = page == p.pages - 1;
                        const int valid = !(there >> i & 1) ? 0 : tree ? p.n : min(KVB, p.len - page * KVB);
                        if (valid == KVB && !tree) continue;
#pragma unroll
                        for (int e = lane; e < 256; e += 32) {
                            const int key = warp * 16 + (e >> 4), pc = e & 15;
                            uint4* const at = reinterpret_cast<uint4*>(v0 + i * PAGE_BYTES + (pc >> 3) * (PAGE_BYTES / 2) + sw128_off(key, pc & 7));
                            if (key >= valid) {
                                *at = make_uint4(0u, 0u, 0u, 0u);
                            } else if (tree) {
                                const uint4 x = *at;
                                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                                bool bad = false;
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    if (!finite16(w[u])) { w[u] &= 0xFFFF0000u; bad = true; }
                                    if (!finite16(w[u] >> 16)) { w[u] &= 0xFFFFu; bad = true; }
                                }
                                if (bad) {
                                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                                    atomicOr(&p.bad[key >> 5], 1u << (key & 31));
                                }
                            }
                        }
                    }
                    fence_async();
                }
                float alpha = 1.f;
                if (mine) {
                    const uint32_t at = lanes + (uint32_t)((tile & 1) * 128);
                    uint32_t s[L::KT];
#pragma unroll
                    for (int i = 0; i < L::KT; i += 32) tm_ld32_nw(at + i, s + i);
                    tm_wait_ld();
                    if (partial) {
#pragma unroll
                        for (int i = 0; i < L::KT; ++i)
                            if (!(keys[i >> 6] >> (i & 63) & 1)) s[i] = 0xFF800000u;  // -inf
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < L::KT; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (top > m) {
                        alpha = at_ex2(mc - top * cs);
                        m = top;
                        mc = top * cs;
                    }
                    const float base = m == -INFINITY ? 0.f : mc;
                    const u64 cs2 = pair(cs, cs), base2 = pair(-base, -base), minus = pair(-1.f, -1.f);
                    u64 sum[2] = {0, 0};
#pragma unroll
                    for (int i0 = 0; i0 < L::KT; i0 += 64) {
                        uint32_t w[L::PPARTS][32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float x, y;
                            halves(fma2(pair(__uint_as_float(s[i0 + 2 * i]), __uint_as_float(s[i0 + 2 * i + 1])), cs2, base2), x, y);
                            u64 e = pair(at_ex2(x), at_ex2(y));
                            sum[i & 1] = add2(sum[i & 1], e);
#pragma unroll
                            for (int part = 0; part < L::PPARTS; ++part) {
                                halves(e, x, y);
                                w[part][i] = bf16_pair(x, y);
                                if (part + 1 < L::PPARTS)
                                    e = fma2(pair(__uint_as_float(w[part][i] << 16), __uint_as_float(w[part][i] & 0xFFFF0000u)), minus, e);
                            }
                        }
#pragma unroll
                        for (int part = 0; part < L::PPARTS; ++part) tm_st32(at + (uint32_t)(part * (L::KT / 2) + i0 / 2), w[part]);
                    }
                    float x, y, z, u;
                    halves(sum[0], x, y);
                    halves(sum[1], z, u);
                    l = l * alpha + ((x + y) + (z + u));
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                sh.alpha[tile % RING][r] = alpha;
                if (t + 1 == nt) {
                    sh.m[tile % RING][r] = m == -INFINITY ? -INFINITY : mc;
                    sh.l[tile % RING][r] = l;
                }
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    arrive(&sh.p_full[tile & 1]);
                    arrive(&sh.o_full[tile & 1]);
                }
            }
            if (!ok) break;
            slot_at += 2 * nt;
            __syncwarp();
            if (lane == 0) arrive(&sh.piece_empty[slot]);
        }
    } else {
        // ---------------- a row's sums over the tiles: thread = row
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + 256 + ((uint32_t)(quarter * 32) << 16);
        int tile = 0;
        for (int k = 0; ok; ++k) {
            const int slot = k % PIECES;
            if (!wait(&sh.piece_full[slot], (k / PIECES) & 1)) break;
            const Piece& p = sh.piece[slot];
            if (p.b < 0) break;
            const int nt = p.t1 - p.t0, rows = 2 * p.n;
            const bool mine = quarter * 32 < rows;
            u64 o[HD / 2];
#pragma unroll
            for (int i = 0; i < HD / 2; ++i) o[i] = 0;
            float m = 0.f, l = 0.f;
            for (int t = 0; t < nt; ++t, ++tile) {
                if (!wait(&sh.o_full[tile & 1], (tile >> 1) & 1)) break;
                tc_after();
                if (mine) {
                    const float f = sh.alpha[tile % RING][r];
                    const u64 f2 = pair(f, f);
#pragma unroll
                    for (int i = 0; i < HD; i += 32) {
                        uint32_t x[32];
                        tm_ld32_nw(lanes + (uint32_t)((tile & 1) * 128 + i), x);
                        tm_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[i / 2 + j] = fma2(o[i / 2 + j], f2, pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])));
                    }
                    m = sh.m[tile % RING][r];
                    l = sh.l[tile % RING][r];
                }
                tc_before();
                __syncwarp();
                if (lane == 0) arrive(&sh.o_empty[tile & 1]);
            }
            if (!ok) break;
            if (r < rows) {
                float x[HD];
#pragma unroll
                for (int i = 0; i < HD / 2; ++i) halves(o[i], x[2 * i], x[2 * i + 1]);
                const u64 bad = ((u64)p.bad[1] << 32 | p.bad[0]) & (p.bad[0] | p.bad[1] ? p.seen[r >> 1] : 0ull);
                for (u64 left = bad; left; left &= left - 1) {  // what was set aside
                    const bf16* const v = a.v + ((size_t)p.b * a.N + __ffsll(left) - 1) * a.kv_stride + p.g * HD;
#pragma unroll
                    for (int d = 0; d < HD; ++d) {
                        const uint32_t half = *reinterpret_cast<const uint16_t*>(v + d);
                        if (!finite16(half)) x[d] += __uint_as_float(half << 16);
                    }
                }
                if (p.whole) {
                    if (p.ok) store_row(static_cast<T*>(a.out) + (((size_t)p.b * a.N + (r >> 1)) * NQ + 2 * p.g + (r & 1)) * HD, x, l == 0.f ? 0.f : 1.f / l);
                } else {
                    float* const to = a.part + (((size_t)me * 2 + !p.first) * 2 * a.N + r) * PART;
                    store_row(to, x, 1.f);
                    to[HD] = m;
                    to[HD + 1] = l;
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.piece_empty[slot]);
        }
    }
    if (!ok && lane == 0) set_err(c.err, TTS_BB_TREE_ERR_TIMEOUT);
    tc_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
    }
}

// grid (shares - 1, rows / 4), 128 threads: the pieces of the (sequence, KV head) that the end of share blockIdx.x cuts first. A warp a
// row, a lane 4 of the 128 dims. A share's first piece stands in its place 0, the piece that ends it in place 1.
template <typename T>
__global__ void __launch_bounds__(128) k_tree_combine(TreeArgs a, int shares) {
    pdl_wait();
    pdl_trigger();
    const int s0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y * 4 + warp;
    // the first pieces of this share and of those behind it: at most 20 shares hold parts of one of 8 or more (sequence, head)
    const int4 meta = s0 + lane < shares ? a.meta[s0 + lane] : make_int4(-1, 0, 0, 0);
    const int it = __shfl_sync(0xffffffffu, meta.x, 1);
    const uint32_t goes_on = __ballot_sync(0xffffffffu, lane > 0 && meta.x == it && (meta.z & 1));
    if (it < 0 || !(goes_on & 2)) return;  // the share behind begins with a new one
    const int head = __shfl_sync(0xffffffffu, meta.x, 0), inside = __shfl_sync(0xffffffffu, meta.z, 0) & 1;
    if (head == it && inside) return;  // begun before this share
    const int more = __ffs(~(goes_on >> 1)) - 1;  // shares behind this one
    const int n = __shfl_sync(0xffffffffu, meta.y, 1);
    const bool in_order = __shfl_sync(0xffffffffu, meta.z, more) >> 2 & 1;  // the last piece holds the tree
    if (r >= 2 * n || !in_order) return;
    const auto at = [&](int i) { return a.part + (((size_t)(s0 + i) * 2 + (i == 0 && head != it)) * 2 * a.N + r) * PART; };
    float M = lane <= more ? at(lane)[HD] : -INFINITY;
    M = warp_max(M);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i <= more; ++i) {
        const float* const p = at(i);
        const float f = at_ex2(p[HD] - base);
        const float4 x = *reinterpret_cast<const float4*>(p + lane * 4);
        l += f * p[HD + 1];
        o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    T* const to = static_cast<T*>(a.out) + (((size_t)(it / NKV) * a.N + (r >> 1)) * NQ + 2 * (it % NKV) + (r & 1)) * HD + lane * 4;
    if constexpr (std::is_same_v<T, float>) *reinterpret_cast<float4*>(to) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    else *reinterpret_cast<uint2*>(to) = make_uint2(bf16_pair(o.x * f, o.y * f), bf16_pair(o.z * f, o.w * f));
}

// Blocks of the launch: one an SM, or one a tile where there are fewer.
int share_count(int B, int max_len, int pages_a_tile) {
    return (int)std::min<long long>(SHARES, (long long)B * NKV * tiles_of(max_len, pages_a_tile));
}
constexpr size_t META_BYTES = (SHARES * sizeof(int4) + 255) / 256 * 256;

}  // namespace

TTS_API size_t tts_bb_tree_attention_workspace(int B, int N, int max_len) {
    if (!tree_ok(B, N) || max_len < 0 || max_len > (1 << 30)) return 0;
    return META_BYTES + (size_t)share_count(B, max_len, 1) * 2 * 2 * N * PART * sizeof(float);  // of both types
}

TTS_API tts_bb_status tts_bb_tree_attention(const tts_bb_kv_cache* cache, int layer, int B, int N, const void* q, int type,
                                            int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                            const int32_t* parents, const int32_t* n_nodes, const int32_t* seqs,
                                            const int32_t* kv_lens, int max_len, void* out, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    if (!cache_ok(cache) || layer < 0 || layer >= cache->n_layers || !tree_ok(B, N) || !q || !k || !v || !parents || !kv_lens || !out ||
        (type != TTS_BB_T_F32 && type != TTS_BB_T_BF16) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        q_stride < NQ * HD || q_stride % (type == TTS_BB_T_F32 ? 4 : 8) || kv_stride < NKV * HD || kv_stride % 8 || kv_stride > (1ll << 38) ||
        max_len < 0 || max_len > (1 << 30) || (long long)max_len > (long long)cache->blocks_per_seq * KVB || (!seqs && B > cache->n_seqs) ||
        !words_aligned(parents, n_nodes, seqs, kv_lens))
        return TTS_BB_E_INVALID;
    if (!workspace || workspace_bytes < tts_bb_tree_attention_workspace(B, N, max_len) || !aligned16(workspace)) return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const Pages c = pages_of(cache, layer);
    CUtensorMap pool_map, k_map, v_map;
    if (!tc_make_map_strided(&pool_map, c.pool, c.n_blocks * 2 * NKV * KVB, HD, HD, KVB) ||
        !tc_make_map_strided(&k_map, k, B * N, NKV * HD, kv_stride, KVB) || !tc_make_map_strided(&v_map, v, B * N, NKV * HD, kv_stride, KVB))
        return TTS_BB_E_CUDA;
    const TreeArgs a{q, static_cast<const bf16*>(v), q_stride, kv_stride, parents, n_nodes, seqs, kv_lens, B, N, max_len, out,
                     static_cast<int4*>(workspace), reinterpret_cast<float*>(static_cast<char*>(workspace) + META_BYTES)};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto go = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value;
        static SmemState state;
        allow_smem(state, k_tree_attn<F32>, SMEM<F32>);
        const int shares = share_count(B, max_len, Lay<F32>::PAGES);
        launch_pdl(k_tree_attn<F32>, shares, NT, SMEM<F32>, st, pool_map, k_map, v_map, c, a);
        if (tiles_of(max_len, Lay<F32>::PAGES) > 1)
            launch_pdl(k_tree_combine<std::conditional_t<F32, float, bf16>>, dim3(shares - 1, (2 * N + 3) / 4), 128, 0, st, a, shares);
    };
    if (type == TTS_BB_T_F32) go(std::true_type{});
    else go(std::false_type{});
    return launched();
}
