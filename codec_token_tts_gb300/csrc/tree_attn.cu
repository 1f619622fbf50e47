// Attention of a tree of drafted tokens over the paged bf16 cache: a node sees the cached keys, itself and its ancestors.
//
// The two query heads of a KV head and up to 64 nodes are the 128 rows of a tile of the tensor cores: row 2 i + h is node i's
// head 2 g + h. A sequence's keys are its cache pages of 64 and, behind them, one page of the tree's own keys, masked by
// each node's ancestors. Sums: out = sum_j 2^(c (s_j - m)) v_j / sum_j 2^(c (s_j - m)), c = log2 e / sqrt 128, with the running
// maximum m of the tiles so far (bf16: within a factor of 4 of it). Scores, softmax and sums are fp32; the sums of a tile (bf16: of two) are
// added to those before in registers, since the tensor cores' own accumulation cuts off what it shifts out.
//
// Each key's 512 bytes a KV head are read once and meet up to 128 rows: 256 products a byte at most, which needs tcgen05, and stays
// bound by memory. The least that a call reads is the cache: see k_tree_attn for what is reached.
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
    int4* meta;   // [blocks]: the first piece of each
    float4* part; // [blocks][2][PART][128]
};

constexpr int PAGE_BYTES = KVB * HD * 2;  // K or V of a page and head
constexpr int PART = HD / 4 + 1;          // a row's 128 sums by four, then its reference and weight: rows side by side
constexpr int SHARES = 152 / NKV;         // times 8 blocks: one an SM

// Exponents of 2 are (score - reference) CS, the difference first: in score CS - reference CS the rounding of the second product, up to 2^-25 of
// it, would be the exponent of the largest weight, which beyond 2^31 is 0 or infinite. One instruction more for two weights: 1 x 333 keys, 6
// nodes 8.5 us for 8.3, 8 x 65537, 31 nodes 255 for 250 from L2 and 309 for 309 from memory.
constexpr float CS = 0.08838834764831845f * 1.4426950408889634f;

// A share's work: a piece of the tiles (a page each) of one (sequence, KV head), the last of which is the tree.
struct Piece {
    int b, g, row, len, n;  // b < 0: no more
    int t0, t1, tiles;
    int whole, first;
    uint32_t bad[2];        // nodes whose values are not all finite
    // of pieces that hold the tree, a little later:
    int ok;                 // the tree is in order
    u64 seen[MAX_NODES];    // ancestors and self
};

// bf16: queries as they are, weights in two bf16 parts (17 bits, both rounded). fp32: queries and weights in three parts
// each, which is all of their bits.
template <bool F32>
struct Lay {
    static constexpr int QPARTS = F32 ? 3 : 1, PPARTS = F32 ? 3 : 2, QBUFS = F32 ? 1 : 2;
    // Regions of 64 columns of TMEM for a tile's scores, where weights replace them: of 32 keys' 32 columns the first part of their weights
    // takes 16, the second the others. The third part of tile t has 32 columns of its own by t & 1, behind three regions (two regions of
    // 96, which need no wait for them: 2500 cycles a tile, 3 regions 2100). Values are loaded AHEAD tiles behind keys
    static constexpr int REGIONS = F32 ? 3 : 4, AHEAD = 2;
    // Tiles whose sums the tensor cores add up where no row's reference rises between them, before warps 8 .. 11 take them: with one of
    // two buffers a tile, products that end late and the taking of their sums bounded a tile (8 x 65537 keys, 31 nodes, from L2: 272 us, of
    // pairs 253; 255 since weights take the difference first).
    // So that references rise seldom, one lags up to 2^SLACK behind the maximum: weights reach 4 then.
    static constexpr int GROUP = F32 ? 1 : 2;
    static constexpr float SLACK = F32 ? 0.f : 2.f;
    // the column of a part of 32 keys' weights of tile u
    static __device__ __forceinline__ uint32_t part_at(uint32_t u, int part, int chunk) {
        return part < 2 ? u % REGIONS * KVB + chunk * 32 + part * 16 : 192 + (u & 1) * 32 + chunk * 16;
    }
    static constexpr int STAGE = F32 ? 4096 : 0;  // of each warp that writes sums: 32 rows of 128 bytes
};
// Warps of single tasks: the loader and the issuer of sums beside the rows that trees of up to 32 nodes leave empty (warps of one index modulo
// 4 share a scheduler, and 0 and 1 are busy then): 8 x 65537 keys, 31 nodes 326 us, with the loader beside warp 0 or 1 375.
constexpr int W_SUM = 8, W_REST = 12, W_SAFE = 12, W_S = 13, W_LOAD = 14, W_PV = 15, WARPS = 16, NT = WARPS * 32;
// registers of a thread: the launch's 128 are dealt anew (208 for the sums and 80 for the rest: fp32 spills, 16 x 200..2000 keys 33.6 us, now 33.0)
constexpr int REGS_SOFT = 112, REGS_SUM = 200, REGS_REST = 88;
static_assert(2 * REGS_SOFT + REGS_SUM + REGS_REST == 4 * 128, "registers of the launch");
constexpr int PIECES = 4;       // descriptors in flight
constexpr int RING = 8;         // tiles whose references and weights are kept
constexpr int MAX_SLOTS = 8;    // of K, and of V
constexpr int TMEM_COLS = 512;  // the regions, then the sums of tile t at 256 + 128 (t & 1)

struct Shared {
    u64 k_full[MAX_SLOTS], k_empty[MAX_SLOTS], v_full[MAX_SLOTS], v_ready[MAX_SLOTS], v_empty[MAX_SLOTS];
    u64 s_full[4], p_full[4], w_empty[4];  // of a region: scores there (products, their issuer), weights there (4 warps), weights taken
    u64 o_full[2], o_empty[2];  // one or two tiles' sums there (products, their issuer), taken (4)
    u64 m_full[4][2];           // a tile's references of 32 rows there
    u64 q_full[2], q_empty[2], piece_full[PIECES], seen_full[PIECES], piece_empty[PIECES], fin[2];
    uint32_t sums[WARPS];
    uint32_t tmem;
    int abort;
    int start[5];
    int last[2];    // of the tiles whose sums a buffer holds
    unsigned char rose[4][4];  // of a region's weights and 32 rows: whether a reference rose
    int page[16];   // of tile t, at t % 16: -1 where its page is out of range
    Piece piece[PIECES];
    float m[RING][128], l[RING][128];
};
constexpr int SMEM_MAX = 232448;
// Of dynamic shared memory: the queries of `rows` rows (a multiple of 8), pages of K and of V, the stages, then Shared.
struct Plan {
    int rows, k_slots, v_slots;
    template <bool F32>
    __host__ __device__ int q_bytes() const { return Lay<F32>::QPARTS * rows * HD * 2; }  // of one buffer
    template <bool F32>
    __host__ __device__ int ring() const { return Lay<F32>::QBUFS * q_bytes<F32>(); }
    template <bool F32>
    __host__ __device__ int stages() const { return ring<F32>() + (k_slots + v_slots) * PAGE_BYTES; }
    template <bool F32>
    __host__ __device__ int shared() const { return stages<F32>() + 4 * Lay<F32>::STAGE; }
    template <bool F32>
    __host__ __device__ int bytes() const { return shared<F32>() + (int)sizeof(Shared); }
};

__device__ __forceinline__ void arrive(u64* bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s_addr(bar)) : "memory"); }
__device__ __forceinline__ void arrive_tx(u64* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e != 0;
}
// Operand descriptors: the words that do not change (stride 1024 bytes, 128-byte swizzle), and the low ones: the address and, for
// values (whose dims are two halves PAGE_BYTES / 2 apart), the leading offset.
constexpr uint32_t DESC_HI = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return saddr >> 4 | (PAGE_BYTES / 2 >> 4) << 16; }
// D (+)= A B, both in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"((uint32_t)acc));
}
// D (+)= A B with A (bf16 pairs, a column a pair) in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"((uint32_t)acc));
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
        "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
        : "memory");
}
// A warp's wait for one to three phases, at most 2^22 rounds of tries (each takes some 20 cycles at least, and the hardware holds a try
// back for a while where it has to wait): false then, and where another warp has given up.
#define TREE_TRY(p, bar, par) "mbarrier.try_wait.parity.shared::cta.b64 " p ", [" bar "], " par ";\n"
#define TREE_RETRY                                                                                                             \
    "ld.volatile.shared.u32 s, [%1];\nadd.u32 n, n, 1;\nsetp.gt.u32 q, n, 4194304;\n@q st.volatile.shared.u32 [%1], 1;\n" \
    "setp.eq.u32 q, s, 0;\n@q bra AGAIN;\nTHERE:\nselp.u32 %0, 1, 0, p;\n}"
__device__ __forceinline__ bool wait_for(int* stop, u64* bar, uint32_t par) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p, q;\n.reg .u32 n, s;\nmov.u32 n, 0;\nAGAIN:\n" TREE_TRY("p", "%2", "%3") "@p bra THERE;\n" TREE_RETRY
                 : "=r"(ok)
                 : "r"(s_addr(stop)), "r"(s_addr(bar)), "r"(par)
                 : "memory");
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_for(int* stop, u64* bar, uint32_t par, u64* bar2, uint32_t par2) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p, q;\n.reg .u32 n, s;\nmov.u32 n, 0;\nAGAIN:\n" TREE_TRY("p", "%2", "%3") TREE_TRY("q", "%4", "%5")
                 "and.pred p, p, q;\n@p bra THERE;\n" TREE_RETRY
                 : "=r"(ok)
                 : "r"(s_addr(stop)), "r"(s_addr(bar)), "r"(par), "r"(s_addr(bar2)), "r"(par2)
                 : "memory");
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_for(int* stop, u64* bar, uint32_t par, u64* bar2, uint32_t par2, u64* bar3, uint32_t par3) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p, q, r;\n.reg .u32 n, s;\nmov.u32 n, 0;\nAGAIN:\n" TREE_TRY("p", "%2", "%3") TREE_TRY("q", "%4", "%5")
                 TREE_TRY("r", "%6", "%7") "and.pred p, p, q;\nand.pred p, p, r;\n@p bra THERE;\n" TREE_RETRY
                 : "=r"(ok)
                 : "r"(s_addr(stop)), "r"(s_addr(bar)), "r"(par), "r"(s_addr(bar2)), "r"(par2), "r"(s_addr(bar3)), "r"(par3)
                 : "memory");
    return __all_sync(0xffffffffu, ok);
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
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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
__host__ __device__ constexpr int tiles_of(int len) { return (len + KVB - 1) / KVB + 1; }

// What each node sees, by doubling: what is seen within 2^k steps, and the node 2^k steps up. Nodes lane and lane + 32 of a warp. 200 x 3..30
// keys, 64 nodes: 54 us, through shared memory 63.
struct Line {
    u64 seen[2];
    int up[2];
    bool in_order;  // or a parent was not (taken as -1)

    __device__ __forceinline__ void begin(const int32_t* parents, int n, int lane) {
        in_order = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            up[h] = j < n ? parents[j] : -1;
            seen[h] = 1ull << j;
        }
    }
    // one round; whether there are more
    __device__ __forceinline__ bool step(int lane) {
        bool bad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool wrong = up[h] < -1 || up[h] >= lane + 32 * h;
            bad |= wrong;
            if (wrong) up[h] = -1;
        }
        in_order &= !__any_sync(0xffffffffu, bad);
        u64 more[2];
        int above[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u64 s0 = __shfl_sync(0xffffffffu, seen[0], up[h] & 31), s1 = __shfl_sync(0xffffffffu, seen[1], up[h] & 31);
            const int v0 = __shfl_sync(0xffffffffu, up[0], up[h] & 31), v1 = __shfl_sync(0xffffffffu, up[1], up[h] & 31);
            more[h] = up[h] < 0 ? 0ull : up[h] < 32 ? s0 : s1;
            above[h] = up[h] < 0 ? -1 : up[h] < 32 ? v0 : v1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            seen[h] |= more[h];
            up[h] = above[h];
        }
        return __any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0);
    }
};

__device__ __forceinline__ bool finite16(uint32_t half) { return (half & 0x7F80u) != 0x7F80u; }

// grid: 8 blocks a share, 512 threads. The tiles of all sequences are one line, cut into equal shares, and the 8 KV heads walk it side
// by side, a block each: what they read at a time lies together (64 x 200..2000 keys, 64 nodes: 74 us then; heads one after the other 81). Warp
// 14 deals the pieces of its share and loads pages (and bf16 queries) by TMA, 12 finds the nodes' ancestors and makes values safe to be
// multiplied by 0, 13 issues the scores S = Q K^T and 15 the sums O = P V (two warps, since an issuer waits for its products: one took
// turns, and the tensor cores waited meanwhile: 90 us for 97). Warps 0 .. 7 turn scores into weights (a thread a row, even and odd
// tiles by four each), which replace them in TMEM as the A operand of P V; they hand the running maximum on. Warps 8 .. 11 add
// the tiles' sums to those in their registers. Every wait is bounded.
//
// Measured: 8 x 65537 keys, 31 nodes 309 us, 7.0 TB/s: memory. 64 x 200..2000 keys, 64 nodes 71 us, 4.8 TB/s: 5 us until the first
// scores (one third of it instructions that come from L2), some 1400 cycles a tile, which memory needs too, 3 us at the end of each
// piece and of the launch, 7 for the launch that merges (8 x 16384 keys, 31 nodes: 5). fp32, 8 x 16384 keys, 64 nodes 134 us: the tensor cores (24 products of 128 x 64 x 16 for the
// scores of a tile, 12 of 128 x 128 x 16 for its sums, 2100 cycles).
//
// ONE: a share is a sequence, and none is cut.
template <bool F32, bool ONE>
__global__ void __launch_bounds__(NT, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap pool_map, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ CUtensorMap q_map, Pages c, TreeArgs a, Plan plan) {
    typedef Lay<F32> L;
    typedef std::conditional_t<F32, float, bf16> T;
    extern __shared__ __align__(1024) unsigned char smem[];
    if (s_addr(smem) & 1023u) {  // the swizzled tiles need a 1 KB-aligned base
        if (threadIdx.x == 0) {
            set_err(c.err, TTS_BB_TREE_ERR_TIMEOUT);
            pdl_wait();
            if (!ONE) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        return;
    }
    unsigned char* const k_ring = smem + plan.ring<F32>();
    unsigned char* const v_ring = k_ring + plan.k_slots * PAGE_BYTES;
    Shared& sh = *reinterpret_cast<Shared*>(smem + plan.shared<F32>());
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, me = blockIdx.x;
    if (warp == 0) {
        const auto init = [&](u64* b, int n, int of) {
            if (lane < of) tc_mbar_init((uint64_t*)b + lane, n);
        };
        init(sh.k_full, 1, 3 * MAX_SLOTS);  // and k_empty, v_full
        init(sh.v_ready, 1, 2 * MAX_SLOTS);  // and v_empty
        init(sh.s_full, 2, 4);
        init(sh.p_full, 4, 4);
        init(sh.w_empty, 1, 4);
        init(sh.o_full, 2, 2);
        init(sh.o_empty, 4, 2);
        init(&sh.m_full[0][0], 1, 8);
        init(sh.q_full, F32 ? 8 : 1, 2);
        init(sh.q_empty, 1, 2);
        init(sh.piece_full, 1, PIECES);
        init(sh.seen_full, 1, PIECES);
        init(sh.piece_empty, 2 + 8 + 4, PIECES);
        init(sh.fin, 1, 2);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_PV) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s_addr(&sh.tmem)), "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    // where the share begins: the sequences' tiles, one a thread at a time; the sum of all first, where one turn is not enough
    uint32_t before = 0, first = 0, units = 0, share = 0;
    const bool one_turn = a.B <= NT;
    const uint32_t shares = gridDim.x / NKV;
    const auto deal = [&](uint32_t tiles) {
        units = tiles;
        share = (units + shares - 1) / shares;
        first = me / NKV * share;
    };
    if constexpr (ONE) {  // a sequence a share: no deal
        if (tid == 0) {
            const int b = me / NKV;
            int row = 0, len = 0, nodes = 0;
            const bool any = sequence(c, a, b, me % NKV == 0, row, len, nodes);
            sh.start[0] = b;
            sh.start[1] = 0;
            sh.start[2] = row;
            sh.start[3] = any ? len : -1;
            sh.start[4] = nodes;
        }
    } else {
#pragma unroll 1
        for (int turn = one_turn; turn < 2; ++turn) {
            before = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < a.B && (turn == 0 || before <= first); i0 += NT) {
                const int i = i0 + tid;
                int row = 0, len = 0, nodes = 0;
                const uint32_t n = i < a.B && sequence(c, a, i, turn == one_turn && me == 0, row, len, nodes) ? tiles_of(len) : 0;
                uint32_t incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t w = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += w;
                }
                __syncthreads();
                if (lane == 31) sh.sums[warp] = incl;
                __syncthreads();
                uint32_t of = lane < WARPS ? sh.sums[lane] : 0, upto = of;
#pragma unroll
                for (int o = 1; o < WARPS; o <<= 1) {
                    const uint32_t w = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += w;
                }
                const uint32_t mine = before + __shfl_sync(0xffffffffu, upto - of, warp) + incl - n;
                before += __shfl_sync(0xffffffffu, upto, WARPS - 1);
                if (one_turn) deal(before);
                if (turn && first >= mine && first < mine + n) {
                    sh.start[0] = i;
                    sh.start[1] = (int)(first - mine);
                    sh.start[2] = row;
                    sh.start[3] = len;
                    sh.start[4] = nodes;
                }
            }
            if (turn == 0) deal(before);
        }
    }
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t U = ONE ? (sh.start[3] < 0 ? 0 : tiles_of(sh.start[3])) : first >= units ? 0 : min(share, units - first);  // this block's tiles
    bool ok = true;
    const auto wait = [&](u64* bar, uint32_t parity) {  // by whole warps
        ok = wait_for(&sh.abort, bar, parity);
        return ok;
    };
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);  // bf16 times bf16 to fp32, 128 rows
    const auto drain = [&](bool leader) {  // every product that this warp has issued has ended
        if (leader) {
            u64* const fin = &sh.fin[warp == W_S];
            at_commit((uint64_t*)fin);
            const unsigned long long t0 = g_time();
#pragma unroll 1
            while (!tc_mbar_try((uint64_t*)fin, 0) && g_time() - t0 < TC_TIMEOUT_NS) {
            }
        }
        __syncwarp();
    };
    // piece k, once it is there
    const auto piece_bar = [&](uint32_t k) { return &sh.piece_full[k % PIECES]; };
    const auto piece_par = [](uint32_t k) { return k / PIECES & 1u; };

    if (warp >= W_REST) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == W_LOAD) {
            int ks = 0, vs = 0;       // slots
            uint32_t kp = 1, vp = 1;  // parities of what empties them (the first round is empty)
            uint32_t kk = ~0u;
            // the sequence, its next tile, and what of the share has not been dealt
            int b = sh.start[0], at = sh.start[1], row = sh.start[2], len = sh.start[3], n = sh.start[4];
            uint32_t left = U;
            // the next piece (b < 0 where nothing is left), in its place once every warp is done with the one before
            const auto deal_piece = [&](uint32_t k) {
                Piece& p = sh.piece[k % PIECES];
                if (k >= PIECES && !wait(&sh.piece_empty[k % PIECES], (k / PIECES - 1) & 1u)) return false;
                const int nt = tiles_of(len), t0 = at, t1 = (int)min((uint32_t)nt, t0 + left);
                if (lane == 0) {
                    p.b = left ? b : -1;
                    p.g = me % NKV;
                    p.row = row;
                    p.len = len;
                    p.n = n;
                    p.t0 = t0;
                    p.t1 = t1;
                    p.tiles = nt;
                    p.whole = t0 == 0 && t1 == nt;
                    p.first = k == 0;
                    p.bad[0] = p.bad[1] = 0;
                    arrive(piece_bar(k));
                }
                __syncwarp();
                if (left == 0) return true;
                left -= t1 - t0;
                at += t1 - t0;
                if (at == nt && left > 0) {
                    at = 0;
                    do ++b; while (b < a.B && !sequence(c, a, b, false, row, len, n));
                    if (b >= a.B) left = 0;
                }
                return true;
            };
            // of the piece whose keys are loaded: its tiles (all, and its next and last here), its sequence, row and keys
            int tiles = 0, kt = 0, t1 = 0, from = 0, pb = 0, prow = 0;
            const int g = me % NKV;
            const auto entry = [&](int t) { return t < t1 && t < tiles - 1 ? c.table[(size_t)prow * c.bps + t] : 0; };
            // the first row of a tile's keys in what holds them, the pool or the tree's own; -1 where its page is out of range
            const auto rows_at = [&](int t, int page) {
                if (t == tiles - 1) return pb * a.N;
                if (page >= 0 && page < c.n_blocks) return (page * 2 * NKV + g) * KVB;
                set_err(c.err, TTS_BB_TREE_ERR_PAGE);
                return -1;
            };
            int here = 0, next = 0;  // that of the tiles from + lane, and the pages of the tiles from + 32 + lane
            // Keys are loaded a tile a round, and the values of AHEAD rounds ago: where these are. The round is short, since this warp's
            // instructions were what bounded a tile before: 8 x 65537 keys from L2, 64 nodes 282 us, with two waits and the piece read
            // from shared memory for keys and for values 325.
            int y[L::AHEAD + 1] = {};
            bool tree[L::AHEAD + 1] = {};
            int k_landing = 0, v_landing = 0;
#pragma unroll 1
            for (uint32_t i = 0; ok && i < U + L::AHEAD; ++i) {
                // both at once: an empty slot for the keys, and one for the values (behind the last keys, and before the first values,
                // of one that nothing is loaded to)
                const bool k_turn = i < U, v_turn = i >= L::AHEAD;
                if (k_turn) {
                    if (kt == t1) {
                        ++kk;
                        if (!deal_piece(kk)) break;
                        const Piece& p = sh.piece[kk % PIECES];
                        tiles = p.tiles, from = kt = p.t0, t1 = p.t1, pb = p.b, prow = p.row;
                        here = rows_at(from + lane, entry(from + lane));
                        next = entry(from + 32 + lane);
                        if constexpr (!F32) {
                            const uint32_t qb = kk & 1;
                            if (kk >= 2 && !wait(&sh.q_empty[qb], ((kk >> 1) - 1) & 1u)) {
                                --kk;
                                break;
                            }
                            if (lane == 0) {
                                unsigned char* const to = smem + qb * plan.q_bytes<F32>();
                                arrive_tx(&sh.q_full[qb], (uint32_t)a.N * 512);
                                tma_load_3d(to, &q_map, 0, 2 * g, pb * a.N, (uint64_t*)&sh.q_full[qb]);
                                tma_load_3d(to + plan.rows * 128, &q_map, 64, 2 * g, pb * a.N, (uint64_t*)&sh.q_full[qb]);
                            }
                        }
                    } else if (kt == from + 32) {
                        from = kt;
                        here = rows_at(from + lane, next);
                        next = entry(from + 32 + lane);
                    }
                }
#pragma unroll
                for (int j = L::AHEAD; j > 0; --j) y[j] = y[j - 1], tree[j] = tree[j - 1];
                y[0] = __shfl_sync(0xffffffffu, here, kt - from);
                tree[0] = kt == tiles - 1;
                ok = wait_for(&sh.abort, &sh.k_empty[ks], kp, &sh.v_empty[vs], vp);
                if (!ok) break;
                if (lane == 0) {
                    // K (which 0) or V of a tile
                    const auto fetch = [&](unsigned char* to, u64* bar, int j, int which) {
                        arrive_tx(bar, y[j] < 0 ? 0 : PAGE_BYTES);
                        if (y[j] >= 0)
                            tma_load_3d(to, !tree[j] ? &pool_map : which ? &v_map : &k_map, 0, y[j] + (tree[j] ? 0 : which * NKV * KVB),
                                        tree[j] ? 2 * g : 0, (uint64_t*)bar);
                    };
                    if (k_turn) {
                        sh.page[i % 16] = y[0];
                        fetch(k_ring + ks * PAGE_BYTES, &sh.k_full[ks], 0, 0);
                    }
                    if (v_turn) fetch(v_ring + vs * PAGE_BYTES, &sh.v_full[vs], L::AHEAD, 1);
                }
                if (k_turn) {
                    ++kt;
                    ++k_landing;
                    if (++ks == plan.k_slots) ks = 0, kp ^= 1;
                }
                if (v_turn) {
                    ++v_landing;
                    if (++vs == plan.v_slots) vs = 0, vp ^= 1;
                }
            }
            if (ok) ok = deal_piece(kk + 1);  // no more
            if (*(volatile int*)&sh.abort && lane == 0) {  // copies in flight land before the block ends
                const auto landed = [&](u64* full, int n, int slots) {
#pragma unroll 1
                    for (int j = max(0, n - slots); j < n; ++j) {
                        const unsigned long long t0 = g_time();
#pragma unroll 1
                        while (!tc_mbar_try((uint64_t*)&full[j % slots], (uint32_t)(j / slots) & 1u) && g_time() - t0 < TC_TIMEOUT_NS) {
                        }
                    }
                };
                landed(sh.k_full, k_landing, plan.k_slots);
                landed(sh.v_full, v_landing, plan.v_slots);
                if (!F32) landed(sh.q_full, (int)(kk + 1), 2);
            }
        } else if (warp == W_S) {
            constexpr uint32_t IDESC_S = IDESC | ((uint32_t)(KVB >> 3) << 17);
            const uint32_t q0 = desc_k(s_addr(smem)), k0 = desc_k(s_addr(k_ring)), half = (uint32_t)plan.rows * 128 >> 4,
                           q_buf = (uint32_t)plan.q_bytes<F32>() >> 4;
            const bool leader = elect();
            uint32_t ks = 0, kp = 0, k = ~0u;  // slot, its parity, piece
            int left = 0;
#pragma unroll 1
            for (uint32_t u = 0; u < U; ++u) {
                if (left == 0) {
                    ++k;
                    if (!wait(piece_bar(k), piece_par(k))) break;
                    left = sh.piece[k % PIECES].t1 - sh.piece[k % PIECES].t0;
                    if (!wait(&sh.q_full[F32 ? 0 : k & 1], (F32 ? k : k >> 1) & 1u)) break;
                }
                // the keys; and the weights that tile u - REGIONS left in the region were taken (of none: the phase before the first)
                const uint32_t region = u % L::REGIONS;
                ok = wait_for(&sh.abort, &sh.k_full[ks], kp, &sh.w_empty[region], (u / L::REGIONS - 1) & 1u);
                if (!ok) break;
                tc_after();
                const uint32_t d = tmem + region * KVB, k1 = k0 + ks * (PAGE_BYTES >> 4), q1 = q0 + (F32 ? 0u : (k & 1) * q_buf);
                --left;
                if (leader) {
#pragma unroll
                    for (int part = L::QPARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ss(d, q1 + (uint32_t)(part * 2 + (kk >> 2)) * half + (kk & 3) * 2, k1 + (uint32_t)((kk >> 2) * (PAGE_BYTES / 2) + (kk & 3) * 32) / 16,
                                   IDESC_S, part < L::QPARTS - 1 || kk > 0);
                    arrive(&sh.s_full[region]);
                    at_commit((uint64_t*)&sh.s_full[region]);
                    at_commit((uint64_t*)&sh.k_empty[ks]);
                    if (!F32 && left == 0) at_commit((uint64_t*)&sh.q_empty[k & 1]);
                }
                __syncwarp();
                if (++ks == (uint32_t)plan.k_slots) ks = 0, kp ^= 1;
            }
            drain(leader);
        } else if (warp == W_PV) {
            constexpr uint32_t IDESC_PV = IDESC | ((uint32_t)(HD >> 3) << 17) | (1u << 16);
            const uint32_t v0 = desc_mn(s_addr(v_ring));
            const bool leader = elect();
            uint32_t vs = 0, vp = 0, k = ~0u;  // slot, its parity, piece
            uint32_t o = 0;                    // the buffer's turn
            int left = 0, t = 0, tiles = 0, len = 0, n = 0, held = 0;  // tiles in it
            const auto close = [&](uint32_t last) {
                if (leader) {
                    sh.last[o & 1] = (int)last;
                    arrive(&sh.o_full[o & 1]);
                    at_commit((uint64_t*)&sh.o_full[o & 1]);
                }
                ++o;
                held = 0;
            };
#pragma unroll 1
            for (uint32_t u = 0; u < U; ++u) {
                if (left == 0) {
                    ++k;
                    if (!wait(piece_bar(k), piece_par(k))) break;
                    const Piece& p = sh.piece[k % PIECES];
                    t = p.t0;
                    left = p.t1 - t;
                    tiles = p.tiles;
                    len = p.len;
                    n = p.n;
                }
                // 16 keys a step of the products, of those that there are
                const int keys = t == tiles - 1 ? n : min(KVB, len - t * KVB), steps = (keys + 15) / 16;
                const uint32_t region = u % L::REGIONS;
                if (L::GROUP > 1 && held) {
                    ok = wait_for(&sh.abort, &sh.p_full[region], (u / L::REGIONS) & 1u, &sh.v_ready[vs], vp);
                    if (!ok) break;
                    if (*reinterpret_cast<const volatile uint32_t*>(sh.rose[region])) {
                        __syncwarp();
                        close(u - 1);
                        ok = wait(&sh.o_empty[o & 1], ((o >> 1) - 1) & 1u);
                    }
                } else {
                    ok = wait_for(&sh.abort, &sh.p_full[region], (u / L::REGIONS) & 1u, &sh.v_ready[vs], vp, &sh.o_empty[o & 1], ((o >> 1) - 1) & 1u);
                }
                if (!ok) break;
                tc_after();
                const bool adds = held > 0;
                const uint32_t d = tmem + 256 + (o & 1) * 128, v1 = v0 + vs * (PAGE_BYTES >> 4);
                ++t;
                --left;
                if (leader) {
#pragma unroll
                    for (int part = L::PPARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int kk = 0; kk < KVB / 16; ++kk)  // 8 columns of weights
                            if (kk < steps) mma_ts(d, tmem + L::part_at(u, part, kk >> 1) + (kk & 1) * 8, v1 + (uint32_t)(kk * 2048 / 16), IDESC_PV, adds || part < L::PPARTS - 1 || kk > 0);
                    at_commit((uint64_t*)&sh.v_empty[vs]);
                    at_commit((uint64_t*)&sh.w_empty[region]);
                    if (left == 0) arrive(&sh.piece_empty[k % PIECES]);
                }
                if (++held == L::GROUP || left == 0) close(u);
                __syncwarp();
                if (++vs == (uint32_t)plan.v_slots) vs = 0, vp ^= 1;
            }
            drain(leader);
        } else if (warp == W_SAFE) {
            // Values that weights of 0 may meet: rows behind a page's keys (up to a step of 16) and pages that were not there become
            // zeros, and so does what is not finite among the tree's: it is added to the rows that see it at the end.
            int t = 0, vs = 0;
            uint32_t vp = 0, k = ~0u;
            Piece* p = nullptr;
            if (U == 0 && lane == 0 && !ONE) a.meta[me] = make_int4(-1, 0, 0, 0);
#pragma unroll 1
            for (uint32_t u = 0; ok && u < U; ++u) {
                if (!p) {
                    ++k;
                    if (!wait(piece_bar(k), piece_par(k))) break;
                    p = &sh.piece[k % PIECES];
                    t = p->t0;
                    bool tree_ok = true;
                    if (p->t1 == p->tiles) {  // the tiles' values wait meanwhile, so all of it stays in registers
                        Line line;
                        line.begin(a.parents + (size_t)p->b * a.N, p->n, lane);
                        while (line.step(lane)) {
                        }
                        p->seen[lane] = line.seen[0];
                        p->seen[lane + 32] = line.seen[1];
                        tree_ok = line.in_order;
                        if (!tree_ok && lane == 0) set_err(c.err, TTS_BB_TREE_ERR_TREE);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        p->ok = tree_ok;
                        arrive(&sh.seen_full[k % PIECES]);
                        // of the share's first piece: its sequence, nodes, and whether it begins inside of that; bit 2: in order
                        if (k == 0 && !ONE) a.meta[me] = make_int4(p->b, p->n, (t > 0) | tree_ok << 2, 0);
                    }
                }
                if (!wait(&sh.v_full[vs], vp)) break;
                const bool tree = t == p->tiles - 1;
                const int keys = tree ? p->n : min(KVB, p->len - t * KVB), valid = sh.page[u % 16] >= 0 ? keys : 0;
                if (tree || valid < KVB) {
                    unsigned char* const v1 = v_ring + vs * PAGE_BYTES;
                    const auto at = [&](int key, int pc) {
                        return reinterpret_cast<uint4*>(v1 + (pc >> 3) * (PAGE_BYTES / 2) + sw128_off(key, pc & 7));
                    };
                    // 2 keys an instruction
#pragma unroll 1
                    for (int key = valid + (lane >> 4); key < (keys + 15) / 16 * 16; key += 2) *at(key, lane & 15) = make_uint4(0u, 0u, 0u, 0u);
                    if (tree) {
                        // 0 times what is finite is 0, and NaN else; the rows behind are zeros by now
                        __syncwarp();
                        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
                        __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 2
                        for (int key0 = lane >> 4; key0 < (valid + 15) / 16 * 16; key0 += 8) {
                            uint4 x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i] = *at(key0 + 2 * i, lane & 15);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __nv_bfloat162* const y = reinterpret_cast<const __nv_bfloat162*>(&x[i]);
#pragma unroll
                                for (int h = 0; h < 4; ++h) sum[h] = __hfma2(y[h], zero, sum[h]);
                            }
                        }
                        const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
                        if (__any_sync(0xffffffffu, __hisnan(__low2bfloat16(all)) || __hisnan(__high2bfloat16(all)))) {
#pragma unroll 1
                            for (int key = lane >> 4; key < valid; key += 2) {
                                const uint4 x = *at(key, lane & 15);
                                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                                bool bad = false;
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    if (!finite16(w[h])) { w[h] &= 0xFFFF0000u; bad = true; }
                                    if (!finite16(w[h] >> 16)) { w[h] &= 0xFFFFu; bad = true; }
                                }
                                if (!bad) continue;
                                *at(key, lane & 15) = make_uint4(w[0], w[1], w[2], w[3]);
                                atomicOr(&p->bad[key >> 5], 1u << (key & 31));
                            }
                        }
                    }
                    fence_async();
                }
                __syncwarp();
                if (lane == 0) arrive(&sh.v_ready[vs]);
                if (++vs == plan.v_slots) vs = 0, vp ^= 1;
                if (++t == p->t1) {
                    if (lane == 0) arrive(&sh.piece_empty[k % PIECES]);
                    p = nullptr;
                }
            }
        }
    } else if (warp < W_SUM) {
        // ---------------- scores to weights: thread = row; warps 0 .. 3 the share's even tiles, 4 .. 7 the odd ones
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
        const int group = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t u0 = 0;  // tiles before the piece
#pragma unroll 1
        for (uint32_t k = 0; ok; ++k) {
            if (!wait(piece_bar(k), piece_par(k))) break;
            const Piece& p = sh.piece[k % PIECES];
            if (p.b < 0) break;
            const int nt = p.t1 - p.t0, rows = 2 * p.n;
            if constexpr (F32) {
                // the queries, a warp 16 rows; those of the piece before were read by products that have ended
                if (u0 > 0 && !wait(&sh.s_full[(u0 - 1) % L::REGIONS], ((u0 - 1) / L::REGIONS) & 1u)) break;
                if (warp * 16 < rows) {
                    const float* const q = static_cast<const float*>(a.q) + (size_t)p.b * a.N * a.q_stride + 2 * p.g * HD;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        float4 x[4][2];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = (half * 4 + i) * 32 + lane, qr = warp * 16 + (e >> 4), pc = e & 15;
                            x[i][0] = x[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (qr < rows) {
                                const float4* const src = reinterpret_cast<const float4*>(q + (qr >> 1) * a.q_stride + (qr & 1) * HD + pc * 8);
                                x[i][0] = src[0];
                                x[i][1] = src[1];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = (half * 4 + i) * 32 + lane, qr = warp * 16 + (e >> 4), pc = e & 15;
                            if (qr >= plan.rows) continue;
                            unsigned char* const to = smem + (pc >> 3) * plan.rows * 128 + sw128_off(qr, pc & 7);
                            float f[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                            uint32_t w[4];
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    w[h] = bf16_pair(f[2 * h], f[2 * h + 1]);
                                    f[2 * h] -= __uint_as_float(w[h] << 16);
                                    f[2 * h + 1] -= __uint_as_float(w[h] & 0xFFFF0000u);
                                }
                                *reinterpret_cast<uint4*>(to + part * plan.rows * 256) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    fence_async();
                }
                __syncwarp();
                if (lane == 0) arrive(&sh.q_full[0]);
            }
            const bool mine = quarter * 32 < rows;
            float before = -INFINITY, l = 0.f;  // of this warp's tiles: the reference, and the sum of weights
#pragma unroll 1
            for (int j = (int)(u0 ^ group) & 1; j < nt; j += 2) {
                const int t = p.t0 + j;
                const uint32_t u = u0 + j, region = u % L::REGIONS, at = lanes + region * KVB;
                if (!wait(&sh.s_full[region], (u / L::REGIONS) & 1u)) break;
                float m = -INFINITY;
                bool rose = false;
                // the keys that count, a bit each, where not all do
                const bool tree = t == p.tiles - 1;
                const int valid = p.len - t * KVB;
                const bool there = sh.page[u % 16] >= 0, special = tree || valid < KVB || !there;
                u64 keys = ~0ull;
                if (special) {
                    if (tree && !wait(&sh.seen_full[k % PIECES], piece_par(k))) break;
                    keys = !there ? 0ull : tree ? (r < rows ? p.seen[r >> 1] : 0ull) : (1ull << valid) - 1;
                }
                if (mine) {
                    tc_after();
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int chunk = 0; chunk < 2; ++chunk) {
                        uint32_t s[32];
                        tm_ld32_nw(at + chunk * 32, s);
                        tm_wait_ld();
                        if (special) {  // and back: what follows is the same for all tiles
                            const uint32_t count = (uint32_t)(keys >> (chunk * 32));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(count >> i & 1)) s[i] = 0xFF800000u;  // -inf
                            tm_st32(at + chunk * 32, s);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
                    }
                    m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                // the maximum so far, from the warp of the tile before (waited for at a new piece too: no warp is two tiles ahead)
                if (u > 0) {
                    if (!wait(&sh.m_full[quarter][(u - 1) & 1], ((u - 1) >> 1) & 1u)) break;
                    if (u > u0) {
                        const float other = sh.m[(u - 1) % RING][r];
                        if ((m - other) * CS > L::SLACK) rose = r < rows;
                        else m = other;
                    }
                }
                if constexpr (L::GROUP > 1) {
                    rose = __any_sync(0xffffffffu, rose);
                    if (lane == 0) sh.rose[region][quarter] = rose;
                }
                sh.m[u % RING][r] = m;
                __syncwarp();
                if (lane == 0) arrive(&sh.m_full[quarter][u & 1]);
                if (mine) {
                    const float base = m == -INFINITY ? 0.f : m;
                    const u64 cs2 = pair(CS, CS), base2 = pair(-base, -base), minus = pair(-1.f, -1.f);
                    u64 sum[2] = {0, 0};
                    // the third parts' columns were taken by the product of this group's tile before
                    if (F32 && u >= 2 && !wait(&sh.w_empty[(u - 2) % L::REGIONS], ((u - 2) / L::REGIONS) & 1u)) break;
#pragma unroll 1
                    for (int chunk = 0; chunk < 2; ++chunk) {
                        uint32_t s[32], w[L::PPARTS][16];
                        tm_ld32_nw(at + chunk * 32, s);
                        tm_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x, y;
                            halves(mul2(add2(pair(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), base2), cs2), x, y);
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
                        for (int part = 0; part < L::PPARTS; ++part) tm_st16(lanes + L::part_at(u, part, chunk), w[part]);
                    }
                    float x, y, z, v;
                    halves(sum[0], x, y);
                    halves(sum[1], z, v);
                    l = (l == 0.f ? 0.f : l * at_ex2((before - base) * CS)) + ((x + y) + (z + v));
                    before = m;
                    if (j + 2 >= nt) sh.l[u % RING][r] = l;
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                tc_before();
                __syncwarp();
                if (lane == 0) arrive(&sh.p_full[region]);
            }
            if (!ok) break;
            u0 += nt;
            __syncwarp();
            if (lane == 0) arrive(&sh.piece_empty[k % PIECES]);
        }
    } else {
        // ---------------- a row's sums over the tiles: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SUM));
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + 256 + ((uint32_t)(quarter * 32) << 16);
        uint32_t u = 0, turn = 0;
#pragma unroll 1
        for (uint32_t k = 0; ok; ++k) {
            if (!wait(piece_bar(k), piece_par(k))) break;
            const Piece& p = sh.piece[k % PIECES];
            if (p.b < 0) break;
            const int nt = p.t1 - p.t0, rows = 2 * p.n;
            const bool mine = quarter * 32 < rows;
            u64 o[HD / 2];
#pragma unroll
            for (int i = 0; i < HD / 2; ++i) o[i] = 0;
            float m = -INFINITY, l = 0.f;  // the reference
#pragma unroll 1
            for (int t = 0; t < nt; ++t, ++u, ++turn) {
                if (!wait(&sh.o_full[turn & 1], (turn >> 1) & 1u)) break;
                // the buffer's tiles: from one on, to t
                const bool first = t == 0;
                const int more = sh.last[turn & 1] - (int)u;
                t += more;
                u += more;
                if (mine) {
                    tc_after();
                    const float now = sh.m[u % RING][r], f = first ? 0.f : now == m ? 1.f : at_ex2((m - now) * CS);
                    const u64 f2 = pair(f, f);
                    const uint32_t at = lanes + (turn & 1) * 128;
                    uint32_t x[2][32];  // the next 32 dims are on their way while these are added
                    tm_ld32_nw(at, x[0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tm_wait_ld();
                        if (i < 3) tm_ld32_nw(at + 32 * (i + 1), x[(i + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[16 * i + j] = fma2(o[16 * i + j], f2, pair(__uint_as_float(x[i & 1][2 * j]), __uint_as_float(x[i & 1][2 * j + 1])));
                    }
                    if (t + 2 >= nt) {  // of even and of odd tiles
                        l = (first || l == 0.f ? 0.f : l * f) + sh.l[u % RING][r];
                        if (more && t + 1 == nt) l += sh.l[(u - 1) % RING][r];
                    }
                    m = now;
                }
                tc_before();
                __syncwarp();
                if (lane == 0) arrive(&sh.o_empty[turn & 1]);
            }
            if (!ok) break;
            // the piece's end: code that runs this seldom comes from beyond the instruction cache, so it is kept short
            if (p.t1 == p.tiles && !wait(&sh.seen_full[k % PIECES], piece_par(k))) break;
            if (mine) {
                T* const to = static_cast<T*>(a.out) + ((size_t)p.b * a.N * NQ + 2 * p.g) * HD;
                T* const row = to + ((size_t)(r >> 1) * NQ + (r & 1)) * HD;
                float4* const part = a.part + ((size_t)me * 2 + !p.first) * PART * 128 + r;
                const auto four = [&](int i) {
                    float4 x;
                    halves(o[2 * i], x.x, x.y);
                    halves(o[2 * i + 1], x.z, x.w);
                    return x;
                };
                if (!ONE && !p.whole) {
                    if (r < rows) {  // rows side by side: whole lines
#pragma unroll
                        for (int i = 0; i < HD / 4; ++i) part[i * 128] = four(i);
                        part[(HD / 4) * 128] = make_float4(m, l, 0.f, 0.f);
                    }
                } else if (p.ok) {
                    const float f = 1.f / l;  // l is 0 where all scores are -inf: NaN, as the formula's
                    const u64 f2 = pair(f, f), none = pair(-0.f, -0.f);
#pragma unroll
                    for (int i = 0; i < HD / 2; ++i) o[i] = fma2(o[i], f2, none);
                    if constexpr (F32) {
                        // 128 bytes of each row at a time through the warp's stage: whole lines (straight from the lanes, which hold a row each, 32
                        // lines an instruction)
                        unsigned char* const stage = smem + plan.stages<F32>() + quarter * L::STAGE;
#pragma unroll
                        for (int d0 = 0; d0 < HD; d0 += 32) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(stage + sw128_off(lane, i)) = four(d0 / 4 + i);
                            __syncwarp();
#pragma unroll 1
                            for (int at = quarter * 32 + (lane >> 3); at < min(rows, quarter * 32 + 32); at += 4)
                                *reinterpret_cast<float4*>(to + ((size_t)(at >> 1) * NQ + (at & 1)) * HD + d0 + (lane & 7) * 4) =
                                    *reinterpret_cast<const float4*>(stage + sw128_off(at & 31, lane & 7));
                        }
                    } else if (r < rows) {
#pragma unroll
                        for (int i = 0; i < HD / 8; ++i) {
                            const float4 x = four(2 * i), y = four(2 * i + 1);
                            *reinterpret_cast<uint4*>(row + i * 8) = make_uint4(bf16_pair(x.x, x.y), bf16_pair(x.z, x.w), bf16_pair(y.x, y.y), bf16_pair(y.z, y.w));
                        }
                    }
                }
                if (p.bad[0] | p.bad[1]) {  // what was set aside is added to what stands there now
                    __syncwarp();
#pragma unroll 1
                    for (u64 left = r < rows ? ((u64)p.bad[1] << 32 | p.bad[0]) & p.seen[r >> 1] : 0ull; left; left &= left - 1) {
                        const bf16* const v = a.v + ((size_t)p.b * a.N + __ffsll(left) - 1) * a.kv_stride + p.g * HD;
#pragma unroll 1
                        for (int d = 0; d < HD; ++d) {
                            const float y = bf2f(v[d]);
                            if (fabsf(y) <= 3.4028235e38f) continue;
                            if (!ONE && !p.whole) reinterpret_cast<float*>(part + (d >> 2) * 128)[d & 3] += y;
                            else if (p.ok) row[d] = (T)((float)row[d] + y);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.piece_empty[k % PIECES]);
        }
    }
    if (!ok && lane == 0) set_err(c.err, TTS_BB_TREE_ERR_TIMEOUT);
    tc_before();
    __syncthreads();
    if (warp == W_PV) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
    }
}

// grid (8 (shares - 1), rows / 32, 4), 128 threads: the pieces of the (sequence, KV head) that the end of a share cuts first. A lane
// a row, a warp 8 of the 128 dims. A share's first piece stands in its place 0, the piece that ends it in place 1.
template <typename T>
__global__ void __launch_bounds__(128) k_tree_combine(TreeArgs a, int shares) {
    pdl_wait();
    pdl_trigger();
    const int s0 = blockIdx.x / NKV, g = blockIdx.x % NKV, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y * 32 + lane;
    // the first pieces of this share and of those behind it: fewer than 32
    const int4 meta = s0 + lane < shares ? a.meta[(s0 + lane) * NKV + g] : make_int4(-1, 0, 0, 0);
    const int it = __shfl_sync(0xffffffffu, meta.x, 1);
    const uint32_t goes_on = __ballot_sync(0xffffffffu, lane > 0 && meta.x == it && (meta.z & 1));
    // (and after a wait that ran out a place may hold anything)
    if (it < 0 || it >= a.B || !(goes_on & 2)) return;  // the share behind begins with a new one
    const int head = __shfl_sync(0xffffffffu, meta.x, 0), inside = __shfl_sync(0xffffffffu, meta.z, 0) & 1;
    if (head == it && inside) return;  // begun before this share
    const int more = __ffs(~(goes_on >> 1)) - 1;  // shares behind this one
    const int n = min(__shfl_sync(0xffffffffu, meta.y, 1), a.N);
    const bool in_order = __shfl_sync(0xffffffffu, meta.z, more) >> 2 & 1;  // the last piece holds the tree
    if (r >= 2 * n || !in_order) return;
    const auto at = [&](int i) { return a.part + ((size_t)((s0 + i) * NKV + g) * 2 + (i == 0 && head != it)) * PART * 128 + r; };
    float M = -INFINITY, l = 0.f;
    float4 o[2] = {};
    const int d0 = (blockIdx.z * 4 + warp) * 2;
#pragma unroll 1
    for (int i0 = 0; i0 <= more; i0 += 8) {  // eight pieces at once
        float4 w[8], x[8][2];
        float top = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4* const p = at(min(i0 + i, more));
            w[i] = p[(HD / 4) * 128];
            x[i][0] = p[d0 * 128];
            x[i][1] = p[(d0 + 1) * 128];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, w[i].x);
        const float base = top == -INFINITY ? 0.f : top, f0 = at_ex2((M - base) * CS);
        M = top;
        l *= f0;
#pragma unroll
        for (int d = 0; d < 2; ++d) { o[d].x *= f0; o[d].y *= f0; o[d].z *= f0; o[d].w *= f0; }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i > more) break;
            const float f = at_ex2((w[i].x - base) * CS);
            l += f * w[i].y;
#pragma unroll
            for (int d = 0; d < 2; ++d) { o[d].x += f * x[i][d].x; o[d].y += f * x[i][d].y; o[d].z += f * x[i][d].z; o[d].w += f * x[i][d].w; }
        }
    }
    const float f = 1.f / l;
    T* const to = static_cast<T*>(a.out) + (((size_t)it * a.N + (r >> 1)) * NQ + 2 * g + (r & 1)) * HD + d0 * 4;
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
        for (int d = 0; d < 2; ++d) *reinterpret_cast<float4*>(to + d * 4) = make_float4(o[d].x * f, o[d].y * f, o[d].z * f, o[d].w * f);
    } else {
        *reinterpret_cast<uint4*>(to) = make_uint4(bf16_pair(o[0].x * f, o[0].y * f), bf16_pair(o[0].z * f, o[0].w * f), bf16_pair(o[1].x * f, o[1].y * f),
                                                   bf16_pair(o[1].z * f, o[1].w * f));
    }
}

// Shares of the launch: 8 blocks each, one an SM in all, or a tile a share where there are fewer. Few and short sequences are not cut, which
// saves the deal and the launch that merges, as long as what a cut would take from the longest is worth fewer than 10 tiles (fp32: 5). bf16, 6
// nodes: 1 x 333 keys 8.5 us (and 3 of the host's less), in shares 9.4; 1 x 600 10.6 and 10.8; 1 x 1200 15.6 and 11.5; 19 x 120..1200 16.5 and
// 18.7. fp32, 25 nodes: 1 x 100 9.5 and 9.4, 1 x 320 12.4 and 10.4, 12 x 64..640 18.1 and 19.9. Up to 20 tiles: where only one sequence is
// long, it bounds all.
constexpr int ONE_TILES = 20;
bool one_block(int B, int max_len, bool f32) {
    const int t = tiles_of(max_len);
    return B <= SHARES && t <= ONE_TILES && t * (SHARES - B) <= SHARES * (f32 ? 5 : 10);
}
int share_count(int B, int max_len) { return (int)std::min<long long>(SHARES, (long long)B * tiles_of(max_len)); }
constexpr size_t META_BYTES = (SHARES * NKV * sizeof(int4) + 255) / 256 * 256;
// As many pages of K and V as fit behind the queries.
template <bool F32>
Plan plan_of(int N) {
    Plan p{(2 * N + 7) / 8 * 8, 0, 0};
    const int pages = (SMEM_MAX - p.bytes<F32>()) / PAGE_BYTES;
    p.k_slots = std::min(MAX_SLOTS, pages / 2);
    p.v_slots = std::min(MAX_SLOTS, pages - p.k_slots);
    return p;
}

}  // namespace

TTS_API size_t tts_bb_tree_attention_workspace(int B, int N, int max_len) {
    if (!tree_ok(B, N) || max_len < 0 || max_len > (1 << 30) || (long long)B * max_len > (1ll << 33)) return 0;
    // (what bf16 calls cut, fp32 calls cut too)
    return one_block(B, max_len, true) ? 0 : META_BYTES + (size_t)share_count(B, max_len) * NKV * 2 * PART * 128 * sizeof(float4);
}

TTS_API tts_bb_status tts_bb_tree_attention(const tts_bb_kv_cache* cache, int layer, int B, int N, const void* q, int type,
                                            int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                            const int32_t* parents, const int32_t* n_nodes, const int32_t* seqs,
                                            const int32_t* kv_lens, int max_len, void* out, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    if (!cache_ok(cache) || layer < 0 || layer >= cache->n_layers || !tree_ok(B, N) || !q || !k || !v || !parents || !kv_lens || !out ||
        (type != TTS_BB_T_F32 && type != TTS_BB_T_BF16) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
        q_stride < NQ * HD || q_stride % (type == TTS_BB_T_F32 ? 4 : 8) || kv_stride < NKV * HD || kv_stride % 8 ||
        q_stride > (1ll << 38) || kv_stride > (1ll << 38) || max_len < 0 || max_len > (1 << 30) || (long long)B * max_len > (1ll << 33) ||
        (long long)max_len > (long long)cache->blocks_per_seq * KVB || (!seqs && B > cache->n_seqs) || !words_aligned(parents, n_nodes, seqs, kv_lens))
        return TTS_BB_E_INVALID;
    const size_t need = tts_bb_tree_attention_workspace(B, N, max_len);
    if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const Pages c = pages_of(cache, layer);
    CUtensorMap pool_map, k_map, v_map, q_map;
    if (!tc_make_map_parts(&pool_map, c.pool, c.n_blocks * 2 * NKV * KVB, 2, HD, KVB) ||
        !tc_make_map_parts(&k_map, k, B * N, 2 * NKV, kv_stride, KVB) || !tc_make_map_parts(&v_map, v, B * N, 2 * NKV, kv_stride, KVB) ||
        (type == TTS_BB_T_BF16 && !tc_make_map_heads(&q_map, q, B * N, NQ, q_stride, N)))
        return TTS_BB_E_CUDA;
    if (type != TTS_BB_T_BF16) q_map = k_map;  // not used
    const TreeArgs a{q, static_cast<const bf16*>(v), q_stride, kv_stride, parents, n_nodes, seqs, kv_lens, B, N, max_len, out,
                     static_cast<int4*>(workspace), reinterpret_cast<float4*>(static_cast<char*>(workspace) + META_BYTES)};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    bool regs = true;
    const bool one = one_block(B, max_len, type == TTS_BB_T_F32);
    const auto go = [&](auto f32, auto single) {
        constexpr bool F32 = decltype(f32)::value, ONE = decltype(single)::value;
        static SmemState state;
        allow_smem(state, k_tree_attn<F32, ONE>, SMEM_MAX);
        // what its warps deal anew has to be there at the launch: they would wait for it
        static const bool enough = [] {
            cudaFuncAttributes f{};
            return cudaFuncGetAttributes(&f, k_tree_attn<F32, ONE>) == cudaSuccess && f.numRegs >= 128;
        }();
        regs = enough;
        if (!regs) return;
        const Plan plan = plan_of<F32>(N);
        const int shares = ONE ? B : share_count(B, max_len);
        launch_pdl(k_tree_attn<F32, ONE>, shares * NKV, NT, plan.bytes<F32>(), st, pool_map, k_map, v_map, q_map, c, a, plan);
        if (!ONE && shares > 1 && tiles_of(max_len) > 1)
            launch_pdl(k_tree_combine<std::conditional_t<F32, float, bf16>>, dim3((shares - 1) * NKV, (2 * N + 31) / 32, 4), 128, 0, st, a, shares);
    };
    if (type == TTS_BB_T_F32) one ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else one ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    return regs ? launched() : TTS_BB_E_CUDA;
}
