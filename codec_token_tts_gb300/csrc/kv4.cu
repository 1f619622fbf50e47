// Paged KV cache held in 4 bits: append (q/k RMSNorm, half-rotate RoPE, quantisation), read-back and
// grouped-query attention (16 query heads, 8 KV heads of 128), all on the caller's buffers.
//
// Format. A cache block holds K then V of 64 tokens for the 8 KV heads as 16 tiles of 4608 bytes. A
// tile: 64 code rows of 64 bytes, then 64 parameter rows of 8 bytes. The 128 dims of a token's head are
// two groups of 64 (dims 0..63 and 64..127, the two halves that RoPE pairs). Word w of a code row holds
// dims 64 (w & 1) + 8 (w >> 1) + i in nibble i, so that both 8-byte pieces (V: one piece a lane) and
// 16-byte pieces (K: one piece a lane) carry both groups. A parameter row: (bf16 scale, bf16 offset) of
// each group, value = scale * (code + 128 + offset). The offset is a whole number, -249 .. -7, so code +
// 128 + offset is a whole number below 256 in magnitude: exact in bf16, which is what the tensor cores
// of the attention take.
//
// Quantisation of a group x[64]: scale = bf16(max((hi - lo) / 15, max|x| / 120)), zero = rint(lo / scale),
// code = clamp(rint(x / scale) - zero, 0, 15), offset = zero - 128. The second term bounds zero by 121.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "../../include/tts_bb.h"

#define TTS_API extern "C" __attribute__((visibility("default")))

using namespace ttsbb;

namespace {

constexpr int TILE = TTS_BB_KV4_TILE_BYTES;
constexpr size_t BLOCK = TTS_BB_KV4_BLOCK_BYTES;
constexpr int PAR = KVB * HD / 2;  // byte offset of a tile's parameter rows
static_assert(TILE == PAR + KVB * 8 && BLOCK == (size_t)2 * NKV * TILE, "tile layout");
constexpr float LOG2E = 1.4426950408889634f;

struct Cache {
    uint8_t* pool;
    const int32_t* table;
    int32_t* err;
    int n_blocks, n_seqs, bps;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
// The block of (sequence row, position), or -1 with the reason in *err.
__device__ __forceinline__ int find_block(const Cache& c, int seq, int pos, bool report) {
    if (seq >= c.n_seqs || pos < 0 || pos / KVB >= c.bps) {
        if (report) set_err(c.err, TTS_BB_KV4_ERR_RANGE);
        return -1;
    }
    const int p = c.table[(size_t)seq * c.bps + pos / KVB];
    if (p < 0 || p >= c.n_blocks) {
        if (report) set_err(c.err, TTS_BB_KV4_ERR_PAGE);
        return -1;
    }
    return p;
}

// ---------------------------------------------------------------- append
// A head is held by 8 lanes (a warp holds four heads): lane l of them has dims 8l .. 8l + 7 of both groups, so the pairs
// (i, i + 64) that RoPE rotates are a lane's own, and so are words 2l and 2l + 1 of the code row. x[0..7]: group 0, x[8..15]:
// group 1.
struct Quant {
    uint32_t codes[2];  // a word of each group
    uint32_t par[2];    // bf16 scale | bf16 offset << 16
};

__device__ __forceinline__ float min3(float a, float b, float c) {
    float m;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
// two floats an instruction
typedef unsigned long long f2;
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
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
// over a head's 8 lanes; a NaN stays one
__device__ __forceinline__ float head_min(float v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) { const float w = __shfl_xor_sync(0xffffffffu, v, o); v = min3(v, w, w); }
    return v;
}
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) { const float w = __shfl_xor_sync(0xffffffffu, v, o); v = max3(v, w, w); }
    return v;
}
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return bf2f(x); }
__device__ __forceinline__ uint32_t bf_bits(float x) { return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// 8 values as they stand in memory (so few registers hold a row ahead of its use), and as pairs
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + i);
    return r;
}
__device__ __forceinline__ void pairs_of(const Raw8<float>& r, f2* v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[2 * i] = pair(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
        v[2 * i + 1] = pair(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
    }
}
__device__ __forceinline__ void pairs_of(const Raw8<bf16>& r, f2* v) {
    float f[8];
    unpack8(r.v[0], f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}
// 8 values as pairs; 16- (bf16) or 32-byte pieces
__device__ __forceinline__ void load8(const float* p, f2* v) {
    const float4 a = load4(p), b = load4(p + 4);
    v[0] = pair(a.x, a.y); v[1] = pair(a.z, a.w); v[2] = pair(b.x, b.y); v[3] = pair(b.z, b.w);
}
__device__ __forceinline__ void load8(const bf16* p, f2* v) {
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(p), f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}
__device__ __forceinline__ void store8(float* p, const f2* v) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) halves(v[e], f[2 * e], f[2 * e + 1]);
    store4(p, f);
    store4(p + 4, f + 4);
}
__device__ __forceinline__ void store8(bf16* p, const f2* v) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        halves(v[e], a, b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        o[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Numbers as the unevaluated sum of two floats, h the rounding of h + l: 48 bits, by error-free sums (Knuth) and products
// (by fma). Doubles would do as well, but this GPU has few units for them: a pair of heads took 10 us in them.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two norm2(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two sum2(float a, float b) {
    const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    const Two s = sum2(a.h, b.h);
    return norm2(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h);
    return norm2(p, __fmaf_rn(a.h, b.h, -p) + __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h)));
}
__device__ __forceinline__ Two neg2(Two a) { return {-a.h, -a.l}; }
__device__ __forceinline__ bool less2(Two a, Two b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }
__device__ __forceinline__ Two div2(Two a, float b) {  // b a whole number: its products with 24 bits are kept by fma
    const float q = __fdiv_rn(a.h, b);
    return norm2(q, __fdiv_rn(__fadd_rn(__fmaf_rn(-q, b, a.h), a.l), b));
}
__device__ __forceinline__ Two peer2(Two a, int o) { return {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)}; }
// x / s to the nearest whole number, ties to even, from one of the two next to it: s has 8 bits, so (k + 1/2) s is exact and
// one fma tells on which side of it x lies
__device__ __forceinline__ float rint2(float k, Two x, float s) {
    const float up = __fadd_rn(__fmaf_rn(-(k + 0.5f), s, x.h), x.l), down = __fadd_rn(__fmaf_rn(-(k - 0.5f), s, x.h), x.l);
    const bool odd = (int)k & 1;
    return up > 0.f || (up == 0.f && odd) ? k + 1.f : down < 0.f || (down == 0.f && odd) ? k - 1.f : k;
}
__device__ __forceinline__ float rint2(Two x, float s) { return rint2(rintf(__fdiv_rn(x.h, s)), x, s); }

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The inverse root mean square of a head's row (x: at this lane's first dim), in 48 bits
template <typename T>
__device__ __forceinline__ Two inverse_norm(const T* x, float eps) {
    Two part[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const Two a = {to_float(x[e]), 0.f}, b = {to_float(x[HD / 2 + e]), 0.f}, c = {to_float(x[4 + e]), 0.f}, d = {to_float(x[HD / 2 + 4 + e]), 0.f};
        part[e] = add2(add2(mul2(a, a), mul2(b, b)), add2(mul2(c, c), mul2(d, d)));
    }
    Two ss = add2(add2(part[0], part[1]), add2(part[2], part[3]));
#pragma unroll
    for (int o = 4; o; o >>= 1) ss = add2(ss, peer2(ss, o));
    ss = add2({ss.h * (1.f / HD), ss.l * (1.f / HD)}, {eps, 0.f});
    // one Newton step doubles the 23 bits of rsqrtf: r (1 + (1 - ss r r) / 2)
    const Two r = {rsqrtf(ss.h), 0.f};
    const Two err = add2({1.f, 0.f}, neg2(mul2(ss, mul2(r, r))));
    return norm2(r.h, r.h * 0.5f * err.h);
}
// dims e and 64 + e of this lane's of a key: normalised, with its gain, rotated
template <typename T>
__device__ __forceinline__ void key_values(const T* x, const bf16* gain, const float* cs, const float* sn, Two r, int e, Two (&z)[2]) {
    const Two a = mul2(mul2({to_float(x[e]), 0.f}, r), {bf2f(gain[e]), 0.f});
    const Two b = mul2(mul2({to_float(x[HD / 2 + e]), 0.f}, r), {bf2f(gain[HD / 2 + e]), 0.f});
    const Two c = {cs[e], 0.f}, s = {sn[e], 0.f};
    z[0] = add2(mul2(a, c), neg2(mul2(b, s)));
    z[1] = add2(mul2(b, c), mul2(a, s));
}

// The definition, in 48 bits: of the head's row x (normalised with its gain and rotated here where gain is given), lane l's dims;
// all pointers at this lane's first dim. Seldom needed, so its code is kept short (what a launch runs once comes from
// memory): value by value, in one loop that goes over them twice, for the ranges and for the codes.
template <typename T>
__device__ __forceinline__ void quant48(const T* x, const bf16* gain, const float* cs, const float* sn, float eps, Quant& q) {
    Two r = {1.f, 0.f};
    if (gain) r = inverse_norm(x, eps);
    Two lo[2], hi[2];
    float s[2] = {1.f, 1.f}, zero[2] = {0.f, 0.f};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        lo[g] = {INFINITY, 0.f};
        hi[g] = {-INFINITY, 0.f};
        q.codes[g] = 0u;
    }
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        const int e = i & 7;
        Two z[2] = {{to_float(x[e]), 0.f}, {to_float(x[HD / 2 + e]), 0.f}};
        if (gain) key_values(x, gain, cs, sn, r, e, z);
        if (i < 8) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                lo[g] = less2(z[g], lo[g]) ? z[g] : lo[g];
                hi[g] = less2(hi[g], z[g]) ? z[g] : hi[g];
            }
            if (i < 7) continue;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
                for (int o = 4; o; o >>= 1) {
                    const Two a = peer2(lo[g], o), b = peer2(hi[g], o);
                    lo[g] = less2(a, lo[g]) ? a : lo[g];
                    hi[g] = less2(hi[g], b) ? b : hi[g];
                }
                const Two range = div2(add2(hi[g], neg2(lo[g])), 15.f), most = div2(less2(hi[g], neg2(lo[g])) ? neg2(lo[g]) : hi[g], 120.f);
                const uint32_t sb = bf_bits(less2(range, most) ? most.h : range.h);
                s[g] = __uint_as_float(sb << 16);
                zero[g] = s[g] > 0.f ? rint2(lo[g], s[g]) : 0.f;
                q.par[g] = sb | bf_bits(zero[g] - 128.f) << 16;
            }
        } else {
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (s[g] > 0.f) q.codes[g] |= (uint32_t)fminf(rint2(z[g], s[g]) - zero[g], 15.f) << (4 * e);
        }
    }
}

// The same for one group (the pairs x of a lane) in 32 bits. Keys are known to within delta; values are exact (EXACT), and
// x / scale is then divided out in full: a value halfway between two codes, which bf16 rows meet often, goes to the even whole
// number. SURE_SCALE: the scale's rounding could not fall the other way (nor is the group too small for this arithmetic);
// FINITE: all values are; unsure: a bit for each value whose code could be another. Rounding is by adding and subtracting
// 1.5 2^23; the lowest value is one of the x, so its code is 0 and no code is below.
enum { SURE_SCALE = 1, FINITE = 2 };
constexpr float MAGIC = 12582912.f;
template <bool EXACT>
__device__ __forceinline__ int quant32(const f2* x, float delta, uint32_t& codes, uint32_t& par, uint32_t& unsure) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) halves(x[e], v[2 * e], v[2 * e + 1]);
    const float lo = head_min(min3(min3(min3(v[0], v[1], v[2]), v[3], v[4]), min3(v[5], v[6], v[7]), v[7]));
    const float hi = head_max(max3(max3(max3(v[0], v[1], v[2]), v[3], v[4]), max3(v[5], v[6], v[7]), v[7]));
    const float amax = max3(hi, -lo, -lo);
    const float s0 = fmaxf((hi - lo) * (1.f / 15.f), amax * (1.f / 120.f));
    const float es = 0.15f * delta + s0 * 0x1p-22f;  // three roundings, and x's
    const uint32_t sb = bf_bits(s0 - es);
    const float s = __uint_as_float(sb << 16), inv = rcp(s);
    // bound of the error of x / s: EXACT: one rounding; else two and the reciprocal's, and x's
    const float rel = EXACT ? 0x1p-23f * amax * inv : 0x1p-22f * amax * inv + delta * inv;
    float t0 = lo * inv;
    if (EXACT) t0 = fmaf(fmaf(-t0, s, lo), inv, t0);
    const float zero = (t0 + MAGIC) - MAGIC;
    const f2 inv2 = both(inv), magic = both(MAGIC), unmagic = both(-MAGIC), minus = both(-1.f), unzero = both(-zero), ms = both(-s);
    float c[8], d[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f2 t = mulp(x[e], inv2);
        if (EXACT) t = fmap(fmap(t, ms, x[e]), inv2, t);
        const f2 k = addp(addp(t, magic), unmagic);
        halves(fmap(k, minus, t), d[2 * e], d[2 * e + 1]);
        halves(addp(k, unzero), c[2 * e], c[2 * e + 1]);
    }
    unsure = 0u;
    const float far = max3(max3(max3(fabsf(d[0]), fabsf(d[1]), fabsf(d[2])), fabsf(d[3]), fabsf(d[4])), max3(fabsf(d[5]), fabsf(d[6]), fabsf(d[7])), 0.f);
    if (far >= 0.5f - rel)  // from a whole number
#pragma unroll
        for (int e = 0; e < 8; ++e) unsure |= fabsf(d[e]) >= 0.5f - rel ? 1u << e : 0u;
    uint32_t h[2];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = fminf(c[e], 15.f);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        h[i] = __float_as_uint(fmaf(fmaf(c[4 * i + 3], 16.f, c[4 * i + 2]), 256.f, fmaf(c[4 * i + 1], 16.f, c[4 * i])) + 8388608.f);
    codes = __byte_perm(h[0], h[1], 0x5410);
    par = sb | bf_bits(zero - 128.f) << 16;
    return (sb == bf_bits(s0 + es) && s0 > 1e-30f ? SURE_SCALE : 0) | (amax < INFINITY ? FINITE : 0);
}
// The unsure codes of keys whose scale is sure, decided in 48 bits: the warp goes through the places that any lane asks for.
// False where one of them is a group's lowest value (code 0), whose rounding moves the zero point.
template <typename T>
__device__ __forceinline__ bool settle(const T* x, const bf16* gain, const float* cs, const float* sn, float eps, uint32_t unsure, Quant& q) {
    const Two r = inverse_norm(x, eps);
    uint32_t all = __reduce_or_sync(0xffffffffu, unsure);
    bool fine = true;
    while (all) {
        const int e = __ffs(all) - 1, g = e >> 3, d = e & 7;
        all &= all - 1;
        Two z[2];
        key_values(x, gain, cs, sn, r, d, z);
        const uint32_t par = g ? q.par[1] : q.par[0];
        const float s = __uint_as_float(par << 16), zero = __uint_as_float(par & 0xFFFF0000u) + 128.f;
        const float k = rint2(g ? z[1] : z[0], s) - zero;
        if (unsure >> e & 1u) {
            fine = fine && k > 0.f && ((g ? q.codes[1] : q.codes[0]) >> (4 * d) & 15u) != 0u;
            const uint32_t put = (uint32_t)fminf(fmaxf(k, 0.f), 15.f) << (4 * d), keep = ~(15u << (4 * d));
            if (g) q.codes[1] = (q.codes[1] & keep) | put;
            else q.codes[0] = (q.codes[0] & keep) | put;
        }
    }
    return fine;
}

// grid (tokens at most, parts), 128 threads: a token's 16 q heads, or its 8 k and 8 v heads, four a warp; a block goes on with
// the token a grid further, whose row is on its way meanwhile. q and k: RMSNorm over the head with its gain, then the
// pairs (i, i + 64) rotated by the token's row of the cos / sin tables.
// Bound by memory (8 or 16 KB read, 4 or 8 KB + 1152 B written for a token) and, nearly as much, by its instructions: 24463 bf16
// tokens (16 prompts padded to 2048) 107 us, 3.2 TB/s (memory alone: 50 us); fp32 159 us, 4.0 TB/s (95 us).
//
// A code next to a border between two would fall either way on the rounding of a 32-bit norm, and one
// code off is a whole scale. Where quant32 is not sure (about 3 % of the fours of k heads) those codes, or the four heads where
// it is the scale, are done again in 48 bits, so that all are those of the definition.
// delta bounds the 32-bit error of a rotated key: relative to |x_i cos| + |x_j sin|, 2^-24 times 5 (half of the sum of
// squares' 8 roundings, and the mean's two) + 2 (Newton's step) + 2 (norm and gain) + 2 (rotation) is below 12 * 2^-24.
// WHAT: HEADS_Q, HEADS_KV, or both
enum { HEADS_Q = 1, HEADS_KV = 2 };
template <int WHAT, typename TI, typename TQ>
__global__ void __launch_bounds__(128, 6) k_kv4_append(int T, const TI* __restrict__ qkv, long long stride,
                                                    const bf16* __restrict__ gq, const bf16* __restrict__ gk, float eps,
                                                    const float* __restrict__ cos_t, const float* __restrict__ sin_t,
                                                    int n_pos, const int32_t* __restrict__ seqs,
                                                    const int32_t* __restrict__ positions, Cache c, TQ* __restrict__ q_out) {
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    const int warp = (WHAT == HEADS_KV ? 4 : blockIdx.y * 4) + (threadIdx.x >> 5), lane = threadIdx.x & 31, l = lane & 7;
    const int head = warp * 4 + (lane >> 3);
    // a token's row is fetched while the one before is at hand, its place one token earlier (rows of padding stay unread)
    int t = blockIdx.x, next_seq = seqs[t], next_pos = positions[t], far_seq = -1, far_pos = 0;
    Raw8<TI> next0 = {}, next1 = {};
    if (t + (int)gridDim.x < T) { far_seq = seqs[t + gridDim.x]; far_pos = positions[t + gridDim.x]; }
    {
        const TI* const first = qkv + (size_t)t * stride + head * HD + l * 8;
        next0 = raw8(first);
        next1 = raw8(first + HD / 2);
    }
    for (; t < T; t += gridDim.x) {
        const TI* const row = qkv + (size_t)t * stride + head * HD + l * 8;
        const int seq = next_seq, pos = next_pos;
        f2 x[8];  // pairs of dims of group 0, then of group 1
        pairs_of(next0, x);
        pairs_of(next1, x + 4);
        next_seq = far_seq;
        next_pos = far_pos;
        far_seq = -1;
        if (next_seq >= 0) {
            const TI* const ahead = row + (size_t)gridDim.x * stride;
            next0 = raw8(ahead);
            next1 = raw8(ahead + HD / 2);
        }
        if (t + 2ll * gridDim.x < T) { far_seq = seqs[t + 2 * gridDim.x]; far_pos = positions[t + 2 * gridDim.x]; }
        if (seq < 0) continue;
        if (pos >= n_pos) {
            if (threadIdx.x == 0) set_err(c.err, TTS_BB_KV4_ERR_RANGE);
            continue;
        }
        const int phys = find_block(c, seq, pos, threadIdx.x == 0);
        if (phys < 0) continue;
        const bool is_q = WHAT == HEADS_Q || (WHAT != HEADS_KV && warp < 4), norm = is_q || warp < 6;
        f2 y[8];
        float delta = 0.f;
        if (norm) {
            f2 g[8], cs[4], sn[4];
            const bf16* const gain = (is_q ? gq : gk) + l * 8;
            load8(gain, g);
            load8(gain + HD / 2, g + 4);
            load8(cos_t + (size_t)pos * (HD / 2) + l * 8, cs);
            load8(sin_t + (size_t)pos * (HD / 2) + l * 8, sn);
            f2 ss[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) ss[e] = fmap(x[e], x[e], mulp(x[4 + e], x[4 + e]));
            float s0, s1;
            halves(addp(addp(ss[0], ss[1]), addp(ss[2], ss[3])), s0, s1);
            const float ms = head_sum(s0 + s1) * (1.f / HD) + eps, r0 = rsqrtf(ms);
            // a step of Newton's takes rsqrtf's last bits
            const f2 r = both(fmaf(r0 * 0.5f, fmaf(-ms * r0, r0, 1.f), r0)), minus = both(-1.f);
            f2 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mulp(mulp(x[e], r), g[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = fmap(v[e], cs[e], mulp(mulp(v[4 + e], sn[e]), minus));
                y[4 + e] = fmap(v[4 + e], cs[e], mulp(v[e], sn[e]));
            }
            if (is_q) {
                if (q_out) {
                    TQ* const to = q_out + ((size_t)t * NQ + head) * HD + l * 8;
                    store8(to, y);
                    store8(to + HD / 2, y + 4);
                }
                continue;
            }
            float m = 0.f, n = 0.f;  // |v_i cos| + |v_j sin| is at most m n
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a, b;
                halves(v[e], a, b);
                m = max3(m, fabsf(a), fabsf(b));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, b, p, q;
                halves(cs[e], a, b);
                halves(sn[e], p, q);
                n = max3(n, fabsf(a) + fabsf(p), fabsf(b) + fabsf(q));
            }
            delta = 0x1.8p-21f * head_max(m * n);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e];
    }
        Quant q;
        uint32_t un0, un1;
        int sure0, sure1;
        bool again;  // in 48 bits
        const size_t at = (size_t)pos * (HD / 2) + l * 8;
        if (norm) {
            sure0 = quant32<false>(y, delta, q.codes[0], q.par[0], un0);
            sure1 = quant32<false>(y + 4, delta, q.codes[1], q.par[1], un1);
            again = __any_sync(0xffffffffu, !(sure0 & sure1 & SURE_SCALE));
            if (!again && __any_sync(0xffffffffu, un0 | un1))
                again = __any_sync(0xffffffffu, !settle(row, gk + l * 8, cos_t + at, sin_t + at, eps, un0 | un1 << 8, q));
        } else {
            sure0 = quant32<true>(y, 0.f, q.codes[0], q.par[0], un0);
            sure1 = quant32<true>(y + 4, 0.f, q.codes[1], q.par[1], un1);
            // quotients of two bf16 numbers that are not halfway stay further from it than their rounding
            again = __any_sync(0xffffffffu, !(sure0 & sure1 & SURE_SCALE) || (sizeof(TI) == 4 && (un0 | un1)));
        }
        if (again) quant48(row, norm ? gk + l * 8 : nullptr, cos_t + at, sin_t + at, eps, q);
        // a group with a value that is not finite is held as NaN
        if (!(sure0 & FINITE)) { q.codes[0] = 0u; q.par[0] = 0xC3007FC0u; }
        if (!(sure1 & FINITE)) { q.codes[1] = 0u; q.par[1] = 0xC3007FC0u; }
        uint8_t* const tile = c.pool + (size_t)phys * BLOCK + (size_t)(head - NQ) * TILE;  // k heads 0..7, then v heads
        const int tok = pos % KVB;
        *reinterpret_cast<uint2*>(tile + tok * (HD / 2) + l * 8) = make_uint2(q.codes[0], q.codes[1]);
        if (l == 0) *reinterpret_cast<uint2*>(tile + PAR + tok * 8) = make_uint2(q.par[0], q.par[1]);
    }
}

// ---------------------------------------------------------------- read
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// grid ceil(T / N), 256 threads: thread (K or V, head, word) unpacks one word (8 dims) of each of N tokens, whose addresses
// and words are all on their way before the first is unpacked: bound by the latency of three loads in a row where a thread has
// one token, so long calls take four (24463 tokens and 8305 of padding 26 us, 4.9 TB/s; by one 46 us).
template <int N>
__global__ void __launch_bounds__(256) k_kv4_read(int T, const int32_t* __restrict__ seqs, const int32_t* __restrict__ positions,
                                                  Cache c, bf16* __restrict__ k_out, bf16* __restrict__ v_out) {
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    const int t0 = blockIdx.x * N, unit = threadIdx.x >> 4, w = threadIdx.x & 15;  // unit: which * 8 + head
    int pos[N], phys[N];
    uint32_t word[N], par[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        phys[i] = -1;
        if (t0 + i < T) {
            const int seq = seqs[t0 + i];
            pos[i] = positions[t0 + i];
            if (seq >= 0) phys[i] = find_block(c, seq, pos[i], threadIdx.x == 0);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (phys[i] < 0) continue;
        const uint8_t* tile = c.pool + (size_t)phys[i] * BLOCK + (size_t)unit * TILE;
        const int tok = pos[i] % KVB;
        word[i] = *reinterpret_cast<const uint32_t*>(tile + tok * (HD / 2) + w * 4);
        par[i] = *reinterpret_cast<const uint32_t*>(tile + PAR + tok * 8 + (w & 1) * 4);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (phys[i] < 0) continue;
        // pairs of dims (d, d + 4): 128 + code, the offset added (exact), times the scale (rounded once); then side by side
        const uint32_t s = __byte_perm(par[i], 0u, 0x1010), off = __byte_perm(par[i], 0u, 0x3232);
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul_bf16x2(add_bf16x2((word[i] >> (4 * e) & 0x000F000Fu) | 0x43004300u, off), s);
        const uint32_t o[4] = {__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                               __byte_perm(v[2], v[3], 0x7632)};
        bf16* out = (unit < NKV ? k_out : v_out) + ((size_t)(t0 + i) * NKV + (unit & 7)) * HD + 64 * (w & 1) + 8 * (w >> 1);
        *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------- attention
// A row is a query token, or two tokens of a sequence that follow one another (the last of an odd number alone).
struct AttnArgs {
    const int32_t* seqs;
    const int32_t* kv_lens;
    int S, max_len;
    int each, per_seq, rows;  // query tokens of a row, rows of a sequence, rows in all
    int n_splits;
    float* part;  // pieces: 128 output sums, reference, sum of weights
    __device__ __forceinline__ int token(int r) const { return r / per_seq * S + r % per_seq * each; }     // its first
    __device__ __forceinline__ bool two(int r) const { return each == 2 && 2 * (r % per_seq) + 1 < S; }
};

// Row r: the cache row it reads and the keys its last token sees; false where the row is left as it was.
__device__ __forceinline__ bool attn_row(const Cache& c, const AttnArgs& a, int r, bool report, int& seq, int& seen) {
    const int b = r / a.per_seq, s = min((r - b * a.per_seq + 1) * a.each, a.S) - 1;
    seq = a.seqs ? a.seqs[b] : b;
    if (seq < 0) return false;
    int len = a.kv_lens[b];
    if (seq >= c.n_seqs || len < 0 || len > a.max_len) {
        if (report) set_err(c.err, TTS_BB_KV4_ERR_RANGE);
        return false;
    }
    seen = max(0, len - (a.S - 1 - s));
    return true;
}

// Tensor-core attention of one (row, KV head, split). 4 warps; a warp takes 32 keys at a time (warps 0, 1 the halves of the
// split's even cache blocks, 2, 3 of the odd ones), copied by cp.async through a ring of its own: no barrier between
// warps until the end. What bounds it beside memory are the integer instructions that take nibbles apart (two a cycle
// and SM), so both products take the codes with as few of them as they can:
//
// Scores, S[key][column] = K Q^T, by m16n8k16 on fp16: the half word 000c is the fp16 number c 2^-24 and 00c0 16 c 2^-24
// (subnormals and the first binade are evenly spaced), so a word of 8 codes is two steps' operands after one shift and
// four masks. Lane (r = lane / 4, c = lane % 4) reads 16 bytes of the code rows of keys r and r + 8: 16 dims of each group, in
// pairs (d, d + 4), which only permutes the contraction; Q of the dims that come as 16 c is divided by 16. Products are exact
// and sums fp32. The zero point joins by the queries' sum: s (sum q code + zero sum q). Q is scaled by a power of two to a
// largest magnitude in [2^14, 2^15). bf16 queries are then exact in fp16 (down to 2^-25 of the head's largest); column n
// holds head n & 1, so every lane has both heads' scores of its keys. fp32 queries enter as two fp16 parts, to within one fp32
// step together, part (n >> 1) & 1 of head n & 1 in column n; and their codes become (code + zero) 2^-9 first, by one exact
// multiply-add each: the subnormal numbers as operands lose up to 5 bits of a product's sum. bf16 results do not show that: with
// those multiply-adds as many of them round to another number than the exact ones do, and 8 x 65537 keys take 117 us, not 111.
// Each lane then keeps one score of 16 keys: key r + 8 (c & 1), head c >> 1. (By m16n8k32 on e4m3, where a byte of two masks
// is 4 operands, the same took longer: that form is carried out by fp16 products after conversions.)
//
// Output, O^T[dim][column] += V^T P, by m16n8k16 on bf16, V's codes as A: rows are dims, and a register holds one dim of
// two keys: one byte of both keys' words side by side, then one mask for the byte's even dim and one for its odd dim:
// 000c is the bf16 number c 2^-133 and 00c0 16 c 2^-133 (subnormals again). A multiply-add makes them (code + zero) 2^-7,
// exact in 8 bits: whole numbers around zero, not 0..15 with a middle added later, because where a softmax is flat the
// sums cancel and a common offset would cost their digits. P times V's scale of the key and group is B, as bf16 parts in
// columns of their own: for fp32 three by truncation, all 24 bits; for bf16 two, both rounded: within 2^-18 of the weight, on
// either side. Two of 1000 bf16 outputs then round to another number than the exact ones do; of the plain form in 32 bits one of
// 3000 does. (Two parts by truncation, no faster, are low by 2^-17 on average: 6 of 1000. Three, as for fp32, cost about a tenth of the time.)
//
// Two query tokens that follow one another (N = 2): the columns that one token only repeats are the second one's, query
// c & 1 in a lane, which then has both of 16 keys' scores r and r + 8 of its head; fp32's third parts of the weights take
// products of their own (and registers: three blocks an SM). Codes are taken apart once for both: 8 sequences of 8 tokens and
// 200..2000 keys 28 -> 19 us (fp32 33 -> 28). The first token does not see the second's key: its weight is 0 there.
//
// Softmax: a running reference m for each head, moved only when a score exceeds it by 8 (log2): then sums and O are
// rescaled. It starts at about the lowest number, not -inf, so that no difference of infinities arises, and no finite score
// has a weight of 0 beside nothing larger.
constexpr int WARPS = 4, STAGES = 2, UNIT = 32, UNIT_BYTES = 4608;  // K and V codes 2048 each, parameters 256 each
constexpr int V_AT = 2048, KP_AT = 4096, VP_AT = 4352, RING_BYTES = WARPS * STAGES * UNIT_BYTES;
constexpr float M_START = -3.4e38f, M_SLACK = 8.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ float as_f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t as_u(float x) { return __float_as_uint(x); }
__device__ __forceinline__ float scale_of(uint32_t par) { return as_f(par << 16); }
__device__ __forceinline__ float zero_of(uint32_t par) { return as_f(par & 0xFFFF0000u) + 128.f; }
// bf16 part (0, 1, 2) of x: 8 significant bits each, by truncation; m1, m2 cover the upper half where part >= 1, 2
__device__ __forceinline__ uint32_t part_of(float x, uint32_t m1, uint32_t m2) {
    x -= as_f(as_u(x) & m1);
    return as_u(x - as_f(as_u(x) & m2));
}
// x as two bf16 parts, the first in the high half, the second (of the rest) in the low one
__device__ __forceinline__ uint32_t two_parts(float x) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x), "f"(0.f));
    const float first = as_f(d);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(first), "f"(x - first));
    return d;
}
// One warp's share of the queries: a head's 128 values (lane l: dims 4l .. 4l + 3) as fp16 parts in `to` ([part][2 heads] rows of
// 128, to: this head's; 8 dims stand as 0 4 1 5 2 6 3 7; with one part (bf16 queries) the odd ones divided by 16) and in
// `about` its group sums, in the units of the products' sums, and the factor that turns those into scores times log2(e) (NaN
// where a query is not finite).
template <int PARTS, int N>
__device__ __forceinline__ void stage_q(const float4 v, int lane, __half* to, float* about) {
    const float a = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
    // fmaxf drops a NaN
    const bool fine = __all_sync(0xffffffffu, a < INFINITY && v.x == v.x && v.y == v.y && v.z == v.z && v.w == v.w);
    // 2^(14 - exponent of the largest), the largest taken as at least 2^-103
    const float up = __uint_as_float((268u - max(__float_as_uint(fine ? warp_max(a) : 1.f) >> 23, 24u)) << 23);
    float s = (v.x + v.y) + (v.z + v.w);
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((lane & 15) == 0) about[lane >> 4] = s * up * 0x1p-24f;
    if (lane == 0) about[2] = fine ? rsqrtf((float)HD) * LOG2E * (PARTS == 1 ? 0x1p24f : 0x1p9f) / up : __int_as_float(0x7FC00000);
    float x[4] = {v.x * up, v.y * up, v.z * up, v.w * up};
    to += (lane >> 1) * 8 + (lane & 1);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half h = __float2half_rn(x[e]);
            x[e] -= __half2float(h);
            to[p * 2 * N * HD + e * 2] = PARTS == 1 && (e & 1) ? __hmul(h, __float2half_rn(0.0625f)) : h;
        }
}

__device__ __forceinline__ float peer(const float* p, int rank) {  // *p in the shared memory of a block of the cluster
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int N> constexpr int AN_SM = sizeof(T) * N == 8 ? 3 : 4;  // blocks an SM
// What a block has in common for its pieces
struct Shared {
    __half q[4][2][HD];  // [2 part + query, or part][head]
    float about[4][4];   // of head h of query j at 2 j + h, here and below
    float m[WARPS][4], l[WARPS][4];
};

// One piece: the cache blocks [b0, b1) of KV head g of a row that reads cache row seq and whose last token sees `seen` keys;
// q: its two heads; gap: 1 where there is a second token, whose heads are NQ rows further and which sees one key more.
template <typename T> struct Piece {
    const T* q;
    int seq, seen, gap, g, b0, b1;
    // units of a warp: unit i is keys 32 (warp & 1) .. + 31 of block b0 + (warp >> 1) + 2 i
    __device__ __forceinline__ int units(int warp) const { return max(0, (b1 - b0 - (warp >> 1) + 1) >> 1); }
    __device__ __forceinline__ const int32_t* pages(const Cache& c, int warp) const {
        return c.table + (size_t)seq * c.bps + b0 + (warp >> 1);
    }
};
// What is on its way for a piece before its turn: the first unit (STAGES - 1 of them) and the queries
struct Ahead {
    float4 q;
    int page;          // of the first unit not fetched yet
    uint32_t missing;  // bit s: the block in stage s has no page
};
// A unit's codes and parameters into stage s of the warp's ring; the group is committed by the caller
__device__ __forceinline__ void fetch_unit(const Cache& cache, int g, uint8_t* ring, int s, int page, uint32_t& missing) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool ok = page >= 0 && page < cache.n_blocks;
    missing = missing & ~(1u << s) | (ok ? 0u : 1u << s);
    if (ok) {
        const uint8_t* const b = cache.pool + (size_t)page * BLOCK + (size_t)g * TILE + (warp & 1) * 2048 + lane * 16;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(ring) + (warp * STAGES + s) * UNIT_BYTES;
        // 16-byte pieces of V rows are swapped between the row's halves for rows 2, 3 of every 4, so that the 8-byte reads
        // of 4 rows meet all 32 banks
        const uint32_t vd = d + V_AT + (lane * 16 ^ (lane >> 3 & 1) * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cp16(d + lane * 16 + 512 * i, b + 512 * i);
            cp16(vd + 512 * i, b + NKV * TILE + 512 * i);
        }
        cp16(d + KP_AT + lane * 16, b + (lane & 16 ? NKV * TILE : 0) + PAR + (warp & 1) * (256 - 2048) + ((lane & 15) - lane) * 16);
    } else if (lane == 0) {
        set_err(cache.err, TTS_BB_KV4_ERR_PAGE);
    }
}
template <typename T>
__device__ __forceinline__ void start_piece(const Piece<T>& p, const Cache& cache, uint8_t* ring, int page0, Ahead& a) {
    static_assert(STAGES == 2, "one unit ahead");
    const int warp = threadIdx.x >> 5, n = p.units(warp);
    a.missing = 0u;
    if (n > 0) fetch_unit(cache, p.g, ring, 0, page0, a.missing);
    asm volatile("cp.async.commit_group;" ::: "memory");
    a.page = n > 1 ? p.pages(cache, warp)[2] : 0;
}
template <int N, typename T>
__device__ __forceinline__ void load_queries(const Piece<T>& p, Ahead& a) {
    // a head a warp; the second token's by warps 2, 3 (where there is none, the first's again, and nobody reads the results)
    if (threadIdx.x < 64 * N) a.q = load4(p.q + (threadIdx.x >> 6) * p.gap * (NQ * HD) + (threadIdx.x & 63) * 4);
}

// A piece that is started already; the next one (where more) is started before the warps' results are merged, so that its
// keys come meanwhile. Thread d ends with the piece's reference M, sum of weights L and output sums O of dim d of both
// heads of each of the N query tokens. All threads of the block call it, with the same arguments; `so` is free again when the next call has merged.
template <typename T, int N>
__device__ __forceinline__ void attend_piece(const Piece<T>& p, bool more, const Piece<T>& next, const Cache& cache, uint8_t* ring, float* so,
                                             Shared& sh, Ahead& ahead, float (&M)[2 * N], float (&L)[2 * N], float (&O)[2 * N]) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int P = F32 ? 3 : 2;  // bf16 parts of a weight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int seen = p.seen, j0 = p.b0 + (warp >> 1), n = p.units(warp);
    uint8_t* const mine = ring + warp * STAGES * UNIT_BYTES;
    const int32_t* const pages = p.pages(cache, warp);

    if (warp < 2 * N) stage_q<F32 ? 2 : 1, N>(ahead.q, lane, sh.q[warp >> 1][warp & 1], sh.about[warp]);
    __syncthreads();
    int next_page = 0;
    if (more) {
        if (next.units(warp) > 0) next_page = next.pages(cache, warp)[0];
        load_queries<N>(next, ahead);
    }
    uint4 qb[4];       // of word w: the B registers of its two steps
    const int hq = N == 1 ? c >> 1 : (c >> 1) + 2 * (c & 1);  // this lane's head (and query)
    const float qsum[2] = {sh.about[hq][0], sh.about[hq][1]};
    const float factor = sh.about[hq][2];
#pragma unroll
    for (int w = 0; w < 4; ++w)
        qb[w] = *reinterpret_cast<const uint4*>(&sh.q[F32 && N == 2 ? r >> 1 : F32 || N == 2 ? r >> 1 & 1 : 0][r & 1][64 * (w & 1) + 16 * c + 8 * (w >> 1)]);
    const uint32_t m1 = r >= 2 * N ? 0xFFFF0000u : 0u, m2 = N == 1 && r >= 4 ? 0xFFFF0000u : 0u;
    const uint32_t half_sel = r & (N == 1 ? 2 : 4) ? 0x5410u : 0x7632u;  // bf16: part 0 in the high halves, part 1 in the low ones
    const int from = 4 * c + 2 * (r & 1) + (N == 1 ? 0 : r >> 1 & 1);    // the lane that has the weight of key c of this column
    const int my = N == 1 ? r + 8 * (c & 1) : r;                         // this lane's key of 16 (the first; the second 8 behind)
    const int sees = seen - (N == 2 && !(c & 1) ? p.gap : 0);
    const uint8_t* const kat = mine + r * 64 + c * 16;
    const uint8_t* const vat = mine + V_AT + c * 64 + (r * 8 ^ (c >> 1) * 32);
    float o[8][4] = {}, m = M_START, l = 0.f;
    [[maybe_unused]] float o3[F32 && N == 2 ? 8 : 1][4] = {};  // the third parts' sums, by columns 0 to 3 of products of their own

    // 16 keys: codes at byte `at` of the ring, parameters at `par`
    auto step = [&](auto tail, const int at, const int par, const int key0) {
        constexpr bool TAIL = decltype(tail)::value;

        float z[N];
        {
            const uint4 k0 = *reinterpret_cast<const uint4*>(kat + at);
            const uint4 k1 = *reinterpret_cast<const uint4*>(kat + at + 512);
            uint2 kp[N];
#pragma unroll
            for (int j = 0; j < N; ++j) kp[j] = *reinterpret_cast<const uint2*>(mine + par + KP_AT + my * 8 + j * 64);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
            [[maybe_unused]] uint32_t kz[2][2] = {};  // fp32: zero 2^-9 of keys r, r + 8 and each group, twice
            if constexpr (F32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint2 rp = *reinterpret_cast<const uint2*>(mine + par + KP_AT + r * 8 + h * 64);
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        const __half2 v = __float2half2_rn(zero_of(gr ? rp.y : rp.x) * 0x1p-9f);
                        kz[h][gr] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
            }
            float s[2][4] = {};  // of each group
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t u0 = w0[w] >> 8, u1 = w1[w] >> 8;
                uint32_t x[4] = {w0[w] & 0x000F000Fu, w1[w] & 0x000F000Fu, w0[w] & 0x00F000F0u, w1[w] & 0x00F000F0u};
                uint32_t y[4] = {u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x00F000F0u};
                if constexpr (F32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // times 2^15 and 2^11
                        x[e] = fma_f16x2(x[e], e < 2 ? 0x78007800u : 0x68006800u, kz[e & 1][w & 1]);
                        y[e] = fma_f16x2(y[e], e < 2 ? 0x78007800u : 0x68006800u, kz[e & 1][w & 1]);
                    }
                }
                mma_f16(s[w & 1], x, qb[w].x, qb[w].y);
                mma_f16(s[w & 1], y, qb[w].z, qb[w].w);
            }
            // this lane's keys and head: sums e = 2 (key r + 8) + head
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float y[2];
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    const float a0 = c & 2 ? s[gr][1] : s[gr][0], a1 = c & 2 ? s[gr][3] : s[gr][2];
                    y[gr] = N == 2 ? (j ? a1 : a0) : c & 1 ? a1 : a0;
                    // the other part's sum
                    if (F32 && N == 1) y[gr] += __shfl_xor_sync(0xffffffffu, c & 1 ? a0 : a1, 1);
                    if (F32 && N == 2) y[gr] += __shfl_xor_sync(0xffffffffu, c & 2 ? s[gr][2 * j] : s[gr][2 * j + 1], 2);
                }
                if (!F32) {
                    y[0] += zero_of(kp[j].x) * qsum[0];
                    y[1] += zero_of(kp[j].y) * qsum[1];
                }
                z[j] = scale_of(kp[j].x) * y[0] + scale_of(kp[j].y) * y[1];
                z[j] *= factor;
            }
        }
        bool on[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            on[j] = !TAIL || key0 + my + 8 * j < sees;
            if (!on[j]) z[j] = -INFINITY;
        }
        if (__any_sync(0xffffffffu, z[0] > m + M_SLACK || z[N - 1] > m + M_SLACK)) {
            float mx = fmaxf(z[0], z[N - 1]);
            if (N == 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float nm = fmaxf(m, mx), f = ex2(m - nm), other = __shfl_xor_sync(0xffffffffu, f, 2);
            const float f0 = c & 2 ? other : f, f1 = c & 2 ? f : other;
            m = nm;
            l *= f;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                o[t][0] *= f0; o[t][1] *= f1;
                o[t][2] *= f0; o[t][3] *= f1;
                if constexpr (F32 && N == 2) {
                    o3[t][0] *= f0; o3[t][1] *= f1;
                    o3[t][2] *= f0; o3[t][3] *= f1;
                }
            }
        }
        {
            float ps[N][2];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float p = ex2(z[j] - m);
                l += p;
                const uint2 vp = *reinterpret_cast<const uint2*>(mine + par + VP_AT + my * 8 + j * 64);
                ps[j][0] = p * scale_of(vp.x);
                ps[j][1] = p * scale_of(vp.y);
                if (TAIL && !on[j]) ps[j][0] = ps[j][1] = 0.f;  // parameters behind the keys may be anything
            }
            uint2 w[4], pp[4];  // codes and parameters of keys c, c + 4, c + 8, c + 12
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = *reinterpret_cast<const uint2*>(vat + at + k * 256);
                pp[k] = *reinterpret_cast<const uint2*>(mine + par + VP_AT + c * 8 + k * 32);
            }
            if constexpr (TAIL) {  // nor an offset that is not finite times a zero
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (key0 + c + 4 * k >= seen) pp[k] = make_uint2(0u, 0u);
            }
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                uint32_t y[4], b0, b1;
                [[maybe_unused]] uint32_t b2 = 0u, b3 = 0u;
                if constexpr (F32 && N == 2) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x = __shfl_sync(0xffffffffu, ps[k >> 1][gr], from + (k & 1) * 16);
                        const float rest = x - as_f(as_u(x) & 0xFFFF0000u);
                        y[k] = r >= 4 ? as_u(rest) : as_u(x);
                        const uint32_t third = r >= 4 ? 0u : as_u(rest - as_f(as_u(rest) & 0xFFFF0000u));
                        if (k < 2) b2 |= third >> 16 << (16 * (k & 1));
                        else b3 |= third >> 16 << (16 * (k & 1));
                    }
                    b0 = highs(y[0], y[1]);
                    b1 = highs(y[2], y[3]);
                } else if constexpr (F32) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = part_of(__shfl_sync(0xffffffffu, ps[0][gr], from + (k & 1) * 16 + (k >> 1)), m1, m2);
                    b0 = highs(y[0], y[1]);
                    b1 = highs(y[2], y[3]);
                } else {
                    uint32_t both[N];  // part 1 below part 0
#pragma unroll
                    for (int j = 0; j < N; ++j) both[j] = two_parts(ps[j][gr]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = __shfl_sync(0xffffffffu, both[N == 2 ? k >> 1 : 0], from + (k & 1) * 16 + (N == 1 ? k >> 1 : 0));
                    b0 = __byte_perm(y[0], y[1], half_sel);
                    b1 = __byte_perm(y[2], y[3], half_sel);
                }
                uint32_t zero[2];  // keys 0 1, keys 2 3: zero 2^-7
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t off = highs(gr ? pp[2 * h].y : pp[2 * h].x, gr ? pp[2 * h + 1].y : pp[2 * h + 1].x);
                    zero[h] = fma_bf16x2(off, 0x3C003C00u, 0x3F803F80u);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {  // byte t of the words: dims 2 t, 2 t + 1 of lane r's 8
                    const uint32_t sel = 0x0400u + 0x1111u * t;
                    const uint32_t u01 = __byte_perm(gr ? w[0].y : w[0].x, gr ? w[1].y : w[1].x, sel);
                    const uint32_t u23 = __byte_perm(gr ? w[2].y : w[2].x, gr ? w[3].y : w[3].x, sel);
                    // times 2^126 and 2^122
                    const uint32_t x4[4] = {fma_bf16x2(u01 & 0x000F000Fu, 0x7E807E80u, zero[0]), fma_bf16x2(u01 & 0x00F000F0u, 0x7C807C80u, zero[0]),
                                            fma_bf16x2(u23 & 0x000F000Fu, 0x7E807E80u, zero[1]), fma_bf16x2(u23 & 0x00F000F0u, 0x7C807C80u, zero[1])};
                    mma_bf16(o[4 * gr + t], x4, b0, b1);
                    if constexpr (F32 && N == 2) mma_bf16(o3[4 * gr + t], x4, b2, b3);
                }
            }
        }
    };
    for (int i = 0; i < n; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncwarp();
        if (i + STAGES - 1 < n) fetch_unit(cache, p.g, ring, (i + STAGES - 1) % STAGES, ahead.page, ahead.missing);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (i + STAGES < n) ahead.page = pages[2 * (i + STAGES)];
        const int key0 = (j0 + 2 * i) * KVB + (warp & 1) * UNIT;
        if (key0 >= seen || (ahead.missing >> (i % STAGES) & 1)) continue;
        const int at = (i % STAGES) * UNIT_BYTES;
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
            const int k = key0 + 16 * u;
            if (k + 16 <= seen - (N == 2 ? p.gap : 0)) step(std::false_type{}, at + 1024 * u, at + 128 * u, k);
            else if (k < seen) step(std::true_type{}, at + 1024 * u, at + 128 * u, k);
        }
    }
    // merge the warps: every part of O to shared memory (so: [warp][part][query][head][128]), then one thread for each dim
    if (N == 1) l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (more) {
        __syncwarp();  // the warp's ring is free
        start_piece(next, cache, ring, next_page, ahead);
    }
    if (N == 2 || c < P) {
        const int at = N == 1 ? warp * P + c : (warp * P + (c >> 1)) * 2 + (c & 1);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int d = 64 * (t >> 2) + 8 * r + 2 * (t & 3);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(so + (at * 2 + h) * HD + d) =
                    make_float2(o[t][h] * 128.f, o[t][2 + h] * 128.f);
            if constexpr (F32 && N == 2) {
                if (c < 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2*>(so + (((warp * P + 2) * 2 + c) * 2 + h) * HD + d) =
                            make_float2(o3[t][h] * 128.f, o3[t][2 + h] * 128.f);
                }
            }
        }
    }
    if (lane < 4 && (N == 2 || !(lane & 1))) { sh.m[warp][hq] = m; sh.l[warp][hq] = l; }
    __syncthreads();
    const int d = threadIdx.x;
#pragma unroll
    for (int h = 0; h < 2 * N; ++h) {
        M[h] = M_START;
        L[h] = O[h] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M[h] = fmaxf(M[h], sh.m[w][h]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = ex2(sh.m[w][h] - M[h]);
            float x = 0.f;
#pragma unroll
            for (int part = P - 1; part >= 0; --part) x += so[((w * P + part) * 2 * N + h) * HD + d];
            L[h] += f * sh.l[w][h];
            O[h] += f * x;
        }
    }
}

// grid (splits, 8, rows), 128 threads: 64 rows of 200..2000 keys, fp32, 32 us; 1 of 8000, bf16, 7.9. One piece a block, the blocks of a row's keys dealt evenly to its splits. The splits of a (row,
// head) are one cluster (at most 16), which merges them through its shared memory.
template <typename T, int N>
__global__ void __launch_bounds__(WARPS * 32, AN_SM<T, N>) k_kv4_attn(const T* __restrict__ q, Cache cache, AttnArgs a, T* __restrict__ out) {
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) Shared sh;
    const int split = blockIdx.x, g = blockIdx.y, row = blockIdx.z, d = threadIdx.x;
    int seq, seen;
    if (!attn_row(cache, a, row, d == 0 && split == 0 && g == 0, seq, seen)) return;
    const int nblk = (seen + KVB - 1) / KVB, bps = (nblk + a.n_splits - 1) / a.n_splits;
    float M[2 * N], L[2 * N], O[2 * N];
    const int gap = N == 2 && a.two(row);
    const size_t token = N == 1 ? row : a.token(row);
    const Piece<T> p = {q + (token * NQ + 2 * g) * HD, seq, seen, gap, g, split * bps, min(nblk, (split + 1) * bps)};
    Ahead ahead;
    load_queries<N>(p, ahead);
    start_piece(p, cache, ring, p.units(d >> 5) > 0 ? p.pages(cache, d >> 5)[0] : 0, ahead);
    attend_piece<T, N>(p, false, p, cache, ring, reinterpret_cast<float*>(ring + RING_BYTES), sh, ahead, M, L, O);
    T* const to = out + (token * NQ + 2 * g) * HD;
    const int heads = N == 1 ? 2 : 2 + 2 * gap;
    if (a.n_splits == 1) {
#pragma unroll
        for (int h = 0; h < 2 * N; ++h)
            if (h < heads) to[((h >> 1) * NQ + (h & 1)) * HD + d] = (T)(L[h] == 0.f ? 0.f : O[h] / L[h]);
        return;
    }
    float(*const all)[HD] = reinterpret_cast<float(*)[HD]>(ring);  // which is free: every copy was waited for
    __shared__ float ml[2 * N][2];
#pragma unroll
    for (int h = 0; h < 2 * N; ++h) {
        all[h][d] = O[h];
        if (d == 0) { ml[h][0] = M[h]; ml[h][1] = L[h]; }
    }
    cluster_sync();
    for (int i = split * WARPS * 32 + d; i < heads * HD; i += a.n_splits * WARPS * 32) {
        const int h = i / HD;
        float m1 = M_START, l1 = 0.f, o1 = 0.f;
#pragma unroll 8
        for (int s = 0; s < a.n_splits; ++s) m1 = fmaxf(m1, peer(&ml[h][0], s));
#pragma unroll 8
        for (int s = 0; s < a.n_splits; ++s) {
            const float f = ex2(peer(&ml[h][0], s) - m1);
            l1 += f * peer(&ml[h][1], s);
            o1 += f * peer(&all[h][i % HD], s);
        }
        to[((h >> 1) * NQ + (h & 1)) * HD + i % HD] = (T)(l1 == 0.f ? 0.f : o1 / l1);
    }
    cluster_sync();  // no block leaves while another reads its sums
}

// All cache blocks of all rows and heads as one line, (row, head, block) in that order, cut into equal shares: ragged rows
// then cost what their keys cost, and no wave of blocks waits for the longest. Share i is blocks [i Q, (i + 1) Q) of the
// line. A (row, head) that lies in one share is written at once, the others' pieces go to the workspace, two places a share:
// the piece that starts the share, and the one that ends it.
struct Line {
    long long units;  // blocks in all
    int share;        // blocks of one share
};
__device__ __forceinline__ int row_blocks(const Cache& c, const AttnArgs& a, int row, bool report) {
    int seq, seen;
    return row < a.rows && attn_row(c, a, row, report, seq, seen) ? (seen + KVB - 1) / KVB : 0;
}
__device__ __forceinline__ Line line_of(long long blocks, int shares) {
    const long long u = blocks * NKV;
    return {u, max(2, (int)((u + shares - 1) / shares))};
}
// the place of a piece: [share][first, last][N queries][2 heads][128 sums, reference, weight]
constexpr int PIECE = HD + 4;  // 16-byte rows
template <int N>
__device__ __forceinline__ float* place(float* part, int share, int which) { return part + ((size_t)share * 2 + which) * 2 * N * PIECE; }

// grid: the shares; rows <= LINE_ROWS. 8 rows of 65537 keys, bf16: 110 us with the launch that merges, 5.4 TB/s.
constexpr int LINE_ROWS = 1024;
template <typename T, int N>
__global__ void __launch_bounds__(WARPS * 32, AN_SM<T, N>) k_kv4_attn_line(const T* __restrict__ q, Cache cache, AttnArgs a, T* __restrict__ out) {
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) Shared sh;
    __shared__ int start[4];  // the share's first row, the blocks of it before the share, its cache row and its keys
    __shared__ long long sums[WARPS];
    const int me = blockIdx.x, d = threadIdx.x, warp = d >> 5, lane = d & 31;
    // where the share begins: the rows' blocks, a row a thread at a time; the sums of all rows first, where one turn is not enough
    long long total = 0, before = 0, first = 0;
    Line line = {0, 0};
    const bool one_turn = a.rows <= WARPS * 32;
    if (!one_turn) {
        for (int i = d; i < a.rows; i += WARPS * 32) total += row_blocks(cache, a, i, me == 0);
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) sums[warp] = total;
        __syncthreads();
        total = sums[0] + sums[1] + sums[2] + sums[3];
        line = line_of(total, gridDim.x);
        first = (long long)me * line.share;
    }
    for (int i = d; i - d < a.rows && before * NKV <= first; i += WARPS * 32) {
        int row_seq = 0, row_seen = 0;
        const int n = i < a.rows && attn_row(cache, a, i, one_turn && me == 0, row_seq, row_seen) ? (row_seen + KVB - 1) / KVB : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += w;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long mine = before + incl - n;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) mine += sums[w];
            before += sums[w];
        }
        if (one_turn) {
            line = line_of(before, gridDim.x);
            first = (long long)me * line.share;
        }
        if (first >= mine * NKV && first < (mine + n) * NKV) {
            start[0] = i;
            start[1] = (int)(first - mine * NKV);
            start[2] = row_seq;
            start[3] = row_seen;
        }
    }
    __syncthreads();
    if (first < line.units) {
        int row = start[0], at = start[1], seq = start[2], seen = start[3], left = (int)min((long long)line.share, line.units - first);
        // the piece from `at` of the row on; then the place behind it
        const auto take = [&](Piece<T>& p, int& piece_row, bool& whole) {
            const int nblk = (seen + KVB - 1) / KVB, g = at / nblk, b0 = at - g * nblk, b1 = min(nblk, b0 + left);
            p = {q + ((size_t)(N == 1 ? row : a.token(row)) * NQ + 2 * g) * HD, seq, seen, N == 2 && a.two(row), g, b0, b1};
            piece_row = row;
            whole = b0 == 0 && b1 == nblk;
            left -= b1 - b0;
            at += b1 - b0;
            if (at == nblk * NKV) {
                at = 0;
                if (left > 0)
                    do ++row; while (row < a.rows && (!attn_row(cache, a, row, false, seq, seen) || seen == 0));
                if (row >= a.rows) left = 0;
            }
        };
        Piece<T> p, next;
        int piece_row, next_row = 0;
        bool whole, next_whole = false, begins = true;  // the share's first piece
        take(p, piece_row, whole);
        Ahead ahead;
        load_queries<N>(p, ahead);
        start_piece(p, cache, ring, p.units(warp) > 0 ? p.pages(cache, warp)[0] : 0, ahead);
        for (bool more = true; more;) {
            more = left > 0;
            if (more) take(next, next_row, next_whole);
            float M[2 * N], L[2 * N], O[2 * N];
            attend_piece<T, N>(p, more, next, cache, ring, reinterpret_cast<float*>(ring + RING_BYTES), sh, ahead, M, L, O);
            if (whole) {
#pragma unroll
                for (int h = 0; h < 2 * N; ++h)
                    if (h < 2 || p.gap)
                        out[((size_t)((N == 1 ? piece_row : a.token(piece_row)) + (h >> 1)) * NQ + 2 * p.g + (h & 1)) * HD + d] =
                            (T)(L[h] == 0.f ? 0.f : O[h] / L[h]);
            } else {
                float* const to = place<N>(a.part, me, begins ? 0 : 1);
#pragma unroll
                for (int h = 0; h < 2 * N; ++h) {
                    to[h * PIECE + d] = O[h];
                    if (d == 0) { to[h * PIECE + HD] = M[h]; to[h * PIECE + HD + 1] = L[h]; }
                }
            }
            begins = false;
            p = next;
            piece_row = next_row;
            whole = next_whole;
        }
    }
    // rows that see nothing: zeros, by the blocks in turn
    for (int i = me; i < a.rows; i += gridDim.x) {
        int seq, seen;
        if (attn_row(cache, a, i, false, seq, seen) && seen == 0)
            for (int e = d; e < (N == 2 && a.two(i) ? 2 : 1) * NQ * HD; e += WARPS * 32)
                out[(size_t)(N == 1 ? i : a.token(i)) * NQ * HD + e] = (T)0.f;
    }
}

// grid (16 N, rows), 128 threads: the pieces of a (row, query, head) that lies in several shares. Warp w sums pieces w, w + 4, ..., lane l
// dims 4l .. 4l + 3, all weighted to the largest reference; then the warps' sums are added in their order.
template <typename T, int N>
__global__ void __launch_bounds__(128) k_kv4_combine(Cache c, AttnArgs a, int shares, T* __restrict__ out) {
    pdl_wait();  // upstream results are read below
    pdl_trigger();
    __shared__ long long sums[2][4];
    __shared__ float4 part[4][32];
    __shared__ float weight[4];
    const int g = blockIdx.x / (2 * N), h = blockIdx.x % (2 * N), row = blockIdx.y, d = threadIdx.x, warp = d >> 5, lane = d & 31;
    long long before = 0, total = 0;
    for (int i = d; i < a.rows; i += 128) {
        const int n = row_blocks(c, a, i, false);
        total += n;
        if (i < row) before += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) { sums[0][warp] = before; sums[1][warp] = total; }
    __syncthreads();
    before = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    total = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
    const Line line = line_of(total, shares);
    const int nblk = row_blocks(c, a, row, false);
    if (nblk == 0 || (h >= 2 && !a.two(row))) return;
    const long long from = before * NKV + (long long)g * nblk;
    const int s0 = (int)(from / line.share), n = (int)((from + nblk - 1) / line.share) - s0 + 1;
    if (n == 1) return;  // written by its share
    const bool inside = from != (long long)s0 * line.share;  // the first piece ends its share
    auto at = [&](int i) { return place<N>(a.part, s0 + i, i == 0 && inside) + h * PIECE; };
    float M = M_START;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, at(i)[HD]);
    M = warp_max(M);
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = warp; i < n; i += 4) {
        const float* p = at(i);
        const float f = ex2(p[HD] - M);
        const float4 x = *reinterpret_cast<const float4*>(p + lane * 4);
        L += f * p[HD + 1];
        o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
    }
    part[warp][lane] = o;
    if (lane == 0) weight[warp] = L;
    __syncthreads();
    const float* const s = reinterpret_cast<const float*>(part);
    L = weight[0] + weight[1] + weight[2] + weight[3];
    const float O = s[d] + s[HD + d] + s[2 * HD + d] + s[3 * HD + d];
    out[((size_t)((N == 1 ? row : a.token(row)) + (h >> 1)) * NQ + 2 * g + (h & 1)) * HD + d] = (T)(L == 0.f ? 0.f : O / L);
}

struct Plan {
    int splits;  // a cluster's blocks; 0: a line
    int shares;
};
// Caches of up to 16 blocks of keys a block of the launch (32 where the pairs fill half the SMs' slots by themselves): one
// block, or one cluster of up to 8 as the slots allow, for each (row, KV head), in one launch; clusters of 16 for few rows, up
// to 24 blocks of keys each. Longer ones: a line in `slots`
// shares (as many blocks as are resident: one wave) and the launch that merges it. Measured, us: 1 x 8000 keys 7.9 by a
// cluster of 16, 9.9 of 8, 14.1 by a line; 1 x 20000 14.2 and 16.4 by a line; 4 x 4000 fp32 8.5 by clusters of 8, 10.6 of 16,
// 4 x 16000 20.2 of 16 and 24.1 by a line; 64 x 20..200 keys 6.0 by a block each, 14.3 by a line; 64 x 100..1000 fp32 17.7
// and 22.9, 64 x 200..2000 31.7 and 31.0 (even rows of 2000 37.1 and 42.7), 64 x 400..4000 56 and 46 (even 69 and 73), 64 x 800..8000
// 78 and 69. A twentieth of the slots stays free, since clusters do not fill every SM: 19 x 1000 keys in
// clusters of 3 of 4 blocks an SM 11.1, of 4 (all slots, two waves) 12.6.
Plan attn_plan(long long rows, int max_len, int slots) {
    const long long pairs = rows * NKV, nblk = (max_len + KVB - 1) / KVB, most = (nblk + 1) / 2, room = slots * 19 / 20;
    long long n = std::min({8ll, room / pairs, most});
    if (16 * pairs <= room && nblk > (32 * pairs <= slots ? 32 : 128)) n = 16;
    if (rows > LINE_ROWS || nblk <= (n == 16 ? 24 * n : n >= 2 ? 16 * n : 32)) return {(int)std::max(n, 1ll), 0};
    return {0, (int)std::min<long long>(slots, pairs * most)};
}

bool cache_ok(const tts_bb_kv4* c) {
    return c && c->pool && c->page_table && c->n_blocks >= 1 && c->n_seqs >= 1 && c->blocks_per_seq >= 1 &&
           (uintptr_t)c->pool % 16 == 0 && words_aligned(c->page_table, c->err);
}
Cache cache_of(const tts_bb_kv4* c) {
    return Cache{static_cast<uint8_t*>(c->pool), c->page_table, c->err, c->n_blocks, c->n_seqs, c->blocks_per_seq};
}
bool type_ok(int t) { return t == TTS_BB_T_F32 || t == TTS_BB_T_BF16; }
bool aligned(const void* p) { return (uintptr_t)p % 16 == 0; }
tts_bb_status status() { return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA; }

// launch_pdl with clusters of n blocks along x
template <typename... KArgs, typename... Args>
void launch_cluster(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int n, Args... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = n;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, k, static_cast<KArgs>(args)...);
}

// fp32 prompts take two launches: the q heads need half of the registers, and twice as many of their warps then hide memory:
// 24463 tokens 159 us, 168 in one. bf16 ones, whose values on the way take half the registers, take one: 107 us, 110 in two.
constexpr int SPLIT_TOKENS = 4096;
template <typename TI, typename TQ>
void append(int T, const void* qkv, int64_t stride, const void* gq, const void* gk, float eps, const float* cos_t,
            const float* sin_t, int n_pos, const int32_t* seqs, const int32_t* positions, const tts_bb_kv4* c, void* q_out,
            cudaStream_t st) {
    const auto go = [&](auto k, int parts) {
        launch_pdl(k, dim3(std::min(T, 6 * 152), parts), 128, 0, st, T, static_cast<const TI*>(qkv), (long long)stride, static_cast<const bf16*>(gq),
                   static_cast<const bf16*>(gk), eps, cos_t, sin_t, n_pos, seqs, positions, cache_of(c), static_cast<TQ*>(q_out));
    };
    if constexpr (sizeof(TI) == 4) {
        if (T >= SPLIT_TOKENS) {
            go(k_kv4_append<HEADS_KV, TI, TQ>, 1);
            if (q_out) go(k_kv4_append<HEADS_Q, TI, TQ>, 1);
            return;
        }
    }
    go(k_kv4_append<HEADS_Q | HEADS_KV, TI, TQ>, 2);
}

}  // namespace

TTS_API tts_bb_status tts_bb_rope_tables(double theta, int n_pos, float* cos_table, float* sin_table) {
    if (n_pos < 1 || !(theta > 0.0) || !cos_table || !sin_table) return TTS_BB_E_INVALID;
    for (int i = 0; i < HD / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / HD);
        for (int p = 0; p < n_pos; ++p) {
            cos_table[(size_t)p * (HD / 2) + i] = (float)std::cos(p * f);
            sin_table[(size_t)p * (HD / 2) + i] = (float)std::sin(p * f);
        }
    }
    return TTS_BB_OK;
}

TTS_API tts_bb_status tts_bb_kv4_append(const tts_bb_kv4* cache, int T, const void* qkv, int qkv_type, int64_t qkv_stride,
                                        const void* q_norm, const void* k_norm, float eps, const float* cos_table,
                                        const float* sin_table, int n_pos, const int32_t* seqs, const int32_t* positions,
                                        void* q_out, int q_type, void* stream) {
    if (!cache_ok(cache) || T < 1 || !qkv || !q_norm || !k_norm || !cos_table || !sin_table || n_pos < 1 || !seqs ||
        !positions || !type_ok(qkv_type) || !type_ok(q_type) || !(eps >= 0.f) || qkv_stride < QKV || qkv_stride % (qkv_type == TTS_BB_T_F32 ? 4 : 8) ||
        !aligned(qkv) || !aligned(q_out) || !aligned(q_norm) || !aligned(k_norm) || !aligned(cos_table) || !aligned(sin_table) ||
        !words_aligned(seqs, positions))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool fi = qkv_type == TTS_BB_T_F32, fq = q_type == TTS_BB_T_F32;
    auto go = [&](auto f) {
        f(T, qkv, qkv_stride, q_norm, k_norm, eps, cos_table, sin_table, n_pos, seqs, positions, cache, q_out, st);
    };
    if (fi && fq) go(append<float, float>);
    else if (fi) go(append<float, bf16>);
    else if (fq) go(append<bf16, float>);
    else go(append<bf16, bf16>);
    return status();
}

TTS_API tts_bb_status tts_bb_kv4_read(const tts_bb_kv4* cache, int T, const int32_t* seqs, const int32_t* positions,
                                      void* k_out, void* v_out, void* stream) {
    if (!cache_ok(cache) || T < 1 || !seqs || !positions || !k_out || !v_out || (uintptr_t)k_out % 16 || (uintptr_t)v_out % 16 ||
        !words_aligned(seqs, positions))
        return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const auto go = [&](auto k, int n) {
        launch_pdl(k, (T + n - 1) / n, 256, 0, static_cast<cudaStream_t>(stream), T, seqs, positions, cache_of(cache),
                   static_cast<bf16*>(k_out), static_cast<bf16*>(v_out));
    };
    if (T < 4 * 8 * 152) go(k_kv4_read<1>, 1);  // fewer than four tokens for each of the 8 blocks an SM holds
    else go(k_kv4_read<4>, 4);
    return status();
}

TTS_API size_t tts_bb_kv4_attention_workspace(int B, int S, int max_len) {
    if (B < 1 || S < 1 || S > TTS_BB_KV4_MAX_QUERIES || max_len < 1 || max_len > (1 << 30) || (long long)B * S > 65535) return 0;
    size_t most = 0;  // of both types
    for (int each = 1; each <= std::min(S, 2); ++each)
        for (int an_sm = each == 1 ? 4 : 3; an_sm <= 4; ++an_sm)
            most = std::max(most, (size_t)attn_plan((long long)B * ((S + each - 1) / each), max_len, an_sm * 152).shares * 2 * 2 * each * PIECE *
                                      sizeof(float));
    return most;
}

TTS_API tts_bb_status tts_bb_kv4_attention(const tts_bb_kv4* cache, int B, int S, const void* q, int type,
                                           const int32_t* seqs, const int32_t* kv_lens, int max_len, void* out,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!cache_ok(cache) || B < 1 || S < 1 || S > TTS_BB_KV4_MAX_QUERIES || (long long)B * S > 65535 || !q || !kv_lens ||
        !out || !type_ok(type) || !aligned(q) || !aligned(out) || max_len < 1 || max_len > (1 << 30) ||
        (long long)max_len > (long long)cache->blocks_per_seq * KVB || (!seqs && B > cache->n_seqs) ||
        !words_aligned(seqs, kv_lens))
        return TTS_BB_E_INVALID;
    const size_t need = tts_bb_kv4_attention_workspace(B, S, max_len);
    if (need && (!workspace || workspace_bytes < need || (uintptr_t)workspace % 16)) return TTS_BB_E_INVALID;
    if (cudaPeekAtLastError() != cudaSuccess) return TTS_BB_E_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Cache c = cache_of(cache);
    // query tokens of a sequence two at a time, in the columns of the products that one leaves empty
    auto go = [&](auto type_of, auto tokens) {
        typedef decltype(type_of) T;
        constexpr int N = decltype(tokens)::value;
        const int per_seq = (S + N - 1) / N, rows = B * per_seq;
        const Plan p = attn_plan(rows, max_len, AN_SM<T, N> * 152);
        const AttnArgs a{seqs, kv_lens, S, max_len, N, per_seq, rows, p.splits, static_cast<float*>(workspace)};
        constexpr size_t smem = RING_BYTES + (size_t)WARPS * (sizeof(T) == 4 ? 3 : 2) * 2 * N * HD * sizeof(float);
        static SmemState grid_state, line_state;
        allow_smem(grid_state, k_kv4_attn<T, N>, smem, true);
        allow_smem(line_state, k_kv4_attn_line<T, N>, smem);
        const T* const qt = static_cast<const T*>(q);
        T* const to = static_cast<T*>(out);
        if (p.splits > 1) {
            launch_cluster(k_kv4_attn<T, N>, dim3(p.splits, NKV, rows), WARPS * 32, smem, st, p.splits, qt, c, a, to);
        } else if (p.splits) {
            launch_pdl(k_kv4_attn<T, N>, dim3(1, NKV, rows), WARPS * 32, smem, st, qt, c, a, to);
        } else {
            launch_pdl(k_kv4_attn_line<T, N>, p.shares, WARPS * 32, smem, st, qt, c, a, to);
            launch_pdl(k_kv4_combine<T, N>, dim3(NQ * N, rows), 128, 0, st, c, a, p.shares, to);
        }
    };
    if (type == TTS_BB_T_F32 && S == 1) go(float{}, std::integral_constant<int, 1>{});
    else if (type == TTS_BB_T_F32) go(float{}, std::integral_constant<int, 2>{});
    else if (S == 1) go(bf16{}, std::integral_constant<int, 1>{});
    else go(bf16{}, std::integral_constant<int, 2>{});
    return status();
}
