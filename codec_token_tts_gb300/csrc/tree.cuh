// What the speculative decoding operators share: the paged bf16 cache's view, and the checks of trees and arguments.
#pragma once
#include "common.cuh"
#include "../../include/tts_bb.h"

namespace ttsbb {

constexpr int MAX_NODES = TTS_BB_TREE_MAX_NODES;
constexpr size_t KV_BLOCK = TTS_BB_KV_BLOCK_ELEMS;
static_assert(KV_BLOCK == (size_t)2 * NKV * KVB * HD, "block layout");

// One layer's pool, or (commit) the first of several.
struct Pages {
    bf16* pool;
    const int32_t* table;
    int32_t* err;
    long long layer_stride;
    int n_blocks, n_seqs, bps;
};
// The cache row of sequence b: -1 padding, -2 out of range.
__device__ __forceinline__ int row_of(const Pages& c, const int32_t* seqs, int b) {
    const int r = seqs ? seqs[b] : b;
    return r < 0 ? -1 : r < c.n_seqs ? r : -2;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool cache_ok(const tts_bb_kv_cache* c) {
    return c && c->pool && c->page_table && c->n_layers >= 1 && c->n_blocks >= 1 && c->n_blocks <= (1 << 20) && c->n_seqs >= 1 &&
           c->blocks_per_seq >= 1 && aligned16(c->pool) && words_aligned(c->page_table, c->err) &&
           (c->n_layers == 1 || (c->layer_stride >= (int64_t)(c->n_blocks * KV_BLOCK) && c->layer_stride % 8 == 0));
}
inline bool tree_ok(int B, int N) { return B >= 1 && N >= 1 && N <= MAX_NODES && (long long)B * N <= 65535; }
inline Pages pages_of(const tts_bb_kv_cache* c, int layer) {
    const long long stride = c->n_layers == 1 ? 0 : c->layer_stride;
    return Pages{static_cast<bf16*>(c->pool) + layer * stride, c->page_table, c->err, stride, c->n_blocks, c->n_seqs, c->blocks_per_seq};
}
inline tts_bb_status launched() { return cudaPeekAtLastError() == cudaSuccess ? TTS_BB_OK : TTS_BB_E_CUDA; }

}  // namespace ttsbb
