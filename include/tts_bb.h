/*
 * tts_bb.h — C ABI of the GB300 (sm_103a) engine for the forward step of the
 * Qwen3-0.6B-shaped backbone that drives codec-token speech generation.
 *
 * The backbone (28 layers, hidden 1024, 16 query / 8 KV heads of 128, SwiGLU
 * 3072, RMSNorm eps 1e-6, q/k RMSNorm before half-rotate RoPE theta 1e6) is the
 * one described on "omnivoice-cpp docs/ARCHITECTURE.md" (GGUF layout;
 * Component architecture, Qwen3 specifics) and "Qwen3-TTS ncnn port"
 * (Tencent/ncnn discussion 6877; model structure, Talker and Code Predictor;
 * single-token SDPA and host attention; mRoPE conclusion).
 *
 * Conventions follow the public C99 ABI of omnivoice-cpp (Public API and ABI
 * guarantee): an opaque handle, a default-initialiser for the config struct,
 * a negative status enum, caller-owned outputs, a version string. The header
 * is plain C99; the library exports only tts_bb_* symbols.
 *
 * Pointers. Unless a parameter says otherwise:
 *   - "device" arrays are CUDA device pointers (e.g. torch CUDA tensors) on
 *     the device that was current at tts_bb_create; they must stay valid
 *     until the work enqueued on the handle's stream has finished;
 *   - "host" arrays are ordinary CPU memory read before the call returns.
 * All compute calls are asynchronous on the handle's stream. Host-side
 * argument errors return before anything is enqueued and change no state.
 * Device-side errors (an out-of-range id) are latched in a device error word:
 * with config.sync_errors = 1 every call ends by reading it (one stream
 * synchronisation); with 0 the caller reads it with tts_bb_sync().
 * A handle is not thread-safe: one host thread at a time.
 */
#ifndef TTS_BB_H
#define TTS_BB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TTS_BB_VERSION_MAJOR 0
#define TTS_BB_VERSION_MINOR 1
#define TTS_BB_VERSION_PATCH 0

#define TTS_BB_MAX_CODEBOOKS 16
#define TTS_BB_MAX_HEADS 16
#define TTS_BB_KV_BLOCK 64

typedef struct tts_bb tts_bb; /* opaque engine handle */

typedef enum {
    TTS_BB_OK = 0,
    TTS_BB_E_INVALID = -1,         /* bad argument; nothing was enqueued */
    TTS_BB_E_UNSUPPORTED = -2,     /* valid C, a shape the kernels are not built for */
    TTS_BB_E_CUDA = -3,            /* a CUDA runtime call failed */
    TTS_BB_E_OOM = -4,             /* device memory or KV blocks exhausted */
    TTS_BB_E_DEVICE_TIMEOUT = -5,  /* a bounded device-side wait ran out */
    TTS_BB_E_BAD_ID = -6,          /* a token id was out of its table (it was skipped) */
    TTS_BB_E_NOT_IMPLEMENTED = -7
} tts_bb_status;

/* Backbone and engine shape. Field names follow the Code Predictor config of
 * "rightkit-qts 0.2.0" (Mode API: hidden_size, n_layers, heads, kv heads,
 * intermediate_size, head_dim, rms_norm_eps, rope_theta, vocab_size). */
typedef struct {
    int n_layers;          /* 28 Talker / OmniVoice, 5 Code Predictor */
    int hidden;            /* 1024 (the only value the kernels support) */
    int n_q_heads;         /* 16 */
    int n_kv_heads;        /* 8 */
    int head_dim;          /* 128 */
    int ffn;               /* 3072 */
    float rms_eps;         /* 1e-6 */
    float rope_theta;      /* 1e6 */
    /* Input embedding: the codebook tables E_0..E_{n_codebooks-1} are summed
     * (Qwen3-TTS ncnn port, model structure: the 16 embeddings of a frame are
     * added to form the next Talker input). */
    int n_codebooks;
    int codebook_rows[TTS_BB_MAX_CODEBOOKS];
    /* OmniVoice hybrid input (omnivoice-cpp, Component architecture): a text
     * table of text_vocab rows and an audio table of audio_codebooks *
     * audio_vocab rows. 0 = absent. */
    int text_vocab;
    int audio_codebooks;
    int audio_vocab;
    /* Output heads: n_heads bf16 matrices of [head_rows][hidden] (Talker 1 x
     * 3072, Code Predictor 15 x 2048). For OmniVoice set n_heads = audio_codebooks
     * and head_rows = audio_vocab: one [n_heads*head_rows][hidden] matrix
     * (audio_heads) is passed in head[0]. 0 heads = hidden-state only. */
    int n_heads;
    int head_rows;
    /* KV cache: paged, TTS_BB_KV_BLOCK tokens per block. */
    int max_slots;         /* concurrent sequences (stream slots), at most 2^20 */
    int max_ctx;           /* longest sequence, tokens, at most 2^20 */
    int kv_blocks;         /* physical blocks; 0 = max_slots * ceil(max_ctx / 64) */
    int max_batch;         /* largest B of one call (scratch sizing) */
    int max_tokens;        /* largest B*S of one prefill / MaskGIT call, at most 2^20 */
    int sync_errors;       /* 1 = each call synchronises to report device errors */
} tts_bb_config;

/* Per-layer tensor roles (PyTorch (out, in) row-major, bf16). */
enum {
    TTS_BB_W_IN_NORM = 0,  /* [hidden]           input_layernorm */
    TTS_BB_W_Q,            /* [heads*128][hidden] q_proj */
    TTS_BB_W_K,            /* [kv*128][hidden]   k_proj */
    TTS_BB_W_V,            /* [kv*128][hidden]   v_proj */
    TTS_BB_W_Q_NORM,       /* [128]              q_norm */
    TTS_BB_W_K_NORM,       /* [128]              k_norm */
    TTS_BB_W_O,            /* [hidden][heads*128] o_proj */
    TTS_BB_W_POST_NORM,    /* [hidden]           post_attention_layernorm */
    TTS_BB_W_GATE,         /* [ffn][hidden]      gate_proj */
    TTS_BB_W_UP,           /* [ffn][hidden]      up_proj */
    TTS_BB_W_DOWN,         /* [hidden][ffn]      down_proj */
    TTS_BB_LAYER_TENSORS
};

/* Weight pointers, bf16 bit patterns. Host or device memory (anything
 * cudaMemcpy with cudaMemcpyDefault accepts). tts_bb_create copies them into
 * engine-owned device memory (fusing q/k/v and interleaving gate/up), so the
 * caller may free its copies once tts_bb_create has returned. */
typedef struct {
    const void* codebook[TTS_BB_MAX_CODEBOOKS]; /* [codebook_rows[k]][hidden] */
    const void* text_table;                     /* [text_vocab][hidden] or NULL */
    const void* audio_table;                    /* [audio_codebooks*audio_vocab][hidden] or NULL */
    const void* const* layer;                   /* n_layers * TTS_BB_LAYER_TENSORS pointers */
    const void* final_norm;                     /* [hidden] */
    const void* head[TTS_BB_MAX_HEADS];         /* [head_rows][hidden] each */
} tts_bb_weights;

/* Optional per-call inputs and outputs. NULL options = all defaults. */
typedef struct {
    /* device bf16 [tokens][hidden], added to the codebook sum (the Code
     * Predictor's Talker-hidden row, or a plain embedding input). */
    const void* embeds;
    /* device fp32 [tokens][hidden]: the residual after the last layer, before
     * the final norm. */
    float* hidden_out;
    /* element stride between consecutive rows of argmax_out (0 = 1): lets a
     * Talker / Code-Predictor loop write codes straight into the next frame's
     * id matrix. */
    int argmax_stride;
} tts_bb_opts;

/* Fill *cfg with the Qwen3-TTS Talker shape: 28 layers, 16 codebooks
 * (E_0 3072 rows, E_1..E_15 2048 rows), one 3072-row head, 64 slots, 4096 ctx. */
void tts_bb_default_config(tts_bb_config* cfg);

/* Create an engine on the current CUDA device; `stream` is a cudaStream_t
 * (NULL = the legacy default stream) on which every call of the handle runs.
 * Allocates the weights, the KV block pool and scratch. Returns
 * TTS_BB_E_INVALID for a bad config, TTS_BB_E_UNSUPPORTED for a shape the
 * kernels are not built for (or max_slots, max_ctx, max_tokens above 2^20),
 * TTS_BB_E_OOM when device or host memory runs out. No exception leaves the
 * call. */
tts_bb_status tts_bb_create(const tts_bb_config* cfg, const tts_bb_weights* w,
                            void* stream, tts_bb** out);

/* Wait for the handle's work and free everything it owns. NULL is a no-op. */
void tts_bb_free(tts_bb* h);

/* Causal prefill (Qwen3-TTS ncnn port: prompt prefill fills the per-layer
 * KV cache). Sequence b appends lens[b] tokens (1..S) to slot slots[b],
 * starting at the slot's current length, so a prefill can extend a cache.
 *   B, S      batch and padded length; B*S <= max_tokens, B <= max_batch
 *   slots     host int32 [B], distinct, in [0, max_slots)
 *   lens      host int32 [B], 1..S
 *   ids       device int32 [B][S][n_codebooks]; -1 = no token from that
 *             codebook at that position; NULL = embeddings only
 *   head_idx  head applied to the last valid position of each row (-1 = none)
 *   logits_out device fp32 [B][head_rows] or NULL
 *   argmax_out device int32 [B] (stride opts->argmax_stride) or NULL; the
 *             lowest index wins a tie
 *   opts->embeds     [B][S][hidden]; opts->hidden_out [B][S][hidden]
 * An out-of-table id is skipped and reported as TTS_BB_E_BAD_ID. */
tts_bb_status tts_bb_prefill(tts_bb* h, int B, int S, const int32_t* slots, const int32_t* lens,
                             const int32_t* ids, int head_idx, float* logits_out,
                             int32_t* argmax_out, const tts_bb_opts* opts);

/* One decode step, query length 1, for B sequences (Qwen3-TTS ncnn port,
 * single-token SDPA and host attention: RoPE, KV append and GQA attention over
 * the cache for a query of length 1).
 *   slots    host int32 [B], distinct
 *   kv_lens  host int32 [B]: tokens already cached in each slot; must equal
 *            the engine's length for the slot (TTS_BB_E_INVALID otherwise).
 *            The new token is written at position kv_lens[b] and attention
 *            covers kv_lens[b] + 1 tokens.
 *   ids      device int32 [B][n_codebooks] (-1 = absent) or NULL
 *   logits_out / argmax_out as in tts_bb_prefill, one row per sequence
 *   opts->embeds [B][hidden]; opts->hidden_out [B][hidden] */
tts_bb_status tts_bb_decode_step(tts_bb* h, int B, const int32_t* slots, const int32_t* kv_lens,
                                 const int32_t* ids, int head_idx, float* logits_out,
                                 int32_t* argmax_out, const tts_bb_opts* opts);

/* tts_bb_decode_step with HOST buffers, for a caller that keeps its ids and
 * reads each step's tokens on the host (a streaming loop): copies ids (host
 * int32 [B][n_codebooks], pinned for an asynchronous copy) to the device, runs
 * the step, copies argmax_out (host int32 [B] or NULL) and logits_out (host
 * fp32 [B][head_rows] or NULL) back, and returns once they have landed (one
 * stream synchronisation, which also reads the device error word). Other
 * arguments and errors as in tts_bb_decode_step. Device staging for max_batch
 * rows is allocated on the first call. */
tts_bb_status tts_bb_decode_step_host(tts_bb* h, int B, const int32_t* slots, const int32_t* kv_lens,
                                      const int32_t* ids, int head_idx, int32_t* argmax_out, float* logits_out);

/* One full bidirectional MaskGIT pass without a KV cache (omnivoice-cpp,
 * MaskGIT decoder: every step is a full prefill with non-causal attention;
 * Component architecture: hybrid text/audio embedding and audio heads;
 * Inner-loop optimisations: logits only over the audio window).
 *   ids         device int32 [B][audio_codebooks][S] (text id on every row at
 *               text positions, audio codes 0..audio_vocab-1 at audio positions)
 *   audio_mask  device uint8 [B][S], 1 = audio position
 *   key_lens    host int32 [B] (keys >= key_lens[b] are padding) or NULL = S
 *   audio_start first position of the audio window, 0 <= audio_start < S
 *   logits_out  device fp32 [B][n_heads][S - audio_start][head_rows]:
 *               logits[b][k][s][v] = final_norm(x[b][audio_start+s]) . W[k*head_rows + v]
 *   opts->hidden_out [B][S][hidden]
 * Requires a handle with text and audio tables; B*S <= max_tokens. */
tts_bb_status tts_bb_maskgit_pass(tts_bb* h, int B, int S, const int32_t* ids,
                                  const uint8_t* audio_mask, const int32_t* key_lens,
                                  int audio_start, float* logits_out, const tts_bb_opts* opts);

/* One frame of the Talker -> Code Predictor loop (Qwen3-TTS ncnn port, model
 * structure: the Talker predicts codebook 0 of each frame, the Code Predictor
 * the other 15 in 15 autoregressive steps, and the frame's 16 embeddings
 * summed are the Talker's next input), for B streams at once, greedy:
 *   1. the Talker decodes `codes` (this frame's input, [B][16], -1 = absent)
 *      at position kv_lens[b] of slot slots[b] (as tts_bb_decode_step), head 0
 *      -> code 0, and its last-layer hidden state;
 *   2. the Code Predictor runs a 2-token prefill in its slots 0..B-1: position
 *      0 = the Talker hidden state after the Talker's final norm (bf16),
 *      position 1 = E_0[code 0]; head 0 -> code 1; then calls j = 1..14 feed
 *      E_j[code j] at position j + 1, head j -> code j + 1; its slots are
 *      released afterwards;
 *   3. codes[b] = the frame's 16 codes (the next frame's input).
 *   talker, cp     handles on the same stream; cp has 16 codebooks (the
 *                  Talker's tables), >= 15 heads, B <= max_slots, max_batch,
 *                  2 B <= max_tokens, max_ctx >= 16
 *   slots, kv_lens host int32 [B] for the Talker, as in tts_bb_decode_step
 *   codes          device int32 [B][16], read then overwritten
 *   talker_logits  device fp32 [B][Talker head_rows] or NULL
 * Everything runs on the shared stream (about 2 + 16 launches and, for B > 2,
 * graph replays); scratch is allocated on the first call that needs more.
 * Errors as in tts_bb_decode_step / tts_bb_prefill (status of the first call
 * that failed); TTS_BB_E_INVALID for handles that do not fit. */
tts_bb_status tts_bb_frame_step(tts_bb* talker, tts_bb* cp, int B, const int32_t* slots,
                                const int32_t* kv_lens, int32_t* codes, float* talker_logits);

/* Greedy token update of one MaskGIT refinement step on the device
 * (omnivoice-cpp, MaskGIT decoder, class and position temperatures 0). The
 * batch of a pass holds n_items conditional rows (0..n_items-1) followed by
 * their n_items unconditional rows (n_items..2 n_items-1). For every target
 * cell (item i, codebook k < n_heads, position t < T):
 *   z     = c + cfg_scale (c - u), float32, c the conditional and u the
 *           unconditional logits of the cell (one rounding per operation)
 *   pred  = argmax of z over the ids other than the mask id (head_rows - 1),
 *           lowest id on ties
 *   score = z[pred] - logsumexp(z over all head_rows ids) - k layer_penalty
 * Cells whose current id (conditional row) is not the mask id are kept. Of
 * the masked cells of each item, the min(n_unmask, masked) with the highest
 * score (ties: lowest k T + t) take pred, written to the conditional and the
 * unconditional rows.
 *   logits  device fp32 [2 n_items][n_heads][S_logits][head_rows] (the
 *           maskgit_pass output); the cell's logits sit at position
 *           cond_pos0 + t (conditional rows) and uncond_pos0 + t
 *           (unconditional rows)
 *   ids     device int32 [2 n_items][n_heads][S_ids], updated in place at
 *           positions cond_ids_pos0 + t and uncond_ids_pos0 + t
 *   cfg_scale 2.0 and layer_penalty 5.0 on the page.
 * Two kernel launches on the handle's stream; the scratch (12 bytes per cell)
 * is allocated on the first call that needs more. TTS_BB_E_INVALID for
 * windows outside their tensors, n_items < 1, T < 1, n_unmask < 0 or a
 * handle without audio heads (or with more than 1056 ids per head). */
tts_bb_status tts_bb_maskgit_update(tts_bb* h, int n_items, int T, const float* logits, int S_logits,
                                    int cond_pos0, int uncond_pos0, int32_t* ids, int S_ids,
                                    int cond_ids_pos0, int uncond_ids_pos0, int n_unmask,
                                    float cfg_scale, float layer_penalty);

/* Cells newly unmasked at each of num_step MaskGIT steps, host only:
 * counts[i] = ceil(n_total (t'[i+1] - t'[i])) with t[i] = i / num_step
 * shifted by t' = s t / (s t + (1 - t)), s = t_shift (0.1 on the page, whose
 * time-step function is not printed: this shift is a reading). The counts sum
 * to at least n_total. TTS_BB_E_INVALID for num_step < 1, n_total < 0,
 * t_shift <= 0 or a NULL counts. */
tts_bb_status tts_bb_maskgit_schedule(int num_step, int n_total, double t_shift, int32_t* counts);

/* RVQ codec decode (omnivoice-cpp, Audio tokenizer pipeline, Decode, and RVQ
 * codec): codes of K codebooks -> out_dim frame features,
 *   out[b][t] = sum_k ( embed_k[codes[b][k][t]] . proj_w_k^T + proj_b_k )
 * with embed_k [codebook_size][dim] (codebook.embed), proj_w_k [out_dim][dim]
 * (project_out.weight) and proj_b_k [out_dim] (project_out.bias), all device
 * bf16 pointers, K of each; the OmniVoice codec has K = 8, 1024 x 64 tables and
 * out_dim 1024. tts_bb_rvq_create copies them (the caller may free its copies)
 * and returns TTS_BB_E_INVALID for NULL pointers or sizes outside
 * 1 <= K <= 64, dim a multiple of 8 with K * dim a multiple of 64,
 * TTS_BB_E_OOM, TTS_BB_E_UNSUPPORTED without tcgen05 tensor maps. */
typedef struct tts_bb_rvq tts_bb_rvq;
tts_bb_status tts_bb_rvq_create(int n_codebooks, int codebook_size, int dim, int out_dim,
                                const void* const* embed, const void* const* proj_w,
                                const void* const* proj_b, void* stream, tts_bb_rvq** out);
/* codes device int32 [B][K][T]; out device fp32 [B][T][out_dim]. Asynchronous
 * on the handle's stream (a gather kernel and one GEMM); a code outside
 * 0..codebook_size-1 contributes nothing and is reported by tts_bb_rvq_sync as
 * TTS_BB_E_BAD_ID. Scratch (K * dim bf16 per frame) grows on the first call
 * that needs more. */
tts_bb_status tts_bb_rvq_decode(tts_bb_rvq* r, int B, int T, const int32_t* codes, float* out);
/* Wait for the handle's work; returns (and clears) a latched device error. */
tts_bb_status tts_bb_rvq_sync(tts_bb_rvq* r);
/* Wait and free. NULL is a no-op. */
void tts_bb_rvq_free(tts_bb_rvq* r);

/* Qwen3-TTS codec quantizer lookup (Qwen3-TTS ncnn port, Codec Decoder split,
 * steps 1-4): the frame's 16 codes -> the 512-channel float hidden that the
 * codec body reads,
 *   out[b][o][t] = P_sem[o] . C_0[codes[b][0][t]]
 *                + P_ac[o] . sum_{k=1..K-1} C_k[codes[b][k][t]]
 * i.e. the first (semantic) codebook through its own projection and the
 * other K-1 (acoustic) codebooks summed through the second projection.
 *   codebooks     K device bf16 pointers, each [codebook_size][dim]
 *   proj_semantic device bf16 [out_dim][dim]; proj_acoustic the same
 * (the page: 16 codebooks of 2048 entries, out_dim 512; it does not print the
 * codebook width, so dim is a parameter; the projections are bias-free).
 * tts_bb_quantizer_create copies them (the caller may free its copies) and
 * returns TTS_BB_E_INVALID for NULL pointers or sizes outside 2 <= K <= 32,
 * dim a multiple of 64 in 64..1024, 1 <= out_dim <= 8192; TTS_BB_E_OOM. */
typedef struct tts_bb_quantizer tts_bb_quantizer;
tts_bb_status tts_bb_quantizer_create(int n_codebooks, int codebook_size, int dim, int out_dim,
                                      const void* const* codebooks, const void* proj_semantic,
                                      const void* proj_acoustic, void* stream, tts_bb_quantizer** out);
/* codes device int32 [B][K][T]; out device fp32 [B][out_dim][T] (channel-major,
 * the [1, 512, T] layout the page feeds to the codec body). Asynchronous on the
 * handle's stream (a gather kernel and one GEMM); the acoustic sum is carried
 * as bf16 high + low parts, so the result keeps fp32-level accuracy over the
 * bf16 tables. A code outside 0..codebook_size-1 contributes nothing and is
 * reported by tts_bb_quantizer_sync as TTS_BB_E_BAD_ID. Scratch (3 * dim bf16
 * per frame, rounded up to 256) grows on the first call that needs more. */
tts_bb_status tts_bb_quantizer_decode(tts_bb_quantizer* q, int B, int T, const int32_t* codes, float* out);
/* Wait for the handle's work; returns (and clears) a latched device error. */
tts_bb_status tts_bb_quantizer_sync(tts_bb_quantizer* q);
/* Wait and free. NULL is a no-op. */
void tts_bb_quantizer_free(tts_bb_quantizer* q);

/* DAC decoder: frame features -> 24 kHz audio (omnivoice-cpp, Audio tokenizer
 * pipeline, Decode; DAC decoder block channels; Snake activation;
 * ConvTranspose1d): fc2 Linear 1024 -> 256, conv1 (256 -> 1024, k 7, pad 3),
 * five blocks with ratios r = 8, 5, 4, 2, 3 and channels 1024 -> 512 -> 256 ->
 * 128 -> 64 -> 32 (snake; ConvTranspose1d k 2r, stride r, padding ceil(r/2),
 * output_padding r % 2; three residual units with dilations 1, 3, 9: snake,
 * Conv1d k 7 pad 3d, snake, Conv1d k 1, add), snake, conv2 (32 -> 1, k 7,
 * pad 3). Snake: y = x + sin(alpha x)^2 / (alpha + 1e-9), alpha per channel.
 * Every convolution and the Linear have a bias. All weights are device fp32
 * in PyTorch layouts; tts_bb_dac_create copies them. */
typedef struct {
    const float* alpha;          /* [IC] snake before the upsampling convolution */
    const float* up_w;           /* [IC][OC][2r] ConvTranspose1d weight */
    const float* up_b;           /* [OC] */
    const float* res_alpha1[3];  /* [OC] */
    const float* res_w1[3];      /* [OC][OC][7] */
    const float* res_b1[3];      /* [OC] */
    const float* res_alpha2[3];  /* [OC] */
    const float* res_w2[3];      /* [OC][OC][1] */
    const float* res_b2[3];      /* [OC] */
} tts_bb_dac_block;
typedef struct {
    const float* fc2_w;          /* [256][1024] */
    const float* fc2_b;          /* [256] */
    const float* conv1_w;        /* [1024][256][7] */
    const float* conv1_b;        /* [1024] */
    tts_bb_dac_block block[5];
    const float* final_alpha;    /* [32] */
    const float* conv2_w;        /* [1][32][7] */
    const float* conv2_b;        /* [1] */
} tts_bb_dac_weights;
typedef struct tts_bb_dac tts_bb_dac;
/* TTS_BB_E_INVALID for a NULL pointer, TTS_BB_E_OOM when memory runs out. */
tts_bb_status tts_bb_dac_create(const tts_bb_dac_weights* w, void* stream, tts_bb_dac** out);
/* features device fp32 [B][T][1024] (the RVQ decode output); audio device fp32
 * [B][960 T]. Asynchronous on the handle's stream; three activation buffers of
 * 30720 T floats per item are allocated on the first call that needs more.
 * fc2, conv1 and every convolution of the five blocks run on the tensor cores
 * (39 launches) with fp32 operands split into bf16 high + low parts (three
 * products per pair, fp32 accumulation) and time-major activations; conv2 runs
 * in fp32 on the CUDA cores. Environment TTS_BB_DAC=fp32 at create: every
 * convolution in fp32 on the CUDA cores, channel-major (38 launches).
 * TTS_BB_E_INVALID for NULL buffers, B < 1 or B > 65535, T < 1, or B x 960 T
 * above 2^31 - 1 samples. */
tts_bb_status tts_bb_dac_decode(tts_bb_dac* d, int B, int T, const float* features, float* audio);
/* Wait for the handle's work; returns (and clears) a latched device error
 * (TTS_BB_E_DEVICE_TIMEOUT: a bounded wait of a tensor-core kernel ran out). */
tts_bb_status tts_bb_dac_sync(tts_bb_dac* d);
/* Wait and free. NULL is a no-op. */
void tts_bb_dac_free(tts_bb_dac* d);

/* Return the slot's KV blocks to the pool; its length becomes 0. */
tts_bb_status tts_bb_release(tts_bb* h, int slot);

/* Shorten a slot to `len` tokens (0 <= len <= current length); blocks past
 * the new end go back to the pool. Positions >= len are rewritten by the next
 * prefill or decode step. */
tts_bb_status tts_bb_truncate(tts_bb* h, int slot, int len);

/* Current cached length of a slot, or -1 for a bad handle or slot. */
int tts_bb_slot_len(const tts_bb* h, int slot);

/* Wait for the handle's stream and report (then clear) any latched device error. */
tts_bb_status tts_bb_sync(tts_bb* h);

/* Text of the last error on this handle (empty string if none). */
const char* tts_bb_last_error(const tts_bb* h);

/* "MAJOR.MINOR.PATCH (sm_103a)". */
const char* tts_bb_version(void);

/* Test hooks: read or write n tokens of one layer's cache of one slot,
 * positions pos0..pos0+n-1, through the page table.
 *   k, v  device bf16 [n][n_kv_heads][head_dim] (keys after q/k-norm and RoPE)
 * tts_bb_debug_kv_write extends the slot to pos0+n if it was shorter
 * (allocating blocks); pos0 must not exceed the current length. */
tts_bb_status tts_bb_debug_kv_read(tts_bb* h, int layer, int slot, int pos0, int n,
                                   void* k_out, void* v_out);
tts_bb_status tts_bb_debug_kv_write(tts_bb* h, int layer, int slot, int pos0, int n,
                                    const void* k, const void* v);

/* Test hooks for failure handling (no counterpart on the pages): they force
 * device-side waits to run out without faulting the GPU.
 *   what = TTS_BB_DEBUG_WAIT_LIMIT_NS: every wait of the persistent decode
 *          step (exchange polls, weight-ring slots) gives up after arg ns
 *          (default 2e9; arg in 1e6 .. 1e10, else TTS_BB_E_INVALID).
 *   what = TTS_BB_DEBUG_STALL_NEXT_STEP: the next persistent decode step
 *          (batch <= 2) withholds one CTA's exchange words, so every CTA's
 *          wait runs out; that step returns TTS_BB_E_DEVICE_TIMEOUT (its
 *          outputs are undefined) and the handle stays usable. arg unused.
 * Returns TTS_BB_E_INVALID for a null handle or an unknown `what`. The
 * environment variable TTS_BB_FAIL_ALLOC_AT=n makes the n-th device
 * allocation of a handle being created fail (creation returns TTS_BB_E_OOM). */
enum { TTS_BB_DEBUG_WAIT_LIMIT_NS = 1, TTS_BB_DEBUG_STALL_NEXT_STEP = 2 };
tts_bb_status tts_bb_debug_fault(tts_bb* h, int what, int64_t arg);

/* Number of kernel launches the handle has enqueued since creation (a
 * counter kept on the host; lets a caller count launches in a timed region). */
uint64_t tts_bb_launch_count(const tts_bb* h);

/* Per-kernel timing. tts_bb_profile(h, 1) clears the record and brackets
 * every later kernel launch of the handle with CUDA events on its stream;
 * tts_bb_profile(h, 0) stops. tts_bb_profile_report waits for the stream and
 * returns a JSON summary {"kernels": [{"kind", "launches", "ms", "bytes",
 * "flops"}]}: per kernel kind, the launches, their summed event time and
 * their algorithmic bytes and flops. The string stays valid until the next
 * report or tts_bb_free. The events add a little time between launches, so
 * time a clean run without profiling. */
tts_bb_status tts_bb_profile(tts_bb* h, int on);
const char* tts_bb_profile_report(tts_bb* h);

/* Decode attention that allocates nothing (the pages have no counterpart: it
 * exists for callers of this library that may not call cudaMalloc — a plug-in
 * whose host framework owns every device allocation, or a real-time audio
 * thread that must not block in the allocator).
 *
 * It runs the same GQA decode attention kernels as tts_bb_decode_step on the
 * caller's own buffers (split-K flash decode; for max_position < 32 one warp
 * per query and KV head, which writes no partials); the split partials go to
 * a fixed array in device memory that is part of the library (TTS_BB_STATIC_ATTN_MAX_B x 16 heads x
 * TTS_BB_STATIC_ATTN_MAX_SPLITS x 130 floats = 4.26 MB, held by every GPU that
 * loads the library until the process exits). No cudaMalloc or cudaFree, no
 * allocating library call.
 *   q           device bf16 [B][16][128]: queries after q-norm and RoPE
 *   kv_pool     device bf16 blocks [n][2][8][64][128]: block p holds K then V
 *               of 64 positions for the 8 KV heads (the engine's pool layout)
 *   page_table  device int32 [B][blocks_per_seq]: physical block of each
 *               64-token block of sequence b
 *   positions   device int32 [B]: position of the query token of sequence b;
 *               its K/V must already be in the pool, attention covers
 *               positions 0..positions[b]. Values outside 0..max_position
 *               are clamped into that range on the device before any read
 *               (so no access leaves the caller's page-table rows); the
 *               output of such a sequence is then not meaningful
 *   max_position the largest value in positions (host int)
 *   out         device bf16 [B][16][128]
 *   stream      cudaStream_t (NULL = legacy default stream)
 * Returns TTS_BB_E_INVALID for NULL pointers, B outside
 * 1..TTS_BB_STATIC_ATTN_MAX_B or a max_position the page table cannot hold;
 * TTS_BB_E_CUDA if a CUDA error is already pending when the call starts (it
 * is left pending, not cleared) or a launch fails. The first call on a device looks up the
 * array's device address (cudaGetSymbolAddress) with that device current. Every call shares the
 * array and overwrites all the partials it reads, so nothing needs clearing
 * between calls; calls that overlap on the GPU (other streams, other host
 * threads) race on it and must be serialised by the caller. */
#define TTS_BB_STATIC_ATTN_MAX_B 64
#define TTS_BB_STATIC_ATTN_MAX_SPLITS 8
tts_bb_status tts_bb_gqa_decode_attention_static(const void* q, const void* kv_pool, const int32_t* page_table,
                                                 int blocks_per_seq, const int32_t* positions, int B,
                                                 int max_position, void* out, void* stream);

/* ------------------------------------------------------------------------
 * Low-bit decode operators: a paged KV cache held in 4 bits, products with
 * 4-bit weights, and log probabilities of the answers. Like
 * tts_bb_gqa_decode_attention_static they work on the caller's buffers alone:
 * every array is device memory of the current device, every call is
 * asynchronous on `stream` (a cudaStream_t of that device, NULL = legacy
 * default stream), allocates nothing, keeps nothing between calls and may be
 * captured into a CUDA graph. Calls on several streams or threads at once are
 * independent as long as what they write (outputs, workspaces, the same cache
 * rows) is not shared. Arrays of int32, uint32 and fp32 are 4-byte aligned, others as
 * stated. Host-side argument errors return TTS_BB_E_INVALID before anything is
 * enqueued; TTS_BB_E_CUDA: a CUDA error was already pending (it is left pending)
 * or a launch failed. */

/* Element types of arrays that may have several. */
enum { TTS_BB_T_F32 = 0, TTS_BB_T_BF16 = 1, TTS_BB_T_F16 = 2 };

/* A paged KV cache in 4 bits: 4.5 bits a value. One block holds 64 tokens (the
 * positions 64 j .. 64 j + 63 of a sequence) as K then V tiles of the 8 KV heads:
 *   pool[block][2][8] tiles of TTS_BB_KV4_TILE_BYTES: 64 code rows of 64 bytes,
 *   then 64 parameter rows of 8 bytes, one of each for a token.
 * The 128 dims of a head are two groups of 64 (dims 0..63 and 64..127). Word w
 * (32 bits, little endian) of a code row holds dims 64 (w & 1) + 8 (w >> 1) + i
 * in nibble i (bits 4 i .. 4 i + 3); a parameter row holds (bf16 scale, bf16
 * offset) of group 0, then of group 1. A value is scale * (code + 128 + offset).
 * A group x is quantised with scale = bf16(max((hi - lo) / 15, max|x| / 120)),
 * zero = rint(lo / scale), code = clamp(rint(x / scale) - zero, 0, 15) and offset =
 * zero - 128 (codes 0 and offset -128 where scale is 0; a group with a value
 * that is not finite is held as NaN; magnitudes up to 1e38).
 * A pool must be zeroed or written before it is read: blocks past a sequence's
 * keys may hold anything. */
#define TTS_BB_KV4_TILE_BYTES 4608
#define TTS_BB_KV4_BLOCK_BYTES 73728 /* 2 * 8 tiles; a bf16 block has 262144 */
#define TTS_BB_KV4_MAX_QUERIES 64    /* query tokens of a sequence in one attention call */
/* Bits of a cache's error word. */
enum {
    TTS_BB_KV4_ERR_PAGE = 1, /* a page-table entry outside 0..n_blocks-1 was met */
    TTS_BB_KV4_ERR_RANGE = 2 /* a sequence row >= n_seqs, a position outside the page table or the
                                cos / sin tables, or a key count outside 0..max_len */
};
typedef struct {
    void* pool;                /* device, 16-byte aligned: n_blocks * TTS_BB_KV4_BLOCK_BYTES */
    const int32_t* page_table; /* device int32 [n_seqs][blocks_per_seq]: block of each 64 positions */
    int32_t* err;              /* device word, or NULL: the bits of what calls skipped are ORed into it */
    int n_blocks;
    int n_seqs;
    int blocks_per_seq;
} tts_bb_kv4;

/* cos and sin of pos * theta^(-2 i / 128), i < 64, for positions 0 .. n_pos - 1, host only: fills two
 * host fp32 arrays [n_pos][64] (angles and functions in 64 bits, rounded once), to be copied to the
 * device for tts_bb_kv4_append. TTS_BB_E_INVALID for n_pos < 1, theta <= 0 or a NULL array. */
tts_bb_status tts_bb_rope_tables(double theta, int n_pos, float* cos_table, float* sin_table);

/* Append T tokens: q/k RMSNorm, half-rotate RoPE and the 4-bit quantisation of keys and values, in one
 * launch (fp32 prompts in two). Token t belongs to cache row seqs[t] at position positions[t]; a negative seqs[t] is padding:
 * nothing is done for it. A token whose row, position or page is out of range is skipped as a whole (its
 * q_out row too) and reported in cache->err. The (row, position) pairs of one call must differ, else what
 * that position holds is unspecified.
 *   qkv        [T] rows of 4096 (16 q, 8 k, 8 v heads of 128), fp32 or bf16 (qkv_type), rows
 *              qkv_stride elements apart (>= 4096), every row 16-byte aligned
 *   q_norm, k_norm  bf16 [128] gains, 16-byte aligned; eps inside the root
 *   cos_table, sin_table  fp32 [n_pos][64], 16-byte aligned; the pairs (i, i + 64) rotate by row positions[t]
 *   seqs, positions int32 [T]
 *   q_out      fp32 or bf16 (q_type) [T][16][128]: the rotated queries, 16-byte aligned, or NULL
 * The codes and parameters are those of the exact arithmetic (values next to a border between two codes are decided
 * in 48 bits), for q and k up to 1e18 in magnitude, beyond which their squares overflow. */
tts_bb_status tts_bb_kv4_append(const tts_bb_kv4* cache, int T, const void* qkv, int qkv_type, int64_t qkv_stride,
                                const void* q_norm, const void* k_norm, float eps, const float* cos_table,
                                const float* sin_table, int n_pos, const int32_t* seqs, const int32_t* positions,
                                void* q_out, int q_type, void* stream);

/* The values the cache holds for T tokens (seqs, positions as in tts_bb_kv4_append), rounded to bf16:
 * k_out, v_out bf16 [T][8][128], 16-byte aligned. Rows of padding and of tokens out of range are left as they were. */
tts_bb_status tts_bb_kv4_read(const tts_bb_kv4* cache, int T, const int32_t* seqs, const int32_t* positions,
                              void* k_out, void* v_out, void* stream);

/* Grouped-query attention over the cache, S causal query tokens for each of B sequences: a decode step
 * (S = 1) or a short chunk whose keys are already appended. Query head h reads KV head h / 2, scale
 * 1 / sqrt(128), softmax and sums in fp32: keys and values of magnitudes up to 1e25 leave room for them.
 *   q, out    fp32 or bf16 (type) [B][S][16][128], 16-byte aligned
 *   seqs      int32 [B], the cache row of each sequence (negative: padding, its out rows are left as
 *             they were), or NULL: sequence b reads row b
 *   kv_lens   int32 [B], the sequence's keys, those of the S query tokens among them: query s sees the first
 *             kv_lens[b] - (S - 1 - s); a query that sees none gives zeros
 *   max_len   an upper bound of kv_lens (host), at most 64 * blocks_per_seq and 2^30; it sets the split and
 *             the workspace, a tight one is faster. A sequence whose row or key count is out of range is
 *             left as it was; keys behind a page out of range are left out of the sums; both are reported
 *             in cache->err.
 *   workspace at least tts_bb_kv4_attention_workspace(B, S, max_len) bytes, 16-byte aligned (NULL where that is 0);
 *             written before it is read, not shared by calls that overlap
 * Results do not depend on the order in which blocks of the launch run. TTS_BB_E_INVALID also for
 * S > TTS_BB_KV4_MAX_QUERIES or B * S > 65535. */
size_t tts_bb_kv4_attention_workspace(int B, int S, int max_len);
tts_bb_status tts_bb_kv4_attention(const tts_bb_kv4* cache, int B, int S, const void* q, int type, const int32_t* seqs,
                                   const int32_t* kv_lens, int max_len, void* out, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Products with 4-bit weights, y = x W^T for T <= TTS_BB_W4_MAX_TOKENS rows of x: W[n][k] = scale[n][k / group] *
 * (code[n][k] - zero[n][k / group]).
 * tts_bb_w4_pack lays the weights out once (tts_bb_w4_packed_bytes bytes, 16-byte aligned; 0 for
 * sizes that are refused) from
 *   codes   uint8 [N][K / 2]: code 2 i in the low, 2 i + 1 in the high nibble of byte i
 *   scales  bf16 [N][K / group]
 *   zeros   uint8 [N][K / group], 0..15, or NULL: 8 everywhere (above 15: taken modulo 16)
 * group 32, 64 or 128; K a multiple of group, at most 2^18; N at most 2^20. */
#define TTS_BB_W4_MAX_TOKENS 64
size_t tts_bb_w4_packed_bytes(int N, int K, int group);
tts_bb_status tts_bb_w4_pack(int N, int K, int group, const void* codes, const void* scales, const void* zeros,
                             void* packed, void* stream);
/*   x  fp32 or bf16 (type) [T] rows of K, x_stride elements apart (>= K, and 16-byte aligned rows)
 *   y  fp32 or bf16 (the same type) [T][N], 4- or 2-byte aligned
 * A row of x enters to within one fp32 step of each value, or 2^-39 of the row's largest magnitude where that is
 * more; products are exact and summed in fp32, in an order that depends on the sizes alone. An infinity or a NaN
 * in a row of x makes that row of y NaN. */
tts_bb_status tts_bb_w4_linear(int T, int N, int K, int group, const void* x, int type, int64_t x_stride,
                               const void* packed, void* y, void* stream);

/* Log probabilities of R <= 2^27 rows of V <= 2^30 logits: of a given token, the entropy, the log-sum-exp and the n_top most
 * probable tokens.
 *   logits   fp32, bf16 or fp16 (type) [R] rows, row_stride elements apart (>= V), aligned to the element
 *   targets  int32 [R] or NULL; logprob fp32 [R]: log p(targets[r]); -inf for a target outside 0..V-1, a
 *            masked one, or one of logit -inf
 *   allowed  NULL, or uint32 words of 32 ids each (id i: bit i & 31 of word i >> 5; (V + 31) / 32
 *            words a row, allowed_stride words apart, 0 = one row for all): an id whose bit is 0 has
 *            probability 0, whatever its logit
 *   entropy  fp32 [R] (nats); lse fp32 [R]: log of the sum of exp(logit)
 *   top_ids, top_logprobs  int32 and fp32 [R][n_top], 0 <= n_top <= TTS_BB_LOGPROBS_MAX_TOP: by logit
 *            downward, ties to the lowest id; ids of probability 0 are no alternatives: (-1, -inf) behind the last
 * Outputs may be NULL (top_* where n_top is 0, logprob where targets is NULL). A row with nothing left
 * has logprob and lse -inf and entropy 0; an allowed NaN or +inf makes the row's numbers NaN and its
 * ids -1.
 * Slower, with the same results: many rows of up to 96 * 32 logits that hold an allowed one of -inf or beyond 1e30 in
 * magnitude (49152 x 1025: ten times), alternatives of rows whose ids of probability above 0 all lie in one of their parts
 * (64 x 151676, 1500 ids side by side: ten times), and rows of more than 393216 fp32 or 786432 16-bit logits, which
 * a single block reads once more for each alternative. The allowed bits exclude ids at no cost.
 *   workspace  not used: no sizes need one so far, tts_bb_token_logprobs_workspace gives 0 and NULL will do. Callers that
 *            ask and pass what is asked for need no change where that ends */
#define TTS_BB_LOGPROBS_MAX_TOP 32
size_t tts_bb_token_logprobs_workspace(int R, int V, int n_top);
tts_bb_status tts_bb_token_logprobs(int R, int V, const void* logits, int type, int64_t row_stride,
                                    const int32_t* targets, const uint32_t* allowed, int64_t allowed_stride, int n_top,
                                    float* logprob, float* entropy, float* lse, int32_t* top_ids, float* top_logprobs,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Speculative decoding operators: a pass over a tree of drafted tokens for each sequence. tts_bb_tree_attention runs the
 * tree's attention over a paged bf16 cache, tts_bb_tree_verify (or _greedy) finds the path that the target model accepts
 * and the token behind it, tts_bb_tree_commit appends the path's keys and values to the caches of all layers. Drafted
 * keys and values stay in the caller's own arrays until then: a rejected token never owns a place of the cache. The
 * conventions of the low-bit operators hold: the caller's buffers alone, asynchronous on `stream`, no allocation, nothing
 * kept between calls, capturable into a CUDA graph, TTS_BB_E_INVALID before anything is enqueued.
 *
 * A tree has 1 .. N nodes, N <= TTS_BB_TREE_MAX_NODES, B * N <= 65535:
 *   parents  int32 [B][N]: parents[b][i] is a node below i, or -1: a child of the cached context. Node 0 is the pending token
 *            (known, its keys not yet cached). Verification starts there: further nodes of parent -1 are never reached
 *   n_nodes  int32 [B], 0 .. N, or NULL: N each. Nodes behind them are padding, whatever they hold; 0: a padding sequence
 * A sequence of a parent out of order or of n_nodes out of range is skipped (below) and reported. */
#define TTS_BB_TREE_MAX_NODES 64
/* Bits of an error word. */
enum {
    TTS_BB_TREE_ERR_PAGE = 1,  /* a page-table entry outside 0..n_blocks-1 was met */
    TTS_BB_TREE_ERR_RANGE = 2, /* a cache row, a key count, a node count or a position out of range */
    TTS_BB_TREE_ERR_TREE = 4,  /* a parent that is not below its node, or a path's node outside 0..N-1 */
    TTS_BB_TREE_ERR_TIMEOUT = 8 /* a bounded wait inside a kernel ran out: that call's out is undefined */
};
/* A paged bf16 KV cache of n_layers layers: each a pool of blocks [n_blocks][2][8][64][128] (block: K then V of 64 positions
 * for the 8 KV heads, as tts_bb_gqa_decode_attention_static reads it), all under one page table. */
#define TTS_BB_KV_BLOCK_ELEMS 131072
typedef struct {
    void* pool;                /* device bf16, 16-byte aligned: layer 0 */
    const int32_t* page_table; /* device int32 [n_seqs][blocks_per_seq]: block of each 64 positions */
    int32_t* err;              /* device word, or NULL: the bits of what calls skipped are ORed into it */
    int64_t layer_stride;      /* elements from a layer's pool to the next, a multiple of 8 (not used for one layer) */
    int n_layers;
    int n_blocks;              /* at most 2^20 */
    int n_seqs;
    int blocks_per_seq;
} tts_bb_kv_cache;

/* Grouped-query attention of N tree nodes for each of B sequences: node i sees the first kv_lens[b] cached keys, itself and its
 * ancestors. Query head h reads KV head h / 2, scale 1 / sqrt(128), softmax and sums in fp32.
 *   cache, layer  the cache, and which of its layers
 *   q        fp32 or bf16 (type) [B * N] rows of 2048 (16 heads of 128, normed and rotated), q_stride elements apart
 *   k, v     bf16 [B * N] rows of 1024 (8 heads of 128, k normed and rotated): the nodes' own, kv_stride elements apart
 *   out      [B][N][16][128] of the type of q
 *            all rows of q, k, v, out 16-byte aligned; k, v and q may be parts of wider rows
 *   seqs     int32 [B], the cache row of each sequence (negative: padding), or NULL: sequence b reads row b
 *   kv_lens  int32 [B], the sequence's cached keys, 0 .. max_len
 *   max_len  an upper bound of kv_lens (host), 0 .. 64 * blocks_per_seq, at most 2^30, B * max_len at most 2^33; it sets the
 *            split and the workspace, a tight one is faster
 *   workspace at least tts_bb_tree_attention_workspace(B, N, max_len) bytes (20.6 MB at most), 16-byte aligned (NULL where that
 *            is 0); written before it is read, not shared by calls that overlap
 * out and the workspace overlap no input. Rows of out of padding and of skipped sequences are left as they were; keys behind a page out
 * of range are left out of the sums. What masked keys, places behind a sequence's keys and padding nodes hold does not matter, NaN and
 * infinities among it. Where the formula gives NaN or an infinity the number is one of the two; queries and keys of magnitudes up
 * to 1e18 and values up to 1e28 leave fp32 room for scores and sums; an infinite key that a node sees gives bf16 queries what
 * the formula gives, fp32 ones that or NaN. Results do not depend on the order in which blocks of the launch run. */
size_t tts_bb_tree_attention_workspace(int B, int N, int max_len);
tts_bb_status tts_bb_tree_attention(const tts_bb_kv_cache* cache, int layer, int B, int N, const void* q, int type,
                                    int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                    const int32_t* parents, const int32_t* n_nodes, const int32_t* seqs,
                                    const int32_t* kv_lens, int max_len, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* The path of drafted tokens that the target's probabilities accept, by given random numbers, so that the tokens are distributed
 * as the target's own. At node i (first: node 0) with the target's row p and the draft's row q, the children x in the order of
 * their index: r = p, Z = 1 at first; x is accepted where u q(x) Z < r(x), and the walk goes on from it. Else r(y) becomes
 * max(r(y) - Z q(y), 0) for all y, and Z the sum of r. With draft NULL (drafts that were chosen, not drawn, such as the most
 * probable ones): accepted where u Z < r(x), else r(x) becomes 0 and Z loses what it was. Behind the last accepted node the
 * next token is the smallest x where the sum of r(0 .. x) exceeds u_next times the sum of all r; where that is 0, the
 * most probable one of p, the lowest of them.
 *   tokens   int32 [B][N]; a drafted token outside 0..V-1 is no draw: never accepted, r stays
 *   target   fp32 [B * N] rows of V probabilities, target_stride elements apart (>= V): row b N + i holds the target's for
 *            the token behind node i. 0 <= p <= 1, each row's sum near 1 (others, NaN among them: some path of the tree and some
 *            next token in 0..V-1)
 *   draft    fp32, the same for the draft model, draft_stride apart: the distribution from which all children of node i were
 *            drawn, independently of each other; or NULL
 *   u        fp32 [B][N] in [0, 1): node j's number; u_next fp32 [B]
 *   n_accepted int32 [B]: nodes of the path, node 0 among them; 0 for padding and skipped sequences
 *   path     int32 [B][N]: its nodes, -1 behind the last;  next_token int32 [B]: -1 where n_accepted is 0
 *   err      device word, or NULL
 * Masses are held to some 2^-46 of the 1 of a row for each rejected child of a node, whatever their own size (rows beyond 2^24 ids: to
 * a few bits fewer): the answers are those of exact arithmetic but where two masses lie that close to each other. What rejections
 * by a draft next to the target leave may itself be of the size of 2^-25. V at most 2^30, fp32 and int32 arrays 4-byte aligned. Rows of
 * target and draft that begin at different places of 16 bytes are read an id at a time: 64 x 151676 ids, 12 nodes 45 us instead of 40. */
tts_bb_status tts_bb_tree_verify(int B, int N, int V, const int32_t* tokens, const int32_t* parents, const int32_t* n_nodes,
                                 const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                                 const float* u, const float* u_next, int32_t* n_accepted, int32_t* path,
                                 int32_t* next_token, int32_t* err, void* stream);
/* The same for greedy decoding: target_ids int32 [B][N] holds the target's choice behind each node (such as argmax_out); of a
 * node's children the first of that token is accepted, and next_token is the choice behind the last accepted node. */
tts_bb_status tts_bb_tree_verify_greedy(int B, int N, const int32_t* tokens, const int32_t* parents, const int32_t* n_nodes,
                                        const int32_t* target_ids, int32_t* n_accepted, int32_t* path, int32_t* next_token,
                                        int32_t* err, void* stream);

/* Append the accepted paths to the caches of all layers: node path[b][j] of sequence b becomes position kv_lens[b] + j of its cache
 * row, for j < n_accepted[b].
 *   k, v     bf16 [n_layers][B * N] rows of 1024 as tts_bb_tree_attention takes them, rows row_stride and layers layer_stride
 *            elements apart, every row 16-byte aligned; not a part of the cache
 *   path, n_accepted  as tts_bb_tree_verify gives them (0: nothing is appended)
 *   seqs, kv_lens     as in tts_bb_tree_attention. kv_lens is not changed: adding n_accepted to it is the caller's
 * The rows of one call must differ. Tokens whose position, page or node is out of range are skipped, as is a sequence whose
 * row, key count or n_accepted is, and reported in cache->err. */
tts_bb_status tts_bb_tree_commit(const tts_bb_kv_cache* cache, int B, int N, const void* k, const void* v, int64_t row_stride,
                                 int64_t layer_stride, const int32_t* path, const int32_t* n_accepted, const int32_t* seqs,
                                 const int32_t* kv_lens, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TTS_BB_H */
