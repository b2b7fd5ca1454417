/*
 * rrq.h — random-rotation vector quantisation for KV-cache and embedding vectors
 * on NVIDIA B200 (sm_100a).  C ABI of librrq.so.
 *
 * The method ("Random-rotation quantization" page, brain.bigb.es, intro "the
 * scheme", steps 1–3): rotate each vector by a random orthogonal Π, quantise
 * every rotated coordinate independently with one fixed codebook computed once
 * for the post-rotation marginal, and at decode time dequantise and apply Πᵀ.
 * Π is the randomized Hadamard transform (section "Why rotation works";
 * "TurboQuant and per-layer outlier-aware K" page, section "TurboQuant 2026":
 * the FWHT):
 *
 *     Π = H·D/√d,  D = diag(s_0 .. s_{d-1}),  s_i = ±1,
 *     H = Sylvester–Hadamard matrix of order d in natural order,
 *     H_ij = (−1)^popcount(i & j).
 *
 * s_i = −1 exactly when bit 63 of SplitMix64 output number i is set, where
 * output c of a generator seeded with `seed` is mix(seed + (c+1)·0x9E3779B97F4A7C15)
 * (Steele, Lea & Flood 2014).  One D per call, shared by every vector.
 *
 * Common conventions
 * ------------------
 *  - Every data pointer is a DEVICE pointer owned by the caller, except where
 *    an argument says "host".  The library allocates no device memory and
 *    keeps no per-call state; it never synchronises the stream.
 *  - Every call is asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL = the legacy default stream).  Inputs and outputs must not alias.
 *  - Vectors are rows of a dense row-major [n × d] array; a KV tensor
 *    [tokens × heads × d] is n = tokens·heads rows, row t·heads + h.
 *  - d is a power of two in [64, 512]; bits in 1..4; n ≥ 0 (n = 0 is a
 *    no-op returning RRQ_OK).
 *  - Vector and code arrays must be 32-byte aligned (the kernels move whole
 *    32-byte sectors); norm arrays 4-byte; other alignments are stated per
 *    entry point.
 *  - Element types: RRQ_F32 (float), RRQ_F16 (IEEE binary16), RRQ_BF16.
 *  - Arguments are validated before any launch; an invalid call returns
 *    RRQ_ERR_INVALID and touches no memory.  A failed launch returns
 *    RRQ_ERR_CUDA.  Non-finite inputs give unspecified codes (no fault).
 *  - fp32 / bf16 inputs need 1e-18 < ‖x‖₂ < 1e18 (the squared norm is
 *    accumulated in fp32); fp16 inputs have no range restriction.
 *
 * Codebook (`codebook` arguments)
 * -------------------------------
 *  A HOST pointer to 2^bits strictly ascending finite floats, copied by value
 *  at the call, or NULL for the Lloyd–Max codebook of N(0,1) ("Random-rotation
 *  quantization" page, section "History", EDEN bullet: 1-bit ±√(2/π),
 *  2-bit ±0.453, ±1.510).  Decision thresholds are the midpoints
 *  τ_k = (c_k + c_{k+1})/2 (nearest-centroid cells; section "Three decoders,
 *  one rotation", MSE decoder).  A codebook that is exactly symmetric
 *  (c_k = −c_{L−1−k}) takes a faster path; any ascending codebook is accepted.
 *
 * Packed code format (RRQ_FORMAT_VERSION 1)
 * -----------------------------------------
 *  Per vector d·bits/8 bytes; coordinate i occupies bits [i·bits, (i+1)·bits)
 *  of the byte string, least significant bit first (bits = 4: coordinate 2j
 *  in the low nibble of byte j).  Code k means level c_k (code 0 = most
 *  negative).  The per-vector scale is a separate fp32 array: ν = ‖x‖₂.
 */
#ifndef RRQ_H
#define RRQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RRQ_FORMAT_VERSION 1

/* status codes */
#define RRQ_OK 0
#define RRQ_ERR_INVALID 1     /* bad argument, detected before any launch       */
#define RRQ_ERR_CUDA 2        /* a CUDA launch or runtime call failed           */
#define RRQ_ERR_UNSUPPORTED 3 /* valid request the library does not implement  */
#define RRQ_ERR_SCRATCH 4     /* request larger than the fixed scratch of
                                 rrq_attention_decode_noalloc                   */

/* element types */
#define RRQ_F32 0
#define RRQ_F16 1
#define RRQ_BF16 2

/* GGML block types for rrq_ggml_rot (the numbers of ggml's own type enumeration) */
#define RRQ_GGML_Q4_0 2
#define RRQ_GGML_Q4_1 3
#define RRQ_GGML_Q5_0 6
#define RRQ_GGML_Q5_1 7
#define RRQ_GGML_Q8_0 8

/* Packed-format version this library writes and reads. */
int rrq_format_version(void);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* rrq_strerror(int status);

/*
 * rrq_codebook — the default codebook: ascending Lloyd–Max levels for N(0,1).
 * "Random-rotation quantization" page, section "History", EDEN bullet.
 * Computed on the host in double by Lloyd's iteration (centroid of each
 * nearest-level cell under the normal density, thresholds at midpoints) and
 * rounded to float; exactly symmetric.
 *   bits    1..4
 *   levels  HOST, float[2^bits], written in ascending order
 * Returns RRQ_OK or RRQ_ERR_INVALID.  Thread-safe; no CUDA call.
 */
int rrq_codebook(int bits, float* levels);

/*
 * rrq_rotate — y = Πx (inverse = 0) or y = Πᵀx (inverse = 1), fp32 output.
 * "Random-rotation quantization" page, scheme steps 1 and 3, and section
 * "Why rotation works" (randomized Hadamard transform).
 *   x      [n × d] of x_dtype
 *   y      [n × d] float
 * Errors: RRQ_ERR_INVALID (d, dtype, n, null or misaligned pointer),
 * RRQ_ERR_CUDA.
 */
int rrq_rotate(const void* x, int x_dtype, int64_t n, int d, uint64_t seed, int inverse,
               float* y, void* stream);

/*
 * rrq_encode — quantise n vectors.
 * "Random-rotation quantization" page: scheme steps 1–2; "History", EDEN
 * bullet (normalise to ≈N(0,1), Lloyd–Max codebook) and TurboQuant bullet
 * (constant per-vector scale); "Three decoders, one rotation", MSE decoder.
 * For each vector x:
 *     ν = ‖x‖₂,  u = √d·Πx/ν  (u = 0 when ν = 0),
 *     code_i = #{k : u_i > τ_k}   (a value on a threshold takes the lower code),
 * codes are packed as described above and ν is stored as fp32.
 *
 * Optional QJL stage ("History", QJL and TurboQuant bullets: a 1-bit sign
 * sketch of the residual makes inner products unbiased; "Bias vs
 * unbiasedness"): when qjl_S is non-NULL, also
 *     r = Πx − ŷ,  ŷ = (ν/√d)·c[code]  (the decoder's rotated-domain value),
 *     qjl_bits bit i = [ (S·r)_i > 0 ],  qjl_rnorm = ‖r‖₂,
 * with S the d×d matrix at qjl_S (bf16, row-major, see rrq_qjl_matrix).
 * The product S·r runs on the tensor cores (tcgen05): for fp32 x with r split
 * exactly into three bf16 parts (an fp32-accurate product); for 16-bit x with
 * r scaled by a power of two and split into two fp16 parts and S rounded to
 * fp16 (the sign of an output can differ only where |(S·r)_i| < 1e-5·‖r‖₂).
 *   x          [n × d] of x_dtype
 *   codes      [n × d·bits/8] bytes (output)
 *   norms      [n] float (output)
 *   qjl_S      bf16 [d × d] or NULL (no QJL; then qjl_bits/qjl_rnorm ignored)
 *   qjl_bits   [n × d/8] bytes (output, with qjl_S)
 *   qjl_rnorm  [n] float (output, with qjl_S)
 * Errors: RRQ_ERR_INVALID (bad d / bits / dtype / codebook, null or
 * misaligned pointer), RRQ_ERR_UNSUPPORTED (QJL with d other than 128),
 * RRQ_ERR_CUDA.
 */
int rrq_encode(const void* x, int x_dtype, int64_t n, int d, int bits, uint64_t seed,
               const float* codebook, uint8_t* codes, float* norms,
               const uint16_t* qjl_S, uint8_t* qjl_bits, float* qjl_rnorm, void* stream);

/*
 * rrq_decode — reconstruct n vectors from codes and norms.
 * "Random-rotation quantization" page, scheme step 3 and "Three decoders,
 * one rotation", MSE decoder:
 *     ŷ_i = (ν/√d)·c[code_i],   x̂ = Πᵀŷ = (ν/d)·D·H·c[code],
 * computed in fp32 and rounded to out_dtype (round to nearest even).
 *   codes  [n × d·bits/8] bytes;  norms [n] float
 *   out    [n × d] of out_dtype
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_CUDA.
 */
int rrq_decode(const uint8_t* codes, const float* norms, int64_t n, int d, int bits,
               uint64_t seed, const float* codebook, void* out, int out_dtype, void* stream);

/*
 * rrq_drive_encode — DRIVE's one-bit encoder.
 * "Random-rotation quantization" page, "History", DRIVE bullet (one bit per
 * coordinate, sign(R(x)), plus one scale; ‖R(x)‖₁/d is the biased, MSE-optimal
 * choice and ‖x‖₂²/‖R(x)‖₁ the unbiased one), and "Three decoders, one
 * rotation", mean decoder x̂ = S·Πᵀ·sign(Πx).  For each vector x:
 *     bit_i = [ (Πx)_i > 0 ]   (0 decodes to −1, 1 to +1),
 *     S = ‖Πx‖₁/d (unbiased = 0) or ‖x‖₂²/‖Πx‖₁ (unbiased = 1; 0 when x = 0),
 *     scales = fp32(S·√d).
 * Bits are packed as rrq_encode's one-bit codes, and the stored value is what
 * rrq_decode and rrq_qk_scores read as the norm, so rrq_decode(bits = 1,
 * codebook {−1, +1}) returns S·Πᵀ·sign(Πx) and rrq_qk_scores with the same
 * codebook returns scale·S·⟨Πq, sign(Πx)⟩.
 *   x       [n × d] of x_dtype
 *   codes   [n × d/8] bytes (output);  scales [n] float (output)
 * Errors: RRQ_ERR_INVALID (d, dtype, unbiased not 0/1, null or misaligned
 * pointer), RRQ_ERR_CUDA.
 */
int rrq_drive_encode(const void* x, int x_dtype, int64_t n, int d, uint64_t seed, int unbiased,
                     uint8_t* codes, float* scales, void* stream);

/*
 * rrq_qk_scores — decode-time attention scores against a quantised K cache,
 * without decoding it.  "Random-rotation quantization" page, "Three decoders,
 * one rotation", inner-product decoder: <q, x> is recovered from <Πq, code(Πx)>
 * and a normalising scalar.  With q' = Πq (rotated once per call):
 *     scores[h][t] = scale · (ν_{t,g}/√d) · Σ_i q'_{h,i} · c[code_{t,g,i}]
 *                  = scale · <q_h, x̂_{t,g}>,    g = ⌊h·hkv/hq⌋ (GQA groups).
 *   q       [hq × d] half (unrotated query heads)
 *   codes   [T·hkv × d·bits/8] bytes, row t·hkv + g;  norms [T·hkv] float
 *   scores  [hq × T] float (output)
 * hq must be a multiple of hkv with hq/hkv in {1, 2, 4, 8}.
 * Accuracy: fp16 query values (each head scaled by a power of two) times fp16
 * levels, summed in fp32 (tensor-core tiles for 4-bit codes at d ≤ 128, fp16 pairs
 * with fp32 partial sums otherwise); the error is far below 1e-3·‖q‖·‖x̂‖ for
 * bits ≤ 4.
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_UNSUPPORTED (group size), RRQ_ERR_CUDA.
 */
int rrq_qk_scores(const void* q, int hq, const uint8_t* codes, const float* norms, int64_t T,
                  int hkv, int d, int bits, uint64_t seed, const float* codebook, float scale,
                  float* scores, void* stream);

/*
 * rrq_qk_scores_qjl — unbiased decode-time attention scores on keys stored as
 * b-bit MSE codes plus the QJL one-bit residual sketch (rrq_encode with qjl_S).
 * "Random-rotation quantization" page: "History", TurboQuant bullet (a biased
 * MSE quantiser followed by an unbiased one-bit stage on the residual) and QJL
 * bullet; "Three decoders, one rotation", inner-product decoder; "Bias vs
 * unbiasedness".  With g = ⌊h·hkv/hq⌋:
 *     scores[h][t] = scale · ( <q_h, x̂_{t,g}>
 *                              + √(π/2)/d · ρ_{t,g} · <S·Π·q_h, sign_{t,g}> ),
 * x̂ the b-bit MSE reconstruction (as rrq_qk_scores), sign_i = +1 where QJL bit i
 * is set and −1 elsewhere, ρ the stored residual norm.  Averaged over the
 * Gaussian S the score is unbiased for scale·<q_h, x_{t,g}>.
 *   q          [hq × d] fp16 (unrotated)
 *   codes      [T·hkv × d·bits/8] bytes, row t·hkv + g;  norms [T·hkv] float
 *   qjl_bits   [T·hkv × d/8] bytes;  qjl_rnorm [T·hkv] float (as rrq_encode writes)
 *   qjl_S      bf16 [d × d] (the S given to rrq_encode)
 *   scores     [hq × T] float (output)
 * d must be 128; hq a multiple of hkv with hq/hkv in {1, 2, 4, 8}.
 * Accuracy: both dot products as fp16 × fp16 products summed in fp32 (tensor-core
 * tiles), each head's query and projected query scaled by a power of two.
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_UNSUPPORTED (d other than 128, group size),
 * RRQ_ERR_CUDA.
 */
int rrq_qk_scores_qjl(const void* q, int hq, const uint8_t* codes, const float* norms,
                      const uint8_t* qjl_bits, const float* qjl_rnorm, const uint16_t* qjl_S,
                      int64_t T, int hkv, int d, int bits, uint64_t seed, const float* codebook,
                      float scale, float* scores, void* stream);

/*
 * rrq_attention_decode — one decode step of attention over a quantised K/V cache.
 * "Attn-rot (TurboQuant lite) in llama.cpp" page, "What kind of beast is
 * Attn-rot" (keys and values both quantised after a rotation);
 * "Random-rotation quantization" page, "Three decoders, one rotation" (the MSE
 * decoder is the one for KV-cache compression).  With g = ⌊h·hkv/hq⌋:
 *     s[h][t] = scale · <q_h, k̂_{t,g}>         (as rrq_qk_scores, K codebook and seed),
 *     p[h][t] = exp(s[h][t] − max_t s[h][·]) / Σ_t exp(s[h][t] − max_t s[h][·]),
 *     out[h]  = Σ_t p[h][t] · v̂_{t,g}          (v̂ as rrq_decode, V codebook and seed).
 * The values are summed in their rotated domain and rotated back once per head.
 *   q          [hq × d] fp16
 *   k_codes    [T·hkv × d·k_bits/8] bytes, row t·hkv + g;  k_norms [T·hkv] float
 *   v_codes    [T·hkv × d·v_bits/8] bytes;                 v_norms [T·hkv] float
 *   k_codebook, v_codebook: HOST float[2^bits] or NULL (the default codebook)
 *   workspace  device scratch of workspace_bytes ≥ rrq_attention_workspace_bytes(
 *              hq, hkv, d, k_bits, v_bits, T), 256-byte aligned, owned by the caller,
 *              and ZERO before its first use: each call leaves its counters at zero
 *              again.  Calls that share a workspace must not overlap on the GPU.
 *   out        [hq × d] float (output)
 * d ∈ {64, 128, 256, 512}, K and V codes of 1 to 4 bits; hq a multiple of hkv
 * with hq/hkv in {1, 2, 4, 8} (at most 4 for d = 512); T ≥ 1.  Scores as
 * rrq_qk_scores (fp16 operands, fp32 sums); softmax in fp32.  d = 128 with 4-bit
 * K and V runs as one fused kernel whose value sums take fp16 levels and fp16
 * weights with fp32 accumulation; the weights are p·ν relative to the largest
 * p·ν of the head (exponent and log2 ν added before the one exponential), so any
 * finite value norm keeps its precision.  Every other shape writes the scores
 * to the workspace (hq × T floats) and sums the values in fp32.  Either way, per
 * head the output is within 2e-3·Σ_t p_t·‖v̂_t‖ of the exact softmax-weighted sum
 * of the reconstructions.
 * Errors: RRQ_ERR_INVALID (incl. a workspace that is too small), RRQ_ERR_UNSUPPORTED
 * (d, bits, group size; for d = 128 with 4-bit codes also a device whose
 * per-block reserved shared memory is not the 1 KB the fused kernel's shared
 * layout assumes), RRQ_ERR_CUDA.
 */
int rrq_attention_decode(const void* q, int hq, const uint8_t* k_codes, const float* k_norms,
                         const uint8_t* v_codes, const float* v_norms, int64_t T, int hkv, int d,
                         int k_bits, uint64_t k_seed, const float* k_codebook, int v_bits,
                         uint64_t v_seed, const float* v_codebook, float scale, void* workspace,
                         size_t workspace_bytes, float* out, void* stream);

/*
 * rrq_attention_decode_noalloc — rrq_attention_decode without a workspace argument
 * and without allocating anything.  The pages have no counterpart: this entry is
 * for callers that cannot allocate device memory at the point of the call, such
 * as a serving loop whose memory is reserved up front by its own allocator (a
 * cudaMalloc there would synchronise the device and fragment the pool) or code
 * deep in a call chain that has no workspace to pass down.
 * Its scratch is a fixed 4 MiB array inside the library's device image, so every
 * GPU that loads the library holds those 4 MiB until the process exits.  Requests
 * whose workspace (rrq_attention_workspace_bytes) exceeds 4 MiB are rejected with
 * RRQ_ERR_SCRATCH before anything is launched.
 * The first call on a device looks up the array's address on that device (once)
 * and keeps it for the life of the process; make that first call before any
 * stream capture.  A cudaDeviceReset() of that device invalidates the kept
 * address: do not call this entry on a device after resetting it.  Each call clears the array's
 * counters on `stream` before its kernel runs.  All calls share the one array:
 * calls whose GPU work overlaps (other streams, other host threads) race and
 * give wrong results; calls ordered on one stream are safe.
 * Arguments, outputs and the other errors as rrq_attention_decode.
 */
int rrq_attention_decode_noalloc(const void* q, int hq, const uint8_t* k_codes,
                                 const float* k_norms, const uint8_t* v_codes,
                                 const float* v_norms, int64_t T, int hkv, int d, int k_bits,
                                 uint64_t k_seed, const float* k_codebook, int v_bits,
                                 uint64_t v_seed, const float* v_codebook, float scale,
                                 float* out, void* stream);

/*
 * rrq_attention_workspace_bytes — the workspace rrq_attention_decode needs for
 * (hq, hkv, d, k_bits, v_bits, T) on the current device (it depends on the SM
 * count and, for the shapes other than d = 128 with 4-bit K and V, on how many
 * CTAs of the value kernel for that d and V width one SM holds), or 0 for an
 * invalid shape.  d = 128 with 4-bit K and V needs the counters and partial
 * states only (well under 1 MB for 32 query heads); every other shape adds
 * hq × T floats of scores.  No CUDA work beyond reading the device's attributes
 * and the kernels' occupancy.
 */
size_t rrq_attention_workspace_bytes(int hq, int hkv, int d, int k_bits, int v_bits, int64_t T);

/*
 * rrq_attention_shared — one decode step of attention for a batch of sequences
 * that share a quantised prefix, each followed by a quantised tail of its own.
 * The pages define the quantised cache ("Attn-rot (TurboQuant lite) in llama.cpp"
 * page, "What kind of beast is Attn-rot": K and V both quantised after a rotation;
 * "Random-rotation quantization" page, "Three decoders, one rotation": the MSE
 * decoder); serving a batch from it is this library's addition.  For sequence b and
 * query head h, g = ⌊h·hkv/hq⌋, over the tokens t of the prefix and then of the
 * first n_b = tail_lens[b] rows of tail b:
 *     s[t] = scale · <q_{b,h}, k̂_{t,g}>,   p = softmax(s),   out_{b,h} = Σ_t p[t]·v̂_{t,g},
 * k̂ and v̂ as rrq_decode.  The prefix is read and dequantised once for every 128 query rows
 * (sequences × heads per kv head; for d = 512, a plain kernel, it is dequantised once for
 * every 8).  A sequence without any token (no prefix and n_b = 0) gets zeros.
 *   q           [batch × hq × d] of q_dtype (RRQ_F16 or RRQ_BF16), unrotated
 *   pk_codes    [prefix·hkv × d·k_bits/8] bytes, row t·hkv + g;  pk_norms [prefix·hkv]
 *   pv_codes    [prefix·hkv × d·v_bits/8] bytes;                 pv_norms [prefix·hkv]
 *   tk_codes    [batch·tail_cap·hkv × d·k_bits/8] bytes, row (b·tail_cap + t)·hkv + g;
 *   tk_norms, tv_codes, tv_norms likewise
 *   tail_lens   [batch] int32 on the device, read by the kernels: values outside
 *               [0, tail_cap] count as the nearer end.  Rows behind n_b do not count,
 *               whatever they hold.
 *   workspace   device scratch of workspace_bytes ≥ rrq_attention_shared_workspace_bytes(
 *               batch, hq, hkv, d, prefix, tail_cap), 256-byte aligned, of any content.
 *               Calls that share a workspace must not overlap on the GPU (also where
 *               they were captured into graphs).
 *   out         [batch × hq × d] of q_dtype (output)
 * prefix ≥ 0 and tail_cap ≥ 0; the arrays of a part of size 0 (and tail_lens with
 * tail_cap = 0) may be NULL.  batch = 0 is a no-op.  d ∈ {64, 128, 256, 512}, 1- to
 * 4-bit K and V; hq a multiple of hkv, at most 128 query heads per kv head.
 * Alignment: codes, q and out 16 bytes, norms and tail_lens 4.
 * Accuracy: softmax statistics, sums and the rotations in fp32 (all of it for d = 512).  For
 * d ≤ 256 both products run on the tensor cores with fp16 operands and fp32 sums:
 *  - the weights p_t·‖v̂_t‖, relative to the largest of their head: 11 bits down to 2^-18 of
 *    it, within 2^-29 of it below, whatever p_t and ‖v̂_t‖ are on their own (value norms below
 *    2^-90 lose precision, and weights p_t below 2^-90 of the largest may count as zero);
 *  - the levels of a codebook: 11 bits within 2^-14 of its largest, within 2^-25 of that
 *    below; the default ones of 1 to 3 bits to 2^-14 of themselves or better, of 4 bits to
 *    3.8e-5 on average;
 *  - the rotated queries: 22 bits.
 * A score is therefore off by at most 2^-11·scale·‖q‖·‖k̂_t‖, and √d times less on average, all
 * but 2^-11 of it from the key levels.  While the scores' errors stay below 5e-4, and no more
 * than 2^18 tokens of a head have weights below 2^-18 of its largest, the output of a head is
 * within 2e-3·Σ_t p_t·‖v̂_t‖ of the exact one before it is rounded to q_dtype.
 * Errors: RRQ_ERR_INVALID (incl. a workspace that is too small), RRQ_ERR_UNSUPPORTED
 * (q_dtype RRQ_F32, more than 128 heads per kv head, 2^31 − 128 or more tokens in the
 * prefix or over all tails, 10^8 or more tiles of 64 or 128 tokens over all units of work,
 * or a device whose per-block reserved shared memory is not the 1 KB that the tensor-core
 * kernel's layout assumes), RRQ_ERR_CUDA.
 */
int rrq_attention_shared(const void* q, int q_dtype, int64_t batch, int hq,
                         const uint8_t* pk_codes, const float* pk_norms, const uint8_t* pv_codes,
                         const float* pv_norms, int64_t prefix, const uint8_t* tk_codes,
                         const float* tk_norms, const uint8_t* tv_codes, const float* tv_norms,
                         int64_t tail_cap, const int32_t* tail_lens, int hkv, int d, int k_bits,
                         uint64_t k_seed, const float* k_codebook, int v_bits, uint64_t v_seed,
                         const float* v_codebook, float scale, void* workspace,
                         size_t workspace_bytes, void* out, void* stream);

/*
 * rrq_attention_shared_workspace_bytes — the workspace rrq_attention_shared needs
 * on the current device (it depends on the SM count), or 0 for an invalid or
 * unsupported shape.  It grows with batch, hq and d, and with prefix and tail_cap
 * only until every SM has work.
 */
size_t rrq_attention_shared_workspace_bytes(int64_t batch, int hq, int hkv, int d, int64_t prefix,
                                            int64_t tail_cap);

/*
 * rrq_attention_mass — the attention weight that every cached token has drawn so
 * far, from a decode step's scores (rrq_qk_scores, rrq_qk_scores_qjl): what
 * rrq_evict keeps tokens by.  Not on the pages.  With p = softmax of a head's
 * scores over the tokens t < n_b = lens[b]:
 *     out[b][g][t] = decay · mass[b][g][t] + Σ_{h in group g} p[b][h][t],   t < n_b,
 *     out[b][g][t] = mass[b][g][t],                                        t ≥ n_b.
 * The weights are those among the tokens whose scores are given.  For a sequence behind a
 * shared prefix pass the scores of prefix and tail together: with the tail's alone the
 * weights of its tokens add up to 1 per head, whatever the prefix draws.
 * A score of −inf masks its token (weight 0); a head whose scores are all −inf adds
 * nothing.  +inf and NaN scores give unspecified values for the tokens of their
 * kv head (no fault).
 *   scores  [batch × hq × T] float
 *   lens    [batch] int32 on the device, or NULL (all T tokens); values outside
 *           [0, T] count as the nearer end
 *   mass    [batch × hkv × T] float, or NULL (zeros);  out may be the same array
 *   out     [batch × hkv × T] float (output)
 * hq a multiple of hkv, at most 1024 query heads per kv head.  batch = 0 or T = 0 is a
 * no-op.  T < 2^31, batch·hkv ≤ 2^27.  Arrays 4-byte aligned (16-byte vectors are used where addresses and T allow).  fp32 throughout;
 * the result does not depend on the order in which the GPU runs blocks.
 * Errors: RRQ_ERR_INVALID (incl. a decay that is not finite), RRQ_ERR_UNSUPPORTED (more
 * than 1024 query heads per kv head), RRQ_ERR_CUDA.
 */
int rrq_attention_mass(const float* scores, int64_t batch, int hq, int hkv, int64_t T,
                       const int32_t* lens, float decay, const float* mass, float* out,
                       void* stream);

/*
 * rrq_evict — cut every sequence of a quantised cache back to at most `keep` tokens
 * per kv head: the first `sink` tokens and the last `recent` ones stay, the others
 * by the largest mass (rrq_attention_mass), equal masses in favour of the lower
 * token.  Not on the pages.  The kept rows move, in their order, to the front of
 * another cache; each kv head keeps tokens of its own.  With n_b = lens[b]:
 *     m_b = min(n_b, keep) → out_lens[b];
 *     index[b][g][s] = the s-th kept token (ascending), s < m_b;
 *     row (b·keep + s)·hkv + g of the output cache = row (b·cap + index[b][g][s])·hkv + g;
 *     out_mass[b][g][s] = mass[b][g][index[b][g][s]].
 * Entries s ≥ m_b of every output are left as they were.  The new cache's capacity is keep: a
 * full one has no room for a next token.  To evict into caches of more tokens, call once
 * per sequence (batch = 1) with the beginning of that sequence's cache as the output.
 *   mass      [batch × hkv × cap] float (a NaN counts as less than −inf, −0 as +0)
 *   lens      [batch] int32 on the device, or NULL (all cap tokens); values outside
 *             [0, cap] count as the nearer end
 *   k_codes   [batch·cap·hkv × d·k_bits/8] bytes;  k_norms [batch·cap·hkv] float;
 *   v_codes, v_norms likewise
 *   index     [batch × hkv × keep] int32;  out_lens [batch] int32;
 *   out_mass  [batch × hkv × keep] float, or NULL;
 *   ok_codes, ok_norms, ov_codes, ov_norms: the output cache of capacity keep
 * Inputs and outputs must not overlap.  keep ≥ 1, sink, recent ≥ 0 with
 * sink + recent ≤ keep; cap < 2^31, batch·hkv ≤ 2^27.  batch = 0 or cap = 0: out_lens is set to 0 for
 * every sequence, nothing else is written.  Alignment: codes 16 bytes, the rest 4.
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_CUDA.
 */
int rrq_evict(const float* mass, int64_t batch, int hkv, int64_t cap, const int32_t* lens,
              int64_t keep, int64_t sink, int64_t recent, int d, int k_bits, int v_bits,
              const uint8_t* k_codes, const float* k_norms, const uint8_t* v_codes,
              const float* v_norms, int32_t* index, int32_t* out_lens, float* out_mass,
              uint8_t* ok_codes, float* ok_norms, uint8_t* ov_codes, float* ov_norms, void* stream);

/* frequency schedules of rrq_rope_frequencies */
#define RRQ_ROPE_NONE 0
#define RRQ_ROPE_LINEAR 1
#define RRQ_ROPE_NTK 2
#define RRQ_ROPE_YARN 3

/*
 * rrq_rope_frequencies — rotary frequencies for rrq_rope, on the HOST, in double.
 * Not on the pages.  For the pair i < rot/2 the unscaled frequency is
 * θ_i = base^(−2i/rot) radians per position, and with the stretch f ≥ 1:
 *   RRQ_ROPE_NONE    θ_i
 *   RRQ_ROPE_LINEAR  θ_i / f (positions interpolated)
 *   RRQ_ROPE_NTK     (base·f^(rot/(rot−2)))^(−2i/rot) (θ_i for rot = 2)
 *   RRQ_ROPE_YARN    θ_i·(1 − r_i) + θ_i/f·r_i, where r_i rises linearly from 0 at the
 *                    pair that turns `fast` times over `original` positions to 1 at
 *                    the pair that turns `slow` times: r_i = clamp((i − lo)/(hi − lo), 0, 1),
 *                    lo = max(⌊c(fast)⌋, 0), hi = min(⌈c(slow)⌉, rot − 1), hi − lo at least
 *                    0.001, c(n) = rot·ln(original/(2πn))/(2 ln base)
 * *factor is the factor on cos and sin: 0.1·ln f + 1 for YARN, else 1.
 *   freqs   HOST, double[rot/2] (output);  factor HOST, double (output)
 * rot even in [2, 512]; base > 1 and stretch ≥ 1 finite; for YARN original > 0 and
 * fast ≥ slow > 0, finite.  Errors: RRQ_ERR_INVALID.  Thread-safe; no CUDA call.
 */
int rrq_rope_frequencies(int schedule, int rot, double base, double stretch, double original,
                         double fast, double slow, double* freqs, double* factor);

/*
 * rrq_rope — rotary positions of queries and keys, before rrq_encode and the scores.
 * Not on the pages.  Vector x of a token at position p: for the pair i < rot/2,
 * (a, b) = (x_i, x_{i + rot/2}) (interleaved = 0) or (x_{2i}, x_{2i+1}) (interleaved = 1),
 *     (a', b') = factor · (a·cos φ − b·sin φ, a·sin φ + b·cos φ),   φ = p·freqs[i],
 * and coordinates from rot on are copied.  inverse = 1 takes −φ: the transposed map,
 * which is also the gradient with respect to x.
 * The angle is formed as p times the frequency in turns as a 64-bit fixed-point
 * fraction, modulo one turn, and cut to 32 bits: within 2^-32 + |p|·2^-65 turns of the
 * exact one.  Products in fp32, rounded once to dtype.
 *   x          [n × heads × d] of dtype;  y the same (output), which may be x itself
 *   positions  [n] int64 on the device, of any sign
 *   freqs      HOST, double[rot/2], finite, |freqs| < 2^31
 * d ∈ {64, 128, 256, 512}; rot even in [2, d]; heads ≥ 1; n = 0 is a no-op.  Alignment:
 * x and y 16 bytes, positions 8.
 * Errors: RRQ_ERR_INVALID (incl. a factor that is not finite), RRQ_ERR_CUDA.
 */
int rrq_rope(const void* x, int dtype, int64_t n, int heads, int d, int rot, int interleaved,
             const int64_t* positions, const double* freqs, double factor, int inverse, void* y,
             void* stream);

/*
 * rrq_q4_0_rot — "Attn-rot" (TurboQuant lite): rotate, then q4_0.
 * "Attn-rot (TurboQuant lite) in llama.cpp" page: rotate K/V before an
 * ordinary block format, q4_0 first of all.  With y = Πx (rotate = 1) or
 * y = x (rotate = 0), per block of 32 consecutive coordinates:
 *     m = the element of largest |y| (first on ties), Δ = m/−8 (fp32),
 *     q_j = min(15, ⌊fp32(fp32(y_j·inv) + 8.5)⌋),  inv = fp32(1/Δ) (0 when Δ = 0),
 * stored as 18 bytes: fp16(Δ) little endian, then byte j = q_j | q_{j+16}<<4
 * (the public llama.cpp q4_0 block, kept identical for interoperability).
 *   x       [n × d] of x_dtype (d a multiple of 32 within [64, 512])
 *   blocks  [n × d/32 × 18] bytes (output; 16-byte aligned)
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_CUDA.
 */
int rrq_q4_0_rot(const void* x, int x_dtype, int64_t n, int d, uint64_t seed, int rotate,
                 void* blocks, void* stream);

/*
 * rrq_q4_0_rot_decode — inverse of rrq_q4_0_rot: ŷ_j = (q_j − 8)·fp16(Δ), then
 * x̂ = Πᵀŷ when rotate = 1; fp32 arithmetic, rounded to out_dtype.
 *   blocks  [n × d/32 × 18] bytes;  out [n × d] of out_dtype
 */
int rrq_q4_0_rot_decode(const void* blocks, int64_t n, int d, uint64_t seed, int rotate,
                        void* out, int out_dtype, void* stream);

/*
 * rrq_ggml_block_bytes — bytes of one block of 32 values of a GGML block type:
 * 18 (q4_0), 20 (q4_1), 22 (q5_0), 24 (q5_1), 34 (q8_0); 0 for any other type.
 */
int rrq_ggml_block_bytes(int type);

/*
 * rrq_ggml_rot — "Attn-rot" with any of the GGML block types the page lists:
 * rotate (rotate = 1: y = Πx, orthonormal; rotate = 0: y = x), then blocks of 32.
 * "Attn-rot (TurboQuant lite) in llama.cpp" page, "How to use it": q4_0 first of
 * all, also q4_1, q5_0, q5_1 (and q8_0).  The page names the types without
 * defining them; the public llama.cpp blocks are used, kept identical for
 * interoperability, with every decision in fp32 (y rounded to fp32, each
 * product, sum and quotient rounded, no fused multiply-add), inv = fp32(1/Δ),
 * 0 when Δ = 0:
 *   q4_0  as rrq_q4_0_rot (18 bytes);
 *   q4_1  lo, hi = first min / max in index order, Δ = (hi − lo)/15,
 *         q_j = min(15, ⌊(y_j − lo)·inv + 0.5⌋); 20 bytes: fp16 Δ, fp16 lo, then
 *         byte j = q_j | q_{j+16} << 4;
 *   q5_0  m = first element of largest |y| (+0 for a block of zeros), Δ = m/−16,
 *         q_j = min(31, ⌊y_j·inv + 16.5⌋); 22 bytes: fp16 Δ, a little-endian
 *         32-bit word whose bit j is bit 4 of q_j, then byte j = (q_j & 15) |
 *         (q_{j+16} & 15) << 4;
 *   q5_1  as q4_1 with Δ = (hi − lo)/31 and no clamp; 24 bytes: fp16 Δ, fp16 lo,
 *         the high-bit word, the nibble bytes;
 *   q8_0  Δ = max|y|/127, q_j = round(y_j·inv) (halves away from zero); 34
 *         bytes: fp16 Δ, then q_j as signed bytes.
 *   x       [n × d] of x_dtype (d in {64, 128, 256, 512})
 *   type    RRQ_GGML_Q4_0 / _Q4_1 / _Q5_0 / _Q5_1 / _Q8_0
 *   blocks  [n × d/32 × rrq_ggml_block_bytes(type)] bytes (output; 16-byte aligned)
 * Errors: RRQ_ERR_INVALID (type, d, dtype, rotate, null or misaligned pointer),
 * RRQ_ERR_CUDA.
 */
int rrq_ggml_rot(const void* x, int x_dtype, int64_t n, int d, uint64_t seed, int rotate, int type,
                 void* blocks, void* stream);

/*
 * rrq_ggml_rot_decode — inverse of rrq_ggml_rot: with the stored fp16 values,
 * ŷ_j = q_j·Δ + lo (q4_1, q5_1), (q_j − 16)·Δ (q5_0), q_j·Δ (q8_0), (q_j − 8)·Δ
 * (q4_0); then x̂ = Πᵀŷ when rotate = 1.  fp32 arithmetic (q·Δ + lo as one fused
 * multiply-add), rounded to out_dtype.
 *   blocks  [n × d/32 × rrq_ggml_block_bytes(type)] bytes;  out [n × d] of out_dtype
 * Errors: RRQ_ERR_INVALID, RRQ_ERR_CUDA.
 */
int rrq_ggml_rot_decode(const void* blocks, int type, int64_t n, int d, uint64_t seed, int rotate,
                        void* out, int out_dtype, void* stream);

/*
 * rrq_qjl_matrix — the QJL projection S for a seed, on the HOST.
 * Entry e = i·d + j: u1, u2 = top 53 bits of SplitMix64 outputs 2e, 2e+1 as
 * uniforms in [0,1); z = sqrt(−2 ln(1 − u1))·cos(2π·u2) (Box–Muller);
 * S[i][j] = bf16(z) (nearest even).  Written as bf16 bit patterns; the
 * caller copies S to the device once and passes it to rrq_encode.
 *   S  HOST, uint16_t[d × d]
 * d a power of two in [64, 512].  Errors: RRQ_ERR_INVALID.
 */
int rrq_qjl_matrix(uint64_t seed, int d, uint16_t* S);

#ifdef __cplusplus
}
#endif

#endif /* RRQ_H */
