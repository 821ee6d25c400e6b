/*
 * gpt2_ops.h - the kernels of the GPT-2 training step, one entry point each.
 *
 * These are the same kernels gpt2_forward/gpt2_backward/gpt2_adamw_step run,
 * exposed on caller-owned device buffers so that each can be checked alone.
 * The kernel list is the one of llm.c "State of the Union [May 3, 2024]",
 * kernel table under "Runtime, DRAM traffic, instructions": encoder forward
 * and backward, layernorm forward and backward, the bf16 matmuls, attention
 * forward and backward, GELU forward and backward, residual, the fused
 * classifier, the bias-gradient reduction and AdamW.
 *
 * Conventions:
 *   - dtype: GPT2_MODE_FP32 (0) for fp32 activations, GPT2_MODE_BF16 (1) for
 *     bf16 activations. Arithmetic inside a kernel is fp32 in both.
 *   - Every pointer is a device pointer unless stated. All tensors are
 *     dense and row-major. Activation buffers need 16-byte alignment.
 *   - stream is a cudaStream_t (NULL = legacy default stream). Calls only
 *     enqueue work; they never synchronise, allocate or free.
 *   - scratch: caller-owned device memory of at least the size the matching
 *     *_scratch_bytes() call returns (256-byte aligned); its contents on
 *     entry do not matter. Two calls that share a scratch buffer must not
 *     overlap on the device.
 *   - d_status: optional device int; kernels OR an error bit into it
 *     (1 = token id out of range, 2 = bounded wait timed out, 4 = target id
 *     out of range, 8 = sequence offsets out of order or out of range) and
 *     never trap.
 *   - Return GPT2_OK or a negative gpt2_status (see gpt2.h) for bad
 *     arguments or a failed launch.
 */
#ifndef GPT2_OPS_H
#define GPT2_OPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* x0[b,t,:] = wte[tokens[b,t],:] + wpe[t,:] (section "Single GPU training":
 * GPT-2's token plus learned position embedding; kernel "encoder_forward").
 * x0 [B*T, C], wte [>=V, C], wpe [>=T, C] in dtype. An id outside [0,V) sets
 * bit 1 of *d_status and reads row 0 instead. */
int gpt2_op_encoder_forward(int dtype, void* x0, const int32_t* tokens, const void* wte,
                            const void* wpe, int B, int T, int C, int V, int* d_status,
                            void* stream);

/* Embedding backward ("encoder_backward"): dwte[v,:] += sum of dx0 rows
 * whose token is v, summed in ascending position order (deterministic);
 * dwpe[t,:] = sum_b dx0[b,t,:] for t < T (rows t >= T untouched).
 * dwte [Vp, C] fp32 (accumulated into), dwpe [>=T, C] fp32 (overwritten),
 * dx0 [B*T, C] dtype, tokens in [0, Vp). */
size_t gpt2_op_encoder_backward_scratch(int B, int T, int C);
int gpt2_op_encoder_backward(int dtype, float* dwte, float* dwpe, const void* dx0,
                             const int32_t* tokens, int B, int T, int C, int Vp,
                             void* scratch, size_t scratch_bytes, void* stream);

/* LayerNorm forward ("layernorm_forward"): per row of x [N, C],
 * y = (x - mean) * rstd * gamma + beta, rstd = 1/sqrt(biased var + 1e-5);
 * mean and rstd [N] fp32 are saved for the backward. C % 8 == 0, C <= 2048. */
int gpt2_op_layernorm_forward(int dtype, void* y, float* mean, float* rstd, const void* x,
                              const void* gamma, const void* beta, int N, int C, void* stream);

/* LayerNorm backward ("layernorm_backward"): with xhat = (x-mean)*rstd and
 * dxhat = dy*gamma, dx = rstd (dxhat - mean(dxhat) - xhat mean(dxhat xhat))
 * (dtype, overwritten); dgamma = sum_rows dy xhat, dbeta = sum_rows dy (fp32,
 * overwritten, deterministic two-stage reduction through scratch). */
size_t gpt2_op_layernorm_backward_scratch(int N, int C);
int gpt2_op_layernorm_backward(int dtype, void* dx, float* dgamma, float* dbeta, const void* dy,
                               const void* x, const void* gamma, const float* mean,
                               const float* rstd, int N, int C, void* scratch,
                               size_t scratch_bytes, void* stream);

/* Residual join followed by LayerNorm, one pass: xsum = x + r (rounded to
 * dtype, stored), then y, mean, rstd = LayerNorm of xsum exactly as
 * gpt2_op_layernorm_forward computes it. In the GPT-2 block every residual
 * sum ("residual_forward") is read next by a LayerNorm ("layernorm_forward";
 * llm.c "State of the Union", section "Runtime, DRAM traffic,
 * instructions"). xsum must not overlap x, r or y. Limits as for
 * gpt2_op_layernorm_forward. */
int gpt2_op_residual_layernorm_forward(int dtype, void* y, float* mean, float* rstd, void* xsum,
                                       const void* x, const void* r, const void* gamma,
                                       const void* beta, int N, int C, void* stream);

/* LayerNorm backward into the residual-stream gradient: with dx as in
 * gpt2_op_layernorm_backward, dres = dx (accumulate = 0) or dres += dx
 * (accumulate = 1, the residual join of the backward pass; dres is read and
 * written in place). dgamma, dbeta as in gpt2_op_layernorm_backward; if
 * dres_colsum is not null it receives the column sums of the resulting dres
 * (as stored, in dtype), fp32 [C], overwritten: the bias gradient
 * ("matmul_backward_bias") of the projection whose output joined the
 * residual stream at this point. Scratch: gpt2_op_layernorm_backward_scratch. */
int gpt2_op_layernorm_backward_residual(int dtype, void* dres, int accumulate, float* dgamma,
                                        float* dbeta, float* dres_colsum, const void* dy,
                                        const void* x, const void* gamma, const float* mean,
                                        const float* rstd, int N, int C, void* scratch,
                                        size_t scratch_bytes, void* stream);

/* Matmul (the bf16 GEMMs of the kernel table, "ampere_bf16" and
 * "cutlass::Kernel2"): D[M,N] = sum_k A(m,k) B(n,k) (+ bias[n]).
 * A(m,k) is A[m*K + k] (a_mn_major = 0) or A[k*M + m] (a_mn_major = 1);
 * B(n,k) is B[n*K + k] (b_mn_major = 0) or B[k*N + n] (b_mn_major = 1).
 * So the linear forward is (0,0) with B = W [N,K]; the input gradient
 * dX = dY W is (0,1); the weight gradient dW = dY^T X is (1,1).
 * A, B and bias (optional, length N, dtype) are in dtype; D is fp32 if
 * d_fp32 else dtype, overwritten. bf16: tcgen05 tensor cores (TMA-fed,
 * fp32 accumulate in tensor memory); fp32: fp32 FMA. Needs K % 8 == 0 and
 * N % 8 == 0 (and M % 8 == 0 when a_mn_major); 16-byte aligned buffers.
 * K >= 1 (K = 0 is GPT2_ERR_ARG); M = 0 or N = 0 launches nothing.
 * Scratch holds split-K partial sums (fp32 D only). */
size_t gpt2_op_matmul_scratch(int dtype, int M, int N, int K, int d_fp32);
int gpt2_op_matmul(int dtype, void* D, int d_fp32, const void* A, int a_mn_major, const void* B,
                   int b_mn_major, const void* bias, int M, int N, int K, void* scratch,
                   size_t scratch_bytes, int* d_status, void* stream);

/* FP8 linear layer (the modded-nanogpt project page, "NanoGPT (124M) in 90
 * seconds", "How it works": FP8 for the MLP, the QKV projections and the
 * head), with per-tensor scaling to one of two 8-bit floating-point formats
 * (OCP 8-bit floating point):
 *   GPT2_FP8_E4M3  1 sign, 4 exponent bits (bias 7), 3 mantissa bits, largest
 *                  finite value fmax = 448 (weights and activations);
 *   GPT2_FP8_E5M2  1 sign, 5 exponent bits (bias 15), 2 mantissa bits,
 *                  largest finite value fmax = 57344 (gradients).
 *
 * gpt2_op_quantize_fp8: q[i] = fp8(x[i] * scales[0]) for n bf16 values x in
 * the given format, with scales[0] = fmax / amax and scales[1] = amax / fmax
 * written on the device (both 1 when amax = max |x| is 0); the product is
 * rounded to fp32, then to the nearest value of the format (ties to even),
 * saturating at +-fmax; a NaN stays NaN and does not enter amax. q: n bytes
 * (8-byte aligned), x 16-byte aligned, scales: 2 floats; scratch:
 * gpt2_op_quantize_fp8_scratch() bytes. An unknown format is GPT2_ERR_ARG.
 *
 * gpt2_op_matmul_fp8: D[M,N] (bf16, overwritten) = (A B^T)[m,n] *
 * a_scales[1] * b_scales[1] (+ bias[n], bf16, optional), A [M,K] and B [N,K]
 * FP8 codes row-major (B is the [out, in] weight), each in its own format
 * (an e5m2 gradient times an e4m3 weight, for instance), the scale arrays as
 * written by gpt2_op_quantize_fp8 (read on the device). tcgen05 tensor cores
 * (kind::f8f6f4, TMA-fed, fp32 accumulation in tensor memory). Needs K % 16
 * == 0 and N % 8 == 0, 16-byte aligned A, B, D and bias; an unknown format is
 * GPT2_ERR_ARG. */
#define GPT2_FP8_E4M3 0
#define GPT2_FP8_E5M2 1
size_t gpt2_op_quantize_fp8_scratch(void);
int gpt2_op_quantize_fp8(void* q, float* scales, const void* x, int64_t n, int format, void* scratch,
                         size_t scratch_bytes, void* stream);
int gpt2_op_matmul_fp8(void* D, const void* A, int a_format, const float* a_scales, const void* B, int b_format,
                       const float* b_scales, const void* bias, int M, int N, int K, int* d_status, void* stream);

/* The codes of x [R][C] (bf16, row-major, C % 8 == 0, 16-byte aligned) under
 * the scales of an earlier gpt2_op_quantize_fp8 of the same values (scales[0]
 * multiplies, as there), written transposed to qt [C][R] and, when q is not
 * null, also as they are to q [R][C]: the same codes gpt2_op_quantize_fp8
 * gives, in the K-major layout the weight-gradient and input-gradient
 * products of an FP8 linear layer read. */
int gpt2_op_quantize_fp8_transpose(void* qt, void* q, const float* scales, const void* x, int R, int C,
                                   int format, void* stream);

/* The general FP8 product: epi 0: D[M,N] = (A B^T) a_scales[1] b_scales[1]
 * (+ bias), in bf16 or (d_fp32) fp32, accumulate (fp32 only): D += instead;
 * epi 1 (the MLP's first linear and its GELU): u = that product + bias
 * rounded to bf16, D = gelu'(u), D2 = gelu(u) (bf16); epi 2 (the input
 * gradient through the GELU): D = bf16(A B^T scales) * aux[m,n] (aux bf16
 * [M,N]). A [M,K], B [N,K] FP8 codes, K-major, K % 16 == 0, N % 8 == 0;
 * scratch: gpt2_op_matmul_fp8_scratch(M, N, K, d_fp32, accumulate) bytes
 * (split-K partial tiles of an fp32 product). */
size_t gpt2_op_matmul_fp8_scratch(int M, int N, int K, int d_fp32, int accumulate);
int gpt2_op_matmul_fp8_ex(int epi, void* D, void* D2, const void* aux, int d_fp32, int accumulate, const void* A,
                          int a_format, const float* a_scales, const void* B, int b_format, const float* b_scales,
                          const void* bias, int M, int N, int K, void* scratch, size_t scratch_bytes, int* d_status,
                          void* stream);

/* Linear forward with the GELU after it fused into the GEMM epilogue (the
 * MLP's first linear, "matmul_forward", followed by "gelu_forward" in the
 * kernel table): u = A W^T + bias (A [M,K], W [N,K] row-major, bias [N]
 * optional), rounded to dtype; out = gelu(u) with the tanh-approximation
 * GELU of gpt2_op_gelu_forward, and dgelu = gelu'(u), the factor the
 * backward needs (the backward of the step uses nothing else of u). Both
 * outputs [M,N] in dtype, overwritten, not overlapping. bf16: one
 * tensor-core GEMM whose epilogue writes both; fp32: the fp32 GEMM (into
 * dgelu) then one elementwise pass. Same shape and alignment rules as
 * gpt2_op_matmul. */
int gpt2_op_matmul_gelu(int dtype, void* dgelu, void* out, const void* A, const void* W,
                        const void* bias, int M, int N, int K, int* d_status, void* stream);

/* The input gradient of that GELU's input, fused ("gelu_backward" of the
 * kernel table folded into the preceding "matmul_backward"): du[M,N] =
 * (dY W)[m,n] * dgelu[m,n] with dY [M,K], W [K,N] row-major (the weight of
 * the linear that read gelu(u)) and dgelu from gpt2_op_matmul_gelu; the
 * product dY W is rounded to dtype before the multiply. du overwritten, in
 * dtype; it may not overlap dgelu. */
int gpt2_op_matmul_gelu_backward(int dtype, void* du, const void* dY, const void* W,
                                 const void* dgelu, int M, int N, int K, int* d_status,
                                 void* stream);

/* The same, and the bias gradient of the linear whose output gradient du is
 * ("matmul_backward"'s bias part): dbias[n] = sum over m of du[m,n], fp32
 * [N], overwritten, summed from the values as stored in du. bf16: the sums
 * of each 32-row slice are formed in the matmul's epilogue and reduced by a
 * second launch; fp32: a separate column-sum pass over du. scratch: at least
 * gpt2_op_matmul_gelu_backward_bias_scratch(M, N) bytes (else
 * GPT2_ERR_WORKSPACE). */
size_t gpt2_op_matmul_gelu_backward_bias_scratch(int M, int N);
int gpt2_op_matmul_gelu_backward_bias(int dtype, void* du, float* dbias, const void* dY,
                                      const void* W, const void* dgelu, int M, int N, int K,
                                      void* scratch, size_t scratch_bytes, int* d_status,
                                      void* stream);

/* Causal multi-head attention forward ("flash attention", section "Single
 * GPU training"; kernel "cudnn_generated_fort_native_sdpa"): qkv [B*T, 3C]
 * holds q | k | v column blocks, head h at columns h*hd..h*hd+hd-1 of each.
 * o [B*T, C] (dtype) = softmax(q k^T / sqrt(hd), causal) v per head; lse
 * [B, H, T] fp32 = log-sum-exp of each scaled score row. The T x T score
 * matrix is never stored. hd == 64 for bf16; hd <= 64 for fp32. */
int gpt2_op_attention_forward(int dtype, void* o, float* lse, const void* qkv, int B, int T,
                              int C, int H, void* stream);

/* Attention backward (kernels "compute_dot_do_o", the SDPA backward and
 * "rearrange_n_convert_dq" of the table): D = rowsum(dO * O) into scratch,
 * then with P recomputed from lse: dV = P^T dO, dS = P (dO V^T - D),
 * dQ = dS K / sqrt(hd), dK = dS^T Q / sqrt(hd), written to dqkv [B*T, 3C]
 * (dtype, overwritten) in the q | k | v layout. Deterministic (no atomics). */
size_t gpt2_op_attention_backward_scratch(int B, int T, int H);
int gpt2_op_attention_backward(int dtype, void* dqkv, const void* dout, const void* qkv,
                               const void* o, const float* lse, int B, int T, int C, int H,
                               void* scratch, size_t scratch_bytes, void* stream);

/* Causal attention over packed sequences of different lengths, with grouped
 * heads (an addition of this library: the attention of the step, which takes
 * B sequences of one length, for a batch of documents laid end to end).
 * Sequence s has the queries cu_q[s] .. cu_q[s+1]-1 and the keys
 * cu_k[s] .. cu_k[s+1]-1 (cu_q, cu_k: n_seq + 1 ascending int32 offsets in
 * device memory, read by the kernels, so a captured graph follows them; they
 * may be one array). Its query i sees its keys 0 .. i + lk - lq (lq, lk the
 * sequence's own lengths: the last query sees every key, so lq < lk continues
 * a prompt whose first keys are cached, lq = 1 is one new token). Query head h
 * reads key head h / (Hq / Hkv).
 *   o[i,h,:] = softmax(q[i,h,:] . k / sqrt(hd)) v, lse[h,i] = log-sum-exp of
 *   the scaled scores. A query that sees no key (lk < lq) gets o = 0 and
 *   lse = -inf.
 * q, o [total_q] rows of Hq * hd values, k, v [total_k] rows of Hkv * hd,
 * head h at columns h*hd .. of a row; *_stride: elements from one row to the
 * next (so q, k and v may be column blocks of one fused buffer). lse [Hq,
 * total_q] fp32. Rows of o and lse that belong to no sequence (before
 * cu_q[0], at or after cu_q[n_seq]) are left as they were, and no row's
 * result depends on rows of another sequence, whatever they hold. Within a
 * sequence, a NaN or infinity at a position may reach the results of earlier
 * positions of the same 128-row tile (in the backward also gradients of the
 * tile's keys that its query does not see). o and lse must not overlap the
 * inputs.
 *   - max_q, max_k: at least the longest sequence's queries and keys (they
 *     choose the kernel; a longer sequence sets bit 8 of *d_status).
 *   - Offsets that descend or leave [0, total] set bit 8 of *d_status; they
 *     are clamped, so no memory outside the buffers is touched.
 *   - hd == 64 for bf16; hd 8, 16, 32 or 64 for fp32. Hq a multiple of Hkv,
 *     at most 128 query heads to a key head. Pointers 16-byte aligned, strides
 *     multiples of 16 bytes and at least the row. total_q * Hq, total_k * Hkv
 *     and n_seq * Hq below 2^30 (else GPT2_ERR_ARG).
 *   - n_seq = 0 or total_q = 0 launches nothing.
 *   - Every wait of the bf16 kernels is bounded by 4e9 cycles (bit 2 of
 *     *d_status): a sequence of more than 5e7 keys may run into it.
 * Scratch: the list of work items and links of those that come again, or
 * partial results of keys split over blocks (few queries). */
size_t gpt2_op_attention_packed_forward_scratch(int dtype, int n_seq, int total_q, int total_k, int max_q, int max_k,
                                                int Hq, int Hkv, int hd);
int gpt2_op_attention_packed_forward(int dtype, void* o, int64_t o_stride, float* lse, const void* q,
                                     int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                     int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int n_seq,
                                     int total_q, int total_k, int max_q, int max_k, int Hq, int Hkv, int hd,
                                     void* scratch, size_t scratch_bytes, int* d_status, void* stream);

/* Its backward, from the forward's o and lse: with D = rowsum(dO * O) and P
 * recomputed from lse, dV = P^T dO, dS = P (dO V^T - D), dQ = dS K / sqrt(hd),
 * dK = dS^T Q / sqrt(hd); dK and dV are summed over the query heads of their
 * group. dq [total_q] rows, dk, dv [total_k] rows (dtype, their own strides,
 * overwritten; rows of no sequence are left as they were, a key that no query
 * sees gets 0). Deterministic (no atomics). dq, dk, dv must not overlap the
 * inputs. Sequences, strides and limits as in the forward. Scratch (bf16): lse
 * and D, the lists of work items. */
size_t gpt2_op_attention_packed_backward_scratch(int dtype, int n_seq, int total_q, int total_k, int Hq, int Hkv,
                                                 int hd);
int gpt2_op_attention_packed_backward(int dtype, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride, void* dv,
                                      int64_t dv_stride, const void* dout, int64_t dout_stride, const void* q,
                                      int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, const void* o, int64_t o_stride, const float* lse,
                                      const int32_t* cu_q, const int32_t* cu_k, int n_seq, int total_q, int total_k,
                                      int max_q, int max_k, int Hq, int Hkv, int hd, void* scratch,
                                      size_t scratch_bytes, int* d_status, void* stream);

/* GELU, tanh form ("gelu_forward"): g = 0.5 u (1 + tanh(sqrt(2/pi)(u + 0.044715 u^3))).
 * n % 8 == 0. In place (g == u) is allowed. */
int gpt2_op_gelu_forward(int dtype, void* g, const void* u, int64_t n, void* stream);

/* GELU backward ("gelu_backward"): du = dg * g'(u). In place (du == dg) allowed. */
int gpt2_op_gelu_backward(int dtype, void* du, const void* u, const void* dg, int64_t n,
                          void* stream);

/* Residual forward ("residual_forward"): out = a + b, n % 8 == 0. */
int gpt2_op_residual_forward(int dtype, void* out, const void* a, const void* b, int64_t n,
                             void* stream);

/* Residual backward: the gradient reaching a residual join from the
 * branch is added to the stream gradient, dres += dbranch, n % 8 == 0.
 * llm.c's kernel table has no row of its own for it (the step folds it into
 * the LayerNorm backward, gpt2_op_layernorm_backward_residual). */
int gpt2_op_residual_backward(int dtype, void* dres, const void* dbranch, int64_t n,
                              void* stream);

/* Bias gradient ("matmul_backward_bias"): dbias[c] = sum_rows dy[r, c]
 * (fp32, overwritten), dy [N, C] dtype; deterministic two-stage reduction. */
size_t gpt2_op_bias_backward_scratch(int N, int C);
int gpt2_op_bias_backward(int dtype, float* dbias, const void* dy, int N, int C, void* scratch,
                          size_t scratch_bytes, void* stream);

/* Bias gradient without caller scratch (no counterpart on the pages; in
 * place of a citation: an addition of this library). It serves callers that
 * cannot allocate or lend device memory (for example a program whose device memory is wholly owned by
 * another runtime's allocator or a fixed pool, or code that must not call
 * cudaMalloc because it can synchronise the device). It computes exactly
 * what gpt2_op_bias_backward computes, dbias[c] = sum_rows dy[r, c] (fp32,
 * overwritten), but its partial sums go to a fixed 4 MiB array inside the
 * library instead of caller scratch. It calls no cudaMalloc, cudaFree or
 * allocating library routine.
 *   - Limit: ceil(N/128) * C <= 1,048,576 (e.g. N = 32768 rows with
 *     C <= 4096). Larger sizes return GPT2_ERR_WORKSPACE and launch nothing.
 *   - The array is held by every GPU that loads the library until the
 *     process exits. The first call on each device looks up its device
 *     address (cudaGetSymbolAddress) with that device current; make that
 *     first call before any stream capture.
 *   - All calls share the one array. Calls that overlap on the GPU (on
 *     different streams, or from several threads) race and give wrong
 *     results; order them on one stream. Nothing in the array needs to
 *     start at zero: each call writes every partial it reads.
 * Arguments as gpt2_op_bias_backward, without the scratch. */
int gpt2_op_bias_backward_noalloc(int dtype, float* dbias, const void* dy, int N, int C,
                                  void* stream);

/* Fused classifier ("fused_classifier", section "Single GPU training" and
 * "Fine print"): per row i of logits [N, Vp] (dtype), over columns j < V only:
 * lse_i = log sum exp z_ij, losses[i] = lse_i - z_i,targets[i] (fp32), and in
 * place z_ij <- dloss * (exp(z_ij - lse_i) - [j == target_i]) for j < V,
 * 0 for V <= j < Vp. Normalised logits are never stored. dloss is the
 * gradient of the loss w.r.t. each row's loss (1/N for a mean).
 * A target outside [0,V) sets bit 4 of *d_status and is treated as 0. */
int gpt2_op_classifier(int dtype, void* logits, float* losses, const int32_t* targets, int N,
                       int V, int Vp, float dloss, int* d_status, void* stream);

/* Log-probabilities of given tokens, with entropy and the top alternatives
 * (an addition of this library: the classifier's softmax kept for scoring; the
 * logits are read once and left as they are). Per row i of logits [N, Vp]
 * (dtype), over columns j < V only (Vp % 8 == 0):
 *   lse[i]  = log sum exp z_ij,  logp[i] = z_i,targets[i] - lse[i],
 *   entropy[i] = -sum_j p_ij log p_ij with p = exp(z - lse) (0 log 0 = 0),
 *   top_ids[i, 0..k-1] = the columns of the k largest logits, largest first,
 *   equal logits by the lowest column, top_logp[i, r] their log-probability.
 * Log-probabilities are (z - max) - ln S: accurate to a few 2^-24 and their own
 * size however far the logits are from 0, never positive; no entropy is
 * negative. All outputs fp32 (top_ids int32); 0 <= k <= 64, k <= V, top_logp and top_ids
 * [N, k] (unused for k = 0); entropy may be null; logp and targets may both be
 * null. A target outside [0,V) sets bit 4 of *d_status and is treated as 0. A
 * row whose every logit is -inf has no distribution: lse = logp = top_logp =
 * -inf, entropy = 0. A row with a NaN gets NaN in all of them; one with +inf
 * (and no NaN) gets lse = inf, entropy = NaN, and log-probabilities of -inf
 * (NaN for its infinite columns). top_ids stay in [0,V); a NaN counts as
 * the largest. */
int gpt2_op_token_logprobs(int dtype, float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids,
                           int k, const void* logits, const int32_t* targets, int N, int V, int Vp, int* d_status,
                           void* stream);

/* Its gradient: with g = dlogp[i], a = dlse[i], b = dentropy[i] (each array
 * may be null: 0) and p, log p from the forward's lse,
 *   dlogits_ij = g ([j == target_i] - p_ij) + a p_ij - b p_ij (log p_ij + entropy_i)
 * for j < V (0 where p_ij = 0, and in a row that has no distribution), 0 for
 * V <= j < Vp. dlogits [N, Vp] (dtype, overwritten) may be logits itself.
 * entropy is needed with dentropy, targets with dlogp; targets out of range as
 * above. p carries lse's own rounding (|lse| 2^-24, relative). Nothing is summed across rows: deterministic. */
int gpt2_op_token_logprobs_backward(int dtype, void* dlogits, const void* logits, const int32_t* targets,
                                    const float* lse, const float* entropy, const float* dlogp, const float* dlse,
                                    const float* dentropy, int N, int V, int Vp, int* d_status, void* stream);

/* Mean of losses [N] into *out (device fp32): fixed-order tree, deterministic.
 * The mean loss of the forward with targets (llm.c "State of the Union",
 * "Single GPU training"). */
int gpt2_op_mean_loss(float* out, const float* losses, int N, void* stream);

/* AdamW ("adamw_kernel"): over n fp32 elements, m = b1 m + (1-b1) g;
 * v = b2 v + (1-b2) g^2; theta -= lr (m/(1-b1^t) / (sqrt(v/(1-b2^t)) + eps)
 * + wd theta); if param_bf16 != NULL also writes bf16(theta) (round to
 * nearest even) there. n % 4 == 0. */
int gpt2_op_adamw(float* master, void* param_bf16, const float* grad, float* m, float* v,
                  int64_t n, float lr, float beta1, float beta2, float eps, float weight_decay,
                  int t, void* stream);

/* Norms of queries and keys for each head with the position rotation, in one
 * pass (an addition of this library: positions for packed sequences, whose
 * tokens the encoder's learned positions do not count). For N rows (tokens) of
 * Hq query heads and Hk key heads of hd values, each head x becomes
 *   n = x * rstd * gamma, rstd = 1 / sqrt(mean(x^2) + eps)   (norm != 0; else n = x)
 *   y_a = amplitude (n_a cos t - n_b sin t), y_b = amplitude (n_a sin t + n_b cos t)
 * for the pairs of its first rot values: (j, j + rot / 2) (interleaved = 0) or
 * (2 j, 2 j + 1) (interleaved != 0), j < rot / 2; the other values keep n. The
 * angle t is pos[row] * turns[j] * 2^-64 turns, modulo one turn: turns is a
 * device array of rot / 2 fractions of a turn per position (gpt2_rotary_turns
 * fills one on the host, good to 2^-34 of a turn at any int32 position); cos and
 * sin are formed in fp32 from the exact product's distance to its nearest quarter
 * turn, which is rounded to 2^-28 of a turn.
 *   q, qo: rows of Hq * hd values, k, ko: rows of Hk * hd (dtype), head h at
 *   columns h*hd .. of a row; *_stride: elements from one row to the next, so
 *   they may be column blocks of one fused buffer. qo may be q and ko k (with
 *   the same stride); otherwise outputs must not overlap inputs.
 *   q_gamma, k_gamma: [hd] in dtype, or null (ones); unused without norm.
 *   - hd 8, 16, 32, 64 or 128; rot a multiple of 8, 0 <= rot <= hd (turns may
 *     be null for 0). Hq, Hk >= 0, not both 0 (pointers of none are unused).
 *     Pointers 16-byte aligned, strides multiples of 16 bytes and at least the
 *     row. eps > 0 with norm; amplitude finite. N = 0 launches nothing.
 *   - Squares are formed in fp32: a head with values from about 1e19 on has an
 *     infinite mean and comes out as 0. */
int gpt2_op_qk_norm_rotary_forward(int dtype, void* qo, int64_t qo_stride, void* ko, int64_t ko_stride, const void* q,
                                   int64_t q_stride, const void* k, int64_t k_stride, const void* q_gamma,
                                   const void* k_gamma, const int32_t* pos, const uint64_t* turns, int N, int Hq,
                                   int Hk, int hd, int rot, int interleaved, int norm, float eps, float amplitude,
                                   void* stream);

/* Its backward: from dqo, dko (gradients of qo, ko) and the forward's q, k
 * (read with norm only; they may be null without), with dn the gradient turned
 * back, xhat = x rstd: dx = rstd (dn gamma - xhat mean(dn gamma xhat)) into dq,
 * dk (dtype, overwritten; dq may be dqo and dk dko with the same stride),
 * dq_gamma, dk_gamma [hd] fp32 = the sums of dn xhat over rows and heads
 * (overwritten; either may be null, both are unused without norm).
 * Deterministic (no atomics). N = 0 sets the gammas' gradients to 0. Scratch:
 * partial sums of the gammas' gradients. Limits as in the forward. */
size_t gpt2_op_qk_norm_rotary_backward_scratch(int N, int hd);
int gpt2_op_qk_norm_rotary_backward(int dtype, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                                    float* dq_gamma, float* dk_gamma, const void* dqo, int64_t dqo_stride,
                                    const void* dko, int64_t dko_stride, const void* q, int64_t q_stride,
                                    const void* k, int64_t k_stride, const void* q_gamma, const void* k_gamma,
                                    const int32_t* pos, const uint64_t* turns, int N, int Hq, int Hk, int hd, int rot,
                                    int interleaved, int norm, float eps, float amplitude, void* scratch,
                                    size_t scratch_bytes, void* stream);

/* Host: turns[j] = round(2^64 f_j / (2 pi)) for j < rot / 2 (host memory), with
 * the frequencies f_j = base^(-2 j / rot) stretched for contexts longer than
 * the model's own:
 *   GPT2_ROTARY_PLAIN   as they are;
 *   GPT2_ROTARY_LINEAR  divided by factor (positions interpolated);
 *   GPT2_ROTARY_BASE    base * factor^(rot / (rot - 2)) in place of base: the
 *                       fastest pair stays, the slowest is divided by factor;
 *   GPT2_ROTARY_PARTS   divided by factor where a pair turns less than slow
 *                       times over `context` positions, kept where it turns
 *                       more than fast times, blended linearly in the number
 *                       of turns between.
 * rot even and >= 0, base > 1, factor >= 1, and for PARTS context >= 1, fast > slow >= 0
 * (else GPT2_ERR_ARG). */
#define GPT2_ROTARY_PLAIN 0
#define GPT2_ROTARY_LINEAR 1
#define GPT2_ROTARY_BASE 2
#define GPT2_ROTARY_PARTS 3
int gpt2_rotary_turns(uint64_t* turns, int rot, double base, int scaling, double factor, double context, double fast,
                      double slow);

/* Softmax cross entropy from hidden states and the head's weight, without
 * keeping the logits (an addition of this library: gpt2_op_matmul with the
 * head's weight followed by gpt2_op_classifier, without the N x V buffer
 * between them). With z = x W^T over the first V rows of W:
 *   lse[i] = log sum_j<V exp z_ij, losses[i] = lse[i] - z_i,targets[i] (fp32),
 * formed as (max - z_target) + ln sum exp(z - max): never negative, and as
 * exact far from 0 as near it. x [N, C], w [>= V, C] in dtype (the rows of w
 * from V on are not used, whatever they hold); the logits are fp32 and are not
 * rounded. A target outside [0,V) sets bit 4 of *d_status and is treated as 0.
 * Rows of x are independent. A logit of -inf counts as nothing (a row of nothing
 * else gets lse = -inf and a loss of +inf); a row with a NaN or +inf gets NaN.
 * C % 8 == 0, C >= 8, V >= 1, x and w 16-byte aligned; N * C, V * C and the
 * 64 x 64 tiles of N x V below 2^31 - 2048; N = 0 launches nothing. Scratch: row statistics of the
 * vocabulary's tiles. */
size_t gpt2_op_linear_classifier_forward_scratch(int dtype, int N, int C, int V);
int gpt2_op_linear_classifier_forward(int dtype, float* losses, float* lse, const void* x, const void* w,
                                      const int32_t* targets, int N, int C, int V, void* scratch,
                                      size_t scratch_bytes, int* d_status, void* stream);

/* Its gradient from the forward's lse: with p = exp(z - lse) formed again, in
 * pieces of the vocabulary,
 *   dz_ij = (dloss[i] + dlse[i]) p_ij - dloss[i] [j == targets[i]],
 *   dx = dz W (dtype, overwritten), dw = dz^T x.
 * dloss, dlse: [N] fp32, gradients of losses and lse, either may be null (0). A
 * row whose dloss and dlse are 0, or whose lse is -inf, has dz = 0 whatever its
 * logits are (a prompt's or padding's tokens; it costs what any row costs, and x
 * and the first V rows of w have to be finite all the same: the products add 0
 * times them). dw [Vp, C], Vp >= V, Vp % 8 == 0: fp32 (dw_fp32 = 1; the only
 * form in fp32) or bf16; rows from V on get 0. accumulate (fp32 dw only): dw +=
 * instead, rows from V on stay. In bf16 dz is rounded to bf16 for the products, in units of the largest |dloss|
 * and |dloss + dlse|: half a step (2^-8) of each value (what is below 2^-126 of
 * that unit loses bits, and is 0 below 2^-134); sums are fp32. p carries lse's own
 * rounding (|lse| 2^-24, relative). Deterministic: sums are taken in a fixed
 * order (the one atomic is the largest |dloss|, the same in any). dx and dw must
 * not overlap the inputs or each other. Limits as in the forward; N = 0 sets
 * dw to 0 (or leaves it, with accumulate). Scratch: a piece of dz (up to 1 GB,
 * or 2048 columns where that is more: all columns where they fit, 824 MB for
 * 8192 rows of 50257 in bf16), dx in fp32 where there are several pieces,
 * partial products (with accumulate, a piece of dw in fp32). */
size_t gpt2_op_linear_classifier_backward_scratch(int dtype, int N, int C, int V, int Vp, int accumulate);
int gpt2_op_linear_classifier_backward(int dtype, void* dx, void* dw, int dw_fp32, int accumulate, const void* x,
                                       const void* w, const int32_t* targets, const float* lse, const float* dloss,
                                       const float* dlse, int N, int C, int V, int Vp, void* scratch,
                                       size_t scratch_bytes, int* d_status, void* stream);

/* AdamW over many tensors at once, with moments in 32 or in 8 bits (an
 * addition of this library: gpt2_op_adamw for a list of tensors of any sizes).
 * For each value of each tensor, with g = grad * grad_scale * clip, clip =
 * min(1, max_grad_norm / (||grad|| |grad_scale| + 1e-6)) over all tensors if
 * max_grad_norm > 0, else 1 (as gpt2_adamw_step_ex). Squares are formed in
 * fp32: from about 1e19 on ||grad|| is infinite, and clip 0; a NaN clips nothing.
 *   m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2;
 *   theta -= lr (m/(1-b1^t) / (sqrt(v/(1-b2^t)) + eps) + weight_decay theta),
 * and bf16(theta) to param_bf16 where that is not null. grad_norm, if not
 * null, receives ||grad|| (before grad_scale; device float). Deterministic.
 *
 * The list is host memory and is read during the call only. grads are all in
 * grad_dtype. n >= 0 values of any count (n = 0: nothing to do); addresses need
 * the alignment of their type only (16 bytes are faster). Tensors must not
 * overlap. At most 2^24 tensors of together fewer than 2^42 values.
 *
 * bits = 32: m and v are fp32 [n]; m_scale and v_scale are unused. bits = 8: m
 * and v are n bytes each, m_scale and v_scale ceil(n / 128) bytes; zeros are
 * moments of 0. The value of a code under its block's scale byte s (128
 * consecutive values share one) is code * 2^(s - 127):
 *   m   sign, 4 exponent bits (bias 7), 3 mantissa bits; the largest magnitude
 *       of a block lies in [2^7, 2^8]; 0x7F and 0xFF are NaN;
 *   v   5 exponent bits (bias 15), 3 mantissa bits, no sign (the top of an
 *       fp16 number); the largest lies in [2^14, 2^15]; NaN is written as 0xFF.
 * Both have subnormals. The new m and v are formed in fp32, with each product
 * and sum rounded on its own (b1 m + (1-b1) g, b2 v + (1-b2) (g g)), and used
 * for theta as they are; stored, they are rounded up or down to a neighbouring code so
 * that they are right on average: up where (what is left over the lower code)
 * / (the codes' distance) + u >= 1, with u = r / 2^16 and r 16 bits of
 * splitmix64's finaliser mix: values 2p and 2p + 1 of tensor k (from 0 in the
 * list) take bits 0-15 and 32-47 (m) and 16-31 and 48-63 (v) of
 *   mix(mix(seed + t G) + (k 2^40 + p) G), G = 0x9E3779B97F4A7C15.
 * A v above 0 is stored as its lowest code at least. What is not finite is
 * stored as NaN and leaves its block's scale alone.
 *
 * Tensors are numbered within their list: two lists of one step want two seeds.
 * A captured call keeps its numbers (lr, t and so its bias corrections, seed,
 * grad_scale) and its addresses: a replay is that step t again, on the values
 * that the tensors hold then.
 *
 * beta1, beta2 in [0, 1), eps >= 0, t >= 1, max_grad_norm >= 0. Scratch: partial
 * sums of the norm (needed with max_grad_norm > 0 or grad_norm). */
typedef struct gpt2_adamw_tensor {
    float* master;
    void* param_bf16;
    const void* grad;
    void* m;
    void* v;
    uint8_t* m_scale;
    uint8_t* v_scale;
    int64_t n;
    float weight_decay;
} gpt2_adamw_tensor;
size_t gpt2_op_adamw_many_scratch(const gpt2_adamw_tensor* tensors, int n_tensors);
int gpt2_op_adamw_many(const gpt2_adamw_tensor* tensors, int n_tensors, int grad_dtype, int bits, float lr,
                       float beta1, float beta2, float eps, float grad_scale, float max_grad_norm, float* grad_norm,
                       int t, uint64_t seed, void* scratch, size_t scratch_bytes, void* stream);

/* The values of 8-bit moments of the tensors, in dtype (bf16 holds every one
 * of them exactly, down to its subnormals): m_values[i] and v_values[i] (host
 * arrays of device pointers) receive tensors[i].n values each. Of the tensors,
 * m, v, m_scale, v_scale and n are read. */
int gpt2_op_adamw_many_states(const gpt2_adamw_tensor* tensors, void* const* m_values, void* const* v_values,
                              int n_tensors, int dtype, void* stream);

/* Failure-path testing of the bounded device waits (the design's failure
 * detection: a wait that runs out sets a status bit and the kernel returns;
 * nothing traps or hangs).
 * gpt2_debug_set_wait_limit: the bound, in SM clock cycles, of every
 * mbarrier wait of the tensor-core GEMM, the attention kernels and the
 * classifier on the current device; cycles <= 0 restores the default
 * (about 2 s). Takes effect for kernels launched after it returns; must not
 * be called while such kernels run.
 * gpt2_debug_stall_matmul: on != 0 makes every tensor-core GEMM launched
 * afterwards on the current device wait, before its first product, on a
 * barrier that nothing arrives at. The wait runs out after the bound above;
 * the kernel then sets the timeout bit (2) of its status word, stops its
 * other warps, waits (bounded) for its copies in flight, frees its tensor
 * memory and returns, leaving its output unwritten; the model's calls
 * report GPT2_ERR_TIMEOUT. on = 0 restores normal operation.
 * Both return GPT2_OK or GPT2_ERR_CUDA. Test hooks, not for the hot path. */
int gpt2_debug_set_wait_limit(int64_t cycles);
int gpt2_debug_stall_matmul(int on);

/* gpt2_debug_matmul_pair: on = 1 (the default) routes the plain bf16
 * matmuls with M >= 512 and one k-range per tile (no GELU epilogue) to the
 * CTA-pair kernel when N >= 1024, or when N is 384 to 960, a multiple of 192,
 * and K is 2048 to 16384 (192-wide pair tiles); the pair kernel issues one M = 256
 * tensor-core product for two neighbouring SMs (tcgen05 .cta_group::2) so
 * that each SM loads half of the B tile; on = 2 routes the GELU and GELU-gradient matmuls of that size there
 * too; 0 keeps every matmul on the one-CTA kernel. Process-wide; takes effect
 * for matmuls launched after it returns (a captured step graph keeps the
 * kernels it was captured with); on > 2 also sets the number of two-CTA
 * clusters launched (else the number the device keeps resident). Returns
 * the number of clusters the pair kernel launches (on != 0) or 0. A switch
 * for measurements and tests, not needed in normal use. */
int gpt2_debug_matmul_pair(int on);

/* gpt2_debug_linear_classifier_piece: the bytes that a piece of dz may take in
 * gpt2_op_linear_classifier_backward (and its scratch call), instead of 1 GB;
 * bytes <= 0 restores that. Process-wide, for measurements and tests: not
 * between a scratch call and the call that uses the scratch. Returns GPT2_OK. */
int gpt2_debug_linear_classifier_piece(int64_t bytes);

#ifdef __cplusplus
}
#endif
#endif /* GPT2_OPS_H */
