/*
 * lpgemm: 4-bit weights with group scales, and the gated feed-forward block,
 * for one AMD Instinct MI355X (gfx950).
 *
 *   lpgemm_quantize_w4, lpgemm_dequantize_w4   16-bit weights to 4-bit codes,
 *                             one scale (and zero point) per group along k
 *   lpgemm_w4                 C = X . W^T for 16-bit rows and such weights
 *   lpgemm_gated_w4           act(X . G^T) * (X . U^T) for such weights
 *   lpgemm_gated_ffn          (act(X . G^T) * (X . U^T)) . D^T, 16-bit weights
 *   lpgemm_gated_ffn_backward its gradients
 *
 * The conventions of lpgemm.h and lpgemm_moe.h hold: device pointers owned by
 * the caller, work enqueued on `stream` without synchronising, nothing
 * allocated, no state kept between calls, the same status codes checked on the
 * host in the same order (sizes, shape rules, empty problem, NULL pointers,
 * alignment, then the device, the workspace's size and the launch).  Weights are N rows
 * of K values.  Outputs must not overlap inputs, each other or the workspace.
 *
 * Sixteen-bit tensors are binary16 or bfloat16; `type` is the type of every
 * 16-bit tensor of a call.  Sums are held in binary32; their order depends on
 * the sizes and the device's number of compute units only, so equal calls on
 * equal devices give equal bits.  Infinities and NaN go the way the formulas
 * send them, but for rows of X at lpgemm_w4.
 *
 * Workspaces are scratch: a call writes every byte that it reads, nothing has
 * to be cleared, and nothing is kept from one call for the next.  Calls that
 * share one must not overlap in time.
 */
#ifndef LPGEMM_FFN_H
#define LPGEMM_FFN_H

#include "lpgemm_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The activation of a gated block:
 *   LPGEMM_SILU  g / (1 + exp(-g))
 *   LPGEMM_GELU  g (1 + tanh(z)) / 2 = g / (1 + exp(-2 z)),
 *                z = sqrt(2 / pi) (g + 0.044715 g^3) */
typedef enum lpgemm_activation {
    LPGEMM_SILU = 0,
    LPGEMM_GELU = 1
} lpgemm_activation;

/* Weights in 4 bits.  W is N x K; `group` consecutive values of a row share a
 * scale and, where there are zero points, a zero:
 *   W[n][k] = (code[n][k] - zero[n][k / group]) * scale[n][k / group].
 * Codes are signed (-8..7), two to a byte along k, the even k in the low
 * nibble, two's complement: N rows of K / 2 bytes, the operand layout of
 * lpgemm_i4.  Scales and zeros are N x (K / group) values of a 16-bit type;
 * zeros may hold any value, integers or not, and NULL stands for zeros of 0.
 * group is 32, 64, 128 or 256 and divides K; K is at most LPGEMM_MAX_K_W4. */
#define LPGEMM_MAX_K_W4 1048576

/* W of `type` to codes, scales and (zeros not NULL) zeros.  For each group,
 * in binary32 and rounded to nearest even:
 *   without zeros: s = type(max |w| / 7), code = clamp(rne(w / s), -8, 7);
 *   with zeros: lo = min(0, min w), hi = max(0, max w), s = type((hi - lo) / 15),
 *     zero = clamp(-8 - rne(lo / s), -8, 7), an integer,
 *     code = clamp(rne(w / s) + zero, -8, 7).
 * A group whose max |w| (hi - lo) is below 2^-100, or whose s is 0, gets s = 0
 * and codes and zero 0; one with an infinity or a NaN gets s = NaN and codes
 * and zero 0; where hi - lo leaves binary32 (bfloat16 near its largest), s is
 * an infinity, codes and zero 0.
 * w_stride in elements, at least K, a multiple of 8.  Pointers 16-byte
 * aligned, scales and zeros 2-byte.  N = 0 or K = 0 is a no-op. */
lpgemm_status lpgemm_quantize_w4(int64_t N, int64_t K, int64_t group, lpgemm_type type, const void *W,
                                 int64_t w_stride, uint8_t *codes, void *scales, void *zeros,
                                 hipStream_t stream);

/* The values the codes stand for: Y = N x K of `out_type` (any of the three),
 * (code - zero) * scale, each operation rounded to binary32, then once to
 * out_type.  `type`: that of scales and zeros. */
lpgemm_status lpgemm_dequantize_w4(int64_t N, int64_t K, int64_t group, lpgemm_type type, const uint8_t *codes,
                                   const void *scales, const void *zeros, lpgemm_type out_type, void *Y,
                                   hipStream_t stream);

/* C = X . W^T: X M rows of K values of `type` (x_stride in elements, at least
 * K, a multiple of 8, at most LPGEMM_MAX_STRIDE), W in 4 bits with scales and
 * zeros of the same type, C M x N of `out_type`.  Up to LPGEMM_W4_EXACT_M rows
 * the weights enter the sums exactly: C[m][n] = sum over groups of scale * (sum
 * of x * code - zero * sum of x), every sum in binary32.  (The kernels sum x *
 * (code + 24) and take 24 times the sum of x off: a row of X with an infinity or
 * a NaN gives NaN, and so may one with magnitudes above 2^115.)  Beyond, each
 * weight is first rounded once to `type`, into the workspace, and the product is
 * that of 16-bit weights; a weight row that may hold values past the type's range
 * is divided by a power of two before and its sums multiplied by it after, so
 * that such weights stay finite.  (Exact weights for more rows: calls of up to
 * LPGEMM_W4_EXACT_M rows each.)  M = 0 or N = 0 is a no-op; K = 0 sets C to 0.
 * X, codes and C 16-byte aligned, scales and zeros 2-byte.  M is at most
 * LPGEMM_MAX_M_W4, N at most LPGEMM_MAX_N_W4, with below 2^24 tiles of 64 x 64 of
 * C (UNSUPPORTED_SHAPE otherwise).
 * `workspace`, 256-byte aligned, holds at least lpgemm_w4_workspace(M, N, K,
 * group, 0) bytes (0 up to LPGEMM_W4_SHORT_M rows; -1 for sizes out of range or
 * no device), which depends on the current device's number of compute units;
 * INVALID_VALUE where it is missing or too small. */
#define LPGEMM_MAX_STRIDE 2097152
#define LPGEMM_MAX_M_W4 134217728
#define LPGEMM_MAX_N_W4 16777216
#define LPGEMM_W4_SHORT_M 4
#define LPGEMM_W4_EXACT_M 384
int64_t lpgemm_w4_workspace(int64_t M, int64_t N, int64_t K, int64_t group, int gated);
lpgemm_status lpgemm_w4(int64_t M, int64_t N, int64_t K, int64_t group, lpgemm_type type, const void *X,
                        int64_t x_stride, const uint8_t *codes, const void *scales, const void *zeros,
                        lpgemm_type out_type, void *C, void *workspace, int64_t workspace_bytes,
                        hipStream_t stream);

/* H = act(X . G^T) * (X . U^T), M x F of out_type, where the first F of the 2 F
 * weight rows are G and the others U; both products, the activation and the
 * product of the two in binary32, rounded once.  Otherwise as lpgemm_w4 with
 * N = 2 F (and the workspace of gated = 1). */
lpgemm_status lpgemm_gated_w4(int64_t M, int64_t F, int64_t K, int64_t group, lpgemm_type type,
                              lpgemm_activation activation, const void *X, int64_t x_stride,
                              const uint8_t *codes, const void *scales, const void *zeros, lpgemm_type out_type,
                              void *H, void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* The gated feed-forward block with 16-bit weights, everything of `type`:
 *   [g u] = X . W_gate_up^T    X: M x D, W_gate_up: 2 F x D, gate rows first
 *   h = act(g) * u             from the binary32 sums, rounded to `type` (past
 *                              binary16's 65504 to an infinity)
 *   Y = h . W_down^T           W_down: D x F, Y: M x D
 * GU, if not NULL, receives [g u] (M x 2 F, each rounded once), which the
 * backward pass reads.  D and F are multiples of 8, at most LPGEMM_MAX_D_FFN;
 * M at most 2^31 - 257, with below 2^24 tiles of 64 x 64 of each M x 2 F, M x D
 * and 2 F x D matrix.  x_stride as for lpgemm_w4.  Pointers 16-byte aligned.
 * M = 0 is a no-op; F = 0 sets Y to 0, D = 0 sets GU to 0.
 * `workspace`, 256-byte aligned, holds at least
 * lpgemm_gated_ffn_workspace(M, D, F) bytes, which depends on the current
 * device's number of compute units (-1 for sizes out of range or no device). */
#define LPGEMM_MAX_D_FFN 262144
int64_t lpgemm_gated_ffn_workspace(int64_t M, int64_t D, int64_t F);
lpgemm_status lpgemm_gated_ffn(int64_t M, int64_t D, int64_t F, lpgemm_type type, lpgemm_activation activation,
                               const void *X, int64_t x_stride, const void *W_gate_up, const void *W_down,
                               void *GU, void *Y, void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* The block's gradients, from dY (M x D, dy_stride as x_stride) and what the
 * forward pass had and kept:
 *   dh = dY . W_down, h = act(g) * u, du = dh act(g), dg = dh u act'(g)
 *   dX = [dg du] . W_gate_up            M x D, of `type`
 *   dW_gate_up = [dg du]^T . X          2 F x D, of grad_type
 *   dW_down = dY^T . h                  D x F, of grad_type
 * h, dg and du are formed in binary32 from GU and the binary32 sums dh and
 * rounded once to `type`, as operands of the products behind them.  grad_type
 * is LPGEMM_F32 or `type`.  Any of dX, dW_gate_up and dW_down may be NULL: it
 * is then not computed.  M = 0 sets the weights' gradients to 0, F = 0 sets dX
 * to 0; D = 0 is a no-op. */
int64_t lpgemm_gated_ffn_backward_workspace(int64_t M, int64_t D, int64_t F);
lpgemm_status lpgemm_gated_ffn_backward(int64_t M, int64_t D, int64_t F, lpgemm_type type,
                                        lpgemm_activation activation, const void *dY, int64_t dy_stride,
                                        const void *X, int64_t x_stride, const void *W_gate_up,
                                        const void *W_down, const void *GU, lpgemm_type grad_type, void *dX,
                                        void *dW_gate_up, void *dW_down, void *workspace,
                                        int64_t workspace_bytes, hipStream_t stream);

/* Ablation hook, as lpgemm_force_config: every call takes its kernels by its
 * sizes; lpgemm_force_ffn_config(c) pins one for every later call in the process
 * that can run it, or restores the choice for any other value (-1), and returns
 * the previous setting.  0, 1, 2: the block's products on tiles of 64, 128 and
 * 256 rows; 3: its forward pass and the 4-bit products on the kernel for few
 * rows; 4, 5, 6: the 4-bit products on tiles of 32 and 64 rows and through
 * 16-bit weights (4-bit products of up to LPGEMM_W4_SHORT_M rows stay on the
 * kernel for few rows).  The sums' order depends on it, and with it the bits of
 * the results, and how large a workspace has to be: ask after setting it. */
int lpgemm_ffn_config_count(void);
int lpgemm_force_ffn_config(int config);

#ifdef __cplusplus
}
#endif

#endif /* LPGEMM_FFN_H */
