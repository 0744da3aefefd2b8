// C entry points of the gated feed-forward block (include/lpgemm_ffn.h).
#include "ffn.hpp"
#include "few_rows.hpp"

namespace lpgemm {
std::atomic<int> g_forced_ffn{-1};
}  // namespace lpgemm

using namespace lpgemm;

namespace {

bool is_16bit(lpgemm_type t) { return t == LPGEMM_F16 || t == LPGEMM_BF16; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

bool bad_sizes(int64_t M, int64_t D, int64_t F) { return M < 0 || D < 0 || F < 0 || M > INT32_MAX; }
bool bad_shape(int64_t M, int64_t D, int64_t F) {
  if (D % 8 != 0 || F % 8 != 0 || D > LPGEMM_MAX_D_FFN || F > LPGEMM_MAX_D_FFN || M > INT32_MAX - 256) return true;
  const int64_t m = (M + 63) / 64, d = (D + 63) / 64, f = (2 * F + 63) / 64, most = (int64_t)1 << 24;
  return m * f >= most || m * d >= most || f * d >= most;
}
bool bad_stride(int64_t stride, int64_t D) { return stride < D || stride % 8 != 0 || stride > LPGEMM_MAX_STRIDE; }

// Whether the forward pass runs its products on few_rows: a handful of rows, or
// small weights (us, both products, few_rows against tiles: 8 x 4096 x 14336 75
// and 77, 16 rows 85 and 78; 33 x 1024 x 2816 16.2 and 19.6, 64 rows 21.0 and
// 20.2).
bool few_rows_forward(int64_t M, int64_t D, int64_t F) {
  const int forced = forced_ffn();
  if (forced >= FFN_TILE_64 && forced <= FFN_TILE_256) return false;
  if (forced == FFN_FEW_ROWS) return M <= 16 * 65535;
  return M <= 8 || (M <= 48 && D * F <= (int64_t)4 << 20);
}

// The workspace's parts, in bytes from its start.
struct ForwardSpace {
  int64_t h, part, total;
  ForwardSpace(int64_t M, int64_t D, int64_t F, int cu_count) {
    h = 0;
    part = round256(2 * M * F);
    int64_t sums = 0;
    if (!few_rows_forward(M, D, F)) {
      const int64_t a = split_bytes(plan_tiles(JOB_GATED, M, 2 * F, D, cu_count), JOB_GATED, M, 2 * F);
      const int64_t b = split_bytes(plan_tiles(JOB_DOWN, M, D, F, cu_count), JOB_DOWN, M, D);
      sums = a > b ? a : b;
    }
    total = part + round256(sums);
  }
};
struct BackwardSpace {
  int64_t dgu, h, part, total;
  BackwardSpace(int64_t M, int64_t D, int64_t F, int cu_count) {
    dgu = 0;
    h = round256(4 * M * F);
    part = h + round256(2 * M * F);
    int64_t sums = 0;
    auto add = [&](int job, int64_t m, int64_t n, int64_t k) {
      const int64_t b = split_bytes(plan_tiles(job, m, n, k, cu_count), job, m, n);
      if (b > sums) sums = b;
    };
    add(JOB_GATED_GRAD, M, F, D);
    add(JOB_DX, M, D, 2 * F);
    add(JOB_DW, 2 * F, D, M);
    add(JOB_DW, D, F, M);
    total = part + round256(sums);
  }
};

template <typename Space>
int64_t workspace_bytes_of(int64_t M, int64_t D, int64_t F) {
  if (bad_sizes(M, D, F) || bad_shape(M, D, F)) return -1;
  DeviceInfo dev;
  if (current_device(dev) != LPGEMM_SUCCESS) return -1;
  return Space(M, D, F, dev.cu_count).total;
}

// The forward pass.  h goes into the second product as T, which its matrix
// instructions take: y is then 0.0023 from 64 bits in bf16 and 0.0003 in fp16
// (root mean square, of y's), with h in binary32 0.0017 and 0.0002, most of which is
// y's own rounding.  h in two parts, the rounded one and the rest, would take the
// product's time twice (363 of 1130 us at 4096 x 4096 x 14336 bf16).
template <typename T>
lpgemm_status forward(int64_t M, int64_t D, int64_t F, int activation, const void* X, int64_t x_stride,
                      const void* w_gate_up, const void* w_down, void* GU, void* Y, uint8_t* ws, int64_t ws_bytes,
                      int cu_count, hipStream_t stream) {
  const ForwardSpace space(M, D, F, cu_count);
  uint8_t* const h = ws + space.h;
  lpgemm_status st = LPGEMM_SUCCESS;
  if (few_rows_forward(M, D, F)) {
    FewRowsArgs p{};
    p.X = static_cast<const uint8_t*>(X);
    p.W = static_cast<const uint8_t*>(w_gate_up);
    p.C = h;
    p.GU = static_cast<uint8_t*>(GU);
    p.out_type = kIsF16<T> ? LPGEMM_F16 : LPGEMM_BF16;
    p.M = (int)M;
    p.N = (int)(2 * F);
    p.F = (int)F;
    p.K = (int)D;
    p.activation = activation;
    p.x_stride = (int)(2 * x_stride);
    p.row_bytes = (int)(2 * D);
    if (F > 0) st = run_few_rows<T>(p, 0, cu_count, stream);
    if (st != LPGEMM_SUCCESS || D == 0) return st;
    p.X = h;
    p.W = static_cast<const uint8_t*>(w_down);
    p.C = static_cast<uint8_t*>(Y);
    p.GU = nullptr;
    p.N = (int)D;
    p.F = 0;
    p.K = (int)F;
    p.x_stride = p.row_bytes = (int)(2 * F);
    return run_few_rows<T>(p, 0, cu_count, stream);
  }
  float* const part = reinterpret_cast<float*>(ws + space.part);
  const int64_t part_bytes = ws_bytes - space.part;
  TileArgs p{};
  p.A = static_cast<const uint8_t*>(X);
  p.B = static_cast<const uint8_t*>(w_gate_up);
  p.a_stride = 2 * x_stride;
  p.b_stride = 2 * D;
  p.H = h;
  p.GU = static_cast<uint8_t*>(GU);
  p.out_type = kIsF16<T> ? LPGEMM_F16 : LPGEMM_BF16;
  p.activation = activation;
  p.M = (int)M;
  p.N = (int)(2 * F);
  p.F = (int)F;
  p.K = (int)D;
  if (F > 0) st = run_tile<T>(JOB_GATED, p, part, part_bytes, cu_count, stream);
  if (st != LPGEMM_SUCCESS || D == 0) return st;
  TileArgs q{};
  q.A = h;
  q.B = static_cast<const uint8_t*>(w_down);
  q.a_stride = q.b_stride = 2 * F;
  q.C = static_cast<uint8_t*>(Y);
  q.out_type = kIsF16<T> ? LPGEMM_F16 : LPGEMM_BF16;
  q.M = (int)M;
  q.N = (int)D;
  q.K = (int)F;
  return run_tile<T>(JOB_DOWN, q, part, part_bytes, cu_count, stream);
}

// The gradients.  dg, du and h as T: the same distances from 64 bits as in the
// forward pass; two parts of each would take 1930 of 2500 us twice at that size.
template <typename T>
lpgemm_status backward(int64_t M, int64_t D, int64_t F, int activation, const void* dY, int64_t dy_stride,
                       const void* X, int64_t x_stride, const void* w_gate_up, const void* w_down, const void* GU,
                       lpgemm_type grad_type, void* dX, void* dw_gate_up, void* dw_down, uint8_t* ws,
                       int64_t ws_bytes, int cu_count, hipStream_t stream) {
  const BackwardSpace space(M, D, F, cu_count);
  uint8_t *const dgu = ws + space.dgu, *const h = ws + space.h;
  float* const part = reinterpret_cast<float*>(ws + space.part);
  const int64_t part_bytes = ws_bytes - space.part;
  const int own_type = kIsF16<T> ? LPGEMM_F16 : LPGEMM_BF16;
  lpgemm_status st = LPGEMM_SUCCESS;
  if (M > 0 && F > 0) {
    TileArgs p{};
    p.A = static_cast<const uint8_t*>(dY);
    p.B = static_cast<const uint8_t*>(w_down);
    p.a_stride = 2 * dy_stride;
    p.b_stride = 2 * F;
    p.H = h;
    p.GU = const_cast<uint8_t*>(static_cast<const uint8_t*>(GU));
    p.DGU = dgu;
    p.activation = activation;
    p.M = (int)M;
    p.N = p.F = (int)F;
    p.K = (int)D;
    st = run_tile<T>(JOB_GATED_GRAD, p, part, part_bytes, cu_count, stream);
  }
  if (st == LPGEMM_SUCCESS && dX && M > 0) {
    TileArgs p{};
    p.A = dgu;
    p.B = static_cast<const uint8_t*>(w_gate_up);
    p.a_stride = 4 * F;
    p.b_stride = 2 * D;
    p.C = static_cast<uint8_t*>(dX);
    p.out_type = own_type;
    p.M = (int)M;
    p.N = (int)D;
    p.K = (int)(2 * F);
    st = run_tile<T>(JOB_DX, p, part, part_bytes, cu_count, stream);
  }
  if (st == LPGEMM_SUCCESS && dw_gate_up && F > 0) {
    TileArgs p{};
    p.A = dgu;
    p.B = static_cast<const uint8_t*>(X);
    p.a_stride = 4 * F;
    p.b_stride = 2 * x_stride;
    p.C = static_cast<uint8_t*>(dw_gate_up);
    p.out_type = grad_type;
    p.M = (int)(2 * F);
    p.N = (int)D;
    p.K = (int)M;
    st = run_tile<T>(JOB_DW, p, part, part_bytes, cu_count, stream);
  }
  if (st == LPGEMM_SUCCESS && dw_down && F > 0) {
    TileArgs p{};
    p.A = static_cast<const uint8_t*>(dY);
    p.B = h;
    p.a_stride = 2 * dy_stride;
    p.b_stride = 2 * F;
    p.C = static_cast<uint8_t*>(dw_down);
    p.out_type = grad_type;
    p.M = (int)D;
    p.N = (int)F;
    p.K = (int)M;
    st = run_tile<T>(JOB_DW, p, part, part_bytes, cu_count, stream);
  }
  return st;
}

}  // namespace

extern "C" {

int lpgemm_ffn_config_count(void) { return FFN_CONFIG_COUNT; }

int lpgemm_force_ffn_config(int config) {
  return g_forced_ffn.exchange(config >= 0 && config < FFN_CONFIG_COUNT ? config : -1);
}

int64_t lpgemm_gated_ffn_workspace(int64_t M, int64_t D, int64_t F) { return workspace_bytes_of<ForwardSpace>(M, D, F); }

int64_t lpgemm_gated_ffn_backward_workspace(int64_t M, int64_t D, int64_t F) {
  return workspace_bytes_of<BackwardSpace>(M, D, F);
}

lpgemm_status lpgemm_gated_ffn(int64_t M, int64_t D, int64_t F, lpgemm_type type, lpgemm_activation activation,
                               const void* X, int64_t x_stride, const void* W_gate_up, const void* W_down, void* GU,
                               void* Y, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (bad_sizes(M, D, F) || !is_16bit(type) || (activation != LPGEMM_SILU && activation != LPGEMM_GELU) ||
      workspace_bytes < 0)
    return LPGEMM_ERROR_INVALID_VALUE;
  if (bad_shape(M, D, F) || bad_stride(x_stride, D)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (M == 0 || (D == 0 && (F == 0 || !GU))) return LPGEMM_SUCCESS;
  const bool products = D > 0 && F > 0;
  if ((D > 0 && !Y) || (products && (!X || !W_gate_up || !W_down)) || (F > 0 && !workspace))
    return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(Y) || !aligned16(GU) || !aligned256(workspace) ||
      (products && (!aligned16(X) || !aligned16(W_gate_up) || !aligned16(W_down))))
    return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  const lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  if (workspace_bytes < ForwardSpace(M, D, F, dev.cu_count).total) return LPGEMM_ERROR_INVALID_VALUE;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  return type == LPGEMM_F16
             ? forward<TypeF16>(M, D, F, activation, X, x_stride, W_gate_up, W_down, GU, Y, ws, workspace_bytes, dev.cu_count, stream)
             : forward<TypeBF16>(M, D, F, activation, X, x_stride, W_gate_up, W_down, GU, Y, ws, workspace_bytes, dev.cu_count, stream);
}

lpgemm_status lpgemm_gated_ffn_backward(int64_t M, int64_t D, int64_t F, lpgemm_type type,
                                        lpgemm_activation activation, const void* dY, int64_t dy_stride,
                                        const void* X, int64_t x_stride, const void* W_gate_up, const void* W_down,
                                        const void* GU, lpgemm_type grad_type, void* dX, void* dW_gate_up,
                                        void* dW_down, void* workspace, int64_t workspace_bytes,
                                        hipStream_t stream) {
  if (bad_sizes(M, D, F) || !is_16bit(type) || (activation != LPGEMM_SILU && activation != LPGEMM_GELU) ||
      (grad_type != LPGEMM_F32 && grad_type != type) || workspace_bytes < 0)
    return LPGEMM_ERROR_INVALID_VALUE;
  if (bad_shape(M, D, F) || bad_stride(x_stride, D) || bad_stride(dy_stride, D)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (D == 0 || (M == 0 && F == 0) || (!dX && !dW_gate_up && !dW_down)) return LPGEMM_SUCCESS;
  const bool products = M > 0 && F > 0;
  if (products && (!dY || !X || !W_gate_up || !W_down || !GU || !workspace)) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(dX) || !aligned16(dW_gate_up) || !aligned16(dW_down) ||
      (products && (!aligned16(dY) || !aligned16(X) || !aligned16(W_gate_up) || !aligned16(W_down) || !aligned16(GU) ||
                    !aligned256(workspace))))
    return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  const lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  if (products && workspace_bytes < BackwardSpace(M, D, F, dev.cu_count).total) return LPGEMM_ERROR_INVALID_VALUE;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  return type == LPGEMM_F16
             ? backward<TypeF16>(M, D, F, activation, dY, dy_stride, X, x_stride, W_gate_up, W_down, GU, grad_type, dX,
                                 dW_gate_up, dW_down, ws, workspace_bytes, dev.cu_count, stream)
             : backward<TypeBF16>(M, D, F, activation, dY, dy_stride, X, x_stride, W_gate_up, W_down, GU, grad_type, dX,
                                  dW_gate_up, dW_down, ws, workspace_bytes, dev.cu_count, stream);
}

}  // extern "C"
