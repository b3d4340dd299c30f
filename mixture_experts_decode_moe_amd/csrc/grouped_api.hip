// Host side of the grouped products and the MXFP4 conversions: argument
// checks, then one launch (two for a split dw, whose parts take the only
// workspace here).  Nothing keeps state or allocates.
#include <stdint.h>

#include "grouped.h"

using namespace moe;

namespace {

constexpr int32_t kMaxWidth = 65536;         // N and K
constexpr int32_t kMaxRows = INT32_MAX / 2;  // as moe_permute
constexpr int64_t kMaxStride = 1 << 24;      // of 16-bit operands: a step's rows are addressed in 32 bits
constexpr int kTileRows = 128, kTileCols = 64;  // the smallest tiles of the kernels that count so

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int64_t type_size(int32_t t) { return t == MOE_T_F32 ? 4 : 2; }

bool known_type(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_F16 || t == MOE_T_F32; }

// What every grouped product asks of its groups and sizes.
int check_groups(int32_t n_rows, int32_t E, int32_t N, int32_t K, const int32_t *offsets) {
  if (n_rows < 0 || E <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || N > kMaxWidth || K > kMaxWidth || n_rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits, whatever the offsets hold
  const int64_t tiles = E * (n_rows / kTileRows + static_cast<int64_t>(1));
  const int64_t cols = (N > K ? N : K) / kTileCols + 1;
  return tiles * cols > INT32_MAX / 2 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows that are gathered from T source rows.
int check_rows(const void *x, int32_t T, int32_t n_rows, const int32_t *row_tok, const float *row_w) {
  if (T < 0 || (!row_tok && n_rows > T)) return MOE_ERR_INVALID_ARG;
  if (n_rows > 0 && !x) return MOE_ERR_INVALID_ARG;
  if (!aligned(row_tok, 4) || !aligned(row_w, 4)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// A 16-bit operand's rows: whole 16-byte pieces.
int check_operand(const void *p, int64_t ld, int32_t width) {
  if (ld < width || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  return ld % 8 || ld > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_16bit(int32_t type, int32_t out_type, int32_t N, int32_t K) {
  if (type != MOE_T_BF16 && type != MOE_T_F16) return known_type(type) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (!known_type(out_type)) return MOE_ERR_INVALID_ARG;
  if (out_type != type && out_type != MOE_T_F32) return MOE_ERR_UNSUPPORTED;
  return N % 8 || K % 8 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

GroupedArgs grouped_args(int32_t kind, int32_t type, int32_t out_type, int32_t T, int32_t n_rows, int32_t E,
                         const int32_t *offsets, const int32_t *row_tok, const float *row_w, void *out,
                         int64_t out_ld) {
  GroupedArgs a{};
  a.kind = kind;
  a.type = type;
  a.out_type = out_type;
  a.T = T;
  a.n_rows = n_rows;
  a.E = E;
  a.offsets = offsets;
  a.row_tok = row_tok;
  a.row_w = row_w;
  a.out = static_cast<char *>(out);
  a.out_ld = out_ld;
  a.splits = 1;
  return a;
}

int check_mx(const moe_mx_rows *m) {
  return m && m->q && m->s && aligned(m->q, 16) && aligned(m->s, 16) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int moe_mx_quantize(const void *x, int32_t x_type, int64_t x_ld, int32_t rows, int32_t cols, uint8_t *q, uint8_t *s,
                    void *stream) {
  if (rows < 0 || cols <= 0 || !known_type(x_type) || x_ld < cols) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !s || !aligned(x, type_size(x_type)) || !aligned(q, 16) || !aligned(s, 16)) return MOE_ERR_INVALID_ARG;
  if (cols > INT32_MAX - kMxPad) return MOE_ERR_UNSUPPORTED;
  return hip_status(launch_mx_quantize(MxQuantArgs{x, x_ld, rows, cols, x_type, q, s}, static_cast<hipStream_t>(stream)));
}

int moe_mx_dequantize(const uint8_t *q, const uint8_t *s, int32_t rows, int32_t cols, void *out, int32_t out_type,
                      int64_t out_ld, void *stream) {
  if (rows < 0 || cols <= 0 || !known_type(out_type) || out_ld < cols) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!out || !q || !s || !aligned(out, type_size(out_type)) || !aligned(q, 16) || !aligned(s, 16))
    return MOE_ERR_INVALID_ARG;
  if (cols > INT32_MAX - kMxPad) return MOE_ERR_UNSUPPORTED;
  return hip_status(
      launch_mx_dequantize(MxDequantArgs{q, s, rows, cols, out_type, out, out_ld}, static_cast<hipStream_t>(stream)));
}

int moe_mx_grouped_gemm(const moe_mx_rows *x, int32_t T, int32_t n_rows, const moe_mx_rows *w, const moe_mx_rows *up,
                        int32_t E, int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_tok,
                        const float *row_w, void *out, int32_t out_type, int64_t out_ld, void *stream) {
  int rc = check_groups(n_rows, E, N, K, offsets);
  if (rc != MOE_OK) return rc;
  if (!known_type(out_type) || out_ld < N) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if ((rc = check_mx(x)) != MOE_OK || (rc = check_mx(w)) != MOE_OK || (up && (rc = check_mx(up)) != MOE_OK)) return rc;
  if ((rc = check_rows(x->q, T, n_rows, row_tok, row_w)) != MOE_OK) return rc;
  if (!out || !aligned(out, type_size(out_type))) return MOE_ERR_INVALID_ARG;
  GroupedArgs a = grouped_args(kGroupedMx, 0, out_type, T, n_rows, E, offsets, row_tok, row_w, out, out_ld);
  const int32_t kp = (K + kMxPad - 1) / kMxPad * kMxPad;
  a.a = reinterpret_cast<const char *>(w->q);
  a.as = reinterpret_cast<const char *>(w->s);
  a.a2 = up ? reinterpret_cast<const char *>(up->q) : nullptr;
  a.as2 = up ? reinterpret_cast<const char *>(up->s) : nullptr;
  a.b = reinterpret_cast<const char *>(x->q);
  a.bs = reinterpret_cast<const char *>(x->s);
  a.a_ld = a.b_ld = kp / 2;
  a.a_expert = static_cast<int64_t>(N) * (kp / 2);
  a.s_ld = kp / kMxBlock;
  a.na = N;
  a.red = kp / 2;
  return hip_status(launch_grouped(a, static_cast<hipStream_t>(stream)));
}

int moe_grouped_gemm(const void *x, int64_t x_ld, int32_t T, int32_t n_rows, const void *w, int32_t type, int32_t E,
                     int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_tok, const float *row_w,
                     void *out, int32_t out_type, int64_t out_ld, void *stream) {
  int rc = check_groups(n_rows, E, N, K, offsets);
  if (rc == MOE_OK) rc = check_16bit(type, out_type, N, K);
  if (rc != MOE_OK) return rc;
  if (n_rows == 0) return MOE_OK;
  if ((rc = check_rows(x, T, n_rows, row_tok, row_w)) != MOE_OK) return rc;
  if (!w || !aligned(w, 16) || !out) return MOE_ERR_INVALID_ARG;
  if ((rc = check_operand(x, x_ld, K)) != MOE_OK || (rc = check_operand(out, out_ld, N)) != MOE_OK) return rc;
  GroupedArgs a = grouped_args(kGroupedFwd, type, out_type, T, n_rows, E, offsets, row_tok, row_w, out, out_ld);
  a.a = static_cast<const char *>(w);
  a.b = static_cast<const char *>(x);
  a.a_ld = 2 * static_cast<int64_t>(K);
  a.b_ld = 2 * x_ld;
  a.a_expert = static_cast<int64_t>(N) * a.a_ld;
  a.na = N;
  a.red = 2 * K;
  return hip_status(launch_grouped(a, static_cast<hipStream_t>(stream)));
}

int moe_grouped_gemm_dx(const void *dy, int64_t dy_ld, int32_t n_rows, const void *w, int32_t type, int32_t E,
                        int32_t N, int32_t K, const int32_t *offsets, void *dx, int32_t out_type, int64_t dx_ld,
                        void *stream) {
  int rc = check_groups(n_rows, E, N, K, offsets);
  if (rc == MOE_OK) rc = check_16bit(type, out_type, N, K);
  if (rc != MOE_OK) return rc;
  if (n_rows == 0) return MOE_OK;
  if (!dy || !w || !aligned(w, 16) || !dx) return MOE_ERR_INVALID_ARG;
  if ((rc = check_operand(dy, dy_ld, N)) != MOE_OK || (rc = check_operand(dx, dx_ld, K)) != MOE_OK) return rc;
  GroupedArgs a = grouped_args(kGroupedDx, type, out_type, n_rows, n_rows, E, offsets, nullptr, nullptr, dx, dx_ld);
  a.a = static_cast<const char *>(w);
  a.b = static_cast<const char *>(dy);
  a.a_ld = 2 * static_cast<int64_t>(K);
  a.b_ld = 2 * dy_ld;
  a.a_expert = static_cast<int64_t>(N) * a.a_ld;
  a.na = K;
  a.red = N;
  return hip_status(launch_grouped(a, static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_gemm_dw_workspace_bytes(int32_t n_rows, int32_t E, int32_t N, int32_t K) {
  if (n_rows < 0 || E <= 0 || N <= 0 || K <= 0 || E > 1024 || N > kMaxWidth || K > kMaxWidth) return 0;
  const int32_t parts = grouped_dw_splits(n_rows, E, N, K);
  return parts > 1 ? align_up(static_cast<size_t>(parts) * E * N * K * sizeof(float), 256) : 0;
}

int moe_grouped_gemm_dw(const void *dy, int64_t dy_ld, const void *x, int64_t x_ld, int32_t T, int32_t n_rows,
                        int32_t type, int32_t E, int32_t N, int32_t K, const int32_t *offsets,
                        const int32_t *row_tok, void *dw, int32_t out_type, void *ws, size_t ws_bytes, void *stream) {
  int rc = check_groups(n_rows, E, N, K, offsets);
  if (rc == MOE_OK) rc = check_16bit(type, out_type, N, K);
  if (rc == MOE_OK) rc = check_rows(x, T, n_rows, row_tok, nullptr);
  if (rc != MOE_OK) return rc;
  if (!dw || !aligned(dw, 16) || (n_rows > 0 && !dy)) return MOE_ERR_INVALID_ARG;
  if (n_rows > 0 &&
      ((rc = check_operand(dy, dy_ld, N)) != MOE_OK || (rc = check_operand(x, x_ld, K)) != MOE_OK))
    return rc;
  GroupedArgs a = grouped_args(kGroupedDw, type, out_type, T, n_rows, E, offsets, row_tok, nullptr, dw, K);
  a.a = static_cast<const char *>(x);
  a.b = static_cast<const char *>(dy);
  a.a_ld = 2 * x_ld;
  a.b_ld = 2 * dy_ld;
  a.na = K;
  a.nb = N;
  const size_t need = moe_grouped_gemm_dw_workspace_bytes(n_rows, E, N, K);
  if (need > 0) {
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return MOE_ERR_WORKSPACE;
    a.splits = grouped_dw_splits(n_rows, E, N, K);
    a.parts = static_cast<char *>(ws);
  }
  return hip_status(launch_grouped(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
