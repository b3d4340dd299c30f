// Arguments of the grouped products and of the MXFP4 conversions, shared by
// their host side and kernels.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMxBlock = 32;  // elements under one scale
constexpr int kMxPad = 128;   // rows are padded to a multiple of this

struct MxQuantArgs {
  const void *x;
  int64_t x_ld;
  int32_t rows, cols, type;
  uint8_t *q, *s;
};
hipError_t launch_mx_quantize(const MxQuantArgs &a, hipStream_t s);

struct MxDequantArgs {
  const uint8_t *q, *s;
  int32_t rows, cols, type;
  void *out;
  int64_t out_ld;
};
hipError_t launch_mx_dequantize(const MxDequantArgs &a, hipStream_t s);

// One grouped product.  The output tile is [b][a]: `a` is the operand whose
// rows become the contiguous output columns (the matrices; for dw: x), `b`
// the one whose rows become output rows (the grouped rows; for dw: dy).
enum GroupedKind : int32_t { kGroupedFwd, kGroupedDx, kGroupedDw, kGroupedMx };

struct GroupedArgs {
  int32_t kind, type, out_type;
  const char *a, *a2;    // matrices (and SwiGLU's up matrices); dw: x
  const char *b;         // rows; dw: dy
  const char *as, *as2, *bs;  // MXFP4 scales
  int64_t a_ld, b_ld;    // bytes a row
  int64_t a_expert;      // bytes a matrix (0 for dw)
  int32_t s_ld;          // MXFP4: scale bytes a row
  int32_t T, n_rows, E;
  int32_t na;            // output columns
  int32_t nb;            // dw: output rows (N)
  int32_t red;           // length of the reduction: bytes of a row (fwd, mx) or rows (dx); dw: per group
  const int32_t *offsets, *row_tok;
  const float *row_w;
  char *out;
  int64_t out_ld;        // elements
  int32_t splits;        // dw: parts of a group's rows (1: none)
  char *parts;           // dw with parts: float [splits][E][nb][na]
};
hipError_t launch_grouped(const GroupedArgs &a, hipStream_t s);
int32_t grouped_dw_splits(int32_t n_rows, int32_t E, int32_t N, int32_t K);
// fwd and mx with few rows an expert: the blocks such a launch has, and the
// launch, which wants fewer than 2^31
int64_t grouped_few_blocks(const GroupedArgs &a);
hipError_t launch_grouped_few(const GroupedArgs &a, hipStream_t s);

}  // namespace moe
