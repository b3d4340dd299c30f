// Products grouped by expert: 16-bit rows and matrices with both gradients,
// and MXFP4 rows and matrices, on 128-column tiles of the matrix cores.
//
//   fwd  out[r][n]   = sum_k x[r][k]  w_e[n][k]
//   dx   dx[r][k]    = sum_n dy[r][n] w_e[n][k]
//   dw   dw_e[n][k]  = sum_r dy[r][n] x[r][k]   (r over the rows of e)
//   mx   fwd with MXFP4 operands, optionally the SwiGLU of two products
//
// One kernel.  Operand `a` supplies the contiguous output columns (the
// matrices; x for dw) and is the matrix instruction's first operand, so that
// a lane ends with four neighbouring columns of one output row; operand `b`
// supplies the output rows.  All four products are the same walk over the
// reduction in steps of 128 bytes a row, because 16 bytes are a lane's
// operand of every instruction used: eight 16-bit elements of
// v_mfma_f32_16x16x32_{bf16,f16}, one 32-element MXFP4 block of
// v_mfma_scale_f32_16x16x128_f8f6f4.  An operand whose reduction runs along
// its rows (fwd, mx; dy of dx) is staged as rows of eight 16-byte pieces; one
// whose reduction runs across its rows (the matrices of dx; both of dw) is
// staged as it lies, 64 rows of 128 columns, and read with the LDS's
// transposing load (ds_read_b64_tr_b16: 16 lanes take a 4 x 16 patch and get
// a column of four each).
//
// Staging is direct loads into LDS (no registers), one step ahead, two
// buffers.  Requests that would leave the matrix, the group or the reduction
// read a page of zeros instead, so tails need no masks in the product and
// never meet another group's NaN.  The pieces of a row are permuted by an XOR
// with row bits so that operand reads meet every bank equally.
//
// A block of four waves (2 x 2) loops over items (expert, column tile, row
// tile); the row tiles of one column tile follow one another, so a matrix
// tile comes from HBM once, and each XCD works on its own range of items.
#include "grouped.h"

#include "mfma_common.h"

namespace moe {

namespace {

constexpr int kGrThreads = 256;
constexpr int kGrMaxExperts = 1024;
constexpr int kGrCols = 128;  // rows of the `a` tile
constexpr int kGrStep = 128;  // bytes of a row a step (reduction along rows)
constexpr int kGrRed = 64;    // rows a step (reduction across rows)

__device__ const uint4 g_zero_page = {0u, 0u, 0u, 0u};

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Direct loads: every lane's 16 (4) bytes go to LDS at `dst` + lane * 16 (4).
// Written in assembly because the compiler would otherwise wait for them
// before any LDS read of the same loop; they have no destination registers,
// and the kernel waits for them itself.
MOE_DEV void direct16(const char *p, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(p) : "memory", "m0");
}
MOE_DEV void direct4(const char *p, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(dst), "v"(p) : "memory", "m0");
}
MOE_DEV uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)p));
}

// XOR of the piece index of staged row R.  `a` rows are read in the order
// 32 j + 8 i + 4 h + b (i, b = 0..3 over 16 lanes), `b` rows in order; a row is
// half of the 64 banks, so rows that differ in bit 0 never collide and the
// other three varying bits choose the piece.
MOE_DEV int swz_a(int R) { return ((R >> 1) & 1) | (((R >> 3) & 3) << 1); }
MOE_DEV int swz_b(int R) { return (R >> 1) & 7; }
// the same for transposed reads: eight rows of a half wave read 32 bytes each
MOE_DEV int swz_t(int R) { return ((R & 3) | (((R >> 3) & 1) << 2)) << 1; }

template <int TYPE>
MOE_DEV f32x4_t mfma16(const u32x4_t &a, const u32x4_t &b, const f32x4_t &c) {
  if constexpr (TYPE == MOE_T_BF16)
    return mfma_bf16(a, b, c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// MXFP4: sa and sb hold the lane's scale byte in their low byte
MOE_DEV f32x4_t mfma_mx(const u32x4_t &a, const u32x4_t &b, const f32x4_t &c, uint32_t sa, uint32_t sb) {
  const i32x8_t A = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8_t B = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, static_cast<int>(sa), 0,
                                                          static_cast<int>(sb));
}

// pre[e] = row tiles of the groups before e; pre[E] = all of them
template <int BT>
MOE_DEV void row_tiles(const GroupedArgs &a, int *pre, int *scratch) {
  constexpr int kPer = kGrMaxExperts / kGrThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int cnt[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    cnt[i] = e < a.E ? (group_range(a, e).n + BT - 1) / BT : 0;
    mine += cnt[i];
  }
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 63) scratch[wave] = inc;
  lds_barrier();
  int base = inc - mine;
  for (int w = 0; w < wave; ++w) base += scratch[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e <= a.E) pre[e] = base;
    base += cnt[i];
  }
  if (tid == kGrThreads - 1 && a.E == kGrMaxExperts) pre[kGrMaxExperts] = base;
  lds_barrier();
}

// The expert of row tile j (pre[e] <= j < pre[e + 1]), found by the whole
// wave: among every 16th entry, then among those 16.
MOE_DEV int tile_expert(const int *pre, int E, int j) {
  const int lane = lane_id();
  const int c = __popcll(__ballot(16 * lane < E && pre[16 * lane] <= j)) - 1;
  const int i = 16 * c + (lane & 15);
  return 16 * c + __popcll(__ballot(lane < 16 && i < E && pre[i] <= j)) - 1;
}

// N (4 or 8) neighbouring columns of one output row
template <int N>
MOE_DEV void store_cols(const GroupedArgs &a, int64_t at, int col, const float (&v)[N]) {
  const bool whole = a.out_vec && col + N <= a.na;
  if (a.out_type == MOE_T_F32) {
    float *o = reinterpret_cast<float *>(a.out) + at + col;
    if (whole) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col + i < a.na) o[i] = v[i];
    }
    return;
  }
  uint32_t p[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (a.out_type == MOE_T_BF16) {
      p[i] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
    } else {
      const f32x2v_t f = {v[2 * i], v[2 * i + 1]};
      p[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2_t));
    }
  }
  uint16_t *o = reinterpret_cast<uint16_t *>(a.out) + at + col;
  if (whole) {
    if constexpr (N == 8)
      *reinterpret_cast<uint4 *>(o) = make_uint4(p[0], p[1], p[2], p[3]);
    else
      *reinterpret_cast<uint2 *>(o) = make_uint2(p[0], p[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + i < a.na) o[i] = static_cast<uint16_t>(p[i / 2] >> (16 * (i & 1)));
  }
}

// One operand's requests of this lane: piece i of step s is read at p[i] +
// s * advance while s * unit < lim[i], else from the page of zeros.
template <int N>
struct Requests {
  const char *p[N];
  int32_t lim[N];
};

template <int KIND, int TYPE, int BT, bool SWIGLU>
__global__ void __launch_bounds__(kGrThreads, 2) grouped_tile_kernel(GroupedArgs a, int32_t col_tiles, int32_t dw_tiles) {
  constexpr bool MX = KIND == kGroupedMx, DW = KIND == kGroupedDw;
  constexpr bool ACROSS_A = KIND == kGroupedDx || DW, ACROSS_B = DW;  // reduction across the operand's rows
  constexpr int NA = 4, NB = BT / 32;  // 1 KB requests a wave, a step
  constexpr int FB = BT / 32;          // 16-row fragments of a wave along b
  constexpr int kUnit = ACROSS_A && ACROSS_B ? kGrRed : kGrStep;
  constexpr uint32_t kDataA = kGrCols * kGrStep, kDataB = BT * kGrStep;
  constexpr uint32_t kScale = MX ? (kGrCols + BT) * 8 : 0;
  constexpr uint32_t kBuf = kDataA + kDataB + kScale;
  static_assert(!DW || BT == kGrCols, "dw tiles are square");
  __shared__ __align__(1024) char lds[2 * kBuf];
  __shared__ int pre[kGrMaxExperts + 1];
  __shared__ int scratch[kGrThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wa = wave & 1, wb = wave >> 1;
  const int l16 = lane & 15, g = lane >> 4;
  const char *zero = reinterpret_cast<const char *>(&g_zero_page);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));

  int n_items;
  if constexpr (DW) {
    n_items = a.E * col_tiles * dw_tiles;
  } else {
    row_tiles<BT>(a, pre, scratch);
    n_items = pre[a.E] * col_tiles;
  }
  // blocks go to the XCDs in turn: XCD x takes the x-th eighth of the items
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  const int end = static_cast<int>(static_cast<int64_t>(n_items) * (xcd + 1) / 8);
  for (int item = static_cast<int>(static_cast<int64_t>(n_items) * xcd / 8) + (blockIdx.x >> 3); item < end; item += per) {
    int e, ct, bt;
    if constexpr (DW) {
      e = item / (col_tiles * dw_tiles);
      const int in = item - e * (col_tiles * dw_tiles);
      ct = in / dw_tiles;
      bt = in - ct * dw_tiles;
    } else {
      e = __builtin_amdgcn_readfirstlane(tile_expert(pre, a.E, item / col_tiles));
      const int mt = pre[e + 1] - pre[e];
      const int in = item - pre[e] * col_tiles;
      ct = in / mt;
      bt = in - ct * mt;
      if (bt < 0 || bt >= mt) continue;  // only where offsets overlap
    }
    const GroupRange gr = group_range(a, e);
    const int b0 = bt * BT;                        // first output row of the tile
    const int b_rows = (DW ? a.nb : gr.n) - b0;    // output rows from there on
    const int c0 = ct * (SWIGLU ? kGrCols / 2 : kGrCols);
    const int red = DW ? gr.n : a.red;             // rows (across) or bytes (along)
    constexpr int kRedUnit = KIND == kGroupedDx ? kGrRed : kUnit;
    const int steps = (red + kRedUnit - 1) / kRedUnit;

    Requests<NA> ra;
    Requests<NB> rb;
    const char *abase = a.a + static_cast<int64_t>(e) * a.a_expert;
    const char *upbase = SWIGLU ? a.a2 + static_cast<int64_t>(e) * a.a_expert : nullptr;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      if constexpr (ACROSS_A) {
        const int R = 4 * (wave + 4 * i) + g;
        const int col = c0 + 8 * (l16 ^ swz_t(R));
        const bool ok = col < a.na;
        if constexpr (DW)
          ra.p[i] = a.a + 2 * static_cast<int64_t>(ok ? col : 0);  // the row is added a step at a time
        else
          ra.p[i] = abase + R * a.a_ld + 2 * static_cast<int64_t>(ok ? col : 0);
        ra.lim[i] = ok ? red - R : INT32_MIN;
      } else {
        const int R = 8 * (wave + 4 * i) + (lane >> 3);
        const int piece = (lane & 7) ^ swz_a(R);
        // SwiGLU: 32 gate rows, then their 32 up rows, for each half of the tile
        const int col = SWIGLU ? c0 + 32 * (R >> 6) + (R & 31) : c0 + R;
        const char *base = SWIGLU && (R & 32) ? upbase : abase;
        const bool ok = col < a.na;
        ra.p[i] = base + (ok ? col : 0) * a.a_ld + 16 * piece;
        ra.lim[i] = ok ? red - 16 * piece : INT32_MIN;
      }
    }
    // Row of x or dy behind grouped row r (inside the group), or -1
    auto source = [&](int r) __attribute__((always_inline)) {
      const int at = gr.r0 + r;
      if (KIND == kGroupedDx || !a.row_tok) return at;
      const int t = a.row_tok[at];
      return static_cast<uint32_t>(t) < static_cast<uint32_t>(a.T) ? t : -1;
    };
    int tok[NA];  // dw: the x row of each request of the next step
    auto next_rows = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int r = s * kGrRed + 4 * (wave + 4 * i) + g;
        tok[i] = r < red ? source(r) : -1;
      }
    };
    if constexpr (DW) next_rows(0);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if constexpr (ACROSS_B) {
        const int R = 4 * (wave + 4 * i) + g;
        const int col = b0 + 8 * (l16 ^ swz_t(R));
        const bool ok = col < a.nb;
        rb.p[i] = a.b + (gr.r0 + static_cast<int64_t>(R)) * a.b_ld + 2 * static_cast<int64_t>(ok ? col : 0);
        rb.lim[i] = ok ? red - R : INT32_MIN;
      } else {
        const int R = 8 * (wave + 4 * i) + (lane >> 3);
        const int piece = (lane & 7) ^ swz_b(R);
        const int src = R < b_rows ? source(b0 + R) : -1;
        rb.p[i] = a.b + (src < 0 ? 0 : src) * a.b_ld + 16 * piece;
        const int bytes = KIND == kGroupedDx ? 2 * red : red;
        rb.lim[i] = src >= 0 ? bytes - 16 * piece : INT32_MIN;
      }
    }
    // MXFP4: eight scale bytes a row and step, two 4-byte requests; request
    // q of a wave covers 32 rows of a (q = 0) or b
    const char *sp[2] = {zero, zero};
    int slim[2] = {INT32_MIN, INT32_MIN};
    if constexpr (MX) {
      const int j = 4 * (lane & 1);
      const int R = 32 * wave + (lane >> 1);
      const int col = SWIGLU ? c0 + 32 * (R >> 6) + (R & 31) : c0 + R;
      const char *base = SWIGLU && (R & 32) ? a.as2 : a.as;
      if (col < a.na) {
        sp[0] = base + (static_cast<int64_t>(e) * a.na + col) * a.s_ld + j;
        slim[0] = a.s_ld - j;
      }
      const int src = R < BT && R < b_rows ? source(b0 + R) : -1;
      if (src >= 0) {
        sp[1] = a.bs + static_cast<int64_t>(src) * a.s_ld + j;
        slim[1] = a.s_ld - j;
      }
    }

    auto issue = [&](int s) __attribute__((always_inline)) {
      const uint32_t buf = lds0 + (s & 1) * kBuf;
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const char *p;
        if constexpr (DW) {
          p = ra.lim[i] > s * kGrRed && tok[i] >= 0 ? ra.p[i] + tok[i] * a.a_ld : zero;
        } else if constexpr (ACROSS_A) {
          p = ra.lim[i] > s * kGrRed ? ra.p[i] + s * (kGrRed * a.a_ld) : zero;
        } else {
          p = ra.lim[i] > s * kGrStep ? ra.p[i] + s * static_cast<int64_t>(kGrStep) : zero;
        }
        direct16(p, buf + 1024 * (wave + 4 * i));
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const char *p;
        if constexpr (ACROSS_B)
          p = rb.lim[i] > s * kGrRed ? rb.p[i] + s * (kGrRed * a.b_ld) : zero;
        else
          p = rb.lim[i] > s * kGrStep ? rb.p[i] + s * static_cast<int64_t>(kGrStep) : zero;
        direct16(p, buf + kDataA + 1024 * (wave + 4 * i));
      }
      if constexpr (MX) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (q == 0 || 32 * wave < BT)
            direct4(slim[q] > 8 * s ? sp[q] + 8 * s : zero,
                    buf + kDataA + kDataB + (q == 0 ? 0u : kGrCols * 8u) + 256 * wave);
      }
    };

    f32x4_t acc[4][FB];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int h = 0; h < FB; ++h) acc[f][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    lds_barrier();  // the previous item's operand reads are done
    if (steps > 0) {
      issue(0);
      if constexpr (DW) next_rows(1);
    }
    for (int s = 0; s < steps; ++s) {
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      lds_barrier();
      if (s + 1 < steps) {
        issue(s + 1);
        if constexpr (DW) next_rows(s + 2);
      }
      const char *ta = lds + (s & 1) * kBuf;
      const char *tb = ta + kDataA;
      const char *ts = tb + kDataB;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        auto along = [&](const char *t, int R, int sw) __attribute__((always_inline)) {
          const uint4 v = *reinterpret_cast<const uint4 *>(t + R * kGrStep + 16 * ((4 * kk + g) ^ sw));
          return u32x4_t{v.x, v.y, v.z, v.w};
        };
        // columns col .. col + 15 of staged rows 32 kk + 8 g .. + 7
        auto across = [&](const char *t, int col) __attribute__((always_inline)) {
          u32x4_t r;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int R = 32 * kk + 8 * g + 4 * j + (l16 >> 2);
            const int piece = (col / 8 + ((l16 >> 1) & 1)) ^ swz_t(R);
            const char *p = t + R * 256 + 16 * piece + 8 * (l16 & 1);
            const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4_t *)(const_cast<char *>(p)));
            const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
            r[2 * j] = u.x;
            r[2 * j + 1] = u.y;
          }
          return r;
        };
        u32x4_t A[4], B[FB];
        uint32_t sa[4] = {}, sb[FB] = {};
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if constexpr (ACROSS_A) {
            A[f] = across(ta, 64 * wa + 16 * f);
          } else {
            const int R = 64 * wa + 32 * (f >> 1) + 8 * (l16 >> 2) + 4 * (f & 1) + (l16 & 3);
            A[f] = along(ta, R, swz_a(R));
            if constexpr (MX) sa[f] = *reinterpret_cast<const uint32_t *>(ts + 8 * R + 4 * kk) >> (8 * g);
          }
        }
#pragma unroll
        for (int h = 0; h < FB; ++h) {
          const int R = wb * (BT / 2) + 16 * h + l16;
          if constexpr (ACROSS_B) {
            B[h] = across(tb, wb * (BT / 2) + 16 * h);
          } else {
            B[h] = along(tb, R, swz_b(R));
            if constexpr (MX) sb[h] = *reinterpret_cast<const uint32_t *>(ts + 8 * (kGrCols + R) + 4 * kk) >> (8 * g);
          }
        }
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int h = 0; h < FB; ++h) {
            if constexpr (MX)
              acc[f][h] = mfma_mx(A[f], B[h], acc[f][h], sa[f], sb[h]);
            else
              acc[f][h] = mfma16<TYPE>(A[f], B[h], acc[f][h]);
          }
      }
    }

#pragma unroll
    for (int h = 0; h < FB; ++h) {
      const int r = wb * (BT / 2) + 16 * h + l16;  // output row inside the tile
      if (r >= b_rows) continue;
      const int64_t row = DW ? static_cast<int64_t>(e) * a.nb + b0 + r : static_cast<int64_t>(gr.r0) + b0 + r;
      const float w = !DW && a.row_w ? a.row_w[row] : 1.f;
      const int64_t at = row * a.out_ld;
      if constexpr (ACROSS_A) {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int col = c0 + 64 * wa + 16 * f + 4 * g;
          const float v[4] = {acc[f][h].x, acc[f][h].y, acc[f][h].z, acc[f][h].w};
          if (col < a.na) store_cols<4>(a, at, col, v);
        }
      } else if constexpr (SWIGLU) {
        const int col = c0 + 32 * wa + 8 * g;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gv = acc[i >> 2][h][i & 3], uv = acc[2 + (i >> 2)][h][i & 3];
          v[i] = w * (gv / (1.f + expf(-gv)) * uv);
        }
        if (col < a.na) store_cols<8>(a, at, col, v);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = c0 + 64 * wa + 32 * j + 8 * g;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = w * acc[2 * j + (i >> 2)][h][i & 3];
          if (col < a.na) store_cols<8>(a, at, col, v);
        }
      }
    }
  }
}

template <int KIND, int TYPE, int BT, bool SWIGLU>
hipError_t launch_tile(const GroupedArgs &a, hipStream_t s) {
  const int32_t cols = SWIGLU ? kGrCols / 2 : kGrCols;
  const int32_t col_tiles = (a.na + cols - 1) / cols;
  const int32_t dw_tiles = (a.nb + kGrCols - 1) / kGrCols;
  // items at most (host): the kernel counts them itself
  const int64_t tiles = KIND == kGroupedDw ? static_cast<int64_t>(a.E) * dw_tiles
                                           : a.n_rows / BT + static_cast<int64_t>(a.E < a.n_rows ? a.E : a.n_rows);
  const int64_t items = tiles * col_tiles;
  const int64_t blocks = (items + 7) / 8 * 8;
  constexpr int64_t kMost = 512;  // two blocks a compute unit
  grouped_tile_kernel<KIND, TYPE, BT, SWIGLU>
      <<<dim3(static_cast<uint32_t>(blocks < kMost ? blocks : kMost)), kGrThreads, 0, s>>>(a, col_tiles, dw_tiles);
  return hipGetLastError();
}

template <int KIND, int TYPE, bool SWIGLU>
hipError_t launch_rows(const GroupedArgs &a, hipStream_t s) {
  return launch_tile<KIND, TYPE, 128, SWIGLU>(a, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t s) {
  const bool bf = a.type == MOE_T_BF16;
  switch (a.kind) {
    case kGroupedMx:
      return a.a2 ? launch_rows<kGroupedMx, 0, true>(a, s) : launch_rows<kGroupedMx, 0, false>(a, s);
    case kGroupedDx:
      return bf ? launch_rows<kGroupedDx, MOE_T_BF16, false>(a, s) : launch_rows<kGroupedDx, MOE_T_F16, false>(a, s);
    case kGroupedDw:
      return bf ? launch_tile<kGroupedDw, MOE_T_BF16, 128, false>(a, s)
                : launch_tile<kGroupedDw, MOE_T_F16, 128, false>(a, s);
    default:
      return bf ? launch_rows<kGroupedFwd, MOE_T_BF16, false>(a, s) : launch_rows<kGroupedFwd, MOE_T_F16, false>(a, s);
  }
}

}  // namespace moe
