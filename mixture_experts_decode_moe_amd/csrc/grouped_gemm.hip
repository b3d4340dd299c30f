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
#include "grouped_device.h"

namespace moe {

namespace {

constexpr int kGrThreads = 256;
constexpr int kGrMaxExperts = 1024;
constexpr int kGrCols = 128;  // rows of the `a` tile
constexpr int kGrStep = 128;  // bytes of a row a step (reduction along rows)
constexpr int kGrRed = 64;    // rows a step (reduction across rows)

// Direct loads: every lane's 16 (4) bytes go to LDS at `dst` + lane * 16 (4).
// Written in assembly because the compiler would otherwise wait for them
// before any LDS read of the same loop; they have no destination registers,
// and the kernel waits for them itself.  `dst` is the same in every lane.
MOE_DEV void direct16(const char *p, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(
                       __builtin_amdgcn_readfirstlane(dst)),
                   "v"(p) : "memory", "m0");
}
MOE_DEV void direct4(const char *p, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(
                       __builtin_amdgcn_readfirstlane(dst)),
                   "v"(p) : "memory", "m0");
}
MOE_DEV uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)p));
}

// XOR of the piece index of staged row R.  A row is half of the 64 banks, so
// rows that differ in bit 0 never collide and the other three bits that vary
// over 16 lanes choose the piece: rows in order, or (PAIRS) 32 j + 8 i + 4 h +
// b with i, b = 0..3 over the lanes.
template <bool PAIRS>
MOE_DEV int swz(int R) {
  return PAIRS ? ((R >> 1) & 1) | (((R >> 3) & 3) << 1) : (R >> 1) & 7;
}
// the same for transposed reads: eight rows of a half wave read 32 bytes each
MOE_DEV int swz_t(int R) { return ((R & 3) | (((R >> 3) & 1) << 2)) << 1; }

// Fills lo[e] (e = 0 .. E) with the groups' first rows, inside [0, n_rows]
// whatever the offsets hold, and (BT > 0) pre[e] with the row tiles of the
// groups before e, pre[E] = all of them.  Group e has max(lo[e + 1] - lo[e],
// 0) rows.
template <int BT>
MOE_DEV void group_table(const GroupedArgs &a, int *lo, int *pre, int *scratch) {
  constexpr int kPer = kGrMaxExperts / kGrThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.E; e += kGrThreads)
    lo[e] = a.offsets ? min(max(a.offsets[e], 0), a.n_rows) : e * a.n_rows;  // without offsets E is 1
  lds_barrier();
  if constexpr (BT > 0) {
    int cnt[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      cnt[i] = e < a.E ? (max(lo[e + 1] - lo[e], 0) + BT - 1) / BT : 0;
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
}

// The expert of row tile j (pre[e] <= j < pre[e + 1]), found by the whole
// wave: among every 16th entry, then among those 16.
MOE_DEV int tile_expert(const int *pre, int E, int j) {
  const int lane = lane_id();
  const int c = __popcll(__ballot(16 * lane < E && pre[16 * lane] <= j)) - 1;
  const int i = 16 * c + (lane & 15);
  return 16 * c + __popcll(__ballot(lane < 16 && i < E && pre[i] <= j)) - 1;
}

// One operand's requests of this lane: piece i of step s is read at p[i] +
// s * advance while s * unit < lim[i], else from the page of zeros.
template <int N>
struct Requests {
  const char *p[N];
  int32_t lim[N];
};

// One output tile (the same in every lane).
struct Tile {
  int e, ct, bt;
  int r0, n;   // the group's rows
  int b_rows;  // output rows from the tile's first on
  int steps;
};

template <int KIND, int TYPE, int OUT, int BT, bool SWIGLU>
__global__ void __launch_bounds__(kGrThreads, 2) grouped_tile_kernel(GroupedArgs a, int32_t col_tiles, int32_t dw_tiles) {
  constexpr bool MX = KIND == kGroupedMx, DW = KIND == kGroupedDw;
  constexpr bool ACROSS_A = KIND == kGroupedDx || DW, ACROSS_B = DW;  // reduction across the operand's rows
  constexpr int NA = 4, NB = BT / 32;  // 1 KB requests a wave, a step
  constexpr int FB = BT / 32;          // 16-row fragments of a wave along b
  constexpr int kCols = SWIGLU ? kGrCols / 2 : kGrCols;
  constexpr uint32_t kDataA = kGrCols * kGrStep, kDataB = BT * kGrStep;
  constexpr uint32_t kScale = MX ? (kGrCols + BT) * 8 : 0;
  constexpr uint32_t kBuf = kDataA + kDataB + kScale;
  // The matrices' rows behind a lane's accumulators: fragments f and f + 1
  // interleaved in fours where that makes eight neighbouring 16-bit columns
  // a lane, else fragment by fragment.
  constexpr bool kPairs = OUT != MOE_T_F32 && !ACROSS_A;
  constexpr int kWords = OUT == MOE_T_F32 || kPairs ? 4 : 2;
  constexpr int kChunks = (SWIGLU ? 2 : 4) / (kPairs ? 2 : 1);  // stores of a lane a row fragment
  using Out = Packed<OUT, kWords>;
  static_assert(!DW || BT == kGrCols, "dw tiles are square");
  __shared__ __align__(1024) char lds[2 * kBuf];
  __shared__ float row_scale[2][BT];
  constexpr int kTokens = DW ? kGrRed : BT;
  __shared__ int row_token[2][kTokens];
  __shared__ int lo[kGrMaxExperts + 1], pre[DW ? 1 : kGrMaxExperts + 1];
  __shared__ int scratch[kGrThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wa = wave & 1, wb = wave >> 1;
  const int l16 = lane & 15, g = lane >> 4;
  const char *zero = reinterpret_cast<const char *>(&g_zero_page);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const uint32_t token0 = __builtin_amdgcn_readfirstlane(lds_addr(row_token));
  const uint32_t scale0 = __builtin_amdgcn_readfirstlane(lds_addr(row_scale));

  group_table<DW ? 0 : BT>(a, lo, pre, scratch);
  const int n_items = DW ? a.E * col_tiles * dw_tiles : __builtin_amdgcn_readfirstlane(pre[DW ? 0 : a.E]) * col_tiles;
  // blocks go to the XCDs in turn: XCD x takes the x-th eighth of the items
  const int xcd = blockIdx.x & 7, per = gridDim.x >> 3;
  const int end = static_cast<int>(static_cast<int64_t>(n_items) * (xcd + 1) / 8);
  const int begin = static_cast<int>(static_cast<int64_t>(n_items) * xcd / 8) + (blockIdx.x >> 3);

  auto locate = [&](int item) __attribute__((always_inline)) {
    Tile t;
    if constexpr (DW) {
      t.e = item / (col_tiles * dw_tiles);
      const int in = item - t.e * (col_tiles * dw_tiles);
      t.bt = in / col_tiles;
      t.ct = in - t.bt * col_tiles;
    } else {
      t.e = __builtin_amdgcn_readfirstlane(tile_expert(pre, a.E, item / col_tiles));
      const int j = item / col_tiles;
      t.ct = item - j * col_tiles;
      t.bt = j - __builtin_amdgcn_readfirstlane(pre[t.e]);
    }
    t.r0 = __builtin_amdgcn_readfirstlane(lo[t.e]);
    t.n = max(__builtin_amdgcn_readfirstlane(lo[t.e + 1]) - t.r0, 0);
    t.b_rows = (DW ? a.nb : t.n) - t.bt * BT;
    const int red = DW ? t.n : a.red;
    constexpr int kUnit = ACROSS_A ? kGrRed : kGrStep;
    t.steps = (red + kUnit - 1) / kUnit;
    if (!DW && (t.bt < 0 || t.b_rows <= 0)) t.steps = 0;  // only where offsets overlap
    return t;
  };
  // ---- The requesting side runs one step ahead of the products, across the
  // tiles: while a tile's last step is multiplied and its results are
  // stored, the next tile's first step is on its way.  The tokens of the
  // rows that a request gathers are brought to LDS a step earlier still; they
  // never pass through registers on the way, where the compiler would wait
  // for them (and so for all requests before them).
  int next = begin;  // item of the next request
  int next_step = 0;
  int tiles_begun = 0;
  int slot = 0;  // of row_token: the next request's tokens
  Tile nt{};
  Requests<NA> ra;
  Requests<NB> rb;
  const char *sp[2] = {zero, zero};
  int slim[2] = {INT32_MIN, INT32_MIN};
  const bool gather = KIND != kGroupedDx && a.row_tok;

  auto request_tokens = [&]() __attribute__((always_inline)) {
    if (!gather || (!DW && next_step > 0)) return;
    slot ^= 1;
    if (64 * wave < kTokens) {
      const int r = (DW ? next_step * kGrRed : nt.bt * BT) + 64 * wave + lane;
      direct4(reinterpret_cast<const char *>(a.row_tok + nt.r0 + (r < nt.n ? r : 0)),
              token0 + (slot * kTokens + 64 * wave) * 4);
    }
  };
  // row of the gathered operand behind row r of the group, `at` of the
  // request's; -1: none
  auto source = [&](int r, int at) __attribute__((always_inline)) {
    if (r >= nt.n) return -1;
    if (!gather) return nt.r0 + r;
    const int k = row_token[slot][at];
    return static_cast<uint32_t>(k) < static_cast<uint32_t>(a.T) ? k : -1;
  };
  auto find_next = [&]() __attribute__((always_inline)) {
    while (next < end) {
      nt = locate(next);
      if (nt.steps > 0) break;
      next += per;
    }
    if (next < end) request_tokens();
  };
  // addresses of tile nt's requests
  auto set_up = [&]() __attribute__((always_inline)) {
    const int c0 = nt.ct * kCols, b0 = nt.bt * BT;
    const int red = DW ? nt.n : a.red;
    const char *abase = a.a + static_cast<int64_t>(nt.e) * a.a_expert;
    const char *upbase = SWIGLU ? a.a2 + static_cast<int64_t>(nt.e) * a.a_expert : nullptr;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      if constexpr (ACROSS_A) {
        const int R = 4 * (wave + 4 * i) + g;
        const int col = c0 + 8 * (l16 ^ swz_t(R));
        const bool ok = col < a.na;
        // dw: the row is added a step at a time
        ra.p[i] = (DW ? a.a : abase + R * a.a_ld) + 2 * static_cast<int64_t>(ok ? col : 0);
        ra.lim[i] = ok ? red - R : INT32_MIN;
      } else {
        const int R = 8 * (wave + 4 * i) + (lane >> 3);
        const int piece = (lane & 7) ^ swz<kPairs>(R);
        // SwiGLU: 32 gate rows, then their 32 up rows, for each half of the tile
        const int col = SWIGLU ? c0 + 32 * (R >> 6) + (R & 31) : c0 + R;
        const char *base = SWIGLU && (R & 32) ? upbase : abase;
        const bool ok = col < a.na;
        ra.p[i] = base + (ok ? col : 0) * a.a_ld + 16 * piece;
        ra.lim[i] = ok ? red - 16 * piece : INT32_MIN;
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if constexpr (ACROSS_B) {
        const int R = 4 * (wave + 4 * i) + g;
        const int col = b0 + 8 * (l16 ^ swz_t(R));
        const bool ok = col < a.nb;
        rb.p[i] = a.b + (nt.r0 + static_cast<int64_t>(R)) * a.b_ld + 2 * static_cast<int64_t>(ok ? col : 0);
        rb.lim[i] = ok ? red - R : INT32_MIN;
      } else {
        const int R = 8 * (wave + 4 * i) + (lane >> 3);
        const int piece = (lane & 7) ^ swz<false>(R);
        const int src = source(b0 + R, R);
        rb.p[i] = a.b + max(src, 0) * a.b_ld + 16 * piece;
        rb.lim[i] = src >= 0 ? (KIND == kGroupedDx ? 2 * red : red) - 16 * piece : INT32_MIN;
      }
    }
    // MXFP4: eight scale bytes a row and step, two 4-byte requests a lane,
    // each request of a wave 32 rows of a or b
    if constexpr (MX) {
      const int j = 4 * (lane & 1);
      const int R = 32 * wave + (lane >> 1);
      const int col = SWIGLU ? c0 + 32 * (R >> 6) + (R & 31) : c0 + R;
      const char *base = SWIGLU && (R & 32) ? a.as2 : a.as;
      sp[0] = base + (static_cast<int64_t>(nt.e) * a.na + (col < a.na ? col : 0)) * a.s_ld + j;
      slim[0] = col < a.na ? a.s_ld - j : INT32_MIN;
      const int src = R < BT ? source(b0 + R, R) : -1;
      sp[1] = a.bs + static_cast<int64_t>(max(src, 0)) * a.s_ld + j;
      slim[1] = src >= 0 ? a.s_ld - j : INT32_MIN;
    }
  };
  // requests the next step into buffer `b`
  auto issue = [&](int b) __attribute__((always_inline)) {
    if (next >= end) return;
    const int s = next_step;
    const uint32_t buf = lds0 + b * kBuf;
    if (s == 0) {
      set_up();
      if (!DW && a.row_w && 64 * wave < BT) {
        const int r = 64 * wave + lane;
        direct4(r < nt.b_rows ? reinterpret_cast<const char *>(a.row_w + nt.r0 + nt.bt * BT + r) : zero,
                scale0 + ((tiles_begun & 1) * BT + 64 * wave) * 4);
      }
      ++tiles_begun;
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const char *p;
      if constexpr (DW) {
        const int at = 4 * (wave + 4 * i) + g;
        const int src = source(s * kGrRed + at, at);
        p = ra.lim[i] > s * kGrRed && src >= 0 ? ra.p[i] + src * a.a_ld : zero;
      } else if constexpr (ACROSS_A)
        p = ra.lim[i] > s * kGrRed ? ra.p[i] + s * (kGrRed * a.a_ld) : zero;
      else
        p = ra.lim[i] > s * kGrStep ? ra.p[i] + s * static_cast<int64_t>(kGrStep) : zero;
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
      direct4(slim[0] > 8 * s ? sp[0] + 8 * s : zero, buf + kDataA + kDataB + 256 * wave);
      if (32 * wave < BT)
        direct4(slim[1] > 8 * s ? sp[1] + 8 * s : zero, buf + kDataA + kDataB + kGrCols * 8 + 256 * wave);
    }
    if (++next_step == nt.steps) {
      next_step = 0;
      next += per;
      find_next();
    } else {
      request_tokens();
    }
  };

  find_next();
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  lds_barrier();
  issue(0);
  int buf = 0;
  int tiles_done = 0;
  bool younger = false;  // the tile's first requests were followed by a whole tile's stores
  for (int item = begin; item < end; item += per) {
    const Tile t = locate(item);
    f32x4_t acc[4][FB];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int h = 0; h < FB; ++h) acc[f][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < t.steps; ++s) {
      // this step's requests have landed; requests and stores are counted in
      // the order they were made, so the stores behind them may be under way
      if (s == 0 && younger)
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(FB * kChunks));
      else
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      lds_barrier();
      if (next < end) issue(buf ^ 1);
      const char *ta = lds + buf * kBuf;
      const char *tb = ta + kDataA;
      const char *ts = tb + kDataB;
      buf ^= 1;
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
            const int R = 64 * wa + (kPairs ? 32 * (f >> 1) + 8 * (l16 >> 2) + 4 * (f & 1) + (l16 & 3) : 16 * f + l16);
            A[f] = along(ta, R, swz<kPairs>(R));
            if constexpr (MX) sa[f] = *reinterpret_cast<const uint32_t *>(ts + 8 * R + 4 * kk) >> (8 * g);
          }
        }
#pragma unroll
        for (int h = 0; h < FB; ++h) {
          const int R = wb * (BT / 2) + 16 * h + l16;
          if constexpr (ACROSS_B) {
            B[h] = across(tb, wb * (BT / 2) + 16 * h);
          } else {
            B[h] = along(tb, R, swz<false>(R));
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
    if (!DW && t.steps == 0) continue;

    const float *scale = row_scale[tiles_done++ & 1];
    auto store_tile = [&](auto whole_t) __attribute__((always_inline)) {
      constexpr bool WHOLE = decltype(whole_t)::value != 0;
#pragma unroll
      for (int h = 0; h < FB; ++h) {
        const int r0 = wb * (BT / 2) + 16 * h;  // the fragment's first row in the tile
        const float w = !DW && a.row_w ? scale[r0 + l16] : 1.f;
        const int r = r0 + (lane >> 2);  // the row that this lane stores
        const bool in = WHOLE || r < t.b_rows;
        const int64_t at =
            ((DW ? static_cast<int64_t>(t.e) * a.nb : static_cast<int64_t>(t.r0)) + t.bt * BT + r) * a.out_ld;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float v[Out::kCols];
#pragma unroll
          for (int i = 0; i < Out::kCols; ++i) {
            const int f = kPairs ? 2 * c + (i >> 2) : c;
            v[i] = acc[f][h][i & 3];
            if constexpr (SWIGLU) v[i] = v[i] / (1.f + expf(-v[i])) * acc[f + 2][h][i & 3];
            v[i] *= w;
          }
          Out o;
          o.set(v);
          o.by_row();
          const int col = t.ct * kCols + (SWIGLU ? 32 : 64) * wa + Out::kCols * (4 * c + (lane & 3));
          if (WHOLE || (in && col < a.na)) o.template store<WHOLE>(a, at, col);
        }
      }
    };
    younger = a.out_vec && t.b_rows >= BT && (t.ct + 1) * kCols <= a.na;
    if (younger)
      store_tile(IntC<1>{});
    else
      store_tile(IntC<0>{});
  }
}

template <int KIND, int TYPE, int OUT, int BT, bool SWIGLU = false>
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
  grouped_tile_kernel<KIND, TYPE, OUT, BT, SWIGLU>
      <<<dim3(static_cast<uint32_t>(blocks < kMost ? blocks : kMost)), kGrThreads, 0, s>>>(a, col_tiles, dw_tiles);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_16bit(const GroupedArgs &a, hipStream_t s) {
  if (a.type == MOE_T_BF16)
    return a.out_type == MOE_T_F32 ? launch_tile<KIND, MOE_T_BF16, MOE_T_F32, 128>(a, s)
                                   : launch_tile<KIND, MOE_T_BF16, MOE_T_BF16, 128>(a, s);
  return a.out_type == MOE_T_F32 ? launch_tile<KIND, MOE_T_F16, MOE_T_F32, 128>(a, s)
                                 : launch_tile<KIND, MOE_T_F16, MOE_T_F16, 128>(a, s);
}

template <bool SWIGLU>
hipError_t launch_mx(const GroupedArgs &a, hipStream_t s) {
  switch (a.out_type) {
    case MOE_T_BF16:
      return launch_tile<kGroupedMx, 0, MOE_T_BF16, 128, SWIGLU>(a, s);
    case MOE_T_F16:
      return launch_tile<kGroupedMx, 0, MOE_T_F16, 128, SWIGLU>(a, s);
    default:
      return launch_tile<kGroupedMx, 0, MOE_T_F32, 128, SWIGLU>(a, s);
  }
}

// Whether the few-row kernel takes the call: up to 256 rows, and tiles for
// less than one block a compute unit.  Below that the tiles leave most of the
// chip idle and a tile's long walk is the whole time: one row each of eight
// experts of 1024 x 2048 in 16 bits 27.9 us against 12.2, one row of a single
// 1024 x 1024 matrix 15.7 against 4.8, 256 rows of it 15.9 against 10.3.  Above
// it the tiles read every matrix once: 64 experts of 1024 x 1024, a row each,
// 29.8 against 32.4 us, MXFP4 12.0 against 20.0; 1024 rows of one matrix 17.0
// against 34.3.
bool few_rows(const GroupedArgs &a) {
  if (a.kind != kGroupedFwd && a.kind != kGroupedMx) return false;
  const int32_t cols = a.a2 ? kGrCols / 2 : kGrCols;
  const int32_t tiles = a.n_rows / 128 + (a.E < a.n_rows ? a.E : a.n_rows);
  return a.n_rows <= 256 && static_cast<int64_t>(tiles) * ((a.na + cols - 1) / cols) <= 256;
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, hipStream_t s) {
  if (few_rows(a)) return launch_grouped_few(a, s);
  switch (a.kind) {
    case kGroupedMx:
      return a.a2 ? launch_mx<true>(a, s) : launch_mx<false>(a, s);
    case kGroupedDx:
      return launch_16bit<kGroupedDx>(a, s);
    case kGroupedDw:
      return launch_16bit<kGroupedDw>(a, s);
    default:
      return launch_16bit<kGroupedFwd>(a, s);
  }
}

}  // namespace moe
