// Products of 16-bit and 8-bit integer operands, dense and grouped over experts of ragged sizes, and the
// 16-bit product's gradients.
//
//   rows      out[r, n]  = sum_k a[src(r), k] * w[e, n, k]        (gate+up: SiLU of one half times the other)
//   across    out[r, n]  = sum_k a[r, k] * w[e, k, n]             (the rows' gradient)
//   weights   dw[e,n,k]  = sum over the expert's rows r of dy[r, n] * x[src(r), k]
//
// The matrix instruction's A operand is the side whose index is contiguous in the output (weights, or x), its B
// operand the other (token rows, or dy): a lane then ends with four consecutive columns of one output row.  Lane
// (r, g) of a 16-row fragment holds 16 bytes of its row, the same 16 bytes of K on both sides.
#include <atomic>
#include <utility>

#include "device_common.h"
#include "internal.h"
#include "lds_dma.h"

namespace megamoe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kGtDevices = 64;
constexpr int kGtPlain = 0, kGtGateUp = 1, kGtAcross = 2;  // operations of gt_kernel
constexpr int kGtGrid = 256;                        // one workgroup a CU
constexpr int kGtWaves = 8, kGtThreads = kGtWaves * kWave;
constexpr int kGtCols = 256, kGtRows = 256;         // A-side and B-side rows of the largest tile
constexpr int kGtStage = 128;                       // bytes of K a stage (64 or 128 elements)
constexpr int kGtSide = kGtCols * kGtStage;         // LDS bytes of a stage's A side
constexpr int kGtLds = 160 * 1024;
// ns of a tile, by its rows (of 256 columns, and of the tiles of 64 x 64): a stage of 128 bytes of K, and the rest.
constexpr int kGtNs4[2] = {1300, 4000}, kGtNs2[2] = {1150, 5000}, kGtNs1[2] = {1050, 5000}, kGtNsFine[2] = {250, 1500};
constexpr int kGwTile = 60, kGwFineTile = 20;  // the weights' gradient's tiles, beside their stages, in tenths of a us
constexpr int kGtNsFineAlone = 330;  // of a stage where no two tiles of 64 rows share weights
constexpr int kGtBand = 8;                          // m-tiles walked together, for L2 reuse of the weights
// The kernels have no static LDS: addresses start at 0.  At the end: two list lengths, m-tile prefix int32 [E + 1],
// two lists uint16 [E].
constexpr int kGtLists = kGtLds - 8224;
static_assert(8 + 4 * (MEGAMOE_MAX_EXPERTS + 1) + 4 * MEGAMOE_MAX_EXPERTS <= kGtLds - kGtLists, "the lists fit");

__device__ const uint32_t g_zeros[4] = {0u, 0u, 0u, 0u};  // what a load brings beyond the reduced dimension

__device__ __forceinline__ float g_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// Parts of at most `of` that n is cut into, for any n of 31 bits (n + of - 1 would not fit).
__device__ __forceinline__ int g_parts(int n, int of) { return n / of + (n % of > 0 ? 1 : 0); }

// Workgroup barrier that no LDS access is moved across.  Vector memory loads stay in flight.
__device__ __forceinline__ void g_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void g_wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

// A word of a table that the kernel does not write, from a wave-uniform address: a scalar load, which does not wait
// for the vector loads in flight.
__device__ __forceinline__ int g_scalar(const int32_t* p) {
  const uint64_t at = scalar_addr(reinterpret_cast<const uint8_t*>(p));
  return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(at);
}

// Sum of a value over the lanes up to this one.
__device__ __forceinline__ int g_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

__device__ __forceinline__ int g_total(int v) { return __builtin_amdgcn_readlane(g_scan(v), kWave - 1); }

// What follows from the lane is computed where it is used, not held in registers through a loop.
__device__ __forceinline__ int g_here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Operand types: the accumulator and the 16x16 matrix instruction over 64 bytes of K (16x16x32 or 16x16x64).  Inline
// assembly keeps the accumulators in accumulation registers, 128 of them in the largest tile: left to itself the
// compiler moves them to and fro (408 moves beside 64 products, when there were 256).  What it does not know of these
// instructions is kept by hand: an accumulator is met again after at least 7 others, and g_settle stands between the
// products and any other write or read of it.  From registers the instructions reach 2025 TFLOP/s (bf16) and 4121 TOPS
// (int8) on random numbers, 2468 and 4926 on zeros: the clock falls with the power.
template <int kDtype>
struct GType {
  typedef f32x4 acc;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ void mfma(u32x4 a, u32x4 b, acc& c) {
    if constexpr (kDtype == MEGAMOE_DTYPE_BF16)
      asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else
      asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ acc product(u32x4 a, u32x4 b, acc c) {  // (the compiler's own, for chains)
    if constexpr (kDtype == MEGAMOE_DTYPE_BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct GType<kOperandI8> {
  typedef i32x4 acc;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ void mfma(u32x4 a, u32x4 b, acc& c) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ acc product(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};
// Accumulators in front of other instructions than the products: a result can be read 18 cycles after its
// instruction, and is read by the next one 2 after a write.
template <typename A, int n>
__device__ __forceinline__ void g_settle(A (&c)[n]) {
  static_assert(n == 4 || n == 8, "fragments of a wave");
  if constexpr (n == 8)
    asm volatile("s_nop 15\n\ts_nop 7"
                 : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]), "+a"(c[4]), "+a"(c[5]), "+a"(c[6]), "+a"(c[7]));
  else
    asm volatile("s_nop 15\n\ts_nop 7" : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]));
}

__device__ __forceinline__ u32x4 lds_read16(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(at);
}
__device__ __forceinline__ void lds_write16(uint32_t at, u32x4 v) {
  *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at) = v;
}
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(at);
}

// A 16-row fragment of a side that lies across: LDS holds rows of the reduced dimension, kRow bytes each (512: the
// 256 columns of a large tile; 128: the 64 of a small one).  The transposing read gives lane i of 16 lanes column i of
// the four rows by 16 columns whose 8-byte pieces the lanes point at: two of them make the lane's eight values of K.
template <int kRow>
__device__ __forceinline__ u32x4 lds_read_across(uint32_t at) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(at + 4 * kRow));
  const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
  return u32x4{l[0], l[1], h[0], h[1]};
}

__device__ __forceinline__ uint32_t g_pack2(float a, float b, bool f16) {
  return f16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2))
             : __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
// Two 16-column blocks of an output row, four consecutive columns of each a lane (g = lane / 16: columns 4g) ->
// eight consecutive ones: of block g % 2, from column 8 (g / 2) on.
__device__ __forceinline__ u32x4 g_gather8(u32x2 lo, u32x2 hi) {
  const auto a = __builtin_amdgcn_permlane16_swap(lo[0], hi[0], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(lo[1], hi[1], false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}

// A step: the products of one 64-byte piece of K, with the next step's operands read from LDS (read(i)) and a
// stage's loads requested (load(j)) between them, each behind a product of its own: a wave issues in order, and a load
// holds it for some 70 cycles, which only the SIMD's other wave's products fill.  Reads and loads are out after three
// quarters of the products (half, or all of them: the same times).
template <int V>
struct GTag {
  static constexpr int value = V;
};
template <typename F, int... V>
__device__ __forceinline__ void gt_each(const F& f, std::integer_sequence<int, V...>) {
  (f(GTag<V>{}), ...);
}
template <typename T, int MF, int NF, int kReads, int kLoads, typename Read, typename Load>
__device__ __forceinline__ void gt_step(typename T::acc (&acc)[MF][NF], const u32x4 (&a)[NF], const u32x4 (&b)[MF],
                                        const Read& read, const Load& load) {
  constexpr int span = MF * NF * 3 / 4;
  gt_each(
      [&](auto tag) __attribute__((always_inline)) {
        constexpr int at = decltype(tag)::value;
        T::mfma(a[at / MF], b[at % MF], acc[at % MF][at / MF]);
        __builtin_amdgcn_sched_barrier(0);
        // item i of n stands behind product i * span / n, loads one later
        constexpr int r0 = (at * kReads + span - 1) / span, r1 = ((at + 1) * kReads + span - 1) / span;
#pragma unroll
        for (int i = r0; i < (r1 < kReads ? r1 : kReads); ++i) read(i);
        constexpr int l0 = ((at - 1) * kLoads + span - 1) / span, l1 = (at * kLoads + span - 1) / span;
#pragma unroll
        for (int j = at > 0 ? l0 : 0; j < (at == 0 ? 0 : l1 < kLoads ? l1 : kLoads); ++j) load(j);
        __builtin_amdgcn_sched_barrier(0);
      },
      std::make_integer_sequence<int, MF * NF>{});
}
struct GtNothing {
  __device__ __forceinline__ void operator()(int) const {}
};

// A lane's 16 bytes of two neighbouring 64-byte blocks of its output row (lane % 16) -> of both blocks of a row of the
// lower eight, and of one of the upper eight: row (lane % 8), block (lane % 16) / 8.  A store then covers eight
// rows of 128 bytes, whole lines, not sixteen of half a line: non-temporal stores of half lines took the weights'
// gradient of 64 experts of 32 rows (float32, 7168 x 4096) 2400 us.
__device__ __forceinline__ void g_whole_lines(u32x4& lo, u32x4& hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = (int)lo[i], b = (int)hi[i];
    lo[i] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false);  // row_ror 8 into lanes 8-15
    hi[i] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false);  // into lanes 0-7
  }
}

// ============================================================================================
// rows, gate+up and across: 256 weight rows x BM token rows a tile, BM = 64 WB = 256, or 128 or 64 for an
// expert's last rows when they fit; one persistent workgroup of 8 waves a CU takes all tiles of 256 rows, then
// those of 128, then those of 64.
//
// A stage is 128 bytes of K of every row.  Stages go from global memory straight into a ring of LDS slots (2 of
// 64 KB, or 3 of the lower tiles' 48 or 40) and run on across tiles.  A stage is two steps of 64 bytes; a step's
// operands are read from LDS while the step before is multiplied.  Between the two steps of stage s a wave has
// read all of s: it waits for its loads of stage s + 1, and one barrier makes everyone's visible and says that
// s's slot is free, into which the second step requests the stage after the ring's last.
//
// Many rows: matrix instructions, memory's latency and the power.  int8 16384 x 4096 x 7168 takes 350 us in runs of
// 50 ms (2750 TOPS; 275 us on zeros) and up to 400 in longer ones, as the clock falls; bf16 16384 x 7168 x 4096 727 (1320
// TFLOP/s), 16384 x 2048 x 7168 362, 24 experts of 1024 rows across, 7168 to 4096, 1150.  Few rows: the weights' bytes,
// 48 experts of 40 rows, 7168 to 4096, 404 us (7.1 TB/s), 8 experts of one row across 80 (5.9).  4 waves of 128 x 128
// read a third less from LDS: 657 us for the bf16 product, the same for int8, 942 where 8 waves take 789 for the
// weights' gradient.  Operands staged through registers: 379 where these loads took 358.  Touching the next stages in
// the L2 first: 3 to 10% slower.
// ============================================================================================
template <int WB>
struct GtShape {
  static constexpr int WM = WB == 4 ? 4 : 2, WN = kGtWaves / WM;  // waves along token rows, weight rows
  static constexpr int MF = 4 * WB / WM, NF = 16 / WN;            // a wave's fragments of either side
  static constexpr int D = WB == 4 ? 2 : 3;                       // slots
  static constexpr int kBufs = D + 1;                             // tiles whose scales are in LDS at a time
  static constexpr int kSlot = kGtSide + 64 * WB * kGtStage;
  static constexpr int kLoads = 4 + WB;                           // load instructions a wave and stage
  // LDS behind the slots: the tokens of two tiles' rows, the scales of kBufs tiles
  static constexpr int kRowsAt = D * kSlot, kScalesAt = kRowsAt + 2 * 64 * WB * 4;
  static constexpr int kScaleBuf = 4 * (kGtCols + 64 * WB);
  static constexpr int kTilesAt = kScalesAt + kBufs * kScaleBuf;  // and what the epilogue needs of as many tiles
  static_assert(kTilesAt + kBufs * 16 <= kGtLists, "the LDS layout fits");
};

struct GtTile {
  int e, nt, left;  // expert, n-tile, real rows from row0 on
  int64_t row0;
};

template <int kOp, int kDtype, int WB, typename Find>
__device__ __forceinline__ void gt_phase(const GroupedArgs& p, int t0, int total, const Find& find) {
  typedef GtShape<WB> S;
  typedef GType<kDtype> T;
  constexpr bool kL1 = kOp == kGtGateUp, kAcross = kOp == kGtAcross, kI8 = kDtype == kOperandI8;
  constexpr int cols = kL1 ? kGtCols / 2 : kGtCols;  // output columns of a tile
  constexpr int WN = S::WN, MF = S::MF, NF = S::NF, D = S::D, L = S::kLoads;
  if (t0 >= total) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int64_t RB = (int64_t)p.K * T::kBytes;                    // bytes of a row of K
  const int64_t NB = (int64_t)p.N * T::kBytes;                    // across: bytes of a weight row
  const int nks = (int)((RB + kGtStage - 1) / kGtStage);
  const int piece = (lane & 7) ^ (lane >> 4);  // of 8 rows of an even load instruction (odd: ^ 4)

  // ---- loads -------------------------------------------------------------------------------------
  GtTile ld, nx = find(t0);  // of the loads, and the next
  int lt = t0;
  int lks = 0, lseq = 0;
  const uint8_t* w_at = nullptr;                   // of the stage to request
  uint32_t w_off[kAcross ? 2 : 4];                 // across: of even and odd load instructions
  uint64_t a_at[WB];
  const auto fetch_rows = [&](int buf) __attribute__((always_inline)) {  // tokens of the next tile's rows
    if (!kAcross && p.row_token != nullptr && wave < WB) {
      const int R = 64 * wave + g_here(lane);
      dma4(reinterpret_cast<const uint8_t*>(p.row_token + nx.row0 + (R < nx.left ? R : nx.left - 1)),
           S::kRowsAt + 4 * (64 * WB * buf + 64 * wave));
    }
  };
  // Source of the tile's token row R, and weight row (output column) of its row R; rows past the tile's end read
  // its last row, columns past the last one the last: what they feed is not stored.
  const auto a_row = [&](int R) __attribute__((always_inline)) -> uint32_t {
    if (!kAcross && p.row_token != nullptr) return lds_read<uint32_t>(S::kRowsAt + 4 * (64 * WB * (lseq & 1) + R));
    return (uint32_t)((int)ld.row0 + (R < ld.left ? R : ld.left - 1));
  };
  const auto w_col = [&](int R) __attribute__((always_inline)) {
    constexpr int per = kGtCols / WN;  // rows of a wave: kL1: the first half gate, the second up
    const int c = ld.nt * cols + (kL1 ? R / per * (per / 2) + R % (per / 2) : R);
    return c < p.N ? c : p.N - 1;
  };
  const auto is_up = [&](int R) { return R % (kGtCols / WN) >= kGtCols / WN / 2; };
  const auto a_piece = [&](int i) { return piece ^ (((WB * wave + i) & 1) << 2); };
  const auto uniform = [](const uint8_t* at) __attribute__((always_inline)) {
    return reinterpret_cast<const uint8_t*>(scalar_addr(at));
  };
  const auto enter = [&]() __attribute__((always_inline)) {  // tile lt
    const int ln = g_here(lane);
    ld = nx;
    if (wave == 0 && lane == 0)
      lds_write16(S::kTilesAt + 16 * (lseq % S::kBufs),
                  u32x4{(uint32_t)ld.nt, (uint32_t)ld.left, (uint32_t)ld.row0, (uint32_t)(ld.row0 >> 32)});
#pragma unroll
    for (int i = 0; i < WB; ++i)
      a_at[i] = reinterpret_cast<uint64_t>(p.a) + (uint64_t)a_row(8 * (WB * wave + i) + ln / 8) * (uint64_t)(uint32_t)RB +
                16 * a_piece(i);
    if constexpr (kAcross) {
      w_at = uniform(static_cast<const uint8_t*>(p.w) + ((int64_t)ld.e * p.K + 8 * wave) * NB +
                     (int64_t)ld.nt * cols * T::kBytes);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = (ln & 31) ^ (((2 * q + (ln >> 5)) | ((wave & 1) << 2)) << 1);
        const int last = p.N / 8 - 1 - ld.nt * (cols / 8);
        w_off[q] = (uint32_t)(ln >> 5) * (uint32_t)NB + 16 * (c < last ? c : last);
      }
    } else {  // (gate+up: a wave's rows are all gate's or all up's)
      const int64_t c0 = (int64_t)ld.nt * cols + (kL1 && is_up(32 * wave) ? p.N : 0);
      w_at = uniform(static_cast<const uint8_t*>(p.w) + ((int64_t)ld.e * (kL1 ? 2 : 1) * p.N + c0) * RB);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w_off[j] = (uint32_t)(w_col(32 * wave + 8 * j + ln / 8) - ld.nt * cols) * (uint32_t)RB + 16 * (piece ^ ((j & 1) << 2));
    }
    if constexpr (kI8) {  // the tile's scales: weight rows by four waves, token rows by WB others
      const uint32_t to = S::kScalesAt + (lseq % S::kBufs) * S::kScaleBuf;
      const int R = 64 * (wave & 3) + ln;
      if (wave < 4)
        dma4(reinterpret_cast<const uint8_t*>(p.w_scales + (int64_t)ld.e * (kL1 ? 2 : 1) * p.N +
                                              (kL1 && is_up(R) ? p.N : 0) + w_col(R)),
             to + 256 * wave);
      else if (wave - 4 < WB)
        dma4(reinterpret_cast<const uint8_t*>(p.a_scales + a_row(R)), to + 4 * kGtCols + 256 * (wave - 4));
    }
    if (lt + kGtGrid < total) {  // (its table entries are on their way while the tile's stages are multiplied)
      nx = find(lt + kGtGrid);
      fetch_rows((lseq + 1) & 1);
    }
    ++lseq;
  };
  bool done = false;  // with nothing left the last stage is loaded again, and not used
  const auto last_stage = [&]() { return lks + 1 == nks && lt + kGtGrid >= total; };
  // Load j of the stage at (lt, lks): weights, then token rows.
  const auto load = [&](int j, uint64_t a_step, int slot) __attribute__((always_inline)) {
    if (j < 4) {
      const uint8_t* const base = kAcross ? w_at + 2 * j * NB : w_at;
      const uint32_t off = w_off[kAcross ? j & 1 : j], to = slot * S::kSlot + 1024 * (4 * wave + j);
      // the lower tiles are mostly an expert's only ones: its weights are read once, past the caches
      if constexpr (WB < 4) dma16snt(base, off, to);
      else dma16s(base, off, to);
    } else {
      dma16(reinterpret_cast<const uint8_t*>(a_at[j - 4]), slot * S::kSlot + kGtSide + 1024 * (WB * wave + j - 4));
      a_at[j - 4] += a_step;
    }
  };
  // A row's last stage, when K ends inside it: lanes whose piece lies behind the end load the stage's first piece
  // instead (across: waves whose weight rows do, the first rows), and clear() writes zeros over what they brought,
  // before the barrier that shows it.
  const bool ragged = (RB & (kGtStage - 1)) != 0;
  const int left = (int)((RB & (kGtStage - 1)) / 16);  // pieces (across: eights of weight rows) in the last stage
  const auto trim = [&]() __attribute__((always_inline)) {
    if constexpr (kAcross) {
      if (wave >= left) w_at -= 8 * wave * NB;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((piece ^ ((j & 1) << 2)) >= left) w_off[j] -= 16 * (piece ^ ((j & 1) << 2));
    }
#pragma unroll
    for (int i = 0; i < WB; ++i)
      if (a_piece(i) >= left) a_at[i] -= 16 * a_piece(i);
  };
  const auto clear = [&](uint32_t slot) __attribute__((always_inline)) {
    const uint32_t to = slot + 16 * g_here(lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((kAcross ? wave : piece ^ ((j & 1) << 2)) >= left) lds_write16(to + 1024 * (4 * wave + j), u32x4{0u, 0u, 0u, 0u});
#pragma unroll
    for (int i = 0; i < WB; ++i)
      if (a_piece(i) >= left) lds_write16(to + kGtSide + 1024 * (WB * wave + i), u32x4{0u, 0u, 0u, 0u});
  };
  const auto tail_stage = [&]() { return ragged && lks + 1 == nks; };
  const auto loaded = [&]() __attribute__((always_inline)) {
    if (last_stage()) {
      done = true;
      return;
    }
    w_at += kAcross ? 64 * NB : kGtStage;
    if (++lks == nks) {
      lks = 0;
      lt += kGtGrid;
    }
  };

  // ---- operands ------------------------------------------------------------------------------------
  const int wm = wave / WN, wn = wave % WN, r = lane & 15, g = lane >> 4;
  const uint32_t along = r * kGtStage + 16 * (g ^ ((r >> 1) & 7));
  const uint32_t b_base = kGtSide + wm * (16 * MF) * kGtStage + along;
  const int jj = (lane & 15) >> 2;
  const uint32_t a_base = kAcross ? (8 * g + jj) * 512 + (((NF * wn) ^ (jj | ((g & 1) << 2))) * 32) + (lane & 3) * 8
                                  : wn * (16 * NF) * kGtStage + along;
  u32x4 a[2][NF], b[2][MF];
  // Operands of step st of a slot: bases in registers, so that a read is one instruction.
  uint32_t ra, rb;
  const auto aim = [&](int slot, int st) __attribute__((always_inline)) {
    rb = (b_base ^ (st * 64)) + slot * S::kSlot;
    ra = (kAcross ? a_base : a_base ^ (st * 64)) + slot * S::kSlot;
    asm volatile("" : "+v"(ra), "+v"(rb));
  };
  const auto read_one = [&](int st, int i) __attribute__((always_inline)) {
    if (i < MF) b[st][i] = lds_read16(rb + i * 16 * kGtStage);
    else if constexpr (kAcross) a[st][i - MF] = lds_read_across<512>((ra ^ ((i - MF) * 32)) + st * 32 * 512);
    else a[st][i - MF] = lds_read16(ra + (i - MF) * 16 * kGtStage);
  };

  g_wait_lds();
  g_barrier();  // the phase before is done with LDS
  fetch_rows(0);
  wait_vmcnt<0>();
  g_barrier();
  int issued = 0;
  const auto first_loads = [&]() __attribute__((always_inline)) {
    if (!done && lks == 0) {
      if (issued > 0) {  // its rows were asked for with the tile before
        wait_vmcnt<0>();
        g_barrier();
      }
      enter();
    }
    if (!done && tail_stage()) trim();
    const uint64_t a_step = last_stage() ? 0 : kGtStage;
#pragma unroll
    for (int j = 0; j < L; ++j) load(j, a_step, issued);
    loaded();
  };
  for (; issued < D; ++issued) first_loads();
  wait_vmcnt<(D - 1) * L>();
  if (ragged && nks == 1) clear(0);
  g_wait_lds();
  g_barrier();
  aim(0, 0);
#pragma unroll
  for (int i = 0; i < MF + NF; ++i) read_one(0, i);

  int slot = 0, seq = 0;
  for (int t = t0; t < total; t += kGtGrid) {
    typename T::acc acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][f][q] = 0;
#pragma unroll
    for (int m = 0; m < MF; ++m) g_settle(acc[m]);
    for (int ks = 0; ks < nks; ++ks) {
      const int nslot = slot + 1 == D ? 0 : slot + 1;
      aim(slot, 1);
      gt_step<T, MF, NF, MF + NF, 0>(acc, a[0], b[0], [&](int i) __attribute__((always_inline)) { read_one(1, i); }, GtNothing{});
      wait_vmcnt<(D - 2) * L>();  // the next stage's
      if (ragged && (ks + 2 == nks || nks == 1)) clear(nslot * S::kSlot);
      g_wait_lds();
      g_barrier();
      if (!done && lks == 0) enter();
      if (!done && tail_stage()) trim();
      const uint64_t a_step = last_stage() ? 0 : kGtStage;
      aim(nslot, 0);
      gt_step<T, MF, NF, MF + NF, L>(acc, a[1], b[1], [&](int i) __attribute__((always_inline)) { read_one(0, i); },
                                     [&](int j) __attribute__((always_inline)) { load(j, a_step, slot); });
      if (!done) loaded();
      slot = nslot;
    }

    // Output: row 16 m + r of the wave, columns 16 f + 4 g ..+3 of block f.
    const u32x4 info = lds_read16(S::kTilesAt + 16 * (seq % S::kBufs));  // of the tile, as its loads left it
    struct {
      int nt, left;
      int64_t row0;
    } cur;
    cur.nt = __builtin_amdgcn_readfirstlane((int)info[0]);
    cur.left = __builtin_amdgcn_readfirstlane((int)info[1]);
    cur.row0 = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)info[2]) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)info[3]) << 32);
    const uint32_t sc = S::kScalesAt + (seq % S::kBufs) * S::kScaleBuf;
    ++seq;
    const bool f16 = p.out_dtype == MEGAMOE_DTYPE_F16;
    constexpr int kOutF = kL1 ? NF / 2 : NF;  // column blocks of a wave
    const int le = g_here(lane), r = le & 15, g = le >> 4;
    const int c0 = cur.nt * cols + wn * 16 * kOutF + 16 * (g & 1) + 8 * (g >> 1);
    const auto put = [&](int R, int c, u32x4 v) __attribute__((always_inline)) {
      if (R < cur.left && c < p.N)
        __builtin_nontemporal_store(
            v, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + (cur.row0 + R) * (int64_t)p.N + c));
    };
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      __builtin_amdgcn_sched_barrier(0);  // an output row at a time in registers
      g_settle(acc[m]);
      const int R0 = (wm * MF + m) * 16;
      float sa = 0.0f;
      if constexpr (kI8) sa = lds_read<float>(sc + 4 * (kGtCols + R0 + r));
      u32x4 line = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int f = 0; f < kOutF; f += 2) {
        u32x2 half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto value = [&](int blk) __attribute__((always_inline)) {
            if constexpr (kI8) {
              const f32x4 sw = lds_read<f32x4>(sc + 4 * (wn * 16 * NF + 16 * blk + 4 * g));
              f32x4 v;
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = (float)acc[m][blk][q] * sw[q] * sa;
              return v;
            } else {
              return acc[m][blk];
            }
          };
          f32x4 z = value(f + h);
          if constexpr (kL1) {
            const f32x4 u = value(f + h + NF / 2);
#pragma unroll
            for (int q = 0; q < 4; ++q) z[q] = g_silu(z[q]) * u[q];
          }
          half[h] = u32x2{g_pack2(z[0], z[1], f16), g_pack2(z[2], z[3], f16)};
        }
        u32x4 v = g_gather8(half[0], half[1]);
        if constexpr (kOutF == 2) {
          put(R0 + r, c0, v);
        } else if (f & 2) {
          g_whole_lines(line, v);
          const int c = c0 + 16 * (f - 2) + 32 * (r >> 3);
          put(R0 + (r & 7), c, line);
          put(R0 + 8 + (r & 7), c, v);
        } else {
          line = v;
        }
      }
    }
  }
  wait_vmcnt<0>();  // no load is on its way into LDS when the phase, or the workgroup, ends
}

// ============================================================================================
// The same products where tiles of 256 columns would leave most of the chip empty: 64 weight rows (gate+up: 32 of
// each) x 64 token rows a tile, by the same workgroups of 8 waves.
//
// A stage is 256 bytes of K, 32 KB, and the ring holds four: with few products a stage, a tile waits for memory and for
// the barrier (with stages of 128 bytes, 64 x 4096 x 7168 int8 took 26.9 us).  Waves 0-3 multiply a stage's first
// 128 bytes of K, waves 4-7 its second, 32 x 32 each; at a tile's end the second four leave their sums in
// LDS and the first four add and store.  One barrier a stage: behind it everyone's loads of the stage are visible and
// the slot of the stage before is free.
// ============================================================================================
constexpr int kGfStage = 256, kGfSide = 64 * kGfStage, kGfSlot = 2 * kGfSide, kGfD = 4;
constexpr int kGfRedAt = kGfD * kGfSlot, kGfRowsAt = kGfRedAt + 4 * kWave * 64, kGfScalesAt = kGfRowsAt + 2 * 64 * 4;
constexpr int kGfScaleBuf = 4 * (64 + 64);
static_assert(kGfScalesAt + (kGfD + 1) * kGfScaleBuf <= kGtLists, "the LDS layout fits");

template <int kOp, int kDtype, typename Find>
__device__ __forceinline__ void gt_fine_phase(const GroupedArgs& p, int t0, int total, const Find& find) {
  typedef GType<kDtype> T;
  constexpr bool kL1 = kOp == kGtGateUp, kAcross = kOp == kGtAcross, kI8 = kDtype == kOperandI8;
  constexpr int cols = kL1 ? 32 : 64, D = kGfD, L = 4;
  if (t0 >= total) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int64_t RB = (int64_t)p.K * T::kBytes, NB = (int64_t)p.N * T::kBytes;
  const int nks = (int)((RB + kGfStage - 1) / kGfStage);
  const bool tokens = wave >= 4;  // whose rows this wave loads: 16 of the tile's weight rows or token rows
  const int ww = wave & 3;
  const auto piece = [&](int j) { return (lane & 15) ^ (4 * j + (lane >> 4)); };  // of load instruction j: 4 rows by 16

  // ---- loads -------------------------------------------------------------------------------------
  GtTile ld, nx = find(t0);
  int lt = t0;
  int lks = 0, lseq = 0;
  bool done = false;
  uint64_t at[L];
  const auto fetch_rows = [&](int buf) __attribute__((always_inline)) {
    if (!kAcross && p.row_token != nullptr && wave == 0)
      dma4(reinterpret_cast<const uint8_t*>(p.row_token + nx.row0 + (lane < nx.left ? lane : nx.left - 1)),
           kGfRowsAt + 4 * 64 * buf);
  };
  const auto a_row = [&](int R) __attribute__((always_inline)) -> uint32_t {
    if (!kAcross && p.row_token != nullptr) return lds_read<uint32_t>(kGfRowsAt + 4 * (64 * (lseq & 1) + R));
    return (uint32_t)((int)ld.row0 + (R < ld.left ? R : ld.left - 1));
  };
  // Weight row of the tile's row R: gate+up: 16 gate and 16 up rows for either half of the waves.
  const auto w_row = [&](int R) __attribute__((always_inline)) -> int64_t {
    const int c = ld.nt * cols + (kL1 ? R / 32 * 16 + R % 16 : R);
    return (int64_t)ld.e * (kL1 ? 2 : 1) * p.N + (c < p.N ? c : p.N - 1) + (kL1 && (R & 16) ? p.N : 0);
  };
  const auto enter = [&]() __attribute__((always_inline)) {
    ld = nx;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int R = 16 * ww + 4 * j + lane / 16;
      if (tokens) {
        at[j] = reinterpret_cast<uint64_t>(p.a) + (uint64_t)a_row(R) * (uint64_t)RB + 16 * piece(j);
      } else if constexpr (kAcross) {  // 128 rows of the reduced dimension, 128 bytes each, 8 a load
        const int R = 8 * (4 * ww + j) + lane / 8;
        const int c = (lane & 7) ^ ((((R >> 1) & 1) | ((R >> 3) & 1) << 1) << 1), last = p.N / 8 - 1 - ld.nt * 8;
        at[j] = reinterpret_cast<uint64_t>(p.w) + (uint64_t)(((int64_t)ld.e * p.K + R) * NB) + 128 * (uint64_t)ld.nt +
                16 * (c < last ? c : last);
      } else {
        at[j] = reinterpret_cast<uint64_t>(p.w) + (uint64_t)(w_row(R) * RB) + 16 * piece(j);
      }
    }
    if constexpr (kI8) {
      const uint32_t to = kGfScalesAt + (lseq % (D + 1)) * kGfScaleBuf;
      if (wave == 1) dma4(reinterpret_cast<const uint8_t*>(p.w_scales + w_row(lane)), to);
      if (wave == 2) dma4(reinterpret_cast<const uint8_t*>(p.a_scales + a_row(lane)), to + 256);
    }
    if (lt + kGtGrid < total) {
      nx = find(lt + kGtGrid);
      fetch_rows((lseq + 1) & 1);
    }
    ++lseq;
  };
  const bool ragged = (RB & (kGfStage - 1)) != 0;
  const int left = (int)((RB & (kGfStage - 1)) / 16);
  const auto last_stage = [&]() { return lks + 1 == nks && lt + kGtGrid >= total; };
  const auto beyond = [&](int j) __attribute__((always_inline)) {  // what load j brings of a row's last stage lies behind its end
    return (kAcross && !tokens ? 4 * ww + j : piece(j)) >= left;
  };
  // The next stage into a slot.  Behind a row's end: the stage's first piece (or rows) instead, cleared later.
  const auto load = [&](int slot) __attribute__((always_inline)) {
    if (!done && lks == 0) {
      if (nks < D && lseq > 0) {  // its rows were asked for with the tile before, less than a ring ago
        wait_vmcnt<0>();
        g_barrier();
      }
      enter();
    }
    if (ragged && !done && lks + 1 == nks) {
#pragma unroll
      for (int j = 0; j < L; ++j)
        if (beyond(j)) at[j] -= kAcross && !tokens ? (uint64_t)(8 * (4 * ww + j)) * (uint64_t)NB : (uint64_t)(16 * piece(j));
    }
    const uint64_t step = last_stage() ? 0 : kAcross && !tokens ? 128 * (uint64_t)NB : kGfStage;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      dma16(reinterpret_cast<const uint8_t*>(at[j]), slot * kGfSlot + (tokens ? kGfSide : 0) + 1024 * (4 * ww + j));
      at[j] += step;
    }
    if (last_stage()) {
      done = true;
    } else if (++lks == nks) {
      lks = 0;
      lt += kGtGrid;
    }
  };
  const auto clear = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < L; ++j)
      if (beyond(j))
        lds_write16(slot * kGfSlot + (tokens ? kGfSide : 0) + 1024 * (4 * ww + j) + 16 * lane, u32x4{0u, 0u, 0u, 0u});
  };

  g_wait_lds();
  g_barrier();  // the phase before is done with LDS
  fetch_rows(0);
  wait_vmcnt<0>();
  g_barrier();
#pragma unroll 1
  for (int i = 0; i < D - 1; ++i) load(i);

  // ---- products ------------------------------------------------------------------------------------
  const int half = wave >> 2, wm = ww >> 1, wn = ww & 1, r = lane & 15, g = lane >> 4, jj = r >> 2;
  const uint32_t along = r * kGfStage + 16 * ((8 * half + g) ^ r);
  const uint32_t b_at = kGfSide + wm * 32 * kGfStage + along;
  const uint32_t a_at = kAcross ? (64 * half + 8 * g + jj) * 128 + (((2 * wn) ^ ((jj >> 1) | (g & 1) << 1)) * 32) + (lane & 3) * 8
                                : wn * 32 * kGfStage + along;
  int slot = 0, seq = 0;
  for (int t = t0; t < total; t += kGtGrid) {
    typename T::acc acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i / 2][i % 2][q] = 0;
    for (int ks = 0; ks < nks; ++ks) {
      wait_vmcnt<(D - 2) * L>();
      if (ragged && ks + 1 == nks) clear(slot);
      g_wait_lds();
      g_barrier();
      u32x4 a[2][2], b[2][2];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          b[st][i] = lds_read16(slot * kGfSlot + (b_at ^ (st * 64)) + i * 16 * kGfStage);
          if constexpr (kAcross) {
            a[st][i] = lds_read_across<128>(slot * kGfSlot + (a_at ^ (i * 32)) + st * 32 * 128);
          } else {
            a[st][i] = lds_read16(slot * kGfSlot + (a_at ^ (st * 64)) + i * 16 * kGfStage);
          }
        }
      load(slot == 0 ? D - 1 : slot - 1);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int f = 0; f < 2; ++f) acc[m][f] = T::product(a[st][f], b[st][m], acc[m][f]);
      slot = slot + 1 == D ? 0 : slot + 1;
    }
    const uint32_t red = kGfRedAt + (ww * kWave + lane) * 16;
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lds_write16(red + i * 4 * kWave * 16, __builtin_bit_cast(u32x4, acc[i / 2][i % 2]));
    }
    g_wait_lds();
    g_barrier();
    const uint32_t sc = kGfScalesAt + (seq % (D + 1)) * kGfScaleBuf;
    ++seq;
    if (half == 1) continue;
    const GtTile cur = find(t);
    const bool f16 = p.out_dtype == MEGAMOE_DTYPE_F16;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int R = wm * 32 + 16 * m + r;
      f32x4 z[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const typename T::acc sum =
            acc[m][f] + __builtin_bit_cast(typename T::acc, lds_read16(red + (2 * m + f) * 4 * kWave * 16));
        if constexpr (kI8) {
          const f32x4 sw = lds_read<f32x4>(sc + 4 * (wn * 32 + 16 * f + 4 * g));
          const float sa = lds_read<float>(sc + 256 + 4 * R);
#pragma unroll
          for (int q = 0; q < 4; ++q) z[f][q] = (float)sum[q] * sw[q] * sa;
        } else {
          z[f] = sum;
        }
      }
      uint16_t* const out = static_cast<uint16_t*>(p.out) + (cur.row0 + R) * (int64_t)p.N;
      if constexpr (kL1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) z[0][q] = g_silu(z[0][q]) * z[1][q];
        const int c = cur.nt * cols + wn * 16 + 4 * g;
        if (R < cur.left && c < p.N)
          *reinterpret_cast<u32x2*>(out + c) = u32x2{g_pack2(z[0][0], z[0][1], f16), g_pack2(z[0][2], z[0][3], f16)};
      } else {
        const u32x4 v = g_gather8(u32x2{g_pack2(z[0][0], z[0][1], f16), g_pack2(z[0][2], z[0][3], f16)},
                                  u32x2{g_pack2(z[1][0], z[1][1], f16), g_pack2(z[1][2], z[1][3], f16)});
        const int c = cur.nt * cols + wn * 32 + 16 * (g & 1) + 8 * (g >> 1);
        if (R < cur.left && c < p.N) *reinterpret_cast<u32x4*>(out + c) = v;
      }
    }
  }
  wait_vmcnt<0>();
}

// Whether the tiles of 64 take the call: the time of the fullest workgroup either way, of tiles of nks stages.
// (Large and small tiles, us: int8 256 x 4096 x 7168 71 and 16, 1024 rows 86 and 51, 2048 rows 88 and 99; bf16 16
// experts of 288 rows, 3640 to 176, 118 and 19; 64 of 94 rows, 2048 to 7168, 402 and 534; 48 of 40 rows, 7168 to 4096,
// 404 and 479; 8 of 32, 512 to 1024, 10.7 and 7.2; across, 24 of 100 rows, 2048 to 1024, 39 and 28.)
// In float32: a division of 64-bit integers lasts longer than all of the rest.
__device__ __forceinline__ bool gt_fine(int m4, int m2, int m1, int mf, int ntn, int ntf, int nks) {
  const float t4 = (float)(nks * kGtNs4[0] + kGtNs4[1]), t2 = (float)(nks * kGtNs2[0] + kGtNs2[1]);
  const float t1 = (float)(nks * kGtNs1[0] + kGtNs1[1]);
  const float tf = (float)(nks * (m4 || m2 ? kGtNsFine[0] : kGtNsFineAlone) + kGtNsFine[1]);
  const float one = m4 ? t4 : m2 ? t2 : t1, n = (float)(m4 + m2 + m1), per = 1.0f / kGtGrid;
  const float rounds = ceilf(n * (float)ntn * per);
  const float all = n > 0.0f ? ((float)m4 * t4 + (float)m2 * t2 + (float)m1 * t1) * __builtin_amdgcn_rcpf(n) * rounds : 0.0f;
  return ceilf((float)mf * (float)ntf * per) * tf < (all < one ? one : all);
}

template <int kOp, int kDtype>
__global__ __launch_bounds__(kGtThreads, 1) void gt_kernel(GroupedArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_gt[];
  int* const s_n = reinterpret_cast<int*>(s_gt + kGtLists);
  int* const pref = s_n + 2;                                              // 256-row m-tiles before each expert [E + 1]
  uint16_t* const list2 = reinterpret_cast<uint16_t*>(pref + p.E + 1);    // experts with a last tile of 128 rows
  uint16_t* const list1 = list2 + p.E;                                    // of 64
  const int E = p.E, lane = lane_id();
  constexpr int cols = kOp == kGtGateUp ? kGtCols / 2 : kGtCols;
  const int ntn = (p.N + cols - 1) / cols, ntf = (p.N + cols / 4 - 1) / (cols / 4);
  if (threadIdx.x < kWave) {
    const auto rows_of = [&](int e) {
      return e < E ? p.counts ? p.counts[e] : (int)p.M : 0;
    };
    const auto last = [&](int rest) { return rest > 128 ? 4 : rest > 64 ? 2 : rest > 0 ? 1 : 0; };  // tile of a last part
    int own4 = 0, own2 = 0, own1 = 0, ownf = 0;
    for (int c = lane; c < E; c += kWave) {
      const int cnt = rows_of(c), l = last(cnt % kGtRows);
      own4 += cnt / kGtRows + (l == 4);
      own2 += l == 2;
      own1 += l == 1;
      ownf += g_parts(cnt, 64);
    }
    const bool fine = gt_fine(g_total(own4), g_total(own2), g_total(own1), g_total(ownf), ntn, ntf,
                              (int)(((int64_t)p.K * GType<kDtype>::kBytes + kGtStage - 1) / kGtStage));
    int carry = 0, n2 = 0, n1 = 0;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (int c = 0; c < E; c += kWave) {
      const int cnt = rows_of(c + lane), l = last(cnt % kGtRows);
      const int own = fine ? g_parts(cnt, 64) : cnt / kGtRows + (l == 4);
      const int incl = g_scan(own);
      if (c + lane < E) pref[c + lane] = carry + incl - own;
      carry += __builtin_amdgcn_readlane(incl, kWave - 1);
      const uint64_t b2 = __ballot(l == 2), b1 = __ballot(l == 1);
      if (l == 2) list2[n2 + __popcll(b2 & below)] = (uint16_t)(c + lane);
      if (l == 1) list1[n1 + __popcll(b1 & below)] = (uint16_t)(c + lane);
      n2 += __popcll(b2);
      n1 += __popcll(b1);
    }
    if (lane == 0) {
      pref[E] = carry;
      s_n[0] = fine ? -1 : n2;
      s_n[1] = n1;
    }
  }
  __syncthreads();
  const bool fine = __builtin_amdgcn_readfirstlane(s_n[0]) < 0;
  const int total4 = __builtin_amdgcn_readfirstlane(pref[E]) * (fine ? ntf : ntn);
  const int total2 = __builtin_amdgcn_readfirstlane(s_n[0]) * ntn;
  const int total1 = __builtin_amdgcn_readfirstlane(s_n[1]) * ntn;
  const auto count = [&](int e) { return p.counts ? g_scalar(p.counts + e) : (int)p.M; };
  const auto offset = [&](int e) { return (int64_t)(p.padded_offsets ? g_scalar(p.padded_offsets + e) : 0); };
  // (Tile numbers fit 32 bits: a tile has 4096 outputs and more, and 2^31 of them would not fit the GPU.)
  // Tile t of those of 256 (or 64) rows: its expert by two steps of 64 comparisons (at most 1024 experts).
  const auto find_tile = [&](int t, int rows, int ntn) __attribute__((always_inline)) {
    const int step = (E + kWave - 1) / kWave;
    const int at = lane * step;
    const int chunk = __popcll(__ballot(at < E && pref[at < E ? at : 0] * ntn <= t)) - 1;
    const int at2 = chunk * step + lane;
    const int e = __builtin_amdgcn_readfirstlane(
        chunk * step - 1 + __popcll(__ballot(lane < step && at2 < E && pref[at2 < E ? at2 : 0] * ntn <= t)));
    const int first = __builtin_amdgcn_readfirstlane(pref[e]);
    const int mts = __builtin_amdgcn_readfirstlane(pref[e + 1]) - first;
    const int local = t - first * ntn;
    const int band = local / (kGtBand * ntn), in = local % (kGtBand * ntn);
    const int width = min(kGtBand, mts - band * kGtBand);
    const int mt = band * kGtBand + in % width;
    return GtTile{e, in / width, count(e) - mt * rows, offset(e) + (int64_t)mt * rows};
  };
  const auto find4 = [&](int t) __attribute__((always_inline)) { return find_tile(t, kGtRows, ntn); };
  const auto find_last = [&](const uint16_t* list, int t) __attribute__((always_inline)) {
    const int e = __builtin_amdgcn_readfirstlane((int)list[t / ntn]);
    const int cnt = count(e), mt = cnt / kGtRows;
    return GtTile{e, t % ntn, cnt - mt * kGtRows, offset(e) + (int64_t)mt * kGtRows};
  };
  // XCD b % 8 takes 32 tiles in a row of every 256: they share rows and weights in its L2.  The lists follow each
  // other, so that a workgroup that has one tile more of one list has one less of the next.
  const int wg = (blockIdx.x % 8) * (kGtGrid / 8) + blockIdx.x / 8;
  const auto first = [&](int before) { return (wg - before % kGtGrid + kGtGrid) % kGtGrid; };
  if (fine) {
    gt_fine_phase<kOp, kDtype>(p, wg, total4, [&](int t) __attribute__((always_inline)) { return find_tile(t, 64, ntf); });
    return;
  }
  gt_phase<kOp, kDtype, 4>(p, wg, total4, find4);
  gt_phase<kOp, kDtype, 2>(p, first(total4), total2, [&](int t) { return find_last(list2, t); });
  gt_phase<kOp, kDtype, 1>(p, first(total4 + total2), total1, [&](int t) { return find_last(list1, t); });
}

// ============================================================================================
// weights: 256 columns of x by 256 columns of dy a tile, both read across: the expert's rows are the reduced
// dimension, 64 a stage.  The ring, the barrier and the steps are those above.
//
// Long experts: as the rows (16384 x 7168 x 4096: 789 us, 1220 TFLOP/s).  Short ones: the gradients' stores, which
// no products run beside, since all workgroups store at about the same time (48 experts of 512 rows, float32 7168 x
// 4096: 2080 us, 1250 without the stores; of 64 experts of 32 rows 1440, 5.3 TB/s; in 16 bits 1590 and 840).  With
// accumulate the old values are read between the products and the stores, beside nothing else: 3470 and 3550 (3.4 and
// 4.2 TB/s), in 16 bits 2640 and 2520.  Tiles of another order for each XCD, so that they store at other times: slower.
// ============================================================================================
constexpr int kGwSlot = 2 * kGtSide;
constexpr int kGwTokens = 2 * kGwSlot;               // LDS: the waves' tokens of two stages' rows
static_assert(kGwTokens + kGtWaves * 2 * 64 * 4 <= kGtLds, "the LDS layout fits");

// Old values added to four consecutive gradients, at `out` (accumulate).
__device__ __forceinline__ f32x4 gw_add(f32x4 z, const uint8_t* out, int dtype) {
  if (dtype == MEGAMOE_DTYPE_F32) return z + *reinterpret_cast<const f32x4*>(out);
  const u32x2 old = *reinterpret_cast<const u32x2*>(out);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t bits = (old[q / 2] >> (16 * (q & 1))) & 0xFFFFu;
    const uint16_t b16 = (uint16_t)bits;
    z[q] += dtype == MEGAMOE_DTYPE_F16 ? (float)__builtin_bit_cast(_Float16, b16) : bf16_bits_to_f32(bits);
  }
  return z;
}

// Small matrices: 64 columns of x by 64 of dy a tile, 128 of the expert's rows a stage, as the tiles of 64 x 64 above:
// a ring of four slots, one barrier a stage, half of the waves on either half of its rows.  Gathered rows: the
// expert's tokens lie in LDS (at most kGwMaxTokens; longer experts are left to the large tiles).
constexpr int kGwFineStage = 128, kGwMaxTokens = 3584, kGwFineTokens = kGfRedAt + 4 * kWave * 64;
static_assert(kGwFineTokens + 4 * kGwMaxTokens <= kGtLds, "the LDS layout fits");

template <int kDtype, bool kGather>
__device__ __forceinline__ void gw_fine_phase(const GroupedWgradArgs& p) {
  typedef GType<kDtype> T;
  constexpr int D = kGfD, L = 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id(), ww = wave & 3;
  const bool dy = wave >= 4;  // whose columns this wave loads: 32 of a stage's rows
  const int64_t KB = (int64_t)p.K * 2, NB = (int64_t)p.N * 2, own_bytes = dy ? NB : KB;
  const int ntk = (p.K + 63) / 64, ntn = (p.N + 63) / 64, per = ntk * ntn;
  const int64_t total = (int64_t)p.E * per;
  struct Tile {
    int e, kt, nt, cnt;
    int64_t row0;
  };
  const auto find = [&](int64_t t) __attribute__((always_inline)) {
    Tile x;
    x.e = (int)(t / per);
    const int in = (int)(t % per);
    x.nt = in % ntn;
    x.kt = in / ntn;
    x.cnt = g_scalar(p.counts + x.e);
    x.row0 = g_scalar(p.padded_offsets + x.e);
    return x;
  };
  const auto stages = [&](const Tile& x) { return x.cnt > 0 ? g_parts(x.cnt, kGwFineStage) : 1; };
  const int64_t t0 = (blockIdx.x % 8) * (kGtGrid / 8) + blockIdx.x / 8;
  if (t0 >= total) return;

  Tile ld;
  int64_t lt = t0;
  int lks = 0, lnks = 0, l_expert = -1;
  bool done = false;
  uint64_t base[L];
  const auto row = [&](int j) { return 8 * (4 * ww + j) + lane / 8; };  // of a stage's 128, of load instruction j
  const auto load = [&](int slot) __attribute__((always_inline)) {
    if (!done && lks == 0) {
      ld = find(lt);
      lnks = stages(ld);
      if (kGather && ld.e != l_expert && ld.cnt > 0) {
        g_wait_lds();
        g_barrier();  // the tokens before have been read
        for (int at = 64 * wave; at < ld.cnt; at += 64 * kGtWaves)
          dma4(reinterpret_cast<const uint8_t*>(p.row_token + ld.row0 + (at + lane < ld.cnt ? at + lane : ld.cnt - 1)),
               kGwFineTokens + 4 * at);
        wait_vmcnt<0>();
        g_barrier();
        l_expert = ld.e;
      }
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int R = row(j), c = (lane & 7) ^ ((((R >> 1) & 1) | ((R >> 3) & 1) << 1) << 1);
        const int last = (int)(own_bytes / 16) - 1 - (dy ? ld.nt : ld.kt) * 8;
        base[j] = reinterpret_cast<uint64_t>(dy ? p.dy : p.x) + 128 * (uint64_t)(dy ? ld.nt : ld.kt) +
                  16 * (c < last ? c : last) + (kGather && !dy ? 0 : (uint64_t)(ld.row0 * own_bytes));
      }
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int at = kGwFineStage * lks + row(j), r = at < ld.cnt ? at : ld.cnt - 1;  // behind the last row: that; cleared later
      const uint32_t src = kGather && !dy ? lds_read<uint32_t>(kGwFineTokens + 4 * (r < 0 ? 0 : r)) : (uint32_t)r;
      const uint64_t from = base[j] + (uint64_t)src * (uint64_t)(uint32_t)own_bytes;
      dma16(ld.cnt > 0 ? reinterpret_cast<const uint8_t*>(from) : reinterpret_cast<const uint8_t*>(g_zeros),
            slot * kGfSlot + (dy ? kGfSide : 0) + 1024 * (4 * ww + j));
    }
    if (done) return;
    if (lks + 1 == lnks && lt + kGtGrid >= total) {
      done = true;  // with nothing left the last stage is loaded again, and not used
    } else if (++lks == lnks) {
      lks = 0;
      lt += kGtGrid;
    }
  };
#pragma unroll 1
  for (int i = 0; i < D - 1; ++i) load(i);

  const int half = wave >> 2, wm = ww >> 1, wn = ww & 1, r = lane & 15, g = lane >> 4, jj = r >> 2;
  const uint32_t across = (64 * half + 8 * g + jj) * 128 + (lane & 3) * 8, v = (jj >> 1) | (g & 1) << 1;
  const uint32_t a_at = across + ((2 * wn) ^ v) * 32, b_at = kGfSide + across + ((2 * wm) ^ v) * 32;
  int slot = 0;
  for (int64_t t = t0; t < total; t += kGtGrid) {
    const Tile cur = find(t);
    const int nks = stages(cur);
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i / 2][i % 2][q] = 0.0f;
    for (int ks = 0; ks < nks; ++ks) {
      wait_vmcnt<(D - 2) * L>();
      if (cur.cnt - kGwFineStage * ks < kGwFineStage) {
#pragma unroll
        for (int j = 0; j < L; ++j)
          if (kGwFineStage * ks + row(j) >= cur.cnt)
            lds_write16(slot * kGfSlot + (dy ? kGfSide : 0) + 1024 * (4 * ww + j) + 16 * lane, u32x4{0u, 0u, 0u, 0u});
      }
      g_wait_lds();
      g_barrier();
      u32x4 a[2][2], b[2][2];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[st][i] = lds_read_across<128>(slot * kGfSlot + (a_at ^ (i * 32)) + st * 32 * 128);
          b[st][i] = lds_read_across<128>(slot * kGfSlot + (b_at ^ (i * 32)) + st * 32 * 128);
        }
      load(slot == 0 ? D - 1 : slot - 1);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int f = 0; f < 2; ++f) acc[m][f] = T::product(a[st][f], b[st][m], acc[m][f]);
      slot = slot + 1 == D ? 0 : slot + 1;
    }
    const uint32_t red = kGfRedAt + (ww * kWave + lane) * 16;
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lds_write16(red + i * 4 * kWave * 16, __builtin_bit_cast(u32x4, acc[i / 2][i % 2]));
    }
    g_wait_lds();
    g_barrier();
    if (half == 1 || (cur.cnt == 0 && p.accumulate)) continue;
    const bool f32 = p.dw_dtype == MEGAMOE_DTYPE_F32, f16 = p.dw_dtype == MEGAMOE_DTYPE_F16;
    const int64_t bytes = f32 ? 4 : 2;
    const auto place = [&](int n, int k) __attribute__((always_inline)) {
      return static_cast<uint8_t*>(p.dw) + (((int64_t)cur.e * p.N + n) * p.K + k) * bytes;
    };
    const int k0 = cur.kt * 64 + wn * 32;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int n0 = cur.nt * 64 + wm * 32 + 16 * m, n = n0 + r;
      f32x4 z[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        z[f] = acc[m][f] + __builtin_bit_cast(f32x4, lds_read16(red + (2 * m + f) * 4 * kWave * 16));
        const int k = k0 + 16 * f + 4 * g;
        if (p.accumulate && n < p.N && k < p.K) z[f] = gw_add(z[f], place(n, k), p.dw_dtype);
      }
      const auto put = [&](int n, int k, u32x4 v) __attribute__((always_inline)) {
        if (n < p.N && k < p.K) *reinterpret_cast<u32x4*>(place(n, k)) = v;
      };
      if (f32) {
        u32x4 lo = __builtin_bit_cast(u32x4, z[0]), hi = __builtin_bit_cast(u32x4, z[1]);
        g_whole_lines(lo, hi);
        put(n0 + (r & 7), k0 + 16 * (r >> 3) + 4 * g, lo);
        put(n0 + 8 + (r & 7), k0 + 16 * (r >> 3) + 4 * g, hi);
      } else {
        put(n, k0 + 16 * (g & 1) + 8 * (g >> 1),
            g_gather8(u32x2{g_pack2(z[0][0], z[0][1], f16), g_pack2(z[0][2], z[0][3], f16)},
                      u32x2{g_pack2(z[1][0], z[1][1], f16), g_pack2(z[1][2], z[1][3], f16)}));
      }
    }
  }
  wait_vmcnt<0>();
}

// Whether the tiles of 64 x 64 take the call: the time of the fullest workgroup either way, from the counts.  (Large and
// small tiles, us: 4 experts of 945 rows, 40 x 696, 25.8 and 8.2; 4 of 2233, 160 x 816, 57 and 16; 1 of 469, 3496 x 456,
// 22 and 11; 8 of 15, 520 x 1032, 12.3 and 13.3; 48 of 100, 1024 x 1024, 42 and 91.)
__device__ __forceinline__ bool gw_fine(const GroupedWgradArgs& p, bool gather) {
  const int64_t per = (int64_t)((p.K + 255) / 256) * ((p.N + 255) / 256), perf = (int64_t)((p.K + 63) / 64) * ((p.N + 63) / 64);
  int coarse = 0, fine = 0, most = 0;  // a tile of every expert, in tenths of a us; the largest count
  for (int e = lane_id(); e < p.E; e += kWave) {
    const int cnt = p.counts[e];
    coarse += 14 * g_parts(cnt, 64) + kGwTile;
    fine += 5 * g_parts(cnt, kGwFineStage) + kGwFineTile;
    most = most > cnt ? most : cnt;
  }
  const int64_t all = (int64_t)g_total(coarse) * per, all_fine = (int64_t)g_total(fine) * perf;
  most = (int)wave_max_u32((uint32_t)most);
  if (gather && most > kGwMaxTokens) return false;
  const int64_t one = 14 * (int64_t)g_parts(most, 64) + kGwTile;
  const int64_t one_fine = 5 * (int64_t)g_parts(most, kGwFineStage) + kGwFineTile;
  return (all_fine / kGtGrid > one_fine ? all_fine / kGtGrid : one_fine) < (all / kGtGrid > one ? all / kGtGrid : one);
}

template <int kDtype, bool kGather>
__global__ __launch_bounds__(kGtThreads, 1) void gt_weights_kernel(GroupedWgradArgs p) {
  if (gw_fine(p, kGather)) {
    gw_fine_phase<kDtype, kGather>(p);
    return;
  }
  extern __shared__ __attribute__((aligned(16))) uint8_t s_gt[];
  typedef GType<kDtype> T;
  constexpr int MF = 4, NF = 8, L = 8;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int64_t KB = (int64_t)p.K * 2, NB = (int64_t)p.N * 2;
  const int ntk = (p.K + kGtCols - 1) / kGtCols, ntn = (p.N + kGtRows - 1) / kGtRows;
  const int per = ntk * ntn;
  const int64_t total = (int64_t)p.E * per;
  const uint8_t* const pad = reinterpret_cast<const uint8_t*>(g_zeros);

  struct Tile {
    int e, kt, nt, cnt;
    int64_t row0;
  };
  const auto find = [&](int64_t t) __attribute__((always_inline)) {
    Tile x;
    x.e = (int)(t / per);
    const int in = (int)(t % per), band = in / (kGtBand * ntk), ib = in % (kGtBand * ntk);
    const int width = min(kGtBand, ntn - band * kGtBand);
    x.nt = band * kGtBand + ib % width;
    x.kt = ib / width;
    x.cnt = g_scalar(p.counts + x.e);
    x.row0 = g_scalar(p.padded_offsets + x.e);
    return x;
  };
  const auto stages = [&](const Tile& x) { return x.cnt > 0 ? g_parts(x.cnt, 64) : 1; };

  const int64_t t0 = (blockIdx.x % 8) * (kGtGrid / 8) + blockIdx.x / 8;
  if (t0 >= total) return;
  const auto row = [&]() __attribute__((always_inline)) { return 8 * wave + (g_here(lane) >> 5); };  // of a stage's 64, of load 0
  Tile ld = find(t0), ldn = ld;
  int64_t lt = t0;
  int lks = 0, lnks = 0, lq = 0;  // lq: parity of the stage's tokens
  uint32_t x_off[2], y_off[2];  // of even and odd load instructions
  const uint8_t *x_at = nullptr, *y_at = nullptr;
  const uint32_t tok_at = kGwTokens + wave * 2 * 64 * 4;
  const auto fetch = [&](const Tile& x, int ks, int q) __attribute__((always_inline)) {  // tokens of the stage's rows
    if (kGather && x.cnt > 0) {
      const int R = 64 * ks + g_here(lane);
      dma4(reinterpret_cast<const uint8_t*>(p.row_token + x.row0 + (R < x.cnt ? R : x.cnt - 1)), tok_at + 256 * (q & 1));
    }
  };
  const auto enter = [&]() __attribute__((always_inline)) {
    const int ln = g_here(lane);
    lnks = stages(ld);
    if (lt + kGtGrid < total) ldn = find(lt + kGtGrid);
    x_at = static_cast<const uint8_t*>(p.x) + (int64_t)ld.kt * kGtCols * 2 + (kGather ? 0 : (ld.row0 + 8 * wave) * KB);
    y_at = static_cast<const uint8_t*>(p.dy) + (int64_t)ld.nt * kGtRows * 2 + (ld.row0 + 8 * wave) * NB;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = (ln & 31) ^ (((2 * q + (ln >> 5)) | ((wave & 1) << 2)) << 1);
      const int lk = p.K / 8 - 1 - ld.kt * 32, lnn = p.N / 8 - 1 - ld.nt * 32;
      x_off[q] = 16 * (c < lk ? c : lk) + (kGather ? 0u : (uint32_t)(ln >> 5) * (uint32_t)KB);
      y_off[q] = 16 * (c < lnn ? c : lnn) + (uint32_t)(ln >> 5) * (uint32_t)NB;
    }
  };
  uint32_t tok[4];
  bool done = false;  // with nothing left the last stage is loaded again, into a slot that no product reads
  const auto begin = [&]() __attribute__((always_inline)) {  // of the stage at (lt, lks)
    if (lks == 0) enter();
    if (kGather) {
      if (lks + 1 < lnks) fetch(ld, lks + 1, lq + 1);
      else if (lt + kGtGrid < total) fetch(ldn, 0, lq + 1);
    }
  };
  // Load j of the stage: dy, then x.  tail: the expert's rows end in it.
  const auto load = [&](int j, bool tail, int slot) __attribute__((always_inline)) {
    const int i = j & 3;
    const uint32_t to = slot * kGwSlot + (j < 4 ? kGtSide : 0) + 1024 * (4 * wave + i);
    const auto in = [&]() __attribute__((always_inline)) { return row() + 2 * i < ld.cnt - 64 * lks; };
    if (j >= 4 && kGather) {
      const uint8_t* src = x_at + ((uint64_t)tok[i] * (uint64_t)(uint32_t)KB + x_off[i & 1]);
      if (__builtin_expect(tail, 0)) src = in() ? src : pad;
      dma16(src, to);
    } else {
      const uint8_t* const base = j < 4 ? y_at + 2 * i * NB : x_at + 2 * i * KB;
      const uint32_t off = (j < 4 ? y_off : x_off)[i & 1];
      if (__builtin_expect(tail, 0)) dma16(in() ? base + off : pad, to);
      else dma16s(base, off, to);
    }
    if (kGather && j < 4)  // row j's token, four loads before it is used
      tok[j] = lds_read<uint32_t>(tok_at + 256 * (lq & 1) + 4 * (row() + 2 * j));
  };
  const auto tail_stage = [&]() { return ld.cnt - 64 * lks < 64; };
  const auto loaded = [&]() __attribute__((always_inline)) {
    if (lks + 1 == lnks && lt + kGtGrid >= total) {
      done = true;
      return;
    }
    if (!kGather) x_at += 64 * KB;
    y_at += 64 * NB;
    ++lq;
    if (++lks == lnks) {
      lks = 0;
      lt += kGtGrid;
      ld = ldn;
    }
  };

  const int wm = wave / 2, wn = wave % 2, g = lane >> 4, jj = (lane & 15) >> 2;  // 64 rows of dy by 128 of x a wave
  const uint32_t v = jj | ((g & 1) << 2), lane_at = (8 * g + jj) * 512 + (lane & 3) * 8;
  const uint32_t a_base = lane_at + wn * 256 + v * 32, b_base = kGtSide + lane_at + ((4 * wm) ^ v) * 32;
  u32x4 a[2][NF], b[2][MF];
  uint32_t ra, rb;
  const auto aim = [&](int slot) __attribute__((always_inline)) {
    ra = a_base + slot * kGwSlot;
    rb = b_base + slot * kGwSlot;
    asm volatile("" : "+v"(ra), "+v"(rb));
  };
  const auto read_one = [&](int st, int i) __attribute__((always_inline)) {
    if (i < MF) b[st][i] = lds_read_across<512>((rb ^ (i * 32)) + st * 32 * 512);
    else a[st][i - MF] = lds_read_across<512>((ra ^ ((i - MF) * 32)) + st * 32 * 512);
  };

  fetch(ld, 0, 0);
  for (int n = 0; n < 2; ++n) {
    wait_vmcnt<0>();  // the stage's tokens (the wave's own)
    asm volatile("" ::: "memory");
    if (!done) begin();
#pragma unroll
    for (int j = 0; j < L; ++j) load(j, tail_stage(), n);
    if (!done) loaded();
  }
  wait_vmcnt<L>();
  g_barrier();
  aim(0);
#pragma unroll
  for (int i = 0; i < MF + NF; ++i) read_one(0, i);

  int slot = 0;
  for (int64_t t = t0; t < total; t += kGtGrid) {
    const Tile cur = find(t);
    const int nks = stages(cur);
    f32x4 acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][f][q] = 0.0f;
#pragma unroll
    for (int m = 0; m < MF; ++m) g_settle(acc[m]);
    for (int ks = 0; ks < nks; ++ks) {
      gt_step<T, MF, NF, MF + NF, 0>(acc, a[0], b[0], [&](int i) __attribute__((always_inline)) { read_one(1, i); }, GtNothing{});
      g_wait_lds();
      wait_vmcnt<0>();
      g_barrier();
      if (!done) begin();
      const bool tail = tail_stage();
      aim(slot ^ 1);
      gt_step<T, MF, NF, MF + NF, L>(acc, a[1], b[1], [&](int i) __attribute__((always_inline)) { read_one(0, i); },
                                     [&](int j) __attribute__((always_inline)) { load(j, tail, slot); });
      if (!done) loaded();
      slot ^= 1;
    }
    if (cur.cnt == 0 && p.accumulate) continue;
    const bool f32 = p.dw_dtype == MEGAMOE_DTYPE_F32, f16 = p.dw_dtype == MEGAMOE_DTYPE_F16;
    const int k0 = cur.kt * kGtCols + wn * 128;
    const int le = g_here(lane), r = le & 15, g = le >> 4;
    uint8_t* const out = static_cast<uint8_t*>(p.dw);
    const int bytes = f32 ? 4 : 2;
    const auto at = [&](int n, int k) __attribute__((always_inline)) { return (((int64_t)cur.e * p.N + n) * p.K + k) * bytes; };
    const auto put = [&](int n, int k, u32x4 v) __attribute__((always_inline)) {
      if (n < p.N && k < p.K) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + at(n, k)));
    };
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      __builtin_amdgcn_sched_barrier(0);
      g_settle(acc[m]);
      const int n0 = cur.nt * kGtRows + wm * 64 + 16 * m, n = n0 + r;
      u32x4 line = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int f = 0; f < NF; f += 2) {
        f32x4 z[2] = {acc[m][f], acc[m][f + 1]};
        if (p.accumulate) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = k0 + 16 * (f + h) + 4 * g;
            if (n >= p.N || k >= p.K) continue;
            z[h] = gw_add(z[h], out + at(n, k), p.dw_dtype);
          }
        }
        if (f32) {
          u32x4 lo = __builtin_bit_cast(u32x4, z[0]), hi = __builtin_bit_cast(u32x4, z[1]);
          g_whole_lines(lo, hi);
          const int k = k0 + 16 * f + 16 * (r >> 3) + 4 * g;
          put(n0 + (r & 7), k, lo);
          put(n0 + 8 + (r & 7), k, hi);
        } else {
          u32x4 v = g_gather8(u32x2{g_pack2(z[0][0], z[0][1], f16), g_pack2(z[0][2], z[0][3], f16)},
                              u32x2{g_pack2(z[1][0], z[1][1], f16), g_pack2(z[1][2], z[1][3], f16)});
          if (f & 2) {
            g_whole_lines(line, v);
            const int k = k0 + 16 * (f - 2) + 32 * (r >> 3) + 16 * (g & 1) + 8 * (g >> 1);
            put(n0 + (r & 7), k, line);
            put(n0 + 8 + (r & 7), k, v);
          } else {
            line = v;
          }
        }
      }
    }
  }
  wait_vmcnt<0>();  // no load is on its way into LDS when the workgroup ends
}

// ============================================================================================
// Experts (or a dense call) of few rows: the weights' bytes are the work.
//
// Work unit: a group, 16 weight rows over the whole of K for one m-tile of up to kGsRows token rows; the groups of
// all m-tiles are laid end to end and every workgroup (4 waves, one a CU) takes an equal range.  A wave streams its
// part of the weight rows through an LDS ring of its own, 16 rows by 256 bytes a slot with the m-tile's token rows
// beside them (they come from the L2), by direct loads: no barrier, no registers, and the ring runs on across groups,
// m-tiles and experts.  kSplit: the 4 waves split K; at a group's end they leave their sums in LDS and one of them
// adds the four in wave order.  Otherwise every wave takes groups of its own.  int8 gate+up of 8 tokens, 7168 to
// 2 x 2048, takes 25 us at 5 experts (5.8 TB/s), 51 at 11 (6.4); bf16, 7168 to 4096, 47 (6.3) and 98 (6.6).  Small
// calls are bound by the start and by groups taken in turn, on the GPU: 8 x 7168 x 2048 int8, whose bytes take 2.1 us,
// takes 6.8 us a call and 7.2 to 7.5 in a kernel trace, as most workgroups take two groups with a barrier each.
//
// Both operands keep 16-byte piece c of row R at place c ^ R of the row's 256 bytes: the 16 rows of one piece are
// read from 16 different places.
// ============================================================================================
constexpr int kGsRows = 16, kGsWaves = 4, kGsChunk = 256, kGsMaxSlots = 8;
constexpr int kGsWeights = 16 * kGsChunk;                                         // LDS bytes of a slot's weights
constexpr int kGsRed = 2 * kGsWaves * kWave * 16;
constexpr int kGsLists = (2 * MEGAMOE_MAX_EXPERTS + 4 * (MEGAMOE_MAX_EXPERTS + 1) + 4 + 15) / 16 * 16;  // experts, m-tile prefix
constexpr int kGsSplitChunks = 16;  // K of so many chunks is split over the waves
constexpr int kGsScales = 256;                                                     // int8: of a slot

__host__ __device__ constexpr int gs_slot_bytes(bool i8, int mrows) {
  return kGsWeights + mrows * kGsChunk + (i8 ? kGsScales : 0);
}

// Waits until at most `after` (<= K) later slots' loads are outstanding for this wave, of at least 5 each.
template <int K>
__device__ __forceinline__ void gs_wait_slots(int after) {
  if constexpr (K > 0) {
    if (after < K) {
      gs_wait_slots<K - 1>(after);
      return;
    }
  }
  wait_vmcnt<5 * K>();
}

template <bool kL1, int kDtype, bool kSplit>
__global__ __launch_bounds__(kGsWaves* kWave, 1) void gs_kernel(GroupedArgs p, int slots, int mrows) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_gt[];
  typedef GType<kDtype> T;
  constexpr bool kI8 = kDtype == kOperandI8;
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int* const pref = reinterpret_cast<int*>(s_gt);                          // m-tiles before each listed expert
  uint16_t* const list = reinterpret_cast<uint16_t*>(pref + MEGAMOE_MAX_EXPERTS + 2);
  const int slot_bytes = gs_slot_bytes(kI8, mrows);
  const uint32_t red_at = kGsLists, ring_at = kGsLists + (kSplit ? kGsRed : 0) + wave * slots * slot_bytes;
  const int64_t RB = (int64_t)p.K * T::kBytes;
  const int nch = (int)((RB + kGsChunk - 1) / kGsChunk), rest = (int)(RB / 16 - (int64_t)(nch - 1) * 16);  // pieces of the last

  // The experts that have rows and their m-tiles.
  int listed = 1;
  if (p.counts != nullptr) {
    if (wave == 0) {
      int n = 0, tiles = 0;
      for (int c = 0; c < p.E; c += kWave) {
        const int cnt = c + lane < p.E ? p.counts[c + lane] : 0;
        const int own = g_parts(cnt, mrows);
        const int incl = g_scan(own);
        const uint64_t any = __ballot(own > 0);
        const int at = n + __popcll(any & (((uint64_t)1 << lane) - 1));
        if (own > 0) {
          list[at] = (uint16_t)(c + lane);
          pref[at] = tiles + incl - own;
        }
        n += __popcll(any);
        tiles += __builtin_amdgcn_readlane(incl, kWave - 1);
      }
      if (lane == 0) {
        pref[n] = tiles;
        pref[MEGAMOE_MAX_EXPERTS + 1] = n;
      }
    }
    __syncthreads();
    listed = __builtin_amdgcn_readfirstlane(pref[MEGAMOE_MAX_EXPERTS + 1]);
  }
  const int64_t tiles = p.counts ? __builtin_amdgcn_readfirstlane(pref[listed]) : (p.M + mrows - 1) / mrows;
  constexpr int unit = kL1 ? 8 : 16;  // output columns of a group
  const int nt = (p.N + unit - 1) / unit;
  const int64_t groups = tiles * nt;
  // XCD b % 8 takes one contiguous eighth.
  const int64_t wg = (blockIdx.x % 8) * (kGtGrid / 8) + blockIdx.x / 8;
  const int64_t part = kSplit ? wg : wg * kGsWaves + wave, parts = kSplit ? kGtGrid : kGtGrid * kGsWaves;
  const int64_t gb = part * groups / parts, ge = (part + 1) * groups / parts;
  if (gb >= ge) return;  // with the split, the whole workgroup
  // this wave's chunks: one at least (the split takes K of four and more)
  const int c0 = kSplit ? wave * nch / kGsWaves : 0, c1 = kSplit ? (wave + 1) * nch / kGsWaves : nch;

  struct Place {
    int i, e, cnt, mt, j;  // listed expert i = expert e of cnt rows, m-tile mt, weight block j
  };
  const auto expert = [&](Place& at) __attribute__((always_inline)) {
    if (p.counts == nullptr) {
      at.e = 0;
      at.cnt = (int)p.M;
    } else {
      at.e = __builtin_amdgcn_readfirstlane((int)list[at.i]);
      at.cnt = g_scalar(p.counts + at.e);
    }
  };
  Place cur;
  {
    const int64_t m = gb / nt;
    cur.j = (int)(gb % nt);
    cur.i = 0;
    if (p.counts != nullptr) {  // by two steps of 64 comparisons
      const int step = (listed + kWave - 1) / kWave, at = lane * step;
      const int chunk = __popcll(__ballot(at < listed && pref[at < listed ? at : 0] <= m)) - 1, at2 = chunk * step + lane;
      cur.i = __builtin_amdgcn_readfirstlane(
          chunk * step - 1 + __popcll(__ballot(lane < step && at2 < listed && pref[at2 < listed ? at2 : 0] <= m)));
    }
    cur.mt = (int)(m - (p.counts ? __builtin_amdgcn_readfirstlane(pref[cur.i]) : 0));
    expert(cur);
  }
  const auto next = [&](Place& at) __attribute__((always_inline)) {  // true: another m-tile
    if (++at.j < nt) return false;
    at.j = 0;
    if ((int64_t)(at.mt + 1) * mrows < at.cnt) {
      ++at.mt;
    } else {
      at.mt = 0;
      ++at.i;
      expert(at);
    }
    return true;
  };
  const auto first_row = [&](const Place& at) __attribute__((always_inline)) {
    return (p.padded_offsets ? g_scalar(p.padded_offsets + at.e) : 0) + (int64_t)at.mt * mrows;
  };

  // ---- the stream ----------------------------------------------------------------------------------
  Place ld = cur;
  int ld_c = c0, ld_slot = 0, ld_quads = 0;
  int64_t ld_left = (ge - gb) * (c1 - c0);  // slots still to be requested
  uint64_t w_at = 0, a_at[4] = {0, 0, 0, 0}, s_at = 0;
  // Loads of 4 rows a 1 KB: lane l brings a piece of row 4 q + l / 16, whose place is l % 16.
  const auto row_of = [&](int R) __attribute__((always_inline)) -> int64_t {  // weight row of row R of the group
    if constexpr (kL1) return ((int64_t)ld.e * 2 + ((R >> 1) & 1)) * p.N + ld.j * 8 + (R >> 2) * 2 + (R & 1);
    const int n = ld.j * 16 + R;
    return (int64_t)ld.e * p.N + (n < p.N ? n : p.N - 1);  // (not stored)
  };
  const auto group_src = [&]() __attribute__((always_inline)) {
    w_at = reinterpret_cast<uint64_t>(p.w) + (uint64_t)(row_of(g) * RB);
    if constexpr (kI8) {
      if (lane < 16) s_at = reinterpret_cast<uint64_t>(p.w_scales + row_of(lane));
    }
  };
  const auto tile_src = [&]() __attribute__((always_inline)) {
    const int64_t row0 = first_row(ld);
    const int left = ld.cnt - ld.mt * mrows < mrows ? ld.cnt - ld.mt * mrows : mrows;
    int tok[kGsRows];
#pragma unroll
    for (int R = 0; R < kGsRows; ++R) {
      const int64_t row = row0 + (R < left ? R : left - 1);
      tok[R] = p.row_token ? g_scalar(p.row_token + row) : (int)row;
    }
    ld_quads = (left + 3) / 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = g == 0 ? tok[4 * q] : g == 1 ? tok[4 * q + 1] : g == 2 ? tok[4 * q + 2] : tok[4 * q + 3];
      a_at[q] = reinterpret_cast<uint64_t>(p.a) + (uint64_t)(uint32_t)t * (uint64_t)RB;
    }
    if constexpr (kI8) {
      int t = tok[0];
#pragma unroll
      for (int R = 1; R < kGsRows; ++R) t = r == R ? tok[R] : t;
      if (lane >= 16) s_at = reinterpret_cast<uint64_t>(p.a_scales + (uint32_t)t);
    }
  };
  const int64_t quad = (kL1 ? 2 : 4) * RB;  // from row R to row R + 4 of the group
  const int last_rows = kL1 ? 16 : p.N - (nt - 1) * 16;  // (a multiple of 8) rows of the last block
  const auto request = [&]() __attribute__((always_inline)) {
    const uint32_t base = ring_at + ld_slot * slot_bytes;
    const int pieces = ld_c + 1 == nch ? rest : 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // a piece beyond K: the chunk's first instead; the compute skips it
      const int piece = (lane & 15) ^ (4 * q + g), off = kGsChunk * ld_c + 16 * (piece < pieces ? piece : 0);
      const int64_t rows = !kL1 && ld.j + 1 == nt && 4 * q >= last_rows ? 0 : q * quad;  // a block's missing rows: its first
      dma16nt(reinterpret_cast<const uint8_t*>(w_at) + rows + off, base + 1024 * q);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q >= ld_quads) break;
      const int piece = (lane & 15) ^ (4 * q + g), off = kGsChunk * ld_c + 16 * (piece < pieces ? piece : 0);
      dma16(reinterpret_cast<const uint8_t*>(a_at[q]) + off, base + kGsWeights + 1024 * q);
    }
    if (kI8 && ld_c + 1 == c1) dma4(reinterpret_cast<const uint8_t*>(s_at), base + slot_bytes - kGsScales);
    ld_slot = ld_slot + 1 == slots ? 0 : ld_slot + 1;
    --ld_left;
    if (++ld_c == c1) {
      ld_c = c0;
      if (ld_left > 0) {
        if (next(ld)) tile_src();
        group_src();
      }
    }
  };
  tile_src();
  group_src();
  for (int i = 0; i < slots && ld_left > 0; ++i) request();

  int slot = 0;
  int64_t row0 = first_row(cur);
  for (int64_t gi = gb; gi < ge; ++gi) {
    typename T::acc acc;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = 0;
    const int left = cur.cnt - cur.mt * mrows < mrows ? cur.cnt - cur.mt * mrows : mrows;
    const int rl = r < left ? r : left - 1;
    f32x4 sw{0.f, 0.f, 0.f, 0.f};
    float sa = 0.0f;
    for (int c = c0; c < c1; ++c) {
      const int64_t ahead = (ge - gi) * (c1 - c0) - (c - c0) - 1 - ld_left;  // slots requested after this one
      gs_wait_slots<kGsMaxSlots - 1>((int)ahead);
      asm volatile("" ::: "memory");
      const uint32_t at = ring_at + slot * slot_bytes;
      u32x4 wv[4], av[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        wv[st] = lds_read16(at + r * kGsChunk + 16 * ((4 * g + st) ^ r));
        av[st] = lds_read16(at + kGsWeights + rl * kGsChunk + 16 * ((4 * g + st) ^ rl));
      }
      if (kI8 && c + 1 == c1) {
        sw = lds_read<f32x4>(at + slot_bytes - kGsScales + 16 * g);
        sa = lds_read<float>(at + slot_bytes - kGsScales + 64 + 4 * r);
      }
      g_wait_lds();  // the slot's operands are in registers
      slot = slot + 1 == slots ? 0 : slot + 1;
      if (ld_left > 0) request();
      if (c + 1 == nch && rest < 16) {
#pragma unroll
        for (int st = 0; st < 4; ++st)
          if (4 * g + st >= rest) wv[st] = av[st] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int st = 0; st < 4; ++st) acc = T::product(wv[st], av[st], acc);
    }
    typename T::acc z = acc;
    if constexpr (kSplit) {
      typedef typename T::acc A;
      const uint32_t red = red_at + (gi & 1) * kGsWaves * kWave * 16 + lane * 16;
      lds_write16(red + wave * kWave * 16, __builtin_bit_cast(u32x4, acc));
      g_wait_lds();  // the partial sums are written; the stream stays in flight
      g_barrier();
      if (wave == (int)(gi % kGsWaves)) {
        z = __builtin_bit_cast(A, lds_read16(red));
#pragma unroll
        for (int k = 1; k < kGsWaves; ++k) z += __builtin_bit_cast(A, lds_read16(red + k * kWave * 16));
      }
    }
    if (!kSplit || wave == (int)(gi % kGsWaves)) {
      // lane: token row r of the m-tile, weight rows 4g .. 4g+3
      f32x4 f;
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = kI8 ? (float)z[q] * sw[q] * sa : (float)z[q];
      const bool f16 = p.out_dtype == MEGAMOE_DTYPE_F16;
      if (r < left) {
        uint16_t* const out = static_cast<uint16_t*>(p.out) + (row0 + r) * (int64_t)p.N;
        if constexpr (kL1) {
          *reinterpret_cast<uint32_t*>(out + cur.j * 8 + 2 * g) = g_pack2(g_silu(f[0]) * f[2], g_silu(f[1]) * f[3], f16);
        } else if (cur.j * 16 + 4 * g < p.N) {
          *reinterpret_cast<u32x2*>(out + cur.j * 16 + 4 * g) = u32x2{g_pack2(f[0], f[1], f16), g_pack2(f[2], f[3], f16)};
        }
      }
    }
    if (gi + 1 < ge && next(cur)) row0 = first_row(cur);
  }
}

// The dynamic LDS limit of a kernel, raised once a device.
template <typename F>
static hipError_t gt_allow_lds(F* kernel, std::atomic<bool> (&done)[kGtDevices]) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev < kGtDevices && done[dev].load(std::memory_order_acquire)) return hipSuccess;
  err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kGtLds);
  if (err == hipSuccess && dev < kGtDevices) done[dev].store(true, std::memory_order_release);
  return err;
}

template <int kOp, int kDtype>
static hipError_t launch_gt(const GroupedArgs& a, hipStream_t stream) {
  static std::atomic<bool> done[kGtDevices];
  const hipError_t err = gt_allow_lds(gt_kernel<kOp, kDtype>, done);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((gt_kernel<kOp, kDtype>), dim3(kGtGrid), dim3(kGtThreads), kGtLds, stream, a);
  return hipGetLastError();
}

template <int kDtype, bool kGather>
static hipError_t launch_gt_weights(const GroupedWgradArgs& a, hipStream_t stream) {
  static std::atomic<bool> done[kGtDevices];
  const hipError_t err = gt_allow_lds(gt_weights_kernel<kDtype, kGather>, done);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((gt_weights_kernel<kDtype, kGather>), dim3(kGtGrid), dim3(kGtThreads), kGtLds, stream, a);
  return hipGetLastError();
}

// How the stream kernel runs: K split or not, token rows of an m-tile, ring slots.
struct GsPlan {
  bool split;
  int mrows, slots;
  size_t lds;
};
static GsPlan gs_plan(const GroupedArgs& a, int64_t rows) {
  GsPlan g;
  const int64_t chunks = ((int64_t)a.K * (a.dtype == kOperandI8 ? 1 : 2) + kGsChunk - 1) / kGsChunk;
  // Split and unsplit, us, int8.  Experts of one row, by chunks of K: 48 with 7168 outputs, 4 chunks 99 and 58, 8 137 and
  // 105, 14 208 and 186, 16 219 and 217; 8 of them, 14 chunks 39 and 36, 16 40 and 49; so from 16 on.  Dense calls of 8
  // rows, which have few groups for the waves, by groups: 300, 8 chunks 6.8 and 7.8, 16 9.0 and 11.6; 448, 4 chunks 6.5
  // and 6.5, 6 6.7 and 6.8, 8 6.9 and 7.8; 512, 8 chunks 6.8 and 7.7; 600, 8 chunks 8.6 and 7.9, 14 11.4 and 10.9; 1024,
  // 8 chunks 10.3 and 8.4, 16 14.5 and 14.1: from 8 chunks on, where no workgroup takes more than two groups.
  const int64_t groups = (a.N + 15) / 16;
  g.split = chunks >= kGsSplitChunks || (chunks >= kGsSplitChunks / 2 && a.counts == nullptr && groups <= 2 * kGtGrid);
  g.mrows = rows > 0 && rows <= 4 ? 4 : rows > 0 && rows <= 8 ? 8 : kGsRows;
  const int slot = gs_slot_bytes(a.dtype == kOperandI8, g.mrows), fixed = kGsLists + (g.split ? kGsRed : 0);
  g.slots = (kGtLds - fixed) / (kGsWaves * slot);
  if (g.slots > kGsMaxSlots) g.slots = kGsMaxSlots;
  g.lds = (size_t)(fixed + kGsWaves * g.slots * slot);
  return g;
}

template <bool kL1, int kDtype, bool kSplit>
static hipError_t launch_gs_as(const GroupedArgs& a, const GsPlan& plan, hipStream_t stream) {
  static std::atomic<bool> done[kGtDevices];
  const hipError_t err = gt_allow_lds(gs_kernel<kL1, kDtype, kSplit>, done);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((gs_kernel<kL1, kDtype, kSplit>), dim3(kGtGrid), dim3(kGsWaves * kWave), plan.lds, stream, a, plan.slots,
                     plan.mrows);
  return hipGetLastError();
}
template <bool kL1, int kDtype>
static hipError_t launch_gs(const GroupedArgs& a, const GsPlan& plan, hipStream_t stream) {
  return plan.split ? launch_gs_as<kL1, kDtype, true>(a, plan, stream) : launch_gs_as<kL1, kDtype, false>(a, plan, stream);
}

hipError_t launch_grouped(const GroupedArgs& a, bool l1, int64_t max_rows, hipStream_t stream) {
  if (a.across)
    return a.dtype == MEGAMOE_DTYPE_BF16 ? launch_gt<kGtAcross, MEGAMOE_DTYPE_BF16>(a, stream)
                                         : launch_gt<kGtAcross, MEGAMOE_DTYPE_F16>(a, stream);
  // The stream kernel takes calls of at most 16 rows an expert, by the caller's bound (it covers every expert, should
  // the bound be wrong), and dense calls of as many.  Without such a bound the tile kernel takes all experts: beside
  // 384 experts of 8 rows (int8, 2048 -> 7168) the stream kernel's 1010 us are its 880, 8 experts of 3 rows (bf16, 7168 ->
  // 4096) take 74 us and 80, and 16 small experts 10.5 us in two launches and 8.7 in one.
  const bool dense = a.counts == nullptr;
  const int64_t rows = dense ? a.M : max_rows;
  if (!(rows > 0 && rows <= kGsRows)) {
    if (a.dtype == kOperandI8)
      return l1 ? launch_gt<kGtGateUp, kOperandI8>(a, stream) : launch_gt<kGtPlain, kOperandI8>(a, stream);
    return a.dtype == MEGAMOE_DTYPE_BF16 ? launch_gt<kGtPlain, MEGAMOE_DTYPE_BF16>(a, stream)
                                         : launch_gt<kGtPlain, MEGAMOE_DTYPE_F16>(a, stream);
  }
  const GsPlan plan = gs_plan(a, rows);
  if (a.dtype == kOperandI8)
    return l1 ? launch_gs<true, kOperandI8>(a, plan, stream) : launch_gs<false, kOperandI8>(a, plan, stream);
  return a.dtype == MEGAMOE_DTYPE_BF16 ? launch_gs<false, MEGAMOE_DTYPE_BF16>(a, plan, stream)
                                       : launch_gs<false, MEGAMOE_DTYPE_F16>(a, plan, stream);
}

hipError_t launch_grouped_wgrad(const GroupedWgradArgs& a, hipStream_t stream) {
  if (a.row_token != nullptr)
    return a.dtype == MEGAMOE_DTYPE_BF16 ? launch_gt_weights<MEGAMOE_DTYPE_BF16, true>(a, stream)
                                         : launch_gt_weights<MEGAMOE_DTYPE_F16, true>(a, stream);
  return a.dtype == MEGAMOE_DTYPE_BF16 ? launch_gt_weights<MEGAMOE_DTYPE_BF16, false>(a, stream)
                                       : launch_gt_weights<MEGAMOE_DTYPE_F16, false>(a, stream);
}

}  // namespace megamoe
