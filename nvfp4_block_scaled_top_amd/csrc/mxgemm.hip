// MXFP4 x MXFP4 products: dense, and grouped over experts (gate+up with SiLU(gate)*up, and down).
//
//   out[m, n] = sum over 32-element blocks b of 2^(ea[m,b] + ew[n,b]) * sum_{k in b} e2m1(a) * e2m1(w)
//
// gfx950 multiplies both operands' codes and scales in the matrix core: lane l of
// v_mfma_scale_f32_16x16x128_f8f6f4 holds the 32 codes (16 bytes) of block l / 16 of row l % 16 and
// that block's scale byte, so an MXFP4 block is one lane's operand and nothing is decoded.
// Products and sums are exact up to the fp32 accumulation.
//
// The weights are the MFMA's A operand and the token rows its B operand, so a lane ends with four
// consecutive output columns of one token.  Gate and up rows of an expert are interleaved two by two
// within a 16-row block: a lane then holds gate and up of the same two h columns.
#include <atomic>

#include "device_common.h"
#include "internal.h"
#include "lds_dma.h"

namespace megamoe {

constexpr int kMxDevices = 64;

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float mx_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// Workgroup barrier that no LDS access is moved across.  Vector memory loads stay in flight.
__device__ __forceinline__ void mx_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int V>
struct IntTag {
  static constexpr int value = V;
};

// Rows of expert e and their first row; without tables there is one group of all p.M rows.
__device__ __forceinline__ int mx_count(const MxGemmArgs& p, int e) { return p.counts ? p.counts[e] : (int)p.M; }

// ============================================================================================
// Experts (or a dense call) of at most kMxSmallRows rows: the weights' bytes are the work.
//
// Work unit: a group, 16 weight rows over the whole of K for one m-tile; the groups of all m-tiles
// are laid end to end and every workgroup takes an equal range (one workgroup of 4 waves a CU).
// The 4 waves split K; each streams its part of the weight rows through an LDS ring of its own, 16 rows
// x 512 elements (256 bytes a row, 16 scale bytes) a slot, by direct global -> LDS loads: no barrier, no
// registers, and some 70 KB in flight a CU.  A slot is requested again as soon as its operands are in
// registers.  The ring runs on across groups and m-tiles.
//
// The token rows' part of K stays in LDS while the groups of their m-tile pass.  Both operands keep
// 16-byte piece c of row R (one MXFP4 block) at slot c ^ R of the row's 256 bytes, so that the 16 rows of
// one g are read from 16 different slots.  (Lanes of two g's still meet in a slot: half of the LDS cycles are
// conflicts by the counter.  LDS is busy for 6 to 18% of the kernel's cycles.)  Lane (r, g) takes blocks 4g .. 4g+3
// of its row, one an MFMA step: its four scale bytes are one word, and the instruction picks the byte.
//
// At the end of a group the waves leave their partial sums in LDS (two buffers, by the group's parity) and
// one of them adds the four in wave order and stores.
//
// Where the token rows of the whole K fit LDS four times beside the rings (K up to 2560), K is not split:
// every wave takes groups of its own and keeps its own copy of the token rows, and nothing is shared
// or waited for.  With K = 2048 split in four a wave has one slot between two barriers: the down projection
// of a 512-token prompt (384 experts, 7168 x 2048) took 814 us, and 632 without the split (528, 5.8 TB/s, with
// the places found as below; these loads alone stream 7.2 TB/s); with
// K = 7168 the split spreads 16 rows' 61 KB over the four waves, which LDS would not hold four times.
// ============================================================================================
constexpr int kMxSmallRows = 16;
constexpr int kMxBn = 256, kMxBm = 256, kMxStageK = 256;  // the tile kernel's weight rows, token rows and stage
constexpr int kMxSplit = 4;                        // waves, K split
constexpr int kMxChunk = 512;                      // K elements of a slot
constexpr int kMxSlotCodes = 16 * kMxChunk / 2;
constexpr int kMxSlot = kMxSlotCodes + 16 * kMxChunk / 32;
constexpr int kMxMaxSlots = 8;
constexpr int kMxLds = 160 * 1024;
constexpr int kMxRed = 2 * kMxSplit * kWave * 16;
constexpr int kMxGrid = 256;                       // one workgroup a CU

// Waits until at most `after` (<= K) later slots' loads are outstanding for this wave.
template <int K>
__device__ __forceinline__ void mx_wait_slots(int after) {
  if constexpr (K > 0) {
    if (after < K) {
      mx_wait_slots<K - 1>(after);
      return;
    }
  }
  wait_vmcnt<5 * K>();
}

template <int S>
__device__ __forceinline__ f32x4 mx_mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

// Which kernel takes the experts of more than kMxSmallRows rows.  A tile costs the tile kernel the same time
// whether the chip is full of tiles or not; the small kernel reads the weights once for every 16 rows, but
// spreads any work over all CUs.  Measured, dense (us, tile kernel / small kernel): 64 rows x 4096 x 7168
// 42.7 / 15.0, 256 x 4096 x 7168 61.2 / 44.5, 400 x 4096 x 7168 67.0 / 69.5, 400 x 7168 x 2048 24.9 / 32.6.
// slots: what the small kernel would stream for them, 0.74 ns each; tiles: of the tile kernel, 256 at a
// time, 1.45, 1.6 or 2.1 us a stage (64, 128 or 256 token rows).  A grouped call is weighed as a whole, with every
// stage at its largest expert's time; the figures are of dense calls.
struct MxLoad {
  int64_t slots, tiles;
  int rows;  // the largest expert's
};
__host__ __device__ inline MxLoad mx_load_of(const MxGemmArgs& p, bool l1, int cnt) {
  if (cnt <= kMxSmallRows || p.mrows == 0) return {0, 0, 0};
  const int64_t groups = l1 ? p.N / 8 : p.N / 16, nch = (p.K + kMxChunk - 1) / kMxChunk;
  const int64_t cols = l1 ? kMxBn / 2 : kMxBn;
  return {(cnt + p.mrows - 1) / p.mrows * groups * nch, (cnt + kMxBm - 1) / kMxBm * ((p.N + cols - 1) / cols), cnt};
}
__host__ __device__ inline bool mx_small_takes_all(const MxGemmArgs& p, const MxLoad& l) {
  const int64_t stages = (p.K + kMxStageK - 1) / kMxStageK * ((l.tiles + kMxGrid - 1) / kMxGrid);
  return l.slots * 74 < stages * (l.rows <= 64 ? 145000 : l.rows <= 128 ? 160000 : 210000);
}
// The same for a grouped call, by one wave, from the counts.
__device__ __forceinline__ bool mx_small_takes_all(const MxGemmArgs& p, bool l1) {
  if (p.cover_large || p.cover_small) return p.cover_large;
  MxLoad sum{0, 0, 0};
  for (int e = lane_id(); e < p.E; e += kWave) {
    const MxLoad l = mx_load_of(p, l1, p.counts[e]);
    sum.slots += l.slots;
    sum.tiles += l.tiles;
    sum.rows = sum.rows > l.rows ? sum.rows : l.rows;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    sum.slots += __shfl_xor(sum.slots, o, kWave);
    sum.tiles += __shfl_xor(sum.tiles, o, kWave);
    const int r = __shfl_xor(sum.rows, o, kWave);
    sum.rows = sum.rows > r ? sum.rows : r;
  }
  return mx_small_takes_all(p, sum);
}

// A place in the list of groups: expert e of cnt rows, m-tile mt of it, 16-row weight block j.
struct MxPlace {
  int e, cnt, mt, j;
};

__device__ __forceinline__ int mx_small_tiles(const MxGemmArgs& p, int cnt, int mrows) {  // p.cover_large: as decided
  return cnt <= kMxSmallRows || p.cover_large ? (cnt + mrows - 1) / mrows : 0;
}

// The first m-tile of an expert from e0 on that has any; p.E if none.
__device__ __forceinline__ void mx_seek(const MxGemmArgs& p, int e0, int mrows, MxPlace& at) {
  at.e = p.E;
  at.mt = 0;
  for (int c = e0; c < p.E && at.e == p.E; c += kWave) {
    const int cnt = c + lane_id() < p.E ? mx_count(p, c + lane_id()) : 0;
    const uint64_t any = __ballot(mx_small_tiles(p, cnt, mrows) > 0);
    if (any) {
      const int l = __ffsll((unsigned long long)any) - 1;
      at.e = c + l;
      at.cnt = __builtin_amdgcn_readlane(cnt, l);
    }
  }
}

// The place of group g of the list, nt groups an m-tile: the experts' m-tiles are summed 64 at a time.
// (Walking the experts one by one, a load each, the last wave of 384 experts began 150 us late.)
__device__ __forceinline__ MxPlace mx_place(const MxGemmArgs& p, int64_t g, int nt, int mrows) {
  MxPlace at;
  int64_t m = g / nt;
  at.j = (int)(g % nt);
  at.e = 0;
  at.cnt = (int)p.M;
  if (p.counts != nullptr) {
    for (int c = 0; c < p.E; c += kWave) {
      const int cnt = c + lane_id() < p.E ? mx_count(p, c + lane_id()) : 0;
      const int own = mx_small_tiles(p, cnt, mrows);
      int incl = own;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(incl, o, kWave);
        if (lane_id() >= o) incl += t;
      }
      const uint64_t past = __ballot((int64_t)incl > m);
      if (past) {
        const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1);
        at.e = c + l;
        at.cnt = __builtin_amdgcn_readlane(cnt, l);
        m -= __builtin_amdgcn_readlane(incl - own, l);
        break;
      }
      m -= __builtin_amdgcn_readlane(incl, kWave - 1);
    }
  }
  at.mt = (int)m;
  return at;
}

template <bool kL1, bool kSplit>
__global__ __launch_bounds__(kMxSplit* kWave, 1) void mx_small_kernel(MxGemmArgs p, int slots) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_mx[];
  const int lane = lane_id(), r = lane & 15, g = lane >> 4, mrows = p.mrows;
  if (p.counts != nullptr) p.cover_large = mx_small_takes_all(p, kL1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int nch = (p.K + kMxChunk - 1) / kMxChunk, nblk = p.K / 32;
  const int64_t Kh = p.K / 2, Ks = p.K / 32;
  const int a_chunk = mrows * (kMxChunk / 2 + kMxChunk / 32);  // LDS bytes of a chunk of the token rows
  uint8_t* const s_a = s_mx + (kSplit ? 0 : wave * nch * a_chunk);
  f32x4* const s_red = reinterpret_cast<f32x4*>(s_mx + nch * a_chunk);
  uint8_t* const s_ring = s_mx + (kSplit ? nch * a_chunk + kMxRed : kMxSplit * nch * a_chunk) + wave * slots * kMxSlot;
  const int c0 = kSplit ? wave * nch / kMxSplit : 0, c1 = kSplit ? (wave + 1) * nch / kMxSplit : nch;  // this wave's chunks
  constexpr int unit = kL1 ? 8 : 16;  // output columns of a group
  const int nt = p.N / unit;

  // The groups [gb, ge) of this workgroup, or of this wave; XCD b % 8 takes one contiguous eighth.
  int64_t tiles = 0;
  if (p.counts == nullptr) {
    tiles = (p.M + mrows - 1) / mrows;
  } else {
    int mine = 0;
    for (int e = lane; e < p.E; e += kWave) mine += mx_small_tiles(p, p.counts[e], mrows);
    tiles = wave_sum_i32(mine);
  }
  const int64_t groups = tiles * nt;
  const int64_t wg = (blockIdx.x % 8) * (kMxGrid / 8) + blockIdx.x / 8;
  const int64_t part = kSplit ? wg : wg * kMxSplit + wave, parts = kSplit ? kMxGrid : kMxGrid * kMxSplit;
  const int64_t gb = part * groups / parts, ge = (part + 1) * groups / parts;
  if (gb >= ge) return;  // with the split, the whole workgroup

  MxPlace cur = mx_place(p, gb, nt, mrows);  // of the group that is computed
  const auto next = [&](MxPlace& at) {
    if (++at.j < nt) return;
    at.j = 0;
    if ((at.mt + 1) * mrows < at.cnt) {
      ++at.mt;
    } else {
      mx_seek(p, at.e + 1, mrows, at);
    }
  };

  // ---- the weight stream -------------------------------------------------------------------------
  MxPlace ld = cur;
  int ld_c = c0, ld_slot = 0;
  int64_t ld_left = (ge - gb) * (c1 - c0);  // slots still to be requested
  const uint8_t *w_src, *ws_src;
  // Loads of 4 rows a 1 KB: lane l brings a piece of row 4q + l / 16, whose LDS place is l % 16.
  const auto row_of = [&](int R) -> int64_t {  // weight row of row R of the group
    if constexpr (kL1) return ((int64_t)ld.e * 2 + ((R >> 1) & 1)) * p.N + ld.j * 8 + (R >> 2) * 2 + (R & 1);
    else return (int64_t)ld.e * p.N + ld.j * 16 + R;
  };
  const auto set_src = [&]() {
    w_src = p.w_codes + row_of(lane >> 4) * Kh;
    ws_src = p.w_scales + row_of(lane >> 2) * Ks;
  };
  const int64_t quad = (kL1 ? 2 : 4) * Kh;  // from row R to row R + 4 of the group
  const auto request = [&]() {
    const uint32_t base = lds_addr(s_ring + ld_slot * kMxSlot);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // a piece beyond K (in the last chunk): the chunk's first instead; the compute skips it
      const int piece = (lane & 15) ^ (4 * q + (lane >> 4));
      const int b = ld_c * 16 + (ld_c * 16 + piece < nblk ? piece : 0);
      dma16nt(w_src + q * quad + 16 * b, base + 1024 * q);
    }
    const int b4 = ld_c * 4 + (ld_c * 4 + (lane & 3) < nblk / 4 ? lane & 3 : 0);
    dma4(ws_src + 4 * b4, base + kMxSlotCodes);
    ld_slot = ld_slot + 1 == slots ? 0 : ld_slot + 1;
    --ld_left;
    if (++ld_c == c1) {
      ld_c = c0;
      if (ld_left > 0) {
        next(ld);
        set_src();
      }
    }
  };

  // This wave's chunks of the m-tile's rows into LDS (rows past the last are left as they are: a row
  // is one column of the product, and theirs are not stored).
  const auto load_rows = [&](const MxPlace& at, int64_t row0, int left) {
    const auto src_row = [&](int R) -> int64_t {
      const int64_t t = row0 + (R < left ? R : 0);
      return p.row_token ? p.row_token[t] : t;
    };
    const uint8_t* a[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = 4 * q < left ? p.a_codes + src_row(4 * q + (lane >> 4)) * Kh : p.a_codes;
    const uint8_t* as = p.a_scales + src_row(lane >> 2) * Ks;
    for (int c = c0; c < c1; ++c) {
      const uint32_t base = lds_addr(s_a + c * a_chunk);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * q >= left) continue;
        const int piece = (lane & 15) ^ (4 * q + (lane >> 4));
        dma16(a[q] + 16 * (c * 16 + (c * 16 + piece < nblk ? piece : 0)), base + 1024 * q);
      }
      const int b4 = c * 4 + (c * 4 + (lane & 3) < nblk / 4 ? lane & 3 : 0);
      if ((lane >> 2) < mrows) dma4(as + 4 * b4, base + mrows * (kMxChunk / 2));
    }
  };

  int64_t row0 = 0;
  int left = 0;
  const auto enter = [&]() {  // the rows of cur's m-tile
    row0 = (p.padded_offsets ? p.padded_offsets[cur.e] : 0) + (int64_t)cur.mt * mrows;
    left = min(cur.cnt - cur.mt * mrows, mrows);
    load_rows(cur, row0, left);
  };
  enter();
  set_src();
  for (int i = 0; i < slots && ld_left > 0; ++i) request();

  int slot = 0;
  const int rl = r & (mrows - 1);
  for (int64_t gi = gb; gi < ge; ++gi) {
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c < c1; ++c) {
      const int64_t ahead = (ge - gi) * (c1 - c0) - (c - c0) - 1 - ld_left;  // slots requested after this one
      mx_wait_slots<kMxMaxSlots - 1>((int)ahead);
      asm volatile("" ::: "memory");
      const uint8_t* w = s_ring + slot * kMxSlot;
      const uint8_t* a = s_a + c * a_chunk;
      u32x4 wv[4], av[4];
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        wv[st] = *reinterpret_cast<const u32x4*>(w + r * 256 + 16 * ((4 * g + st) ^ r));
        av[st] = *reinterpret_cast<const u32x4*>(a + rl * 256 + 16 * ((4 * g + st) ^ rl));
      }
      uint32_t wsc = *reinterpret_cast<const uint32_t*>(w + kMxSlotCodes + r * 16 + 4 * g);
      uint32_t asc = *reinterpret_cast<const uint32_t*>(a + mrows * (kMxChunk / 2) + rl * 16 + 4 * g);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot's operands are in registers
      asm volatile("" ::: "memory");
      slot = slot + 1 == slots ? 0 : slot + 1;
      if (ld_left > 0) request();
      if (c * 4 + 4 > nblk / 4 && c * 4 + g >= nblk / 4) {  // beyond K
        wsc = asc = 0x7F7F7F7Fu;
#pragma unroll
        for (int st = 0; st < 4; ++st) av[st] = u32x4{0u, 0u, 0u, 0u};
      }
      acc = mx_mfma16<0>(wv[0], av[0], acc, wsc, asc);
      acc = mx_mfma16<1>(wv[1], av[1], acc, wsc, asc);
      acc = mx_mfma16<2>(wv[2], av[2], acc, wsc, asc);
      acc = mx_mfma16<3>(wv[3], av[3], acc, wsc, asc);
    }
    f32x4 z = acc;
    if constexpr (kSplit) {
      f32x4* const red = s_red + (gi & 1) * kMxSplit * kWave;
      red[wave * kWave + lane] = acc;
      __builtin_amdgcn_s_waitcnt(0xC07F);  // the partial sums are written; weight loads stay in flight
      mx_barrier();
      if (wave == (int)(gi % kMxSplit)) {
        z = red[lane];
#pragma unroll
        for (int k = 1; k < kMxSplit; ++k) z += red[k * kWave + lane];
      }
    }
    if (!kSplit || wave == (int)(gi % kMxSplit)) {
      // lane: token row r of the m-tile, weight rows 4g .. 4g+3
      if (r < left) {
        uint16_t* out = static_cast<uint16_t*>(p.out) + (row0 + r) * (int64_t)p.N;
        if constexpr (kL1) {
          *reinterpret_cast<uint32_t*>(out + cur.j * 8 + 2 * g) =
              f32_to_bf16_any(mx_silu(z[0]) * z[2]) | f32_to_bf16_any(mx_silu(z[1]) * z[3]) << 16;
        } else {
          *reinterpret_cast<u32x2*>(out + cur.j * 16 + 4 * g) =
              u32x2{f32_to_bf16_any(z[0]) | f32_to_bf16_any(z[1]) << 16,
                    f32_to_bf16_any(z[2]) | f32_to_bf16_any(z[3]) << 16};
        }
      }
    }
    if (gi + 1 < ge) {
      const int e = cur.e, mt = cur.mt;
      next(cur);
      if (cur.e != e || cur.mt != mt) {
        enter();
        wait_vmcnt<0>();  // the new rows, and with them every weight slot requested so far
      }
    }
  }
}

// ============================================================================================
// Experts of more rows: 256 weight rows x BM token rows a tile, BM = 256, or 128 or 64 for an
// expert's last rows when they fit; one persistent workgroup of 8 waves a CU.
//
// Stages of 256 K elements go from global memory straight into one of two LDS slots (no registers): at
// the top of a stage a wave waits for its own loads, one barrier makes everyone's visible and says that
// the other slot is free, the next stage is requested into it, and the stage is computed meanwhile.
// The stages run on across tiles: a tile's last stage requests the next tile's first, whose rows and
// expert were found while this tile was computed.
//
// A stage holds 128 code bytes a row of either operand (a load instruction covers 8 rows; with 128
// contiguous bytes a row it takes 19 cycles, with 64 bytes 28), block c of row R at slot
// c ^ mx_swz(R), so that 16 rows' reads of one block meet the 16 slots of two rows once each (26% of the
// LDS cycles are still conflicts by the counter; which accesses they come from is not known).  Scales come in
// stages of 512 elements, 16 bytes a row: 64 rows cost a load instruction 97 cycles whatever it
// brings of each.
//
// The 32x32x64 form is used: it sustains 9.2 PFLOP/s from registers (6.6 on random data, where the
// chip lowers its clock), the 16x16x128 form 6.9 (5.5).  Lane (r, h) of a 32-row fragment takes blocks
// 4h .. 4h+3 of the stage, one a step: its four scale bytes are one word, and the instruction picks
// the byte.  Both operands use the same order, so every block is met once.
//
// A wave computes 64 token rows x 32 * WB weight rows (WB = 4, 2, 1 for BM = 256, 128, 64).  Gate+up:
// the first half of a wave's weight rows are gate rows, the second half the up rows of the same h
// columns, so both meet in one lane.
// ============================================================================================
constexpr int kMxWaves = 8, kMxThreads = kMxWaves * kWave;
constexpr int kMxBand = 8;                       // m-tiles walked together, for L2 reuse of the weights
constexpr int kMxRowBytes = kMxStageK / 2;
constexpr int kMxACodes = kMxBn * kMxRowBytes;   // within a slot: the weights' codes, then the tokens'
constexpr int kMxStage = kMxACodes + kMxBm * kMxRowBytes;
constexpr int kMxAScales = kMxBn * 16;           // within a scale buffer
constexpr int kMxScaleBuf = kMxAScales + kMxBm * 16;
constexpr int kMxScales = 2 * kMxStage;          // LDS: two slots, two scale buffers, the tables
constexpr int kMxTables = kMxScales + 2 * kMxScaleBuf;
static_assert(kMxTables + 4 * (MEGAMOE_MAX_EXPERTS + 1) + 4 * kMxBm <= kMxLds, "the LDS layout fits");

__device__ __forceinline__ constexpr int mx_swz(int R) { return (R >> 1) & 7; }

// One output tile: BM = 64 * wb token rows from row0 on (left of them real), n-tile nt.
struct MxTile {
  int e, nt, wb, left;
  bool once;  // the expert's only m-tile: its weights are read once
  int64_t row0;
};

// What a load brings for a block beyond K: zero codes, and scales of 1.
__device__ const uint32_t g_mx_pad[8] = {0u, 0u, 0u, 0u, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};

template <int S>
__device__ __forceinline__ f32x16 mx_mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <bool kL1>
__global__ __launch_bounds__(kMxThreads, 1) void mx_tile_kernel(MxGemmArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_mx[];
  int* const s_row = reinterpret_cast<int*>(s_mx + kMxTables);  // tokens of the next tile's rows
  int* const pref = s_row + kMxBm;                              // m-tiles before each expert [E + 1]
  const int E = p.E, K = p.K, nks = (K + kMxStageK - 1) / kMxStageK, nblk = K / 32;
  const int64_t Kh = K / 2, Ks = K / 32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  // whole scale pieces of 16 bytes, aligned
  const bool wide_scales =
      K % 512 == 0 && ((reinterpret_cast<uintptr_t>(p.w_scales) | reinterpret_cast<uintptr_t>(p.a_scales)) & 15) == 0;
  if (wave == 0) {  // exclusive prefix of the experts' m-tiles
    const bool none = p.counts != nullptr && mx_small_takes_all(p, kL1);
    int carry = 0;
    for (int c = 0; c < E; c += kWave) {
      const int cnt = c + lane < E ? mx_count(p, c + lane) : 0;
      int incl = !none && (cnt > kMxSmallRows || p.cover_small) ? (cnt + kMxBm - 1) / kMxBm : 0;
      const int own = incl;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += t;
      }
      if (c + lane < E) pref[c + lane] = carry + incl - own;
      carry += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) pref[E] = carry;
  }
  __syncthreads();
  constexpr int cols = kL1 ? kMxBn / 2 : kMxBn;  // output columns of a tile
  const int ntn = (p.N + cols - 1) / cols;
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(pref[E]) * ntn;

  // Tile t of the list: its expert by two steps of 64 comparisons (at most 1024 experts).
  const auto find = [&](int64_t t) __attribute__((always_inline)) {
    const int step = (E + kWave - 1) / kWave;
    const int at = lane * step;
    const int chunk = __popcll(__ballot(at < E && (int64_t)pref[at < E ? at : 0] * ntn <= t)) - 1;
    const int at2 = chunk * step + lane;
    const int e = __builtin_amdgcn_readfirstlane(
        chunk * step - 1 + __popcll(__ballot(lane < step && at2 < E && (int64_t)pref[at2 < E ? at2 : 0] * ntn <= t)));
    const int first = __builtin_amdgcn_readfirstlane(pref[e]);
    const int mts = __builtin_amdgcn_readfirstlane(pref[e + 1]) - first;
    const int64_t local = t - (int64_t)first * ntn;
    const int band = (int)(local / ((int64_t)kMxBand * ntn)), in = (int)(local % ((int64_t)kMxBand * ntn));
    const int width = min(kMxBand, mts - band * kMxBand);
    const int mt = band * kMxBand + in % width;
    MxTile x;  // wave-uniform, in scalar registers
    x.e = e;
    x.nt = in / width;
    x.left = __builtin_amdgcn_readfirstlane(mx_count(p, e)) - mt * kMxBm;
    x.wb = x.left > 128 ? 4 : x.left > 64 ? 2 : 1;
    x.once = mts == 1;
    x.row0 = (int64_t)(p.padded_offsets ? __builtin_amdgcn_readfirstlane(p.padded_offsets[e]) : 0) + (int64_t)mt * kMxBm;
    return x;
  };
  // Rows past the tile's end read its last row, columns past the last one the last columns' weights:
  // what they feed is not stored.  The tokens of a gathered tile's rows are brought to s_row by loads
  // that a later barrier makes visible.
  const auto fetch_rows = [&](const MxTile& x) __attribute__((always_inline)) {
    if (kL1 && p.row_token != nullptr && wave < 4) {
      const int R = 64 * wave + lane;
      dma4(reinterpret_cast<const uint8_t*>(p.row_token + x.row0 + (R < x.left ? R : x.left - 1)),
           lds_addr(reinterpret_cast<uint8_t*>(s_row + 64 * wave)));
    }
  };
  // Every wave brings an eighth of a stage's weight and token rows.  Under a 256-row tile waves 4-7, which
  // share the SIMDs with waves 0-3, do so after the first quarter of their products, waves 0-3 before
  // theirs: 306 us for 16381 x 4096 x 7168 on random codes, 317 with all of them before, 314 to 316 with
  // waves 4-7 later.  Under lower tiles, which wait for memory, all bring theirs first: 96 experts of 48
  // rows (2048 -> 7168) 183 us, 195 the other way.  What a load adds to its tensor's address is kept in
  // units of 16 bytes for the codes and of 4 for the scales (operands of an expert are below 64 GB), the
  // four weight loads' in the lanes of one register: with all of it computed anew, 40 instructions a load,
  // a stage's loads took 3800 cycles to issue.
  uint32_t w_off = 0, a_off[4] = {0, 0, 0, 0}, s_off = 0;
  const auto set_loads = [&](const MxTile& x) __attribute__((always_inline)) {
    int ln = lane;
    asm volatile("" : "+v"(ln));  // nothing of this is kept in registers across the tile
    const auto a_row = [&](int R) -> uint32_t {
      if (kL1 && p.row_token != nullptr) return (uint32_t)s_row[R];
      return (uint32_t)((int)x.row0 + (R < x.left ? R : x.left - 1));
    };
    const auto w_row = [&](int R) -> uint32_t {  // within the expert; N is a multiple of 8
      if constexpr (kL1) {
        const int half = 16 * x.wb, in = R & (2 * half - 1);
        const int c = x.nt * cols + (R - in) / 2 + (in & (half - 1));
        return (uint32_t)((c < p.N ? c : p.N - 8 + (c & 7)) + (in >= half ? p.N : 0));
      } else {
        const int c = x.nt * cols + R;
        return (uint32_t)(c < p.N ? c : p.N - 8 + (c & 7));
      }
    };
    w_off = w_row(32 * wave + 8 * (ln & 3)) * (uint32_t)(Kh / 16);
    s_off = (wave < 4 ? w_row(64 * wave + ln) : a_row(64 * (wave - 4) + ln)) * (uint32_t)(Ks / 4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a_off[j] = a_row((8 * (x.wb * wave + j) + ln / 8) & (kMxBm - 1)) * (uint32_t)(Kh / 16);
  };
  // Stage ks of tile x into slot `slot`, its scales (even ks) into buffer `buf`.
  const auto issue = [&](const MxTile& x, int ks, int slot, int buf) __attribute__((always_inline)) {
    int ln = lane;
    asm volatile("" : "+v"(ln));  // what follows from the lane is computed here, not held through the tile
    const uint32_t base = lds_addr(s_mx + (slot & 1) * kMxStage);
    const int64_t wn0 = (int64_t)x.e * (kL1 ? 2 : 1) * p.N;
    const uint8_t* const wb = p.w_codes + wn0 * Kh + kMxRowBytes * ks;
    const uint8_t* const pad = reinterpret_cast<const uint8_t*>(g_mx_pad);
    // Lane l of a load brings a block of row l / 8 to place l % 8.
    const int blk0 = (ln & 7) ^ mx_swz(ln / 8);  // of an even 8-row piece (^ 4: odd)
    const uint32_t w_lane = (uint32_t)(ln / 8) * (uint32_t)Kh;
    const uint32_t wl0 = w_lane + 16 * blk0, wl1 = w_lane + 16 * (blk0 ^ 4);
    const uint8_t* const ab = p.a_codes + kMxRowBytes * ks;
    const uint32_t to_w = base + 32 * wave * kMxRowBytes, to_a = base + kMxACodes + 8 * x.wb * wave * kMxRowBytes;
    if ((ks + 1) * 8 <= nblk) {
      // Weights read once bypass the caches: 96 experts of 100 rows (2048 -> 7168) take 202 us instead of
      // 217; weights that the m-tiles of an expert share do not (16381 x 4096 x 7168: 321 us instead of 308).
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* src = wb + ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)w_off, j) << 4);
        if (x.once) dma16snt(src, j & 1 ? wl1 : wl0, to_w + 8 * j * kMxRowBytes);
        else dma16s(src, j & 1 ? wl1 : wl0, to_w + 8 * j * kMxRowBytes);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= x.wb) break;
        const int blk = (x.wb * wave + j) & 1 ? blk0 ^ 4 : blk0;
        dma16(ab + 16 * blk + (uint64_t)a_off[j] * 16, to_a + 8 * j * kMxRowBytes);
      }
    } else {  // the last stage, of four blocks
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int blk = j & 1 ? blk0 ^ 4 : blk0;
        const uint8_t* src = wb + ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)w_off, j) << 4);
        dma16(blk < 4 ? src + (j & 1 ? wl1 : wl0) : pad, to_w + 8 * j * kMxRowBytes);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= x.wb) break;
        const int blk = (x.wb * wave + j) & 1 ? blk0 ^ 4 : blk0;
        dma16(blk < 4 ? ab + 16 * blk + (uint64_t)a_off[j] * 16 : pad, to_a + 8 * j * kMxRowBytes);
      }
    }
    if ((ks & 1) || wave >= 4 + x.wb) return;
    // the scales of 64 weight rows (waves 0-3) or token rows (waves 4-7)
    const uint32_t to = lds_addr(s_mx + kMxScales + (buf & 1) * kMxScaleBuf) + 16 * 64 * wave;
    const uint8_t* const sc = (wave < 4 ? p.w_scales + wn0 * Ks : p.a_scales) + 8 * ks;
    if (wide_scales) {
      dma16(sc + (uint64_t)s_off * 4, to);
    } else {
      // else words, 16 rows a load
      const int word = ln & 3;
      const bool in = 4 * (ks * 2 + word) < nblk;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t o = (uint64_t)(uint32_t)__shfl((int)s_off, 16 * j + ln / 4, kWave) * 4 + 4 * word;
        dma4(in ? sc + o : pad + 16, to + 256 * j);
      }
    }
  };

  // XCD b % 8 takes 32 tiles in a row of every 256: they share rows and weights in its L2.
  int64_t t = (blockIdx.x % 8) * (kMxGrid / 8) + blockIdx.x / 8;
  if (t >= total) return;  // the whole workgroup
  MxTile cur = find(t), nxt = cur;
  fetch_rows(cur);
  wait_vmcnt<0>();
  mx_barrier();
  set_loads(cur);
  issue(cur, 0, 0, 0);
  int stage = 0, sstage = 0;  // parities: of the slot and of the scale buffer in use
  bool first = true;

  const auto run_tile = [&](auto wb_tag) __attribute__((always_inline)) {
    constexpr int WB = decltype(wb_tag)::value;
    constexpr int WM = WB, WN = kMxWaves / WM;
    const int wm = wave / WN, wn = wave % WN;
    const bool more = t + kMxGrid < total;
    f32x16 acc[2][WB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int f = 0; f < WB; ++f)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][f][q] = 0.f;
    for (int ks = 0; ks < nks; ++ks) {
      // A tile's first stage was waited for before the last tile's stores were issued.
      if (ks > 0 || first) __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
      else __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt(0)
      mx_barrier();
      if (ks == 0 && more) {
        nxt = find(t + kMxGrid);
        fetch_rows(nxt);
        if (nks == 1) {  // no later stage waits for these rows
          wait_vmcnt<0>();
          mx_barrier();
        }
      }
      const bool last = ks + 1 == nks;
      if (last && more) set_loads(nxt);
      const bool any = !last || more;
      const int to_ks = last ? 0 : ks + 1, buf = sstage + ((ks & 1) || last ? 1 : 0);
      if (any && (WB < 4 || wave < 4)) issue(last ? nxt : cur, to_ks, stage + 1, buf);
      int ln = lane;
      asm volatile("" : "+v"(ln));  // a few instructions a stage instead of registers
      const int r = ln & 31, h = ln >> 5, swz = mx_swz(r);  // (of rows 32 i + r too)
      const uint8_t* st = s_mx + (stage & 1) * kMxStage;
      const uint8_t* ss = s_mx + kMxScales + (sstage & 1) * kMxScaleBuf + 8 * (ks & 1) + 4 * h;
      const uint8_t* wp = st + (wn * WB * 32 + r) * kMxRowBytes;
      const uint8_t* ap = st + kMxACodes + (wm * 64 + r) * kMxRowBytes;
      uint32_t wsc[WB], asc[2];
#pragma unroll
      for (int f = 0; f < WB; ++f) wsc[f] = *reinterpret_cast<const uint32_t*>(ss + ((wn * WB + f) * 32 + r) * 16);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        asc[i] = *reinterpret_cast<const uint32_t*>(ss + kMxAScales + (wm * 64 + 32 * i + r) * 16);
      const auto read_w = [&](int f, int s) {
        return *reinterpret_cast<const u32x4*>(wp + f * 32 * kMxRowBytes + 16 * ((4 * h + s) ^ swz));
      };
      const auto read_a = [&](int i, int s) {
        return *reinterpret_cast<const u32x4*>(ap + i * 32 * kMxRowBytes + 16 * ((4 * h + s) ^ swz));
      };
      u32x4 w[2][WB], a[2][2];
#pragma unroll
      for (int f = 0; f < WB; ++f) w[0][f] = read_w(f, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) a[0][i] = read_a(i, 0);
      const auto step = [&](auto s_tag) {
        constexpr int S = decltype(s_tag)::value;
        if constexpr (S < 3) {
#pragma unroll
          for (int f = 0; f < WB; ++f) w[(S + 1) & 1][f] = read_w(f, S + 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) a[(S + 1) & 1][i] = read_a(i, S + 1);
        }
        __builtin_amdgcn_sched_barrier(0);  // the next step's reads before this step's products
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int f = 0; f < WB; ++f) acc[i][f] = mx_mfma32<S>(w[S & 1][f], a[S & 1][i], acc[i][f], wsc[f], asc[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int f = 0; f < WB; ++f) asm volatile("" : "+v"(acc[i][f]));  // (products do not move past loads)
      };
      step(IntTag<0>{});
      if (WB == 4 && any && wave >= 4) issue(last ? nxt : cur, to_ks, stage + 1, buf);
      step(IntTag<1>{});
      step(IntTag<2>{});
      step(IntTag<3>{});
      ++stage;
      if ((ks & 1) || ks + 1 == nks) ++sstage;
    }
    if (more) wait_vmcnt<0>();  // the next tile's first stage, ahead of the stores

    // Accumulator q of block (i, f): weight row 32 f + 8 (q / 4) + 4 h + q % 4 of the wave, token row 32 i + r.
    // The wave's 32 token rows of a block go through its eighth of the slot that the tile's last stage was
    // read from (the barrier: by everyone), so that the rows are stored in 16-byte pieces that follow each
    // other: with the accumulators' own 8-byte pieces a 256 x 256 tile took 20 us to store.
    mx_barrier();
    int ln = lane;
    asm volatile("" : "+v"(ln));  // addresses are computed here, not held through the stages
    constexpr int kRow = (kL1 ? 32 : 64) * WB, kPieces = kRow / 16;  // bytes of a wave's output row
    uint8_t* const o_lds = s_mx + ((stage + 1) & 1) * kMxStage + wave * (kMxStage / kMxWaves);
    const auto put = [&](int piece, u32x2 v) {  // 4 columns: half h of a 16-byte piece of row r
      *reinterpret_cast<u32x2*>(o_lds + (ln & 31) * kRow + 16 * (piece ^ (ln & (kPieces - 1))) + 8 * (ln >> 5)) = v;
    };
    const int c0 = cur.nt * cols + wn * kRow / 2;
    const auto store_rows = [&](auto i_tag) __attribute__((always_inline)) {
      constexpr int i = decltype(i_tag)::value;
#pragma unroll
      for (int f = 0; f < (kL1 ? (WB + 1) / 2 : WB); ++f)
#pragma unroll
        for (int q4 = 0; q4 < (kL1 && WB == 1 ? 2 : 4); ++q4) {
          uint32_t b[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float z = acc[i][f][4 * q4 + j];
            if constexpr (kL1) {
              const float up = WB == 1 ? acc[i][0][(4 * q4 + j + 8) & 15] : acc[i][(f + WB / 2) % WB][4 * q4 + j];
              b[j] = f32_to_bf16_any(mx_silu(z) * up);
            } else {
              b[j] = f32_to_bf16_any(z);
            }
          }
          put(4 * f + q4, u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16});
        }
#pragma unroll
      for (int k = 0; k < kPieces / 2; ++k) {
        const int rr = k * (kWave / kPieces) + ln / kPieces, piece = ln % kPieces;
        const int R = wm * 64 + 32 * i + rr, c = c0 + 8 * piece;
        const u32x4 v = *reinterpret_cast<const u32x4*>(o_lds + rr * kRow + 16 * (piece ^ (rr & (kPieces - 1))));
        if (R < cur.left && c < p.N)
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + (cur.row0 + R) * (int64_t)p.N + c));
      }
    };
    store_rows(IntTag<0>{});
    store_rows(IntTag<1>{});
    first = false;
  };
  for (; t < total; t += kMxGrid) {
    if (cur.wb == 4) run_tile(IntTag<4>{});
    else if (cur.wb == 2) run_tile(IntTag<2>{});
    else run_tile(IntTag<1>{});
    cur = nxt;
  }
}

// The dynamic LDS limit of a kernel, raised once a device.
template <typename F>
static hipError_t mx_allow_lds(F* kernel, std::atomic<bool> (&done)[kMxDevices]) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev < kMxDevices && done[dev].load(std::memory_order_acquire)) return hipSuccess;
  err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kMxLds);
  if (err == hipSuccess && dev < kMxDevices) done[dev].store(true, std::memory_order_release);
  return err;
}

// How the small kernel runs for this K: split or not; token rows of its m-tiles, 16, or 8 or 4 where 16
// (or 8) rows of K elements would leave fewer than 4 ring slots a wave; slots.  0 slots: K is too long for it.
struct MxSmallPlan {
  bool split;
  int mrows, slots;
  size_t lds;
};
static MxSmallPlan mx_small_plan(int K) {
  const int64_t nch = (K + kMxChunk - 1) / kMxChunk;
  const auto plan = [&](bool split, int mrows) -> MxSmallPlan {
    const int64_t rows = nch * mrows * (kMxChunk / 2 + kMxChunk / 32);
    const int64_t fixed = split ? rows + kMxRed : kMxSplit * rows;
    int64_t slots = (kMxLds - fixed) / (kMxSplit * kMxSlot);
    if (slots > kMxMaxSlots) slots = kMxMaxSlots;
    if (fixed >= kMxLds || slots < 4) return {split, 0, 0, 0};
    return {split, mrows, (int)slots, (size_t)(fixed + kMxSplit * slots * kMxSlot)};
  };
  MxSmallPlan p = plan(false, kMxSmallRows);
  for (int mrows = kMxSmallRows; p.slots == 0 && mrows >= 4; mrows /= 2) p = plan(true, mrows);
  return p;
}

template <bool kL1>
static hipError_t launch_mx(const MxGemmArgs& a, const MxSmallPlan& plan, bool small, bool large, hipStream_t stream) {
  static std::atomic<bool> whole_done[kMxDevices], split_done[kMxDevices], tile_done[kMxDevices];
  hipError_t err = hipSuccess;
  if (small) {
    const auto kernel = plan.split ? mx_small_kernel<kL1, true> : mx_small_kernel<kL1, false>;
    err = mx_allow_lds(kernel, plan.split ? split_done : whole_done);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(kernel, dim3(kMxGrid), dim3(kMxSplit * kWave), plan.lds, stream, a, plan.slots);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (large) {
    err = mx_allow_lds(mx_tile_kernel<kL1>, tile_done);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(mx_tile_kernel<kL1>, dim3(kMxGrid), dim3(kMxThreads),
                       kMxTables + sizeof(int) * ((size_t)kMxBm + a.E + 1), stream, a);
    err = hipGetLastError();
  }
  return err;
}

hipError_t launch_mx_gemm(const MxGemmArgs& a0, bool l1, int64_t max_rows, hipStream_t stream) {
  MxGemmArgs a = a0;
  const MxSmallPlan plan = mx_small_plan(a.K);
  a.mrows = plan.mrows;
  // A dense call knows its rows.  A grouped one launches both kernels, which decide from the counts, unless
  // the caller's bound says that no expert has more than the small kernel's rows; it then covers every
  // expert, should the bound be wrong.  With a K beyond the small kernel's the tile kernel takes everything.
  bool small = true, large = !(max_rows > 0 && max_rows <= kMxSmallRows);
  if (a.counts == nullptr) {
    small = a.M <= kMxSmallRows || mx_small_takes_all(a, mx_load_of(a, l1, (int)a.M));
    large = !small;
  }
  if (plan.slots == 0) {
    small = false;
    large = true;
  }
  a.cover_large = !large;
  a.cover_small = !small;
  return l1 ? launch_mx<true>(a, plan, small, large, stream) : launch_mx<false>(a, plan, small, large, stream);
}

}  // namespace megamoe
