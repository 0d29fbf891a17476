// Matrix products C = sum_t A_t B_t^T on bf16 MFMAs, with the caller's own
// epilogue, for the 4-bit projection and the vocabulary loss.
//
// An operand lies with the reduction axis contiguous (rows of K elements), or
// turned (K rows, as a weight lies for its input gradient and both operands of a
// weight's gradient do): then the LDS turns it, four rows of 16 columns a read.
// It comes in one or more planes: an fp32 operand is held as bf16 planes
// hi + mid + lo (24 bits), and the product as the sum of the plane pairs
// ("terms") whose size reaches the result's precision.  All terms of a tile
// run through one accumulator.
//
// A workgroup computes a BM x BN tile.  Every wave loads its part of each
// 64-element k-step straight into an NS-slot LDS ring (1 KB a wave
// instruction, whole lines, swizzled) up to NS steps ahead, and multiplies its WM
// x WN part of the tile; one barrier a step hands a landed slot over and a used
// one back.
#pragma once

#include <algorithm>

#include "../../include/dyra.h"
#include "lds_dma.h"

namespace product {
namespace {   // kernels made in one source file are not another's

constexpr int OUT = (int)0x80000000u;   // an offset out of range: reads as zero

// `rows` rows of K elements, or (turned) K rows of `rows` elements; row r of
// plane t at p + t * plane + r * ld (bytes).
struct Operand {
  const void* p;
  int64_t ld, plane;
  int32_t rows;
};

// Plane pairs of a product, four bits each: plane of A, plane of B << 2; the
// first to be added lowest.
constexpr uint32_t pair_of(int a, int b) { return (uint32_t)(a | b << 2); }
constexpr uint32_t TERMS_1 = pair_of(0, 0);
// three planes by three, without those below 2^-24: the smallest first
constexpr uint32_t TERMS_33 = pair_of(2, 0) | pair_of(0, 2) << 4 | pair_of(1, 1) << 8 | pair_of(1, 0) << 12 |
                              pair_of(0, 1) << 16 | pair_of(0, 0) << 20;
// three planes by two
constexpr uint32_t TERMS_32 = pair_of(2, 0) | pair_of(1, 1) << 4 | pair_of(1, 0) << 8 | pair_of(0, 1) << 12 |
                              pair_of(0, 0) << 16;

// What product_kernel computes: a.rows x b.rows results, `terms` plane pairs of
// nk 64-element steps each.  With `live` (a device word) the rows of A, or
// (live_k) the length of the reduction, are what it says, at most those here.
struct Job {
  Operand a, b;
  int32_t kbytes;      // bytes of a row that count, a multiple of 16
  int32_t krows;       // rows of a turned operand that count
  int32_t nk, terms;
  uint32_t pairs;
  int32_t may_split, live_k;
  const int32_t* live;
  float4* part;        // partial tiles, if may_split (part_bytes)
};

// A k-step takes ALONE hundredths of a microsecond with one workgroup on the card,
// ALONE + SHARED with all its places taken (the clock falls with the load).
template <int BM_, int BN_, int NWM_, int NWN_, int NS_, int WGS_, int ALONE_, int SHARED_>
struct Tile {
  static constexpr int ALONE = ALONE_, SHARED = SHARED_;
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NS = NS_;
  static constexpr int NW = NWM * NWN, NT = NW * 64;
  static constexpr int WM = BM / NWM, WN = BN / NWN, FM = WM / 32, FN = WN / 32;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KB loads a wave and step
  static constexpr int SLOT = (BM + BN) * 128;
  static constexpr int LDS = NS * SLOT;
  static constexpr int WPE = WGS_ * NW / 4;                  // waves per SIMD with WGS_ workgroups on a CU
  static constexpr int SLOTS = 256 * WGS_;                   // workgroups on the card at once
  static constexpr bool ALONE_ON_CU = WGS_ == 1;
  static constexpr int QUADS = FM * FN * 4;                  // groups of four results a lane
  static_assert(NW % 2 == 0, "a wave's row blocks have one parity, so one swizzle");
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN, "row blocks divide over the waves");
  static_assert(FM * 32 == WM && WN == 64, "a wave's part is made of 32 x 64 blocks");
};

// 256 x 256: 128 flop a byte loaded, one workgroup a CU (128 KB of LDS)
typedef Tile<256, 256, 2, 4, 2, 1, 100, 75> Big;
// 320 x 256: 142 flop a byte, and other sizes that fill whole rounds (5003 x 4096
// results of 64 steps are 256 of its tiles: a 4-bit projection 140 us instead of 166
// with 320 tiles of 256 x 256, a gradient of 4099 x 4096 of 192 steps 354 instead of
// 379; 1.28 PFLOP/s in whole rounds)
typedef Tile<320, 256, 2, 4, 2, 1, 125, 94> Tall;
// 128 x 128: four times the tiles, two workgroups a CU
typedef Tile<128, 128, 2, 2, 2, 2, 45, 55> Small;
// 64 x 128: a few rows against a matrix that is read once; a deeper ring
typedef Tile<64, 128, 2, 2, 3, 2, 30, 33> Thin;
// The same of an fp32 matrix that is split into its planes on the way (direct_kernel)
struct Direct : Tile<64, 128, 2, 2, 2, 1, 125, 125> {
  static constexpr int A_SLOT = BM * 128, SLOT = 3 * A_SLOT + BN * 256, LDS = NS * SLOT;
};

// How a product's tiles are laid over the workgroups.  The card holds SLOTS of
// them at once: whole rounds of tiles are computed by one workgroup each.  The
// tiles of a last round that would leave much of the card idle are split along
// the reduction, if that saves more than the join costs (600 x 4096 results of 192
// steps: 94 us instead of 145).  Product and join work it out from the sizes
// that they find.
struct Layout {
  int rows, tiles_m, tiles_n, kbytes, krows, nk;
  int whole, tail, split, per;   // tiles computed whole, tiles split, parts of one, steps of a part
  int count;                     // workgroups
  double cost;                   // microseconds, estimated
};

template <class C>
__host__ __device__ inline Layout layout(const Job& j, int live) {
  Layout y;
  y.rows = j.a.rows;
  y.kbytes = j.kbytes;
  y.krows = j.krows;
  y.nk = j.nk;
  if (live >= 0) {
    if (j.live_k) {
      y.krows = live < j.krows ? live : j.krows;
      y.kbytes = 2 * y.krows;
      y.nk = (y.krows + 63) / 64;
    } else {
      y.rows = live < y.rows ? live : y.rows;
    }
  }
  y.tiles_m = (y.rows + C::BM - 1) / C::BM;
  y.tiles_n = (j.b.rows + C::BN - 1) / C::BN;
  const int tiles = y.tiles_m * y.tiles_n, steps = j.terms * y.nk, rest = tiles % C::SLOTS;
  // hundredths of a microsecond of a step of n workgroups
  auto step = [](int n) { return n / C::SLOTS * (C::ALONE + C::SHARED) +
                                 (n % C::SLOTS ? C::ALONE + C::SHARED * (n % C::SLOTS) / C::SLOTS : 0); };
  int split = 1, least = steps * step(rest);
  if (j.may_split && rest) {
    for (int s = 2; s <= 16 && s * 4 <= steps && rest * s <= 2 * C::SLOTS; ++s) {   // at least four steps a part
      // the parts, their way through memory at 5 TB/s, a launch
      const int cost = (steps + s - 1) / s * step(rest * s) + rest * s * (C::BM * C::BN / 1024) / 6 + 600;
      if (cost < least) {
        least = cost;
        split = s;
      }
    }
  }
  y.per = (steps + split - 1) / split;
  y.split = split > 1 ? (steps + y.per - 1) / y.per : 1;   // no part without a step
  y.tail = split > 1 ? rest : 0;
  y.whole = tiles - y.tail;
  y.count = y.whole + y.tail * y.split;
  y.cost = 0.01 * ((double)(tiles / C::SLOTS) * steps * (C::ALONE + C::SHARED) + least);
  return y;
}

// First row and column of a tile.  Consecutive numbers walk bands of four tile
// rows column by column: the 32 workgroups of an XCD then share four row
// blocks of A and eight of B in its L2.
template <class C>
__device__ __forceinline__ void corner(const Layout& y, int t, int& m0, int& n0) {
  const int band = t / (4 * y.tiles_n), first = band * 4, high = min(4, y.tiles_m - first);
  t -= first * y.tiles_n;
  const int tn = t / high;
  m0 = (first + t - tn * high) * C::BM;
  n0 = tn * C::BN;
}

template <class C>
using Acc = f32x16[C::FM][C::FN];

// Eight numbers in N bf16 planes.  The first of several is at most bf16's largest
// number: rounded, a finite number above 2^128 (1 - 2^-9) would become an infinity
// and the next planes NaN; what is cut off fits the other two as well.  A single
// plane is rounded as usual.
template <int N>
__device__ __forceinline__ void split(float (&v)[8], uint4 (&out)[N]) {
  constexpr float TOP = 0x1.fep127f;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (N > 1 && t == 0)
        h[e] = pack_bf16x2(__builtin_amdgcn_fmed3f(v[2 * e], -TOP, TOP),
                           __builtin_amdgcn_fmed3f(v[2 * e + 1], -TOP, TOP));
      else h[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      v[2 * e] -= __uint_as_float(h[e] << 16);
      v[2 * e + 1] -= __uint_as_float(h[e] & 0xffff0000u);
    }
    out[t] = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// A turned operand in a slot: 64 rows of W = BM or BN elements.  A 16-byte chunk
// lies at chunk ^ turn(row): the four rows that 32 lanes read together lie in four
// different quarters of the 256-byte bank window.
template <int W>
__device__ __forceinline__ int turn(int row) {
  return W >= 128 ? (row & 3) << 2 : (row & 2) << 1;
}

// Four elements of one column: of 16 lanes, lane i gives the place of row i / 4,
// columns 4 (i % 4) .. + 3, and receives column i of the four rows.
__device__ __forceinline__ uint2 read_turned(const char* at) {
  typedef short four __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) four*)(uintptr_t)(const __attribute__((address_space(3))) char*)at));
}

// F operands of 32 rows or columns of a wave in a slot, for one sub-step of 16
// after the other.
template <int W, int F, bool TURNED>
struct Feed {
  int off[TURNED ? F : 2];

  __device__ __forceinline__ Feed(int first, int lane) {
    if constexpr (TURNED) {
      const int i = lane & 15;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int chunk = first / 8 + 4 * f + 2 * (lane >> 4 & 1) + (i >> 1 & 1);
        off[f] = (8 * (lane >> 5) + (i >> 2)) * (2 * W) + ((chunk ^ turn<W>(i >> 2)) << 4) + (i & 1) * 8;
      }
    } else {
      off[0] = (first + (lane & 31)) * 128;
      off[1] = (lane >> 5) ^ (lane >> 1 & 7);   // chunk 2 s + lane / 32 at chunk ^ (row / 2 % 8)
    }
  }
  __device__ __forceinline__ uint4 read(const char* slot, int s, int f) const {
    if constexpr (TURNED) {
      const char* at = slot + off[f] + 16 * s * (2 * W);
      const uint2 a = read_turned(at), b = read_turned(at + 4 * (2 * W));
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      return *reinterpret_cast<const uint4*>(slot + off[0] + f * 4096 + (((2 * s) ^ off[1]) << 4));
    }
  }
};

// The L loads with which a wave brings its part of an operand's k-step: 1 KB each,
// eight rows of 128 bytes, or whole rows of a turned operand.
template <int W, int L, int NW, bool TURNED>
struct Bring {
  int v[L], edge;   // offsets from the operand's corner; row or byte of the first within a step
  const char* p;
  int64_t ld;

  // corner: of the tile's first row, or (turned) column; count: rows or columns from there on
  __device__ __forceinline__ void aim(const Operand& o, int at, int plane) {
    p = reinterpret_cast<const char*>(o.p) + plane * o.plane + (TURNED ? 2 * (int64_t)at : at * o.ld);
    ld = o.ld;
  }
  __device__ __forceinline__ void open(const Operand& o, int count, int w, int lane) {
    if constexpr (TURNED) {
      constexpr int CPR = W / 8, RPB = 64 / CPR;   // chunks a row, rows a load
      edge = w * RPB + lane / CPR;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int row = edge + i * NW * RPB, ch = (lane % CPR) ^ turn<W>(row);
        v[i] = ch * 8 < count ? row * (int)o.ld + ch * 16 : OUT;
      }
    } else {
      // row 8 w + lane / 8, 16-byte chunk (lane % 8) ^ (row / 2 % 8); NW is even
      const int row0 = 8 * w + (lane >> 3);
      edge = ((lane & 7) ^ ((row0 >> 1) & 7)) << 4;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int row = row0 + 8 * NW * i;
        v[i] = row < count ? row * (int)o.ld + edge : OUT;
      }
    }
  }
  // step kt to LDS at `to`; live: whether it is one at all
  template <int OFF>
  __device__ __forceinline__ void step(int kt, int kbytes, int krows, bool live, uint32_t to) const {
    if constexpr (TURNED) {
      const i32x4v rs = rsrc_words(p + (int64_t)kt * 64 * ld, 0x7fffffffu);
      constexpr int RPB = 512 / W;
      if (live && kt * 64 + 64 <= krows) {
        static_for<0, L>([&](auto i) __attribute__((always_inline)) {
          constexpr int I = decltype(i)::value;
          dma16k<OFF + I * NW * 1024>(rs, v[I], 0, to);
        });
      } else {
        const int rows = live ? krows - kt * 64 : 0;
        static_for<0, L>([&](auto i) __attribute__((always_inline)) {
          constexpr int I = decltype(i)::value;
          dma16k<OFF + I * NW * 1024>(rs, edge + I * NW * RPB < rows ? v[I] : OUT, 0, to);
        });
      }
    } else {
      const i32x4v rs = rsrc_words(p, 0x7fffffffu);
      const int kb = kt * 128;
      if (live && kb + 128 <= kbytes) {
        static_for<0, L>([&](auto i) __attribute__((always_inline)) {
          constexpr int I = decltype(i)::value;
          dma16k<OFF + I * NW * 1024>(rs, v[I], kb, to);
        });
      } else {
        const bool in = live && edge < kbytes - kb;
        static_for<0, L>([&](auto i) __attribute__((always_inline)) {
          constexpr int I = decltype(i)::value;
          dma16k<OFF + I * NW * 1024>(rs, in ? v[I] : OUT, kb, to);
        });
      }
    }
  }
};

// Epilogues: e.tile<C>(acc, lds, m0, n0, rows, wm, wn) takes a whole tile (the
// ring is its to use), e.block<C>(v, lds, row0, col0, rows) 32 x WN results of
// one wave, which has 32 * WN floats of LDS.
template <class C, bool TA, bool TB, class E>
__global__ __launch_bounds__(C::NT, C::WPE) void product_kernel(Job j, E e) {
  __shared__ __attribute__((aligned(1024))) char ring[C::LDS];
  const Layout y = layout<C>(j, j.live ? *j.live : -1);
  if ((int)blockIdx.x >= y.count) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / C::NWN, wn = w % C::NWN;
  // whole tiles and parts are each dealt over the XCDs; a part if not negative
  const int over = (int)blockIdx.x - y.whole, part = over < 0 ? over : xcd_tile_id(over, y.count - y.whole);
  int m0, n0, first = 0, steps = j.terms * y.nk;
  if (part < 0) {
    corner<C>(y, xcd_tile_id(blockIdx.x, y.whole), m0, n0);
  } else {
    const int z = part / y.tail;
    corner<C>(y, y.whole + part - z * y.tail, m0, n0);
    first = z * y.per;
    steps = max(0, min(y.per, steps - first));
  }
  Bring<C::BM, C::LA, C::NW, TA> a;
  Bring<C::BN, C::LB, C::NW, TB> b;
  a.open(j.a, y.rows - m0, w, lane);
  b.open(j.b, j.b.rows - n0, w, lane);
  const uint32_t base = lds_addr(ring) + w * 1024;
  int term = y.nk ? first / y.nk : 0, kt = first - term * y.nk, left = steps;
  auto aim = [&]() __attribute__((always_inline)) {
    const uint32_t pr = j.pairs >> (4 * term);
    a.aim(j.a, m0, pr & 3);
    b.aim(j.b, n0, pr >> 2 & 3);
  };
  aim();
  // one k-step into a slot; past the last every lane reads out of range, so
  // that each step issues the same number of loads
  auto issue = [&](uint32_t slot) __attribute__((always_inline)) {
    a.template step<0>(kt, y.kbytes, y.krows, left > 0, base + slot);
    b.template step<C::BM * 128>(kt, y.kbytes, y.krows, left > 0, base + slot);
    if (--left > 0 && ++kt == y.nk) {
      kt = 0;
      ++term;
      aim();
    }
  };
  Acc<C> acc;
#pragma unroll
  for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[fm][fn][v] = 0.f;
  const bool busy = m0 + wm * C::WM < y.rows && n0 + wn * C::WN < j.b.rows;   // a wave past the edge has no results
  const Feed<C::BM, C::FM, TA> fa(wm * C::WM, lane);
  const Feed<C::BN, C::FN, TB> fb(wn * C::WN, lane);
  uint4 af[2][C::FM], bf[2][C::FN];
  auto pull = [&](const char* slot, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < C::FM; ++f) af[s & 1][f] = fa.read(slot, s, f);
#pragma unroll
    for (int f = 0; f < C::FN; ++f) bf[s & 1][f] = fb.read(slot + C::BM * 128, s, f);
  };
  // products from .. to - 1 of a sub-step.  The operands are swapped, so that lane
  // (l, g) ends with row l of A and, in element 4 q + e, column 8 q + 4 g + e of B.
  auto multiply = [&](int s, int from, int to) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C::FM * C::FN; ++i)
      if (i >= from && i < to)
        TT<bf16_t>::mma(acc[i / C::FN][i % C::FN], bf[s & 1][i % C::FN], af[s & 1][i / C::FN]);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int ALL = C::FM * C::FN, LOADS = C::LA + C::LB, FIRST = C::ALONE_ON_CU ? C::NS : C::NS - 1;
  uint32_t at = 0, to = FIRST == C::NS ? 0 : (C::NS - 1) * C::SLOT;   // the slot of step t; that which is loaded next
  auto past = [](uint32_t slot) { return slot + C::SLOT == C::LDS ? 0u : slot + C::SLOT; };
#pragma unroll
  for (int s = 0; s < FIRST; ++s) issue(s * C::SLOT);
  auto walk = [&](auto multiplies) __attribute__((always_inline)) {
    constexpr bool MULTIPLIES = decltype(multiplies)::value;
    if constexpr (C::ALONE_ON_CU) {
      // Nobody else keeps the matrix cores busy: sub-step s + 1 is read while s
      // multiplies, and before the last one the wave waits for the next step's
      // loads and for the others to have read this step's slot, so that the last
      // one's products cover the next step's first reads and the loads into the
      // slot that came free (4099 x 32000 x 4096 in 256 x 256 tiles: 927 against 960 us).
      wait_vm_lgkm0<(C::NS - 1) * LOADS>();   // this wave's loads of step 0 have landed
      bare_barrier();                          // everyone's
      if constexpr (MULTIPLIES) pull(ring, 0);
      for (int t = 0; t < steps; ++t) {
        if constexpr (MULTIPLIES) {
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            pull(ring + at, s + 1);
            multiply(s, 0, ALL);
          }
        }
        wait_vm_lgkm0<(C::NS - 2) * LOADS>();   // this wave's loads of step t + 1 have landed
        bare_barrier();                          // everyone's; the slot of step t is free
        if constexpr (MULTIPLIES) {
          pull(ring + past(at), 0);
          multiply(3, 0, ALL / 2);
        }
        issue(at);   // step t + NS
        if constexpr (MULTIPLIES) multiply(3, ALL / 2, ALL);
        at = past(at);
      }
    } else {
      for (int t = 0; t < steps; ++t) {
        wait_vm_lgkm0<(C::NS - 2) * LOADS>();   // this wave's loads of step t have landed
        bare_barrier();                          // everyone's; the slot of step t - 1 is free
        issue(to);                               // step t + NS - 1
        to = past(to);
        if constexpr (MULTIPLIES) {
          pull(ring + at, 0);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s < 3) pull(ring + at, s + 1);
            multiply(s, 0, ALL);
          }
        }
        at = past(at);
      }
    }
  };
  if (busy) walk(std::true_type());
  else walk(std::false_type());
  wait_vm_lgkm0<0>();
  bare_barrier();   // no load is under way, no slot is read: the ring is the epilogue's
  if (part < 0) {
    e.template tile<C>(acc, ring, m0, n0, y.rows, wm, wn);
    return;
  }
  // a part in the order of the registers: whole lines, no staging
  float4* mine = j.part + ((int64_t)part * C::NW + w) * C::QUADS * 64 + lane;
#pragma unroll
  for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[((fm * C::FN + fn) * 4 + q) * 64] = make_float4(acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1],
                                                           acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3]);
}

// The B of direct_kernel: 64 fp32 elements of 128 rows, or (turned) 64 rows of 128
// elements, 32 KB a step, eight loads a wave.
template <bool TURNED>
struct Fp32 {
  static constexpr int LOADS = 8;
  int v[LOADS], edge;
  const char* p;
  int64_t ld;

  __device__ __forceinline__ void open(const Operand& o, int at, int w, int lane) {
    const int count = o.rows - at;
    ld = o.ld;
    p = reinterpret_cast<const char*>(o.p) + (TURNED ? 4 * (int64_t)at : at * ld);
    if constexpr (TURNED) {
      // row 2 w + 8 i + lane / 32; chunk ^ 8 in every other eight rows, which the two
      // halves of a wave read together
      edge = 2 * w + (lane >> 5);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int row = edge + 8 * i, ch = (lane & 31) ^ ((row & 8));
        v[i] = ch * 4 < count ? row * (int)ld + ch * 16 : OUT;
      }
    } else {
      // row 4 w + 16 i + lane / 16, chunk (lane % 16) ^ (row % 16)
      const int row0 = 4 * w + (lane >> 4);
      edge = ((lane & 15) ^ row0) << 4;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int row = row0 + 16 * i;
        v[i] = row < count ? row * (int)ld + edge : OUT;
      }
    }
  }
  // bytes: of a row; rows: that count
  template <int OFF>
  __device__ __forceinline__ void step(int kt, int bytes, int rows, bool live, uint32_t to) const {
    const i32x4v rs = rsrc_words(TURNED ? p + (int64_t)kt * 64 * ld : p, 0x7fffffffu);
    const int kb = TURNED ? 0 : kt * 256, left = live ? (TURNED ? rows - kt * 64 : bytes - kb) : 0;
    static_for<0, LOADS>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      dma16k<OFF + I * 4096>(rs, edge + (TURNED ? 8 * I : 0) < left ? v[I] : OUT, kb, to);
    });
  }
  // 8 elements of row or column `at` for sub-step s
  __device__ __forceinline__ static void read(const char* slot, int s, int at, int g, float (&x)[8]) {
    if constexpr (TURNED) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 16 * s + 8 * g + e;
        x[e] = *reinterpret_cast<const float*>(slot + row * 512 + (((at >> 2) ^ (8 * g)) << 4) + (at & 3) * 4);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = *reinterpret_cast<const float4*>(slot + at * 256 + (((4 * s + 2 * g + h) ^ (at & 15)) << 4));
        x[4 * h] = f.x, x[4 * h + 1] = f.y, x[4 * h + 2] = f.z, x[4 * h + 3] = f.w;
      }
    }
  }
};

// A few rows, in three planes, by an fp32 matrix that is read once, as it lies: each
// wave splits what it multiplies, which takes about as long as the six products do,
// and both less than the matrix takes to arrive.  Loss of fp32 rows, us (with planes
// of W in memory first): 4 x 2048 x 30000 74 (232), 100 x 1024 x 8000 33 (49), 400 x 2048 x
// 4000 75 (74); with more rows the splitting costs more than the planes, 1500 x 512 x
// 8000 123 (85).  Between those the estimate of 128 x 128 tiles is some 15 % high: 700 x
// 1024 x 5000 runs here, 79 (68).
template <bool TB, class E>
__global__ __launch_bounds__(Direct::NT, 1) void direct_kernel(Job j, E e) {
  typedef Direct C;
  __shared__ __attribute__((aligned(1024))) char ring[C::LDS];
  const Layout y = layout<C>(j, j.live ? *j.live : -1);
  if ((int)blockIdx.x >= y.count) return;
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 31, g = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / C::NWN, wn = w % C::NWN;
  const int over = (int)blockIdx.x - y.whole, part = over < 0 ? over : xcd_tile_id(over, y.count - y.whole);
  int m0, n0, kt = 0, steps = y.nk;
  if (part < 0) {
    corner<C>(y, xcd_tile_id(blockIdx.x, y.whole), m0, n0);
  } else {
    const int z = part / y.tail;
    corner<C>(y, y.whole + part - z * y.tail, m0, n0);
    kt = z * y.per;
    steps = max(0, min(y.per, y.nk - kt));
  }
  Bring<C::BM, C::LA, C::NW, false> a[3];
  Fp32<TB> b;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    a[t].open(j.a, y.rows - m0, w, lane);
    a[t].aim(j.a, m0, t);
  }
  b.open(j.b, n0, w, lane);
  const uint32_t base = lds_addr(ring) + w * 1024;
  int left = steps;
  auto issue = [&](uint32_t slot) __attribute__((always_inline)) {
    static_for<0, 3>([&](auto t) __attribute__((always_inline)) {
      constexpr int T = decltype(t)::value;
      a[T].template step<T * C::A_SLOT>(kt, y.kbytes, y.krows, left > 0, base + slot);
    });
    b.template step<3 * C::A_SLOT>(kt, 2 * y.kbytes, y.krows, left > 0, base + slot);
    --left;
    ++kt;
  };
  Acc<C> acc;
#pragma unroll
  for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[0][fn][v] = 0.f;
  const bool busy = m0 + wm * C::WM < y.rows && n0 + wn * C::WN < j.b.rows;
  const Feed<C::BM, C::FM, false> fa(wm * C::WM, lane);
  uint32_t at = 0;
  issue(0);
  auto walk = [&](auto multiplies) __attribute__((always_inline)) {
    for (int t = 0; t < steps; ++t) {
      wait_vm_lgkm0<0>();   // this wave's loads of step t have landed
      bare_barrier();       // everyone's; the other slot is free
      issue(C::SLOT - at);  // step t + 1
      if constexpr (decltype(multiplies)::value) {
        const char* slot = ring + at;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint4 x[3], q[C::FN][3];
#pragma unroll
          for (int t3 = 0; t3 < 3; ++t3) x[t3] = fa.read(slot + t3 * C::A_SLOT, s, 0);
#pragma unroll
          for (int fn = 0; fn < C::FN; ++fn) {
            float f[8];
            Fp32<TB>::read(slot + 3 * C::A_SLOT, s, wn * C::WN + fn * 32 + l, g, f);
            split(f, q[fn]);
          }
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            const uint32_t pr = TERMS_33 >> (4 * i);
#pragma unroll
            for (int fn = 0; fn < C::FN; ++fn) TT<bf16_t>::mma(acc[0][fn], q[fn][pr >> 2 & 3], x[pr & 3]);
          }
        }
      }
      at = C::SLOT - at;
    }
  };
  if (busy) walk(std::true_type());
  else walk(std::false_type());
  wait_vm_lgkm0<0>();
  bare_barrier();
  if (part < 0) {
    e.template tile<C>(acc, ring, m0, n0, y.rows, wm, wn);
    return;
  }
  float4* mine = j.part + ((int64_t)part * C::NW + w) * C::QUADS * 64 + lane;
#pragma unroll
  for (int i = 0; i < C::FN * 4; ++i)
    mine[i * 64] = make_float4(acc[0][i / 4][i % 4 * 4], acc[0][i / 4][i % 4 * 4 + 1], acc[0][i / 4][i % 4 * 4 + 2],
                               acc[0][i / 4][i % 4 * 4 + 3]);
}

// Adds the parts of the split tiles, in their order; one wave for 32 x WN results.
template <class C, class E>
__device__ __forceinline__ void join(const Job& j, const E& e, int block, char* lds) {
  const Layout y = layout<C>(j, j.live ? *j.live : -1);
  const int tail = block / (C::NW * C::FM), sub = block - tail * (C::NW * C::FM);
  if (tail >= y.tail) return;
  const int w = sub / C::FM, fm = sub - w * C::FM;
  int m0, n0;
  corner<C>(y, y.whole + tail, m0, n0);
  const int row0 = m0 + w / C::NWN * C::WM + fm * 32, col0 = n0 + w % C::NWN * C::WN;
  if (row0 >= y.rows || col0 >= j.b.rows) return;
  f32x16 v[C::FN];
#pragma unroll
  for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
    for (int i = 0; i < 16; ++i) v[fn][i] = 0.f;
#pragma unroll 4
  for (int z = 0; z < y.split; ++z) {
    const float4* from =
        j.part + ((int64_t)(z * y.tail + tail) * C::NW + w) * C::QUADS * 64 + fm * C::FN * 256 + threadIdx.x;
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 x = from[(fn * 4 + q) * 64];
        v[fn][4 * q] += x.x;
        v[fn][4 * q + 1] += x.y;
        v[fn][4 * q + 2] += x.z;
        v[fn][4 * q + 3] += x.w;
      }
  }
  e.template block<C>(v, lds, row0, col0, y.rows);
}

constexpr int JOIN_LDS = 32 * 64 * 4;   // every tile's WN is 64

template <class C, class E>
__global__ __launch_bounds__(64) void join_kernel(Job j, E e) {
  __shared__ __attribute__((aligned(1024))) char lds[JOIN_LDS];
  join<C>(j, e, blockIdx.x, lds);
}

// ---------------------------------------------------------------------------
// epilogue: the tile to memory
// ---------------------------------------------------------------------------

// out[row][col] (rows ld elements apart) = (acc + prior[row][col]) * factor + bias[col].
// 32 rows at a time go through LDS, so that every store covers whole 128-byte
// lines.  map: the result's row is out's row map[row].
template <typename T>
struct Store {
  T* out;
  int64_t ld;
  int32_t cols;           // a multiple of 8
  const T* bias;          // or null
  const float* prior;     // fp32 [rows][cols], or null
  const int32_t* map;     // or null
  const float* weight;    // of the factor, or null: 1
  float scale;

  template <class C>
  __device__ __forceinline__ void block(const f32x16 (&v)[C::FN], char* lds, int row0, int col0, int rows) const {
    constexpr int E = 16 / sizeof(T), CPR = C::WN / E;   // elements a chunk, chunks a staged row
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    const bool old = prior && row0 + l < rows;
    const float factor = weight ? *weight * scale : 1.f;
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = fn * 32 + 8 * q + 4 * g;
        float x[4] = {v[fn][4 * q], v[fn][4 * q + 1], v[fn][4 * q + 2], v[fn][4 * q + 3]};
        if (old && col0 + col < cols) {
          const float4 o = *reinterpret_cast<const float4*>(prior + (int64_t)(row0 + l) * cols + col0 + col);
          x[0] += o.x, x[1] += o.y, x[2] += o.z, x[3] += o.w;
        }
        if (weight) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= factor;
        }
        if (bias && col0 + col < cols) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += TT<T>::to_f(bias[col0 + col + e]);
        }
        char* at = lds + l * (CPR * 16) + stage_chunk<CPR>(l, col / E) * 16;
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(at + (col & 4) * 2) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        else *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 32 * CPR / 64; ++i) {
      const int c = lane + i * 64, rr = c / CPR, k = c % CPR;
      const uint4 x = *reinterpret_cast<const uint4*>(lds + rr * (CPR * 16) + stage_chunk<CPR>(rr, k) * 16);
      const int row = row0 + rr, col = col0 + k * E;
      if (row < rows && col < cols) *reinterpret_cast<uint4*>(out + (map ? map[row] : row) * ld + col) = x;
    }
    __builtin_amdgcn_wave_barrier();
  }

  template <class C>
  __device__ __forceinline__ void tile(Acc<C>& acc, char* lds, int m0, int n0, int rows, int wm, int wn) const {
    static_assert(C::NW * 32 * C::WN * 4 <= C::LDS, "staging fits the ring");
    char* mine = lds + (wm * C::NWN + wn) * (32 * C::WN * 4);
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
      block<C>(acc[fm], mine, m0 + wm * C::WM + fm * 32, n0 + wn * C::WN, rows);
  }
};

// ---------------------------------------------------------------------------
// planes
// ---------------------------------------------------------------------------

// A matrix [rows][cols] as bf16 planes, eight elements a thread.  map: only
// its rows map[0 .. *live - 1].
template <typename T>
struct Planes {
  const T* in;
  int64_t ld, plane;
  bf16_t* out;                 // [planes][rows][cols]
  const int32_t *map, *live;   // or null
  int32_t rows, cols;
};

// Eight elements from row `from` to row `to`.
template <typename T>
__device__ __forceinline__ void split_eight(const Planes<T>& a, int64_t from, int64_t to, int col) {
  const T* p = a.in + from * a.ld + col;
  bf16_t* o = a.out + to * a.cols + col;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(p);
  } else {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint4 q[3];
    split(v, q);
#pragma unroll
    for (int t = 0; t < 3; ++t) *reinterpret_cast<uint4*>(o + t * a.plane) = q[t];
  }
}

template <typename T>
__device__ __forceinline__ void make_planes(const Planes<T>& a, int64_t i) {
  const int per = a.cols / 8;
  const int64_t row = i / per;
  if (row >= (a.live ? min(*a.live, a.rows) : a.rows)) return;
  split_eight(a, a.map ? a.map[row] : row, row, (int)(i - row * per) * 8);
}

// Two matrices in one launch, the first in `first` workgroups.
template <typename T>
__global__ __launch_bounds__(256) void planes_kernel(Planes<T> a, Planes<T> b, int first) {
  if ((int)blockIdx.x < first) make_planes(a, (int64_t)blockIdx.x * 256 + threadIdx.x);
  else make_planes(b, (int64_t)(blockIdx.x - first) * 256 + threadIdx.x);
}

// planes of an operand of type T
template <typename T> constexpr int planes_of() { return sizeof(T) == 2 ? 1 : 3; }

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// K: the reduction; Kb: as long as it is in memory where it lies contiguous (a
// multiple of 8).  live: what the rows of A (live_k: the reduction) are found to
// be, or null.
inline Job job(Operand a, Operand b, int64_t K, int64_t Kb, int terms, uint32_t pairs, const int32_t* live = nullptr,
               bool live_k = false) {
  Job j{};
  j.a = a;
  j.b = b;
  j.kbytes = (int32_t)(2 * Kb);
  j.krows = (int32_t)K;
  j.nk = (int32_t)cdiv(K, 64);
  j.terms = terms;
  j.pairs = pairs;
  j.may_split = 1;
  j.live = live;
  j.live_k = live_k;
  return j;
}

inline size_t align256(int64_t b) { return ((size_t)b + 255) & ~(size_t)255; }
inline int64_t up(int64_t a, int64_t m) { return cdiv(a, m) * m; }

// The tile of a product, by the estimated time.
enum Shape { BIG, SMALL, THIN, TALL, DIRECT };

inline Shape shape_of(const Job& j) {
  if (j.a.rows <= 64) return THIN;
  const double big = layout<Big>(j, -1).cost, small = layout<Small>(j, -1).cost;
  // where rows or steps are counted on the device, the least padding: 256 (3280 of
  // 4099 rows, gradients of 4096 x 32000: 2245 us instead of 2315)
  if (!j.live && layout<Tall>(j, -1).cost < std::min(big, small)) return TALL;
  return big <= small ? BIG : SMALL;
}

// Estimated microseconds of a product.
inline double cost(Shape s, const Job& j) {
  return s == DIRECT  ? layout<Direct>(j, -1).cost
         : s == TALL  ? layout<Tall>(j, -1).cost
         : s == BIG   ? layout<Big>(j, -1).cost
         : s == SMALL ? layout<Small>(j, -1).cost
                      : layout<Thin>(j, -1).cost;
}

// Bytes of partial tiles that a product may leave.
template <class C>
inline int64_t part_bytes_as(const Job& j) {
  if (!j.may_split) return 0;
  const Layout y = layout<C>(j, -1);
  // other sizes found on the device may split other tiles
  const int64_t parts = j.live ? std::min<int64_t>(2 * C::SLOTS, 16 * (int64_t)y.tiles_m * y.tiles_n) : y.tail * y.split;
  return parts * C::BM * C::BN * 4;
}

inline int64_t part_bytes(Shape s, const Job& j) {
  return s == DIRECT  ? part_bytes_as<Direct>(j)
         : s == TALL  ? part_bytes_as<Tall>(j)
         : s == BIG   ? part_bytes_as<Big>(j)
         : s == SMALL ? part_bytes_as<Small>(j)
                      : part_bytes_as<Thin>(j);
}

// Workgroups of a product and of its join.
struct Grids {
  int64_t product, join;
};

template <class C>
inline Grids grids_as(const Job& j) {
  const Layout y = layout<C>(j, -1);
  int64_t grid = y.count, tail = y.tail;
  // Fewer live rows or steps may leave other tiles to split; but not where one tile
  // row is all or none, or too short to be split.  A workgroup that finds nothing to
  // do costs its place for some microseconds (300 x 1024 x 2000: 1024 of them 5 us),
  // so that a few sizes are gone through, and only for many the bound is taken:
  // all tiles and 2 SLOTS parts.
  if (j.live && j.may_split && j.terms * y.nk >= 8 && (j.live_k || y.tiles_m > 1)) {
    const int sizes = j.live_k ? y.nk : y.tiles_m, each = j.live_k ? 64 : C::BM;
    for (int i = 1; i < sizes && sizes <= 32; ++i) {
      const Layout z = layout<C>(j, i * each);
      grid = std::max<int64_t>(grid, z.count);
      tail = std::max<int64_t>(tail, z.tail);
    }
    if (sizes > 32) {
      grid = (int64_t)y.tiles_m * y.tiles_n + 2 * C::SLOTS;
      tail = std::min(C::SLOTS, y.tiles_m * y.tiles_n);
    }
  }
  return {grid, tail * C::NW * C::FM};
}

template <class C, bool TA, bool TB, class E>
inline void launch(const Job& j, const E& e, bool joined, hipStream_t st) {
  const Grids g = grids_as<C>(j);
  if (!g.product) return;
  hipLaunchKernelGGL((product_kernel<C, TA, TB, E>), dim3((unsigned)g.product), dim3(C::NT), 0, st, j, e);
  if (joined && g.join) hipLaunchKernelGGL((join_kernel<C, E>), dim3((unsigned)g.join), dim3(64), 0, st, j, e);
}

// TA, TB: operands that lie turned; COUNTED: rows or steps are counted on the device.
// joined: with the join, else the caller launches join_two.
template <bool TA, bool TB, bool COUNTED = false, class E>
void launch_as(Shape s, const Job& j, const E& e, hipStream_t st, bool joined = true) {
  if constexpr (!COUNTED)
    if (s == TALL) return launch<Tall, TA, TB>(j, e, joined, st);
  if (s == BIG) launch<Big, TA, TB>(j, e, joined, st);
  else if (s == SMALL) launch<Small, TA, TB>(j, e, joined, st);
  else launch<Thin, TA, TB>(j, e, joined, st);
}

// The same with B in fp32 (DIRECT): three planes of A in one walk.
template <bool TB, class E>
void launch_direct(const Job& j, const E& e, hipStream_t st, bool joined = true) {
  const Grids g = grids_as<Direct>(j);
  if (!g.product) return;
  hipLaunchKernelGGL((direct_kernel<TB, E>), dim3((unsigned)g.product), dim3(Direct::NT), 0, st, j, e);
  if (joined && g.join) hipLaunchKernelGGL((join_kernel<Direct, E>), dim3((unsigned)g.join), dim3(64), 0, st, j, e);
}

// The joins of two products whose sizes are counted on the device, in one launch.
template <class E>
__device__ __forceinline__ void join_as(Shape s, const Job& j, const E& e, int block, char* lds) {
  if (s == DIRECT) join<Direct>(j, e, block, lds);
  else if (s == BIG) join<Big>(j, e, block, lds);
  else if (s == SMALL) join<Small>(j, e, block, lds);
  else join<Thin>(j, e, block, lds);
}

template <class E>
__global__ __launch_bounds__(64) void join_two_kernel(Shape s, Job j, E e, int first, Shape s2, Job j2, E e2) {
  __shared__ __attribute__((aligned(1024))) char lds[JOIN_LDS];
  if ((int)blockIdx.x < first) join_as(s, j, e, blockIdx.x, lds);
  else join_as(s2, j2, e2, blockIdx.x - first, lds);
}

inline int64_t joins_of(Shape s, const Job& j) {
  return s == DIRECT  ? grids_as<Direct>(j).join
         : s == BIG   ? grids_as<Big>(j).join
         : s == SMALL ? grids_as<Small>(j).join
                      : grids_as<Thin>(j).join;
}

template <class E>
void launch_join_two(Shape s, const Job& j, const E& e, Shape s2, const Job& j2, const E& e2, hipStream_t st) {
  const int64_t first = joins_of(s, j), second = joins_of(s2, j2);
  if (first + second)
    hipLaunchKernelGGL((join_two_kernel<E>), dim3((unsigned)(first + second)), dim3(64), 0, st, s, j, e, (int)first, s2, j2,
                       e2);
}

inline bool misaligned(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

inline bool bad_stride(int64_t ld, int64_t c, int dtype) {
  return ld < c || ld > (int64_t)1 << 20 || ld % (dtype == DYRA_BF16 ? 8 : 4) != 0;
}

template <typename T>
Planes<T> planes(const T* in, int64_t ld, int64_t rows, int64_t cols, void* out, int64_t plane,
                 const int32_t* map = nullptr, const int32_t* live = nullptr) {
  return {in, ld, plane, reinterpret_cast<bf16_t*>(out), map, live, (int32_t)rows, (int32_t)cols};
}

template <typename T>
void launch_planes(const Planes<T>& a, const Planes<T>& b, hipStream_t st) {
  const int64_t na = cdiv((int64_t)a.rows * (a.cols / 8), 256), nb = cdiv((int64_t)b.rows * (b.cols / 8), 256);
  if (na + nb)
    hipLaunchKernelGGL((planes_kernel<T>), dim3((unsigned)(na + nb)), dim3(256), 0, st, a, b, (int)na);
}

}  // namespace
}  // namespace product
