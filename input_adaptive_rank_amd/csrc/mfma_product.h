// Matrix products C = sum_t A_t B_t^T on bf16 MFMAs, with the caller's own
// epilogue, for the 4-bit projection and the vocabulary loss.
//
// Both operands lie with the reduction axis contiguous ("rows" of K elements)
// and come in one or more planes: an fp32 operand is held as bf16 planes
// hi + mid + lo (24 bits), and the product as the sum of the plane pairs
// ("terms") whose size reaches the result's precision.  All terms of a tile
// run through one accumulator.
//
// A workgroup computes a BM x BN tile.  Every wave loads its part of each
// 64-element k-step straight into an NS-slot LDS ring (1 KB a wave
// instruction, rows of 128 bytes swizzled as lds_off does) NS - 1 steps ahead,
// and multiplies its WM x WN part of the tile; one barrier a step hands a
// landed slot over and a used one back.
#pragma once

#include <algorithm>

#include "../../include/dyra.h"
#include "lds_dma.h"

namespace product {
namespace {   // kernels made in one source file are not another's

// Rows of K elements; row r of plane t at p + t * plane + r * ld (bytes).
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
  int32_t nk, terms;
  uint32_t pairs;
  int32_t may_split, live_k;
  const int32_t* live;
  float4* part;        // partial tiles, if may_split (part_bytes)
};

// STEP: tenths of a microsecond that a k-step takes with the card full.
template <int BM_, int BN_, int NWM_, int NWN_, int NS_, int WGS_, int STEP_>
struct Tile {
  static constexpr int STEP = STEP_;
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NS = NS_;
  static constexpr int NW = NWM * NWN, NT = NW * 64;
  static constexpr int WM = BM / NWM, WN = BN / NWN, FM = WM / 32, FN = WN / 32;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KB loads a wave and step
  static constexpr int SLOT = (BM + BN) * 128;
  static constexpr int LDS = NS * SLOT;
  static constexpr int WPE = WGS_ * NW / 4;                  // waves per SIMD with WGS_ workgroups on a CU
  static constexpr int SLOTS = 256 * WGS_;                   // workgroups on the card at once
  static constexpr int QUADS = FM * FN * 4;                  // groups of four results a lane
  static_assert(NW % 2 == 0, "a wave's row blocks have one parity, so one swizzle");
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN, "row blocks divide over the waves");
  static_assert(FM * 32 == WM && WN == 64, "a wave's part is made of 32 x 64 blocks");
};

// 256 x 256: 128 flop a byte loaded, one workgroup a CU (128 KB of LDS); 1.27
// PFLOP/s in whole rounds
typedef Tile<256, 256, 2, 4, 2, 1, 17> Big;
// 128 x 128: four times the tiles, two workgroups a CU
typedef Tile<128, 128, 2, 2, 2, 2, 11> Small;
// 64 x 128: a few rows against a matrix that is read once; a deeper ring
typedef Tile<64, 128, 2, 2, 3, 2, 6> Thin;

// How a product's tiles are laid over the workgroups.  The card holds SLOTS of
// them at once: whole rounds of tiles are computed by one workgroup each.  The
// tiles of a last round that would leave much of the card idle are split along
// the reduction, if that saves more than the join costs (272 tiles of 192 steps:
// 434 us instead of 568).  Product and join work it out from the sizes that
// they find.
struct Layout {
  int rows, tiles_m, tiles_n, kbytes, nk;
  int whole, tail, split, per;   // tiles computed whole, tiles split, parts of one, steps of a part
  int count;                     // workgroups
  double cost;                   // tenths of a microsecond, estimated
};

template <class C>
__host__ __device__ inline Layout layout(const Job& j, int live) {
  Layout y;
  y.rows = j.a.rows;
  y.kbytes = j.kbytes;
  y.nk = j.nk;
  if (live >= 0) {
    if (j.live_k) {
      y.nk = (live + 63) / 64;
      y.nk = y.nk < j.nk ? y.nk : j.nk;
      y.kbytes = y.nk * 128;
    } else {
      y.rows = live < y.rows ? live : y.rows;
    }
  }
  y.tiles_m = (y.rows + C::BM - 1) / C::BM;
  y.tiles_n = (j.b.rows + C::BN - 1) / C::BN;
  const int tiles = y.tiles_m * y.tiles_n, steps = j.terms * y.nk, rest = tiles % C::SLOTS;
  int split = 1, least = rest ? steps * C::STEP : 0;
  if (j.may_split && rest) {
    for (int s = 2; s <= 16 && s * 4 <= steps && rest * s <= 2 * C::SLOTS; ++s) {   // at least four steps a part
      // the rounds of the parts, their way through memory at 5 TB/s, a launch
      const int cost = (rest * s + C::SLOTS - 1) / C::SLOTS * ((steps + s - 1) / s) * C::STEP +
                       rest * s * (C::BM * C::BN / 1024) / 61 + 60;
      if (cost < least) {
        least = cost;
        split = s;
      }
    }
  }
  y.split = split;
  y.tail = split > 1 ? rest : 0;
  y.whole = tiles - y.tail;
  y.per = (steps + split - 1) / split;
  y.count = y.whole + y.tail * split;
  y.cost = (double)(tiles / C::SLOTS) * steps * C::STEP + least;
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

// acc += one k-step of a slot.  Lane (l, g) reads chunk 2 s + g of rows l + 32 f
// of its part; sub-step s + 1 is read while s multiplies.  The operands are
// swapped, so that lane (l, g) ends with row l of A and, in element 4 q + e,
// column 8 q + 4 g + e of B.
template <class C>
__device__ __forceinline__ void multiply(const char* slot, Acc<C>& acc, int wm, int wn, int l, int g) {
  const char* as = slot + (wm * C::WM + l) * 128;
  const char* bs = slot + C::BM * 128 + (wn * C::WN + l) * 128;
  const int h = (l >> 1) & 7;
  uint4 af[2][C::FM], bf[2][C::FN];
  auto load = [&](int s) __attribute__((always_inline)) {
    const int at = (((2 * s + g) ^ h) & 7) << 4;
#pragma unroll
    for (int f = 0; f < C::FM; ++f) af[s & 1][f] = *reinterpret_cast<const uint4*>(as + f * 4096 + at);
#pragma unroll
    for (int f = 0; f < C::FN; ++f) bf[s & 1][f] = *reinterpret_cast<const uint4*>(bs + f * 4096 + at);
  };
  load(0);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s < 3) load(s + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) TT<bf16_t>::mma(acc[fm][fn], bf[s & 1][fn], af[s & 1][fm]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Epilogues: e.tile<C>(acc, lds, m0, n0, rows, wm, wn) takes a whole tile (the
// ring is its to use), e.block<C>(v, lds, row0, col0, rows) 32 x WN results of
// one wave, which has 32 * WN floats of LDS.
template <class C, class E>
__global__ __launch_bounds__(C::NT, C::WPE) void product_kernel(Job j, E e) {
  __shared__ __attribute__((aligned(1024))) char ring[C::LDS];
  const Layout y = layout<C>(j, j.live ? *j.live : -1);
  if ((int)blockIdx.x >= y.count) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / C::NWN, wn = w % C::NWN, l = lane & 31, g = lane >> 5;
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
  // row 8 w + lane / 8 of the wave's row block 0, 16-byte chunk (lane % 8) ^ (row / 2 % 8)
  const int row0 = 8 * w + (lane >> 3), ch = ((lane & 7) ^ ((row0 >> 1) & 7)) << 4;
  const int lda = (int)j.a.ld, ldb = (int)j.b.ld;
  constexpr int OUT = (int)0x80000000u;   // reads as zero
  int va[C::LA], vb[C::LB];
#pragma unroll
  for (int i = 0; i < C::LA; ++i) {
    const int r = row0 + 8 * C::NW * i;
    va[i] = m0 + r < y.rows ? r * lda + ch : OUT;
  }
#pragma unroll
  for (int i = 0; i < C::LB; ++i) {
    const int r = row0 + 8 * C::NW * i;
    vb[i] = n0 + r < j.b.rows ? r * ldb + ch : OUT;
  }
  const uint32_t base = lds_addr(ring) + w * 1024;
  int term = y.nk ? first / y.nk : 0, kt = first - term * y.nk, left = steps;
  i32x4v ra, rb;
  auto aim = [&]() __attribute__((always_inline)) {
    const uint32_t pr = j.pairs >> (4 * term);
    ra = rsrc_words(reinterpret_cast<const char*>(j.a.p) + (int64_t)m0 * j.a.ld + (pr & 3) * j.a.plane, 0x7fffffffu);
    rb = rsrc_words(reinterpret_cast<const char*>(j.b.p) + (int64_t)n0 * j.b.ld + (pr >> 2 & 3) * j.b.plane,
                    0x7fffffffu);
  };
  aim();
  // one k-step into a slot; past the last every lane reads out of range, so
  // that each step issues the same number of loads
  auto issue = [&](uint32_t slot) __attribute__((always_inline)) {
    const int kb = kt * 128;
    const uint32_t to = base + slot;
    if (left > 0 && kb + 128 <= y.kbytes) {
      static_for<0, C::LA>([&](auto i) __attribute__((always_inline)) {
        dma16k<decltype(i)::value * C::NW * 1024>(ra, va[decltype(i)::value], kb, to);
      });
      static_for<0, C::LB>([&](auto i) __attribute__((always_inline)) {
        dma16k<C::BM * 128 + decltype(i)::value * C::NW * 1024>(rb, vb[decltype(i)::value], kb, to);
      });
    } else {
      const bool in = left > 0 && ch < y.kbytes - kb;
      static_for<0, C::LA>([&](auto i) __attribute__((always_inline)) {
        dma16k<decltype(i)::value * C::NW * 1024>(ra, in ? va[decltype(i)::value] : OUT, kb, to);
      });
      static_for<0, C::LB>([&](auto i) __attribute__((always_inline)) {
        dma16k<C::BM * 128 + decltype(i)::value * C::NW * 1024>(rb, in ? vb[decltype(i)::value] : OUT, kb, to);
      });
    }
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
  uint32_t in = 0, out = 0;
#pragma unroll
  for (int s = 0; s < C::NS - 1; ++s) {
    issue(in);
    in += C::SLOT;
  }
  auto walk = [&](auto multiplies) __attribute__((always_inline)) {
    for (int t = 0; t < steps; ++t) {
      wait_vm_lgkm0<(C::NS - 2) * (C::LA + C::LB)>();   // this wave's loads of step t have landed
      bare_barrier();                                    // everyone's; the slot of step t - 1 is free
      issue(in);
      in = in + C::SLOT == C::LDS ? 0 : in + C::SLOT;
      if constexpr (decltype(multiplies)::value) multiply<C>(ring + out, acc, wm, wn, l, g);
      out = out + C::SLOT == C::LDS ? 0 : out + C::SLOT;
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
  float4* to = j.part + ((int64_t)part * C::NW + w) * C::QUADS * 64 + lane;
#pragma unroll
  for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        to[((fm * C::FN + fn) * 4 + q) * 64] = make_float4(acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1],
                                                           acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3]);
}

// Adds the parts of the split tiles, in their order; one wave for 32 x WN results.
template <class C, class E>
__global__ __launch_bounds__(64) void join_kernel(Job j, E e) {
  __shared__ __attribute__((aligned(1024))) char lds[32 * C::WN * 4];
  const Layout y = layout<C>(j, j.live ? *j.live : -1);
  const int tail = blockIdx.x / (C::NW * C::FM), sub = blockIdx.x - tail * (C::NW * C::FM);
  if (tail >= y.tail) return;
  const int w = sub / C::FM, fm = sub - w * C::FM;
  int m0, n0;
  corner<C>(y, y.whole + tail, m0, n0);
  const int row0 = m0 + w / C::NWN * C::WM + fm * 32, col0 = n0 + w % C::NWN * C::WN;
  if (row0 >= ((y.rows + 63) & ~63) || col0 >= j.b.rows) return;   // rows up to 64 more may be padding
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

// ---------------------------------------------------------------------------
// epilogue: the tile to memory
// ---------------------------------------------------------------------------

// out[row][col] (rows ld elements apart) = acc + bias[col] + prior[row][col].
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

  template <class C>
  __device__ __forceinline__ void block(const f32x16 (&v)[C::FN], char* lds, int row0, int col0, int rows) const {
    constexpr int E = 16 / sizeof(T), CPR = C::WN / E;   // elements a chunk, chunks a staged row
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    const bool old = prior && row0 + l < rows;
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = fn * 32 + 8 * q + 4 * g;
        float x[4] = {v[fn][4 * q], v[fn][4 * q + 1], v[fn][4 * q + 2], v[fn][4 * q + 3]};
        if (bias && col0 + col < cols) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += TT<T>::to_f(bias[col0 + col + e]);
        }
        if (old && col0 + col < cols) {
          const float4 o = *reinterpret_cast<const float4*>(prior + (int64_t)(row0 + l) * cols + col0 + col);
          x[0] += o.x, x[1] += o.y, x[2] += o.z, x[3] += o.w;
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
// a bf16 tile in LDS, row by row or transposed to memory
// ---------------------------------------------------------------------------

// 16-byte chunk of a tile whose rows hold a multiple of 16 chunks.  Sixteen
// neighbouring rows, and sixteen rows eight apart (a transposing read), lie in
// sixteen different places of the 256-byte bank window.
__device__ __forceinline__ int tile_at(int row, int chunk, int chunks) {
  return (row * chunks + (chunk ^ ((row ^ (row >> 3)) & 15))) * 16;
}

// rows x cols of the tile (each a multiple of 8 at most ROWS, COLS) to out[row][col]
template <int ROWS, int COLS, int NT>
__device__ __forceinline__ void tile_rows(const char* lds, bf16_t* out, int64_t ld, int rows, int cols) {
  constexpr int CPR = COLS / 8;
  for (int c = threadIdx.x; c < ROWS * CPR; c += NT) {
    const int row = c / CPR, k = c % CPR;
    if (row < rows && k * 8 < cols)
      *reinterpret_cast<uint4*>(out + row * ld + k * 8) = *reinterpret_cast<const uint4*>(lds + tile_at(row, k, CPR));
  }
}

// ... to out[col][row]: a thread turns 8 x 8 elements, neighbouring lanes the
// next eight rows
template <int ROWS, int COLS, int NT>
__device__ __forceinline__ void tile_transposed(const char* lds, bf16_t* out, int64_t ld, int rows, int cols) {
  constexpr int CPR = COLS / 8, RB = ROWS / 8;
  for (int c = threadIdx.x; c < RB * CPR; c += NT) {
    const int r0 = c % RB * 8, k = c / RB;
    if (r0 < rows && k * 8 < cols) {
      uint4 in[8], t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = *reinterpret_cast<const uint4*>(lds + tile_at(r0 + e, k, CPR));
      transpose8x8_b16(in, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(out + (int64_t)(k * 8 + e) * ld + r0) = t[e];
    }
  }
}

// ---------------------------------------------------------------------------
// operands and results beside a product
// ---------------------------------------------------------------------------

// planes of an operand of type T
template <typename T> constexpr int planes_of() { return sizeof(T) == 2 ? 1 : 3; }

// A matrix [rows][cols] as bf16 planes, row by row and transposed (there padded
// with zeros to ldt rows).  map: only its rows map[0 .. *live - 1].
template <typename T>
struct Planes {
  const T* in;
  int64_t ld;
  bf16_t *out, *outt;   // null: not wanted
  int64_t ldo, ldt, plane, plane_t;
  const int32_t *map, *live;   // or null
  int32_t rows, cols;
};

template <typename T>
__global__ __launch_bounds__(256) void planes_kernel(Planes<T> a, int blocks_c) {
  constexpr int NP = planes_of<T>(), E = 8, PER = 128 * 16 / 256;   // 8-element chunks a thread
  __shared__ __attribute__((aligned(1024))) char lds[128 * 256];
  const int r0 = blockIdx.x / blocks_c * 128, c0 = blockIdx.x % blocks_c * 128;
  const int rows = a.live ? min(*a.live, a.rows) : a.rows;
  const int padded = min((rows + 63) & ~63, (int)a.ldt);   // transposed rows that are read
  if (r0 >= max(rows, a.outt ? padded : 0)) return;
  float v[PER][E];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = threadIdx.x + i * 256, row = r0 + c / 16, col = c0 + c % 16 * 8;
#pragma unroll
    for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    if (row < rows && col < a.cols) {
      const T* p = a.in + (a.map ? a.map[row] : row) * a.ld + col;
      if constexpr (sizeof(T) == 2) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[i][2 * e] = __uint_as_float(q[e] << 16);
          v[i][2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
        }
      } else {
        const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        v[i][4] = y.x, v[i][5] = y.y, v[i][6] = y.z, v[i][7] = y.w;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NP; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = threadIdx.x + i * 256, rr = c / 16, row = r0 + rr, col = c0 + c % 16 * 8;
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = pack_bf16x2(v[i][2 * e], v[i][2 * e + 1]);
        v[i][2 * e] -= __uint_as_float(h[e] << 16);
        v[i][2 * e + 1] -= __uint_as_float(h[e] & 0xffff0000u);
      }
      const uint4 x = make_uint4(h[0], h[1], h[2], h[3]);
      if (a.out && row < rows && col < a.cols)
        *reinterpret_cast<uint4*>(a.out + t * a.plane + row * a.ldo + col) = x;
      if (a.outt) *reinterpret_cast<uint4*>(lds + tile_at(rr, c % 16, 16)) = x;
    }
    if (!a.outt) continue;
    __syncthreads();
    tile_transposed<128, 128, 256>(lds, a.outt + t * a.plane_t + (int64_t)c0 * a.ldt + r0, a.ldt,
                                   min(128, padded - r0), min(128, a.cols - c0));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// live: what the rows of A (live_k: the reduction) are found to be, or null.
inline Job job(Operand a, Operand b, int64_t K, int terms, uint32_t pairs, const int32_t* live = nullptr,
               bool live_k = false) {
  Job j{};
  j.a = a;
  j.b = b;
  j.kbytes = (int32_t)(2 * K);
  j.nk = (int32_t)cdiv(2 * K, 128);
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
enum Shape { BIG, SMALL, THIN };

inline Shape shape_of(const Job& j, bool may_be_big = true) {
  if (j.a.rows <= 64) return THIN;
  return may_be_big && layout<Big>(j, -1).cost <= layout<Small>(j, -1).cost ? BIG : SMALL;
}

// Estimated microseconds of a product.
inline double cost(Shape s, const Job& j) {
  return 0.1 * (s == BIG ? layout<Big>(j, -1).cost : s == SMALL ? layout<Small>(j, -1).cost : layout<Thin>(j, -1).cost);
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
  return s == BIG ? part_bytes_as<Big>(j) : s == SMALL ? part_bytes_as<Small>(j) : part_bytes_as<Thin>(j);
}

template <class C, class E>
inline void launch(const Job& j, const E& e, hipStream_t st) {
  const Layout y = layout<C>(j, -1);
  // fewer live rows or steps may leave another number of tiles to split, into 2 SLOTS parts at most
  const int64_t grid = j.live ? (int64_t)y.tiles_m * y.tiles_n + (j.may_split ? 2 * C::SLOTS : 0) : y.count;
  if (!grid) return;
  hipLaunchKernelGGL((product_kernel<C, E>), dim3((unsigned)grid), dim3(C::NT), 0, st, j, e);
  const int64_t tail = j.live ? (j.may_split ? std::min(C::SLOTS, y.tiles_m * y.tiles_n) : 0) : y.tail;
  if (tail)
    hipLaunchKernelGGL((join_kernel<C, E>), dim3((unsigned)(tail * C::NW * C::FM)), dim3(64), 0, st, j, e);
}

template <bool MAY_BE_BIG = true, class E>
void launch_as(Shape s, const Job& j, const E& e, hipStream_t st) {
  if (MAY_BE_BIG && s == BIG) {
    if constexpr (MAY_BE_BIG) launch<Big>(j, e, st);
  } else if (s == SMALL) launch<Small>(j, e, st);
  else launch<Thin>(j, e, st);
}

inline bool misaligned(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

inline bool bad_stride(int64_t ld, int64_t c, int dtype) {
  return ld < c || ld > (int64_t)1 << 20 || ld % (dtype == DYRA_BF16 ? 8 : 4) != 0;
}

template <typename T>
void launch_planes(const T* in, int64_t ld, int64_t rows, int64_t cols, bf16_t* out, bf16_t* outt, int64_t ldt,
                   int64_t plane, int64_t plane_t, const int32_t* map, const int32_t* live, hipStream_t st) {
  const int64_t padded = outt ? ldt : rows;
  const Planes<T> a{in, ld, out, outt, cols, ldt, plane, plane_t, map, live, (int32_t)rows, (int32_t)cols};
  const int64_t bc = cdiv(cols, 128), grid = cdiv(padded, 128) * bc;
  hipLaunchKernelGGL((planes_kernel<T>), dim3((unsigned)grid), dim3(256), 0, st, a, (int)bc);
}

}  // namespace
}  // namespace product
