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

struct Job {
  Operand a, b;        // a.rows x b.rows results
  int32_t kbytes;      // bytes of a row that count, a multiple of 16
  int32_t nk;          // k-steps of a term: ceil(kbytes / 128)
  int32_t terms;
  uint32_t pairs;
  int32_t tiles_m, tiles_n;
  int32_t split, per;  // the terms * nk steps in `split` parts of `per`
};

template <int BM_, int BN_, int NWM_, int NWN_, int NS_, int WGS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NS = NS_;
  static constexpr int NW = NWM * NWN, NT = NW * 64;
  static constexpr int WM = BM / NWM, WN = BN / NWN, FM = WM / 32, FN = WN / 32;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KB loads a wave and step
  static constexpr int SLOT = (BM + BN) * 128;
  static constexpr int LDS = NS * SLOT;
  static constexpr int WPE = WGS_ * NW / 4;                  // waves per SIMD with WGS_ workgroups on a CU
  static_assert(NW % 2 == 0, "a wave's row blocks have one parity, so one swizzle");
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN, "row blocks divide over the waves");
  static_assert(FM * 32 == WM && FN * 32 == WN, "a wave's part is made of 32 x 32 blocks");
};

// 256 x 256: 128 flop a byte loaded, one workgroup a CU (128 KB of LDS)
typedef Tile<256, 256, 2, 4, 2, 1> Big;
// 128 x 128: four times the tiles, two workgroups a CU
typedef Tile<128, 128, 2, 2, 2, 2> Small;
// 64 x 128: a few rows against a matrix that is read once; a deeper ring
typedef Tile<64, 128, 2, 2, 3, 2> Thin;

// Tile (tm, tn) and part z of a workgroup.  Consecutive numbers run on one
// XCD; they walk bands of four tile rows column by column, so that the 32
// workgroups of an XCD share four row blocks of A and eight of B in its L2.
__device__ __forceinline__ void place(const Job& j, int& tm, int& tn, int& z) {
  const int tiles = j.tiles_m * j.tiles_n;
  int t = xcd_tile_id(blockIdx.x, gridDim.x);
  z = t / tiles;
  t -= z * tiles;
  const int band = t / (4 * j.tiles_n), first = band * 4, high = min(4, j.tiles_m - first);
  t -= first * j.tiles_n;
  tn = t / high;
  tm = first + t - tn * high;
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

// The epilogue E is called once a tile as e(acc, lds, m0, n0, z, wm, wn): rows
// from m0 of A, from n0 of B; the whole ring is its to use.
template <class C, class E>
__global__ __launch_bounds__(C::NT, C::WPE) void product_kernel(Job j, E e) {
  __shared__ __attribute__((aligned(1024))) char ring[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / C::NWN, wn = w % C::NWN, l = lane & 31, g = lane >> 5;
  int tm, tn, z;
  place(j, tm, tn, z);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int total = j.terms * j.nk, first = z * j.per, steps = max(0, min(j.per, total - first));
  // row 8 w + lane / 8 of the wave's row block 0, 16-byte chunk (lane % 8) ^ (row / 2 % 8)
  const int row0 = 8 * w + (lane >> 3), ch = ((lane & 7) ^ ((row0 >> 1) & 7)) << 4;
  const int lda = (int)j.a.ld, ldb = (int)j.b.ld;
  constexpr int OUT = (int)0x80000000u;   // reads as zero
  int va[C::LA], vb[C::LB];
#pragma unroll
  for (int i = 0; i < C::LA; ++i) {
    const int r = row0 + 8 * C::NW * i;
    va[i] = m0 + r < j.a.rows ? r * lda + ch : OUT;
  }
#pragma unroll
  for (int i = 0; i < C::LB; ++i) {
    const int r = row0 + 8 * C::NW * i;
    vb[i] = n0 + r < j.b.rows ? r * ldb + ch : OUT;
  }
  const uint32_t base = lds_addr(ring) + w * 1024;
  int term = first / j.nk, kt = first - term * j.nk, left = steps;
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
    if (left > 0 && kb + 128 <= j.kbytes) {
      static_for<0, C::LA>([&](auto i) __attribute__((always_inline)) {
        dma16k<decltype(i)::value * C::NW * 1024>(ra, va[decltype(i)::value], kb, to);
      });
      static_for<0, C::LB>([&](auto i) __attribute__((always_inline)) {
        dma16k<C::BM * 128 + decltype(i)::value * C::NW * 1024>(rb, vb[decltype(i)::value], kb, to);
      });
    } else {
      const bool in = left > 0 && ch < j.kbytes - kb;
      static_for<0, C::LA>([&](auto i) __attribute__((always_inline)) {
        dma16k<decltype(i)::value * C::NW * 1024>(ra, in ? va[decltype(i)::value] : OUT, kb, to);
      });
      static_for<0, C::LB>([&](auto i) __attribute__((always_inline)) {
        dma16k<C::BM * 128 + decltype(i)::value * C::NW * 1024>(rb, in ? vb[decltype(i)::value] : OUT, kb, to);
      });
    }
    if (--left > 0 && ++kt == j.nk) {
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
  uint32_t in = 0, out = 0;
#pragma unroll
  for (int s = 0; s < C::NS - 1; ++s) {
    issue(in);
    in += C::SLOT;
  }
  for (int t = 0; t < steps; ++t) {
    wait_vm_lgkm0<(C::NS - 2) * (C::LA + C::LB)>();   // this wave's loads of step t have landed
    bare_barrier();                                    // everyone's; the slot of step t - 1 is free
    issue(in);
    in = in + C::SLOT == C::LDS ? 0 : in + C::SLOT;
    multiply<C>(ring + out, acc, wm, wn, l, g);
    out = out + C::SLOT == C::LDS ? 0 : out + C::SLOT;
  }
  wait_vm_lgkm0<0>();
  bare_barrier();   // no load is under way, no slot is read: the ring is the epilogue's
  e.template operator()<C>(acc, ring, m0, n0, z, wm, wn);
}

// ---------------------------------------------------------------------------
// epilogue: the tile to memory
// ---------------------------------------------------------------------------

// out[z][row][col] (rows ld elements apart) = acc + bias[col], or += for
// `add`.  A wave takes 32 rows at a time through its part of the ring, so that
// every store covers whole 128-byte lines.
template <typename T>
struct Store {
  T* out;
  int64_t ld, slice;      // elements between rows, between parts
  int32_t rows, cols;     // cols a multiple of 8
  const T* bias;
  int32_t add;

  template <class C>
  __device__ __forceinline__ void operator()(const Acc<C>& acc, char* lds, int m0, int n0, int z, int wm, int wn) const {
    constexpr int E = 16 / sizeof(T), CPR = C::WN / E;   // elements a chunk, chunks a staged row
    static_assert(C::NW * 32 * C::WN * (int)sizeof(T) <= C::LDS, "staging fits the ring");
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    char* mine = lds + (wm * C::NWN + wn) * (32 * CPR * 16);
    const int c0 = n0 + wn * C::WN;
    T* to = out + z * slice;
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = fn * 32 + 8 * q + 4 * g;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[fm][fn][4 * q + e];
          if (bias && c0 + col < cols) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += TT<T>::to_f(bias[c0 + col + e]);
          }
          char* at = mine + l * (CPR * 16) + stage_chunk<CPR>(l, col / E) * 16;
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(at + (col & 4) * 2) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          else *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 32 * CPR / 64; ++i) {
        const int c = lane + i * 64, rr = c / CPR, k = c % CPR;
        uint4 v = *reinterpret_cast<const uint4*>(mine + rr * (CPR * 16) + stage_chunk<CPR>(rr, k) * 16);
        const int row = m0 + wm * C::WM + fm * 32 + rr, col = c0 + k * E;
        if (row < rows && col < cols) {
          uint4* p = reinterpret_cast<uint4*>(to + row * ld + col);
          if constexpr (sizeof(T) == 4) {
            if (add) {
              const uint4 o = *p;
              v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(o.x));
              v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(o.y));
              v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(o.z));
              v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(o.w));
            }
          }
          *p = v;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
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

// A matrix [rows][cols] as bf16 planes, row by row and transposed (rows padded
// with zeros to ldt there); rows whose target is none of the vocabulary's are
// zero in the transposed form, whatever they hold.
template <typename T>
struct Planes {
  const T* in;
  int64_t ld;
  bf16_t *out, *outt;   // null: not wanted
  int64_t ldo, ldt, plane, plane_t;
  const int32_t* targets;   // or null
  int32_t rows, cols, vocab;
};

template <typename T>
__global__ __launch_bounds__(256) void planes_kernel(Planes<T> a, int blocks_c) {
  constexpr int NP = planes_of<T>(), E = 8, PER = 128 * 16 / 256;   // 8-element chunks a thread
  __shared__ __attribute__((aligned(1024))) char lds[128 * 256];
  const int r0 = blockIdx.x / blocks_c * 128, c0 = blockIdx.x % blocks_c * 128;
  float v[PER][E];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = threadIdx.x + i * 256, row = r0 + c / 16, col = c0 + c % 16 * 8;
#pragma unroll
    for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    if (row < a.rows && col < a.cols) {
      const T* p = a.in + row * a.ld + col;
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
      uint4 x = make_uint4(h[0], h[1], h[2], h[3]);
      if (a.out && row < a.rows && col < a.cols)
        *reinterpret_cast<uint4*>(a.out + t * a.plane + row * a.ldo + col) = x;
      if (a.targets && row < a.rows && (a.targets[row] < 0 || a.targets[row] >= a.vocab)) x = zero4();
      if (a.outt) *reinterpret_cast<uint4*>(lds + tile_at(rr, c % 16, 16)) = x;
    }
    if (!a.outt) continue;
    __syncthreads();
    tile_transposed<128, 128, 256>(lds, a.outt + t * a.plane_t + (int64_t)c0 * a.ldt + r0, a.ldt,
                                   min(128, (int)a.ldt - r0), min(128, a.cols - c0));
  }
}

// out = the sum of the parts (+ bias), rounded once.
template <typename T>
__global__ __launch_bounds__(256) void parts_kernel(const float* __restrict__ part, int64_t slice, int parts,
                                                    T* __restrict__ out, int64_t ld, int64_t rows, int cols,
                                                    const T* __restrict__ bias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = cols / 4;
  const int64_t row = i / quads;
  const int col = (int)(i - row * quads) * 4;
  if (row >= rows) return;
  float4 s = *reinterpret_cast<const float4*>(part + row * cols + col);
  for (int p = 1; p < parts; ++p) {
    const float4 v = *reinterpret_cast<const float4*>(part + p * slice + row * cols + col);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  if (bias) s.x += TT<T>::to_f(bias[col]), s.y += TT<T>::to_f(bias[col + 1]), s.z += TT<T>::to_f(bias[col + 2]),
            s.w += TT<T>::to_f(bias[col + 3]);
  T* o = out + row * ld + col;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  else *reinterpret_cast<float4*>(o) = s;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Job job(Operand a, Operand b, int64_t K, int terms, uint32_t pairs) {
  Job j{};
  j.a = a;
  j.b = b;
  j.kbytes = (int32_t)(2 * K);
  j.nk = (int32_t)cdiv(2 * K, 128);
  j.terms = terms;
  j.pairs = pairs;
  return j;
}

template <class C, class E>
inline void launch(Job j, int split, const E& e, hipStream_t st) {
  j.tiles_m = (int32_t)cdiv(j.a.rows, C::BM);
  j.tiles_n = (int32_t)cdiv(j.b.rows, C::BN);
  j.split = split;
  j.per = (int32_t)cdiv((int64_t)j.terms * j.nk, split);
  const int64_t grid = (int64_t)j.tiles_m * j.tiles_n * split;
  if (grid) hipLaunchKernelGGL((product_kernel<C, E>), dim3((unsigned)grid), dim3(C::NT), 0, st, j, e);
}

inline size_t align256(int64_t b) { return ((size_t)b + 255) & ~(size_t)255; }
inline int64_t up(int64_t a, int64_t m) { return cdiv(a, m) * m; }

enum Shape { BIG, SMALL, THIN };

// The tile of a product of m x n results over `steps` k-steps, and into how
// many parts its steps are split (1 where only whole sums will do).
struct Pick {
  Shape shape;
  int split;
};

inline Pick pick(int64_t m, int64_t n, int64_t steps, bool may_split) {
  if (m <= 64) {
    const int64_t tiles = cdiv(n, 128);
    const int64_t s = may_split ? std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(1, tiles), steps / 8)) : 1;
    return {THIN, (int)std::min<int64_t>(s, 16)};
  }
  const int64_t big = cdiv(m, 256) * cdiv(n, 256), small = cdiv(m, 128) * cdiv(n, 128);
  if (big >= 200) return {BIG, 1};
  const int64_t s = may_split ? std::max<int64_t>(1, std::min<int64_t>(cdiv(384, small), steps / 8)) : 1;
  return {SMALL, (int)std::min<int64_t>(s, 16)};
}

template <class E>
void launch_as(const Pick& p, const Job& j, const E& e, hipStream_t st) {
  if (p.shape == BIG) launch<Big>(j, p.split, e, st);
  else if (p.shape == SMALL) launch<Small>(j, p.split, e, st);
  else launch<Thin>(j, p.split, e, st);
}

inline int64_t tile_cols(Shape s) { return s == BIG ? Big::BN : Small::BN; }

inline bool misaligned(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

inline bool bad_stride(int64_t ld, int64_t c, int dtype) {
  return ld < c || ld > (int64_t)1 << 20 || ld % (dtype == DYRA_BF16 ? 8 : 4) != 0;
}

template <typename T>
void launch_planes(const T* in, int64_t ld, int64_t rows, int64_t cols, bf16_t* out, bf16_t* outt, int64_t ldt,
                   int64_t plane, int64_t plane_t, const int32_t* targets, int64_t vocab, hipStream_t st) {
  const int64_t padded = outt ? ldt : rows;
  const Planes<T> a{in, ld, out, outt, cols, ldt, plane, plane_t, targets, (int32_t)rows, (int32_t)cols, (int32_t)vocab};
  const int64_t bc = cdiv(cols, 128), grid = cdiv(padded, 128) * bc;
  hipLaunchKernelGGL((planes_kernel<T>), dim3((unsigned)grid), dim3(256), 0, st, a, (int)bc);
}

}  // namespace
}  // namespace product
