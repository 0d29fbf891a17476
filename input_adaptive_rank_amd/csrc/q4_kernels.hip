// Projections with 4-bit weights: w = scale (code - zero), one scale and zero
// point for each row's group of 32, 64 or 128 columns.
//   forward   Y = X W^T + bias        W [c2][c1]
//   backward  dX = dY W               (the weight is frozen)
//
// Packed weight.  Codes lie in blocks of 16 rows x 128 columns, 1 KB in the
// order in which the lanes of a wave read them as 16-column operands of
// v_mfma_f32_16x16x32_bf16: lane (j, g) holds columns 32 s + 8 g + 0 .. 7 of
// row j in its word s = 0 .. 3, the even columns in the low half.  A pair of
// codes then becomes a pair of bf16 numbers 16 + code with one shift and one
// and-or: 0x4180 is 16, whose upper four mantissa bits are worth 1 to 8.
// Parameters lie as [block of 16 rows][group][16] words, the bf16 scale above the
// bf16 number 128 + zero.
//
// Few rows: each wave multiplies whole blocks of codes, in exact products,
//   sum_k x (16 + code) - (16 + zero) sum_k x,
// the last sum from one more product with ones, and scales each group's sum.  What
// is added and taken off again costs bits: 16 is the least number that an and-or
// can add.  With 128 (a shift of eight less, 1 % at 48 rows) a column of 2^19 that
// every weight meets with 0 moved results by whole units.
// Many rows: W is written out once as bf16 (rounded: at most 2^-8 of a weight, like
// the rounding of the result) and multiplied tile by tile, for the backward pass
// turned on its way; for fp32 operands as two bf16 planes, which hold it exactly (8
// bits of scale times 5).
//
// 4096 -> 4096, group 128: one row 4.5 us (7 with the call), 5003 rows 141 (a product
// at 1.3 PFLOP/s alone 129).  (Times vary by 7 % with the card.)
#include "mfma_product.h"

namespace {

using namespace product;

constexpr int ROW_WAVES = 8;      // waves of a few-row workgroup

struct Weight {
  const uint4* codes;     // [row blocks][column blocks][64]
  const uint32_t* params; // [row blocks][column blocks * groups a block][16]
  int32_t c1, c2, kt;     // kt: column blocks
};

__device__ __forceinline__ float scale_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ float zero_of(uint32_t p) { return __uint_as_float(p << 16) - 112.f; }   // 16 + zero

// 16 + code of a word's eight columns, as bf16.  The constants are held in
// registers, where one v_and_or_b32 can take them both.
__device__ __forceinline__ uint4 widen(uint32_t w) {
  uint32_t mask = 0x00780078u, bias = 0x41804180u;
  asm("" : "+v"(mask));
  asm("" : "+s"(bias));
  return make_uint4((w << 3 & mask) | bias, (w >> 1 & mask) | bias, (w >> 5 & mask) | bias, (w >> 9 & mask) | bias);
}

// code - zero of a word's eight columns, as bf16 (whole numbers below 16: exact).
__device__ __forceinline__ uint4 centre(uint32_t w, float zero) {
  const uint4 v = widen(w);
  auto two = [&](uint32_t p) {
    return pack_bf16x2(__uint_as_float(p << 16) - zero, __uint_as_float(p & 0xffff0000u) - zero);
  };
  return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

struct RowsArgs {
  Weight w;
  const void* X;
  const void* bias;
  void* Y;
  int64_t ldx, ldy;
  int32_t n;
};

// The waves' sums of RT x OB blocks, added in their order, to Y.  Row i, column
// col of a block lie in lane col + 16 (i / 4), register i % 4.
template <typename T, int RT, int OB>
__device__ __forceinline__ void store_sums(const RowsArgs& a, const float* red, int cb0, int t0) {
  const T* bias = reinterpret_cast<const T*>(a.bias);
  for (int u = threadIdx.x; u < RT * OB * 256; u += ROW_WAVES * 64) {
    const int i = u / (16 * OB), col = u % (16 * OB), row = t0 + i, o = cb0 * 16 + col;
    if (row >= a.n || o >= a.w.c2) continue;
    const int at = ((i >> 4) * OB + (col >> 4)) * 256 + ((col & 15) + 16 * (i >> 2 & 3)) * 4 + (i & 3);
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < ROW_WAVES; ++k) v += red[k * RT * OB * 256 + at];
    if (bias) v += TT<T>::to_f(bias[o]);
    reinterpret_cast<T*>(a.Y)[row * a.ldy + o] = TT<T>::from_f(v);
  }
}

// fp32: OB blocks of 16 rows of W (columns of Y) by RT blocks of 16 rows of X a
// workgroup, the column blocks of both dealt to its waves in turn; GPB groups a
// column block.  X enters as three bf16 terms, which the whole numbers code -
// zero multiply exactly; splitting it is what costs (4096 -> 4096, 32 rows: 18
// us), so that two blocks of W share it where there are workgroups enough.
template <int RT, int OB, int GPB>
__global__ __launch_bounds__(ROW_WAVES * 64) void rows_f32_kernel(RowsArgs a) {
  __shared__ float red[ROW_WAVES][RT * OB * 256];
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb0 = blockIdx.x * OB, t0 = blockIdx.y * RT * 16, kt = a.w.kt, c1 = a.w.c1;
  const int blocks = (a.w.c2 + 15) / 16;
  const float* X = reinterpret_cast<const float*>(a.X);
  f32x4 sum[OB][RT];
#pragma unroll
  for (int o = 0; o < OB; ++o)
#pragma unroll
    for (int r = 0; r < RT; ++r) sum[o][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int b = w; b < kt; b += ROW_WAVES) {
    uint4 q[OB];
    uint32_t p[OB][GPB];
#pragma unroll
    for (int o = 0; o < OB; ++o) {
      const int64_t at = (int64_t)min(cb0 + o, blocks - 1) * kt + b;   // past the last: not stored
      q[o] = a.w.codes[at * 64 + lane];
#pragma unroll
      for (int i = 0; i < GPB; ++i) p[o][i] = a.w.params[(at * GPB + i) * 16 + j];
    }
    float4 x[RT][4][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int row = t0 + 16 * r + j, k = b * 128 + 32 * s + 8 * g;
        const bool in = row < a.n && k < c1;
        const float4* at = reinterpret_cast<const float4*>(X + row * a.ldx + k);
#pragma unroll
        for (int h = 0; h < 2; ++h) x[r][s][h] = in ? at[h] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
    for (int i = 0; i < GPB; ++i) {
      f32x4 acc[OB][RT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int o = 0; o < OB; ++o) acc[o][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = i * 4 / GPB; s < (i + 1) * 4 / GPB; ++s) {
        uint4 wq[OB];
#pragma unroll
        for (int o = 0; o < OB; ++o)
          wq[o] = centre(s == 0 ? q[o].x : s == 1 ? q[o].y : s == 2 ? q[o].z : q[o].w, zero_of(p[o][i]));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float v[8] = {x[r][s][0].x, x[r][s][0].y, x[r][s][0].z, x[r][s][0].w,
                        x[r][s][1].x, x[r][s][1].y, x[r][s][1].z, x[r][s][1].w};
          uint4 planes[3];
          split(v, planes);
#pragma unroll
          for (int t = 0; t < 3; ++t)
#pragma unroll
            for (int o = 0; o < OB; ++o) mma16(acc[o][r], planes[t], wq[o]);
        }
      }
#pragma unroll
      for (int o = 0; o < OB; ++o)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[o][r][e] = fmaf(scale_of(p[o][i]), acc[o][r][e], sum[o][r][e]);
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int o = 0; o < OB; ++o) *reinterpret_cast<f32x4*>(&red[w][(r * OB + o) * 256 + lane * 4]) = sum[o][r];
  __syncthreads();
  store_sums<float, RT, OB>(a, &red[0][0], cb0, t0);
}

// bf16: RT blocks of 16 rows of X by OB blocks of 16 rows of W a workgroup, the
// column blocks of both dealt to its waves in turn.  Read as operands, X would
// cost most: 16 rows of 64 bytes touch 16 lines, and a line is what a load
// costs.  So each wave brings its column block of X in whole lines (eight rows
// of 128 bytes a load) into its own part of LDS, half a block at a time, the next
// one while this one is multiplied, and its codes and parameters beside it.
// Nothing is shared between the waves before their sums.  48 rows, 4096 ->
// 12288: 13 us (operands straight from memory 28, one block of W a workgroup 41).
template <int RT, int OB, int GPB>
__global__ __launch_bounds__(ROW_WAVES * 64) void rows_kernel(RowsArgs a) {
  constexpr int XH = RT * 2048, CODES = 2 * XH, PARAMS = CODES + OB * 1024, WAVE = PARAMS + GPB * 256;
  constexpr int RED = RT * OB * 1024;   // a wave's sums
  __shared__ __attribute__((aligned(1024))) char lds[ROW_WAVES * (WAVE > RED ? WAVE : RED)];
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb0 = blockIdx.x * OB, t0 = blockIdx.y * RT * 16, kt = a.w.kt;
  const int blocks = min(OB, (a.w.c2 + 15) / 16 - cb0);
  const char* mine = lds + w * WAVE;
  const uint32_t base = lds_addr(mine);
  constexpr int OUT = (int)0x80000000u;   // reads as zero
  const int ldx = (int)a.ldx * 2, row8 = lane >> 3, end = a.w.c1 * 2;
  int vx[2 * RT];
#pragma unroll
  for (int d = 0; d < 2 * RT; ++d) {
    const int row = 8 * d + row8;
    vx[d] = t0 + row < a.n ? row * ldx + (((lane & 7) ^ (row >> 1 & 7)) << 4) : OUT;
  }
  const int vp = g < blocks ? (g * kt * GPB * 16 + j) * 4 : OUT;
  const i32x4v rx = rsrc_words(reinterpret_cast<const char*>(a.X) + (int64_t)t0 * ldx, 0x7fffffffu);
  const i32x4v rc = rsrc_words(a.w.codes + (int64_t)cb0 * kt * 64, 0x7fffffffu);
  const i32x4v rp = rsrc_words(a.w.params + (int64_t)cb0 * kt * GPB * 16, 0x7fffffffu);
  // half h of X's column block b; past the last block all of it is out of range,
  // so that every turn has the same number of loads
  auto load_x = [&](int b, auto half) __attribute__((always_inline)) {
    constexpr int H = decltype(half)::value;
    const int at = b * 256 + H * 128;
    if (b + 1 < kt) {
      static_for<0, 2 * RT>([&](auto d) __attribute__((always_inline)) {
        constexpr int D = decltype(d)::value;
        dma16k<H * XH + D * 1024>(rx, vx[D], at, base);
      });
    } else {
      static_for<0, 2 * RT>([&](auto d) __attribute__((always_inline)) {
        constexpr int D = decltype(d)::value;
        const int ch = ((lane & 7) ^ ((8 * D + row8) >> 1 & 7)) << 4;
        dma16k<H * XH + D * 1024>(rx, at + ch < end ? vx[D] : OUT, at, base);
      });
    }
  };
  auto load_w = [&](int b) __attribute__((always_inline)) {
    const int vc = b < kt ? lane * 16 : OUT, v = b < kt ? vp : OUT;
    static_for<0, OB>([&](auto o) __attribute__((always_inline)) {
      constexpr int O = decltype(o)::value;
      // past the last block of W: nothing that would be stored
      dma16k<CODES + O * 1024>(rc, vc, (min(O, blocks - 1) * kt + b) * 1024, base);
    });
    static_for<0, GPB>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      dma4(rp, v, (b * GPB + I) * 64, base + PARAMS + I * 256);
    });
  };
  f32x4 sum[OB][RT], acc[OB][RT], all[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int o = 0; o < OB; ++o) sum[o][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
  std::integral_constant<int, 0> first;
  std::integral_constant<int, 1> second;
  load_x(w, first);
  load_w(w);
  load_x(w, second);
  for (int b = w; b < kt; b += ROW_WAVES) {
    uint4 q[OB];
    uint32_t p[OB][GPB];
    auto multiply_half = [&](auto half) __attribute__((always_inline)) {
      constexpr int H = decltype(half)::value;
      uint4 x[2][RT];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int row = 16 * r + j;
          x[s][r] = *reinterpret_cast<const uint4*>(mine + H * XH + row * 128 + (((4 * s + g) ^ (row >> 1 & 7)) << 4));
        }
      if constexpr (H == 0) {
#pragma unroll
        for (int o = 0; o < OB; ++o) {
          q[o] = *reinterpret_cast<const uint4*>(mine + CODES + o * 1024 + lane * 16);
#pragma unroll
          for (int i = 0; i < GPB; ++i)
            p[o][i] = *reinterpret_cast<const uint32_t*>(mine + PARAMS + i * 256 + (o * 16 + j) * 4);
        }
      }
      wait_lgkm0();   // read: the next turn's may land here
      asm volatile("" ::: "memory");
      load_x(b + ROW_WAVES, half);
      if constexpr (H == 0) load_w(b + ROW_WAVES);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        constexpr int STEPS = 4 / GPB;   // of a group
        const int step = 2 * H + s;
        if (step % STEPS == 0) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            all[r] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int o = 0; o < OB; ++o) acc[o][r] = (f32x4){0.f, 0.f, 0.f, 0.f};
          }
        }
        const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
#pragma unroll
        for (int r = 0; r < RT; ++r) mma16(all[r], x[s][r], ones);
#pragma unroll
        for (int o = 0; o < OB; ++o) {
          const uint4 wq = widen(step == 0 ? q[o].x : step == 1 ? q[o].y : step == 2 ? q[o].z : q[o].w);
#pragma unroll
          for (int r = 0; r < RT; ++r) mma16(acc[o][r], x[s][r], wq);
        }
        if (step % STEPS == STEPS - 1) {
#pragma unroll
          for (int o = 0; o < OB; ++o) {
            const float sc = scale_of(p[o][step / STEPS]), zo = zero_of(p[o][step / STEPS]);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sum[o][r][e] = fmaf(sc, fmaf(-zo, all[r][e], acc[o][r][e]), sum[o][r][e]);
          }
        }
      }
    };
    wait_vm_lgkm0<2 * RT>();   // this block's first half, codes and parameters have landed
    asm volatile("" ::: "memory");
    multiply_half(first);
    wait_vm_lgkm0<2 * RT + OB + GPB>();   // its second half
    asm volatile("" ::: "memory");
    multiply_half(second);
  }
  wait_vm_lgkm0<0>();
  __syncthreads();   // no load is under way: the waves' sums
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int o = 0; o < OB; ++o) *reinterpret_cast<f32x4*>(red + ((w * RT + r) * OB + o) * 256 + lane * 4) = sum[o][r];
  __syncthreads();
  store_sums<bf16_t, RT, OB>(a, red, cb0, t0);
}

// ---------------------------------------------------------------------------
// the weight written out
// ---------------------------------------------------------------------------

// 16 x 128 of W as NP bf16 planes [c2][c1], a wave's work.  One plane rounds W, two
// hold it exactly.
template <int NP, int GPB>
__device__ __forceinline__ void write_dense(const Weight& w, bf16_t* out, int64_t plane, int id, char* mine) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int cb = id / w.kt, b = id - cb * w.kt;
  const uint4 q = w.codes[(int64_t)id * 64 + lane];
  const uint32_t words[4] = {q.x, q.y, q.z, q.w};
  float v[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t p = w.params[((int64_t)id * GPB + s * GPB / 4) * 16 + j];
    const float sc = scale_of(p), zo = zero_of(p);
    const uint4 x = widen(words[s]);
    const uint32_t h[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[s][2 * e] = sc * (__uint_as_float(h[e] << 16) - zo);
      v[s][2 * e + 1] = sc * (__uint_as_float(h[e] & 0xffff0000u) - zo);
    }
  }
  uint4 planes[4][NP];
#pragma unroll
  for (int s = 0; s < 4; ++s) split(v[s], planes[s]);
#pragma unroll
  for (int t = 0; t < NP; ++t) {
#pragma unroll
    for (int s = 0; s < 4; ++s)   // row j, chunk 4 s + g at chunk ^ j: 16 rows of a chunk in 16 places
      *reinterpret_cast<uint4*>(mine + j * 256 + (((4 * s + g) ^ j) << 4)) = planes[s][t];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // four rows of whole lines
      const int row = 4 * i + (lane >> 4), k = b * 128 + j * 8;
      const uint4 x = *reinterpret_cast<const uint4*>(mine + row * 256 + ((j ^ row) << 4));
      if (cb * 16 + row < w.c2 && k < w.c1)
        *reinterpret_cast<uint4*>(out + t * plane + (int64_t)(cb * 16 + row) * w.c1 + k) = x;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int GPB>
__global__ __launch_bounds__(256) void dense_kernel(Weight w, bf16_t* out, int waves) {
  __shared__ __attribute__((aligned(1024))) char lds[4][4096];
  const int id = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id < waves) write_dense<1, GPB>(w, out, 0, id, lds[threadIdx.x >> 6]);
}

// The operands of an fp32 product: the weight's two planes in the first
// workgroups, the rows' three in the others.
template <int GPB>
__global__ __launch_bounds__(256) void operands_kernel(Weight w, bf16_t* out, int64_t plane, int waves, int first,
                                                       Planes<float> x) {
  __shared__ __attribute__((aligned(1024))) char lds[4][4096];
  if ((int)blockIdx.x >= first) return make_planes(x, (int64_t)(blockIdx.x - first) * 256 + threadIdx.x);
  const int id = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id < waves) write_dense<2, GPB>(w, out, plane, id, lds[threadIdx.x >> 6]);
}

// W in fp32, exact; eight columns a thread.
__global__ __launch_bounds__(256) void dense_f32_kernel(Weight w, float* out, int gpb) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, words = w.c1 / 8;
  const int64_t row = i / words;
  const int k = (int)(i - row * words) * 8;
  if (row >= w.c2) return;
  const int64_t cb = row / 16, b = k / 128;
  const int lane = (int)(row % 16) + 16 * (k % 32 / 8), s = k % 128 / 32;
  const uint32_t q = reinterpret_cast<const uint32_t*>(w.codes)[((cb * w.kt + b) * 64 + lane) * 4 + s];
  const uint32_t p = w.params[((cb * w.kt + b) * gpb + s * gpb / 4) * 16 + row % 16];
  const float sc = scale_of(p), zo = zero_of(p);
  const uint4 x = widen(q);
  const uint32_t h[4] = {x.x, x.y, x.z, x.w};
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = sc * (__uint_as_float(h[e] << 16) - zo);
    v[2 * e + 1] = sc * (__uint_as_float(h[e] & 0xffff0000u) - zo);
  }
  float4* o = reinterpret_cast<float4*>(out + row * w.c1 + k);
  o[0] = make_float4(v[0], v[1], v[2], v[3]);
  o[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ---------------------------------------------------------------------------
// making a weight
// ---------------------------------------------------------------------------

// The packed form of codes [c2][c1 / 2] (the even column in a byte's low
// half), scales and zero points [c2][groups]; a lane of a block a thread.
__global__ __launch_bounds__(256) void pack_kernel(const uint32_t* __restrict__ codes,
                                                   const bf16_t* __restrict__ scale, const uint8_t* __restrict__ zero,
                                                   uint4* __restrict__ out, uint32_t* __restrict__ params, int c1,
                                                   int c2, int kt, int gpb, int64_t lanes) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= lanes) return;
  const int lane = (int)(i & 63), j = lane & 15, g = lane >> 4;
  const int64_t blk = i >> 6, cb = blk / kt, row = cb * 16 + j;
  const int b = (int)(blk - cb * kt);
  auto half = [](uint32_t v) {   // nibbles 0, 2, 4, 6 side by side
    v &= 0x0f0f0f0fu;
    v = (v | v >> 4) & 0x00ff00ffu;
    return (v | v >> 8) & 0xffffu;
  };
  uint32_t w[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = b * 128 + 32 * s + 8 * g;
    const uint32_t q = row < c2 && k < c1 ? codes[row * (c1 / 8) + k / 8] : 0;
    w[s] = half(q) | half(q >> 4) << 16;
  }
  out[i] = make_uint4(w[0], w[1], w[2], w[3]);
  const int group = 128 / gpb, groups = (c1 + group - 1) / group;
  if (g < gpb) {   // lane group g writes group g of the block
    const int q = b * gpb + g;
    const bool in = row < c2 && q < groups;
    const uint32_t z = in && zero ? zero[row * groups + q] & 15 : 8;
    params[(cb * kt * gpb + q) * 16 + j] = (in ? (uint32_t)scale[row * groups + q] << 16 : 0u) | 0x4300u | z;
  }
}

// Codes of a matrix to the nearest, ties to even.  Without zero points the
// largest magnitude of a group is 7 scales; with them lowest and highest (0
// among them) are 15 scales apart.  A scale is rounded to bf16 first.
template <typename T>
__global__ __launch_bounds__(256) void quantise_kernel(const T* __restrict__ W, int c1, int64_t c2, int group,
                                                       uint8_t* __restrict__ codes, bf16_t* __restrict__ scale,
                                                       uint8_t* __restrict__ zero) {
  const int groups = (c1 + group - 1) / group;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 4;   // four lanes a group
  const int part = threadIdx.x & 3;
  const int64_t row = i / groups;
  const int q = (int)(i - row * groups), k0 = q * group, k1 = min(k0 + group, c1);
  const bool in = row < c2;
  float lo = 0.f, hi = 0.f;
  if (in)
    for (int k = k0 + part * 8; k < k1; k += 32)
      for (int e = 0; e < 8; ++e) {
        const float v = TT<T>::to_f(W[row * c1 + k + e]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
      }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
  }
  if (!in) return;
  const float span = zero ? hi / 15.f - lo / 15.f : fmaxf(hi, -lo) / 7.f;
  const bf16_t sc = f2bf(span);
  const float s = bf2f(sc);
  const float z = !zero ? 8.f : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
  for (int k = k0 + part * 8; k < k1; k += 32)
    for (int e = 0; e < 8; e += 2) {
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float v = s > 0.f ? rintf(TT<T>::to_f(W[row * c1 + k + e + h]) / s) + z : z;
        c[h] = (uint32_t)fminf(fmaxf(v, 0.f), 15.f);
      }
      codes[(row * c1 + k + e) / 2] = (uint8_t)(c[0] | c[1] << 4);
    }
  if (part == 0) {
    scale[row * groups + q] = sc;
    if (zero) zero[row * groups + q] = (uint8_t)z;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

int validate(int64_t c1, int64_t c2, int group) {
  if (group != 32 && group != 64 && group != 128) return DYRA_EINVAL;
  if (c1 <= 0 || c2 <= 0 || c1 % 8 || c2 % 8 || c1 > (int64_t)1 << 20 || c2 > (int64_t)1 << 20) return DYRA_ESHAPE;
  if (c1 * c2 > (int64_t)1 << 34) return DYRA_ESHAPE;   // launches below 2^32 threads
  return DYRA_OK;
}

int validate_call(const dyra_q4* w, int64_t n, int dtype) {
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  const int rc = validate(w->c1, w->c2, w->group);
  if (rc) return rc;
  if (n < 0 || n > (int64_t)1 << 24) return DYRA_ESHAPE;
  if (n * std::max(w->c1, w->c2) >= (int64_t)1 << 33) return DYRA_ESHAPE;
  return DYRA_OK;
}

int64_t code_bytes(int64_t c1, int64_t c2) { return cdiv(c2, 16) * cdiv(c1, 128) * 1024; }
int64_t param_bytes(int64_t c1, int64_t c2, int group) { return cdiv(c2, 16) * cdiv(c1, 128) * (128 / group) * 64; }

Weight weight_of(const dyra_q4& w) {
  const char* p = reinterpret_cast<const char*>(w.packed);
  return {reinterpret_cast<const uint4*>(p), reinterpret_cast<const uint32_t*>(p + code_bytes(w.c1, w.c2)),
          (int32_t)w.c1, (int32_t)w.c2, (int32_t)cdiv(w.c1, 128)};
}

// How few rows run: RT x OB blocks a workgroup, and the estimated microseconds.
struct FewRows {
  int rt, ob;
  double us;
};

// In bf16 workgroups are taken to run in rounds of 256, one a CU: a fit of the times
// below (by its LDS, 43 to 139 KB, up to three of the smallest fit a CU).  A round's time is
// made of its turns of eight column blocks, of its sums' way through LDS and, but for
// the first, of its start.  Measured at 4096 -> 4096, groups of 128 (us): 1 row, RT OB = 1 1
// 4.2, 1 2 4.7, 1 4 6.3; 64 rows, 2 1 9.9, 2 2 7.0, 2 4 8.9, 3 2 8.6; 384 rows, 2 4 26.1, 3 4
// 24.3.  fp32 splits X anew for each pair of blocks of W.
FewRows few_rows(int64_t c1, int64_t c2, int64_t n, int dtype) {
  const int64_t blocks = cdiv(c2, 16), turns_k = cdiv(cdiv(c1, 128), ROW_WAVES);
  FewRows best{0, 0, 1e30};
  if (dtype == DYRA_F32) {
    const int rt = n <= 16 ? 1 : n <= 32 ? 2 : 4;
    const int64_t groups = cdiv(n, 16 * rt);
    const int ob = cdiv(blocks, 2) * groups >= 192 ? 2 : 1;
    return {rt, ob, 2.5 + (double)cdiv(cdiv(blocks, ob) * groups, 256) * turns_k * rt * (2.0 + 0.25 * ob)};
  }
  for (int rt = 1; rt <= 3; ++rt)
    for (int ob = 1; ob <= 4; ++ob) {
      const double rounds = (double)cdiv(cdiv(blocks, ob) * cdiv(n, 16 * rt), 256);
      const double turn = 0.4 + 0.16 * rt + 0.025 * ob + 0.12 * rt * ob;
      const double us = 0.7 + rounds * (1.5 + turns_k * turn + 0.17 * rt * ob);
      if (us < best.us) best = {rt, ob, us};
    }
  return best;
}

// Sizes of a call; few rows need no workspace.
struct Plan {
  bool few;
  FewRows rows;
  Shape tile;
  size_t dense, planes, part, total;
};

// in, out: the reduced and the resulting width
Plan make_plan(int64_t in, int64_t out, int64_t n, int dtype, bool backward) {
  Plan q{};
  const bool wide = dtype == DYRA_F32;
  const Job j = job({nullptr, 0, 0, (int32_t)n}, {nullptr, 0, 0, (int32_t)out}, in, in, wide ? 5 : 1, 0);
  q.tile = shape_of(j);
  if (!backward) {
    // many rows: the weight is written out and read again, two or three launches.
    // Few and many, measured, us: 4096 -> 4096, 384 rows 24 and 38, 768 48 and 56, 1024 69
    // and 58; 4096 -> 12288, 384 rows 72 and 73, 512 104 and 78; fp32, 4096 -> 4096, 128 rows
    // 42 and 60, 256 80 and 73.
    q.rows = few_rows(in, out, n, dtype);
    q.few = n <= (int64_t)1 << 16 && q.rows.us <= 8 + (wide ? 4 + in * out / 2e6 : in * out / 3e6) + cost(q.tile, j);
    if (q.few) return q;
  }
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  q.dense = take((wide ? 4 : 2) * in * out);
  if (wide) q.planes = take(6 * n * in);
  q.part = take(part_bytes(q.tile, j));
  q.total = at;
  return q;
}

template <typename T, int RT, int OB>
void launch_rows_as(const RowsArgs& a, int group, hipStream_t st) {
  const dim3 grid((unsigned)cdiv(a.w.c2, 16 * OB), (unsigned)cdiv(a.n, 16 * RT)), nt(ROW_WAVES * 64);
  if constexpr (sizeof(T) == 2) {
    if (group == 128) hipLaunchKernelGGL((rows_kernel<RT, OB, 1>), grid, nt, 0, st, a);
    else if (group == 64) hipLaunchKernelGGL((rows_kernel<RT, OB, 2>), grid, nt, 0, st, a);
    else hipLaunchKernelGGL((rows_kernel<RT, OB, 4>), grid, nt, 0, st, a);
  } else {
    if (group == 128) hipLaunchKernelGGL((rows_f32_kernel<RT, OB, 1>), grid, nt, 0, st, a);
    else if (group == 64) hipLaunchKernelGGL((rows_f32_kernel<RT, OB, 2>), grid, nt, 0, st, a);
    else hipLaunchKernelGGL((rows_f32_kernel<RT, OB, 4>), grid, nt, 0, st, a);
  }
}

template <typename T, int RT>
void launch_rows(const RowsArgs& a, int ob, int group, hipStream_t st) {
  if (ob == 1) launch_rows_as<T, RT, 1>(a, group, st);
  else if (ob == 2) launch_rows_as<T, RT, 2>(a, group, st);
  else if constexpr (sizeof(T) == 2) {
    if (ob == 3) launch_rows_as<T, RT, 3>(a, group, st);
    else launch_rows_as<T, RT, 4>(a, group, st);
  }
}

void launch_dense(const Weight& w, int group, bf16_t* out, hipStream_t st) {
  const int64_t waves = cdiv(w.c2, 16) * w.kt;
  const dim3 grid((unsigned)cdiv(waves, 4)), nt(256);
  if (group == 128) hipLaunchKernelGGL((dense_kernel<1>), grid, nt, 0, st, w, out, (int)waves);
  else if (group == 64) hipLaunchKernelGGL((dense_kernel<2>), grid, nt, 0, st, w, out, (int)waves);
  else hipLaunchKernelGGL((dense_kernel<4>), grid, nt, 0, st, w, out, (int)waves);
}

void launch_operands(const Weight& w, int group, bf16_t* out, const Planes<float>& x, hipStream_t st) {
  const int64_t waves = cdiv(w.c2, 16) * w.kt, plane = (int64_t)w.c1 * w.c2, first = cdiv(waves, 4);
  const dim3 grid((unsigned)(first + cdiv((int64_t)x.rows * (x.cols / 8), 256))), nt(256);
  if (group == 128) hipLaunchKernelGGL((operands_kernel<1>), grid, nt, 0, st, w, out, plane, (int)waves, (int)first, x);
  else if (group == 64)
    hipLaunchKernelGGL((operands_kernel<2>), grid, nt, 0, st, w, out, plane, (int)waves, (int)first, x);
  else hipLaunchKernelGGL((operands_kernel<4>), grid, nt, 0, st, w, out, plane, (int)waves, (int)first, x);
}

// out [n][cout] = in [n][cin] times the weight, transposed or (BACK) as it is
template <typename T, bool BACK>
int many(const dyra_q4& w, const T* in, int64_t ldi, const T* bias, T* out, int64_t ldo, int64_t n, const Plan& q,
         char* ws, hipStream_t st) {
  constexpr bool wide = sizeof(T) == 4;
  const int64_t cin = BACK ? w.c2 : w.c1, cout = BACK ? w.c1 : w.c2;
  bf16_t* dense = reinterpret_cast<bf16_t*>(ws + q.dense);
  Operand a{in, 2 * ldi, 0, (int32_t)n};
  if constexpr (wide) {
    launch_operands(weight_of(w), w.group, dense, planes(in, ldi, n, cin, ws + q.planes, n * cin), st);
    a = {ws + q.planes, 2 * cin, 2 * n * cin, (int32_t)n};
  } else {
    launch_dense(weight_of(w), w.group, dense, st);
  }
  Job j = job(a, {dense, 2 * w.c1, 2 * w.c1 * w.c2, (int32_t)cout}, cin, cin, wide ? 5 : 1, wide ? TERMS_32 : TERMS_1);
  j.part = reinterpret_cast<float4*>(ws + q.part);
  launch_as<false, BACK>(q.tile, j, Store<T>{out, ldo, (int32_t)cout, bias, nullptr, nullptr, nullptr, 1.f}, st);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

template <typename T>
int forward_impl(const dyra_q4& w, const T* X, int64_t ldx, const T* bias, T* Y, int64_t ldy, int64_t n,
                 const Plan& q, char* ws, hipStream_t st) {
  if (!q.few) return many<T, false>(w, X, ldx, bias, Y, ldy, n, q, ws, st);
  const RowsArgs a{weight_of(w), X, bias, Y, ldx, ldy, (int32_t)n};
  if (q.rows.rt == 1) launch_rows<T, 1>(a, q.rows.ob, w.group, st);
  else if (q.rows.rt == 2) launch_rows<T, 2>(a, q.rows.ob, w.group, st);
  else launch_rows<T, sizeof(T) == 2 ? 3 : 4>(a, q.rows.ob, w.group, st);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

}  // namespace

extern "C" int dyra_q4_packed_size(int64_t c1, int64_t c2, int32_t group, size_t* bytes) {
  if (!bytes) return DYRA_EINVAL;
  const int rc = validate(c1, c2, group);
  if (rc) return rc;
  *bytes = (size_t)(code_bytes(c1, c2) + param_bytes(c1, c2, group));
  return DYRA_OK;
}

extern "C" int dyra_q4_pack(int64_t c1, int64_t c2, int32_t group, const void* codes, const void* scale,
                            const void* zero, void* packed, void* stream) {
  if (!codes || !scale || !packed) return DYRA_EINVAL;
  const int rc = validate(c1, c2, group);
  if (rc) return rc;
  if (misaligned(codes, 3) || misaligned(scale, 1) || misaligned(packed, 15)) return DYRA_EINVAL;
  const int64_t kt = cdiv(c1, 128), lanes = cdiv(c2, 16) * kt * 64;
  char* p = reinterpret_cast<char*>(packed);
  hipLaunchKernelGGL(pack_kernel, dim3((unsigned)cdiv(lanes, 256)), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), reinterpret_cast<const uint32_t*>(codes),
                     reinterpret_cast<const bf16_t*>(scale), reinterpret_cast<const uint8_t*>(zero),
                     reinterpret_cast<uint4*>(p), reinterpret_cast<uint32_t*>(p + code_bytes(c1, c2)), (int)c1, (int)c2,
                     (int)kt, 128 / group, lanes);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

extern "C" int dyra_q4_quantise(const void* W, int64_t c1, int64_t c2, int32_t group, int32_t dtype, void* codes,
                                void* scale, void* zero, void* stream) {
  if (!W || !codes || !scale) return DYRA_EINVAL;
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  const int rc = validate(c1, c2, group);
  if (rc) return rc;
  if (misaligned(W, 15) || misaligned(codes, 3) || misaligned(scale, 1)) return DYRA_EINVAL;
  const dim3 grid((unsigned)cdiv(c2 * cdiv(c1, group) * 4, 256)), nt(256);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  uint8_t *q = reinterpret_cast<uint8_t*>(codes), *z = reinterpret_cast<uint8_t*>(zero);
  bf16_t* s = reinterpret_cast<bf16_t*>(scale);
  if (dtype == DYRA_BF16)
    hipLaunchKernelGGL((quantise_kernel<bf16_t>), grid, nt, 0, st, reinterpret_cast<const bf16_t*>(W), (int)c1, c2,
                       group, q, s, z);
  else
    hipLaunchKernelGGL((quantise_kernel<float>), grid, nt, 0, st, reinterpret_cast<const float*>(W), (int)c1, c2,
                       group, q, s, z);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

extern "C" int dyra_q4_dense(const dyra_q4* w, void* out, int32_t dtype, void* stream) {
  if (!w || !w->packed || !out) return DYRA_EINVAL;
  const int rc = validate_call(w, 0, dtype);
  if (rc) return rc;
  if (misaligned(w->packed, 15) || misaligned(out, 15)) return DYRA_EINVAL;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == DYRA_BF16) launch_dense(weight_of(*w), w->group, reinterpret_cast<bf16_t*>(out), st);
  else
    hipLaunchKernelGGL(dense_f32_kernel, dim3((unsigned)cdiv(w->c2 * (w->c1 / 8), 256)), dim3(256), 0, st,
                       weight_of(*w), reinterpret_cast<float*>(out), 128 / w->group);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

extern "C" int dyra_q4_workspace_size(int64_t c1, int64_t c2, int64_t n, int32_t dtype, int32_t backward,
                                      size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return DYRA_EINVAL;
  const dyra_q4 w{c1, c2, 128, nullptr};
  const int rc = validate_call(&w, n, dtype);
  if (rc) return rc;
  *bytes = n ? (backward ? make_plan(c2, c1, n, dtype, true) : make_plan(c1, c2, n, dtype, false)).total : 0;
  return DYRA_OK;
}

extern "C" int dyra_q4_forward(const dyra_q4* w, const void* X, int64_t ldx, const void* bias, void* Y, int64_t ldy,
                               int64_t n, int32_t dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!w || !w->packed) return DYRA_EINVAL;
  const int rc = validate_call(w, n, dtype);
  if (rc) return rc;
  if (misaligned(w->packed, 15)) return DYRA_EINVAL;
  if (n == 0) return DYRA_OK;
  if (!X || !Y || misaligned(X, 15) || misaligned(bias, 15) || misaligned(Y, 15) || misaligned(workspace, 15))
    return DYRA_EINVAL;
  if (bad_stride(ldx, w->c1, dtype) || bad_stride(ldy, w->c2, dtype)) return DYRA_ESHAPE;
  const Plan q = make_plan(w->c1, w->c2, n, dtype, false);
  if (q.total && !workspace) return DYRA_EINVAL;
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == DYRA_BF16)
    return forward_impl(*w, reinterpret_cast<const bf16_t*>(X), ldx, reinterpret_cast<const bf16_t*>(bias),
                        reinterpret_cast<bf16_t*>(Y), ldy, n, q, ws, st);
  return forward_impl(*w, reinterpret_cast<const float*>(X), ldx, reinterpret_cast<const float*>(bias),
                      reinterpret_cast<float*>(Y), ldy, n, q, ws, st);
}

extern "C" int dyra_q4_backward(const dyra_q4* w, const void* dY, int64_t lddy, void* dX, int64_t lddx, int64_t n,
                                int32_t dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!w || !w->packed) return DYRA_EINVAL;
  const int rc = validate_call(w, n, dtype);
  if (rc) return rc;
  if (misaligned(w->packed, 15)) return DYRA_EINVAL;
  if (n == 0) return DYRA_OK;
  if (!dY || !dX || !workspace || misaligned(dY, 15) || misaligned(dX, 15) || misaligned(workspace, 15))
    return DYRA_EINVAL;
  if (bad_stride(lddy, w->c2, dtype) || bad_stride(lddx, w->c1, dtype)) return DYRA_ESHAPE;
  const Plan q = make_plan(w->c2, w->c1, n, dtype, true);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == DYRA_BF16)
    return many<bf16_t, true>(*w, reinterpret_cast<const bf16_t*>(dY), lddy, nullptr, reinterpret_cast<bf16_t*>(dX),
                              lddx, n, q, ws, st);
  return many<float, true>(*w, reinterpret_cast<const float*>(dY), lddy, nullptr, reinterpret_cast<float*>(dX), lddx, n,
                           q, ws, st);
}
