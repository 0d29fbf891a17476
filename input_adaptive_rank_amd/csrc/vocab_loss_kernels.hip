// Softmax cross entropy over a vocabulary, from hidden rows H [n][C] and a
// head W [V][C], without the logits in memory:
//   a_tv = scale H_t . W_v,  lse_t = log sum_v exp a_tv,  loss_t = lse_t - a_t,target
//   d_tv = scale dloss_t (exp(a_tv - lse_t) - [v = target_t])
//   dH = d W,  dW = d^T H
//
// Forward: one product whose epilogue leaves, for each row and 64 columns, the
// maximum and the sum of exponentials below it; a second launch joins them.  4099 x
// 4096 x 32000: 885 us, a library's product alone 830 to 870.  Backward: the rows
// that count are gathered; for one piece of the vocabulary after the other their
// logits are multiplied again, d goes to memory as bf16, and the two gradients are
// products of the piece, whose operands the LDS turns where they lie across the
// reduction.  The pieces keep d in bf16 within the 256 MB of the last-level cache, up to
// 2^19 rows (a piece has at least 256 words); its three planes in fp32 take up to three
// times that.  The same sizes, 3280 rows that count: 2310 us, 1.12 PFLOP/s.  (Times vary
// by 7 % with the card.)
//
// bf16: logits are sums of exact products in fp32; d is rounded to bf16 for
// the two products of the backward pass (at most 2^-8 of a term, like the
// rounding of the gradients, which are bf16).  fp32: every operand is three
// bf16 planes (24 bits), a product the six pairs of planes that reach 2^-24; W is
// split on its way where few rows read it, else written out as planes first.
#include "mfma_product.h"

namespace {

using namespace product;

constexpr float LOG2E = 1.44269504088896340736f;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Each row's softmax over 64 columns: the largest logit m and the sum of
// exp(a - m), and the target's logit where it lies among them.  Every exponent
// is a difference times log2 e, never a difference of rounded products, and m is
// rounded as the target's logit is: a sum of exponentials is at least 1, m at
// least the target's logit, so that no loss is negative.
struct RowStats {
  float2* part;             // [blocks of 64 columns][rows]
  float* mine;              // [rows] logit of the target
  const int32_t* targets;
  float scale;
  int32_t cols, v0;         // of this piece of W; its first, a multiple of 64

  template <class C>
  __device__ __forceinline__ void block(const f32x16 (&v)[C::FN], char*, int row0, int col0, int rows) const {
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5, row = row0 + l;
    if (col0 >= cols) return;
    const float k2 = scale * LOG2E;
    const int at = (int)((unsigned)(row < rows ? targets[row] : -1) - (unsigned)(v0 + col0));
    const bool has = (unsigned)at < (unsigned)min(C::WN, cols - col0) && (at >> 2 & 1) == g;
    if (__any(has)) {
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i)
        if (has && i == ((at >> 5) * 16 + (at >> 3 & 3) * 4 + (at & 3))) mine[row] = v[i / 16][i % 16] * scale;
    }
    const int edge = cols - col0 - 4 * g;   // columns from here on are none
    float a[16 * C::FN];
#pragma unroll
    for (int i = 0; i < 16 * C::FN; ++i) {
      a[i] = v[i / 16][i % 16];
      if (edge < C::WN) a[i] = i / 16 * 32 + (i % 16 / 4) * 8 + i % 4 < edge ? a[i] : -INFINITY;
    }
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16 * C::FN; ++i) top = fmaxf(top, a[i]);
    top = fmaxf(top, __shfl_xor(top, 32));
    // nothing above -inf: exponents are taken from 0, so that a NaN stays
    const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < 16 * C::FN; ++i) sum += __builtin_amdgcn_exp2f((a[i] - from) * k2);
    sum += __shfl_xor(sum, 32);
    if (g == 0 && row < rows) part[(int64_t)((v0 + col0) / 64) * rows + row] = make_float2(top * scale, sum);
  }

  template <class C>
  __device__ __forceinline__ void tile(Acc<C>& acc, char* lds, int m0, int n0, int rows, int wm, int wn) const {
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
      block<C>(acc[fm], lds, m0 + wm * C::WM + fm * 32, n0 + wn * C::WN, rows);
      __builtin_amdgcn_sched_barrier(0);   // one block after the other: registers
    }
  }
};

// Joins a row's parts: 32 rows a workgroup, 32 lanes a row.
__global__ __launch_bounds__(1024) void row_loss_kernel(const float2* __restrict__ part, const float* __restrict__ mine,
                                                        const int32_t* __restrict__ targets, float* __restrict__ loss,
                                                        float* __restrict__ lse, int rows, int vocab, int blocks) {
  __shared__ float2 st[32][32];
  const int rr = threadIdx.x & 31, k = threadIdx.x >> 5, row = blockIdx.x * 32 + rr;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 s) {
    const float t = fmaxf(top, s.x);
    sum = (top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f((top - t) * LOG2E)) +
          (s.x == -INFINITY ? s.y : s.y * __builtin_amdgcn_exp2f((s.x - t) * LOG2E));
    top = t;
  };
  if (row < rows) {
#pragma unroll 8
    for (int t = k; t < blocks; t += 32) join(part[(int64_t)t * rows + row]);
  }
  st[k][rr] = make_float2(top, sum);
  __syncthreads();
  if (k < 4) {
#pragma unroll
    for (int i = 1; i < 8; ++i) join(st[k + 4 * i][rr]);
    st[k][rr] = make_float2(top, sum);
  }
  __syncthreads();
  if (k || row >= rows) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) join(st[i][rr]);
  const float rest = logf(sum);
  lse[row] = top == -INFINITY ? rest : top + rest;
  const int t = targets[row];
  loss[row] = t >= 0 && t < vocab ? (top - mine[row]) + rest : 0.f;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// What the device finds out about a backward call.
struct Found {
  int32_t live;     // rows that count
  float weight;     // the largest finite |dloss| among them, or 1: what d is relative to
};

// The rows that count: map[0 .. live - 1], ascending, by the first workgroup;
// the others set the rest's gradients to zero.
template <typename T>
__global__ __launch_bounds__(1024) void live_kernel(const int32_t* __restrict__ targets,
                                                    const float* __restrict__ dloss, int n, int vocab,
                                                    Found* __restrict__ found, int32_t* __restrict__ map,
                                                    T* __restrict__ dH, int64_t ld, int C) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (blockIdx.x) {
    const int row = (blockIdx.x - 1) * 16 + w;
    if (row >= n) return;
    const int t = targets[row];
    if (t >= 0 && t < vocab) return;
    constexpr int E = 16 / sizeof(T);
    for (int c = lane * E; c < C; c += 64 * E) *reinterpret_cast<uint4*>(dH + row * ld + c) = zero4();
    return;
  }
  constexpr int PER = 8;
  __shared__ int sums[2][16];
  __shared__ float tops[16];
  int base = 0, flip = 0;
  float top = 0.f;
  for (int r0 = 0; r0 < n; r0 += 1024 * PER, flip ^= 1) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int row = r0 + tid * PER + i, t = row < n ? targets[row] : -1;
      const bool in = t >= 0 && t < vocab;
      const float g = in ? fabsf(dloss[row]) : 0.f;
      bits |= (uint32_t)in << i;
      if (g < INFINITY) top = fmaxf(top, g);
    }
    const int mine = __popc(bits);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 63) sums[flip][w] = upto;
    __syncthreads();
    int at = base + upto - mine;
    for (int i = 0; i < 16; ++i) {
      const int o = sums[flip][i];
      base += o;
      if (i < w) at += o;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (bits >> i & 1) map[at++] = r0 + tid * PER + i;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane == 0) tops[w] = top;
  __syncthreads();
  if (tid) return;
  for (int i = 1; i < 16; ++i) top = fmaxf(top, tops[i]);
  *found = Found{base, top > 0.f ? top : 1.f};
}

// The same for a few thousand rows, and their planes, in one launch: `per` rows a
// workgroup, which counts the rows before them itself; workgroup `groups` finds the
// rest out, and those behind it make the planes of W.
template <typename T>
__global__ __launch_bounds__(256) void gather_kernel(const int32_t* __restrict__ targets,
                                                     const float* __restrict__ dloss, int n, int vocab,
                                                     Found* __restrict__ found, int32_t* __restrict__ map,
                                                     T* __restrict__ dH, int64_t ld, Planes<T> h, int per, int groups,
                                                     Planes<T> w) {
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (b > groups) return make_planes(w, (int64_t)(b - groups - 1) * 256 + tid);
  __shared__ int sums[4], place[64];
  __shared__ float tops[4];
  const bool all = b == groups;
  const int r0 = all ? n : b * per;
  int count = 0;
  float top = 0.f;
#pragma unroll 4
  for (int i = tid; i < r0; i += 256) {
    const int t = targets[i];
    const bool in = t >= 0 && t < vocab;
    count += in;
    const float g = all && in ? fabsf(dloss[i]) : 0.f;
    if (g < INFINITY) top = fmaxf(top, g);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    count += __shfl_xor(count, d);
    top = fmaxf(top, __shfl_xor(top, d));
  }
  if (lane == 0) {
    sums[wave] = count;
    tops[wave] = top;
  }
  __syncthreads();
  const int base = sums[0] + sums[1] + sums[2] + sums[3];
  if (all) {
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    if (tid == 0) *found = Found{base, top > 0.f ? top : 1.f};
    return;
  }
  const int rows = min(per, n - r0);
  if (wave == 0) {
    const int t = lane < rows ? targets[r0 + lane] : -1;
    const bool in = t >= 0 && t < vocab;
    const uint64_t ins = __ballot(in);
    const int at = base + __popcll(ins & (((uint64_t)1 << lane) - 1));
    place[lane] = in ? at : -1;
    if (in) map[at] = r0 + lane;
  }
  __syncthreads();
  const int chunks = h.cols / 8;
  for (int i = tid; i < rows * chunks; i += 256) {
    const int r = i / chunks, col = (i - r * chunks) * 8, at = place[r];
    if (at >= 0) {
      split_eight(h, r0 + r, at, col);
    } else if (dH) {
#pragma unroll
      for (int e = 0; e < 8; e += 16 / sizeof(T)) *reinterpret_cast<uint4*>(dH + (r0 + r) * ld + col + e) = zero4();
    }
  }
}

// d of a tile over scale times the largest weight, in NP bf16 planes; columns past
// the piece's are zero up to the padded width.  So the entry of a target that is
// far from likely is 1 whatever the weights are, if they are all the same (the
// mean's): rounded with its weight it would be off by the same part of itself in
// every row, and the gradients with it.
template <int NP>
struct Gradient {
  bf16_t* d;                    // [NP][rows][ldd]
  int64_t ldd, plane;
  const float *lse, *dloss;
  const int32_t *targets, *map;
  const Found* found;
  float scale;
  int32_t cols, v0;             // of this piece

  // a row's logits to its d, in 32 x WN results
  template <class C>
  __device__ __forceinline__ void values(f32x16 (&v)[C::FN], int row, int col0, int rows) const {
    const int g = (threadIdx.x & 63) >> 5;
    const bool in = row < rows;
    const int r = in ? map[row] : 0;
    const float w = in ? dloss[r] / found->weight : 0.f, from = in ? lse[r] : 0.f;
    const int at = in ? targets[r] - v0 - col0 : -1;
    const bool has = (unsigned)at < (unsigned)C::WN && (at >> 2 & 1) == g;
#pragma unroll
    for (int i = 0; i < 16 * C::FN; ++i)
      v[i / 16][i % 16] = __builtin_amdgcn_exp2f(fmaf(v[i / 16][i % 16], scale, -from) * LOG2E);
    if (__any(has)) {
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i)
        v[i / 16][i % 16] -= has && i == ((at >> 5) * 16 + (at >> 3 & 3) * 4 + (at & 3)) ? 1.f : 0.f;
    }
    const int edge = in ? cols - col0 - 4 * g : 0;   // columns from here on are none
    if (__all(edge >= C::WN)) {
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i) v[i / 16][i % 16] *= w;
    } else {
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i)
        v[i / 16][i % 16] = i / 16 * 32 + (i % 16 / 4) * 8 + i % 4 < edge ? v[i / 16][i % 16] * w : 0.f;
    }
  }

  // two neighbouring results as bf16; what is left of them for the next plane
  __device__ static __forceinline__ uint32_t peel(f32x16& v, int i) {
    const uint32_t h = pack_bf16x2(v[i], v[i + 1]);
    if constexpr (NP > 1) {
      v[i] -= __uint_as_float(h << 16);
      v[i + 1] -= __uint_as_float(h & 0xffff0000u);
    }
    return h;
  }

  // 32 rows of one line
  template <class C>
  __device__ __forceinline__ void block(f32x16 (&v)[C::FN], char* lds, int row0, int col0, int rows) const {
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    values<C>(v, row0 + l, col0, rows);
#pragma unroll
    for (int t = 0; t < NP; ++t) {
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t x = peel(v[fn], 4 * q), y = peel(v[fn], 4 * q + 2);
          *reinterpret_cast<uint2*>(lds + lds_off(l, fn * 4 + q) + 8 * g) = make_uint2(x, y);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = i * 8 + (lane >> 3), k = lane & 7, col = col0 + k * 8;
        const uint4 x = *reinterpret_cast<const uint4*>(lds + lds_off(rr, k));
        if (row0 + rr < rows && col < ldd) *reinterpret_cast<uint4*>(d + t * plane + (row0 + rr) * ldd + col) = x;
      }
      __builtin_amdgcn_wave_barrier();
    }
  }

  template <class C>
  __device__ __forceinline__ void tile(Acc<C>& acc, char* lds, int m0, int n0, int rows, int wm, int wn) const {
    char* mine = lds + (wm * C::NWN + wn) * 4096;
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
      block<C>(acc[fm], mine, m0 + wm * C::WM + fm * 32, n0 + wn * C::WN, rows);
      __builtin_amdgcn_sched_barrier(0);   // one block after the other: registers
    }
  }
};

template <typename T>
__global__ __launch_bounds__(256) void zero_kernel(T* __restrict__ out, int64_t elems) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < elems / 8; i += (int64_t)gridDim.x * 256)
    for (int e = 0; e < 8; e += 16 / sizeof(T)) *reinterpret_cast<uint4*>(out + i * 8 + e) = zero4();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The three products of a call, without operands: their sizes and shapes.
Operand rows_of(int64_t rows) { return {nullptr, 0, 0, (int32_t)rows}; }

// Sizes of a call.
struct Plan {
  int64_t np;                           // planes of an operand
  int64_t piece;                        // columns of the vocabulary at a time
  Shape logits, dh, dw;                 // logits and dh both DIRECT: W is read as it is
  double us;                            // estimated, of what depends on that
  size_t part, mine, live, map, hp, wp, d, acc, parts, dw_parts, total;
};

const int32_t* const SOME = reinterpret_cast<const int32_t*>(4);   // "found on the device", for sizes alone

Plan plan_as(bool direct, int64_t n, int64_t C, int64_t V, int dtype, bool backward, bool need_dh, bool need_dw) {
  Plan q{};
  const bool wide = dtype == DYRA_F32;
  q.np = wide ? 3 : 1;
  const int terms = wide ? 6 : 1, once = direct ? 1 : terms;
  // d of a piece is at most 2^27 elements a plane (in bf16 256 MB, the last-level cache)
  // or 256 words of it, planes of fp32 weights at most 2^28 elements
  int64_t most = (int64_t)1 << 20;
  if (backward) most = std::min<int64_t>(most, ((int64_t)1 << 27) / n);
  if (wide && !direct) most = std::min<int64_t>(most, ((int64_t)1 << 28) / (3 * C));
  most = std::max<int64_t>(256, most & ~(int64_t)255);
  q.piece = std::min(up(V, 64), up(cdiv(V, cdiv(V, most)), 256));
  const int32_t* live = backward ? SOME : nullptr;
  const Job logits = job(rows_of(n), rows_of(q.piece), C, C, once, 0, live);
  q.logits = direct ? DIRECT : shape_of(logits);
  // a last piece of fewer columns may be split into more parts
  const Job rest = job(rows_of(n), rows_of(V - (cdiv(V, q.piece) - 1) * q.piece), C, C, once, 0, live);
  // the planes of W go to memory at 5 TB/s, 10 bytes an element, after a launch
  q.us = cost(q.logits, logits) + (wide && !direct ? 4 + 2e-6 * q.piece * C : 0.);
  int64_t parts = std::max(part_bytes(q.logits, logits), part_bytes(q.logits, rest));
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (wide && !direct) q.wp = take(2 * q.np * q.piece * C);
  if (wide || backward) q.hp = take(2 * q.np * n * C);
  if (!backward) {
    q.part = take(8 * cdiv(V, 64) * n);
    q.mine = take(4 * n);
  } else {
    q.live = take(sizeof(Found));
    q.map = take(4 * n);
    q.d = take(2 * q.np * n * q.piece);
    const Job j = job(rows_of(n), rows_of(C), q.piece, q.piece, once, 0, live);
    q.dh = direct ? DIRECT : shape_of(j);
    q.us += cost(q.dh, j);   // wanted or not, so that dW does not depend on it
    if (need_dh) {
      parts = std::max(parts, part_bytes(q.dh, j));
      if (q.piece < V) q.acc = take(4 * n * C);
    }
    if (need_dw) {
      const Job j = job(rows_of(q.piece), rows_of(C), n, n, terms, 0, live, true);
      q.dw = shape_of(j);
      // both gradients' parts are joined in one launch
      if (need_dh) q.dw_parts = take(part_bytes(q.dw, j));
      else parts = std::max(parts, part_bytes(q.dw, j));
    }
  }
  q.parts = take(parts);
  if (!(need_dh && need_dw)) q.dw_parts = q.parts;
  q.total = at;
  q.us *= (double)V / q.piece;
  return q;
}

Plan make_plan(int64_t n, int64_t C, int64_t V, int dtype, bool backward, bool need_dh, bool need_dw) {
  const Plan q = plan_as(false, n, C, V, dtype, backward, need_dh, need_dw);
  if (dtype != DYRA_F32) return q;
  const Plan d = plan_as(true, n, C, V, dtype, backward, need_dh, need_dw);
  return d.us < q.us ? d : q;
}

// exponents are taken in base two, so that scale / log 2 has to be a number
bool bad_scale(float scale) { return !(scale > 0.f && scale <= 0x1p126f); }

int validate(int64_t n, int64_t C, int64_t V, int dtype) {
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  if (n < 0 || n > (int64_t)1 << 20 || C <= 0 || C % 8 || C > (int64_t)1 << 17 || V <= 0 || V > (int64_t)1 << 24)
    return DYRA_ESHAPE;
  // every launch has fewer than 2^32 threads
  if (n * C >= (int64_t)1 << 33 || n * V >= (int64_t)1 << 37) return DYRA_ESHAPE;
  return DYRA_OK;
}

// The logits of a piece: rows of H (or of its planes) by rows of W from v0.
template <typename T>
Job logits_job(Operand h, const T* W, int64_t v0, int64_t cols, int64_t C, const Plan& q, char* ws,
               const int32_t* live) {
  Job j;
  if constexpr (sizeof(T) == 2) j = job(h, {W + v0 * C, 2 * C, 0, (int32_t)cols}, C, C, 1, TERMS_1, live);
  else if (q.logits == DIRECT) j = job(h, {W + v0 * C, 4 * C, 0, (int32_t)cols}, C, C, 1, 0, live);
  else j = job(h, {ws + q.wp, 2 * C, 2 * q.piece * C, (int32_t)cols}, C, C, 6, TERMS_33, live);
  j.part = reinterpret_cast<float4*>(ws + q.parts);
  return j;
}

template <typename T>
int forward_impl(const T* H, int64_t ldh, const T* W, const int32_t* targets, float scale, float* loss, float* lse,
                 int64_t n, int64_t C, int64_t V, const Plan& q, char* ws, hipStream_t st) {
  constexpr bool wide = sizeof(T) == 4;
  float2* part = reinterpret_cast<float2*>(ws + q.part);
  float* mine = reinterpret_cast<float*>(ws + q.mine);
  Operand h{H, 2 * ldh, 0, (int32_t)n};
  if constexpr (wide) h = {ws + q.hp, 2 * C, 2 * n * C, (int32_t)n};
  for (int64_t v0 = 0; v0 < V; v0 += q.piece) {
    const int64_t cols = std::min(q.piece, V - v0);
    if constexpr (wide)
      launch_planes<T>(planes(H, ldh, v0 ? 0 : n, C, ws + q.hp, n * C),
                       q.logits == DIRECT ? Planes<T>{} : planes(W + v0 * C, C, cols, C, ws + q.wp, q.piece * C), st);
    const Job j = logits_job<T>(h, W, v0, cols, C, q, ws, nullptr);
    const RowStats e{part, mine, targets, scale, (int32_t)cols, (int32_t)v0};
    if (wide && q.logits == DIRECT) launch_direct<false>(j, e, st);
    else launch_as<false, false>(q.logits, j, e, st);
  }
  hipLaunchKernelGGL(row_loss_kernel, dim3((unsigned)cdiv(n, 32)), dim3(1024), 0, st, part, mine, targets, loss, lse,
                     (int)n, (int)V, (int)cdiv(V, 64));
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

template <typename T>
int backward_impl(const T* H, int64_t ldh, const T* W, const int32_t* targets, const float* lse, const float* dloss,
                  float scale, T* dH, int64_t lddh, T* dW, int64_t n, int64_t C, int64_t V, const Plan& q, char* ws,
                  hipStream_t st) {
  constexpr int NP = planes_of<T>(), terms = NP == 3 ? 6 : 1;
  constexpr uint32_t pairs = NP == 3 ? TERMS_33 : TERMS_1;
  Found* found = reinterpret_cast<Found*>(ws + q.live);
  int32_t *live = &found->live, *map = reinterpret_cast<int32_t*>(ws + q.map);
  float* acc = reinterpret_cast<float*>(ws + q.acc);
  bf16_t* d = reinterpret_cast<bf16_t*>(ws + q.d);
  // Counting anew in each workgroup costs less than a launch up to some thousand rows,
  // us (in two launches): 8 x 1024 x 4000 41 (44), fp32 1031 x 512 x 5003 147 (150), 8192 x
  // 256 x 256 54 (58), 16384 x 4096 x 256 297 (254)
  const bool few = n <= 8192;
  const bool direct = NP == 3 && q.logits == DIRECT;
  if (!few)
    hipLaunchKernelGGL((live_kernel<T>), dim3((unsigned)(1 + (dH ? cdiv(n, 16) : 0))), dim3(1024), 0, st, targets,
                       dloss, (int)n, (int)V, found, map, dH, lddh, (int)C);
  const Operand h{ws + q.hp, 2 * C, 2 * n * C, (int32_t)n};
  for (int64_t v0 = 0; v0 < V; v0 += q.piece) {
    const int64_t cols = std::min(q.piece, V - v0), ldd = up(cols, 64);
    const Planes<T> wp = NP == 3 && !direct ? planes(W + v0 * C, C, cols, C, ws + q.wp, q.piece * C) : Planes<T>{};
    if (few && v0 == 0) {
      const int per = (int)std::min<int64_t>(64, std::max<int64_t>(1, 8192 / C)), groups = (int)cdiv(n, per);
      const int64_t grid = groups + 1 + cdiv((int64_t)wp.rows * (wp.cols / 8), 256);
      hipLaunchKernelGGL((gather_kernel<T>), dim3((unsigned)grid), dim3(256), 0, st, targets, dloss, (int)n, (int)V,
                         found, map, dH, lddh, planes(H, ldh, n, C, ws + q.hp, n * C), per, groups, wp);
    } else {
      launch_planes<T>(planes(H, ldh, v0 ? 0 : n, C, ws + q.hp, n * C, map, live), wp, st);
    }
    const Gradient<NP> e{d, ldd, n * q.piece, lse, dloss, targets, map, found, scale, (int32_t)cols,
                         (int32_t)v0};
    const Job lj = logits_job<T>(h, W, v0, cols, C, q, ws, live);
    if constexpr (NP == 3) {
      if (direct) launch_direct<false>(lj, e, st);
    }
    if (!direct) launch_as<false, false, true>(q.logits, lj, e, st);
    const bool last = v0 + cols == V, both = dH && dW && last;
    Job hj, wj;
    Store<T> he, we;
    if (dH) {
      Operand w = lj.b;   // turned: its rows are the reduction
      w.rows = (int32_t)C;
      hj = job({d, 2 * ldd, 2 * n * q.piece, (int32_t)n}, w, cols, ldd, direct ? 1 : terms, pairs, live);
      hj.part = lj.part;
      // pieces add up in fp32; the last rounds and puts the rows in their places
      const float* prior = v0 ? acc : nullptr;
      he = {dH, lddh, (int32_t)C, nullptr, prior, map, &found->weight, scale};
      const Store<float> add{acc, C, (int32_t)C, nullptr, prior, nullptr, nullptr, 1.f};
      if constexpr (NP == 3) {
        if (direct) launch_direct<true>(hj, last ? he : add, st, !both);
      }
      if (!direct && last) launch_as<false, true, true>(q.dh, hj, he, st, !both);
      else if (!direct) launch_as<false, true, true>(q.dh, hj, add, st);
    }
    if (dW) {
      Operand hr = h;   // both turned
      hr.rows = (int32_t)C;
      wj = job({d, 2 * ldd, 2 * n * q.piece, (int32_t)cols}, hr, n, n, terms, pairs, live, true);
      wj.part = reinterpret_cast<float4*>(ws + q.dw_parts);
      we = {dW + v0 * C, C, (int32_t)C, nullptr, nullptr, nullptr, &found->weight, scale};
      launch_as<true, true, true>(q.dw, wj, we, st, !both);
    }
    if (both) launch_join_two(q.dh, hj, he, q.dw, wj, we, st);
  }
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

template <typename T>
int zero(T* out, int64_t elems, hipStream_t st) {
  if (elems)
    hipLaunchKernelGGL((zero_kernel<T>), dim3((unsigned)std::min<int64_t>(cdiv(elems, 2048), 2048)), dim3(256), 0, st, out,
                       elems);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

}  // namespace

extern "C" int dyra_vocab_loss_workspace_size(int64_t n, int64_t C, int64_t V, int32_t dtype, int32_t backward,
                                              int32_t need_dh, int32_t need_dw, size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return DYRA_EINVAL;
  const int rc = validate(n, C, V, dtype);
  if (rc) return rc;
  *bytes = n ? make_plan(n, C, V, dtype, backward, need_dh, need_dw).total : 0;
  return DYRA_OK;
}

extern "C" int dyra_vocab_loss_forward(const void* H, int64_t ldh, const void* W, const int32_t* targets, float scale,
                                       float* loss, float* lse, int64_t n, int64_t C, int64_t V, int32_t dtype,
                                       void* workspace, size_t ws_bytes, void* stream) {
  const int rc = validate(n, C, V, dtype);
  if (rc) return rc;
  if (bad_scale(scale)) return DYRA_EINVAL;
  if (n == 0) return DYRA_OK;
  if (!H || !W || !targets || !loss || !lse || !workspace) return DYRA_EINVAL;
  if (misaligned(H, 15) || misaligned(W, 15) || misaligned(workspace, 15) || misaligned(targets, 3) ||
      misaligned(loss, 3) || misaligned(lse, 3))
    return DYRA_EINVAL;
  if (bad_stride(ldh, C, dtype)) return DYRA_ESHAPE;
  const Plan q = make_plan(n, C, V, dtype, false, false, false);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == DYRA_BF16)
    return forward_impl(reinterpret_cast<const bf16_t*>(H), ldh, reinterpret_cast<const bf16_t*>(W), targets, scale,
                        loss, lse, n, C, V, q, ws, st);
  return forward_impl(reinterpret_cast<const float*>(H), ldh, reinterpret_cast<const float*>(W), targets, scale, loss,
                      lse, n, C, V, q, ws, st);
}

extern "C" int dyra_vocab_loss_backward(const void* H, int64_t ldh, const void* W, const int32_t* targets,
                                        const float* lse, const float* dloss, float scale, void* dH, int64_t lddh,
                                        void* dW, int64_t n, int64_t C, int64_t V, int32_t dtype, void* workspace,
                                        size_t ws_bytes, void* stream) {
  const int rc = validate(n, C, V, dtype);
  if (rc) return rc;
  if (bad_scale(scale) || (!dH && !dW)) return DYRA_EINVAL;
  if (misaligned(dW, 15)) return DYRA_EINVAL;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (n == 0) {
    if (!dW) return DYRA_OK;
    return dtype == DYRA_BF16 ? zero(reinterpret_cast<bf16_t*>(dW), V * C, st)
                              : zero(reinterpret_cast<float*>(dW), V * C, st);
  }
  if (!H || !W || !targets || !lse || !dloss || !workspace) return DYRA_EINVAL;
  if (misaligned(H, 15) || misaligned(W, 15) || misaligned(dH, 15) || misaligned(workspace, 15) ||
      misaligned(targets, 3) || misaligned(lse, 3) || misaligned(dloss, 3))
    return DYRA_EINVAL;
  if (bad_stride(ldh, C, dtype) || (dH && bad_stride(lddh, C, dtype))) return DYRA_ESHAPE;
  const Plan q = make_plan(n, C, V, dtype, true, dH != nullptr, dW != nullptr);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  if (dtype == DYRA_BF16)
    return backward_impl(reinterpret_cast<const bf16_t*>(H), ldh, reinterpret_cast<const bf16_t*>(W), targets, lse,
                         dloss, scale, reinterpret_cast<bf16_t*>(dH), lddh, reinterpret_cast<bf16_t*>(dW), n, C, V, q,
                         ws, st);
  return backward_impl(reinterpret_cast<const float*>(H), ldh, reinterpret_cast<const float*>(W), targets, lse, dloss,
                       scale, reinterpret_cast<float*>(dH), lddh, reinterpret_cast<float*>(dW), n, C, V, q, ws, st);
}
