// Softmax cross entropy over a vocabulary, from hidden rows H [n][C] and a
// head W [V][C], without the logits in memory:
//   a_tv = scale H_t . W_v,  lse_t = log sum_v exp a_tv,  loss_t = lse_t - a_t,target
//   d_tv = scale dloss_t (exp(a_tv - lse_t) - [v = target_t])
//   dH = d W,  dW = d^T H
//
// Forward: one product whose epilogue leaves, for each row and tile of
// columns, the maximum and the sum of exponentials below it; a second launch
// joins them.  Backward: for one piece of the vocabulary after the other the
// logits are multiplied again, d goes to memory as bf16 (row by row for dH,
// transposed for dW, so that both products find their reduction axis
// contiguous), and the two gradients are products of the piece.  The pieces
// keep d within what the last-level cache holds.
//
// bf16: logits are sums of exact products in fp32; d is rounded to bf16 for
// the two products of the backward pass (2^-9 of each term, below the
// rounding of the gradients, which are bf16).  fp32: every operand is three
// bf16 planes (24 bits), a product the six pairs of planes that reach 2^-24.
#include <cmath>

#include "mfma_product.h"

namespace {

using namespace product;

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// The tile's part of each row's softmax, in powers of two: maximum m and
// sum of 2^(a - m) over its columns; the target's logit where it lies here.
struct RowStats {
  float2* part;             // [tiles of columns][rows]
  float* mine;              // [rows] logit of the target
  const int32_t* targets;
  float scale;
  int32_t rows, cols;       // of H, of this piece of W
  int32_t v0, t0;           // first column and tile of the piece

  template <class C>
  __device__ __forceinline__ void operator()(Acc<C>& acc, char* lds, int m0, int n0, int, int wm, int wn) const {
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    const float k2 = scale * LOG2E;
    float2* st = reinterpret_cast<float2*>(lds);
    const int c0 = n0 + wn * C::WN;
    const bool edge = c0 + C::WN > cols;
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
      const int rr = wm * C::WM + fm * 32 + l, row = m0 + rr;
      const int at = (int)((unsigned)(row < rows ? targets[row] : -1) - (unsigned)(v0 + c0));
      const bool has = c0 < cols && (unsigned)at < (unsigned)min(C::WN, cols - c0) && (at >> 2 & 1) == g;
      if (__any(has)) {
#pragma unroll
        for (int i = 0; i < 16 * C::FN; ++i)
          if (has && i == ((at >> 5) * 16 + (at >> 3 & 3) * 4 + (at & 3))) mine[row] = acc[fm][i / 16][i % 16] * scale;
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < 16 * C::FN; ++i)
          if (c0 + i / 16 * 32 + (i % 16 / 4) * 8 + 4 * g + i % 4 >= cols) acc[fm][i / 16][i % 16] = -INFINITY;
      }
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i) top = fmaxf(top, acc[fm][i / 16][i % 16]);
      top = fmaxf(top, __shfl_xor(top, 32));
      // nothing above -inf: exponents are taken from 0, so that a NaN stays
      const float m2 = top == -INFINITY ? 0.f : top * k2;
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i) sum += __builtin_amdgcn_exp2f(fmaf(acc[fm][i / 16][i % 16], k2, -m2));
      sum += __shfl_xor(sum, 32);
      if (g == 0) st[rr * C::NWN + wn] = make_float2(top == -INFINITY ? -INFINITY : m2, sum);
    }
    __syncthreads();
    for (int rr = threadIdx.x; rr < C::BM; rr += C::NT) {
      if (m0 + rr >= rows) break;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < C::NWN; ++i) top = fmaxf(top, st[rr * C::NWN + i].x);
#pragma unroll
      for (int i = 0; i < C::NWN; ++i) {
        const float2 s = st[rr * C::NWN + i];
        sum += s.x == -INFINITY ? s.y : s.y * __builtin_amdgcn_exp2f(s.x - top);   // an empty sum is 0, or NaN
      }
      part[(int64_t)(t0 + n0 / C::BN) * rows + m0 + rr] = make_float2(top, sum);
    }
  }
};

// Joins a row's parts: 32 rows a workgroup, eight lanes a row.
__global__ __launch_bounds__(256) void row_loss_kernel(const float2* __restrict__ part, const float* __restrict__ mine,
                                                       const int32_t* __restrict__ targets, float* __restrict__ loss,
                                                       float* __restrict__ lse, int rows, int vocab, int tiles) {
  __shared__ float2 st[8][32];
  const int rr = threadIdx.x & 31, k = threadIdx.x >> 5, row = blockIdx.x * 32 + rr;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 s) {
    const float t = fmaxf(top, s.x);
    sum = (top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f(top - t)) +
          (s.x == -INFINITY ? s.y : s.y * __builtin_amdgcn_exp2f(s.x - t));
    top = t;
  };
  if (row < rows) {
#pragma unroll 8
    for (int t = k; t < tiles; t += 8) join(part[(int64_t)t * rows + row]);
  }
  st[k][rr] = make_float2(top, sum);
  __syncthreads();
  if (k || row >= rows) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) join(st[i][rr]);
  const float all = top == -INFINITY ? logf(sum) : fmaf(top, LN2, logf(sum));
  lse[row] = all;
  const int t = targets[row];
  loss[row] = t >= 0 && t < vocab ? all - mine[row] : 0.f;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// d of the tile, in NP bf16 planes, row by row and transposed.  Columns past
// the piece's and rows past n are zero up to the padded sizes.
template <int NP>
struct Gradient {
  bf16_t *d, *dt;               // [NP][rows][ldd], [NP][cols][ldt]; null: not wanted
  int64_t ldd, ldt, plane, plane_t;
  const float *lse, *dloss;
  const int32_t* targets;
  float scale;
  int32_t rows, cols, vocab;    // of H, of this piece, in all
  int32_t v0;

  template <class C>
  __device__ __forceinline__ void operator()(Acc<C>& acc, char* lds, int m0, int n0, int, int wm, int wn) const {
    static_assert(C::BM * C::BN * 2 <= C::LDS && C::BN % 128 == 0, "the tile fits the ring");
    constexpr int CPR = C::BN / 8;
    const int lane = threadIdx.x & 63, l = lane & 31, g = lane >> 5;
    const float k2 = scale * LOG2E;
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
      const int row = m0 + wm * C::WM + fm * 32 + l;
      const int target = row < rows ? targets[row] : -1;
      const bool live = target >= 0 && target < vocab;
      const float w = live ? dloss[row] * scale : 0.f, l2 = live ? -lse[row] * LOG2E : 0.f;
      const int at = target - v0 - n0 - wn * C::WN - 4 * g;
#pragma unroll
      for (int i = 0; i < 16 * C::FN; ++i) {
        const int c = i / 16 * 32 + (i % 16 / 4) * 8 + i % 4;
        const float p = __builtin_amdgcn_exp2f(fmaf(acc[fm][i / 16][i % 16], k2, l2)) - (c == at ? 1.f : 0.f);
        acc[fm][i / 16][i % 16] = live && n0 + wn * C::WN + 4 * g + c < cols ? w * p : 0.f;
      }
    }
    const int valid = min(C::BM, rows - m0), padded = min(C::BM, (int)ldt - m0), wide = min(C::BN, (int)ldd - n0);
#pragma unroll
    for (int t = 0; t < NP; ++t) {
      if (t) __syncthreads();   // the plane before has been copied out
#pragma unroll
      for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = 4 * q + 2 * e;
              h[e] = pack_bf16x2(acc[fm][fn][i], acc[fm][fn][i + 1]);
              if constexpr (NP > 1) {   // the rest is the next plane's
                acc[fm][fn][i] -= __uint_as_float(h[e] << 16);
                acc[fm][fn][i + 1] -= __uint_as_float(h[e] & 0xffff0000u);
              }
            }
            const int row = wm * C::WM + fm * 32 + l, col = wn * C::WN + fn * 32 + 8 * q + 4 * g;
            *reinterpret_cast<uint2*>(lds + tile_at(row, col / 8, CPR) + 8 * g) = make_uint2(h[0], h[1]);
          }
      __syncthreads();
      if (d) tile_rows<C::BM, C::BN, C::NT>(lds, d + t * plane + (int64_t)m0 * ldd + n0, ldd, valid, wide);
      if (dt) tile_transposed<C::BM, C::BN, C::NT>(lds, dt + t * plane_t + (int64_t)n0 * ldt + m0, ldt, padded, wide);
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

// Sizes of a call.
struct Plan {
  int64_t np, nrow;                     // n padded
  int64_t piece, pieces;                // columns of the vocabulary at a time
  Pick logits, dh, dw;
  int64_t tiles;                        // forward: tiles of columns in all
  bool direct;                          // dH needs no fp32 parts
  size_t part, mine, hp, ht, wp, wt, d, dt, acc, total;
};

Plan make_plan(int64_t n, int64_t C, int64_t V, int dtype, bool backward, bool need_dh, bool need_dw) {
  Plan q{};
  const bool wide = dtype == DYRA_F32;
  q.np = wide ? 3 : 1;
  const int terms = wide ? 6 : 1;
  q.nrow = up(std::max<int64_t>(n, 1), 64);
  // d of a piece, both ways, is at most 2^26 elements a plane pair (256 MB in
  // bf16, the last-level cache); planes of fp32 weights at most 2^28
  int64_t most = V;
  if (backward) most = std::min<int64_t>(most, ((int64_t)1 << 26) / q.nrow);
  if (wide) most = std::min<int64_t>(most, ((int64_t)1 << 28) / (3 * C));
  most = std::max<int64_t>(256, most & ~(int64_t)255);
  q.pieces = cdiv(V, most);
  q.piece = std::min(up(V, 64), up(cdiv(V, q.pieces), 256));
  q.pieces = cdiv(V, q.piece);
  const int64_t step = cdiv(C, 64);
  q.logits = pick(n, q.piece, terms * step, false);
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (wide) {
    q.hp = take(2 * q.np * n * C);
    q.wp = take(2 * q.np * q.piece * C);
  }
  if (!backward) {
    q.tiles = (q.pieces - 1) * cdiv(q.piece, tile_cols(q.logits.shape)) +
              cdiv(V - (q.pieces - 1) * q.piece, tile_cols(q.logits.shape));
    q.part = take(8 * q.tiles * n);
    q.mine = take(4 * n);
  } else {
    if (need_dh) {
      q.dh = pick(n, C, terms * cdiv(q.piece, 64), true);
      q.direct = q.pieces == 1 && q.dh.split == 1;
      q.wt = take(2 * q.np * C * q.piece);
      q.d = take(2 * q.np * n * q.piece);
      if (!q.direct) q.acc = take(4 * q.dh.split * n * C);
    }
    if (need_dw) {
      q.dw = pick(q.piece, C, terms * cdiv(q.nrow, 64), false);
      q.ht = take(2 * q.np * C * q.nrow);
      q.dt = take(2 * q.np * q.piece * q.nrow);
    }
  }
  q.total = at;
  return q;
}

int validate(int64_t n, int64_t C, int64_t V, int dtype) {
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  if (n < 0 || n > (int64_t)1 << 20 || C <= 0 || C % 8 || C > (int64_t)1 << 17 || V <= 0 || V > (int64_t)1 << 24)
    return DYRA_ESHAPE;
  // every launch has fewer than 2^32 threads
  if (n * C >= (int64_t)1 << 33 || n * V >= (int64_t)1 << 37) return DYRA_ESHAPE;
  return DYRA_OK;
}

// The operands of the logits of a piece: H and W rows from v0.
template <typename T>
Job logits_job(const T* H, int64_t ldh, const T* W, int64_t v0, int64_t cols, int64_t n, int64_t C, const Plan& q,
               char* ws) {
  if constexpr (sizeof(T) == 2)
    return job({H, 2 * ldh, 0, (int32_t)n}, {W + v0 * C, 2 * C, 0, (int32_t)cols}, C, 1, TERMS_1);
  else
    return job({ws + q.hp, 2 * C, 2 * n * C, (int32_t)n}, {ws + q.wp, 2 * C, 2 * q.piece * C, (int32_t)cols}, C, 6,
               TERMS_33);
}

template <typename T>
int forward_impl(const T* H, int64_t ldh, const T* W, const int32_t* targets, float scale, float* loss, float* lse,
                 int64_t n, int64_t C, int64_t V, const Plan& q, char* ws, hipStream_t st) {
  constexpr bool wide = sizeof(T) == 4;
  float2* part = reinterpret_cast<float2*>(ws + q.part);
  float* mine = reinterpret_cast<float*>(ws + q.mine);
  if constexpr (wide)
    launch_planes<T>(H, ldh, n, C, reinterpret_cast<bf16_t*>(ws + q.hp), nullptr, 0, n * C, 0, nullptr, 0, st);
  int64_t t0 = 0;
  for (int64_t v0 = 0; v0 < V; v0 += q.piece) {
    const int64_t cols = std::min(q.piece, V - v0);
    if constexpr (wide)
      launch_planes<T>(W + v0 * C, C, cols, C, reinterpret_cast<bf16_t*>(ws + q.wp), nullptr, 0, q.piece * C, 0,
                       nullptr, 0, st);
    const RowStats e{part, mine, targets, scale, (int32_t)n, (int32_t)cols, (int32_t)v0, (int32_t)t0};
    launch_as(q.logits, logits_job<T>(H, ldh, W, v0, cols, n, C, q, ws), e, st);
    t0 += cdiv(cols, tile_cols(q.logits.shape));
  }
  hipLaunchKernelGGL(row_loss_kernel, dim3((unsigned)cdiv(n, 32)), dim3(256), 0, st, part, mine, targets, loss, lse,
                     (int)n, (int)V, (int)q.tiles);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

template <typename T>
int backward_impl(const T* H, int64_t ldh, const T* W, const int32_t* targets, const float* lse, const float* dloss,
                  float scale, T* dH, int64_t lddh, T* dW, int64_t n, int64_t C, int64_t V, const Plan& q, char* ws,
                  hipStream_t st) {
  constexpr int NP = planes_of<T>(), terms = NP == 3 ? 6 : 1;
  constexpr uint32_t pairs = NP == 3 ? TERMS_33 : TERMS_1;
  auto at = [&](size_t o) { return reinterpret_cast<bf16_t*>(ws + o); };
  bf16_t* hp = NP == 3 ? at(q.hp) : nullptr;
  bf16_t* ht = dW ? at(q.ht) : nullptr;
  if (hp || ht)
    launch_planes<T>(H, ldh, n, C, hp, ht, q.nrow, n * C, C * q.nrow, targets, V, st);
  for (int64_t v0 = 0; v0 < V; v0 += q.piece) {
    const int64_t cols = std::min(q.piece, V - v0);
    bf16_t* wp = NP == 3 ? at(q.wp) : nullptr;
    bf16_t* wt = dH ? at(q.wt) : nullptr;
    if (wp || wt)
      launch_planes<T>(W + v0 * C, C, cols, C, wp, wt, up(cols, 64), q.piece * C, C * q.piece, nullptr, 0, st);
    const int64_t ldd = up(cols, 64);
    const Gradient<NP> e{dH ? at(q.d) : nullptr, dW ? at(q.dt) : nullptr, ldd, q.nrow, n * q.piece,
                         q.piece * q.nrow, lse, dloss, targets, scale, (int32_t)n, (int32_t)cols, (int32_t)V,
                         (int32_t)v0};
    launch_as(q.logits, logits_job<T>(H, ldh, W, v0, cols, n, C, q, ws), e, st);
    if (dH) {
      const Job j = job({at(q.d), 2 * ldd, 2 * n * q.piece, (int32_t)n}, {wt, 2 * ldd, 2 * C * q.piece, (int32_t)C}, ldd,
                        terms, pairs);
      if (q.direct) {
        launch_as(q.dh, j, Store<T>{dH, lddh, 0, (int32_t)n, (int32_t)C, nullptr, 0}, st);
      } else {
        launch_as(q.dh, j, Store<float>{reinterpret_cast<float*>(ws + q.acc), C, n * C, (int32_t)n, (int32_t)C, nullptr,
                                        v0 > 0}, st);
      }
    }
    if (dW) {
      const Job j = job({at(q.dt), 2 * q.nrow, 2 * q.piece * q.nrow, (int32_t)cols},
                        {ht, 2 * q.nrow, 2 * C * q.nrow, (int32_t)C}, q.nrow, terms, pairs);
      launch_as(q.dw, j, Store<T>{dW + v0 * C, C, 0, (int32_t)cols, (int32_t)C, nullptr, 0}, st);
    }
  }
  if (dH && !q.direct)
    hipLaunchKernelGGL((parts_kernel<T>), dim3((unsigned)cdiv(n * (C / 4), 256)), dim3(256), 0, st,
                       reinterpret_cast<const float*>(ws + q.acc), n * C, q.dh.split, dH, lddh, n, (int)C,
                       (const T*)nullptr);
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
  if (!(scale > 0.f) || !std::isfinite(scale)) return DYRA_EINVAL;
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
  if (!(scale > 0.f) || !std::isfinite(scale) || (!dH && !dW)) return DYRA_EINVAL;
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
