// The norms before and after a block, fused with its gate and residual scale,
// on gfx950.  Per row, with y the block's output and x the residual stream:
//   u  = post(y),  x' = alpha x + g * u,  z = pre(x')
// post is the identity, an RMS norm or a layer norm with weight and bias, pre
// an RMS or layer norm; the gate g is absent, one vector, or one vector per
// request.  Backward, from dz and the gradient dx' that reaches x' directly:
//   d = dx' + pre^T(dz),  dx = alpha d,  du = g * d,  dy = post^T(du)
//   dg = sum over rows of d * u, and the weights' and biases' column sums.
//
// Forward moves 4 rows, backward 6, for some tens of operations an element:
// memory bounds both where a row and the column sums fit the registers.  A row
// stays there from its load to its store (fp32, rounded once), so each operand
// crosses memory once.  Measured, bf16:
// forward 32928 x 1024 (layer norm, channel gate) 44 us, 6.1 TB/s; its
// backward 74 + 5 us for the joined column sums, 5.1 TB/s; backward 4099 x
// 4096 (both norms, a gate per request) 44 + 5 us, 4.1 TB/s.  A copy of the
// first size runs at 5.2 TB/s, of 2 GiB at 4.85.
// The widest rows spill, and then the spills bound them.  Forward: fp32 above
// 8192 columns 115 registers (1000 x 16384 with all parameters 102 us, 2.6
// TB/s), bf16 12 (1500 x 12288 41 us, 3.6 TB/s).  Backward: see its kernel.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/dyra.h"
#include "device_common.h"
#include "spec.h"

using namespace dyra_spec_util;

namespace {

constexpr int MAX_C = 16384;   // 16 waves of 64 lanes, two 8-element chunks each

struct NormArgs {
  const void *x, *y, *dz, *dxn;   // forward: x, y; backward: x', y, dz, dx' (dxn may be null)
  void *o0, *o1;                  // forward: x', z; backward: dx, dy
  const void *pw, *pb, *qw, *qb;  // pre weight / bias, post weight / bias, or null
  const void* gate;
  const int32_t* off;             // requests' offsets, gate per request only
  float *part, *gpart, *dgate;    // backward: column partials, gate partials, per-request gate gradient
  int64_t n;
  int32_t c, B, pre, post, per_request;
  int32_t rows;                   // consecutive rows of a row group
  float eps, alpha;
};

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load8(const void* base, int64_t at, bool live) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    r.v[i] = live ? reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(base) + at)[i] : zero4();
  return r;
}

// load8 of rows that the backward pass reads once (non-temporal): 32928 x 1024
// in bf16 goes from 75 to 65 us (with a gate 85 to 73), 4099 x 4096 in fp32
// from 90 to 87; between, the two are within 3 us of each other (6263 x 4232:
// 55 and 56.5).  In the forward pass it changes nothing, and non-temporal
// stores cost either pass 4 to 8 us.
template <typename T>
__device__ __forceinline__ Raw<T> load8_once(const void* base, int64_t at, bool live) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    r.v[i] = live ? __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(reinterpret_cast<const T*>(base) + at) + i))
                  : zero4();
  return r;
}

// A parameter vector's chunk, `other` everywhere where there is none.
template <typename T>
__device__ __forceinline__ Raw<T> load_param(const void* base, int64_t at, bool live, uint32_t other) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(other, other, other, other);
  return base ? load8<T>(base, at, live) : r;
}
template <typename T> constexpr uint32_t ones() { return sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u; }

// Element e of a chunk as fp32.
template <typename T>
__device__ __forceinline__ float elem(const Raw<T>& r, int e) {
  const uint4& u = r.v[sizeof(T) == 2 ? 0 : e >> 2];
  const int w = sizeof(T) == 2 ? e >> 1 : e & 3;
  const uint32_t x = w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
  if constexpr (sizeof(T) == 2) return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
  else return __uint_as_float(x);
}

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f2bf(v[2 * i]) | (uint32_t)f2bf(v[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(reinterpret_cast<bf16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// v of the lane that a DPP control names (row_mask: the 16-lane rows that
// take part; the others add 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}

// The sum over a wave, in every lane: within quads, halves of 16 and 16 by
// permutations, then across the four rows of 16 to lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xb1, 0xf>(v);    // quad_perm 1 0 3 2
  v += dpp<0x4e, 0xf>(v);    // quad_perm 2 3 0 1
  v += dpp<0x141, 0xf>(v);   // row_half_mirror
  v += dpp<0x140, 0xf>(v);   // row_mirror
  v += dpp<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
  v += dpp<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums K values over a row's WPR waves.  Every lane gets the sums.  With
// several waves the partial sums meet in LDS; two alternating buffers leave
// one barrier per call.  All row groups of the workgroup call it together.
template <int WPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& flip) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6, first = wave / WPR * WPR;
    float* buf = lds + flip * (16 * 4);
    flip ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) buf[wave * 4 + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s += buf[(first + w) * 4 + k];
      v[k] = s;
    }
  }
}

// The request of a row, going on from that of an earlier row of the group.
struct RequestWalk {
  const int32_t* off;
  int B, b;
  int64_t next;   // first row past request b
  __device__ __forceinline__ void load_next() { next = b + 1 < B ? off[b + 1] : INT64_MAX; }
  __device__ __forceinline__ void start(int64_t row) {   // the last request that starts at or before `row`
    int a = 0, z = B;
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (off[mid] <= row) a = mid;
      else z = mid;
    }
    b = a;
    load_next();
  }
  __device__ __forceinline__ void advance(int64_t row) {
    while (next <= row) {
      ++b;
      load_next();
    }
  }
};

constexpr int LAYER = DYRA_NORM_LAYER;

// Statistics of a row held as NCH chunks: mean (0 for RMS) and 1 / deviation.
// The layer norm's squares are taken about the mean, in a second pass over
// the registers: E[v^2] - mean^2 would cancel where the mean is large.
template <int WPR, int NCH>
__device__ __forceinline__ void row_stats(const float (&v)[NCH][8], const bool (&live)[NCH], int kind, float inv_c,
                                          float eps, float& mean, float& inv, float* lds, int& flip) {
  mean = 0.f;
  if (kind == LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int h = 0; h < NCH; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += live[h] ? v[h][e] : 0.f;
    row_sum<WPR>(s, lds, flip);
    mean = s[0] * inv_c;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int h = 0; h < NCH; ++h) {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = v[h][e] - mean;
      t += d * d;
    }
    s[0] += live[h] ? t : 0.f;
  }
  row_sum<WPR>(s, lds, flip);
  inv = rsqrtf(s[0] * inv_c + eps);
}

// WPR waves a row, NCH chunks of 8 elements a lane, RPB row groups a
// workgroup; a row group takes `rows` consecutive rows.  The next row is in
// flight while the present one is worked on, and the parameters stay in
// registers as they lie.
template <typename T, int WPR, int NCH, int RPB>
__global__ __launch_bounds__(WPR * RPB * 64) void norm_forward_kernel(NormArgs p) {
  __shared__ float lds[2 * 16 * 4];
  int flip = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / WPR, t = (wave % WPR) * 64 + (threadIdx.x & 63);
  const int64_t r0 = ((int64_t)blockIdx.x * RPB + group) * p.rows;
  const float inv_c = 1.f / (float)p.c;
  int at[NCH];
  bool live[NCH];
  Raw<T> pw[NCH], pb[NCH], qw[NCH], qb[NCH], gt[NCH], xr[NCH], yr[NCH];
  RequestWalk w{p.off, p.B, 0, 0};
  if (p.per_request) w.start(r0);
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const bool ok = live[h] && row < p.n;
      xr[h] = load8<T>(p.x, row * p.c + at[h], ok);
      yr[h] = load8<T>(p.y, row * p.c + at[h], ok);
    }
  };
  auto load_gate = [&] {
#pragma unroll
    for (int h = 0; h < NCH; ++h) gt[h] = load_param<T>(p.gate, (int64_t)w.b * p.c + at[h], live[h], ones<T>());
  };
#pragma unroll
  for (int h = 0; h < NCH; ++h) {
    at[h] = 8 * (t + h * WPR * 64);
    live[h] = at[h] < p.c;
  }
  load_row(r0);
  load_gate();
#pragma unroll
  for (int h = 0; h < NCH; ++h) {
    pw[h] = load_param<T>(p.pw, at[h], live[h], ones<T>());
    pb[h] = load_param<T>(p.pb, at[h], live[h], 0u);
    qw[h] = load_param<T>(p.qw, at[h], live[h], ones<T>());
    qb[h] = load_param<T>(p.qb, at[h], live[h], 0u);
  }
  for (int k = 0; k < p.rows; ++k) {   // the same count in every row group: row_sum has barriers
    const int64_t row = r0 + k;
    const bool in = row < p.n;
    if (WPR == 1 && !in) break;
    if (p.per_request && in && w.next <= row) {
      w.advance(row);
      load_gate();
    }
    float x[NCH][8], y[NCH][8];
#pragma unroll
    for (int h = 0; h < NCH; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[h][e] = elem<T>(xr[h], e);
        y[h][e] = elem<T>(yr[h], e);
      }
    if (k + 1 < p.rows) load_row(row + 1);
    if (p.post != DYRA_NORM_NONE) {
      float mean, inv;
      row_stats<WPR, NCH>(y, live, p.post, inv_c, p.eps, mean, inv, lds, flip);
#pragma unroll
      for (int h = 0; h < NCH; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[h][e] = (y[h][e] - mean) * inv * elem<T>(qw[h], e) + elem<T>(qb[h], e);
    }
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[h][e] = p.alpha * x[h][e] + elem<T>(gt[h], e) * y[h][e];
      if (in && live[h]) store8<T>(p.o0, row * p.c + at[h], x[h]);
    }
    float mean, inv;
    row_stats<WPR, NCH>(x, live, p.pre, inv_c, p.eps, mean, inv, lds, flip);
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[h][e] = (x[h][e] - mean) * inv * elem<T>(pw[h], e) + elem<T>(pb[h], e);
      if (in && live[h]) store8<T>(p.o1, row * p.c + at[h], x[h]);
    }
  }
}

// Column sums a backward pass keeps: pre weight, pre bias, post weight, post
// bias, gate (in that order among those present).
enum { HAS_POST = 1, HAS_GATE = 2, HAS_BIAS = 4 };
constexpr int vectors(int f) {
  return 1 + (f & HAS_BIAS ? 1 : 0) + (f & HAS_POST ? (f & HAS_BIAS ? 2 : 1) : 0) + (f & HAS_GATE ? 1 : 0);
}

// Per row: d = dx' + inv (t - mean(t) - xhat mean(t xhat)), t = dz * weight
// (mean(t) for the layer norm only), likewise for dy through post.  The sums
// of both norms' statistics are taken together.  Column sums stay in
// registers over the group's rows, meet in LDS over the workgroup's row
// groups and go to one partial row a workgroup: no atomics, a fixed order.
// With 16 waves a row (128 registers a lane) sums and row do not fit, and with
// a post norm, gate and biases together (256) nearly; the spills go through the
// caches and bound these.  Spilled registers and times with a post norm, gate
// and biases | without: bf16 512 to 8192 columns 28 - 44 | 0, 4099 x 4096 105 us
// (49 without the biases); bf16 above 8192 267 | 29, 1500 x 12288 414 | 77 us;
// fp32 above 4096 137 | 0, 2000 x 8192 195 | 75 us; above 8192 404 | 54, 1000 x
// 16384 379 | 106 us.
// As forward, the next row is in flight while the present one is worked on
// (but for the widest rows, whose registers do not hold both).
template <typename T, int WPR, int NCH, int RPB, int F>
__global__ __launch_bounds__(WPR * RPB * 64, WPR == 16 ? 4 : 2) void norm_backward_kernel(NormArgs p) {
  constexpr int V = vectors(F);
  constexpr bool POST = F & HAS_POST, GATE = F & HAS_GATE, BIAS = F & HAS_BIAS, AHEAD = WPR < 16;
  constexpr int I_PB = 1, I_QW = 1 + BIAS, I_QB = I_QW + 1, I_G = V - 1;
  __shared__ float lds[2 * 16 * 4];
  __shared__ float meet[RPB > 1 ? (RPB - 1) * WPR * 64 * 8 : 1];
  int flip = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / WPR, t = (wave % WPR) * 64 + (threadIdx.x & 63);
  const int64_t gid = (int64_t)blockIdx.x * RPB + group, r0 = gid * p.rows;
  const float inv_c = 1.f / (float)p.c;
  const bool per_request = GATE && p.per_request;
  int at[NCH];
  bool live[NCH];
#pragma unroll
  for (int h = 0; h < NCH; ++h) {
    at[h] = 8 * (t + h * WPR * 64);
    live[h] = at[h] < p.c;
  }
  float acc[V][NCH][8] = {};
  RequestWalk w{p.off, p.B, 0, 0};
  if (per_request) w.start(r0);
  const int first = w.b;
  Raw<T> xr[NCH], zr[NCH], dr[NCH], yr[NCH], pw[NCH], qw[NCH], qb[NCH], gt[NCH];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const int64_t a = row * p.c + at[h];
      const bool ok = live[h] && row < p.n;
      xr[h] = load8_once<T>(p.x, a, ok);
      zr[h] = load8_once<T>(p.dz, a, ok);
      dr[h] = load8_once<T>(p.dxn, a, ok && p.dxn);
      if constexpr (POST || GATE) yr[h] = load8_once<T>(p.y, a, ok);
    }
  };
  auto load_gate = [&] {
#pragma unroll
    for (int h = 0; h < NCH; ++h) gt[h] = load8<T>(p.gate, (int64_t)w.b * p.c + at[h], live[h]);
  };
  if constexpr (AHEAD) load_row(r0);
#pragma unroll
  for (int h = 0; h < NCH; ++h) {
    pw[h] = load_param<T>(p.pw, at[h], live[h], ones<T>());
    if constexpr (POST) qw[h] = load_param<T>(p.qw, at[h], live[h], ones<T>());
    if constexpr (POST && GATE && BIAS) qb[h] = load_param<T>(p.qb, at[h], live[h], 0u);
  }
  if constexpr (GATE) load_gate();
  for (int k = 0; k < p.rows; ++k) {
    const int64_t row = r0 + k;
    const bool in = row < p.n;
    if (WPR == 1 && !in) break;
    if constexpr (GATE) {
      if (per_request && in && w.next <= row) {
        // request w.b ends: the group's first one may have begun in an earlier
        // group and goes to a partial row, any other lies in this group whole
        float* to = w.b == first ? p.gpart + gid * 2 * p.c : p.dgate + (int64_t)w.b * p.c;
#pragma unroll
        for (int h = 0; h < NCH; ++h) {
          if (live[h]) store8<float>(to, at[h], acc[I_G][h]);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[I_G][h][e] = 0.f;
        }
        w.advance(row);
        load_gate();
      }
    }
    if constexpr (!AHEAD) load_row(row);
    float x[NCH][8], dz[NCH][8], d[NCH][8], y[NCH][8];
#pragma unroll
    for (int h = 0; h < NCH; ++h)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[h][e] = elem<T>(xr[h], e);
        dz[h][e] = elem<T>(zr[h], e);
        d[h][e] = elem<T>(dr[h], e);
        if constexpr (POST || GATE) y[h][e] = elem<T>(yr[h], e);
      }
    if constexpr (AHEAD)
      if (k + 1 < p.rows) load_row(row + 1);
    // means, where a layer norm needs them (idle lanes hold zeros)
    float s1[3] = {0.f, 0.f, 0.f};   // x', t, y
    if (p.pre == LAYER || (POST && p.post == LAYER)) {
#pragma unroll
      for (int h = 0; h < NCH; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s1[0] += x[h][e];
          s1[1] += dz[h][e] * elem<T>(pw[h], e);
          if constexpr (POST) s1[2] += y[h][e];
        }
      row_sum<WPR>(s1, lds, flip);
    }
    const float mx = p.pre == LAYER ? s1[0] * inv_c : 0.f, mt = p.pre == LAYER ? s1[1] * inv_c : 0.f;
    const float my = POST && p.post == LAYER ? s1[2] * inv_c : 0.f;
    float s2[3] = {0.f, 0.f, 0.f};   // (x' - mean)^2, t (x' - mean), (y - mean)^2
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[h][e] -= mx;
        a += x[h][e] * x[h][e];
        s2[1] += dz[h][e] * elem<T>(pw[h], e) * x[h][e];
        if constexpr (POST) {
          y[h][e] -= my;
          b += y[h][e] * y[h][e];
        }
      }
      s2[0] += live[h] ? a : 0.f;
      s2[2] += live[h] ? b : 0.f;
    }
    row_sum<WPR>(s2, lds, flip);
    // past the last row everything is zero, whatever eps
    const float inv = in ? rsqrtf(s2[0] * inv_c + p.eps) : 0.f, proj = s2[1] * inv * inv_c;
    const float iy = POST && in ? rsqrtf(s2[2] * inv_c + p.eps) : 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hat = x[h][e] * inv;
        acc[0][h][e] += dz[h][e] * hat;
        if constexpr (BIAS) acc[I_PB][h][e] += dz[h][e];
        float v = d[h][e] + inv * (dz[h][e] * elem<T>(pw[h], e) - mt - hat * proj);
        o[e] = p.alpha * v;
        if constexpr (POST) y[h][e] *= iy;   // normalised y
        if constexpr (GATE) {
          float u = y[h][e];
          if constexpr (POST) u *= elem<T>(qw[h], e);
          if constexpr (POST && BIAS) u += elem<T>(qb[h], e);
          acc[I_G][h][e] += v * u;           // v is 0 past the last row
          v *= elem<T>(gt[h], e);
        }
        if constexpr (POST) {
          acc[I_QW][h][e] += v * y[h][e];
          if constexpr (BIAS) acc[I_QB][h][e] += v;
          v *= elem<T>(qw[h], e);
        }
        d[h][e] = v;
      }
      if (in && live[h]) store8<T>(p.o0, row * p.c + at[h], o);
    }
    if constexpr (POST) {
      float s3[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < NCH; ++h) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a += d[h][e];
          b += d[h][e] * y[h][e];
        }
        s3[0] += live[h] ? a : 0.f;
        s3[1] += live[h] ? b : 0.f;
      }
      row_sum<WPR>(s3, lds, flip);
      const float m = p.post == LAYER ? s3[0] * inv_c : 0.f, q = s3[1] * inv_c;
#pragma unroll
      for (int h = 0; h < NCH; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[h][e] = iy * (d[h][e] - m - y[h][e] * q);
    }
#pragma unroll
    for (int h = 0; h < NCH; ++h)
      if (in && live[h]) store8<T>(p.o1, row * p.c + at[h], d[h]);
  }
  if constexpr (GATE) {
    if (per_request && r0 < p.n) {
      // the last request of the group: partial row 0 if it is the first too, else 1
      float* to = p.gpart + (gid * 2 + (w.b != first)) * p.c;
#pragma unroll
      for (int h = 0; h < NCH; ++h)
        if (live[h]) store8<float>(to, at[h], acc[I_G][h]);
    }
  }
  const int keep = per_request ? V - 1 : V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v >= keep) break;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if constexpr (RPB > 1) {
        __syncthreads();
        if (group)
#pragma unroll
          for (int e = 0; e < 8; ++e) meet[(((group - 1) * 8 + e) * WPR * 64) + t] = acc[v][h][e];
        __syncthreads();
        if (!group)
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int q = 0; q < RPB - 1; ++q) acc[v][h][e] += meet[((q * 8 + e) * WPR * 64) + t];
      }
      if (!group && live[h]) store8<float>(p.part + ((int64_t)blockIdx.x * V + v) * p.c, at[h], acc[v][h]);
    }
  }
}

// Joins the partial rows: column v of `part` over the workgroups, in order.
// One workgroup: 32 columns, 32 runs of partial rows that meet in LDS.
struct NormJoinArgs {
  const float *part, *gpart;
  float* out[5];         // by vector, null where not wanted
  float* dgate;          // per request
  const int32_t* off;
  int64_t n;
  int32_t c, V, wgs, blocks, B, rows;   // blocks: column blocks of 32
};

__global__ __launch_bounds__(256) void norm_join_kernel(NormJoinArgs p) {
  __shared__ float4 buf[32][9];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int cb = blockIdx.x % p.blocks, which = blockIdx.x / p.blocks;
  const int c = cb * 32 + x * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); };
  float* out;
  if (which < p.V) {
    out = p.out[which];
    if (!out) return;
    if (c < p.c)
#pragma unroll 8
      for (int w = y; w < p.wgs; w += 32)
        v = add(v, *reinterpret_cast<const float4*>(p.part + ((int64_t)w * p.V + which) * p.c + c));
  } else {
    // a request's gate gradient: of every row group it reaches, partial row 0
    // where it is the group's first request, else 1 where it is its last;
    // one that lies inside a group was written by that group
    const int b = which - p.V;
    const int64_t lo = b == 0 ? 0 : p.off[b], hi = b + 1 < p.B ? p.off[b + 1] : p.n;
    out = p.dgate + (int64_t)b * p.c;
    if (lo >= 0 && hi <= p.n && lo < hi) {
      const int64_t g0 = lo / p.rows, g1 = (hi - 1) / p.rows;
      if (g0 == g1 && lo > g0 * p.rows && hi < (g0 + 1) * p.rows && hi < p.n) return;
      if (c < p.c)
#pragma unroll 4
        for (int64_t g = g0 + y; g <= g1; g += 32)
          v = add(v, *reinterpret_cast<const float4*>(p.gpart + (g * 2 + (lo > g * p.rows)) * p.c + c));
    }
  }
  buf[y][x] = v;
  __syncthreads();
  if (y || c >= p.c) return;
  v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 32; ++q) v = add(v, buf[q][x]);
  *reinterpret_cast<float4*>(out + c) = v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

bool misaligned(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }
int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a row lies over lanes: waves (1 to 8, or 16), and chunks of 8 elements a lane.
struct Shape {
  int waves, chunks;
};

// bf16 takes two chunks a lane above 512 columns, fp32 (whose chunk is twice
// the registers) only where 16 waves do not hold the row otherwise.
Shape row_shape(int64_t c, int dtype) {
  const int wide = dtype == DYRA_BF16 ? (c > 512 ? 2 : 1) : (c > 8192 ? 2 : 1);
  const int w = (int)((c + 512 * wide - 1) / (512 * wide));
  return {w <= 8 ? w : 16, wide};
}

struct Split {
  int rpb, rows;   // row groups of a workgroup, rows of a row group
  int64_t wgs;
};

// Workgroups of a pass: `most` at the most, each row group an equal run of rows.
Split split_rows(int64_t n, int rpb, int64_t most) {
  const int64_t groups = std::max<int64_t>(1, std::min(n, most * rpb));
  Split s;
  s.rpb = rpb;
  s.rows = (int)std::max<int64_t>(1, cdiv64(n, groups));
  s.wgs = std::max<int64_t>(1, cdiv64(cdiv64(n, s.rows), rpb));
  return s;
}

// Backward: one workgroup of 8 waves a CU (16 for the widest rows), the
// registers' limit; more would only add partial rows.  Two of 4 waves a CU
// measure the same, four 50 us against 43 (4099 x 4096, both norms, gate).
constexpr int BWAVES = 8, BWGS = 256;
// Forward: up to 4 waves a row 4096 workgroups (25 us at 4099 x 4096; 512:
// 25, 1024: 29), above two a CU, which is what fits (28 us at 2000 x 8192 with
// 512, 34 with 4096).
constexpr int forward_wgs(int waves) { return waves > 4 ? 512 : 4096; }
constexpr int backward_rpb(int waves) { return waves > BWAVES / 2 ? 1 : BWAVES / waves; }
Split backward_split(int64_t n, int waves) { return split_rows(n, backward_rpb(waves), BWGS); }

int flags_of(const dyra_block_norm& p) {
  return (p.post != DYRA_NORM_NONE ? HAS_POST : 0) | (p.gate_kind != DYRA_GATE_NONE ? HAS_GATE : 0) |
         (p.pre_bias || p.post_bias ? HAS_BIAS : 0);
}

struct NormPlan {
  Split s;
  size_t part, gpart, total;
};

NormPlan norm_plan(const dyra_block_norm& p, int64_t n, int dtype) {
  NormPlan q;
  q.s = backward_split(n, row_shape(p.c, dtype).waves);
  q.part = 0;
  q.gpart = align256((size_t)(q.s.wgs * vectors(flags_of(p)) * p.c * 4));
  q.total = q.gpart;
  if (p.gate_kind == DYRA_GATE_REQUEST) q.total += align256((size_t)(q.s.wgs * q.s.rpb * 2 * p.c * 4));
  return q;
}

int validate(const dyra_block_norm* p, int64_t n, int64_t B, int dtype) {
  if (!p) return DYRA_EINVAL;
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  if (p->pre != DYRA_NORM_RMS && p->pre != DYRA_NORM_LAYER) return DYRA_EINVAL;
  if (p->post != DYRA_NORM_NONE && p->post != DYRA_NORM_RMS && p->post != DYRA_NORM_LAYER) return DYRA_EINVAL;
  if (p->gate_kind != DYRA_GATE_NONE && p->gate_kind != DYRA_GATE_CHANNEL && p->gate_kind != DYRA_GATE_REQUEST)
    return DYRA_EINVAL;
  if ((p->gate_kind == DYRA_GATE_NONE) != (p->gate == nullptr) && !(p->gate_kind == DYRA_GATE_REQUEST && B == 0))
    return DYRA_EINVAL;
  if (p->post == DYRA_NORM_NONE && (p->post_weight || p->post_bias)) return DYRA_EINVAL;
  if (!(p->eps >= 0.f) || !(p->eps < 1e30f) || !(p->residual_scale > -1e30f && p->residual_scale < 1e30f))
    return DYRA_EINVAL;
  if (p->c <= 0 || p->c % 8 || p->c > MAX_C || n < 0 || n >= (int64_t)1 << 31 || B < 0 || B >= (int64_t)1 << 24)
    return DYRA_ESHAPE;
  if (p->gate_kind == DYRA_GATE_REQUEST && n > 0 && B == 0) return DYRA_ESHAPE;
  if (misaligned(p->pre_weight, 15) || misaligned(p->pre_bias, 15) || misaligned(p->post_weight, 15) ||
      misaligned(p->post_bias, 15) || misaligned(p->gate, 15))
    return DYRA_EINVAL;
  return DYRA_OK;
}

NormArgs norm_args(const dyra_block_norm& p, int64_t n, int64_t B, const int32_t* off) {
  NormArgs a{};
  a.pw = p.pre_weight;
  a.pb = p.pre_bias;
  a.qw = p.post_weight;
  a.qb = p.post_bias;
  a.gate = p.gate;
  a.off = off;
  a.n = n;
  a.c = (int32_t)p.c;
  a.B = (int32_t)B;
  a.pre = p.pre;
  a.post = p.post;
  a.per_request = p.gate_kind == DYRA_GATE_REQUEST;
  a.eps = p.eps;
  a.alpha = p.residual_scale;
  return a;
}

template <typename T, int WPR, int NCH>
void launch_forward_shape(NormArgs a, hipStream_t st) {
  constexpr int RPB = WPR >= 3 ? 1 : 4 / WPR;
  const Split s = split_rows(a.n, RPB, forward_wgs(WPR));
  a.rows = s.rows;
  hipLaunchKernelGGL((norm_forward_kernel<T, WPR, NCH, RPB>), dim3((unsigned)s.wgs), dim3(WPR * RPB * 64), 0, st, a);
}

template <typename T, int F, int WPR, int NCH>
void launch_backward_shape(const NormArgs& a, const Split& s, hipStream_t st) {
  constexpr int RPB = backward_rpb(WPR);
  hipLaunchKernelGGL((norm_backward_kernel<T, WPR, NCH, RPB, F>), dim3((unsigned)s.wgs), dim3(WPR * RPB * 64), 0, st, a);
}

// Calls f(waves, chunks), as constants, of the shape.
template <typename T, class Fn>
void with_shape(const Shape& sh, Fn&& f) {
  constexpr int N = sizeof(T) == 2 ? 2 : 1;   // chunks of the wide shapes
  auto at = [&](auto w, auto n) { f(w, n); };
  using std::integral_constant;
  const integral_constant<int, N> n{};
  switch (sh.waves) {
    case 1:
      if (sh.chunks == 1) at(integral_constant<int, 1>(), integral_constant<int, 1>());
      else if constexpr (N == 2) at(integral_constant<int, 1>(), n);
      break;
    case 2: at(integral_constant<int, 2>(), n); break;
    case 3: at(integral_constant<int, 3>(), n); break;
    case 4: at(integral_constant<int, 4>(), n); break;
    case 5: at(integral_constant<int, 5>(), n); break;
    case 6: at(integral_constant<int, 6>(), n); break;
    case 7: at(integral_constant<int, 7>(), n); break;
    case 8: at(integral_constant<int, 8>(), n); break;
    default:
      if constexpr (N == 1) {
        if (sh.chunks == 1) {
          at(integral_constant<int, 16>(), integral_constant<int, 1>());
          break;
        }
      }
      at(integral_constant<int, 16>(), integral_constant<int, 2>());
      break;
  }
}

template <typename T>
void launch_forward(const NormArgs& a, hipStream_t st) {
  with_shape<T>(row_shape(a.c, sizeof(T) == 2 ? DYRA_BF16 : DYRA_F32), [&](auto w, auto n) {
    launch_forward_shape<T, decltype(w)::value, decltype(n)::value>(a, st);
  });
}

template <typename T, int F>
void launch_backward_f(const NormArgs& a, const Split& s, hipStream_t st) {
  with_shape<T>(row_shape(a.c, sizeof(T) == 2 ? DYRA_BF16 : DYRA_F32), [&](auto w, auto n) {
    launch_backward_shape<T, F, decltype(w)::value, decltype(n)::value>(a, s, st);
  });
}

template <typename T>
void launch_backward(const NormArgs& a, const Split& s, int flags, hipStream_t st) {
  switch (flags) {
    case 0: launch_backward_f<T, 0>(a, s, st); break;
    case 1: launch_backward_f<T, 1>(a, s, st); break;
    case 2: launch_backward_f<T, 2>(a, s, st); break;
    case 3: launch_backward_f<T, 3>(a, s, st); break;
    case 4: launch_backward_f<T, 4>(a, s, st); break;
    case 5: launch_backward_f<T, 5>(a, s, st); break;
    case 6: launch_backward_f<T, 6>(a, s, st); break;
    default: launch_backward_f<T, 7>(a, s, st); break;
  }
}

}  // namespace

extern "C" int dyra_block_norm_forward(const dyra_block_norm* p, const void* x, const void* y, void* x_new, void* z,
                                       int64_t n, int64_t B, const int32_t* offsets_dev, int32_t dtype,
                                       void* stream) {
  const int rc = validate(p, n, B, dtype);
  if (rc) return rc;
  if (n == 0) return DYRA_OK;
  if (!x || !y || !x_new || !z || (p->gate_kind == DYRA_GATE_REQUEST && !offsets_dev)) return DYRA_EINVAL;
  if (misaligned(x, 15) || misaligned(y, 15) || misaligned(x_new, 15) || misaligned(z, 15) || misaligned(offsets_dev, 3))
    return DYRA_EINVAL;
  NormArgs a = norm_args(*p, n, B, offsets_dev);
  a.x = x;
  a.y = y;
  a.o0 = x_new;
  a.o1 = z;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == DYRA_BF16) launch_forward<bf16_t>(a, st);
  else launch_forward<float>(a, st);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

extern "C" int dyra_block_norm_workspace_size(const dyra_block_norm* p, int64_t n, int64_t B, int32_t dtype,
                                              size_t* bytes) {
  if (!bytes) return DYRA_EINVAL;
  const int rc = validate(p, n, B, dtype);
  if (rc) return rc;
  *bytes = norm_plan(*p, n, dtype).total;
  return DYRA_OK;
}

extern "C" int dyra_block_norm_backward(const dyra_block_norm* p, const void* x_new, const void* y, const void* dz,
                                        const void* dx_new, void* dx, void* dy, const dyra_block_norm_grads* g,
                                        int64_t n, int64_t B, const int32_t* offsets_dev, int32_t dtype,
                                        void* workspace, size_t ws_bytes, void* stream) {
  const int rc = validate(p, n, B, dtype);
  if (rc) return rc;
  if (!g) return DYRA_EINVAL;
  if (misaligned(g->pre_weight, 15) || misaligned(g->pre_bias, 15) || misaligned(g->post_weight, 15) ||
      misaligned(g->post_bias, 15) || misaligned(g->gate, 15) || misaligned(workspace, 15) ||
      misaligned(offsets_dev, 3))
    return DYRA_EINVAL;
  // a bias or gate gradient needs its operand; weights may be implied ones
  if ((g->pre_bias && !p->pre_bias) || (g->post_bias && !p->post_bias) ||
      (g->post_weight && p->post == DYRA_NORM_NONE) || (g->gate && p->gate_kind == DYRA_GATE_NONE))
    return DYRA_EINVAL;
  if (p->gate_kind == DYRA_GATE_REQUEST && B && (!offsets_dev || !g->gate)) return DYRA_EINVAL;
  if (!workspace) return DYRA_EINVAL;
  if (n && (!x_new || !y || !dz || !dx || !dy || misaligned(x_new, 15) || misaligned(y, 15) || misaligned(dz, 15) ||
            misaligned(dx_new, 15) || misaligned(dx, 15) || misaligned(dy, 15)))
    return DYRA_EINVAL;
  const NormPlan q = norm_plan(*p, n, dtype);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  const int F = flags_of(*p), V = vectors(F);
  const int blocks = (int)cdiv64(p->c, 32);
  const int requests = p->gate_kind == DYRA_GATE_REQUEST ? (int)B : 0;
  if (((int64_t)blocks * (V + requests)) << 8 >= (int64_t)1 << 32) return DYRA_ESHAPE;   // threads of the join's launch
  NormArgs a = norm_args(*p, n, B, offsets_dev);
  a.x = x_new;
  a.y = y;
  a.dz = dz;
  a.dxn = dx_new;
  a.o0 = dx;
  a.o1 = dy;
  char* ws = reinterpret_cast<char*>(workspace);
  a.part = reinterpret_cast<float*>(ws + q.part);
  a.gpart = reinterpret_cast<float*>(ws + q.gpart);
  a.dgate = g->gate;
  a.rows = q.s.rows;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  NormJoinArgs j{};
  j.part = a.part;
  j.gpart = a.gpart;
  int v = 0;
  j.out[v++] = g->pre_weight;
  if (F & HAS_BIAS) j.out[v++] = g->pre_bias;
  if (F & HAS_POST) j.out[v++] = g->post_weight;
  if ((F & HAS_POST) && (F & HAS_BIAS)) j.out[v++] = g->post_bias;
  if (F & HAS_GATE) j.out[v++] = requests || p->gate_kind == DYRA_GATE_REQUEST ? nullptr : g->gate;
  j.dgate = g->gate;
  j.off = offsets_dev;
  j.n = n;
  j.c = a.c;
  j.V = V;
  j.wgs = n ? (int)q.s.wgs : 0;
  j.blocks = blocks;
  j.B = (int32_t)B;
  j.rows = q.s.rows;
  // no rows: the row kernel, which would load a row of the gate that a call
  // without requests does not have, has nothing to do, and the join writes zeros
  bool wanted = n || requests;
  for (const float* out : j.out) wanted = wanted || out;
  if (!wanted) return DYRA_OK;
  if (n && dtype == DYRA_BF16) launch_backward<bf16_t>(a, q.s, F, st);
  else if (n) launch_backward<float>(a, q.s, F, st);
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)(blocks * (V + requests))), dim3(256), 0, st, j);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}
