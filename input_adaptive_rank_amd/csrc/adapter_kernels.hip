// Low-rank adapters of many requests beside a shared projection, on gfx950.
//
// Rows of all requests are concatenated; request b (rows off[b] .. off[b+1]-1)
// uses adapter a = slot[b] of a pool A [slots][r][c1], B [slots][c2][r], with
// effective rank k_a <= r and scale s_a.  Per row t of such a request:
//   forward   H_t = X_t A_a^T              (the "shrink", c1 -> k_a)
//             Y_t = base_t + s_a H_t B_a^T (the "expand", k_a -> c2)
//   backward  G_t = s_a dY_t B_a           (shrink with B^T)
//             dX_t = dX_base_t + G_t A_a   (expand with A^T)
//             dA_a = sum_t G_t^T X_t,  dB_a = sum_t s_a dY_t^T H_t
// A row of a request without an adapter (slot < 0 or >= slots) has H = G = 0.
//
// Every pass streams the n-row operands once and touches r-wide ones beside
// them, so memory bounds all of it (r <= 128: at most 2 r flops per operand
// byte).  Rows are grouped by adapter first (group_kernel), so that a tile of
// rows shares its weights whatever the order of the requests.
#include <hip/hip_runtime.h>

#include <climits>

#include "../../include/dyra.h"
#include "device_common.h"
#include "spec.h"

using namespace dyra_spec_util;

namespace {

constexpr int MAX_SLOTS = 2048;   // the grouping kernel holds three counters per slot in LDS
constexpr int GROUP_NT = 1024;
constexpr int TR = 64;            // edge of the weight transposition tiles

__host__ __device__ __forceinline__ int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Requests of a call.  The device arrays are the caller's; whatever they
// hold, every request's rows stay inside [0, n): the first request starts at
// row 0, the last ends at row n, the offsets between are clamped.
struct Requests {
  const int32_t* off;
  const int32_t* slot;
  int32_t n, B, slots;
  __device__ __forceinline__ int count() const { return B > 0 ? B : 1; }   // no request: one without an adapter
  __device__ __forceinline__ int lo(int b) const { return b <= 0 ? 0 : b >= count() ? n : min(max(off[b], 0), n); }
  __device__ __forceinline__ int len(int b) const { return max(lo(b + 1) - lo(b), 0); }
  // slots stands for "no adapter"
  __device__ __forceinline__ int id(int b) const {
    if (B <= 0) return slots;
    const int s = slot[b];
    return s < 0 || s >= slots ? slots : s;
  }
};

// Rows in the order of their slots: perm[p] is the row at grouped position
// p; a tile is a run of at most `tile` positions of one slot.
struct Tile {
  int32_t slot, start, count, pad;
};
struct Grouped {
  int32_t* perm;        // [n]
  Tile* tiles;          // [tile_cap], count 0 past the last
  Tile* chunks;         // [chunk_cap], runs of `chunk` positions (adapter slots only), or null
  int32_t* slot_chunk;  // [slots + 1] first chunk of each slot
  int32_t tile, chunk, tile_cap, chunk_cap;
};

// The row at place i of a tile, or -1.  The guards keep a position or a row
// in range even where inconsistent offsets left part of perm unwritten.
__device__ __forceinline__ int tile_row(const int32_t* perm, const Tile& t, int i, int n) {
  const int pos = t.start + i;
  if (i >= t.count || (unsigned)pos >= (unsigned)n) return -1;
  const int row = perm[pos];
  return (unsigned)row < (unsigned)n ? row : -1;
}

// ---------------------------------------------------------------------------
// grouping (and, for a backward pass, the weights transposed)
// ---------------------------------------------------------------------------

// inclusive sums over the workgroup's threads of three counters
__device__ __forceinline__ void scan3(int (&v)[3], int* wave_sums) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int u = __shfl_up(v[q], d);
      if (lane >= d) v[q] += u;
    }
  if (lane == 63)
#pragma unroll
    for (int q = 0; q < 3; ++q) wave_sums[wave * 3 + q] = v[q];
  __syncthreads();
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int q = 0; q < 3; ++q) v[q] += wave_sums[w * 3 + q];
  __syncthreads();
}

template <typename E>
struct Transpose {   // src [slots][R][C] -> dst [slots][C][R], for the slots in use
  const E* src;
  E* dst;
  int32_t R, C;
  int32_t tiles_r, tiles_c;
};

template <typename E>
__device__ void transpose_tile(const Transpose<E>& t, const Requests& q, int tile, char* lds) {
  const int per = t.tiles_r * t.tiles_c;
  const int slot = tile / per, rt = (tile % per) / t.tiles_c, ct = (tile % per) % t.tiles_c;
  int used = 0;
  for (int b = threadIdx.x; b < q.B; b += GROUP_NT) used |= q.slot[b] == slot && q.len(b) > 0;
  if (!__syncthreads_or(used)) return;
  E(*buf)[TR + 2] = reinterpret_cast<E(*)[TR + 2]>(lds);
  const E* s = t.src + (int64_t)slot * t.R * t.C;
  E* d = t.dst + (int64_t)slot * t.R * t.C;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  for (int i = y; i < TR; i += GROUP_NT / 64) {
    const int r = rt * TR + i, c = ct * TR + x;
    if (r < t.R && c < t.C) buf[i][x] = s[(int64_t)r * t.C + c];
  }
  __syncthreads();
  for (int i = y; i < TR; i += GROUP_NT / 64) {
    const int c = ct * TR + i, r = rt * TR + x;
    if (r < t.R && c < t.C) d[(int64_t)c * t.R + r] = buf[x][i];
  }
}

// Sorts the requests by slot, stably, and lists the rows in that order.  A
// stable order makes every sum over the rows of a slot the same from call to
// call.  Each of the first `group_wgs` workgroups does the whole sort (a few
// thousand cycles for up to 1024 requests) and writes its share of the row
// list and of the tile lists, so no workgroup waits for another; the others
// transpose weight tiles.
template <typename E>
__global__ __launch_bounds__(GROUP_NT) void group_kernel(Requests q, Grouped g, int group_wgs, Transpose<E> ta,
                                                         Transpose<E> tb, int tiles_a) {
  __shared__ __attribute__((aligned(16))) char lds[TR * (TR + 2) * 4 > 4 * GROUP_NT * 4 + 16
                                                       ? TR * (TR + 2) * 4
                                                       : 4 * GROUP_NT * 4 + 16];
  __shared__ int32_t run[MAX_SLOTS + 1], tile0[MAX_SLOTS + 1], chunk0[MAX_SLOTS + 1], start[MAX_SLOTS + 1];
  __shared__ int wave_sums[3 * GROUP_NT / 64];
  const int tid = threadIdx.x, wg = blockIdx.x;
  if (wg >= group_wgs) {
    const int t = wg - group_wgs;
    if (t < tiles_a) transpose_tile(ta, q, t, lds);
    else transpose_tile(tb, q, t - tiles_a, lds);
    return;
  }
  const int B = q.count(), S = q.slots, stride = group_wgs * GROUP_NT;
  // rows of each slot
  for (int s = tid; s <= S; s += GROUP_NT) run[s] = 0;
  __syncthreads();
  for (int b = tid; b < B; b += GROUP_NT) {
    const int len = q.len(b);
    if (len) atomicAdd(&run[q.id(b)], len);
  }
  __syncthreads();
  // first position, first tile and first chunk of each slot; thread t sums slots [t E, (t + 1) E)
  constexpr int EACH = (MAX_SLOTS + 1 + GROUP_NT - 1) / GROUP_NT;
  int own[EACH][3], sum[3] = {0, 0, 0};
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int s = tid * EACH + e, rows = s <= S ? run[s] : 0;
    own[e][0] = rows;
    own[e][1] = (rows + g.tile - 1) / g.tile;
    own[e][2] = s < S && g.chunk ? (rows + g.chunk - 1) / g.chunk : 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] += own[e][k];
  }
  int at[3] = {sum[0], sum[1], sum[2]};
  scan3(at, wave_sums);
#pragma unroll
  for (int k = 0; k < 3; ++k) at[k] -= sum[k];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int s = tid * EACH + e;
    if (s <= S) {
      start[s] = run[s] = at[0];
      tile0[s] = at[1];
      chunk0[s] = at[2];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) at[k] += own[e][k];
  }
  __syncthreads();
  // tile lists: position -> slot by bisection in tile0 / chunk0.  Slots
  // without rows have no tile, so the last s with tile0[s] <= i is the one.
  auto fill = [&](Tile* list, int cap, int size, const int32_t* first, int last_slot) {
    for (int i = wg * GROUP_NT + tid; i < cap; i += stride) {
      int a = 0, z = last_slot + 1;
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (first[mid] <= i) a = mid;
        else z = mid;
      }
      const int end = a < S ? start[a + 1] : q.n;
      const int p = start[a] + (i - first[a]) * size;
      list[i] = Tile{a, p, max(min(end - p, size), 0), 0};
    }
  };
  fill(g.tiles, g.tile_cap, g.tile, tile0, S);
  if (g.chunk) {
    fill(g.chunks, g.chunk_cap, g.chunk, chunk0, S - 1);
    for (int s = wg * GROUP_NT + tid; s <= S; s += stride) g.slot_chunk[s] = chunk0[s];
  }
  // rows, 1024 requests at a time
  int32_t* ids = reinterpret_cast<int32_t*>(lds);
  int32_t *lens = ids + GROUP_NT, *gpos = lens + GROUP_NT, *offs = gpos + GROUP_NT;   // offs has one more
  for (int b0 = 0; b0 < B; b0 += GROUP_NT) {
    const int nb = min(B - b0, GROUP_NT), b = b0 + tid;
    __syncthreads();
    const int id = tid < nb ? q.id(b) : S + 1, len = tid < nb ? q.len(b) : 0;
    ids[tid] = id;
    lens[tid] = len;
    offs[tid] = tid < nb ? q.lo(b) : q.lo(b0 + nb);
    if (tid == 0) offs[GROUP_NT] = q.lo(b0 + nb);
    __syncthreads();
    int before = 0;
    if (tid < nb)
      for (int u = 0; u < tid; ++u) before += ids[u] == id ? lens[u] : 0;
    gpos[tid] = tid < nb ? run[id] + before : 0;
    __syncthreads();
    if (len) atomicAdd(&run[id], len);
    const int lo = offs[0], hi = offs[nb];
    for (int t = lo + wg * GROUP_NT + tid; t < hi; t += stride) {
      int a = 0, z = nb;   // the last request starting at or before row t (empty ones before it share its start)
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (offs[mid] <= t) a = mid;
        else z = mid;
      }
      const int p = gpos[a] + (t - offs[a]);
      if (t - offs[a] < lens[a] && (unsigned)p < (unsigned)q.n) g.perm[p] = t;
    }
  }
}

// ---------------------------------------------------------------------------
// 16x16 matrix products of both element types
// ---------------------------------------------------------------------------

// A 16-byte chunk holds KPC elements; lane (i, g) = (lane & 15, lane >> 4)
// holds elements KPC g .. KPC g + KPC - 1 of row i of a k-step of 4 KPC.
template <typename T> struct Step;
template <> struct Step<bf16_t> {
  static constexpr int KPC = 8, K = 32;
  __device__ static __forceinline__ void mma(f32x4& acc, const uint4& a, const uint4& b) { mma16(acc, a, b); }
};
template <> struct Step<float> {
  static constexpr int KPC = 4, K = 16;
  // v_mfma_f32_16x16x4_f32 takes one element of each lane; the four in a chunk go to four of them
  __device__ static __forceinline__ void mma(f32x4& acc, const uint4& a, const uint4& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), acc, 0, 0, 0);
  }
};

// v = hi + lo to 2^-18 relative, both bf16 (lo = 0 beside an infinite hi,
// which inf - inf would turn into NaN).
__device__ __forceinline__ void split2(float v, bf16_t& hi, float& rest) {
  hi = f2bf(v);
  const float h = bf2f(hi);
  rest = __builtin_isinf(h) ? 0.f : v - h;
}

// ---------------------------------------------------------------------------
// shrink: P[ks][row][j] = sum over a slice of K of X[row][k] W_slot[j][k]
// ---------------------------------------------------------------------------

struct ShrinkArgs {
  const void* X;        // [n][ldx]
  const void* W;        // [slots][r][K]
  const int32_t* rank;  // or null: r
  const float* scale;   // or null: 1
  float* P;             // [KS][n][r]; columns past the rank are 0
  int64_t ldx, K;
  int32_t n, r, slots, sub, tiles, KS;   // sub: row blocks of 16 RT rows a tile is cut into
  Grouped g;
};

constexpr int SHRINK_WAVES = 8;

// One workgroup: 16 RT rows of one slot, one of KS slices of K, which its
// waves divide again; their sums meet in LDS.  A wave reads X straight into
// matrix operands, each 16-byte load one operand of 16 rows; the weights come
// from the L2, one operand per 16 rank columns for every RT operands of X.
template <typename T, int RT, int CT>
__global__ __launch_bounds__(SHRINK_WAVES * 64) void shrink_kernel(ShrinkArgs p) {
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K, W = SHRINK_WAVES;
  constexpr int U = RT + CT > 6 ? 2 : 4;   // k-steps whose loads are in flight together
  constexpr int CB = CT < 4 ? CT : 4;      // 16-column blocks joined at a time
  __shared__ float red[W][CB][256];
  __shared__ int rows[16 * RT];
  const int tile = blockIdx.x / (p.sub * p.KS), rem = blockIdx.x % (p.sub * p.KS);
  const int sub = rem / p.KS, ks = rem % p.KS;
  const Tile t = p.g.tiles[tile];
  if (t.count <= sub * 16 * RT) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  if (tid < 16 * RT) rows[tid] = tile_row(p.g.perm, t, sub * 16 * RT + tid, p.n);
  __syncthreads();
  const bool none = t.slot >= p.slots;
  const int rank = none ? 0 : p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const int nct = (rank + 15) >> 4;
  f32x4 acc[RT][CT] = {};
  if (rank > 0) {
    const T* xr[RT];
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      const int row = rows[16 * a + i];
      xr[a] = reinterpret_cast<const T*>(p.X) + (int64_t)(row < 0 ? max(rows[0], 0) : row) * p.ldx + g * KPC;
    }
    const T* wr[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)   // rows past the pool's r repeat the last one; their sums are dropped
      wr[c] = reinterpret_cast<const T*>(p.W) + ((int64_t)t.slot * p.r + min(16 * c + i, p.r - 1)) * p.K + g * KPC;
    const int64_t steps = cdiv64(p.K, KSTEP), per = cdiv64(steps, (int64_t)p.KS * W);
    const int64_t s0 = ((int64_t)ks * W + wave) * per, s1 = s0 + per < steps ? s0 + per : steps;
    for (int64_t s = s0; s < s1; s += U) {
      uint4 xv[U][RT], wv[U][CT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t k = (s + u) * KSTEP;
        const bool ok = s + u < s1 && k + g * KPC < p.K;
#pragma unroll
        for (int a = 0; a < RT; ++a) xv[u][a] = ok ? *reinterpret_cast<const uint4*>(xr[a] + k) : zero4();
#pragma unroll
        for (int c = 0; c < CT; ++c)
          wv[u][c] = ok && c < nct ? *reinterpret_cast<const uint4*>(wr[c] + k) : zero4();
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < CT; ++c)
          if (c < nct)
#pragma unroll
            for (int a = 0; a < RT; ++a) Step<T>::mma(acc[a][c], xv[u][a], wv[u][c]);
    }
  }
  // join the waves: D[row][j] of a 16x16 block sits at lane j + 16 (row / 4), register row % 4
  const float scale = none || !p.scale ? 1.f : p.scale[t.slot];
  float* P = p.P + (int64_t)ks * p.n * p.r;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int cb = 0; cb < CT; cb += CB) {
      if (16 * cb >= p.r) break;
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CB; ++c)
        if (cb + c < nct) *reinterpret_cast<f32x4*>(&red[wave][c][lane * 4]) = acc[a][cb + c];
      __syncthreads();
      const int cols = min(p.r - 16 * cb, 16 * CB);
      for (int e = tid; e < 16 * cols; e += W * 64) {
        const int row16 = e / cols, j = e % cols, row = rows[16 * a + row16];
        if (row < 0) continue;
        float v = 0.f;
        if (16 * cb + j < rank) {
          const int at = ((j & 15) + 16 * (row16 >> 2)) * 4 + (row16 & 3);
#pragma unroll
          for (int w = 0; w < W; ++w) v += red[w][j >> 4][at];
          v *= scale;
        }
        P[(int64_t)row * p.r + 16 * cb + j] = v;
      }
    }
}

// ---------------------------------------------------------------------------
// expand: out[row][c] = base[row][c] + sum_j scale P[row][j] W_slot[c][j]
// ---------------------------------------------------------------------------

struct ExpandArgs {
  const float* P;       // [KS][n][r]
  const void* W;        // [slots][C][r]
  const int32_t* rank;  // or null: r
  const float* scale;   // or null: 1
  const void* base;     // [n][ldb], or null: 0
  void* out;            // [n][ldo]
  float* H;             // [n][r] receives the sum over ks of P, or null
  int64_t ldb, ldo, C;
  int32_t n, r, slots, KS, tiles, col_blocks;
  Grouped g;
};

constexpr int EXPAND_COLS = 256;   // columns of a workgroup, 64 of each wave

// One workgroup: a tile of 16 RT rows, 256 columns.  P is summed over its
// slices, scaled and put in LDS once: in bf16 as two terms, hi + lo, so that
// Y carries no rounding but its own; the extra product is cheap beside the
// row traffic.  Weights stay in registers for the whole tile.  The weight is
// the left operand, so a lane's results are consecutive columns of one row:
// left row i of the two products of 32 columns is column 8 (i / 4) + 4 h + i % 4
// (h the product), which makes one 16-byte piece of the row.
template <typename T, int RT, int NK>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K, TERMS = BF ? 2 : 1;
  constexpr int PITCH = NK * KSTEP * (int)sizeof(T) + 16;   // bytes of a row in LDS; 16 more spread the banks
  __shared__ __attribute__((aligned(16))) char hs[TERMS * 16 * RT * PITCH];
  __shared__ int rows[16 * RT];
  const int id = xcd_tile_id(blockIdx.x, gridDim.x);
  const Tile t = p.g.tiles[id / p.col_blocks];
  const int cb = id % p.col_blocks;
  if (t.count <= 0) return;
  const bool none = t.slot >= p.slots;
  if (none && p.base == p.out && p.ldb == p.ldo && !(p.H && cb == 0)) return;   // in place: nothing to add
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  if (tid < 16 * RT) rows[tid] = tile_row(p.g.perm, t, tid, p.n);
  __syncthreads();
  const int rank = none ? 0 : p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const int nk = (rank + KSTEP - 1) / KSTEP;
  if (p.H && cb == 0)
    for (int e = tid; e < 16 * RT * p.r; e += 256) {
      const int row = rows[e / p.r], j = e % p.r;
      if (row < 0) continue;
      float v = 0.f;
      if (j < rank)
        for (int ks = 0; ks < p.KS; ++ks) v += p.P[((int64_t)ks * p.n + row) * p.r + j];
      p.H[(int64_t)row * p.r + j] = v;
    }
  if (rank > 0) {
    const float scale = p.scale ? p.scale[t.slot] : 1.f;
    const int wide = nk * KSTEP / 4;   // groups of 4 rank columns, zero past the pool's r
    for (int e = tid; e < 16 * RT * wide; e += 256) {
      const int rr = e / wide, j = (e % wide) * 4, row = rows[rr];
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (row >= 0 && j < p.r)
        for (int ks = 0; ks < p.KS; ++ks) {
          const float4 u = *reinterpret_cast<const float4*>(p.P + ((int64_t)ks * p.n + row) * p.r + j);
          v[0] += u.x;
          v[1] += u.y;
          v[2] += u.z;
          v[3] += u.w;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= scale;
      if constexpr (BF) {
        bf16_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float rest;
          split2(v[q], hi[q], rest);
          lo[q] = f2bf(rest);
        }
        *reinterpret_cast<uint2*>(hs + rr * PITCH + j * 2) =
            make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
        *reinterpret_cast<uint2*>(hs + (16 * RT + rr) * PITCH + j * 2) =
            make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
      } else {
        *reinterpret_cast<float4*>(hs + rr * PITCH + j * 4) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
  __syncthreads();
  const int64_t c0 = (int64_t)cb * EXPAND_COLS + wave * 64;
  if (c0 >= p.C) return;
  // weights of the wave's 64 columns: 4 left operands per k-step
  uint4 wv[4][NK];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int64_t col = BF ? c0 + 32 * (h >> 1) + 8 * (i >> 2) + 4 * (h & 1) + (i & 3) : c0 + 16 * h + i;
    const T* wr = reinterpret_cast<const T*>(p.W) + ((int64_t)t.slot * p.C + col) * p.r;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int j = k * KSTEP + g * KPC;
      uint4 v = zero4();
      if (k < nk && col < p.C && j < rank) {
        v = *reinterpret_cast<const uint4*>(wr + j);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};   // what the pool holds past the rank is not used
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (BF) {
            if (j + 2 * q + 1 >= rank) w[q] &= 0xffffu;
            if (j + 2 * q >= rank) w[q] = 0u;
          } else {
            if (j + q >= rank) w[q] = 0u;
          }
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      wv[h][k] = v;
    }
  }
  constexpr int PIECES = BF ? 2 : 4;   // 16-byte pieces of a row a lane holds: columns 32 a + 8 g, or 16 a + 4 g
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    if (16 * a >= t.count) break;
    const int row = rows[16 * a + i];
    uint4 bv[PIECES];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int64_t col = c0 + q * (4 * KPC) + g * KPC;
      bv[q] = row >= 0 && col < p.C && p.base
                  ? *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.base) + (int64_t)row * p.ldb + col)
                  : zero4();
    }
    f32x4 acc[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if constexpr (BF) {
        const uint32_t w0 = h & 1 ? bv[h >> 1].z : bv[h >> 1].x, w1 = h & 1 ? bv[h >> 1].w : bv[h >> 1].y;
        acc[h] = f32x4{__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                       __uint_as_float(w1 & 0xffff0000u)};
      } else {
        acc[h] = __builtin_bit_cast(f32x4, bv[h]);
      }
    }
#pragma unroll
    for (int k = 0; k < NK; ++k)
      if (k < nk) {
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const uint4 hv = *reinterpret_cast<const uint4*>(
              hs + (term * 16 * RT + 16 * a + i) * PITCH + (k * KSTEP + g * KPC) * (int)sizeof(T));
#pragma unroll
          for (int h = 0; h < 4; ++h) Step<T>::mma(acc[h], wv[h][k], hv);
        }
      }
    if (row < 0) continue;
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int64_t col = c0 + q * (4 * KPC) + g * KPC;
      if (col >= p.C) continue;
      uint4 o;
      if constexpr (BF) {
        auto pair = [](float a, float b) { return (uint32_t)f2bf(a) | (uint32_t)f2bf(b) << 16; };
        o = make_uint4(pair(acc[2 * q][0], acc[2 * q][1]), pair(acc[2 * q][2], acc[2 * q][3]),
                       pair(acc[2 * q + 1][0], acc[2 * q + 1][1]), pair(acc[2 * q + 1][2], acc[2 * q + 1][3]));
      } else {
        o = __builtin_bit_cast(uint4, acc[q]);
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + (int64_t)row * p.ldo + col) = o;
    }
  }
}

// ---------------------------------------------------------------------------
// weight gradients: part[chunk][j][c] = sum over the chunk's rows of
// s P[row][j] V[row][c]   (dA: P = G, V = X;  dB: P = s H, V = dY)
// ---------------------------------------------------------------------------

struct GradSide {
  const void* V;       // [n][ldv]
  const float* P;      // [KS][n][r]
  const float* scale;  // or null: 1
  float* part;         // [chunk_cap][r][C]
  int64_t ldv, C;
  int32_t KS, col_blocks;
};
struct GradArgs {
  GradSide side[2];
  const int32_t* rank;
  int32_t n, r, slots, chunk_cap, r_groups;
  Grouped g;
};

constexpr int GRAD_TOK = 64;                  // rows staged together
template <typename T> constexpr int grad_cols() { return sizeof(T) == 2 ? 128 : 64; }   // columns of a wave

// One workgroup: a chunk of rows, 4 waves' columns, up to 16 CT rank columns.
// The row factor (P) goes through LDS, rank-major and, for bf16 V, as three
// bf16 terms (hi + mid + lo, 2^-27 relative: the gradients are fp32, and V is
// exact in bf16).  V is read 8 rows by 8 columns per lane and transposed in
// registers, so that each lane holds 8 consecutive rows of a column, the
// reduction axis; operand e of a lane is column 8 i + e of the wave's 128.
template <typename T, int CT>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int TERMS = BF ? 3 : 1, COLS = grad_cols<T>();
  // bf16: [term][16 CT][GRAD_TOK + 8]; fp32: [GRAD_TOK][16 CT + 4]
  constexpr int PITCH = BF ? GRAD_TOK + 8 : 16 * CT + 4;
  __shared__ __attribute__((aligned(16))) T ps[BF ? TERMS * 16 * CT * PITCH : GRAD_TOK * PITCH];
  __shared__ int rows[GRAD_TOK];
  int id = blockIdx.x;
  const int per0 = p.side[0].col_blocks * p.r_groups * p.chunk_cap;
  const int which = id >= per0;
  id -= which ? per0 : 0;
  const GradSide& v = p.side[which];
  const int cb = id % v.col_blocks, chunk = id / v.col_blocks % p.chunk_cap, rg = id / v.col_blocks / p.chunk_cap;
  const Tile t = p.g.chunks[chunk];
  if (t.count <= 0 || t.slot >= p.slots) return;
  const int rank = p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const int j0 = rg * 16 * CT;
  if (j0 >= rank) return;
  const int nct = min((rank - j0 + 15) >> 4, CT);
  const float scale = v.scale ? v.scale[t.slot] : 1.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int64_t c0 = ((int64_t)cb * 4 + wave) * COLS, col = c0 + i * (COLS / 16);
  const bool live = col < v.C;
  constexpr int E = COLS / 16;   // columns of a lane
  f32x4 acc[CT][E] = {};
  for (int p0 = 0; p0 < t.count; p0 += GRAD_TOK) {
    __syncthreads();
    if (tid < GRAD_TOK) rows[tid] = tile_row(p.g.perm, t, p0 + tid, p.n);
    __syncthreads();
    // P of the staged rows: one unit is 8 rows of one rank column
    for (int u = tid; u < GRAD_TOK / 8 * 16 * CT; u += 256) {
      const int j = u % (16 * CT), tok = u / (16 * CT) * 8;
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int row = rows[tok + q];
        f[q] = 0.f;
        if (row >= 0 && j0 + j < rank)
          for (int ks = 0; ks < v.KS; ++ks) f[q] += v.P[((int64_t)ks * p.n + row) * p.r + j0 + j];
        f[q] *= scale;
      }
      if constexpr (BF) {
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          bf16_t h[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float rest;
            split2(f[q], h[q], rest);
            f[q] = rest;
          }
          *reinterpret_cast<uint4*>(&ps[(term * 16 * CT + j) * PITCH + tok]) =
              make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                         h[6] | (uint32_t)h[7] << 16);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) ps[(tok + q) * PITCH + j] = f[q];
      }
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // 32 rows each
      uint4 in[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // bf16: rows 8 g + e; fp32: rows 4 e + g (one product per element of the chunk, four rows each)
        const int row = rows[half * 32 + (BF ? 8 * g + e : 4 * e + g)];
        in[e] = row >= 0 && live
                    ? *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(v.V) + (int64_t)row * v.ldv + col)
                    : zero4();
      }
      if constexpr (BF) {
        uint4 b[8];
        transpose8x8_b16(in, b);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          if (c < nct)
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const uint4 a = *reinterpret_cast<const uint4*>(&ps[(term * 16 * CT + 16 * c + i) * PITCH + half * 32 + 8 * g]);
#pragma unroll
              for (int e = 0; e < 8; ++e) mma16(acc[c][e], a, b[e]);
            }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            if (c < nct) {
              const float a = ps[(half * 32 + 4 * s + g) * PITCH + 16 * c + i];
              acc[c][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, __uint_as_float(in[s].x), acc[c][0], 0, 0, 0);
              acc[c][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, __uint_as_float(in[s].y), acc[c][1], 0, 0, 0);
              acc[c][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, __uint_as_float(in[s].z), acc[c][2], 0, 0, 0);
              acc[c][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, __uint_as_float(in[s].w), acc[c][3], 0, 0, 0);
            }
      }
    }
  }
  if (!live) return;
  float* out = v.part + (int64_t)chunk * p.r * v.C;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = j0 + 16 * c + 4 * g + q;
      if (j >= rank) continue;
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(out + (int64_t)j * v.C + col + e) =
            make_float4(acc[c][e][q], acc[c][e + 1][q], acc[c][e + 2][q], acc[c][e + 3][q]);
    }
}

// Sums the chunks of each slot in order: dA[s][j][c], and dB[s][c][j]
// (transposed through LDS).  Rows past a slot's rank, and slots without rows,
// are zero.  One workgroup: 64 columns and 64 rank columns of one slot.
struct JoinArgs {
  const float* part[2];
  float* out[2];
  int64_t C[2];
  int32_t blocks[2];
  const int32_t* rank;
  int32_t r, slots, chunk_cap;
  Grouped g;
};

__global__ __launch_bounds__(256) void grad_join_kernel(JoinArgs p) {
  __shared__ float buf[64][65];
  int id = blockIdx.x;
  const int which = id >= p.blocks[0];
  id -= which ? p.blocks[0] : 0;
  const int64_t C = p.C[which];
  const int cbs = (int)cdiv64(C, 64), rbs = (p.r + 63) >> 6;
  const int cb = id % cbs, rb = id / cbs % rbs, slot = id / cbs / rbs;
  const int rank = p.rank ? min(max(p.rank[slot], 0), p.r) : p.r;
  const int lo = min(max(p.g.slot_chunk[slot], 0), p.chunk_cap), hi = min(p.g.slot_chunk[slot + 1], p.chunk_cap);
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int64_t c = (int64_t)cb * 64 + x;
  const int64_t step = (int64_t)p.r * C;
  for (int jj = y; jj < 64; jj += 4) {
    const int j = rb * 64 + jj;
    float v = 0.f;
    if (j < rank && c < C) {
      const float* s = p.part[which] + (int64_t)lo * step + (int64_t)j * C + c;
      for (int k = lo; k < hi; ++k, s += step) v += *s;
    }
    if (which) buf[jj][x] = v;
    else if (j < p.r && c < C) p.out[0][((int64_t)slot * p.r + j) * C + c] = v;
  }
  if (!which) return;
  __syncthreads();
  for (int cc = y; cc < 64; cc += 4) {
    const int64_t oc = (int64_t)cb * 64 + cc;
    const int j = rb * 64 + x;
    if (oc < C && j < p.r) p.out[1][((int64_t)slot * C + oc) * p.r + j] = buf[x][cc];
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Sizes of a call: tile heights, splits and the workspace.
struct Plan {
  int tile, rt, sub;                // rows of a tile; 16-row blocks of a shrink workgroup; those per tile
  int ks1, ks2;                     // slices of c1 (forward) / c2 (backward) in the shrink
  int chunk;                        // rows of a gradient chunk (backward), else 0
  int64_t tile_cap, chunk_cap;
  size_t perm, tiles, chunks, slot_chunk, P, At, Bt, partA, partB, total;
};

int shrink_split(int64_t wgs, int64_t K, int dtype) {
  const int64_t steps = cdiv64(K, dtype == DYRA_BF16 ? 32 : 16);
  int64_t ks = cdiv64(512, wgs);                              // two workgroups per CU
  ks = std::min<int64_t>(ks, cdiv64(steps, 2 * SHRINK_WAVES));   // at least two k-steps per wave
  return (int)std::max<int64_t>(1, std::min<int64_t>(ks, 16));
}

Plan make_plan(int64_t slots, int64_t r, int64_t c1, int64_t c2, int64_t n, int64_t B, int dtype, bool backward) {
  Plan q{};
  q.tile = n <= 512 ? 16 : 64;
  q.rt = n <= 512 ? 1 : 2;
  q.sub = q.tile / (16 * q.rt);
  const int64_t used = std::min(slots + 1, B + 1);   // slots with rows, "no adapter" among them
  q.tile_cap = n / q.tile + used + 1;
  const int64_t wgs = std::max<int64_t>(1, cdiv64(n, 16 * q.rt));
  q.ks1 = shrink_split(wgs, c1, dtype);
  q.ks2 = shrink_split(wgs, c2, dtype);
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += align256((size_t)bytes);
    return here;
  };
  q.perm = take(4 * n);
  q.tiles = take((int64_t)sizeof(Tile) * q.tile_cap);
  q.P = take(4 * n * r * (backward ? q.ks2 : q.ks1));
  if (backward) {
    const int cols = 4 * (dtype == DYRA_BF16 ? grad_cols<bf16_t>() : grad_cols<float>());
    const int64_t blocks = cdiv64(c1, cols) + cdiv64(c2, cols);
    const int64_t chunks = std::max<int64_t>(1, 512 / blocks);
    q.chunk = (int)std::max<int64_t>(GRAD_TOK, cdiv64(cdiv64(n, chunks), GRAD_TOK) * GRAD_TOK);
    q.chunk_cap = n / q.chunk + std::min(slots, B) + 1;
    q.chunks = take((int64_t)sizeof(Tile) * q.chunk_cap);
    q.slot_chunk = take(4 * (slots + 1));
    const int64_t esz = (int64_t)elem_bytes(dtype);
    q.At = take(slots * r * c1 * esz);
    q.Bt = take(slots * r * c2 * esz);
    q.partA = take(4 * q.chunk_cap * r * c1);
    q.partB = take(4 * q.chunk_cap * r * c2);
  }
  q.total = at;
  return q;
}

int validate(int64_t slots, int64_t r, int64_t c1, int64_t c2, int64_t n, int64_t B, int dtype) {
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_EINVAL;
  if (slots <= 0 || slots > MAX_SLOTS || r <= 0 || r > 128 || r % 8) return DYRA_ESHAPE;
  if (c1 <= 0 || c2 <= 0 || c1 % 8 || c2 % 8 || c1 > (int64_t)1 << 24 || c2 > (int64_t)1 << 24) return DYRA_ESHAPE;
  if (n < 0 || B < 0 || n >= ((int64_t)1 << 30) || B >= ((int64_t)1 << 30)) return DYRA_ESHAPE;
  return DYRA_OK;
}

bool misaligned(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

bool bad_stride(int64_t ld, int64_t c, int dtype) {
  return ld < c || ld > (int64_t)1 << 32 || ld % (dtype == DYRA_BF16 ? 8 : 4) != 0;
}

Grouped grouped(const Plan& q, char* ws) {
  Grouped g{};
  g.perm = reinterpret_cast<int32_t*>(ws + q.perm);
  g.tiles = reinterpret_cast<Tile*>(ws + q.tiles);
  g.chunks = reinterpret_cast<Tile*>(ws + q.chunks);
  g.slot_chunk = reinterpret_cast<int32_t*>(ws + q.slot_chunk);
  g.tile = q.tile;
  g.chunk = q.chunk;
  g.tile_cap = (int32_t)q.tile_cap;
  g.chunk_cap = (int32_t)q.chunk_cap;
  return g;
}

template <typename E>
void launch_group(const Requests& rq, const Grouped& g, const Transpose<E>& ta, const Transpose<E>& tb,
                  hipStream_t st) {
  const int wgs = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv64(rq.n, 2 * GROUP_NT), 64));
  const int64_t a = ta.src ? (int64_t)rq.slots * ta.tiles_r * ta.tiles_c : 0;
  const int64_t b = tb.src ? (int64_t)rq.slots * tb.tiles_r * tb.tiles_c : 0;
  hipLaunchKernelGGL((group_kernel<E>), dim3((unsigned)(wgs + a + b)), dim3(GROUP_NT), 0, st, rq, g, wgs, ta, tb,
                     (int)a);
}

template <typename T, int RT>
void launch_shrink_rt(const ShrinkArgs& a, unsigned grid, hipStream_t st) {
  const dim3 nt(SHRINK_WAVES * 64);
  if (a.r <= 16) hipLaunchKernelGGL((shrink_kernel<T, RT, 1>), dim3(grid), nt, 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((shrink_kernel<T, RT, 2>), dim3(grid), nt, 0, st, a);
  else if (a.r <= 64) hipLaunchKernelGGL((shrink_kernel<T, RT, 4>), dim3(grid), nt, 0, st, a);
  else hipLaunchKernelGGL((shrink_kernel<T, RT, 8>), dim3(grid), nt, 0, st, a);
}

template <typename T>
void launch_shrink(const ShrinkArgs& a, int rt, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.tiles * a.sub * a.KS);
  if (rt == 1) launch_shrink_rt<T, 1>(a, grid, st);
  else launch_shrink_rt<T, 2>(a, grid, st);
}

template <typename T, int RT>
void launch_expand_rt(const ExpandArgs& a, unsigned grid, hipStream_t st) {
  const int nk = (a.r + Step<T>::K - 1) / Step<T>::K;
  if (nk <= 1) hipLaunchKernelGGL((expand_kernel<T, RT, 1>), dim3(grid), dim3(256), 0, st, a);
  else if (nk <= 2) hipLaunchKernelGGL((expand_kernel<T, RT, 2>), dim3(grid), dim3(256), 0, st, a);
  else if (nk <= 4) hipLaunchKernelGGL((expand_kernel<T, RT, 4>), dim3(grid), dim3(256), 0, st, a);
  else if constexpr (sizeof(T) == 4) hipLaunchKernelGGL((expand_kernel<T, RT, 8>), dim3(grid), dim3(256), 0, st, a);
}

template <typename T>
void launch_expand(const ExpandArgs& a, int tile, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.tiles * a.col_blocks);
  if (tile == 16) launch_expand_rt<T, 1>(a, grid, st);
  else launch_expand_rt<T, 4>(a, grid, st);
}

template <typename T>
int forward_impl(const dyra_adapters& ad, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y,
                 int64_t ldy, float* H, const Requests& rq, const Plan& q, char* ws, hipStream_t st) {
  const Grouped g = grouped(q, ws);
  const Transpose<T> no{};
  launch_group<T>(rq, g, no, no, st);
  // with one slice the shrink writes H itself
  float* P = H && q.ks1 == 1 ? H : reinterpret_cast<float*>(ws + q.P);
  const ShrinkArgs sa{X, ad.A, ad.rank, nullptr, P, ldx, ad.c1, rq.n, ad.r, ad.slots, q.sub, (int32_t)q.tile_cap, q.ks1, g};
  launch_shrink<T>(sa, q.rt, st);
  const ExpandArgs ea{P,      ad.B, ad.rank, ad.scale, base,  Y,
                      P == H ? nullptr : H, ldb, ldy, ad.c2, rq.n, ad.r, ad.slots, q.ks1, (int32_t)q.tile_cap,
                      (int32_t)cdiv64(ad.c2, EXPAND_COLS), g};
  launch_expand<T>(ea, q.tile, st);
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

template <typename T, int CT>
void launch_grad(GradArgs& a, hipStream_t st) {
  a.r_groups = (a.r + 16 * CT - 1) / (16 * CT);
  const int64_t grid = (int64_t)(a.side[0].col_blocks + a.side[1].col_blocks) * a.r_groups * a.chunk_cap;
  hipLaunchKernelGGL((grad_kernel<T, CT>), dim3((unsigned)grid), dim3(256), 0, st, a);
}

template <typename T>
int backward_impl(const dyra_adapters& ad, const void* X, int64_t ldx, const void* dY, int64_t lddy, const float* H,
                  const void* dXb, int64_t lddb, void* dX, int64_t lddx, float* dA, float* dB, const Requests& rq,
                  const Plan& q, char* ws, hipStream_t st) {
  const Grouped g = grouped(q, ws);
  T* At = reinterpret_cast<T*>(ws + q.At);
  T* Bt = reinterpret_cast<T*>(ws + q.Bt);
  const auto blocks = [](int64_t v) { return (int32_t)cdiv64(v, TR); };
  const Transpose<T> ta{dX ? reinterpret_cast<const T*>(ad.A) : nullptr, At, ad.r, (int32_t)ad.c1, blocks(ad.r),
                        blocks(ad.c1)};
  const Transpose<T> tb{reinterpret_cast<const T*>(ad.B), Bt, (int32_t)ad.c2, ad.r, blocks(ad.c2), blocks(ad.r)};
  launch_group<T>(rq, g, ta, tb, st);
  float* P = reinterpret_cast<float*>(ws + q.P);
  if (rq.n) {
    const ShrinkArgs sa{dY, Bt, ad.rank, ad.scale, P, lddy, ad.c2, rq.n, ad.r, ad.slots, q.sub, (int32_t)q.tile_cap, q.ks2, g};
    launch_shrink<T>(sa, q.rt, st);
  }
  if (dX && rq.n) {
    const ExpandArgs ea{P, At, ad.rank, nullptr, dXb, dX, nullptr, lddb, lddx, ad.c1, rq.n, ad.r, ad.slots, q.ks2,
                        (int32_t)q.tile_cap, (int32_t)cdiv64(ad.c1, EXPAND_COLS), g};
    launch_expand<T>(ea, q.tile, st);
  }
  if (dA) {
    float *pa = reinterpret_cast<float*>(ws + q.partA), *pb = reinterpret_cast<float*>(ws + q.partB);
    const int cols = 4 * grad_cols<T>();
    if (rq.n) {
      GradArgs ga{{{X, P, nullptr, pa, ldx, ad.c1, q.ks2, (int32_t)cdiv64(ad.c1, cols)},
                   {dY, H, ad.scale, pb, lddy, ad.c2, 1, (int32_t)cdiv64(ad.c2, cols)}},
                  ad.rank, rq.n, ad.r, ad.slots, (int32_t)q.chunk_cap, 1, g};
      if (ad.r <= 16) launch_grad<T, 1>(ga, st);
      else if (ad.r <= 32) launch_grad<T, 2>(ga, st);
      else launch_grad<T, 4>(ga, st);
    }
    const int64_t rbs = cdiv64(ad.r, 64);
    const int64_t b0 = cdiv64(ad.c1, 64) * rbs * ad.slots, b1 = cdiv64(ad.c2, 64) * rbs * ad.slots;
    const JoinArgs ja{{pa, pb}, {dA, dB}, {ad.c1, ad.c2}, {(int32_t)b0, (int32_t)b1}, ad.rank, ad.r, ad.slots,
                      (int32_t)q.chunk_cap, g};
    hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)(b0 + b1)), dim3(256), 0, st, ja);
  }
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

// every grid of a call fits a launch
bool grids_fit(const dyra_adapters& ad, const Plan& q, bool backward) {
  const int64_t most = INT_MAX;
  const int64_t c = std::max(ad.c1, ad.c2);
  if (q.tile_cap * q.sub * std::max(q.ks1, q.ks2) > most || q.tile_cap * cdiv64(c, EXPAND_COLS) > most) return false;
  if (!backward) return true;
  const int64_t rbs = cdiv64(ad.r, TR);
  return (cdiv64(ad.c1, TR) + cdiv64(ad.c2, TR)) * rbs * ad.slots + 64 <= most &&
         (cdiv64(ad.c1, 256) + cdiv64(ad.c2, 256)) * 2 * q.chunk_cap <= most;
}

}  // namespace

extern "C" int dyra_adapter_workspace_size(int32_t slots, int32_t r, int64_t c1, int64_t c2, int64_t n, int64_t B,
                                           int32_t dtype, int32_t backward, size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return DYRA_EINVAL;
  const int rc = validate(slots, r, c1, c2, n, B, dtype);
  if (rc) return rc;
  *bytes = make_plan(slots, r, c1, c2, n, B, dtype, backward != 0).total;
  return DYRA_OK;
}

extern "C" int dyra_adapter_forward(const dyra_adapters* ad, const void* X, int64_t ldx, const void* base,
                                    int64_t ldb, void* Y, int64_t ldy, float* H, int64_t n, int64_t B,
                                    const int32_t* offsets_dev, const int32_t* slots_dev, int32_t dtype,
                                    void* workspace, size_t ws_bytes, void* stream) {
  if (!ad || !ad->A || !ad->B) return DYRA_EINVAL;
  const int rc = validate(ad->slots, ad->r, ad->c1, ad->c2, n, B, dtype);
  if (rc) return rc;
  if (misaligned(ad->A, 15) || misaligned(ad->B, 15) || misaligned(ad->rank, 3) || misaligned(ad->scale, 3))
    return DYRA_EINVAL;
  if (n == 0) return DYRA_OK;
  if (!X || !Y || !workspace || (B && (!offsets_dev || !slots_dev))) return DYRA_EINVAL;
  if (misaligned(X, 15) || misaligned(base, 15) || misaligned(Y, 15) || misaligned(H, 15) ||
      misaligned(workspace, 15) || misaligned(offsets_dev, 3) || misaligned(slots_dev, 3))
    return DYRA_EINVAL;
  if (bad_stride(ldx, ad->c1, dtype) || bad_stride(ldy, ad->c2, dtype) || (base && bad_stride(ldb, ad->c2, dtype)))
    return DYRA_ESHAPE;
  const Plan q = make_plan(ad->slots, ad->r, ad->c1, ad->c2, n, B, dtype, false);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  if (!grids_fit(*ad, q, false)) return DYRA_ESHAPE;
  const Requests rq{offsets_dev, slots_dev, (int32_t)n, (int32_t)B, ad->slots};
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == DYRA_BF16 ? forward_impl<bf16_t>(*ad, X, ldx, base, ldb, Y, ldy, H, rq, q, ws, st)
                            : forward_impl<float>(*ad, X, ldx, base, ldb, Y, ldy, H, rq, q, ws, st);
}

extern "C" int dyra_adapter_backward(const dyra_adapters* ad, const void* X, int64_t ldx, const void* dY,
                                     int64_t lddy, const float* H, const void* dX_base, int64_t lddb, void* dX,
                                     int64_t lddx, float* dA, float* dB, int64_t n, int64_t B,
                                     const int32_t* offsets_dev, const int32_t* slots_dev, int32_t dtype,
                                     void* workspace, size_t ws_bytes, void* stream) {
  if (!ad || !ad->A || !ad->B || !dA != !dB || (!dA && !dX)) return DYRA_EINVAL;
  const int rc = validate(ad->slots, ad->r, ad->c1, ad->c2, n, B, dtype);
  if (rc) return rc;
  if (misaligned(ad->A, 15) || misaligned(ad->B, 15) || misaligned(ad->rank, 3) || misaligned(ad->scale, 3) ||
      misaligned(dA, 15) || misaligned(dB, 15) || misaligned(workspace, 15))
    return DYRA_EINVAL;
  if (!workspace || (B && (!offsets_dev || !slots_dev))) return DYRA_EINVAL;
  if (misaligned(offsets_dev, 3) || misaligned(slots_dev, 3)) return DYRA_EINVAL;
  if (n) {
    if (!X || !dY || (dA && !H)) return DYRA_EINVAL;
    if (misaligned(X, 15) || misaligned(dY, 15) || misaligned(H, 15) || misaligned(dX_base, 15) || misaligned(dX, 15))
      return DYRA_EINVAL;
    if (bad_stride(ldx, ad->c1, dtype) || bad_stride(lddy, ad->c2, dtype) || (dX && bad_stride(lddx, ad->c1, dtype)) ||
        (dX_base && bad_stride(lddb, ad->c1, dtype)))
      return DYRA_ESHAPE;
  }
  const Plan q = make_plan(ad->slots, ad->r, ad->c1, ad->c2, n, B, dtype, true);
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  if (!grids_fit(*ad, q, true)) return DYRA_ESHAPE;
  const Requests rq{offsets_dev, slots_dev, (int32_t)n, (int32_t)B, ad->slots};
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == DYRA_BF16
             ? backward_impl<bf16_t>(*ad, X, ldx, dY, lddy, H, dX_base, lddb, dX, lddx, dA, dB, rq, q, ws, st)
             : backward_impl<float>(*ad, X, ldx, dY, lddy, H, dX_base, lddb, dX, lddx, dA, dB, rq, q, ws, st);
}
