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
// A product streams an n-row operand and touches r-wide ones beside it: r flops
// (bf16) or r / 2 (fp32) for a byte of it.  At what a large product and a large
// copy reach on this card, 250 flops a byte in bf16 and 32 in fp32, memory
// bounds all but fp32 above r = 64.  A backward pass reads X once and dY twice,
// for G and for dB.  Rows are grouped by adapter first (group_kernel), so that a tile of
// rows shares its weights whatever the order of the requests.
#include <hip/hip_runtime.h>

#include <climits>
#include <type_traits>

#include "../../include/dyra.h"
#include "device_common.h"
#include "spec.h"

using namespace dyra_spec_util;

namespace {

constexpr int MAX_SLOTS = 2048;   // the grouping kernel holds three counters per slot in LDS
constexpr int GROUP_NT = 1024;

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
  // Packed weights are kept by slot, or, of a pool with more slots than there
  // are requests, by the slot's first request that has rows: time and memory
  // follow the slots that can be in use (forward, 5003 rows of 8 requests,
  // 4096 -> 4096, r = 64: 52 us and 10 MiB at 8, 512 and 2048 slots alike; by
  // slot 52, 105 and 267 us, 10, 514 and 2050 MiB).
  __host__ __device__ __forceinline__ bool by_slot() const { return B >= slots; }
};

// Rows in the order of their slots, in tiles of `tile` places that hold rows
// of one slot: place i of tile t is row perm[t tile + i], -1 past its count.
struct Tile {
  uint16_t slot, pack;   // pack: where the slot's packed weights are
  int32_t count;
};
struct Chunk {   // a run of tiles of one adapter slot
  int32_t slot, first, tiles, pad;
};
struct Grouped {
  int32_t* perm;        // [tile_cap][tile]
  Tile* tiles;          // [tile_cap], count 0 past the last
  Chunk* chunks;        // [chunk_cap], tiles 0 past the last, or null
  int32_t* slot_chunk;  // [slots + 1] first chunk of each slot
  int32_t tile, chunk, tile_cap, chunk_cap;   // chunk: tiles of a chunk
};

// The row at place i of tile t, or -1.  The guard keeps a row in range even
// where inconsistent offsets left a place unwritten.
__device__ __forceinline__ int tile_row(const Grouped& g, int t, int i, int n) {
  const int row = g.perm[(int64_t)t * g.tile + i];
  return (unsigned)row < (unsigned)n ? row : -1;
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

// Loads and stores of rows that pass through the expand once (non-temporal):
// they leave the caches to the inputs.  32928 x 1024 -> 4096 with a base: the
// expand 112 -> 103 us, the shrink of the next call 23 -> 15; 4099 x 4096, rank
// 16: 66 -> 64 us together with a norm that reads the result at once.
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 load_once(const void* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}
__device__ __forceinline__ void store_once(void* p, const uint4& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
}

// v = hi + lo to 2^-18 relative, both bf16 (lo = 0 beside an infinite hi,
// which inf - inf would turn into NaN).
__device__ __forceinline__ void split2(float v, bf16_t& hi, float& rest) {
  hi = f2bf(v);
  const float h = bf2f(hi);
  rest = __builtin_isinf(h) ? 0.f : v - h;
}

// ---------------------------------------------------------------------------
// grouping, and weights laid out as matrix operands
// ---------------------------------------------------------------------------

// inclusive sums over the workgroup's threads of three counters
__device__ __forceinline__ void scan3(int (&v)[3], int* wave_sums, int waves) {   // later waves hold zeros
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
  for (int w = 0; w < min(wave, waves); ++w)
#pragma unroll
    for (int q = 0; q < 3; ++q) v[q] += wave_sums[w * 3 + q];
}

// The weights of a slot as operands: block (rb, kb) is rows 16 rb .. + 15 and
// columns KSTEP kb .. + KSTEP - 1 (the reduction) of a rows x ks matrix, one
// 16-byte chunk of each lane, 1 KB in a row.  Read from the pool as it lies,
// an operand is 16 pieces of 64 bytes a whole weight row apart, which one L2
// channel may have to serve alone; packed it is one contiguous kilobyte.
template <typename T>
struct Pack {
  const T* src;         // [slots][rows][ks], or [slots][ks][rows] if `across`; null: no job
  T* dst;
  int32_t rows, ks;
  int32_t across;
  int32_t by_k;         // block order: kb rows / 16 + rb, else rb ks / KSTEP + kb
  int32_t wgs;          // workgroups per slot (or request)
  __host__ __device__ int64_t blocks() const {
    return ((rows + 15) / 16) * (int64_t)((ks + Step<T>::K - 1) / Step<T>::K);
  }
};

constexpr int PACK_BLOCKS = 16;   // of a workgroup: one per wave, whose loads are one latency

template <typename T>
__device__ void pack_blocks(const Pack<T>& j, const Requests& q, int id) {
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K;
  const int unit = id / j.wgs, part = id % j.wgs;
  const int slot = q.by_slot() ? unit : q.id(unit), end_b = q.by_slot() ? q.B : unit;
  if (!q.by_slot() && (slot >= q.slots || q.len(unit) == 0)) return;
  int other = 0;   // a request with rows of the slot: it is used, or an earlier one's already
  for (int b = threadIdx.x; b < end_b; b += GROUP_NT) other |= q.slot[b] == slot && q.len(b) > 0;
  if ((__syncthreads_or(other) != 0) != q.by_slot()) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int RB = (j.rows + 15) / 16, KB = (j.ks + KSTEP - 1) / KSTEP, total = RB * KB;
  const T* src = j.src + (int64_t)slot * j.rows * j.ks;
  T* dst = j.dst + (int64_t)unit * total * (64 * KPC) + lane * KPC;
  const int end = min((part + 1) * PACK_BLOCKS, total);
  for (int at = part * PACK_BLOCKS + wave; at < end; at += GROUP_NT / 64) {
    const int rb = j.by_k ? at % RB : at / KB, kb = j.by_k ? at / RB : at % KB;
    const int row = rb * 16 + i, k = kb * KSTEP + g * KPC;
    uint4 v = zero4();
    if (row < j.rows && k < j.ks) {
      if (!j.across) {
        v = *reinterpret_cast<const uint4*>(src + (int64_t)row * j.ks + k);
      } else {
        T e[KPC];
#pragma unroll
        for (int u = 0; u < KPC; ++u) e[u] = src[(int64_t)(k + u) * j.rows + row];
        __builtin_memcpy(&v, e, 16);
      }
    }
    *reinterpret_cast<uint4*>(dst + (int64_t)at * (64 * KPC)) = v;
  }
}

// Sorts the requests by slot, stably, and lists the rows in that order.  A
// stable order makes every sum over the rows of a slot the same from call to
// call.  Each of the first `group_wgs` workgroups does the whole sort (a few
// thousand cycles for up to 1024 requests) and writes its share of the row
// list and of the tile lists, so no workgroup waits for another; the others
// pack weights.  Bound by its dependent steps, one workgroup deep: 7 us at up to
// 200 requests and 33000 rows, of which the packing (16 slots of 4096 x 32) and
// the row list are hidden.
template <typename T>
__global__ __launch_bounds__(GROUP_NT) void group_kernel(Requests q, Grouped g, int group_wgs, Pack<T> first,
                                                         Pack<T> second, int first_wgs) {
  __shared__ __attribute__((aligned(16))) int32_t ids[GROUP_NT], lens[GROUP_NT], gpos[GROUP_NT], offs[GROUP_NT + 1];
  __shared__ int32_t run[MAX_SLOTS + 1], tile0[MAX_SLOTS + 1], chunk0[MAX_SLOTS + 1], rows_of[MAX_SLOTS + 1];
  __shared__ int32_t first_of[MAX_SLOTS + 1];   // the first request with rows, where weights are packed by request
  __shared__ int wave_sums[3 * GROUP_NT / 64];
  const int tid = threadIdx.x, wg = blockIdx.x;
  if (wg >= group_wgs) {
    const int t = wg - group_wgs;
    if (t < first_wgs) pack_blocks(first, q, t);
    else pack_blocks(second, q, t - first_wgs);
    return;
  }
  const int B = q.count(), S = q.slots, stride = group_wgs * GROUP_NT;
  // rows of each slot
  for (int s = tid; s <= S; s += GROUP_NT) {
    rows_of[s] = 0;
    first_of[s] = INT_MAX;
  }
  // 1024 requests at a time; the first are loaded once
  int id, len;
  auto load = [&](int b0) {
    const int b = b0 + tid, end = min(b0 + GROUP_NT, B);
    id = b < end ? q.id(b) : S + 1;
    len = b < end ? q.len(b) : 0;
    ids[tid] = id;
    lens[tid] = len;
    offs[tid] = q.lo(min(b, end));
    if (tid == 0) offs[GROUP_NT] = q.lo(end);
  };
  load(0);
  __syncthreads();
  if (len) {
    atomicAdd(&rows_of[id], len);
    if (!q.by_slot()) atomicMin(&first_of[id], tid);
  }
  for (int b = GROUP_NT + tid; b < B; b += GROUP_NT) {
    const int more = q.len(b);
    if (more) {
      atomicAdd(&rows_of[q.id(b)], more);
      if (!q.by_slot()) atomicMin(&first_of[q.id(b)], b);
    }
  }
  __syncthreads();
  // first tile and first chunk of each slot; thread t sums slots [t E, (t + 1) E)
  constexpr int EACH = (MAX_SLOTS + 1 + GROUP_NT - 1) / GROUP_NT;
  int own[EACH][3], sum[3] = {0, 0, 0};
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int s = tid * EACH + e, rows = s <= S ? rows_of[s] : 0, tiles = (rows + g.tile - 1) / g.tile;
    own[e][0] = rows;
    own[e][1] = tiles;
    own[e][2] = s < S && g.chunk ? (tiles + g.chunk - 1) / g.chunk : 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] += own[e][k];
  }
  int at[3] = {sum[0], sum[1], sum[2]};
  scan3(at, wave_sums, S / (64 * EACH) + 1);
#pragma unroll
  for (int k = 0; k < 3; ++k) at[k] -= sum[k];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int s = tid * EACH + e;
    if (s <= S) {
      tile0[s] = at[1];
      run[s] = at[1] * g.tile;   // the next free place of the slot
      chunk0[s] = at[2];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) at[k] += own[e][k];
  }
  __syncthreads();
  // tile i belongs to the last slot s with tile0[s] <= i (slots without rows have no tile)
  auto slot_of = [](const int32_t* from, int i, int last) {
    int a = 0, z = last + 1;
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (from[mid] <= i) a = mid;
      else z = mid;
    }
    return a;
  };
  for (int i = wg * GROUP_NT + tid; i < g.tile_cap; i += stride) {
    const int s = slot_of(tile0, i, S), left = rows_of[s] - (i - tile0[s]) * g.tile;
    const int count = min(max(left, 0), g.tile);
    // the comparison keeps it in range where inconsistent offsets give a tile to a slot without rows
    const int pack = q.by_slot() ? s : first_of[s] < B ? first_of[s] : 0;
    g.tiles[i] = Tile{(uint16_t)s, (uint16_t)pack, count};
    if (count)
      for (int u = count; u < g.tile; ++u) g.perm[(int64_t)i * g.tile + u] = -1;
  }
  if (g.chunk) {
    for (int i = wg * GROUP_NT + tid; i < g.chunk_cap; i += stride) {
      const int s = slot_of(chunk0, i, S - 1), k = (i - chunk0[s]) * g.chunk;
      const int from = tile0[s] + k, tiles = min((rows_of[s] + g.tile - 1) / g.tile - k, g.chunk);
      // inside the tile list, whatever inconsistent offsets add up to
      g.chunks[i] = Chunk{s, from, from < 0 ? 0 : max(min(tiles, g.tile_cap - from), 0), 0};
    }
    for (int s = wg * GROUP_NT + tid; s <= S; s += stride) g.slot_chunk[s] = chunk0[s];
  }
  // rows
  const int64_t places = (int64_t)g.tile_cap * g.tile;
  const int wave = tid >> 6;
  for (int b0 = 0; b0 < B; b0 += GROUP_NT) {
    const int nb = min(B - b0, GROUP_NT);
    if (b0) {
      __syncthreads();
      load(b0);
      __syncthreads();
    }
    int before = 0;   // rows of the same slot in earlier requests of the wave
    if (tid < nb) {
      const int4 *i4 = reinterpret_cast<const int4*>(ids), *l4 = reinterpret_cast<const int4*>(lens);
#pragma unroll 4
      for (int u = wave * 16; u < (tid >> 2); ++u) {
        const int4 a = i4[u], l = l4[u];
        before += (a.x == id ? l.x : 0) + (a.y == id ? l.y : 0) + (a.z == id ? l.z : 0) + (a.w == id ? l.w : 0);
      }
      for (int u = tid & ~3; u < tid; ++u) before += ids[u] == id ? lens[u] : 0;
    }
    // one wave after the other takes its places: at 192 requests 2 us less than
    // counting all earlier requests
    for (int w = 0; w * 64 < nb; ++w) {
      if (wave == w && tid < nb) {
        gpos[tid] = run[id] + before;
        if (len) atomicAdd(&run[id], len);
      }
      __syncthreads();
    }
    const int lo = offs[0], hi = offs[nb];
    for (int t = lo + wg * GROUP_NT + tid; t < hi; t += stride) {
      int a = 0, z = nb;   // the last request starting at or before row t (empty ones before it share its start)
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (offs[mid] <= t) a = mid;
        else z = mid;
      }
      const int64_t p = (int64_t)gpos[a] + (t - offs[a]);
      if (t - offs[a] < lens[a] && p >= 0 && p < places) g.perm[p] = t;
    }
  }
}

// ---------------------------------------------------------------------------
// shrink: P[ks][row][j] = sum over a slice of K of X[row][k] W_slot[j][k]
// ---------------------------------------------------------------------------

struct ShrinkArgs {
  const void* X;        // [n][ldx]
  const void* W;        // [slots][r][K], or packed by k
  const int32_t* rank;  // or null: r
  const float* scale;   // or null: 1
  float* P;             // [KS][n][r]; columns past the rank are 0
  const float* H;       // backward: [n][r], or null
  void *Pf, *Hf;        // backward: P and scale H as left operands of the weight gradients, or null
  int64_t ldx, K;
  int32_t n, r, slots, sub, tiles, KS, packed;   // sub: row blocks of 16 RT rows a tile is cut into
  Grouped g;
};

constexpr int SHRINK_WAVES = 4;
constexpr int GRAD_TILE = 64;   // rows of a tile, but for the smallest forward passes

// Operands of the weight gradients: 32 rows (half a tile) of 16 rank columns,
// lane (i, g) holding rows 8 g .. 8 g + 7 of rank column i.  bf16: three
// terms, hi + mid + lo, 1 KB each (2^-27 relative: the gradients are fp32 and
// the other factor is exact in bf16).  fp32: rows 8 g .. + 3, then + 4 .. + 7.
template <typename T> constexpr int grad_parts() { return sizeof(T) == 2 ? 3 : 2; }
template <typename T>
__device__ __forceinline__ char* grad_block(const void* base, int64_t half_tile, int c, int cts) {
  return const_cast<char*>(reinterpret_cast<const char*>(base)) + (half_tile * cts + c) * (grad_parts<T>() * 1024);
}

// Puts rows 4 q4 .. 4 q4 + 3 of a 16-row block, rank column 16 c + i, there.
template <typename T>
__device__ __forceinline__ void put_grad_rows(void* base, int64_t half_tile, int c, int cts, int upper, int q4, int i,
                                              f32x4 v) {
  const int g = 2 * upper + (q4 >> 1), odd = q4 & 1;
  char* to = grad_block<T>(base, half_tile, c, cts) + (g * 16 + i) * 16;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      bf16_t h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float rest;
        split2(v[q], h[q], rest);
        v[q] = rest;
      }
      *reinterpret_cast<uint2*>(to + term * 1024 + odd * 8) =
          make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
    }
  } else {
    *reinterpret_cast<f32x4*>(to + odd * 1024) = v;
  }
}

// Four rows (4 q4 .. + 3 of a tile's 16-row block) of rank column 16 c + i:
// P, and in a backward pass the operands of the weight gradients.
template <typename T>
__device__ __forceinline__ void shrink_out(const ShrinkArgs& p, float* P, f32x4 v, const int (&rows)[4], int tile,
                                           int block, int c, int i, int q4, int rank, float scale) {
  const int j = 16 * c + i;
  f32x4 h = {0.f, 0.f, 0.f, 0.f};
  if (p.Hf) {   // the four loads together: none is conditional
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = p.H[(int64_t)max(rows[q], 0) * p.r + min(j, p.r - 1)];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = rows[q] >= 0 && j < rank ? h[q] * scale : 0.f;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = rows[q] < 0 ? 0.f : v[q] * scale;
    if (rows[q] >= 0 && j < p.r) P[(int64_t)rows[q] * p.r + j] = v[q];
  }
  if (p.Pf && 16 * c < rank) {
    const int64_t half = (int64_t)tile * 2 + (block >> 1);
    const int cts = (p.r + 15) >> 4;
    put_grad_rows<T>(p.Pf, half, c, cts, block & 1, q4, i, v);
    put_grad_rows<T>(p.Hf, half, c, cts, block & 1, q4, i, h);
  }
}

// Calls f with the number of 16-column blocks as a constant: n, rounded up to
// a power of two, at most CT.
template <int CT, class F>
__device__ __forceinline__ void with_blocks(int n, F&& f) {
  if constexpr (CT == 1) {
    f(std::integral_constant<int, 1>());
  } else {
    if (n > CT / 2) f(std::integral_constant<int, CT>());
    else with_blocks<CT / 2>(n, f);
  }
}

// Lines u0 .. u1 - 1 (128 bytes of each row, two k-steps) of a wave's RT row
// blocks by N weight blocks, the next line in flight.  Eight lanes load a row's
// line; through LDS (of the wave alone, no barrier) its chunks come to the
// lanes that hold them as operands.  Loaded straight into place, an operand is
// 16 rows in 16 neighbouring lanes, and whichever 4 lanes the address unit
// takes together want 4 lines: 32928 x 4096 at r = 64 97 us against 92, 5003 x
// 4096 at r = 32 12.4 and 11.0, 1031 x 1024 in fp32 8.6 and 6.2.  Three lines
// in flight spill.  No load is conditional: behind a branch the compiler could
// not count the loads in flight and would wait for all of them.  Lines and
// rows past the end repeat the last, and the one line that K may end in stands
// by itself.
template <typename T, int RT, int N, int CT>
__device__ __forceinline__ void shrink_slice(f32x4 (&acc)[RT][CT], const T* const (&xr)[RT][2], const T* w, char* lds,
                                             const ShrinkArgs& p, int lane, int u0, int u1, int cts) {
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K, LINE = 2 * KSTEP, D = 2;
  const int i = lane & 15, g = lane >> 4, chunk = lane & 7;
  const int wstep = p.packed ? cts * 64 * KPC : KSTEP;
  int64_t wr[N];
#pragma unroll
  for (int c = 0; c < N; ++c)   // rows past the pool's r repeat the last one; their sums are dropped
    wr[c] = p.packed ? (int64_t)min(c, cts - 1) * 64 * KPC : (int64_t)min(16 * c + i, p.r - 1) * p.K;
  const bool ragged = (int64_t)u1 * LINE > p.K && u0 < u1;
  const int n = u1 - u0 - (ragged ? 1 : 0);
  // chunk c of row r lies at place c ^ (r / 2 % 8) of the row's 128 bytes: 16 lanes reach all banks either way
  char* to[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) to[h] = lds + (8 * h + (lane >> 3)) * 128 + (chunk ^ (4 * h + (lane >> 4))) * 16;
  const char* from[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) from[k] = lds + i * 128 + ((4 * k + g) ^ (i >> 1)) * 16;
  auto put = [&](const u32x4(&x)[RT][2]) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4*>(to[h] + a * 2048) = x[a][h];
    __builtin_amdgcn_wave_barrier();
  };
  auto mul = [&](int k, const uint4(&v)[N]) {
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      const uint4 x = *reinterpret_cast<const uint4*>(from[k] + a * 2048);
#pragma unroll
      for (int c = 0; c < N; ++c) Step<T>::mma(acc[a][c], x, v[c]);
    }
  };
  if (n > 0) {
    // The next line's weights are loaded with its rows, except where they would
    // spill (r = 128, backward at 32928 rows: 349 us against 357).
    constexpr bool AHEAD = RT * N < 16;
    constexpr int DW = AHEAD ? D : 1;
    u32x4 x[D][RT][2];
    uint4 v[DW][2][N];
    auto load_w = [&](int d, int u) {
      u = u0 + min(u, n - 1);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < N; ++c)
          v[d % DW][k][c] = *reinterpret_cast<const uint4*>(w + wr[c] + (int64_t)(2 * u + k) * wstep);
    };
    auto load_x = [&](int d, int u) {
      u = u0 + min(u, n - 1);
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[d][a][h] = *reinterpret_cast<const u32x4*>(xr[a][h] + (int64_t)u * LINE);
    };
    auto line = [&](int d) {
      put(x[d]);
      mul(0, v[d % DW][0]);
      mul(1, v[d % DW][1]);
    };
    load_x(0, 0);
    if (AHEAD) load_w(0, 0);
    int u = 0;
    for (; u + D <= n; u += D)
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (!AHEAD) load_w(d, u + d);
        load_x((d + 1) % D, u + d + 1);
        if (AHEAD) load_w((d + 1) % D, u + d + 1);
        line(d);
      }
    if (u < n) {
      if (!AHEAD) load_w(0, u);
      line(0);
    }
  }
  if (ragged) {
    const int64_t k0 = (int64_t)(u1 - 1) * LINE;
    const bool in = k0 + chunk * KPC < p.K;   // lanes past K read the line's first chunk and use zeros
    u32x4 x[RT][2];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(xr[a][h] + k0 - (in ? 0 : chunk * KPC)), none = {0u, 0u, 0u, 0u};
        x[a][h] = in ? u : none;
      }
    put(x);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k0 + k * KSTEP >= p.K) break;
      const bool has = k0 + k * KSTEP + g * KPC < p.K;
      const int back = has || p.packed ? 0 : g * KPC;
      uint4 v[N];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        v[c] = *reinterpret_cast<const uint4*>(w + wr[c] + (int64_t)(2 * (u1 - 1) + k) * wstep - back);
        v[c] = has ? v[c] : zero4();
      }
      mul(k, v);
    }
  }
}

// One workgroup: 16 RT rows of one slot, one of KS slices of K, which its
// waves divide again; their sums meet in LDS.  The weights come from the L2,
// one operand per 16 rank columns for every RT operands of X.  Bound by the
// rows: 32928 x 1024, r = 16 13.7 us (4.9 TB/s, X in the Infinity Cache);
// 32928 x 4096, r = 64, with the gradients' operands 91 us (270 MB read, 50
// written: 3.5 TB/s), where a tile's 512 KB of weights come from the L2 again
// for every 32 rows and the last third of the workgroups is a second round.
// Tiles of 64 rows with the weights in LDS were slower (125 us where this form
// took 110), as was RT = 4.  RT = 2 at r = 64 spills 3 registers.
template <typename T, int RT, int CT>
__global__ __launch_bounds__(SHRINK_WAVES * 64, CT > 4 ? 2 : 3) void shrink_kernel(ShrinkArgs p) {
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K, W = SHRINK_WAVES;
  constexpr int CB = CT < 4 ? CT : 4;      // 16-column blocks joined at a time
  // a wave's lines of X, then its part of the sums
  constexpr int WAVE_LDS = 1024 * (2 * RT > CB ? 2 * RT : CB);
  __shared__ __attribute__((aligned(16))) char lds[W][WAVE_LDS];
  auto red = [&](int w, int c, int l) { return reinterpret_cast<f32x4*>(lds[w]) + c * 64 + l; };
  const int tile = blockIdx.x / (p.sub * p.KS), rem = blockIdx.x % (p.sub * p.KS);
  const int sub = rem / p.KS, ks = rem % p.KS;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15;
  const int g = lane >> 4;
  const Tile t = p.g.tiles[tile];
  // the operands of the weight gradients are whole half tiles, zero past the rows
  if (t.count <= (p.Pf ? sub * 16 * RT & ~31 : sub * 16 * RT)) return;
  const bool none = t.slot >= p.slots;
  int row_of[RT];
#pragma unroll
  for (int a = 0; a < RT; ++a) row_of[a] = tile_row(p.g, tile, (sub * RT + a) * 16 + i, p.n);
  const int rank = none ? 0 : p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const float scale = none || !p.scale ? 1.f : p.scale[t.slot];
  const int nct = (rank + 15) >> 4, cts = (p.r + 15) >> 4;
  f32x4 acc[RT][CT] = {};
  const int any = __shfl(row_of[0], 0);   // a row to read in the place of one that is not there
  if (rank > 0 && any >= 0) {
    const T* xr[RT][2];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = __shfl(row_of[a], 8 * h + (lane >> 3));
        xr[a][h] = reinterpret_cast<const T*>(p.X) + (int64_t)(row < 0 ? any : row) * p.ldx + (lane & 7) * KPC;
      }
    const int steps = (int)cdiv64(p.K, KSTEP), lines = (steps + 1) >> 1, per = (lines + p.KS * W - 1) / (p.KS * W);
    const int u0 = (ks * W + wave) * per, u1 = min(u0 + per, lines);
    const T* wbase = reinterpret_cast<const T*>(p.W) + (p.packed ? (int64_t)t.pack * steps * cts * 64 * KPC + lane * KPC
                                                                 : (int64_t)t.slot * p.r * p.K + g * KPC);
    with_blocks<CT>(nct, [&](auto blocks) {
      constexpr int N = decltype(blocks)::value;
      shrink_slice<T, RT, N, CT>(acc, xr, wbase, lds[wave], p, lane, u0, u1, cts);
    });
  }
  // join the waves: D[row][j] of a 16x16 block sits at lane j + 16 (row / 4), register row % 4
  float* P = p.P + (int64_t)ks * p.n * p.r;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int cb = 0; cb < CT; cb += CB) {
      if (16 * cb >= p.r) break;
      if (a + cb) __syncthreads();   // the wave's own lines before it need none
#pragma unroll
      for (int c = 0; c < CB; ++c)
        if (cb + c < nct) *red(wave, c, lane) = acc[a][cb + c];
      __syncthreads();
      // four rows of one column a thread: what one lane of the product holds
      for (int e = tid; e < 64 * CB; e += W * 64) {
        const int c = cb + (e >> 6), l = e & 63, j = 16 * c + (l & 15), q4 = l >> 4;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (j < rank)
#pragma unroll
          for (int w = 0; w < W; ++w) v += *red(w, e >> 6, l);
        int rows[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) rows[q] = __shfl(row_of[a], 4 * q4 + q);
        shrink_out<T>(p, P, v, rows, tile, sub * RT + a, c, l & 15, q4, rank, scale);
      }
    }
}

// ---------------------------------------------------------------------------
// the gradients' chunks joined
// ---------------------------------------------------------------------------

// Sums the chunks of each slot in order: dA[s][j][c], and dB[s][c][j]
// (transposed through LDS).  Rows past a slot's rank, and slots without rows,
// are zero.  One workgroup: 64 columns and 16 rank columns of one slot, so that
// even one slot's join is spread over the card (13 us against 86 with a
// workgroup to all rank columns, 4 slots of (1024 + 4096) x 64); it rides in the
// expand's launch, beside rows that do not wait for it.
struct JoinArgs {
  const float* part[2];   // dB's, dA's
  float* out[2];
  int64_t C[2];
  int32_t blocks[2];
  const int32_t* rank;
  int32_t r;
  Grouped g;
};

// The chunks of a slot; one that is alone needs no join: its sums are the
// gradients, which grad_kernel writes itself (1500 rows of 60 slots at r = 128
// 250 us against 370, whose time is the 250 MB of gradients).
__device__ __forceinline__ void slot_chunks(const Grouped& g, int slot, int& lo, int& hi) {
  lo = min(max(g.slot_chunk[slot], 0), g.chunk_cap);
  hi = min(g.slot_chunk[slot + 1], g.chunk_cap);
}
__device__ __forceinline__ bool lone_chunk(const Grouped& g, int slot, int lo, int hi) {
  return hi - lo == 1 && g.chunks[lo].slot == slot && g.chunks[lo].tiles > 0;
}

constexpr int JOIN_LDS = 16 * 68;

__device__ __forceinline__ void join_block(const JoinArgs& p, int id, float* lds) {
  const int which = id >= p.blocks[0];
  id -= which ? p.blocks[0] : 0;
  if (which && id >= p.blocks[1]) return;
  const int64_t C = p.C[which];
  const int cbs = (int)cdiv64(C, 64), rbs = (p.r + 15) >> 4;
  const int cb = id % cbs, rb = id / cbs % rbs, slot = id / cbs / rbs;
  const int rank = p.rank ? min(max(p.rank[slot], 0), p.r) : p.r;
  int lo, hi;
  slot_chunks(p.g, slot, lo, hi);
  const bool lone = lone_chunk(p.g, slot, lo, hi);
  if (lone && rb * 16 + 16 <= rank) return;
  const int x = (threadIdx.x & 15) * 4, y = threadIdx.x >> 4, j = rb * 16 + y;
  const int64_t c = (int64_t)cb * 64 + x, step = (int64_t)p.r * C;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (j < rank && c < C && !lone) {
    const float* s = p.part[which] + (int64_t)lo * step + (int64_t)j * C + c;
#pragma unroll 8
    for (int k = lo; k < hi; ++k, s += step) {
      const float4 u = *reinterpret_cast<const float4*>(s);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
  }
  if (which) {
    if (j < p.r && c < C && !(lone && j < rank))
      *reinterpret_cast<float4*>(p.out[1] + ((int64_t)slot * p.r + j) * C + c) = v;
    return;
  }
  *reinterpret_cast<float4*>(&lds[y * 68 + x]) = v;
  __syncthreads();
  // 4 rank columns of a column a thread
  const int cc = threadIdx.x >> 2, j4 = (threadIdx.x & 3) * 4;
  const int64_t oc = (int64_t)cb * 64 + cc;
  if (oc < C && rb * 16 + j4 < p.r && !(lone && rb * 16 + j4 < rank))
    *reinterpret_cast<float4*>(p.out[0] + ((int64_t)slot * C + oc) * p.r + rb * 16 + j4) =
        make_float4(lds[j4 * 68 + cc], lds[(j4 + 1) * 68 + cc], lds[(j4 + 2) * 68 + cc], lds[(j4 + 3) * 68 + cc]);
}

__global__ __launch_bounds__(256) void grad_join_kernel(JoinArgs p) {
  __shared__ __attribute__((aligned(16))) float lds[JOIN_LDS];
  join_block(p, blockIdx.x, lds);
}

// ---------------------------------------------------------------------------
// expand: out[row][c] = base[row][c] + sum_j scale P[row][j] W_slot[c][j]
// ---------------------------------------------------------------------------

struct ExpandArgs {
  const float* P;       // [KS][n][r]
  const void* W;        // [slots][C][r], or packed by rows
  const int32_t* rank;  // or null: r
  const float* scale;   // or null: 1
  const void* base;     // [n][ldb], or null: 0
  void* out;            // [n][ldo]
  float* H;             // [n][r] receives the sum over ks of P, or null
  int64_t ldb, ldo, C;
  int32_t n, r, slots, KS, tiles, col_blocks, sub, packed;   // sub: row blocks of 16 RT rows a tile is cut into
  Grouped g;
};

constexpr int EXPAND_COLS = 256;   // columns of a workgroup, 64 of each wave
// Row blocks that follow each other on one XCD, which takes all their columns
// (P and the row list are in its L2 then).  An eighth of the list to each XCD
// would leave the last ones the places past the last tile: 5003 x 4096 of 16
// slots 24.5 us against 22.5, with runs of 1 and 4 22.8 and 22.3; 192 rows of 64
// slots 27 against 26.5, 26.8 and 27.9.
constexpr int XCD_RUN = 2;

// One workgroup: 16 RT rows of a tile, 256 columns.  P is summed over its
// slices, scaled and put in LDS once: in bf16 as two terms, hi + lo, so that
// Y carries no rounding but its own; the extra product is cheap beside the
// row traffic.  Weights stay in registers for all the rows.  A product leaves
// 4 columns of one row in a lane; through LDS (wave by wave, no barrier) the
// results come to lanes that hold 16 bytes of a row, 8 lanes to a 128-byte
// line, the form in which base is read and the result written.
// Bound by base and result: 32928 x 4096, r = 16 100 us (540 MB, 5.4 TB/s); with
// few rows a slot by the weights: 192 rows of 61 slots, 12288 columns, ranks to
// 64, 26 us (about 65 MB).  A persistent form with the next tile's rows in flight
// was slower (134 us; 33): its registers cost a workgroup per CU.
template <typename T, int RT, int NK>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs p, JoinArgs join, int join_wgs) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int KPC = Step<T>::KPC, KSTEP = Step<T>::K, TERMS = BF ? 2 : 1;
  constexpr int PITCH = NK * KSTEP * (int)sizeof(T) + 16;   // bytes of a row in LDS; 16 more spread the banks
  constexpr int DP = 68;                 // floats of a row of 64 results in LDS, likewise
  constexpr int LPR = 64 / KPC;          // lanes to a row of 64 columns
  constexpr int RPI = 64 / LPR, PIECES = 16 / RPI;   // rows of a load; loads for 16 rows
  __shared__ __attribute__((aligned(16))) char hs[TERMS * 16 * RT * PITCH];
  __shared__ __attribute__((aligned(16))) float ds[4][16 * DP];
  static_assert(sizeof(ds) >= JOIN_LDS * sizeof(float), "the join's LDS");
  // a backward pass joins the weight gradients in the same launch
  if ((int)blockIdx.x < join_wgs) return join_block(join, blockIdx.x, ds[0]);
  const int id = blockIdx.x - join_wgs, at = (id >> 3) / p.col_blocks, cb = (id >> 3) % p.col_blocks;
  const int part = (at / XCD_RUN * 8 + (id & 7)) * XCD_RUN + at % XCD_RUN, sub = part % p.sub, tile = part / p.sub;
  if (tile >= p.tiles) return;
  const Tile t = p.g.tiles[tile];
  if (t.count <= sub * 16 * RT) return;
  const bool none = t.slot >= p.slots;
  if (none && p.base == p.out && p.ldb == p.ldo && !(p.H && cb == 0)) return;   // in place: nothing to add
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  int row_of[RT];
#pragma unroll
  for (int a = 0; a < RT; ++a) row_of[a] = tile_row(p.g, tile, (sub * RT + a) * 16 + i, p.n);
  const int rank = none ? 0 : p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const int nk = (rank + KSTEP - 1) / KSTEP;
  const float scale = none || !p.scale ? 1.f : p.scale[t.slot];
  const int64_t c0 = (int64_t)cb * EXPAND_COLS + wave * 64;
  // weights of the wave's 64 columns: 4 left operands per k-step
  const int nks = (p.r + KSTEP - 1) / KSTEP;
  uint4 wv[4][NK];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int64_t col = c0 + 16 * h + i;
    const T* wr = reinterpret_cast<const T*>(p.W) +
                  (p.packed ? (((int64_t)t.pack * ((p.C + 15) >> 4) + ((c0 >> 4) + h)) * nks * 64 + lane) * KPC
                            : ((int64_t)t.slot * p.C + col) * p.r + g * KPC);
    const int wstep = p.packed ? 64 * KPC : KSTEP;
#pragma unroll
    for (int k = 0; k < NK; ++k)
      wv[h][k] = k < nk && col < p.C && k * KSTEP + g * KPC < rank
                     ? *reinterpret_cast<const uint4*>(wr + k * wstep)
                     : zero4();
  }
  // the rows of base, all in flight before the first is needed
  const int lr = lane / LPR, lc = (lane % LPR) * KPC;
  const int64_t mine = c0 + lc;
  uint4 bv[RT][PIECES];
  int rv[RT][PIECES];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int row = __shfl(row_of[a], q * RPI + lr);
      rv[a][q] = mine < p.C ? row : -1;
      bv[a][q] = rv[a][q] >= 0 && p.base
                     ? load_once(reinterpret_cast<const T*>(p.base) + (int64_t)row * p.ldb + mine)
                     : zero4();
    }
  // P: thread tid takes rank columns 4 (tid % 16), + 64, ... of row tid / 16 of each 16-row block
  const bool keep_h = p.H && cb == 0;
  if (rank > 0 || keep_h) {
    const int wide = max(nk * KSTEP, keep_h ? p.r : 0) >> 2;   // groups of 4 rank columns, zero past the rank
    const int rr = tid >> 4;
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      const int row = __shfl(row_of[a], rr);   // lanes 0 .. 15 hold the block's rows
      for (int jj = tid & 15; jj < wide; jj += 16) {
        const int j = jj * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (row >= 0 && j < rank)
          for (int ks = 0; ks < p.KS; ++ks) {
            const float4 u = *reinterpret_cast<const float4*>(p.P + ((int64_t)ks * p.n + row) * p.r + j);
            v[0] += u.x;
            v[1] += u.y;
            v[2] += u.z;
            v[3] += u.w;
          }
        if (keep_h && row >= 0 && j < p.r)
          *reinterpret_cast<float4*>(p.H + (int64_t)row * p.r + j) = make_float4(v[0], v[1], v[2], v[3]);
        if (j >= nk * KSTEP) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= scale;
        char* to = hs + (16 * a + rr) * PITCH + j * (int)sizeof(T);
        if constexpr (BF) {
          bf16_t hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float rest;
            split2(v[q], hi[q], rest);
            lo[q] = f2bf(rest);
          }
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
          *reinterpret_cast<uint2*>(to + 16 * RT * PITCH) =
              make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
        } else {
          *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
  }
  __syncthreads();
  if (c0 >= p.C) return;
  if (rank & (KPC - 1)) {   // what the pool holds past a rank that ends inside a chunk is not used
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int j = k * KSTEP + g * KPC;
        uint32_t w[4] = {wv[h][k].x, wv[h][k].y, wv[h][k].z, wv[h][k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (BF) {
            if (j + 2 * q + 1 >= rank) w[q] &= 0xffffu;
            if (j + 2 * q >= rank) w[q] = 0u;
          } else {
            if (j + q >= rank) w[q] = 0u;
          }
        }
        wv[h][k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
  }
  float* d = ds[wave];
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    if ((sub * RT + a) * 16 >= t.count) break;
    f32x4 acc[4] = {};
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
    // columns 16 h + 4 g .. + 3 of row i
#pragma unroll
    for (int h = 0; h < 4; ++h) *reinterpret_cast<f32x4*>(d + i * DP + 16 * h + 4 * g) = acc[h];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const float* s = d + (q * RPI + lr) * DP + lc;
      const uint4& b = bv[a][q];
      uint4 o;
      if constexpr (BF) {
        const float4 u = *reinterpret_cast<const float4*>(s), w = *reinterpret_cast<const float4*>(s + 4);
        auto pair = [](uint32_t x, float lo, float hi) {
          return (uint32_t)f2bf(__uint_as_float(x << 16) + lo) |
                 (uint32_t)f2bf(__uint_as_float(x & 0xffff0000u) + hi) << 16;
        };
        o = make_uint4(pair(b.x, u.x, u.y), pair(b.y, u.z, u.w), pair(b.z, w.x, w.y), pair(b.w, w.z, w.w));
      } else {
        const float4 u = *reinterpret_cast<const float4*>(s);
        o = make_uint4(__float_as_uint(__uint_as_float(b.x) + u.x), __float_as_uint(__uint_as_float(b.y) + u.y),
                       __float_as_uint(__uint_as_float(b.z) + u.z), __float_as_uint(__uint_as_float(b.w) + u.w));
      }
      if (rv[a][q] >= 0) store_once(reinterpret_cast<T*>(p.out) + (int64_t)rv[a][q] * p.ldo + mine, o);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// a few rows: both products in one launch
// ---------------------------------------------------------------------------

struct DirectArgs {
  const void *X, *A, *B, *base;
  const int32_t* rank;
  const float* scale;
  void* out;
  float* H;
  int64_t ldx, ldb, ldo, c1, c2;
  int32_t r, col_blocks;
  Requests q;
};

constexpr int DIRECT_NT = 512;   // threads and columns of a workgroup

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[Step<T>::KPC]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(T) == 2) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    } else {
      v[q] = __uint_as_float(w[q]);
    }
  }
}

// One workgroup: one row, 512 columns.  Every workgroup of a row forms the
// row's whole H again from the L2: r c1 weights, which one CU reads in about
// a microsecond at r = 16, c1 = 4096, where two more launches cost several.
// The waves are JG groups of 16 rank columns (JG 16 >= r) times W / JG parts
// of c1; weights are read a row of A at a time, 1 KB a wave.  Bound by latency:
// 4 rows, 4096 -> 4096, r = 16 6.6 us.  Above r = 16 bf16 spills 5 or 6 of its
// 128 registers; a call of 5 rows takes 14 us at r = 64, 24 at r = 128.
template <typename T, int JG>
__global__ __launch_bounds__(DIRECT_NT, 4) void direct_kernel(DirectArgs p) {
  constexpr int KPC = Step<T>::KPC, W = DIRECT_NT / 64, KG = W / JG, JB = 16;
  __shared__ float part[KG][JG * JB], hs[JG * JB];
  const int row = blockIdx.x / p.col_blocks, cb = blockIdx.x % p.col_blocks;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, jg = wave % JG, kg = wave / JG;
  // the row's request: as many as start at or before it, less one
  int b = 0;
  for (int b0 = 1; b0 < p.q.count(); b0 += DIRECT_NT)
    b += __syncthreads_count(b0 + tid < p.q.count() && p.q.lo(b0 + tid) <= row);
  const int slot = p.q.id(b);
  const bool none = slot >= p.q.slots;
  const int rank = none ? 0 : p.rank ? min(max(p.rank[slot], 0), p.r) : p.r;
  const float scale = none || !p.scale ? 1.f : p.scale[slot];
  const int64_t c = (int64_t)cb * DIRECT_NT + tid;
  const T* x = reinterpret_cast<const T*>(p.X) + (int64_t)row * p.ldx;
  float y = c < p.c2 && p.base ? TT<T>::to_f(reinterpret_cast<const T*>(p.base)[(int64_t)row * p.ldb + c]) : 0.f;
  if (!none) {
    const T* a = reinterpret_cast<const T*>(p.A) + ((int64_t)slot * p.r + jg * JB) * p.c1;
    float acc[JB] = {};
    for (int64_t k = (int64_t)(kg * 64 + lane) * KPC; k < p.c1; k += KG * 64 * KPC) {
      float xv[KPC];
      unpack<T>(*reinterpret_cast<const uint4*>(x + k), xv);
      uint4 w[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j)   // the rank is not waited for: its rows' sums are dropped below
        w[j] = jg * JB + j < p.r ? *reinterpret_cast<const uint4*>(a + (int64_t)j * p.c1 + k) : zero4();
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        float wv[KPC];
        unpack<T>(w[j], wv);
#pragma unroll
        for (int e = 0; e < KPC; ++e) acc[j] += xv[e] * wv[e];
      }
    }
    // 16 sums over 64 lanes: each step halves what a lane holds, lane bits 5 .. 2 pick the value
#pragma unroll
    for (int half = JB / 2, d = 32; half >= 1; half >>= 1, d >>= 1)
#pragma unroll
      for (int q = 0; q < half; ++q) {
        const float keep = lane & d ? acc[q + half] : acc[q], give = lane & d ? acc[q] : acc[q + half];
        acc[q] = keep + __shfl_xor(give, d);
      }
    acc[0] += __shfl_xor(acc[0], 2);
    acc[0] += __shfl_xor(acc[0], 1);
    if ((lane & 3) == 0)
      part[kg][jg * JB + (lane >> 5 & 1) * 8 + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = acc[0];
    __syncthreads();
    if (tid < JG * JB) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < KG; ++w) v += part[w][tid];
      hs[tid] = tid < rank ? v : 0.f;
    }
    __syncthreads();
  }
  if (p.H && cb == 0 && tid < p.r) p.H[(int64_t)row * p.r + tid] = tid < rank ? hs[tid] : 0.f;
  if (c >= p.c2) return;
  const T* wb = reinterpret_cast<const T*>(p.B) + ((int64_t)slot * p.c2 + c) * p.r;
  float d = 0.f;
  for (int j = 0; j < rank; j += KPC) {
    float wv[KPC];
    unpack<T>(*reinterpret_cast<const uint4*>(wb + j), wv);
#pragma unroll
    for (int e = 0; e < KPC; ++e) d += j + e < rank ? hs[j + e] * wv[e] : 0.f;
  }
  reinterpret_cast<T*>(p.out)[(int64_t)row * p.ldo + c] = TT<T>::from_f(rank > 0 ? y + scale * d : y);
}

// ---------------------------------------------------------------------------
// weight gradients: part[chunk][j][c] = sum over the chunk's rows of
// s P[row][j] V[row][c]   (dA: P = G, V = X;  dB: P = s H, V = dY)
// ---------------------------------------------------------------------------

struct GradSide {
  const void* V;       // [n][ldv]
  const void* Pf;      // left operands, written by the shrink
  float* part;         // [chunk_cap][r][C]
  float* out;          // side 0: dB [slots][C][r], side 1: dA [slots][r][C]
  int64_t ldv, C;
  int32_t col_blocks;
};
struct GradArgs {
  GradSide side[2];
  const int32_t* rank;
  int32_t n, r, slots, chunk_cap, r_groups;
  Grouped g;           // tiles of 64 rows
};

constexpr int CHUNK_TILES = 32;   // most tiles of a chunk: their rows are kept in LDS
template <typename T> constexpr int grad_cols() { return sizeof(T) == 2 ? 128 : 64; }   // columns of a wave

// One workgroup: a chunk of tiles, 4 waves' columns, up to 16 CT rank columns.
// V is read 8 rows by 16 bytes per lane; bf16 is transposed in registers, so
// that each lane holds 8 consecutive rows of a column, the reduction axis
// (operand e of a lane is column 8 i + e of the wave's 128); fp32 products
// take one row of each lane group as it is.  The row factors are operands
// already; the four waves share them through LDS, a half tile at a time,
// double-buffered.  Both are in flight a half tile ahead of the products.
// Chunks keep the sums in order without atomics; the partial sums of a slot
// with several are joined by join_block.  Bound by the rows' loads: X 32928 x 1024 and dY x 4096, r = 64
// 84 us (337 MB, 4.0 TB/s) at two workgroups a CU, which the sums' registers
// allow.
template <typename T, int CT>
__global__ __launch_bounds__(256, 2) void grad_kernel(GradArgs p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int COLS = grad_cols<T>(), PARTS = grad_parts<T>(), BYTES = CT * PARTS * 1024;
  constexpr int NA = (BYTES / 16 + 255) / 256;   // 16-byte loads of a thread for a half tile's operands
  __shared__ __attribute__((aligned(16))) char lds[2][BYTES];
  __shared__ __attribute__((aligned(16))) int rows_of[CHUNK_TILES * GRAD_TILE];
  int id = blockIdx.x;
  const int per0 = p.side[0].col_blocks * p.r_groups * p.chunk_cap;
  const int which = id >= per0;
  id -= which ? per0 : 0;
  const GradSide& v = p.side[which];
  // (chunks from the last to the first, against the order in which the shrink
  // read the rows before, take the same time at 4099 and 32928 rows)
  const int cb = id % v.col_blocks, chunk = id / v.col_blocks % p.chunk_cap;
  const int rg = id / v.col_blocks / p.chunk_cap;
  const Chunk t = p.g.chunks[chunk];
  if (t.tiles <= 0 || t.slot >= p.slots) return;
  const int rank = p.rank ? min(max(p.rank[t.slot], 0), p.r) : p.r;
  const int j0 = rg * 16 * CT;
  if (j0 >= rank) return;
  const int nct = min((rank - j0 + 15) >> 4, CT), cts = (p.r + 15) >> 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  constexpr int E = COLS / 16;   // columns of a lane
  const int64_t col = ((int64_t)cb * 4 + wave) * COLS + i * E;
  const bool live = col < v.C;
  const T* V = reinterpret_cast<const T*>(v.V) + col;
  f32x4 acc[CT][E] = {};
  // the second half of the last tile has no operands if it has no row
  const int last_count = p.g.tiles[t.first + t.tiles - 1].count;
  const int halves = t.tiles * 2 - (last_count <= 32 ? 1 : 0);
  const char* ops = grad_block<T>(v.Pf, (int64_t)t.first * 2, j0 >> 4, cts) + tid * 16;
  const int bytes = nct * PARTS * 1024;

  auto load_v = [&](uint4(&in)[8], int h) {
    const int4* s = reinterpret_cast<const int4*>(rows_of + min(h, halves - 1) * 32 + 8 * g);
    const int4 a = s[0], b = s[1];
    const int rows[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      in[e] = h < halves && live && rows[e] >= 0 ? *reinterpret_cast<const uint4*>(V + (int64_t)rows[e] * v.ldv)
                                                 : zero4();
  };
  auto load_a = [&](uint4(&a)[NA], int h) {
#pragma unroll
    for (int n = 0; n < NA; ++n)
      a[n] = h < halves && tid * 16 + n * 4096 < bytes
                 ? *reinterpret_cast<const uint4*>(ops + (int64_t)h * cts * (PARTS * 1024) + n * 4096)
                 : zero4();
  };
  auto put_a = [&](const uint4(&a)[NA], int h) {
#pragma unroll
    for (int n = 0; n < NA; ++n)
      if (tid * 16 + n * 4096 < bytes) *reinterpret_cast<uint4*>(&lds[h & 1][tid * 16 + n * 4096]) = a[n];
  };
  auto mul = [&](const uint4(&in)[8], int h) {
    const char* a = &lds[h & 1][lane * 16];
    if constexpr (BF) {
      uint4 b[8];
      transpose8x8_b16(in, b);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        if (c < nct)
#pragma unroll
          for (int u = 0; u < PARTS; ++u) {
            const uint4 w = *reinterpret_cast<const uint4*>(a + (c * PARTS + u) * 1024);
#pragma unroll
            for (int e = 0; e < 8; ++e) mma16(acc[c][e], w, b[e]);
          }
    } else {
#pragma unroll
      for (int c = 0; c < CT; ++c)
        if (c < nct)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float w = *reinterpret_cast<const float*>(a + (c * PARTS + (q >> 2)) * 1024 + (q & 3) * 4);
            acc[c][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, __uint_as_float(in[q].x), acc[c][0], 0, 0, 0);
            acc[c][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, __uint_as_float(in[q].y), acc[c][1], 0, 0, 0);
            acc[c][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, __uint_as_float(in[q].z), acc[c][2], 0, 0, 0);
            acc[c][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, __uint_as_float(in[q].w), acc[c][3], 0, 0, 0);
          }
    }
  };

  for (int u = tid; u < halves * 32; u += 256) rows_of[u] = tile_row(p.g, t.first, u, p.n);
  uint4 even[8], odd[8], a[NA];
  load_a(a, 0);
  __syncthreads();
  load_v(even, 0);
  put_a(a, 0);
  __syncthreads();
  for (int h = 0; h < halves; h += 2) {
    load_a(a, h + 1);
    load_v(odd, h + 1);
    mul(even, h);
    put_a(a, h + 1);
    __syncthreads();
    if (h + 1 < halves) {
      load_a(a, h + 2);
      load_v(even, h + 2);
      mul(odd, h + 1);
      put_a(a, h + 2);
      __syncthreads();
    }
  }
  if (!live) return;
  int lo, hi;
  slot_chunks(p.g, t.slot, lo, hi);
  const bool lone = lone_chunk(p.g, t.slot, lo, hi);
  if (lone && !which) {   // dB: 4 rank columns of a column a store, zero past the rank
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int j = j0 + 16 * c + 4 * g;
      if (j >= rank) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const f32x4 a = acc[c][e];
        *reinterpret_cast<float4*>(v.out + ((int64_t)t.slot * v.C + col + e) * p.r + j) =
            make_float4(a[0], j + 1 < rank ? a[1] : 0.f, j + 2 < rank ? a[2] : 0.f, j + 3 < rank ? a[3] : 0.f);
      }
    }
    return;
  }
  float* out = lone ? v.out + (int64_t)t.slot * p.r * v.C : v.part + (int64_t)chunk * p.r * v.C;
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Sizes of a call: tile heights, splits and the workspace.
struct Plan {
  int tile, rt, sub, ert;           // rows of a tile; 16-row blocks of a shrink workgroup, those per tile; of an expand one
  int ks;                           // slices of the reduction in the shrink
  int chunk;                        // tiles of a gradient chunk (backward), else 0
  int packed;                       // weights are packed first
  bool direct;                      // forward: one launch, no workspace
  int64_t tile_cap, chunk_cap;
  size_t perm, tiles, chunks, slot_chunk, P, Ws, We, Pf, Hf, partA, partB, total;
};

int shrink_split(int64_t wgs, int64_t K, int dtype) {
  const int64_t steps = cdiv64(K, dtype == DYRA_BF16 ? 32 : 16);
  int64_t ks = cdiv64(512, wgs);                              // two workgroups per CU
  ks = std::min<int64_t>(ks, cdiv64(steps, 2 * SHRINK_WAVES));   // at least one line per wave
  return (int)std::max<int64_t>(1, std::min<int64_t>(ks, 4));   // more slices cost the expand more than they save
}

Plan make_plan(int64_t slots, int64_t r, int64_t c1, int64_t c2, int64_t n, int64_t B, int dtype, bool backward) {
  Plan q{};
  // One launch where its workgroups fit the card at once and what they read
  // of A again and again stays small.  In graph replays, one launch against
  // three: 4 rows of 4096 -> 4096 at r = 16 5.8 and 14.0 us, 64 rows 9.6 and
  // 15.0, 32 rows at r = 64 (128 MiB of A) 16.3 and 18.3.
  const int64_t direct_wgs = n * cdiv64(c2, DIRECT_NT);
  q.direct = !backward && direct_wgs <= 512 && direct_wgs * r * c1 * (int64_t)elem_bytes(dtype) <= (int64_t)128 << 20;
  if (q.direct) return q;
  const bool small = n <= 512 && !backward;
  q.tile = small ? 16 : GRAD_TILE;
  // Row blocks of a shrink workgroup: two share a weight operand, one makes
  // twice the workgroups.  One against two, forward / backward in us: r = 64,
  // 1024 -> 4096, 4099 rows 38 / 63 and 41 / 59, 8192 49 / 82 and 52 / 78, 16500
  // 84 / 141 and 83 / 135, 32928 148 / 238 and 145 / 219; r = 128, 4096 -> 4096,
  // 4099 rows 63 / 140 and 67 / 130, 12000 131 / 249 and 122 / 241, 32928 337 /
  // 578 and 292 / 535; fp32, r = 64, 1024 -> 1024, 16500 rows 85 / 138 and 88 /
  // 143, 32928 144 / 233 and 145 / 232.
  q.rt = r > 32 && n >= 8192 ? 2 : 1;
  q.sub = q.tile / (16 * q.rt);
  q.ert = small ? 1 : 2;   // 2 against 1 and 4: 109, 114 and 113 us at 32928 x 4096, 19, 18 and 21 at 4099 x 4096
  const int64_t used = std::min(slots + 1, B + 1);   // slots with rows, "no adapter" among them
  q.tile_cap = n / q.tile + used + 1;
  q.packed = backward || (n > 512 && n >= 64 * std::min(slots, B));
  const int64_t wgs = std::max<int64_t>(1, std::min(n, q.tile_cap * q.sub));
  q.ks = backward ? 1 : shrink_split(wgs, c1, dtype);
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += align256((size_t)bytes);
    return here;
  };
  q.perm = take(4 * q.tile_cap * q.tile);
  q.tiles = take((int64_t)sizeof(Tile) * q.tile_cap);
  q.P = take(4 * n * r * q.ks);
  if (q.packed) {
    const int64_t kstep = dtype == DYRA_BF16 ? 32 : 16, kin = backward ? c2 : c1, kout = backward ? c1 : c2;
    const int64_t units = std::min(slots, B);
    q.Ws = take(units * cdiv64(r, 16) * cdiv64(kin, kstep) * 1024);
    q.We = take(units * cdiv64(kout, 16) * cdiv64(r, kstep) * 1024);
  }
  if (backward) {
    const int cols = 4 * (dtype == DYRA_BF16 ? grad_cols<bf16_t>() : grad_cols<float>());
    const int parts = dtype == DYRA_BF16 ? grad_parts<bf16_t>() : grad_parts<float>();
    const int64_t blocks = cdiv64(c1, cols) + cdiv64(c2, cols);
    const int64_t most = std::max<int64_t>(1, 512 / blocks), chunks = std::max((most + 1) / 2, most - std::min(slots, B));
    q.chunk = (int)std::min<int64_t>(CHUNK_TILES, std::max<int64_t>(1, cdiv64(cdiv64(n, GRAD_TILE), chunks)));
    q.chunk_cap = n / ((int64_t)q.chunk * GRAD_TILE) + std::min(slots, B) + 1;
    q.chunks = take((int64_t)sizeof(Chunk) * q.chunk_cap);
    q.slot_chunk = take(4 * (slots + 1));
    q.Pf = take(q.tile_cap * 2 * cdiv64(r, 16) * parts * 1024);
    q.Hf = take(q.tile_cap * 2 * cdiv64(r, 16) * parts * 1024);
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
  g.chunks = reinterpret_cast<Chunk*>(ws + q.chunks);
  g.slot_chunk = reinterpret_cast<int32_t*>(ws + q.slot_chunk);
  g.tile = q.tile;
  g.chunk = q.chunk;
  g.tile_cap = (int32_t)q.tile_cap;
  g.chunk_cap = (int32_t)q.chunk_cap;
  return g;
}

template <typename T>
Pack<T> pack_job(const void* src, void* dst, int64_t rows, int64_t ks, bool across, bool by_k) {
  Pack<T> j{reinterpret_cast<const T*>(src), reinterpret_cast<T*>(dst), (int32_t)rows, (int32_t)ks, across, by_k, 0};
  j.wgs = (int32_t)cdiv64(j.blocks(), PACK_BLOCKS);
  return j;
}

// workgroups that sort
int group_wgs(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(cdiv64(n, 2 * GROUP_NT), 64)); }

template <typename T>
void launch_group(const Requests& rq, const Grouped& g, const Pack<T>& a, const Pack<T>& b, hipStream_t st) {
  const int wgs = group_wgs(rq.n);
  const int64_t units = std::min(rq.slots, rq.B), na = a.src ? units * a.wgs : 0, nb = b.src ? units * b.wgs : 0;
  hipLaunchKernelGGL((group_kernel<T>), dim3((unsigned)(wgs + na + nb)), dim3(GROUP_NT), 0, st, rq, g, wgs, a, b,
                     (int)na);
}

template <typename T, int RT, int CT>
void launch_shrink_as(const ShrinkArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.tiles * a.sub * a.KS);
  hipLaunchKernelGGL((shrink_kernel<T, RT, CT>), dim3(grid), dim3(SHRINK_WAVES * 64), 0, st, a);
}

template <typename T>
void launch_shrink(const ShrinkArgs& a, int rt, hipStream_t st) {
  if (a.r <= 16) launch_shrink_as<T, 1, 1>(a, st);
  else if (a.r <= 32) launch_shrink_as<T, 1, 2>(a, st);
  else if (a.r <= 64) rt == 1 ? launch_shrink_as<T, 1, 4>(a, st) : launch_shrink_as<T, 2, 4>(a, st);
  else rt == 1 ? launch_shrink_as<T, 1, 8>(a, st) : launch_shrink_as<T, 2, 8>(a, st);
}

template <typename T, int RT>
void launch_expand_rt(const ExpandArgs& a, const JoinArgs& j, int join_wgs, unsigned grid, hipStream_t st) {
  const int nk = (a.r + Step<T>::K - 1) / Step<T>::K;
  const dim3 nt(256);
  if (nk <= 1) hipLaunchKernelGGL((expand_kernel<T, RT, 1>), dim3(grid), nt, 0, st, a, j, join_wgs);
  else if (nk <= 2) hipLaunchKernelGGL((expand_kernel<T, RT, 2>), dim3(grid), nt, 0, st, a, j, join_wgs);
  else if (nk <= 4) hipLaunchKernelGGL((expand_kernel<T, RT, 4>), dim3(grid), nt, 0, st, a, j, join_wgs);
  else if constexpr (sizeof(T) == 4)
    hipLaunchKernelGGL((expand_kernel<T, RT, 8>), dim3(grid), nt, 0, st, a, j, join_wgs);
}

// workgroups of the expand but for those of a join: whole runs of every XCD
int64_t expand_wgs(int64_t row_blocks, int64_t col_blocks) {
  return cdiv64(row_blocks, 8 * XCD_RUN) * (8 * XCD_RUN) * col_blocks;
}

// join: the weight gradients' join of a backward pass, or null
template <typename T>
void launch_expand(const ExpandArgs& a, int ert, const JoinArgs* join, hipStream_t st) {
  JoinArgs j{};
  int wgs = 0;
  if (join) {
    j = *join;
    wgs = (j.blocks[0] + j.blocks[1] + 7) & ~7;   // the XCDs of the others stay as they are
  }
  const unsigned grid = (unsigned)(expand_wgs((int64_t)a.tiles * a.sub, a.col_blocks) + wgs);
  if (ert == 1) launch_expand_rt<T, 1>(a, j, wgs, grid, st);
  else launch_expand_rt<T, 2>(a, j, wgs, grid, st);
}

template <typename T>
int forward_impl(const dyra_adapters& ad, const void* X, int64_t ldx, const void* base, int64_t ldb, void* Y,
                 int64_t ldy, float* H, const Requests& rq, const Plan& q, char* ws, hipStream_t st) {
  if (q.direct) {
    const int blocks = (int)cdiv64(ad.c2, DIRECT_NT);
    const DirectArgs da{X, ad.A, ad.B, base, ad.rank, ad.scale, Y, H, ldx, ldb, ldy, ad.c1, ad.c2, ad.r, blocks, rq};
    const dim3 grid((unsigned)(rq.n * blocks)), nt(DIRECT_NT);
    if (ad.r <= 16) hipLaunchKernelGGL((direct_kernel<T, 1>), grid, nt, 0, st, da);
    else if (ad.r <= 32) hipLaunchKernelGGL((direct_kernel<T, 2>), grid, nt, 0, st, da);
    else if (ad.r <= 64) hipLaunchKernelGGL((direct_kernel<T, 4>), grid, nt, 0, st, da);
    else hipLaunchKernelGGL((direct_kernel<T, 8>), grid, nt, 0, st, da);
    return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
  }
  const Grouped g = grouped(q, ws);
  const void *Ws = ad.A, *We = ad.B;
  Pack<T> pa{}, pb{};
  if (q.packed) {
    pa = pack_job<T>(ad.A, ws + q.Ws, ad.r, ad.c1, false, true);
    pb = pack_job<T>(ad.B, ws + q.We, ad.c2, ad.r, false, false);
    Ws = pa.dst;
    We = pb.dst;
  }
  launch_group<T>(rq, g, pa, pb, st);
  // with one slice the shrink writes H itself
  float* P = H && q.ks == 1 ? H : reinterpret_cast<float*>(ws + q.P);
  const ShrinkArgs sa{X,     Ws,   ad.rank, nullptr,  P,     nullptr,             nullptr, nullptr,  ldx,
                      ad.c1, rq.n, ad.r,    ad.slots, q.sub, (int32_t)q.tile_cap, q.ks,    q.packed, g};
  launch_shrink<T>(sa, q.rt, st);
  const ExpandArgs ea{P,       We,
                      ad.rank, ad.scale,
                      base,    Y,
                      P == H ? nullptr : H, ldb,
                      ldy,     ad.c2,
                      rq.n,    ad.r,
                      ad.slots, q.ks,
                      (int32_t)q.tile_cap, (int32_t)cdiv64(ad.c2, EXPAND_COLS),
                      q.tile / (16 * q.ert), q.packed,
                      g};
  launch_expand<T>(ea, q.ert, nullptr, st);
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
  const Pack<T> pb = pack_job<T>(ad.B, ws + q.Ws, ad.r, ad.c2, true, true);
  const Pack<T> pa = pack_job<T>(dX ? ad.A : nullptr, ws + q.We, ad.c1, ad.r, true, false);
  launch_group<T>(rq, g, pb, pa, st);
  float* P = reinterpret_cast<float*>(ws + q.P);
  if (rq.n) {
    const ShrinkArgs sa{dY,      pb.dst, ad.rank, ad.scale, P,     dA ? H : nullptr,    dA ? ws + q.Pf : nullptr,
                        dA ? ws + q.Hf : nullptr,  lddy,
                        ad.c2,   rq.n,   ad.r,    ad.slots, q.sub, (int32_t)q.tile_cap, 1,
                        1,       g};
    launch_shrink<T>(sa, q.rt, st);
  }
  JoinArgs join{};
  if (dA) {
    float *pdA = reinterpret_cast<float*>(ws + q.partA), *pdB = reinterpret_cast<float*>(ws + q.partB);
    const int cols = 4 * grad_cols<T>();
    if (rq.n) {
      GradArgs ga{{{dY, ws + q.Hf, pdB, dB, lddy, ad.c2, (int32_t)cdiv64(ad.c2, cols)},
                   {X, ws + q.Pf, pdA, dA, ldx, ad.c1, (int32_t)cdiv64(ad.c1, cols)}},
                  ad.rank, rq.n, ad.r, ad.slots, (int32_t)q.chunk_cap, 1, g};
      if (ad.r <= 16) launch_grad<T, 1>(ga, st);
      else if (ad.r <= 32) launch_grad<T, 2>(ga, st);
      else launch_grad<T, 4>(ga, st);
    }
    const int64_t rbs = cdiv64(ad.r, 16);
    const int64_t b0 = cdiv64(ad.c2, 64) * rbs * ad.slots, b1 = cdiv64(ad.c1, 64) * rbs * ad.slots;
    join = JoinArgs{{pdB, pdA}, {dB, dA}, {ad.c2, ad.c1}, {(int32_t)b0, (int32_t)b1}, ad.rank, ad.r, g};
    if (!dX || !rq.n)
      hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)(b0 + b1)), dim3(256), 0, st, join);
  }
  if (dX && rq.n) {
    const ExpandArgs ea{P,       pa.dst,
                        ad.rank, nullptr,
                        dXb,     dX,
                        nullptr, lddb,
                        lddx,    ad.c1,
                        rq.n,    ad.r,
                        ad.slots, 1,
                        (int32_t)q.tile_cap, (int32_t)cdiv64(ad.c1, EXPAND_COLS),
                        q.tile / (16 * q.ert), 1,
                        g};
    launch_expand<T>(ea, q.ert, dA ? &join : nullptr, st);
  }
  return hipGetLastError() == hipSuccess ? DYRA_OK : DYRA_EHIP;
}

// Every launch of a call has fewer than 2^32 threads, as the runtime demands.
// (Workgroup numbers are then below 2^24, and 32-bit in the kernels.)
bool grids_fit(const dyra_adapters& ad, const Plan& q, int64_t n, int64_t B, int dtype, bool backward) {
  const int64_t most = ((int64_t)1 << 32) - 1, kstep = dtype == DYRA_BF16 ? 32 : 16;
  const int64_t cin = backward ? ad.c2 : ad.c1, cout = backward ? ad.c1 : ad.c2;
  const int64_t packs = cdiv64(cdiv64(ad.r, 16) * cdiv64(cin, kstep), PACK_BLOCKS) +
                        cdiv64(cdiv64(cout, 16) * cdiv64(ad.r, kstep), PACK_BLOCKS);
  if (((q.packed ? packs * std::min<int64_t>(ad.slots, B) : 0) + group_wgs(n)) * GROUP_NT > most) return false;
  if (q.tile_cap * q.sub * q.ks * (SHRINK_WAVES * 64) > most) return false;
  const int64_t joins =
      backward ? (cdiv64(ad.c1, 64) + cdiv64(ad.c2, 64)) * cdiv64(ad.r, 16) * ad.slots + 7 : 0;
  if ((expand_wgs(q.tile_cap * (q.tile / (16 * q.ert)), cdiv64(cout, EXPAND_COLS)) + joins) * 256 > most) return false;
  if (!backward) return true;
  const int64_t cols = 4 * (dtype == DYRA_BF16 ? grad_cols<bf16_t>() : grad_cols<float>());
  const int64_t r_groups = cdiv64(ad.r, ad.r <= 16 ? 16 : ad.r <= 32 ? 32 : 64);
  return (cdiv64(ad.c1, cols) + cdiv64(ad.c2, cols)) * r_groups * q.chunk_cap * 256 <= most;
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
  if (!X || !Y || (B && (!offsets_dev || !slots_dev))) return DYRA_EINVAL;
  if (misaligned(X, 15) || misaligned(base, 15) || misaligned(Y, 15) || misaligned(H, 15) ||
      misaligned(workspace, 15) || misaligned(offsets_dev, 3) || misaligned(slots_dev, 3))
    return DYRA_EINVAL;
  if (bad_stride(ldx, ad->c1, dtype) || bad_stride(ldy, ad->c2, dtype) || (base && bad_stride(ldb, ad->c2, dtype)))
    return DYRA_ESHAPE;
  const Plan q = make_plan(ad->slots, ad->r, ad->c1, ad->c2, n, B, dtype, false);
  if (q.total && !workspace) return DYRA_EINVAL;
  if (ws_bytes < q.total) return DYRA_EWORKSPACE;
  if (!q.direct && !grids_fit(*ad, q, n, B, dtype, false)) return DYRA_ESHAPE;
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
  if (!grids_fit(*ad, q, n, B, dtype, true)) return DYRA_ESHAPE;
  const Requests rq{offsets_dev, slots_dev, (int32_t)n, (int32_t)B, ad->slots};
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return dtype == DYRA_BF16
             ? backward_impl<bf16_t>(*ad, X, ldx, dY, lddy, H, dX_base, lddb, dX, lddx, dA, dB, rq, q, ws, st)
             : backward_impl<float>(*ad, X, ldx, dY, lddy, H, dX_base, lddb, dX, lddx, dA, dB, rq, q, ws, st);
}
