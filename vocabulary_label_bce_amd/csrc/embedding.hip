// Embedding lookup with scaling, and its gradient by sorted ids.
//
//   out[i] = s * table[ids[i]]            (zeros where ids[i] is outside [0, V))
//   dtable[v] = s * sum_{i : ids[i] = v} dout[i]
//
// The gradient sorts the (id, position) pairs by id (stable, so that an item's positions stay in order), sums the
// rows of equal ids in float32 and rounds once: no atomics, the same bits every time. A hot item's positions span
// many chunks of the sorted list; each chunk leaves a partial sum for the item it shares with a neighbour, and a
// second kernel joins them.
#include "encoder.h"

namespace cutbce {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortItems = 1024;  // pairs of one sorting workgroup
constexpr int kMaxBits = 10;      // most bits of one sorting pass
constexpr int kChunk = 32;        // sorted pairs that one lane group sums

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct SortPlan {
  int passes, bits;  // digits of `bits` bits; ids outside [0, V) sort as V, behind the others
  int64_t blocks;
};
SortPlan sort_plan(int64_t n, int64_t V) {
  int total = 1;
  while (((int64_t)1 << total) <= V) ++total;
  SortPlan p;
  p.passes = (int)cdiv(total, kMaxBits);
  p.bits = (int)cdiv(total, p.passes);
  p.blocks = cdiv(n, kSortItems);
  return p;
}

struct BwdLayout {
  size_t keys[2], pos[2], counts, totals, part, total;
  int64_t chunks;
};
BwdLayout bwd_layout(int64_t n, int64_t V, int D) {
  const SortPlan p = sort_plan(n, V);
  BwdLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) L.keys[i] = take(4 * (size_t)n), L.pos[i] = take(4 * (size_t)n);
  L.counts = take(((size_t)p.blocks << p.bits) * 4);
  L.totals = take((size_t)4 << p.bits);
  L.chunks = cdiv(n, kChunk);
  L.part = take((size_t)L.chunks * 2 * D * 4);
  L.total = o;
  return L;
}

// Lanes of a row: the power of two that covers its 16-byte chunks, at most a wave.
int lanes_of(int D, int vec) {
  int l = 1;
  while (l < 64 && l * vec < D) l *= 2;
  return l;
}

template <typename I> __device__ inline int key_of(const I* ids, int64_t i, int V) {
  const int64_t v = (int64_t)ids[i];
  return v >= 0 && v < V ? (int)v : V;
}

template <typename T, typename I>
__global__ __launch_bounds__(256) void k_embed(int64_t n, int V, int D, int lpr, const I* __restrict__ ids,
                                               const T* __restrict__ table, float scale, T* __restrict__ out) {
  constexpr int N = Vec<T>::N;
  const int rpb = 256 / lpr, sub = threadIdx.x % lpr;
  const int64_t i = (int64_t)blockIdx.x * rpb + threadIdx.x / lpr;
  if (i >= n) return;
  const int v = key_of(ids, i, V);
  for (int c = sub * N; c < D; c += lpr * N) {
    float x[N] = {};
    if (v < V) load_cols(table + (int64_t)v * D, c, D, x);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] *= scale;
    store_cols(out + i * D, c, D, x);
  }
}

// Counts of each digit in a workgroup's pairs: counts[digit][block].
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(int64_t n, int V, int shift, int bits, int blocks,
                                                             const I* __restrict__ ids, const int* __restrict__ keys,
                                                             int* __restrict__ counts) {
  __shared__ int h[1 << kMaxBits];
  const int R = 1 << bits;
  for (int d = threadIdx.x; d < R; d += kSortThreads) h[d] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortItems;
  for (int j = threadIdx.x; j < kSortItems && base + j < n; j += kSortThreads) {
    const int key = ids ? key_of(ids, base + j, V) : keys[base + j];
    atomicAdd(&h[(key >> shift) & (R - 1)], 1);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < R; d += kSortThreads) counts[(int64_t)d * blocks + blockIdx.x] = h[d];
}

// Running totals of one digit's counts over the blocks (one wave per digit).
__global__ __launch_bounds__(256) void k_sort_scan(int digits, int blocks, int* __restrict__ counts,
                                                   int* __restrict__ totals) {
  const int d = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (d >= digits) return;
  int* c = counts + (int64_t)d * blocks;
  int run = 0;
  for (int b0 = 0; b0 < blocks; b0 += 64) {
    const int x = b0 + lane < blocks ? c[b0 + lane] : 0;
    int s = x;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int y = __shfl_up(s, o, 64);
      if (lane >= o) s += y;
    }
    if (b0 + lane < blocks) c[b0 + lane] = run + s - x;
    run += __shfl(s, 63, 64);
  }
  if (lane == 0) totals[d] = run;
}

// Moves each pair to its place: digit base + the counts of earlier blocks + its rank among the block's equal digits.
// A wave takes the block's pairs in runs of 64 in order; lanes with equal digits find each other by ballots.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_move(int64_t n, int V, int shift, int bits, int blocks,
                                                            const I* __restrict__ ids, const int* __restrict__ keys,
                                                            const int* __restrict__ pos,
                                                            const int* __restrict__ counts,
                                                            const int* __restrict__ totals, int* __restrict__ keys_out,
                                                            int* __restrict__ pos_out) {
  constexpr int kWaves = kSortThreads / 64, kRuns = kSortItems / kSortThreads;
  __shared__ int base[1 << kMaxBits];
  __shared__ int wc[kWaves][1 << kMaxBits];
  __shared__ int wsum[kWaves];
  const int R = 1 << bits, tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  // digit bases: exclusive totals over the digits
  int carry = 0;
  for (int d0 = 0; d0 < R; d0 += kSortThreads) {
    const int d = d0 + tid, x = d < R ? totals[d] : 0;
    int s = x;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int y = __shfl_up(s, o, 64);
      if (lane >= o) s += y;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) before += wsum[w];
      carry += wsum[w];
    }
    if (d < R) base[d] = before + s - x + counts[(int64_t)d * blocks + blockIdx.x];
    __syncthreads();
  }
  for (int d = tid; d < kWaves * R; d += kSortThreads) wc[d / R][d % R] = 0;
  __syncthreads();
  // each wave: 64 * kRuns consecutive pairs
  const int64_t first = (int64_t)blockIdx.x * kSortItems + (int64_t)wave * 64 * kRuns;
  int key[kRuns], ps[kRuns], rank[kRuns];
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int64_t i = first + r * 64 + lane;
    const bool live = i < n;
    key[r] = live ? (ids ? key_of(ids, i, V) : keys[i]) : 0;
    ps[r] = live ? (ids ? (int)i : pos[i]) : 0;
    const int d = (key[r] >> shift) & (R - 1);
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      same &= ((d >> b) & 1) ? m : ~m;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    int old = 0;
    if (live) old = wc[wave][d];
    rank[r] = old + before;
    if (live && before == 0) wc[wave][d] = old + __popcll(same);
  }
  __syncthreads();
  for (int d = tid; d < R; d += kSortThreads) {
    int s = base[d];
    for (int w = 0; w < kWaves; ++w) {
      const int c = wc[w][d];
      wc[w][d] = s;
      s += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    if (first + r * 64 + lane < n) {
      const int64_t to = (int64_t)wc[wave][(key[r] >> shift) & (R - 1)] + rank[r];
      keys_out[to] = key[r];
      pos_out[to] = ps[r];
    }
  }
}

__global__ __launch_bounds__(256) void k_zero16(uint4* __restrict__ p, int64_t n16, char* __restrict__ tail, int rest) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += step) p[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && (int)threadIdx.x < rest) tail[threadIdx.x] = 0;
}

template <typename T>
__device__ inline void write_row(T* dtable, int v, int c, int D, const float* acc, float scale, bool accumulate) {
  constexpr int N = Vec<T>::N;
  T* row = dtable + (int64_t)v * D;
  float y[N];
#pragma unroll
  for (int j = 0; j < N; ++j) y[j] = acc[j] * scale;
  if (accumulate) {
    float old[N];
    load_cols(row, c, D, old);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] += old[j];
  }
  store_cols(row, c, D, y);
}

// One lane group per chunk of kChunk sorted pairs (and per lpr * N columns: blockIdx.y). An item whose pairs are all
// in the chunk is written; the sum of the first item, where it began earlier, goes to part[chunk][0], that of the
// last, where it began here and goes on, to part[chunk][1].
template <typename T>
__global__ __launch_bounds__(256) void k_embed_grad(int64_t n, int V, int D, int lpr, const int* __restrict__ keys,
                                                    const int* __restrict__ pos, const T* __restrict__ dout,
                                                    float scale, bool accumulate, T* __restrict__ dtable,
                                                    float* __restrict__ part) {
  constexpr int N = Vec<T>::N;
  const int64_t chunk = (int64_t)blockIdx.x * (256 / lpr) + threadIdx.x / lpr;
  const int c = (blockIdx.y * lpr + threadIdx.x % lpr) * N;
  const int64_t e0 = chunk * kChunk;
  if (e0 >= n || c >= D) return;
  const int64_t e1 = e0 + kChunk < n ? e0 + kChunk : n;
  int cur = keys[e0];
  bool began_here = e0 == 0 || keys[e0 - 1] != cur;
  float acc[N] = {};
  for (int64_t e = e0; e < e1; ++e) {
    const int v = keys[e];
    if (v >= V) break;  // the pairs without an item come last
    if (v != cur) {
      if (began_here) write_row(dtable, cur, c, D, acc, scale, accumulate);
      else {
        for (int j = 0; j < N && c + j < D; ++j) part[(chunk * 2 + 0) * D + c + j] = acc[j];
      }
      cur = v;
      began_here = true;
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
    }
    float x[N];
    load_cols(dout + (int64_t)pos[e] * D, c, D, x);
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] += x[j];
  }
  if (cur >= V) return;
  const bool goes_on = e1 < n && keys[e1] == cur;
  if (began_here && !goes_on) {
    write_row(dtable, cur, c, D, acc, scale, accumulate);
  } else {
    float* p = part + (chunk * 2 + (began_here ? 1 : 0)) * D;
    for (int j = 0; j < N && c + j < D; ++j) p[c + j] = acc[j];
  }
}

// Joins the partial sums of the items that span chunks: the chunk where such an item begins adds its own and those
// of the chunks behind it, in order.
template <typename T>
__global__ __launch_bounds__(256) void k_embed_join(int64_t n, int64_t chunks, int V, int D, int lpr,
                                                    const int* __restrict__ keys, float scale, bool accumulate,
                                                    T* __restrict__ dtable, const float* __restrict__ part) {
  constexpr int N = Vec<T>::N;
  const int64_t chunk = (int64_t)blockIdx.x * (256 / lpr) + threadIdx.x / lpr;
  const int c = (blockIdx.y * lpr + threadIdx.x % lpr) * N;
  const int64_t e1 = (chunk + 1) * kChunk;
  if (e1 >= n || c >= D) return;
  const int v = keys[e1 - 1];
  if (v >= V || keys[e1] != v) return;                              // nothing goes on
  const int64_t e0 = chunk * kChunk;
  if (keys[e0] == v && e0 > 0 && keys[e0 - 1] == v) return;         // it began earlier
  float acc[N] = {};
  for (int j = 0; j < N && c + j < D; ++j) acc[j] = part[(chunk * 2 + 1) * D + c + j];
  for (int64_t k = chunk + 1; k < chunks && keys[k * kChunk] == v; ++k)
    for (int j = 0; j < N && c + j < D; ++j) acc[j] += part[(k * 2) * D + c + j];
  write_row(dtable, v, c, D, acc, scale, accumulate);
}

template <typename T, typename I>
hipError_t forward_t(int64_t n, int V, int D, const void* ids, const void* table, float scale, void* out,
                     hipStream_t st) {
  const int lpr = lanes_of(D, Vec<T>::N);
  k_embed<T, I><<<dim3((unsigned)cdiv(n, 256 / lpr)), dim3(256), 0, st>>>(n, V, D, lpr, (const I*)ids,
                                                                         (const T*)table, scale, (T*)out);
  return hipGetLastError();
}

template <typename T, typename I>
hipError_t backward_t(int64_t n, int V, int D, const void* ids, const void* dout, float scale, bool accumulate,
                      void* dtable, char* ws, hipStream_t st) {
  if (!accumulate) {
    const size_t bytes = (size_t)V * D * sizeof(T);
    const int64_t n16 = (int64_t)(bytes / 16);
    const int64_t blocks = cdiv(n16, 256 * 8);
    k_zero16<<<dim3((unsigned)(blocks < 1 ? 1 : (blocks > 8192 ? 8192 : blocks))), dim3(256), 0, st>>>(
        (uint4*)dtable, n16, (char*)dtable + n16 * 16, (int)(bytes % 16));
  }
  if (n == 0) return hipGetLastError();
  const BwdLayout L = bwd_layout(n, V, D);
  const SortPlan p = sort_plan(n, V);
  int* counts = (int*)(ws + L.counts);
  int* totals = (int*)(ws + L.totals);
  const int blocks = (int)p.blocks, digits = 1 << p.bits;
  for (int s = 0; s < p.passes; ++s) {
    const I* id0 = s == 0 ? (const I*)ids : nullptr;
    const int* kin = (const int*)(ws + L.keys[(s + 1) & 1]);
    const int* pin = (const int*)(ws + L.pos[(s + 1) & 1]);
    int* kout = (int*)(ws + L.keys[s & 1]);
    int* pout = (int*)(ws + L.pos[s & 1]);
    k_sort_count<I><<<dim3(blocks), dim3(kSortThreads), 0, st>>>(n, V, s * p.bits, p.bits, blocks, id0, kin, counts);
    k_sort_scan<<<dim3((digits + 3) / 4), dim3(256), 0, st>>>(digits, blocks, counts, totals);
    k_sort_move<I><<<dim3(blocks), dim3(kSortThreads), 0, st>>>(n, V, s * p.bits, p.bits, blocks, id0, kin, pin, counts,
                                                               totals, kout, pout);
  }
  const int* keys = (const int*)(ws + L.keys[(p.passes - 1) & 1]);
  const int* pos = (const int*)(ws + L.pos[(p.passes - 1) & 1]);
  const int lpr = lanes_of(D, Vec<T>::N);
  const dim3 grid((unsigned)cdiv(L.chunks, 256 / lpr), (unsigned)cdiv(D, lpr * Vec<T>::N));
  float* part = (float*)(ws + L.part);
  k_embed_grad<T><<<grid, dim3(256), 0, st>>>(n, V, D, lpr, keys, pos, (const T*)dout, scale, accumulate, (T*)dtable,
                                              part);
  k_embed_join<T><<<grid, dim3(256), 0, st>>>(n, L.chunks, V, D, lpr, keys, scale, accumulate, (T*)dtable, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding_forward(int64_t n, int64_t V, int D, int dtype, int id_bytes, const void* ids,
                                    const void* table, float scale, void* out, hipStream_t st) {
  const int v = (int)V;
  if (dtype == 1)
    return id_bytes == 8 ? forward_t<__bf16, int64_t>(n, v, D, ids, table, scale, out, st)
                         : forward_t<__bf16, int32_t>(n, v, D, ids, table, scale, out, st);
  return id_bytes == 8 ? forward_t<float, int64_t>(n, v, D, ids, table, scale, out, st)
                       : forward_t<float, int32_t>(n, v, D, ids, table, scale, out, st);
}

size_t embedding_backward_bytes(int64_t n, int64_t V, int D, int) { return n > 0 ? bwd_layout(n, V, D).total : 0; }

hipError_t launch_embedding_backward(int64_t n, int64_t V, int D, int dtype, int id_bytes, const void* ids,
                                     const void* dout, float scale, bool accumulate, void* dtable, char* ws,
                                     hipStream_t st) {
  const int v = (int)V;
  if (dtype == 1)
    return id_bytes == 8 ? backward_t<__bf16, int64_t>(n, v, D, ids, dout, scale, accumulate, dtable, ws, st)
                         : backward_t<__bf16, int32_t>(n, v, D, ids, dout, scale, accumulate, dtable, ws, st);
  return id_bytes == 8 ? backward_t<float, int64_t>(n, v, D, ids, dout, scale, accumulate, dtable, ws, st)
                       : backward_t<float, int32_t>(n, v, D, ids, dout, scale, accumulate, dtable, ws, st);
}

}  // namespace cutbce
