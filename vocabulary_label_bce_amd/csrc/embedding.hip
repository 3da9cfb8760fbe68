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

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kSortThreads = 256;
constexpr int kSortItems = 1024;  // pairs of one sorting workgroup
constexpr int kMaxBits = 10;      // most bits of one sorting pass
constexpr int kChunk = 8;         // sorted pairs that one lane group sums
constexpr int kFillBytes = 32768; // what one workgroup clears

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

// Lookup: a group of lanes copies a row, 16 bytes a lane; nothing but memory bounds it. 262,144 rows of 256 bf16 from a
// table of 10 M rows, ids drawn with few hot items: 38 us, 7.0 TB/s read and written (the hot rows come from the
// caches). 32 rows: 1.5 us, an empty kernel 1.4.
template <typename T, typename I>
__global__ __launch_bounds__(256) void k_embed(int64_t n, int V, int D, int lpr, const I* __restrict__ ids,
                                               const T* __restrict__ table, float scale, T* __restrict__ out,
                                               bool past) {
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
    store_cols(out + i * D, c, D, x, past);
  }
}

// The gradient's table is cleared by the sorting kernels, whose own work fills few CUs and is all latency: the
// workgroups behind the sorting ones clear a share of it each. At 876,000 x 128 bf16 (224 MB) and 25,600 ids the six
// launches take 50 us; with the table cleared before them it was 28 us more, and without a table to clear (sums added
// to it) they take 27. At 262,144 x 512 float32 (537 MB) and 12,289 ids they take 94 us, 5.7 TB/s, or 28. The stores
// go past the caches: at 262,144 x 512 float32 (537 MB) the lookup and the row sums around them then still find their
// rows there (13 -> 8 us each).
struct Fill {
  char* p;          // of this launch's share
  int64_t bytes;    // 0: nothing to clear
  int first;        // workgroups from this one on clear
};
__device__ inline bool fill(const Fill& f) {
  if ((int)blockIdx.x < f.first) return false;
  const int64_t at = (int64_t)(blockIdx.x - f.first) * kFillBytes;
#pragma unroll
  for (int i = 0; i < kFillBytes / 16 / kSortThreads; ++i) {
    const int64_t o = at + ((int64_t)i * kSortThreads + threadIdx.x) * 16;
    if (o + 16 <= f.bytes) {
      __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, (u32x4*)(f.p + o));
    } else {
      for (int64_t b = o; b < f.bytes && b < o + 16; ++b) f.p[b] = 0;
    }
  }
  return true;
}
__global__ __launch_bounds__(kSortThreads) void k_fill(Fill f) { fill(f); }

// Counts of each digit in a workgroup's pairs: counts[digit][block]. 10 bits a pass, so that a million items take two:
// the sort is bound by its launches and the latencies in them, not by its bytes. 1,024 pairs a workgroup: 25 workgroups
// at 25,600 positions, and a digit's counts over them are one scan step of a wave.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(Fill f, int64_t n, int V, int shift, int bits, int blocks,
                                                             const I* __restrict__ ids, const int* __restrict__ keys,
                                                             int* __restrict__ counts) {
  if (fill(f)) return;
  constexpr int kPer = kSortItems / kSortThreads;
  __shared__ int h[1 << kMaxBits];
  const int R = 1 << bits;
  const int64_t base = (int64_t)blockIdx.x * kSortItems + threadIdx.x;
  int key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t i = base + j * kSortThreads;
    key[j] = i < n ? (ids ? key_of(ids, i, V) : keys[i]) : -1;
  }
  for (int d = threadIdx.x; d < R; d += kSortThreads) h[d] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (key[j] >= 0) atomicAdd(&h[(key[j] >> shift) & (R - 1)], 1);
  __syncthreads();
  for (int d = threadIdx.x; d < R; d += kSortThreads) counts[(int64_t)d * blocks + blockIdx.x] = h[d];
}

__device__ inline int wave_scan(int x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  return x;
}

// Running totals of one digit's counts over the blocks (one wave per digit).
__global__ __launch_bounds__(kSortThreads) void k_sort_scan(Fill f, int digits, int blocks, int* __restrict__ counts,
                                                            int* __restrict__ totals) {
  if (fill(f)) return;
  const int d = blockIdx.x * (kSortThreads / 64) + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (d >= digits) return;
  int* c = counts + (int64_t)d * blocks;
  int run = 0;
  for (int b0 = 0; b0 < blocks; b0 += 64) {
    const int x = b0 + lane < blocks ? c[b0 + lane] : 0;
    const int s = wave_scan(x, lane);
    if (b0 + lane < blocks) c[b0 + lane] = run + s - x;
    run += __shfl(s, 63, 64);
  }
  if (lane == 0) totals[d] = run;
}

// Moves each pair to its place: digit base + the counts of earlier blocks + its rank among the block's equal digits.
// A wave takes the block's pairs in runs of 64 in order; lanes with equal digits find each other by ballots. Every
// load from memory is issued at the start: the kernel's time is mostly their latency.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_move(Fill f, int64_t n, int V, int shift, int bits, int blocks,
                                                            const I* __restrict__ ids, const int* __restrict__ keys,
                                                            const int* __restrict__ pos,
                                                            const int* __restrict__ counts,
                                                            const int* __restrict__ totals, int* __restrict__ keys_out,
                                                            int* __restrict__ pos_out) {
  if (fill(f)) return;
  constexpr int kWaves = kSortThreads / 64, kRuns = kSortItems / kSortThreads, kMost = 1 << kMaxBits;
  constexpr int kPer = kMost / kSortThreads;  // digits of a thread: kPer consecutive ones
  __shared__ int wc[kWaves][kMost];
  __shared__ int wsum[kWaves];
  const int R = 1 << bits, tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const int64_t first = (int64_t)blockIdx.x * kSortItems + (int64_t)wave * 64 * kRuns;
  int key[kRuns], ps[kRuns], rank[kRuns], tot[kPer], cnt[kPer];
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int64_t i = first + r * 64 + lane;
    const bool live = i < n;
    key[r] = live ? (ids ? key_of(ids, i, V) : keys[i]) : 0;
    ps[r] = live ? (ids ? (int)i : pos[i]) : 0;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int d = tid * kPer + j;
    tot[j] = d < R ? totals[d] : 0;
    cnt[j] = d < R ? counts[(int64_t)d * blocks + blockIdx.x] : 0;
  }
  for (int d = tid; d < kWaves * kMost; d += kSortThreads) ((int*)wc)[d] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const bool live = first + r * 64 + lane < n;
    const int d = (key[r] >> shift) & (R - 1);
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      same &= ((d >> b) & 1) ? m : ~m;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    const int old = live ? wc[wave][d] : 0;
    rank[r] = old + before;
    if (live && before == 0) wc[wave][d] = old + __popcll(same);
  }
  // digit bases: exclusive totals over the digits, kPer consecutive ones a thread
  int sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum += tot[j];
  const int incl = wave_scan(sum, lane);
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int w = 0; w < wave; ++w) base += wsum[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int d = tid * kPer + j;
    int s = base + cnt[j];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = wc[w][d];
      wc[w][d] = s;
      s += c;
    }
    base += tot[j];
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

template <int N> __device__ inline void store_sums(float* row, int c, int D, const float* x) {
#pragma unroll
  for (int j = 0; j < N; j += Vec<float>::N) store_cols(row, c + j, D, x + j);
}

// One lane group per chunk of kChunk sorted pairs (and per lpr * N columns: blockIdx.y). An item whose pairs are all
// in the chunk is written; the sum of the first item, where it began earlier, goes to part[chunk][0], that of the
// last, where it began here and goes on, to part[chunk][1]. The chunk's rows are loaded together before they are
// added: with one row after another the kernel took 39 us at 25,600 x 128 bf16, so 7.1 (6.6 MB read: latency; at 12,289
// x 512 float32, 25 MB, 7.8).
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
  int key[kChunk], at[kChunk];
  const int before = e0 > 0 ? keys[e0 - 1] : -1, after = e0 + kChunk < n ? keys[e0 + kChunk] : V;
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    key[i] = e0 + i < n ? keys[e0 + i] : V;
    at[i] = e0 + i < n ? pos[e0 + i] : 0;
  }
  float x[kChunk][N];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    if (key[i] < V) {
      load_cols(dout + (int64_t)at[i] * D, c, D, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) x[i][j] = 0.f;
    }
  }
  bool began_here = before != key[0];
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = x[0][j];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    if (key[i] >= V) return;  // the pairs without an item come last
    const int next = i + 1 < kChunk ? key[i + 1] : after;
    if (next != key[i]) {
      if (began_here) {
        write_row(dtable, key[i], c, D, acc, scale, accumulate);
      } else {
        store_sums<N>(part + chunk * 2 * D, c, D, acc);
      }
      began_here = true;
    } else if (i + 1 == kChunk) {
      store_sums<N>(part + (chunk * 2 + (began_here ? 1 : 0)) * D, c, D, acc);
    }
    if (i + 1 < kChunk) {
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = (next != key[i] ? 0.f : acc[j]) + x[i + 1][j];
    }
  }
}

// Joins the partial sums of the items that span chunks. A wave looks at one chunk: if an item begins there and goes
// on, it counts the chunks that the item reaches into (64 probes at a time: the keys are sorted). Then the workgroup
// adds the partials of each such item: group g those of the chunks g, g + groups, ... in order, and the groups' sums
// in order of g. 25,600 x 128 bf16: 6.3 us, the chain of probes, partials and sums of the hottest item. An item's
// partials are one workgroup's: 262,144 positions of 1,000 items (1 / rank: the hottest has 3,300 partials) x 512
// float32 take 328 us here, beside 125 for the chunks (537 MB, 4.3 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_embed_join(int64_t n, int64_t chunks, int V, int D, int lpr,
                                                    const int* __restrict__ keys, float scale, bool accumulate,
                                                    T* __restrict__ dtable, const float* __restrict__ part) {
  constexpr int N = Vec<T>::N;
  __shared__ int item[4];
  __shared__ int64_t more[4];
  __shared__ float sums[256][N];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  {
    const int64_t chunk = (int64_t)blockIdx.x * 4 + wave, e0 = chunk * kChunk, e1 = e0 + kChunk;
    int v = V;
    int64_t count = 0;
    if (e1 < n) {
      const int last = keys[e1 - 1], next = keys[e1], head = keys[e0], before = e0 > 0 ? keys[e0 - 1] : -1;
      if (last < V && next == last && !(head == last && before == last)) {
        v = last;
        int64_t lo = chunk + 1, cnt = chunks - lo;  // chunk lo begins with v; the answer is in [lo, lo + cnt)
        while (cnt > 1) {
          const int64_t step = (cnt + 63) / 64, p = lane * step;
          const uint64_t m = __ballot(p < cnt && keys[(lo + p) * kChunk] == v);
          const int64_t k = m ? 63 - __builtin_clzll(m) : 0;
          lo += k * step;
          cnt = cnt - k * step < step ? cnt - k * step : step;
        }
        count = lo - chunk;
      }
    }
    if (lane == 0) item[wave] = v, more[wave] = count;
  }
  __syncthreads();
  const int g = threadIdx.x / lpr, groups = 256 / lpr;
  const int c = (blockIdx.y * lpr + threadIdx.x % lpr) * N;
  for (int w = 0; w < 4; ++w) {
    const int64_t count = more[w];
    if (count == 0) continue;  // the same for the whole workgroup
    const float* p = part + ((int64_t)blockIdx.x * 4 + w) * 2 * D;
    float acc[N] = {};
    if (c < D) {
      // partial 0 is the first chunk's last item, partial k > 0 the first item of the k-th chunk behind it
#pragma unroll 4
      for (int64_t k = g; k <= count; k += groups) {
        float x[N];
        constexpr int M = Vec<float>::N;
        const float* q = p + (k * 2 + (k == 0 ? 1 : 0)) * D;
#pragma unroll
        for (int j = 0; j < N; j += M) load_cols(q, c + j, D, x + j);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += x[j];
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) sums[threadIdx.x][j] = acc[j];
    __syncthreads();
    if (g == 0 && c < D) {
      for (int k = 1; k < groups && k <= count; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += sums[k * lpr + threadIdx.x][j];
      write_row(dtable, item[w], c, D, acc, scale, accumulate);
    }
    __syncthreads();
  }
}

template <typename T, typename I>
hipError_t forward_t(int64_t n, int V, int D, const void* ids, const void* table, float scale, void* out,
                     hipStream_t st) {
  const int lpr = lanes_of(D, Vec<T>::N), rows = 256 / lpr;
  const bool past = goes_past(n * D * (int64_t)sizeof(T));
  for (int64_t i = 0; i < n; i += kMaxGrid * rows) {
    const int64_t m = n - i < kMaxGrid * rows ? n - i : kMaxGrid * rows;
    k_embed<T, I><<<dim3((unsigned)cdiv(m, rows)), dim3(256), 0, st>>>(m, V, D, lpr, (const I*)ids + i, (const T*)table,
                                                                      scale, (T*)out + i * D, past);
  }
  return hipGetLastError();
}

template <typename T, typename I>
hipError_t backward_t(int64_t n, int V, int D, const void* ids, const void* dout, float scale, bool accumulate,
                      void* dtable, char* ws, hipStream_t st) {
  const int64_t bytes = accumulate ? 0 : (int64_t)V * D * (int64_t)sizeof(T);
  if (n == 0) {
    if (bytes) k_fill<<<dim3((unsigned)cdiv(bytes, kFillBytes)), dim3(kSortThreads), 0, st>>>({(char*)dtable, bytes, 0});
    return hipGetLastError();
  }
  const BwdLayout L = bwd_layout(n, V, D);
  const SortPlan p = sort_plan(n, V);
  int* counts = (int*)(ws + L.counts);
  int* totals = (int*)(ws + L.totals);
  const int blocks = (int)p.blocks, digits = 1 << p.bits;
  // A launch's share of the table: a quarter of the pass's to the counting and the scanning each, half to the moving,
  // whose own work takes longest (the sort at 876,000 x 128 bf16 52 -> 49 us against equal shares; 1 : 1 : 3 49).
  const int64_t quarter = cdiv(cdiv(bytes, 4 * p.passes), kFillBytes) * kFillBytes;
  int64_t done = 0;
  int more = 0;  // workgroups that clear
  auto next = [&](int first, int64_t share) {
    const int64_t b = bytes - done < share ? bytes - done : share;
    const Fill f = {(char*)dtable + done, b, first};
    done += b;
    more = (int)cdiv(b, kFillBytes);
    return f;
  };
  for (int s = 0; s < p.passes; ++s) {
    const I* id0 = s == 0 ? (const I*)ids : nullptr;
    const int* kin = (const int*)(ws + L.keys[(s + 1) & 1]);
    const int* pin = (const int*)(ws + L.pos[(s + 1) & 1]);
    int* kout = (int*)(ws + L.keys[s & 1]);
    int* pout = (int*)(ws + L.pos[s & 1]);
    const int scans = (int)cdiv(digits, kSortThreads / 64);
    Fill f = next(blocks, quarter);
    k_sort_count<I><<<dim3(blocks + more), dim3(kSortThreads), 0, st>>>(f, n, V, s * p.bits, p.bits, blocks, id0, kin,
                                                                       counts);
    f = next(scans, quarter);
    k_sort_scan<<<dim3(scans + more), dim3(kSortThreads), 0, st>>>(f, digits, blocks, counts, totals);
    f = next(blocks, 2 * quarter);
    k_sort_move<I><<<dim3(blocks + more), dim3(kSortThreads), 0, st>>>(f, n, V, s * p.bits, p.bits, blocks, id0, kin,
                                                                      pin, counts, totals, kout, pout);
  }
  const int* keys = (const int*)(ws + L.keys[(p.passes - 1) & 1]);
  const int* pos = (const int*)(ws + L.pos[(p.passes - 1) & 1]);
  const int lpr = lanes_of(D, Vec<T>::N);
  const unsigned cols = (unsigned)cdiv(D, lpr * Vec<T>::N);
  float* part = (float*)(ws + L.part);
  k_embed_grad<T><<<dim3((unsigned)cdiv(L.chunks, 256 / lpr), cols), dim3(256), 0, st>>>(
      n, V, D, lpr, keys, pos, (const T*)dout, scale, accumulate, (T*)dtable, part);
  if (L.chunks > 1)
    k_embed_join<T><<<dim3((unsigned)cdiv(L.chunks, 4), cols), dim3(256), 0, st>>>(n, L.chunks, V, D, lpr, keys, scale,
                                                                                   accumulate, (T*)dtable, part);
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
