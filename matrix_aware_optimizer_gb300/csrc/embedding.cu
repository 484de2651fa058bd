// Token embedding: out[t] = scale table[token[t]], and the gradient of the
// table, grad[v] = scale sum_{token[t] = v} dout[t].
//
// Forward: a gather bound by memory; `tpc` threads copy a row, 8 elements
// each, four rows at a time where there are enough tokens, so that a row's
// latency is shared.
//
// Gradient: the tokens are sorted with their positions by a stable radix
// sort (least significant digit first, up to 9 bits a pass), so that equal
// tokens stand together in the order of t. The sorted list is cut into
// pieces of EMB_PIECE entries; a piece sums each of its runs of equal tokens
// in fp32. A run inside one piece goes straight to its row of grad; a run
// that crosses pieces leaves one partial sum per piece, and a last kernel
// adds those in order (very long runs by blocks of EMB_BLOCK pieces first). A
// frequent token's run is thus spread over many SMs, and no sum depends on
// the order in which CTAs run.
//
// Rows without tokens are zero, and writing them is what bounds the call. Up
// to 65536 tokens are sorted by one cluster of eight CTAs that exchange keys
// through distributed shared memory, and the idle SMs clear the first rows of
// the table meanwhile; the other rows without tokens are cleared beside the
// pieces, in the same launch, by CTAs that find the gaps in the sorted list.
// (Clearing everything first and summing afterwards took 108 us instead of
// 80 at 8192 tokens, 64000 x 2048 bf16, both then: scattered reads are slow
// right behind a table of dirty lines in L2.)
//
// Measured, back to back: 62 us there (its bytes at the copy rate: 44) and 138
// at 65521 tokens of 1001 bf16 into 100003 rows of fp32 (78), of which the sort
// takes 31, the pieces about 65 and the runs' partial sums about 20. Past 65536
// tokens, where the sort takes three launches a pass with nothing beside it:
// 131072 tokens, 64000 x 2048 bf16 226 us (118), 1048576 tokens of 512 bf16 into
// 64000 rows of fp32 494 (179).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "blocks.cuh"

namespace prm {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int EMB_TILE = 2048;   // tokens per CTA of a sorting pass
constexpr int EMB_MAX_BITS = 9;  // digit of one pass
constexpr int EMB_MAX_BINS = 1 << EMB_MAX_BITS;
constexpr int EMB_PIECE = 16;
// Partial sums of a long run: by blocks of EMB_BLOCK pieces, EMB_AHEAD under way
// per thread. 65521 tokens, 100003 x 1001: 142 us with blocks of 32, 138 with
// 16, 136 with 8, which doubles what the longest runs add up one by one; 8
// under way took 1 - 3 us more than 4.
constexpr int EMB_BLOCK = 16;
constexpr int EMB_AHEAD = 4;
constexpr int EMB_SPAN_CTAS = 3;  // per SM, of the kernel that adds a run's sums
constexpr int EMB_CLUSTER = 8;
constexpr int EMB_CLUSTER_CHUNK = 8192;  // most keys per CTA of the cluster sort

// Threads that share a row: a power of two, one 8-element vector each per
// step over the columns.
inline int row_threads(int64_t d) {
  int t = 2;
  while (t < EMB_THREADS && static_cast<int64_t>(t) * 8 < d) t *= 2;
  return t;
}

template <bool VEC>
__device__ __forceinline__ int64_t col_index(int64_t c0, int e, int tid, int tpc) {
  return VEC ? c0 + tid * 8 + e : c0 + e * tpc + tid;
}

__device__ __forceinline__ int64_t load_token(const void* token, int bytes, int64_t t) {
  return bytes == 8 ? static_cast<const int64_t*>(token)[t]
                    : static_cast<int64_t>(static_cast<const int32_t*>(token)[t]);
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int64_t c0, int64_t d, int tid, int tpc, float (&o)[8]) {
  if constexpr (VEC) {
    const int64_t c = col_index<true>(c0, 0, tid, tpc);
    Raw8<T> r;
    if (c < d) r.load_cached(row + c);
    else r.zero();
    r.get(o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = col_index<false>(c0, e, tid, tpc);
      o[e] = c < d ? to_f32(row[c]) : 0.f;
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int64_t c0, int64_t d, int tid, int tpc, const float (&o)[8]) {
  if constexpr (VEC) {
    const int64_t c = col_index<true>(c0, 0, tid, tpc);
    if (c < d) {
      Raw8<T> r;
      r.set(o);
      r.store(row + c);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = col_index<false>(c0, e, tid, tpc);
      if (c < d) row[c] = from_f32<T>(o[e]);
    }
  }
}

template <typename TT, typename OT, bool VEC, int ROWS>
__global__ void __launch_bounds__(EMB_THREADS)
    embedding_forward_kernel(const void* __restrict__ token, int token_bytes, const TT* __restrict__ table,
                             OT* __restrict__ out, int64_t tokens, int64_t vocab, int64_t d, float scale, int tpc) {
  const int tid = threadIdx.x & (tpc - 1);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / tpc) + threadIdx.x / tpc) * ROWS;
  pdl_wait();
  pdl_launch_dependents();
  const TT* row[ROWS];
  int64_t width[ROWS];  // d, or 0 for padding: its row is written as zeros
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int64_t v = t0 + k < tokens ? load_token(token, token_bytes, t0 + k) : -1;
    const bool valid = v >= 0 && v < vocab;
    row[k] = table + (valid ? v : 0) * d;
    width[k] = valid ? d : 0;
  }
  for (int64_t c0 = 0; c0 < d; c0 += 8 * tpc) {
    float o[ROWS][8];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) load8<TT, VEC>(row[k], c0, width[k], tid, tpc, o[k]);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (t0 + k >= tokens) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[k][e] *= scale;
      store8<OT, VEC>(out + (t0 + k) * d, c0, d, tid, tpc, o[k]);
    }
  }
}

// ------------------------------------------------------------------ sorting
struct SortPass {
  const void* token;       // first pass: the tokens themselves (key = token, or vocab for padding)
  int token_bytes;         // 0: keys and positions of the pass before
  const uint32_t* keys_in;
  const uint32_t* pos_in;
  uint32_t* keys_out;
  uint32_t* pos_out;
  uint32_t* hist;          // [bins][tiles], then its exclusive scan
  uint32_t count, vocab;
  int shift, bits;
  uint32_t tiles;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& s, uint32_t i) {
  if (s.token_bytes == 0) return s.keys_in[i];
  const int64_t v = load_token(s.token, s.token_bytes, i);
  return v >= 0 && v < s.vocab ? static_cast<uint32_t>(v) : s.vocab;
}

__global__ void __launch_bounds__(EMB_THREADS) sort_hist_kernel(const SortPass s) {
  __shared__ uint32_t bins[EMB_MAX_BINS];
  const uint32_t nbins = 1u << s.bits;
  for (uint32_t b = threadIdx.x; b < nbins; b += EMB_THREADS) bins[b] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t base = blockIdx.x * EMB_TILE;
#pragma unroll
  for (int k = 0; k < EMB_TILE / EMB_THREADS; ++k) {
    const uint32_t i = base + k * EMB_THREADS + threadIdx.x;
    if (i < s.count) atomicAdd(&bins[(sort_key(s, i) >> s.shift) & (nbins - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < nbins; b += EMB_THREADS) s.hist[b * s.tiles + blockIdx.x] = bins[b];
}

// Exclusive scan of the histogram in place, by one CTA.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const SortPass s) {
  __shared__ uint32_t warp_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t n = (1u << s.bits) * s.tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t carry = 0;
  for (uint32_t base = 0; base < n; base += 4096) {
    const uint32_t i = base + threadIdx.x * 4;
    uint32_t v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < n ? s.hist[i + k] : 0;
      sum += v[k];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const uint32_t t = warp_sum[w];
      before += w < warp ? t : 0;
      total += t;
    }
    uint32_t at = carry + before + inc - sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < n) s.hist[i + k] = at;
      at += v[k];
    }
    carry += total;
    __syncthreads();
  }
}

// Moves each key to its place: the tile's offset of its digit, plus the
// number of equal digits before it in the tile. A warp takes 256 consecutive
// keys in eight steps; equal digits of a step find each other by a warp
// match, earlier steps are counted in the warp's own bins.
__global__ void __launch_bounds__(EMB_THREADS) sort_scatter_kernel(const SortPass s) {
  constexpr int WARPS = EMB_THREADS / 32;
  constexpr int STEPS = EMB_TILE / EMB_THREADS;
  __shared__ uint32_t bins[WARPS][EMB_MAX_BINS];
  const uint32_t nbins = 1u << s.bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (uint32_t b = threadIdx.x; b < WARPS * EMB_MAX_BINS; b += EMB_THREADS) bins[0][b] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t base = blockIdx.x * EMB_TILE + warp * (EMB_TILE / WARPS);
  uint32_t key[STEPS], pos[STEPS], rank[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const uint32_t i = base + k * 32 + lane;
    key[k] = i < s.count ? sort_key(s, i) : 0;
    pos[k] = i < s.count && s.token_bytes == 0 ? s.pos_in[i] : i;
  }
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const bool in = base + k * 32 + lane < s.count;
    const uint32_t digit = in ? (key[k] >> s.shift) & (nbins - 1) : EMB_MAX_BINS;
    const uint32_t peers = __match_any_sync(0xffffffffu, digit);
    const uint32_t before = in ? bins[warp][digit] : 0;
    rank[k] = before + __popc(peers & ((1u << lane) - 1));
    __syncwarp();
    if (in && (peers >> lane) == 1u) bins[warp][digit] = rank[k] + 1;  // the last of the peers
    __syncwarp();
  }
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < nbins; b += EMB_THREADS) {
    uint32_t at = s.hist[b * s.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const uint32_t n = bins[w][b];
      bins[w][b] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    if (base + k * 32 + lane < s.count) {
      const uint32_t to = bins[warp][(key[k] >> s.shift) & (nbins - 1)] + rank[k];
      s.keys_out[to] = key[k];
      s.pos_out[to] = pos[k];
    }
  }
}

// The CTA clears `bytes` bytes at p (any alignment), as part `part` of `parts`.
__device__ __forceinline__ void clear_bytes(uint8_t* p, int64_t bytes, int64_t part, int64_t parts) {
  const int64_t head = min(bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15));
  const int64_t body = (bytes - head) / 16;
  const int64_t at = part * EMB_THREADS + threadIdx.x;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = at; i < body; i += parts * EMB_THREADS) __stcs(q + i, make_uint4(0, 0, 0, 0));
  const int64_t tail = head + body * 16;
  if (at < head) p[at] = 0;
  if (at < bytes - tail) p[tail + at] = 0;
}

// Clears the table's first `bytes` bytes. Its successor, the sort, may start
// at once: it does not touch the table.
__global__ void __launch_bounds__(EMB_THREADS) clear_kernel(uint8_t* p, int64_t bytes) {
  pdl_wait();
  pdl_launch_dependents();
  clear_bytes(p, bytes, blockIdx.x, gridDim.x);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// The two halves of a cluster barrier that orders no memory: all CTAs of the
// cluster have started.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

struct ClusterSort {
  const void* token;
  int token_bytes;
  uint32_t count, vocab;
  uint32_t chunk;      // keys per CTA, a multiple of 1024
  int passes, bits;
  int beside;          // runs beside the clearing kernel: waits for it last
  uint32_t* keys;
  uint32_t* pos;
};

// The whole sort by one cluster. A CTA holds `chunk` consecutive (key,
// position) pairs in shared memory. Per pass it ranks its keys (a warp takes
// consecutive keys, 32 a step; equal digits of a step find each other by a
// warp match, earlier steps are counted in the warp's bins), the CTAs share
// their digit counts, and every pair goes to its place in the CTA that holds
// it next.
__global__ void __maxnreg__(48) cluster_sort_kernel(const ClusterSort s) {
  constexpr int WARPS = 32;
  constexpr int MOST = EMB_CLUSTER_CHUNK / 1024;
  extern __shared__ __align__(16) uint32_t sort_smem[];
  uint2* pairs[2] = {reinterpret_cast<uint2*>(sort_smem), reinterpret_cast<uint2*>(sort_smem) + s.chunk};
  uint32_t* counts = sort_smem + 4 * s.chunk;                    // [cluster][bins]: digit counts of every CTA
  uint32_t* base = counts + EMB_CLUSTER * EMB_MAX_BINS;          // [bins]: where this CTA's keys of a digit go
  uint16_t* bins = reinterpret_cast<uint16_t*>(base + EMB_MAX_BINS);  // [warp][bins]
  __shared__ uint32_t warp_sum[WARPS];
  const uint32_t rank_cta = cluster_ctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // this CTA has started; met below, behind the loads of the tokens
  const uint32_t nbins = 1u << s.bits;
  const int steps = static_cast<int>(s.chunk / 1024);
  const uint32_t first = rank_cta * s.chunk;
  const uint32_t mine = first < s.count ? min(s.chunk, s.count - first) : 0;
  if (!s.beside) {
    pdl_wait();
    pdl_launch_dependents();
  }
  uint32_t key[MOST], pos[MOST], rank[MOST];
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    const uint32_t i = (warp * steps + k) * 32 + lane;
    if (k < steps && i < mine) {
      const int64_t v = load_token(s.token, s.token_bytes, first + i);
      key[k] = v >= 0 && v < s.vocab ? static_cast<uint32_t>(v) : s.vocab;
      pos[k] = first + i;
    }
  }
  cluster_wait();  // all eight have: their shared memory may be written
  for (int pass = 0; pass < s.passes; ++pass) {
    const int shift = pass * s.bits;
    for (uint32_t b = threadIdx.x; b < WARPS * EMB_MAX_BINS / 2; b += 1024) reinterpret_cast<uint32_t*>(bins)[b] = 0;
    __syncthreads();
    uint16_t* own = bins + warp * EMB_MAX_BINS;
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      if (k >= steps) break;
      const bool in = (warp * steps + k) * 32 + lane < mine;
      const uint32_t digit = in ? (key[k] >> shift) & (nbins - 1) : EMB_MAX_BINS;
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      rank[k] = (in ? own[digit] : 0) + __popc(peers & ((1u << lane) - 1));
      __syncwarp();
      if (in && (peers >> lane) == 1u) own[digit] = static_cast<uint16_t>(rank[k] + 1);  // the last of the peers
      __syncwarp();
    }
    __syncthreads();
    // offsets of the warps within a digit, and the CTA's count for everyone
    if (threadIdx.x < nbins) {
      uint32_t at = 0;
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) {
        const uint32_t n = bins[w * EMB_MAX_BINS + threadIdx.x];
        bins[w * EMB_MAX_BINS + threadIdx.x] = static_cast<uint16_t>(at);
        at += n;
      }
      const uint32_t slot = smem_u32(counts + rank_cta * EMB_MAX_BINS + threadIdx.x);
#pragma unroll
      for (uint32_t c = 0; c < EMB_CLUSTER; ++c) st_cluster(mapa_shared(slot, c), at);
    }
    cluster_sync_all();
    // exclusive scan of the digits' totals, plus the CTAs before this one
    uint32_t total = 0, before = 0;
    if (threadIdx.x < nbins) {
#pragma unroll
      for (uint32_t c = 0; c < EMB_CLUSTER; ++c) {
        const uint32_t n = counts[c * EMB_MAX_BINS + threadIdx.x];
        before += c < rank_cta ? n : 0;
        total += n;
      }
    }
    uint32_t inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (threadIdx.x < nbins) {
      uint32_t at = before + inc - total;
      for (int w = 0; w < warp; ++w) at += warp_sum[w];
      base[threadIdx.x] = at;
    }
    __syncthreads();
    const uint32_t dst = smem_u32(pairs[pass & 1]);
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      if (k >= steps || (warp * steps + k) * 32 + lane >= mine) break;
      const uint32_t digit = (key[k] >> shift) & (nbins - 1);
      const uint32_t to = base[digit] + own[digit] + rank[k];
      const uint32_t cta = to / s.chunk;
      st_cluster2(mapa_shared(dst + (to - cta * s.chunk) * 8, cta), key[k], pos[k]);
    }
    cluster_sync_all();
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const uint32_t i = (warp * steps + k) * 32 + lane;
      if (k < steps && i < mine) {
        const uint2 p = pairs[pass & 1][i];
        key[k] = p.x;
        pos[k] = p.y;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    const uint32_t i = (warp * steps + k) * 32 + lane;
    if (k < steps && i < mine) {
      s.keys[first + i] = key[k];
      s.pos[first + i] = pos[k];
    }
  }
  if (s.beside) {
    // kernels behind this one also build on the cleared table
    pdl_wait();
    pdl_launch_dependents();
  }
}

// ------------------------------------------------------------------ summing
struct EmbSum {
  const uint32_t* keys;  // sorted; padding (key == vocab) last
  const uint32_t* pos;
  uint32_t count, vocab;
  uint32_t pieces;
  int64_t d;
  float scale;
  int accumulate;
  int tpc;
  uint32_t clear_from;   // first row that the pieces' CTAs look after
  uint32_t clear_ctas;   // 0 when accumulating
  int64_t rows;          // of dout
  uint32_t pitch;        // bytes between rows in shared memory
  int* err;
  // Partial sums, rows of `partial` floats: a thread's 8 columns lie together
  // at (slab tpc + tid) 8, whatever columns they are.
  int64_t partial;
  float* head;  // [piece]: sum of the run that entered from the piece before
  float* tail;  // [piece]: sum of the run that starts here and goes on
  float* block; // [block of pieces]: sum of the heads of a block that one run covers, or NULL
};

__device__ __forceinline__ void load_partial(const float* row, int64_t c0, int tid, float (&o)[8]) {
  const float4* p = reinterpret_cast<const float4*>(row + c0 + tid * 8);
  const float4 a = __ldcg(p), b = __ldcg(p + 1);
  o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}
__device__ __forceinline__ void store_partial(float* row, int64_t c0, int tid, const float (&v)[8]) {
  float4* p = reinterpret_cast<float4*>(row + c0 + tid * 8);
  p[0] = make_float4(v[0], v[1], v[2], v[3]);
  p[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename GT, bool VEC>
__device__ __forceinline__ void finish_row(const EmbSum& s, GT* grad, uint32_t v, int64_t c0, int tid,
                                           float (&acc)[8]) {
  GT* row = grad + static_cast<int64_t>(v) * s.d;
  float old[8];
  if (s.accumulate) load8<GT, VEC>(row, c0, s.d, tid, s.tpc, old);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = s.accumulate ? fmaf(acc[e], s.scale, old[e]) : acc[e] * s.scale;
  store8<GT, VEC>(row, c0, s.d, tid, s.tpc, acc);
}

// First index whose key is at least v, among `count` sorted keys: a warp
// probes 32 places at once, so that a long list takes three or four loads one
// after the other. All lanes of the warp call and get it.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t count, uint32_t v) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0, n = count;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const uint32_t step = n / 32 + 1;
    const uint32_t at = lo + lane * step + step - 1;  // the last place of this lane's part
    const bool below = at < lo + n && keys[at] < v;
    const uint32_t parts = __popc(__ballot_sync(0xffffffffu, below));  // parts that lie below v as a whole
    const uint32_t skipped = min(parts * step, n);
    lo += skipped;
    n = min(step - 1, n - skipped);
  }
  return lo;
}

// CTA `part` of the clearing CTAs: zeroes the rows of its share of
// [clear_from, vocab) that the sorted list does not hold.
template <typename GT>
__device__ __forceinline__ void clear_gaps(const EmbSum& s, GT* grad, uint32_t part) {
  const uint64_t rows = s.vocab - s.clear_from;
  const uint32_t v0 = s.clear_from + static_cast<uint32_t>(rows * part / s.clear_ctas);
  const uint32_t v1 = s.clear_from + static_cast<uint32_t>(rows * (part + 1) / s.clear_ctas);
  const int64_t row_bytes = s.d * static_cast<int64_t>(sizeof(GT));
  uint8_t* const base = reinterpret_cast<uint8_t*>(grad);
  const int lane = threadIdx.x & 31;
  uint32_t i = lower_bound(s.keys, s.count, v0);
  // Every warp reads 32 keys of the list at a time; the CTA clears the gaps in
  // front of them. A run that fills all 32 is left by a search: stepping
  // through a token with thousands of entries took 50 us more.
  for (uint32_t from = v0; from < v1;) {
    const uint32_t key = i + lane < s.count ? min(s.keys[i + lane], v1) : v1;
    const uint32_t up = __shfl_up_sync(0xffffffffu, key, 1);
    const uint32_t prev = lane == 0 ? from - 1 : up;
    for (uint32_t gaps = __ballot_sync(0xffffffffu, key - prev > 1u); gaps != 0; gaps &= gaps - 1) {
      const int k = __ffs(gaps) - 1;
      const uint32_t to = __shfl_sync(0xffffffffu, key, k), at = __shfl_sync(0xffffffffu, prev, k) + 1;
      clear_bytes(base + at * row_bytes, (to - at) * row_bytes, 0, 1);
    }
    const uint32_t first = __shfl_sync(0xffffffffu, key, 0), last = __shfl_sync(0xffffffffu, key, 31);
    from = last + 1;  // (a last of v1 ends the loop)
    i = first == last && from < v1 ? lower_bound(s.keys, s.count, from) : i + 32;
  }
}

// A CTA first asks for all rows of its pieces (bulk copies into shared
// memory), then clears its share of the rows without tokens while they
// arrive, then sums. Blocks behind the last piece only clear.
// ACCESS: VEC rows are read 8 elements a thread, ELEM rows (d % 8 != 0)
// strided by the row's threads; DIRECT (dout off 16 bytes) reads memory.
template <typename DT, typename GT, int ACCESS>
__global__ void __launch_bounds__(EMB_THREADS) piece_kernel(const EmbSum s, const DT* __restrict__ dout, GT* grad) {
  constexpr bool OUT_VEC = ACCESS == VEC;
  extern __shared__ __align__(128) uint8_t rows_smem[];  // [group][entry][pitch]
  __shared__ uint32_t entry_key[EMB_THREADS / 2 * EMB_PIECE];  // [group][entry]
  __shared__ uint8_t entry_off[ACCESS == ELEM ? EMB_THREADS / 2 * EMB_PIECE : 1];  // its row's offset from 16 bytes
  __shared__ uint64_t bar;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x & (s.tpc - 1);
  const int group = threadIdx.x / s.tpc, groups = EMB_THREADS / s.tpc;
  const int64_t slab = 8 * s.tpc;
  const int64_t c0 = blockIdx.y * slab;
  const uint32_t width = static_cast<uint32_t>(min(slab, s.d - c0));
  if constexpr (ACCESS != DIRECT) {
    if (threadIdx.x == 0) {
      mbar_init(&bar, EMB_THREADS);
      abort_flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int64_t piece0 = static_cast<int64_t>(blockIdx.x) * groups;
  const bool sums = piece0 < s.pieces;
  const DT* const dout_end = dout + s.rows * s.d;
  if (ACCESS != DIRECT && sums) {
    uint32_t bytes = 0;
    for (int pass = 0; pass < 2; ++pass) {
      for (int idx = threadIdx.x; idx < groups * EMB_PIECE; idx += EMB_THREADS) {
        // (entries past the list's end: padding, so that their pieces end there)
        const int64_t entry = piece0 * EMB_PIECE + idx;
        const uint32_t key = entry < s.count ? s.keys[entry] : s.vocab;
        const uint32_t pos = entry < s.count ? s.pos[entry] : 0;
        if (pass == 0) entry_key[idx] = key;
        if (key >= s.vocab) continue;
        const DT* src = dout + static_cast<int64_t>(pos) * s.d + c0;
        if (ACCESS == ELEM && pass == 0) entry_off[idx] = static_cast<uint8_t>(ring_offset(src));
        uint8_t* dst = rows_smem + static_cast<size_t>(idx) * s.pitch;
        const uint32_t n = ACCESS == VEC ? width * static_cast<uint32_t>(sizeof(DT)) : ring_bytes(src, width, dout_end);
        if (pass == 0) {
          bytes += n;
          if (ACCESS == ELEM) ring_tail(dst, src, width, dout_end);
        } else {
          ring_load(dst, src, n, &bar);
        }
      }
      if (pass == 0) mbar_arrive_expect_tx(&bar, bytes);
    }
  }
  const int64_t piece = piece0 + group;
  const bool mine = piece < s.pieces;
  const uint32_t i0 = mine ? static_cast<uint32_t>(piece) * EMB_PIECE : 0;
  const uint32_t n = min(s.count - i0, static_cast<uint32_t>(EMB_PIECE));
  const uint32_t before = mine && i0 > 0 ? s.keys[i0 - 1] : 0xffffffffu;
  const uint32_t after = mine && i0 + n < s.count ? s.keys[i0 + n] : 0xffffffffu;
  if (blockIdx.x < s.clear_ctas && blockIdx.y == 0) clear_gaps(s, grad, blockIdx.x);
  if (!sums) return;
  if constexpr (ACCESS != DIRECT) {
    if (!wait_bounded(&bar, 0, &abort_flag, s.err, 2000000000ull)) {
      wait_drain(&bar, 0, 50000000ull);  // let the copies in flight land before the CTA exits
      return;
    }
  }
  if (!mine) return;
  float acc[8];
  uint32_t run = 0xffffffffu;  // key of the run at work
  bool entered = false;        // it entered from the piece before
#pragma unroll 4
  for (uint32_t j = 0; j < n; ++j) {
    uint32_t key;
    if constexpr (ACCESS == DIRECT) key = s.keys[i0 + j];
    else key = entry_key[group * EMB_PIECE + j];
    if (key >= s.vocab) break;  // padding is sorted to the end
    float x[8];
    if constexpr (ACCESS == DIRECT) {
      load8<DT, false>(dout + static_cast<int64_t>(s.pos[i0 + j]) * s.d, c0, s.d, tid, s.tpc, x);
    } else {
      const uint8_t* at = rows_smem + static_cast<size_t>(group * EMB_PIECE + j) * s.pitch;
      if constexpr (ACCESS == VEC) {
        const bool in = tid * 8 < width;
        const DT* p = reinterpret_cast<const DT*>(at) + (in ? tid * 8 : 0);
        if constexpr (sizeof(DT) == 4) {
          const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
          x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
          Raw8<DT> raw;
          raw.a = *reinterpret_cast<const uint4*>(p);
          raw.get(x);
        }
      } else {
        const DT* p = reinterpret_cast<const DT*>(at + entry_off[group * EMB_PIECE + j]) + tid;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e * s.tpc + tid < width ? to_f32(p[e * s.tpc]) : 0.f;
      }
    }
    if (key != run) {
      if (run != 0xffffffffu) {
        if (entered) store_partial(s.head + piece * s.partial, c0, tid, acc);
        else finish_row<GT, OUT_VEC>(s, grad, run, c0, tid, acc);
      }
      entered = j == 0 && key == before;
      run = key;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = x[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[e];
    }
  }
  if (run == 0xffffffffu) return;
  if (entered) store_partial(s.head + piece * s.partial, c0, tid, acc);
  else if (run == after) store_partial(s.tail + piece * s.partial, c0, tid, acc);
  else finish_row<GT, OUT_VEC>(s, grad, run, c0, tid, acc);
}

// Key of the first entry of a piece, or no key at all behind the last piece.
__device__ __forceinline__ uint32_t piece_key(const EmbSum& s, int64_t piece) {
  const uint32_t key = s.keys[min(piece, static_cast<int64_t>(s.pieces) - 1) * EMB_PIECE];
  return piece < s.pieces ? key : 0xffffffffu;
}

// Adds the sums rows[q], rows[q + 1], ... up to `end`, while the run at work
// goes through them: `more(q)`, asked of places that may lie behind the end.
// EMB_AHEAD are loaded at a time, and whether the next ones belong to the run
// is read beside them: one L2 latency for each EMB_AHEAD. Returns the first
// place that the run does not reach.
template <typename More>
__device__ __forceinline__ int64_t add_sums(const float* rows, int64_t partial, int64_t q, int64_t end, int64_t c0,
                                            int tid, float (&acc)[8], More&& more) {
  auto ask = [&](int64_t from) {  // bit k: place from + k belongs to the run
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < EMB_AHEAD; ++k) m |= static_cast<uint32_t>(more(from + k) & (from + k < end)) << k;
    return m;
  };
  constexpr uint32_t ALL = (1u << EMB_AHEAD) - 1;
  for (uint32_t in = ask(q); in != 0;) {
    float x[EMB_AHEAD][8];
#pragma unroll
    for (int k = 0; k < EMB_AHEAD; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
      if (in >> k & 1) load_partial(rows + (q + k) * partial, c0, tid, x[k]);
    }
    const uint32_t next = in == ALL ? ask(q + EMB_AHEAD) : 0;
#pragma unroll
    for (int k = 0; k < EMB_AHEAD; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[k][e];
    q += __popc(in);
    in = next;
  }
  return q;
}

// Whether the run of key v, which enters block b of EMB_BLOCK pieces, goes on
// behind it (and so covers it, as equal keys stand together).
__device__ __forceinline__ bool covers_block(const EmbSum& s, uint32_t v, int64_t block) {
  return piece_key(s, (block + 1) * EMB_BLOCK) == v;
}

// For very long runs: the sum of the heads of each block of pieces that a run
// covers whole.
__global__ void __launch_bounds__(EMB_THREADS) block_kernel(const EmbSum s) {
  const int tid = threadIdx.x & (s.tpc - 1);
  const int64_t block = static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / s.tpc) + threadIdx.x / s.tpc;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 8 * s.tpc;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t q = block * EMB_BLOCK;
  if (q == 0 || q + EMB_BLOCK >= s.pieces) return;
  const uint32_t v = piece_key(s, q), prior = s.keys[q * EMB_PIECE - 1];
  const bool covered = covers_block(s, v, block);
  if (v >= s.vocab || prior != v || !covered) return;
  float acc[8] = {};
  add_sums(s.head, s.partial, q, q + EMB_BLOCK, c0, tid, acc, [](int64_t) { return true; });
  store_partial(s.block + block * s.partial, c0, tid, acc);
}

// Adds up the run that starts in `piece` and goes on into the next ones.
template <typename GT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS, EMB_SPAN_CTAS) span_kernel(const EmbSum s, GT* grad) {
  const int tid = threadIdx.x & (s.tpc - 1);
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / s.tpc) + threadIdx.x / s.tpc;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 8 * s.tpc;
  pdl_wait();
  pdl_launch_dependents();
  if (piece + 1 >= s.pieces) return;
  const uint32_t i1 = static_cast<uint32_t>(piece + 1) * EMB_PIECE;
  const uint32_t i0 = i1 - EMB_PIECE;
  const uint32_t v = s.keys[i1 - 1], next = s.keys[i1], own = s.keys[i0], prior = s.keys[i0 > 0 ? i0 - 1 : 0];
  if (v >= s.vocab || next != v) return;
  if (own == v && i0 > 0 && prior == v) return;  // the run entered from before: an earlier piece's
  float acc[8];
  load_partial(s.tail + piece * s.partial, c0, tid, acc);
  auto heads = [&](int64_t q, int64_t end) {
    return add_sums(s.head, s.partial, q, end, c0, tid, acc, [&](int64_t p) { return piece_key(s, p) == v; });
  };
  int64_t q = piece + 1;
  if (s.block != nullptr) {
    const int64_t whole = min(static_cast<int64_t>(s.pieces), (q + EMB_BLOCK - 1) / EMB_BLOCK * EMB_BLOCK);
    q = heads(q, whole);
    if (q == whole && q < s.pieces)
      q = EMB_BLOCK * add_sums(s.block, s.partial, q / EMB_BLOCK, s.pieces / EMB_BLOCK, c0, tid, acc,
                               [&](int64_t b) { return covers_block(s, v, b); });
    else
      q = s.pieces;
  }
  heads(q, s.pieces);
  finish_row<GT, VEC>(s, grad, v, c0, tid, acc);
}

// ------------------------------------------------------------------- layout
// Most pieces that a run is added up over piece by piece.
constexpr uint32_t EMB_FLAT_PIECES = 1024;

struct EmbPlan {
  int passes, bits;
  bool cluster;         // one cluster sorts
  uint32_t tiles, pieces, blocks;
  int64_t partial;      // floats per row of partial sums
  size_t keys[2], pos[2], hist, head, tail, block, bytes;
};

EmbPlan plan(int64_t tokens, int64_t vocab, int64_t d) {
  EmbPlan p{};
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;  // keys 0 .. vocab
  p.passes = (bits + EMB_MAX_BITS - 1) / EMB_MAX_BITS;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.cluster = tokens <= EMB_CLUSTER * EMB_CLUSTER_CHUNK;
  p.tiles = static_cast<uint32_t>((tokens + EMB_TILE - 1) / EMB_TILE);
  p.pieces = static_cast<uint32_t>((tokens + EMB_PIECE - 1) / EMB_PIECE);
  p.blocks = p.pieces > EMB_FLAT_PIECES ? (p.pieces + EMB_BLOCK - 1) / EMB_BLOCK : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  const size_t entries = static_cast<size_t>(p.pieces) * EMB_PIECE;  // whole pieces: read four entries at a time
  for (int k = 0; k < (p.cluster ? 1 : 2); ++k) {
    p.keys[k] = take(entries * 4);
    p.pos[k] = take(entries * 4);
  }
  p.hist = p.cluster ? at : take((size_t(1) << p.bits) * p.tiles * 4);
  const int64_t slab = 8 * row_threads(d);
  p.partial = (d + slab - 1) / slab * slab;
  p.head = take(static_cast<size_t>(p.pieces) * p.partial * 4);
  p.tail = take(static_cast<size_t>(p.pieces) * p.partial * 4);
  p.block = take(static_cast<size_t>(p.blocks) * p.partial * 4);
  p.bytes = at;
  return p;
}

cudaError_t launch_cluster_sort(const ClusterSort& s, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(s.chunk) * 16 +
                      (EMB_CLUSTER * EMB_MAX_BINS + EMB_MAX_BINS) * sizeof(uint32_t) + 32 * EMB_MAX_BINS * sizeof(uint16_t);
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev].load(std::memory_order_relaxed)) {
    // An SM's split between L1 and shared memory is fixed while CTAs run on it: the clearing kernel asks for the
    // sort's, or the sort would wait for it to drain.
    cudaError_t e = cudaFuncSetAttribute(cluster_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(cluster_sort_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(clear_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(EMB_CLUSTER);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = EMB_CLUSTER;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cluster_sort_kernel, s);
}

// Most dynamic shared memory of a piece kernel: 256 / tpc groups of EMB_PIECE
// rows of 8 tpc fp32 elements and 32 bytes for their ends, with tpc >= 2.
constexpr int EMB_PIECE_SMEM = EMB_THREADS / 2 * EMB_PIECE * (2 * 8 * 4 + 32);

// Allows a piece kernel that once per device. The limit belongs to the kernel,
// not to a launch: set to what each call needs, it could fall below another
// thread's between that one's setting and its launch.
template <typename DT, typename GT, int ACCESS>
cudaError_t piece_setup() {
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(piece_kernel<DT, GT, ACCESS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             EMB_PIECE_SMEM);
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename F>
bool one_type(int dtype, F&& f) {
  if (dtype == PRM_FP32) return f(float{}), true;
  if (dtype == PRM_BF16) return f(__nv_bfloat16{}), true;
  if (dtype == PRM_FP16) return f(__half{}), true;
  return false;
}

int check_sizes(int64_t tokens, int64_t vocab, int64_t d) {
  if (tokens < 0 || vocab < 1 || d < 1) return PRM_ERR_INVALID_ARG;
  if (tokens >= (int64_t(1) << 31) - (1 << 16) || vocab >= (int64_t(1) << 31) || d > (int64_t(1) << 24))
    return PRM_ERR_UNSUPPORTED;
  return PRM_OK;
}

}  // namespace
}  // namespace prm

extern "C" int prm_embedding_forward(const void* token, int token_bytes, const void* table, int table_dtype, void* out,
                                     int out_dtype, int64_t tokens, int64_t vocab, int64_t d, float scale,
                                     void* stream) {
  using namespace prm;
  if ((token_bytes != 4 && token_bytes != 8) || !is_dtype(table_dtype) || !is_dtype(out_dtype) ||
      !std::isfinite(scale))
    return PRM_ERR_INVALID_ARG;
  const int rc = check_sizes(tokens, vocab, d);
  if (rc != PRM_OK || tokens == 0) return rc;
  if (token == nullptr || table == nullptr || out == nullptr) return PRM_ERR_INVALID_ARG;
  const bool vec = d % 8 == 0 && aligned_to(table, 16) && aligned_to(out, 16);
  const int tpc = row_threads(d);
  const int64_t per = EMB_THREADS / tpc;
  // four rows per thread once that leaves every SM a few CTAs
  const int rows = tokens >= 4 * per * 152 * 4 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((tokens + per * rows - 1) / (per * rows)));
  cudaError_t e = cudaErrorInvalidValue;
  one_type(table_dtype, [&](auto tt) {
    one_type(out_dtype, [&](auto ot) {
      using TT = decltype(tt);
      using OT = decltype(ot);
      const cudaStream_t st = static_cast<cudaStream_t>(stream);
      auto go = [&](auto kernel) {
        e = launch_dependent(kernel, grid, dim3(EMB_THREADS), 0, st, token, token_bytes, static_cast<const TT*>(table),
                             static_cast<OT*>(out), tokens, vocab, d, scale, tpc);
      };
      if (vec && rows == 4) go(embedding_forward_kernel<TT, OT, true, 4>);
      else if (vec) go(embedding_forward_kernel<TT, OT, true, 1>);
      else if (rows == 4) go(embedding_forward_kernel<TT, OT, false, 4>);
      else go(embedding_forward_kernel<TT, OT, false, 1>);
    });
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}

extern "C" int prm_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t d, size_t* bytes) {
  using namespace prm;
  if (bytes == nullptr) return PRM_ERR_INVALID_ARG;
  const int rc = check_sizes(tokens, vocab, d);
  if (rc != PRM_OK) return rc;
  *bytes = tokens == 0 ? 0 : plan(tokens, vocab, d).bytes;
  return PRM_OK;
}

extern "C" int prm_embedding_backward(const void* dout, int dout_dtype, const void* token, int token_bytes, void* grad,
                                      int grad_dtype, int accumulate, int64_t tokens, int64_t vocab, int64_t d,
                                      float scale, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace prm;
  if ((token_bytes != 4 && token_bytes != 8) || !is_dtype(dout_dtype) || !is_dtype(grad_dtype) ||
      !std::isfinite(scale))
    return PRM_ERR_INVALID_ARG;
  int rc = check_sizes(tokens, vocab, d);
  if (rc != PRM_OK) return rc;
  if (grad == nullptr) return PRM_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tokens > 0 && (dout == nullptr || token == nullptr)) return PRM_ERR_INVALID_ARG;
  const EmbPlan pl = plan(tokens, vocab, d);
  if (tokens > 0) {
    if (workspace == nullptr || workspace_bytes < pl.bytes) return PRM_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return PRM_ERR_ALIGNMENT;
  }
  // Rows cleared beside the sort: what fits its time (about 8 us and 24 us
  // more for 65536 tokens) at about 6 GB/ms; all of them without tokens.
  const int64_t row_bytes = d * static_cast<int64_t>(dtype_bytes(grad_dtype));
  int64_t cleared = 0;
  if (!accumulate) {
    const double share = pl.cluster ? 6e3 * (8.0 + 24.0 * static_cast<double>(tokens) / 65536.0) : 0.0;
    cleared = tokens == 0 ? vocab : std::min<int64_t>(vocab, static_cast<int64_t>(share * 1e3 / static_cast<double>(row_bytes)));
    const int64_t bytes = cleared * row_bytes;
    // two CTAs per SM leave the sort registers and threads beside them
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((bytes / 16 + EMB_THREADS) / EMB_THREADS, 152 * 2));
    if (bytes > 0) {
      e = launch_dependent(clear_kernel, dim3(blocks), dim3(EMB_THREADS), 0, st, static_cast<uint8_t*>(grad), bytes);
      if (e != cudaSuccess) return PRM_ERR_CUDA;
    }
  }
  if (tokens == 0) return PRM_OK;
  char* ws = static_cast<char*>(workspace);
  SortPass s{};
  if (pl.cluster) {
    ClusterSort c{};
    c.token = token;
    c.token_bytes = token_bytes;
    c.count = static_cast<uint32_t>(tokens);
    c.vocab = static_cast<uint32_t>(vocab);
    c.chunk = static_cast<uint32_t>((tokens + EMB_CLUSTER * 1024 - 1) / (EMB_CLUSTER * 1024)) * 1024;
    c.passes = pl.passes;
    c.bits = pl.bits;
    c.beside = cleared > 0;
    c.keys = s.keys_out = reinterpret_cast<uint32_t*>(ws + pl.keys[0]);
    c.pos = s.pos_out = reinterpret_cast<uint32_t*>(ws + pl.pos[0]);
    if (launch_cluster_sort(c, st) != cudaSuccess) return PRM_ERR_CUDA;
  } else {
    s.token = token;
    s.hist = reinterpret_cast<uint32_t*>(ws + pl.hist);
    s.count = static_cast<uint32_t>(tokens);
    s.vocab = static_cast<uint32_t>(vocab);
    s.bits = pl.bits;
    s.tiles = pl.tiles;
    for (int k = 0; k < pl.passes; ++k) {
      s.token_bytes = k == 0 ? token_bytes : 0;
      s.keys_in = s.keys_out;
      s.pos_in = s.pos_out;
      s.keys_out = reinterpret_cast<uint32_t*>(ws + pl.keys[k & 1]);
      s.pos_out = reinterpret_cast<uint32_t*>(ws + pl.pos[k & 1]);
      s.shift = k * pl.bits;
      if ((e = launch_dependent(sort_hist_kernel, dim3(pl.tiles), dim3(EMB_THREADS), 0, st, s)) != cudaSuccess ||
          (e = launch_dependent(sort_scan_kernel, dim3(1), dim3(1024), 0, st, s)) != cudaSuccess ||
          (e = launch_dependent(sort_scatter_kernel, dim3(pl.tiles), dim3(EMB_THREADS), 0, st, s)) != cudaSuccess)
        return PRM_ERR_CUDA;
    }
  }
  EmbSum m{};
  m.keys = s.keys_out;
  m.pos = s.pos_out;
  m.count = static_cast<uint32_t>(tokens);
  m.vocab = static_cast<uint32_t>(vocab);
  m.pieces = pl.pieces;
  m.d = d;
  m.scale = scale;
  m.accumulate = accumulate != 0;
  m.tpc = row_threads(d);
  m.partial = pl.partial;
  m.head = reinterpret_cast<float*>(ws + pl.head);
  m.tail = reinterpret_cast<float*>(ws + pl.tail);
  m.block = pl.blocks > 0 ? reinterpret_cast<float*>(ws + pl.block) : nullptr;
  const bool vec = d % 8 == 0 && aligned_to(dout, 16) && aligned_to(grad, 16);
  const int per = EMB_THREADS / m.tpc;
  const unsigned blocks = static_cast<unsigned>((pl.pieces + per - 1) / per);
  const unsigned slabs = static_cast<unsigned>((d + 8 * m.tpc - 1) / (8 * m.tpc));
  m.rows = tokens;
  m.clear_from = static_cast<uint32_t>(cleared);
  // enough CTAs to keep the writes busy, where they are not all cleared yet
  const int64_t gap_rows = accumulate ? 0 : vocab - cleared;
  const unsigned ctas = static_cast<unsigned>(std::max<int64_t>(blocks, std::min<int64_t>(gap_rows / 4, 152 * 3)));
  m.clear_ctas = gap_rows > 0 ? std::min(ctas, 152u * 3u) : 0u;  // what runs at once; later CTAs only sum
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;
  m.err = dev->d_err;
  const bool ring = aligned_to(dout, 16);
  const size_t row = static_cast<size_t>(std::min<int64_t>(d, 8 * m.tpc)) * dtype_bytes(dout_dtype);
  m.pitch = static_cast<uint32_t>(vec ? row : round_up(row, 16) + 32);
  const size_t smem = ring ? static_cast<size_t>(per) * EMB_PIECE * m.pitch : 0;
  e = cudaErrorInvalidValue;
  one_type(dout_dtype, [&](auto dt) {
    one_type(grad_dtype, [&](auto gt) {
      using DT = decltype(dt);
      using GT = decltype(gt);
      auto go = [&](auto access, auto span) {
        constexpr int A = decltype(access)::value;
        e = piece_setup<DT, GT, A>();
        if (e == cudaSuccess)
          e = launch_dependent(piece_kernel<DT, GT, A>, dim3(ctas, slabs), dim3(EMB_THREADS), smem, st, m,
                               static_cast<const DT*>(dout), static_cast<GT*>(grad));
        if (e == cudaSuccess && pl.blocks > 0)
          e = launch_dependent(block_kernel, dim3((pl.blocks + per - 1) / per, slabs), dim3(EMB_THREADS), 0, st, m);
        if (e == cudaSuccess && pl.pieces > 1)
          e = launch_dependent(span, dim3(blocks, slabs), dim3(EMB_THREADS), 0, st, m, static_cast<GT*>(grad));
      };
      if (vec) go(std::integral_constant<int, VEC>{}, span_kernel<GT, true>);
      else if (ring) go(std::integral_constant<int, ELEM>{}, span_kernel<GT, false>);
      else go(std::integral_constant<int, DIRECT>{}, span_kernel<GT, false>);
    });
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
