// Token embedding: out[t] = scale table[token[t]], and the gradient of the
// table, grad[v] = scale sum_{token[t] = v} dout[t].
//
// Forward: a gather bound by memory; `tpc` threads copy a row, 8 elements
// each.
//
// Gradient: the tokens are sorted with their positions by a stable radix
// sort (least significant digit first, up to 9 bits a pass), so that equal
// tokens stand together in the order of t. The sorted list is cut into
// pieces of EMB_PIECE entries; a piece sums each of its runs of equal tokens
// in fp32. A run inside one piece goes straight to its row of grad; a run
// that crosses pieces leaves one partial sum per piece, and a last kernel
// adds those in order. A frequent token's run is thus spread over many SMs,
// and no sum depends on the order in which CTAs run. Rows without tokens are
// zeroed beforehand.
#include <algorithm>
#include <cmath>

#include "blocks.cuh"

namespace prm {
namespace {

constexpr int EMB_THREADS = 256;
constexpr int EMB_TILE = 2048;   // tokens per CTA of a sorting pass
constexpr int EMB_MAX_BITS = 9;  // digit of one pass
constexpr int EMB_MAX_BINS = 1 << EMB_MAX_BITS;
constexpr int EMB_PIECE = 32;

// Threads that share a row: a power of two, one 8-element vector each per
// step over the columns.
inline int row_threads(int64_t d) {
  int t = 1;
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

template <typename TT, typename OT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS)
    embedding_forward_kernel(const void* __restrict__ token, int token_bytes, const TT* __restrict__ table,
                             OT* __restrict__ out, int64_t tokens, int64_t vocab, int64_t d, float scale, int tpc) {
  const int tid = threadIdx.x & (tpc - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / tpc) + threadIdx.x / tpc;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= tokens) return;
  const int64_t v = load_token(token, token_bytes, t);
  const bool valid = v >= 0 && v < vocab;
  const TT* row = table + (valid ? v : 0) * d;
  for (int64_t c0 = 0; c0 < d; c0 += 8 * tpc) {
    float o[8];
    load8<TT, VEC>(row, c0, valid ? d : 0, tid, tpc, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= scale;
    store8<OT, VEC>(out + t * d, c0, d, tid, tpc, o);
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
  float* head;  // [piece][d]: sum of the run that entered from the piece before
  float* tail;  // [piece][d]: sum of the run that starts here and goes on
};

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

template <typename DT, typename GT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) piece_kernel(const EmbSum s, const DT* __restrict__ dout, GT* grad) {
  const int tid = threadIdx.x & (s.tpc - 1);
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / s.tpc) + threadIdx.x / s.tpc;
  pdl_wait();
  pdl_launch_dependents();
  if (piece >= s.pieces) return;
  const uint32_t i0 = static_cast<uint32_t>(piece) * EMB_PIECE;
  const uint32_t i1 = min(s.count, i0 + EMB_PIECE);
  const uint32_t before = i0 > 0 ? s.keys[i0 - 1] : 0xffffffffu;
  const uint32_t after = i1 < s.count ? s.keys[i1] : 0xffffffffu;
  for (int64_t c0 = 0; c0 < s.d; c0 += 8 * s.tpc) {
    uint32_t i = i0;
    while (i < i1) {
      const uint32_t v = s.keys[i];
      if (v >= s.vocab) break;  // padding
      const bool from_before = i == i0 && v == before;
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      do {
        float x[8];
        load8<DT, VEC>(dout + static_cast<int64_t>(s.pos[i]) * s.d, c0, s.d, tid, s.tpc, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += x[e];
        ++i;
      } while (i < i1 && s.keys[i] == v);
      if (from_before)
        store8<float, VEC>(s.head + piece * s.d, c0, s.d, tid, s.tpc, acc);
      else if (i == i1 && v == after)
        store8<float, VEC>(s.tail + piece * s.d, c0, s.d, tid, s.tpc, acc);
      else
        finish_row<GT, VEC>(s, grad, v, c0, tid, acc);
    }
  }
}

// Adds up the run that starts in `piece` and goes on into the next ones.
template <typename GT, bool VEC>
__global__ void __launch_bounds__(EMB_THREADS) span_kernel(const EmbSum s, GT* grad) {
  const int tid = threadIdx.x & (s.tpc - 1);
  const int64_t piece = static_cast<int64_t>(blockIdx.x) * (EMB_THREADS / s.tpc) + threadIdx.x / s.tpc;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 8 * s.tpc;
  pdl_wait();
  pdl_launch_dependents();
  if (piece + 1 >= s.pieces) return;
  const uint32_t i1 = static_cast<uint32_t>(piece + 1) * EMB_PIECE;
  const uint32_t v = s.keys[i1 - 1];
  if (v >= s.vocab || s.keys[i1] != v) return;
  const uint32_t i0 = i1 - EMB_PIECE;
  if (s.keys[i0] == v && i0 > 0 && s.keys[i0 - 1] == v) return;  // the run entered from before: an earlier piece's
  float acc[8];
  load8<float, VEC>(s.tail + piece * s.d, c0, s.d, tid, s.tpc, acc);
  // pieces that hold the run: one after another while their first key is v
  uint32_t last = static_cast<uint32_t>(piece) + 1;
  while (last + 1 < s.pieces && s.keys[static_cast<uint32_t>(last + 1) * EMB_PIECE] == v) ++last;
#pragma unroll 4
  for (uint32_t q = static_cast<uint32_t>(piece) + 1; q <= last; ++q) {
    float x[8];
    load8<float, VEC>(s.head + static_cast<int64_t>(q) * s.d, c0, s.d, tid, s.tpc, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += x[e];
  }
  finish_row<GT, VEC>(s, grad, v, c0, tid, acc);
}

// ------------------------------------------------------------------- layout
struct EmbPlan {
  int passes, bits;
  uint32_t tiles, pieces;
  size_t keys[2], pos[2], hist, head, tail, bytes;
};

EmbPlan plan(int64_t tokens, int64_t vocab, int64_t d) {
  EmbPlan p{};
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;  // keys 0 .. vocab
  p.passes = (bits + EMB_MAX_BITS - 1) / EMB_MAX_BITS;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = static_cast<uint32_t>((tokens + EMB_TILE - 1) / EMB_TILE);
  p.pieces = static_cast<uint32_t>((tokens + EMB_PIECE - 1) / EMB_PIECE);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  for (int k = 0; k < 2; ++k) {
    p.keys[k] = take(static_cast<size_t>(tokens) * 4);
    p.pos[k] = take(static_cast<size_t>(tokens) * 4);
  }
  p.hist = take((size_t(1) << p.bits) * p.tiles * 4);
  p.head = take(static_cast<size_t>(p.pieces) * d * 4);
  p.tail = take(static_cast<size_t>(p.pieces) * d * 4);
  p.bytes = at;
  return p;
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
  const dim3 grid(static_cast<unsigned>((tokens + per - 1) / per));
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
      if (vec) go(embedding_forward_kernel<TT, OT, true>);
      else go(embedding_forward_kernel<TT, OT, false>);
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
  if (tokens > 0 && (dout == nullptr || token == nullptr)) return PRM_ERR_INVALID_ARG;
  const EmbPlan pl = plan(tokens, vocab, d);
  if (tokens > 0) {
    if (workspace == nullptr || workspace_bytes < pl.bytes) return PRM_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return PRM_ERR_ALIGNMENT;
  }
  if (!accumulate) {
    const size_t bytes = static_cast<size_t>(vocab) * d * dtype_bytes(grad_dtype);
    if (cudaMemsetAsync(grad, 0, bytes, st) != cudaSuccess) return PRM_ERR_CUDA;
  }
  if (tokens == 0) return PRM_OK;
  char* ws = static_cast<char*>(workspace);
  cudaError_t e;
  SortPass s{};
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
  EmbSum m{};
  m.keys = s.keys_out;
  m.pos = s.pos_out;
  m.count = s.count;
  m.vocab = s.vocab;
  m.pieces = pl.pieces;
  m.d = d;
  m.scale = scale;
  m.accumulate = accumulate != 0;
  m.tpc = row_threads(d);
  m.head = reinterpret_cast<float*>(ws + pl.head);
  m.tail = reinterpret_cast<float*>(ws + pl.tail);
  const bool vec = d % 8 == 0 && aligned_to(dout, 16) && aligned_to(grad, 16);
  const int per = EMB_THREADS / m.tpc;
  const unsigned blocks = static_cast<unsigned>((pl.pieces + per - 1) / per);
  const unsigned slabs = static_cast<unsigned>((d + 8 * m.tpc - 1) / (8 * m.tpc));
  e = cudaErrorInvalidValue;
  one_type(dout_dtype, [&](auto dt) {
    one_type(grad_dtype, [&](auto gt) {
      using DT = decltype(dt);
      using GT = decltype(gt);
      auto go = [&](auto pieces, auto span) {
        e = launch_dependent(pieces, dim3(blocks), dim3(EMB_THREADS), 0, st, m, static_cast<const DT*>(dout),
                             static_cast<GT*>(grad));
        if (e == cudaSuccess && pl.pieces > 1)
          e = launch_dependent(span, dim3(blocks, slabs), dim3(EMB_THREADS), 0, st, m, static_cast<GT*>(grad));
      };
      if (vec) go(piece_kernel<DT, GT, true>, span_kernel<GT, true>);
      else go(piece_kernel<DT, GT, false>, span_kernel<GT, false>);
    });
  });
  return e == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
