// Gated feed-forward block on the tensor cores, forward and backward:
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// Four launches of one persistent tcgen05 kernel with three epilogues:
//   GLU   : x against Wg and Wu at once. A pair of CTAs computes 256 tokens x
//           128 features of g and of u in one accumulator (the even CTA holds
//           the rows of Wg, the odd one those of Wu), so the activation and
//           the product happen in registers: g and u never go to memory as
//           GEMM outputs, only h does (and, for training, g and u once, packed)
//   DGLU  : dh = dy Wd; dh stays in the accumulator, dg and du come out
//   STORE : plain products: y; and dx, dWd, dWg, dWu from one tile queue
// Operands are read in the layout the caller has: K-major or MN-major tiles
// by TMA, without a transposed copy. dx sums over both projections in one
// accumulator (two operand pairs, one after the other, along K).
//
// Rounding: products accumulate in fp32. h, dg and du are rounded to 16 bits
// because they are operands of the next product. g and u are kept for the
// backward pass with 16 significand bits (24-bit floats: fp32 with the low
// byte cut off, 6 bytes for the two), so that the derivative adds no error
// next to those roundings: in an fp64 model of these steps (1024 tokens,
// 512 x 2048) the gradients were 0.0023 from the exact ones, as with g and u
// kept exactly, and with bf16 g and u 0.0029 - 0.0035.
//
// Bound by the tensor cores for more than a few hundred tokens. 8192 tokens,
// 2048 x 8192, bf16: forward 488 us (1.69 PFLOP/s), with g and u saved 515,
// backward 1185 (1.39), both passes 1.65 - 1.77 ms (1.50 - 1.40 PFLOP/s: the SM
// clock under the power cap decides); those of 4096 tokens, 5120 x 20480 4.87 -
// 5.20 ms (1.59 - 1.49). 16384 tokens, 768 x 2048: 0.43 ms (1.07); 65536 tokens, 256 x 704,
// where the tensors' bytes weigh more: 0.66 ms. Each launch alone (8192 tokens,
// 2048 x 8192): GLU 314 us (1.75 PFLOP/s, with 400 MB of g and u written), down
// 193 (1.43), DGLU 198 (1.39, 790 MB moved), gradients 870 (1.58); the tensor
// pipe is active 79, 65, 67 and 68 % of the time: every pair loads all of its
// operands itself, the last rounds are part empty, and DGLU's epilogue waits
// for g and u.
//
// CTA layout, pipeline and TMEM use are those of the Newton-Schulz GEMMs
// (ns5_gemm.cu): 320 threads, warp 0 TMA producer, warp 1 MMA issue in the
// even CTA, warps 2-9 epilogue; 256 x 256 tiles, six 32 KB stages, two
// accumulators.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "ffn.cuh"

namespace prm {
namespace {

constexpr int PAIR_M = 256;
constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BN_HALF = 128;
constexpr int BK = 64;
constexpr int UK = 16;
constexpr int STAGES = 6;
constexpr uint32_t TILE_BYTES = BM * BK * 2;  // 16 KB, A and B alike
constexpr uint32_t STAGE_BYTES = 2 * TILE_BYTES;
constexpr uint32_t PAIR_STAGE_BYTES = 2 * STAGE_BYTES;
constexpr uint32_t MN_CHUNK_BYTES = 64 * BK * 2;  // one 64-column MN-major box
constexpr int NUM_THREADS = 320;
constexpr int EPI_WARPS = 8;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr uint32_t EPI_BUF_BYTES = 32 * 64;  // one 32 x 32 box of 16-bit values
constexpr uint32_t EPI_WARP_BYTES = 2 * EPI_BUF_BYTES;
constexpr size_t EPI_SMEM_BYTES = EPI_WARPS * EPI_WARP_BYTES;
constexpr size_t BARRIER_BYTES = 256;
constexpr size_t SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_SMEM_BYTES + BARRIER_BYTES;
static_assert(SMEM_BYTES <= 232448, "dynamic shared memory above the 227 KB per-block limit");
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

constexpr int EPI_GLU = 0, EPI_DGLU = 1, EPI_STORE = 2;

// One product out = sum over its operand pairs of A B^T (B given K-major) or
// A B (B given MN-major).
struct FfnSegment {
  CUtensorMap a[2];
  CUtensorMap b[2];
  CUtensorMap out[2];   // GLU: h; DGLU: dg, du; STORE: the product
  int M, N;             // output extents (GLU: N = f)
  int k_blocks[2];      // 64-long slices of each pair along K
  int a_mn, b_mn;       // operand stored [K][M] / [K][N]
  int tiles_m, tiles_n;
  int whole;            // tiles that one CTA pair computes; the rest are split
  int splits;           // pairs per split tile, each over a part of K
  int64_t item_begin;
  float* partial;       // splits > 1: fp32 parts of the split tiles
  uint32_t* arrived;    // splits > 1: arrivals per warp region, zero before the launch
};

constexpr int MAX_SEGS = 4;
struct FfnParams {
  FfnSegment seg[MAX_SEGS];
  int nseg;
  int64_t total;        // work items: whole tiles and parts of split ones
  int64_t long_items, hole_end;  // see next_item
  uint4* gu;            // packed g and u (GLU: written when not NULL; DGLU: read)
  uint32_t* zero;       // counters to clear for the next launch
  int zero_count;
  int* err;
};
static_assert(sizeof(FfnParams) <= 4096, "kernel parameters above the 4 KB classic limit");

struct Item {
  int m0, n0;           // first output row; first output column (GLU: first feature)
  int split_tile, split;  // split tiles: index among them and part; else -1
  int kb0, kb1;
};

// Tiles run in groups of GROUP_M row tiles, rows fastest, so that the 76
// pairs at work cover a block of about 8 x 9 tiles: per slice of K they share
// half the operand bytes of a 32 x 2 block.
constexpr int GROUP_M = 8;

__device__ __forceinline__ int ffn_seg(const FfnParams& p, int64_t item) {
  int s = 0;
  while (s + 1 < p.nseg && item >= p.seg[s + 1].item_begin) ++s;
  return s;
}

// The item of CTA pair c of n after `item` (first: item = c - n). Items go
// round the pairs. Where the first product has longer sums than the others
// and its items leave a last round part empty, the pairs without one take
// that many short items more (the hole, up to hole_end), so that all come to
// the end together (17 tile times instead of 18 at 8192 x 2048 x 8192, 106
// instead of 113 at 4096 x 5120 x 20480; both passes, in turn on one machine,
// 1652 us instead of 1674 and 4898 instead of 5031).
template <int EPI>
__device__ __forceinline__ int64_t next_item(const FfnParams& p, int64_t item, int64_t c, int64_t n) {
  if (EPI != EPI_STORE || item >= p.hole_end) return item + n;
  const int64_t rest = static_cast<uint32_t>(p.long_items) % static_cast<uint32_t>(n);  // pairs with an item then
  int64_t to;
  if (item >= p.long_items) {
    to = item + n - rest;
  } else {
    to = item + n;
    if (to < p.long_items) return to;
    if (c < rest) return p.hole_end + c;
    to = p.long_items + c - rest;
  }
  return to < p.hole_end ? to : p.hole_end + c;
}

template <int EPI>
__device__ __forceinline__ Item ffn_item(const FfnSegment& sg, int64_t item) {
  Item it;
  int tile = static_cast<int>(item - sg.item_begin);
  const int kb = sg.k_blocks[0] + sg.k_blocks[1];
  it.split_tile = -1;
  it.split = 0;
  it.kb0 = 0;
  it.kb1 = kb;
  if (EPI == EPI_STORE && tile >= sg.whole) {
    const int q = tile - sg.whole;
    it.split_tile = q / sg.splits;
    it.split = q - it.split_tile * sg.splits;
    it.kb0 = static_cast<int>(static_cast<int64_t>(kb) * it.split / sg.splits);
    it.kb1 = static_cast<int>(static_cast<int64_t>(kb) * (it.split + 1) / sg.splits);
    tile = sg.whole + it.split_tile;
  }
  const int group = tile / (GROUP_M * sg.tiles_n);
  const int rows = min(GROUP_M, sg.tiles_m - group * GROUP_M);
  const int in_group = tile - group * GROUP_M * sg.tiles_n;
  const int tn = in_group / rows;
  it.m0 = (group * GROUP_M + in_group - tn * rows) * PAIR_M;
  it.n0 = tn * (EPI == EPI_GLU ? BN_HALF : BN);
  return it;
}

__device__ __forceinline__ uint32_t ffn_stage_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// Writes this lane's row of a 32 x 32 box (16 packed words) to the staging
// box in the 64-byte swizzle of the output maps.
__device__ __forceinline__ void ffn_stage(uint8_t* box, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(box + ffn_stage_off(lane, c)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// Packed g and u of one 32 x 32 box: 12 vectors of 16 bytes per lane, vector
// k of lane l at box * 384 + k * 32 + l. Words 0..31 hold the high halves of
// g (low 16 bits) and u (high 16 bits) of the lane's 32 columns, words 32..47
// the next 8 bits of both, two columns to a word.
__device__ __forceinline__ int64_t gu_box(int i0, int j0, int f) {
  return (static_cast<int64_t>(i0 >> 5) * ((f + 31) >> 5) + (j0 >> 5)) * 384;
}

template <typename T, int ACT>
__device__ __forceinline__ void glu_chunk(const FfnParams& p, const FfnSegment& sg, int i0, int j0, uint32_t t_g,
                                          uint32_t t_u, uint8_t* stage, int lane) {
  float g[32], u[32];
  tmem_load_32cols(t_g, g);
  tmem_load_32cols(t_u, u);
  if (i0 >= sg.M) return;
  if (p.gu != nullptr) {
    uint4* box = p.gu + gu_box(i0, j0, sg.N) + lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = __byte_perm(__float_as_uint(g[4 * k + e]), __float_as_uint(u[4 * k + e]), 0x7632);
      __stcs(box + k * 32, make_uint4(w[0], w[1], w[2], w[3]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 8 * k + 2 * e;
        const uint32_t lo = __byte_perm(__float_as_uint(g[c]), __float_as_uint(u[c]), 0x0051);
        const uint32_t hi = __byte_perm(__float_as_uint(g[c + 1]), __float_as_uint(u[c + 1]), 0x0051);
        w[e] = __byte_perm(lo, hi, 0x5410);
      }
      __stcs(box + (8 + k) * 32, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  uint32_t w[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float a = ffn_act<ACT>(g[2 * k]) * u[2 * k];
    const float b = ffn_act<ACT>(g[2 * k + 1]) * u[2 * k + 1];
    w[k] = pack2<T>(a, b);
  }
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
  ffn_stage(stage, lane, w);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&sg.out[0], stage, j0, i0);
    bulk_commit_group();
  }
}

__device__ __forceinline__ void gu_load(const FfnParams& p, int i0, int j0, int f, int lane, uint4 (&raw)[12]) {
  const uint4* box = p.gu + gu_box(i0, j0, f) + lane;
#pragma unroll
  for (int k = 0; k < 12; ++k) raw[k] = __ldcs(box + k * 32);
}

template <typename T, int ACT>
__device__ __forceinline__ void dglu_chunk(const FfnParams& p, const FfnSegment& sg, int i0, int j0, uint32_t t_dh,
                                           const uint4 (&raw)[12], uint8_t* stage, int lane) {
  float dh[32];
  tmem_load_32cols(t_dh, dh);
  uint32_t wg[16], wu[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float dg[2], du[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = 2 * k + e;
      const uint4 hv = raw[c >> 2];
      const uint32_t hi = (c & 3) == 0 ? hv.x : (c & 3) == 1 ? hv.y : (c & 3) == 2 ? hv.z : hv.w;
      const uint4 lv = raw[8 + (c >> 3)];
      const int q = (c >> 1) & 3;
      const uint32_t lo = q == 0 ? lv.x : q == 1 ? lv.y : q == 2 ? lv.z : lv.w;
      // lo holds (g, u) of the even column in bytes 0, 1 and of the odd one in bytes 2, 3; the byte
      // below the kept ones repeats the lowest of them, which leaves an infinity what it is
      const float g = __uint_as_float(__byte_perm(lo, hi, (c & 1) ? 0x5422 : 0x5400));
      const float u = __uint_as_float(__byte_perm(lo, hi, (c & 1) ? 0x7633 : 0x7611));
      float a, da;
      ffn_act_grad<ACT>(g, &a, &da);
      dg[e] = dh[c] * u * da;
      du[e] = dh[c] * a;
    }
    wg[k] = pack2<T>(dg[0], dg[1]);
    wu[k] = pack2<T>(du[0], du[1]);
  }
  if (i0 >= sg.M) return;
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
  ffn_stage(stage, lane, wg);
  ffn_stage(stage + EPI_BUF_BYTES, lane, wu);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&sg.out[0], stage, j0, i0);
    tma_store_2d(&sg.out[1], stage + EPI_BUF_BYTES, j0, i0);
    bulk_commit_group();
  }
}

template <typename T>
__device__ __forceinline__ void store_box(const FfnSegment& sg, int i0, int j0, const float (&v)[32], uint8_t* stage,
                                          int lane) {
  if (i0 >= sg.M || j0 >= sg.N) return;
  uint32_t w[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
  ffn_stage(stage, lane, w);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&sg.out[0], stage, j0, i0);
    bulk_commit_group();
  }
}

template <int EPI, typename T, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * TILE_BYTES;
  uint8_t* sEpi = smem + STAGES * STAGE_BYTES;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(sEpi + EPI_SMEM_BYTES);
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* tfull_bar = empty_bar + STAGES;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int64_t cluster_id = blockIdx.x / 2;
  const int64_t num_clusters = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, TMEM_COLS);
    tmem_relinquish_pair();
  }
  // Both CTAs' barriers must exist before either signals the other.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait();
  pdl_launch_dependents();  // the next kernel sets up on SMs that this one leaves or does not use
  if (p.zero != nullptr && blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.zero_count; i += NUM_THREADS) p.zero[i] = 0;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;
      bool ok = true;
      for (int64_t item = next_item<EPI>(p, cluster_id - num_clusters, cluster_id, num_clusters); ok && item < p.total;
         item = next_item<EPI>(p, item, cluster_id, num_clusters)) {
        const FfnSegment& sg = p.seg[ffn_seg(p, item)];
        const Item it = ffn_item<EPI>(sg, item);
        const int m_cta = it.m0 + static_cast<int>(rank) * BM;
        const int n_cta = EPI == EPI_GLU ? it.n0 : it.n0 + static_cast<int>(rank) * BN_HALF;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!wait_bounded(&empty_bar[stage], phase ^ 1u, abort_flag, p.err, WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], PAIR_STAGE_BYTES);
          const uint32_t bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
          uint8_t* a_dst = sA + stage * TILE_BYTES;
          uint8_t* b_dst = sB + stage * TILE_BYTES;
          const int second = kb >= sg.k_blocks[0] ? 1 : 0;  // operand pair
          const int k = (second ? kb - sg.k_blocks[0] : kb) * BK;
          const CUtensorMap* ma = &sg.a[second];
          const CUtensorMap* mb = EPI == EPI_GLU ? &sg.b[rank] : &sg.b[second];
          if (EPI == EPI_STORE && sg.a_mn) {
#pragma unroll
            for (int q = 0; q < BM / 64; ++q)
              tma_load_2d_pair(a_dst + q * MN_CHUNK_BYTES, ma, bar, m_cta + q * 64, k);
          } else {
            tma_load_2d_pair(a_dst, ma, bar, k, m_cta);
          }
          if (EPI == EPI_DGLU || (EPI == EPI_STORE && sg.b_mn)) {
#pragma unroll
            for (int q = 0; q < BN_HALF / 64; ++q)
              tma_load_2d_pair(b_dst + q * MN_CHUNK_BYTES, mb, bar, n_cta + q * 64, k);
          } else {
            tma_load_2d_pair(b_dst, mb, bar, k, n_cta);
          }
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && issued) {
        // Let every load already in flight land before the CTA exits; the
        // odd CTA's complete on the peer's barriers, so it waits an ample time.
        if (rank == 0) {
          for (int s = 0; s < STAGES; ++s)
            if (issued & (1u << s)) wait_drain(&full_bar[s], (issued_parity >> s) & 1u, 50000000ull);
        } else {
          spin_for_ns(2000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr bool FP16 = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true, issued_any = false;
      for (int64_t item = next_item<EPI>(p, cluster_id - num_clusters, cluster_id, num_clusters); ok && item < p.total;
         item = next_item<EPI>(p, item, cluster_id, num_clusters)) {
        const FfnSegment& sg = p.seg[ffn_seg(p, item)];
        const Item it = ffn_item<EPI>(sg, item);
        const bool a_mn = EPI == EPI_STORE && sg.a_mn;
        const bool b_mn = EPI == EPI_DGLU || (EPI == EPI_STORE && sg.b_mn);
        const uint32_t idesc = idesc_f16kind_f32(PAIR_M, BN, a_mn, b_mn, FP16);
        if (!wait_bounded(&tempty_bar[acc], acc_phase ^ 1u, abort_flag, p.err, WAIT_LIMIT_NS)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!wait_bounded(&full_bar[stage], phase, abort_flag, p.err, WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_addr = smem_u32(sA + stage * TILE_BYTES);
          const uint32_t b_addr = smem_u32(sB + stage * TILE_BYTES);
#pragma unroll
          for (int k = 0; k < BK / UK; ++k) {
            const uint64_t ad = a_mn ? smem_desc_sw128(a_addr + k * UK * 128, MN_CHUNK_BYTES, 1024)
                                     : smem_desc_sw128(a_addr + k * UK * 2, 16, 1024);
            const uint64_t bd = b_mn ? smem_desc_sw128(b_addr + k * UK * 128, MN_CHUNK_BYTES, 1024)
                                     : smem_desc_sw128(b_addr + k * UK * 2, 16, 1024);
            umma_bf16_pair(d_tmem, ad, bd, idesc, (kb - it.kb0) | k ? 1u : 0u);
          }
          issued_any = true;
          umma_commit_pair_multicast(&empty_bar[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_multicast(&tfull_bar[acc], 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && issued_any) {
        umma_commit_pair_multicast(drain_bar, 0x1);
        wait_drain(drain_bar, 0, 50000000ull);
      }
    }
  } else {
    const int quarter = warp & 3;
    const int ew = warp - 2;
    const int half = ew >> 2;
    uint8_t* stage = sEpi + ew * EPI_WARP_BYTES;
    const uint32_t tempty_even = mapa_shared(smem_u32(&tempty_bar[0]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t item = next_item<EPI>(p, cluster_id - num_clusters, cluster_id, num_clusters); item < p.total;
         item = next_item<EPI>(p, item, cluster_id, num_clusters)) {
      const FfnSegment& sg = p.seg[ffn_seg(p, item)];
      const Item it = ffn_item<EPI>(sg, item);
      const int i0 = it.m0 + static_cast<int>(rank) * BM + quarter * 32;
      const int jh = it.n0 + half * (EPI == EPI_GLU ? BN_HALF / 2 : BN / 2);  // first column of this warp
      uint4 raw[2][EPI == EPI_DGLU ? 12 : 1];
      if constexpr (EPI == EPI_DGLU) {
        if (i0 < sg.M && jh < sg.N) gu_load(p, i0, jh, sg.N, lane, raw[0]);
      }
      const bool got = wait_bounded(&tfull_bar[acc], acc_phase, abort_flag, p.err, WAIT_LIMIT_NS);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after_sync();
      const uint32_t t_row =
          tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quarter * 32) << 16);
      if constexpr (EPI == EPI_GLU) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int j0 = jh + q * 32;
          if (j0 < sg.N) {
            const uint32_t col = static_cast<uint32_t>(half * (BN_HALF / 2) + q * 32);
            glu_chunk<T, ACT>(p, sg, i0, j0, t_row + col, t_row + BN_HALF + col, stage, lane);
          }
        }
      } else if constexpr (EPI == EPI_DGLU) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j0 = jh + q * 32;
          if (q < 3 && i0 < sg.M && j0 + 32 < sg.N) gu_load(p, i0, j0 + 32, sg.N, lane, raw[(q + 1) & 1]);
          if (j0 < sg.N)
            dglu_chunk<T, ACT>(p, sg, i0, j0, t_row + static_cast<uint32_t>(half * (BN / 2) + q * 32), raw[q & 1], stage,
                          lane);
        }
      } else if (it.split_tile < 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[32];
          tmem_load_32cols(t_row + static_cast<uint32_t>(half * (BN / 2) + q * 32), v);
          store_box<T>(sg, i0, jh + q * 32, v, stage, lane);
        }
      } else {
        // A part of the sum along K: this warp's 32 x 128 values go to the
        // workspace; the warp that arrives last for them adds all parts, in
        // order, and stores the result. Warps without rows have nothing to do.
        const int64_t region = (static_cast<int64_t>(it.split_tile) * 2 + rank) * EPI_WARPS + ew;
        float4* mine = reinterpret_cast<float4*>(sg.partial) + (region * sg.splits + it.split) * (32 * 32) + lane;
        if (i0 < sg.M) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[32];
            tmem_load_32cols(t_row + static_cast<uint32_t>(half * (BN / 2) + q * 32), v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(mine + (q * 8 + k) * 32, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
          }
          __threadfence();
          __syncwarp();
          uint32_t before = 0;
          if (lane == 0) before = atomicAdd(&sg.arrived[region], 1u);
          before = __shfl_sync(0xffffffffu, before, 0);
          if (before + 1 == static_cast<uint32_t>(sg.splits)) {
            __threadfence();
            const float4* all = reinterpret_cast<const float4*>(sg.partial) + region * sg.splits * (32 * 32) + lane;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              float v[32] = {};
              for (int s = 0; s < sg.splits; s += 2) {  // two parts in flight
                float4 a[8], b[8];
                const bool two = s + 1 < sg.splits;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  a[k] = __ldcg(all + s * (32 * 32) + (q * 8 + k) * 32);
                  b[k] = two ? __ldcg(all + (s + 1) * (32 * 32) + (q * 8 + k) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  v[4 * k] = v[4 * k] + a[k].x + b[k].x;
                  v[4 * k + 1] = v[4 * k + 1] + a[k].y + b[k].y;
                  v[4 * k + 2] = v[4 * k + 2] + a[k].z + b[k].z;
                  v[4 * k + 3] = v[4 * k + 3] + a[k].w + b[k].w;
                }
              }
              store_box<T>(sg, i0, jh + q * 32, v, stage, lane);
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_even + static_cast<uint32_t>(acc * sizeof(uint64_t)));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_group_all();
  }
  __syncwarp();
  // No CTA may leave (or free TMEM) while its peer can still touch its
  // barriers, shared memory or accumulators.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

enum MapUse { MAP_ROWS, MAP_COLS, MAP_STORE };  // 128 x 64 boxes, 64 x 64 boxes, 32 x 32 output boxes

// A row-major rows x cols matrix of 16-bit elements with row pitch ld.
bool encode(CUtensorMap* map, const void* base, int dtype, int64_t rows, int64_t cols, int64_t ld, MapUse use) {
  auto enc = map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {use == MAP_STORE ? 32u : 64u, use == MAP_STORE ? 32u : use == MAP_ROWS ? 128u : 64u};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, dtype == PRM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             use == MAP_STORE ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI, typename T, int ACT>
int resident_clusters(int num_sms) {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  const int known = cached[dev].load(std::memory_order_relaxed);
  if (known > 0) return known;
  if (cudaFuncSetAttribute(ffn_gemm_kernel<EPI, T, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(SMEM_BYTES)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, ffn_gemm_kernel<EPI, T, ACT>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = num_sms / 2;
  }
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int EPI, typename T, int ACT>
cudaError_t launch(FfnParams& p, int num_sms, cudaStream_t stream) {
  const int clusters = resident_clusters<EPI, T, ACT>(num_sms);
  if (clusters == 0) return cudaErrorInvalidConfiguration;
  const int64_t n = std::min<int64_t>(p.total, clusters);
  const unsigned grid = static_cast<unsigned>(2 * n);
  p.long_items = p.hole_end = 0;
  if (p.nseg > 1) {
    const int64_t first = p.seg[1].item_begin, kb = p.seg[0].k_blocks[0] + p.seg[0].k_blocks[1];
    const int64_t rounds = (kb + p.seg[1].k_blocks[0] / 2) / p.seg[1].k_blocks[0];  // of short items in a long one's time
    if (rounds > 1 && first % n != 0) {
      p.long_items = first;
      p.hole_end = first + (n - first % n) * rounds;
    }
  }
  return launch_dependent(ffn_gemm_kernel<EPI, T, ACT>, dim3(grid), dim3(NUM_THREADS), SMEM_BYTES, stream, p);
}

template <int EPI, int ACT = 0>
cudaError_t launch(FfnParams& p, int dtype, int num_sms, cudaStream_t stream) {
  return dtype == PRM_BF16 ? launch<EPI, __nv_bfloat16, ACT>(p, num_sms, stream)
                           : launch<EPI, __half, ACT>(p, num_sms, stream);
}

template <int EPI>
cudaError_t launch_act(FfnParams& p, int act, int dtype, int num_sms, cudaStream_t stream) {
  if (act == PRM_ACT_SILU) return launch<EPI, PRM_ACT_SILU>(p, dtype, num_sms, stream);
  if (act == PRM_ACT_GELU) return launch<EPI, PRM_ACT_GELU>(p, dtype, num_sms, stream);
  return launch<EPI, PRM_ACT_GELU_TANH>(p, dtype, num_sms, stream);
}

// Tiles of 256 x tile_n of an M x N product.
int64_t tiles_of(int64_t M, int64_t N, int tile_n) { return ((M + PAIR_M - 1) / PAIR_M) * ((N + tile_n - 1) / tile_n); }
constexpr int64_t AT_ONCE = 76;  // CTA pairs on the 152 SMs

// The tiles of a product that runs alone go to the pairs in waves. Where the
// last wave is not full, its tiles are split along K over the idle pairs: 256
// tiles on 76 pairs take 3.5 tile times instead of 4.
constexpr int MIN_PART = 4;  // slices of K in a part
struct Split {
  int64_t whole, rest;  // tiles computed whole and in parts
  int splits;
};
Split split_last_wave(int64_t M, int64_t N, int64_t K) {
  Split s{0, 0, 1};
  const int64_t items = tiles_of(M, N, BN);
  const int64_t rest = items % AT_ONCE;
  const int64_t kb = (K + BK - 1) / BK;
  // adding up the parts costs about two slices of K per part: no more parts than that pays for
  const int64_t pays = static_cast<int64_t>(std::sqrt(static_cast<double>(kb) / 2)) + 1;
  const int64_t parts = rest == 0 ? 1 : std::min<int64_t>({AT_ONCE / rest, kb / MIN_PART, pays, 16});
  s.whole = parts < 2 ? items : items - rest;
  s.rest = items - s.whole;
  s.splits = parts < 2 ? 1 : static_cast<int>(parts);
  return s;
}
size_t partial_bytes(const Split& s) {
  return static_cast<size_t>(s.rest) * s.splits * PAIR_M * BN * sizeof(float);
}
size_t counter_bytes(const Split& s) { return static_cast<size_t>(s.rest) * 2 * EPI_WARPS * 4; }

// Extents and items of one product, and its place in the queue.
void queue(FfnParams& p, FfnSegment& sg, int64_t M, int64_t N, int64_t K0, int64_t K1, bool a_mn, bool b_mn,
           int tile_n) {
  sg.M = static_cast<int>(M);
  sg.N = static_cast<int>(N);
  sg.k_blocks[0] = static_cast<int>((K0 + BK - 1) / BK);
  sg.k_blocks[1] = static_cast<int>((K1 + BK - 1) / BK);
  sg.a_mn = a_mn;
  sg.b_mn = b_mn;
  sg.tiles_m = static_cast<int>((M + PAIR_M - 1) / PAIR_M);
  const int items = static_cast<int>(tiles_of(M, N, tile_n));
  sg.tiles_n = items / sg.tiles_m;
  if (sg.splits < 2) {
    sg.whole = items;
    sg.splits = 1;
  }
  sg.item_begin = p.total;
  p.total += sg.whole + static_cast<int64_t>(items - sg.whole) * sg.splits;
  p.seg[p.nseg++] = sg;
}

struct FfnSizes {
  size_t saved_h, saved;                                     // gu at saved_h
  size_t fwd_h, fwd_partial, fwd_counters, fwd;              // offsets and size of the forward workspace
  size_t bwd_du, bwd_partial, bwd_counters, bwd;             // dg at 0
  Split down;
};

FfnSizes sizes(int64_t T, int64_t d, int64_t f) {
  FfnSizes s{};
  if (T == 0) return s;
  const size_t act = round_up(static_cast<size_t>(T) * f * 2, 256);
  s.saved_h = act;
  s.saved = act + static_cast<size_t>((T + 31) / 32) * ((f + 31) / 32) * 384 * 16;
  s.down = split_last_wave(T, d, f);
  s.fwd_partial = act;
  s.fwd_counters = act + partial_bytes(s.down);
  s.fwd = s.fwd_counters + round_up(counter_bytes(s.down), 256);
  s.bwd_du = act;
  s.bwd = 2 * act;
  return s;
}

int check(int64_t T, int64_t d, int64_t f) {
  if (T < 0 || d < 1 || f < 1) return PRM_ERR_INVALID_ARG;
  if (d % 8 != 0 || f % 8 != 0) return PRM_ERR_ALIGNMENT;
  if (T >= (int64_t(1) << 31) - 256 || d >= (int64_t(1) << 24) || f >= (int64_t(1) << 24)) return PRM_ERR_UNSUPPORTED;
  // tiles are counted in 32 bits
  constexpr int64_t MOST = int64_t(1) << 30;
  if (tiles_of(T, f, BN_HALF) > MOST || 3 * tiles_of(d, f, BN) + tiles_of(T, d, BN) > MOST) return PRM_ERR_UNSUPPORTED;
  return PRM_OK;
}

}  // namespace
}  // namespace prm

extern "C" int prm_gated_ffn_sizes(int64_t tokens, int64_t d, int64_t f, size_t* saved, size_t* forward_workspace,
                                   size_t* backward_workspace) {
  using namespace prm;
  if (saved == nullptr || forward_workspace == nullptr || backward_workspace == nullptr) return PRM_ERR_INVALID_ARG;
  const int rc = check(tokens, d, f);
  if (rc != PRM_OK) return rc;
  const FfnSizes s = sizes(tokens, d, f);
  *saved = s.saved;
  *forward_workspace = s.fwd;
  *backward_workspace = s.bwd;
  return PRM_OK;
}

extern "C" int prm_gated_ffn_forward(const void* x, int64_t ldx, const void* w_gate, const void* w_up,
                                     const void* w_down, void* y, void* saved, void* workspace,
                                     size_t workspace_bytes, int64_t tokens, int64_t d, int64_t f, int act, int dtype,
                                     void* stream) {
  using namespace prm;
  if ((dtype != PRM_BF16 && dtype != PRM_FP16) || act < PRM_ACT_SILU || act > PRM_ACT_GELU_TANH)
    return PRM_ERR_INVALID_ARG;
  int rc = check(tokens, d, f);
  if (rc != PRM_OK || tokens == 0) return rc;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr || ldx < d)
    return PRM_ERR_INVALID_ARG;
  if (ldx % 8 != 0 || !aligned_to(x, 16) || !aligned_to(w_gate, 16) || !aligned_to(w_up, 16) ||
      !aligned_to(w_down, 16) || !aligned_to(y, 16) || !aligned_to(saved, 256) || !aligned_to(workspace, 256))
    return PRM_ERR_ALIGNMENT;
  const FfnSizes sz = sizes(tokens, d, f);
  if (workspace == nullptr || workspace_bytes < sz.fwd) return PRM_ERR_WORKSPACE;
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  void* h = saved != nullptr ? saved : ws;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (ffn_few(tokens, d, f))
    return ffn_few_forward(x, ldx, w_gate, w_up, w_down, h,
                           saved != nullptr ? reinterpret_cast<uint4*>(static_cast<char*>(saved) + sz.saved_h) : nullptr,
                           y, static_cast<int>(tokens), static_cast<int>(d), static_cast<int>(f), act, dtype,
                           st) == cudaSuccess
               ? PRM_OK
               : PRM_ERR_CUDA;

  FfnParams p{};
  p.err = dev->d_err;
  p.gu = saved != nullptr ? reinterpret_cast<uint4*>(static_cast<char*>(saved) + sz.saved_h) : nullptr;
  uint32_t* counters = reinterpret_cast<uint32_t*>(ws + sz.fwd_counters);
  p.zero = counters;
  p.zero_count = static_cast<int>(counter_bytes(sz.down) / 4);
  FfnSegment sg{};
  if (!encode(&sg.a[0], x, dtype, tokens, d, ldx, MAP_ROWS) || !encode(&sg.b[0], w_gate, dtype, f, d, d, MAP_ROWS) ||
      !encode(&sg.b[1], w_up, dtype, f, d, d, MAP_ROWS) || !encode(&sg.out[0], h, dtype, tokens, f, f, MAP_STORE))
    return PRM_ERR_CUDA;
  queue(p, sg, tokens, f, d, 0, false, false, BN_HALF);
  if (launch_act<EPI_GLU>(p, act, dtype, dev->num_sms, st) != cudaSuccess) return PRM_ERR_CUDA;

  FfnParams q{};
  q.err = dev->d_err;
  FfnSegment dn{};
  if (!encode(&dn.a[0], h, dtype, tokens, f, f, MAP_ROWS) || !encode(&dn.b[0], w_down, dtype, d, f, f, MAP_ROWS) ||
      !encode(&dn.out[0], y, dtype, tokens, d, d, MAP_STORE))
    return PRM_ERR_CUDA;
  dn.whole = static_cast<int>(sz.down.whole);
  dn.splits = sz.down.splits;
  dn.partial = reinterpret_cast<float*>(ws + sz.fwd_partial);
  dn.arrived = counters;
  queue(q, dn, tokens, d, f, 0, false, false, BN);
  return launch<EPI_STORE>(q, dtype, dev->num_sms, st) == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}

extern "C" int prm_gated_ffn_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                      const void* w_up, const void* w_down, const void* saved, void* dx,
                                      void* dw_gate, void* dw_up, void* dw_down, void* workspace,
                                      size_t workspace_bytes, int64_t tokens, int64_t d, int64_t f, int act,
                                      int dtype, void* stream) {
  using namespace prm;
  if ((dtype != PRM_BF16 && dtype != PRM_FP16) || act < PRM_ACT_SILU || act > PRM_ACT_GELU_TANH)
    return PRM_ERR_INVALID_ARG;
  int rc = check(tokens, d, f);
  if (rc != PRM_OK) return rc;
  const bool weights = dw_gate != nullptr || dw_up != nullptr || dw_down != nullptr;
  if (weights && (dw_gate == nullptr || dw_up == nullptr || dw_down == nullptr)) return PRM_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    const size_t n = static_cast<size_t>(d) * f * 2;
    if (weights && (cudaMemsetAsync(dw_gate, 0, n, st) != cudaSuccess ||
                    cudaMemsetAsync(dw_up, 0, n, st) != cudaSuccess ||
                    cudaMemsetAsync(dw_down, 0, n, st) != cudaSuccess))
      return PRM_ERR_CUDA;
    return PRM_OK;
  }
  if (dy == nullptr || x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr ||
      saved == nullptr || lddy < d || ldx < d)
    return PRM_ERR_INVALID_ARG;
  const void* ptrs[9] = {dy, x, w_gate, w_up, w_down, dx, dw_gate, dw_up, dw_down};
  for (const void* q : ptrs)
    if (!aligned_to(q, 16)) return PRM_ERR_ALIGNMENT;
  if (lddy % 8 != 0 || ldx % 8 != 0 || !aligned_to(saved, 256) || !aligned_to(workspace, 256))
    return PRM_ERR_ALIGNMENT;
  const FfnSizes sz = sizes(tokens, d, f);
  if (workspace == nullptr || workspace_bytes < sz.bwd) return PRM_ERR_WORKSPACE;
  if (dx == nullptr && !weights) return PRM_OK;
  const BlockDevice* dev;
  if ((rc = block_device(&dev)) != PRM_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  void* dg = ws;
  void* du = ws + sz.bwd_du;
  const void* h = saved;

  FfnParams p{};
  p.err = dev->d_err;
  p.gu = reinterpret_cast<uint4*>(const_cast<char*>(static_cast<const char*>(saved)) + sz.saved_h);
  FfnSegment sg{};
  if (!encode(&sg.a[0], dy, dtype, tokens, d, lddy, MAP_ROWS) || !encode(&sg.b[0], w_down, dtype, d, f, f, MAP_COLS) ||
      !encode(&sg.out[0], dg, dtype, tokens, f, f, MAP_STORE) ||
      !encode(&sg.out[1], du, dtype, tokens, f, f, MAP_STORE))
    return PRM_ERR_CUDA;
  queue(p, sg, tokens, f, d, 0, false, true, BN);
  if (launch_act<EPI_DGLU>(p, act, dtype, dev->num_sms, st) != cudaSuccess) return PRM_ERR_CUDA;

  // dx (K = 2 f) and the weight gradients (K = tokens) from one queue, the
  // longer sums first, so that the last tiles of the queue are short.
  FfnParams q{};
  q.err = dev->d_err;
  bool ok = true;
  auto add_dx = [&] {
    if (dx == nullptr) return;
    FfnSegment s{};
    ok = ok && encode(&s.a[0], dg, dtype, tokens, f, f, MAP_ROWS) &&
         encode(&s.a[1], du, dtype, tokens, f, f, MAP_ROWS) &&
         encode(&s.b[0], w_gate, dtype, f, d, d, MAP_COLS) && encode(&s.b[1], w_up, dtype, f, d, d, MAP_COLS) &&
         encode(&s.out[0], dx, dtype, tokens, d, d, MAP_STORE);
    queue(q, s, tokens, d, f, f, false, true, BN);
  };
  auto add_weight = [&](const void* a, int64_t lda, int64_t m, const void* b, int64_t ldb, int64_t n, void* out) {
    FfnSegment s{};
    ok = ok && encode(&s.a[0], a, dtype, tokens, m, lda, MAP_COLS) &&
         encode(&s.b[0], b, dtype, tokens, n, ldb, MAP_COLS) && encode(&s.out[0], out, dtype, m, n, n, MAP_STORE);
    queue(q, s, m, n, tokens, 0, true, true, BN);
  };
  const bool dx_first = 2 * f >= tokens;
  if (dx_first) add_dx();
  if (weights) {
    add_weight(dg, f, f, x, ldx, d, dw_gate);
    add_weight(du, f, f, x, ldx, d, dw_up);
    add_weight(dy, lddy, d, h, f, f, dw_down);
  }
  if (!dx_first) add_dx();
  if (!ok) return PRM_ERR_CUDA;
  return launch<EPI_STORE>(q, dtype, dev->num_sms, st) == cudaSuccess ? PRM_OK : PRM_ERR_CUDA;
}
