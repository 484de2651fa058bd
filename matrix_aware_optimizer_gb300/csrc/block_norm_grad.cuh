// Backward pass of the norms around a transformer block. With n = (r - m_r) s_r,
// q = (z - m_z) s_z, P = q post (or z), and dr arriving from r's later uses:
//   dn  = dy (1 + scale_b) pre
//   D   = dr + s_r (dn - n mean(dn n) [- mean(dn)])         (gradient of r in all)
//   dx  = alpha D,   dP = gate_b D,   dq = dP post
//   dz  = s_z (dq - q mean(dq q) [- mean(dq)])              (dP without post)
//   dshift_b = sum dy, dscale_b = sum dy n pre, dgate_b = sum D P,
//   dpre = sum dy (1 + scale_b) n, dpost = sum dP q         (over rows)
// (within a sample dscale_b = pre sum dy n and its part of dpre is (1 +
// scale_b) sum dy n; so with D q, gate_b and post)
// the bracketed terms for the layer norm only. Bound by memory: dy, dr, r and
// z are read once, dx and dz written once.
//
// Persistent CTAs, each with a contiguous range of rows and a fixed thread
// per column, so the column sums stay in registers and need no atomics. Rows
// stream into a ring of shared-memory stages by bulk copies (rows are
// contiguous, so a stage of several short rows is still one copy per array);
// thread 0 fills it. The gains and the sample's scale and gate lie in shared
// memory in fp32. Where a sample ends inside a CTA's range the modulation
// sums are written out: to their place if the whole sample lies in the range,
// else as the range's first or last partial sum, which norm_join_kernel adds
// in order.
//
// Rows of any width and start come through the ring: a copy's ends are
// rounded to 16 bytes and the threads read strided elements (ELEM). Tensors
// that do not start on 16 bytes are read from memory by the threads (DIRECT).
//
// Measured (device time, share of the copy bandwidth on the bytes above):
// 32 x 1024 x 2048 modulated, fp32 stream and bf16 block, 195 us (92 %);
// 8191 x 5120 bf16 with both gains 112 us (66 %); 65536 x 512 bf16 89 us (67
// %); 30000 x 1001 bf16 155 us (34 %; 239 from a kernel compiled for every
// sum), 8000 x 4999 195 us (365); with gains and modulation 8 x 1024 x 2048 bf16
// 69 us (43 %), 8 x 1024 x 8192 fp32 / bf16 346 us (51 %), 8 x 1024 x 3001 bf16
// 284 us (15 %; 239 with five sums per row). What is left is the chain of each
// row -- load, reduce, reduce, store -- behind which only the rows of the
// other CTA of the SM, or the thread's second row, can hide: registers (40
// column sums and their operands per thread) allow no more of them. Fewer
// instructions helped most: packed pairs, two rows per thread and step
// (139 -> 110 us at 5120), values formed again rather than held.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_norm.cuh"

namespace prm {

constexpr int SUM_GATE = 0, SUM_SCALE = 1, SUM_SHIFT = 2, SUM_POST = 3, SUM_PRE = 4, SUM_COUNT = 5;
struct NormGradParams {
  NormParams n;
  int64_t sample_rows;   // rows that share modulation (all rows without any)
  int64_t ctas;
  int groups, stages;
  bool has[SUM_COUNT];
  float* partial_mod;    // [cta][first, last][gate, scale, shift][d]
  float* partial_w;      // [cta][post, pre][d]
  int* err;
};

__device__ __forceinline__ int64_t range_begin(const NormGradParams& p, int64_t cta) {
  return p.n.rows * cta / p.ctas;  // rows < 2^32, ctas <= 304
}

template <typename RT, typename BT>
struct NormGradIo {
  const BT* dy;
  const RT* dr;
  const RT* r;
  const BT* z;
  const float4* stats;
  RT* dx;
  BT* dz;
  BT* mod[3];   // dgate, dscale, dshift
};

__host__ __device__ constexpr bool grad_far(int size, bool mod, bool w) { return w && !mod && size == 2; }

// R: rows that a thread works on at once, to have more than one chain of
// dependent steps and to share what a step costs besides the arithmetic.
template <typename RT, typename BT, int SIZE, int R, int NV, int ACCESS, bool MOD, bool W>
__global__ void __launch_bounds__(norm_threads(SIZE), SIZE == 0 ? 2 : 1)
    norm_backward_kernel(const __grid_constant__ NormGradParams p, const NormGradIo<RT, BT> io) {
  constexpr bool RING = ACCESS != DIRECT;
  // n and q are formed again from the stage behind the reductions instead of held across them: registers.
  constexpr bool AGAIN = ACCESS == VEC;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float scratch[2][128];
  __shared__ uint64_t full_bar[MAX_STAGES], empty_bar[MAX_STAGES];
  __shared__ volatile int abort_flag;
  __shared__ volatile int row_failed[norm_threads(SIZE) / 64];  // [group of rows of more than a warp]
  const int tpr = p.n.tpr, d = p.n.d, groups = p.groups;
  const int threads = tpr * groups;
  const int step_rows = groups * R;
  const int64_t cta = blockIdx.x;
  // stage: rows of dy, dr, r, z and stats one after another (absent arrays
  // take no room, ELEM regions 16 bytes more on either side of 16-byte
  // rounding); after the ring what y's and z's columns are multiplied by for
  // the sample at work, pre (1 + scale) and post gate in fp32, then the groups'
  // exchange area
  const uint32_t slack = ACCESS == ELEM ? 32 : 0;
  auto region = [&](bool there, size_t size) -> uint32_t {
    return there ? ((static_cast<uint32_t>(step_rows * d * size) + slack) & ~15u) : 0u;
  };
  const uint32_t by = region(io.dy != nullptr, sizeof(BT)), bdr = region(io.dr != nullptr, sizeof(RT));
  const uint32_t br = region(io.dy != nullptr, sizeof(RT)), bz = region(io.z != nullptr, sizeof(BT));
  const uint32_t stage_bytes = by + bdr + br + bz + (io.stats ? static_cast<uint32_t>(step_rows) * 16 : 0);
  float* const columns = reinterpret_cast<float*>(smem + p.stages * stage_bytes);
  const int pitch = (d + 3) & ~3;
  float* const col_y = columns;
  float* const col_z = columns + pitch;
  uint64_t* const exchange = reinterpret_cast<uint64_t*>(columns + (W || MOD ? 2 : 0) * pitch);
  // With long rows a thread's gain sums lie in shared memory, where only it
  // touches them: registers are short. With both kinds of sums a row adds to
  // three (dy n, D q and dy); the gains' and the modulation's are formed from
  // them at a sample's end, the gains' in the CTA's row of partial sums.
  constexpr bool FAR = grad_far(SIZE, MOD, W);
  uint64_t* const far_w = exchange + (groups > 1 ? 4 * NV * threads : 0) + threadIdx.x;
  if constexpr (RING) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], threads / 32);
      }
      abort_flag = 0;
      fence_mbar_init();
    }
    if (threadIdx.x < norm_threads(SIZE) / 64) row_failed[threadIdx.x] = -1;
    __syncthreads();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row0 = range_begin(p, cta), row1 = range_begin(p, cta + 1);
  const int64_t all = p.n.rows * d;

  // The ring is filled by thread 0: every stage at first, then one stage per
  // step, when every warp has left the stage before.
  // (Its state lies in shared memory: the other threads need the registers.)
  __shared__ struct {
    int64_t row, sample_end;
    int stage;
    uint32_t phase, issued, parity;
  } fill;
  if (RING && threadIdx.x == 0) {
    fill.row = row0;
    fill.sample_end = (row0 / p.sample_rows + 1) * p.sample_rows;
    fill.stage = 0;
    fill.phase = fill.issued = fill.parity = 0;
  }
  auto refill = [&] {
    if (fill.row >= row1 || abort_flag) return;
    const int64_t stop = min(row1, fill.sample_end);
    const uint32_t n = static_cast<uint32_t>(min(static_cast<int64_t>(step_rows), stop - fill.row));
    if (!wait_bounded(&empty_bar[fill.stage], fill.phase ^ 1u, &abort_flag, p.err, NORM_WAIT_NS)) return;
    uint8_t* dst = smem + fill.stage * stage_bytes;
    uint64_t* bar = &full_bar[fill.stage];
    const uint32_t nd = n * static_cast<uint32_t>(d);
    const int64_t at = fill.row * d;
    if constexpr (ACCESS == ELEM) {
      const uint32_t ny = io.dy ? ring_bytes(io.dy + at, nd, io.dy + all) : 0u;
      const uint32_t nr = io.dy ? ring_bytes(io.r + at, nd, io.r + all) : 0u;
      const uint32_t ndr = io.dr ? ring_bytes(io.dr + at, nd, io.dr + all) : 0u;
      const uint32_t nz = io.z ? ring_bytes(io.z + at, nd, io.z + all) : 0u;
      if (all - at - nd < 8) {  // less than 16 bytes of a tensor behind these rows: its end
        if (io.dy) {
          ring_tail(dst, io.dy + at, nd, io.dy + all);
          ring_tail(dst + by + bdr, io.r + at, nd, io.r + all);
        }
        if (io.dr) ring_tail(dst + by, io.dr + at, nd, io.dr + all);
        if (io.z) ring_tail(dst + by + bdr + br, io.z + at, nd, io.z + all);
      }
      mbar_arrive_expect_tx(bar, ny + nr + ndr + nz + (io.stats ? n * 16 : 0u));
      if (io.dy) {
        ring_load(dst, io.dy + at, ny, bar);
        ring_load(dst + by + bdr, io.r + at, nr, bar);
      }
      if (io.dr) ring_load(dst + by, io.dr + at, ndr, bar);
      if (io.z) ring_load(dst + by + bdr + br, io.z + at, nz, bar);
    } else {
      mbar_arrive_expect_tx(bar, (io.dy ? nd * (sizeof(BT) + sizeof(RT)) : 0u) + (io.dr ? nd * sizeof(RT) : 0u) +
                                     (io.z ? nd * sizeof(BT) : 0u) + (io.stats ? n * 16 : 0u));
      if (io.dy) {
        bulk_load(dst, io.dy + at, nd * sizeof(BT), bar);
        bulk_load(dst + by + bdr, io.r + at, nd * sizeof(RT), bar);
      }
      if (io.dr) bulk_load(dst + by, io.dr + at, nd * sizeof(RT), bar);
      if (io.z) bulk_load(dst + by + bdr + br, io.z + at, nd * sizeof(BT), bar);
    }
    if (io.stats) bulk_load(dst + by + bdr + br + bz, io.stats + fill.row, n * 16, bar);
    fill.issued |= 1u << fill.stage;
    fill.parity = (fill.parity & ~(1u << fill.stage)) | (fill.phase << fill.stage);
    fill.row += n;
    if (fill.row == fill.sample_end) fill.sample_end += p.sample_rows;
    if (++fill.stage == p.stages) {
      fill.stage = 0;
      fill.phase ^= 1u;
    }
  };
  if (RING && threadIdx.x == 0)
    for (int s = 0; s < p.stages; ++s) refill();
  const bool post = W && p.n.post != nullptr;
  const bool pre = W && p.n.pre != nullptr;
  const bool scale = MOD && p.has[SUM_SCALE];
  const bool shift = MOD && p.has[SUM_SHIFT];
  const bool gate = MOD && p.has[SUM_GATE];
  auto fill_columns = [&](int64_t sample) {
    const BT* const sc = static_cast<const BT*>(p.n.scale) + sample * p.n.scale_ld;
    const BT* const g = static_cast<const BT*>(p.n.gate) + sample * p.n.gate_ld;
    for (int i = threadIdx.x; i < d; i += threads) {
      if (pre || scale) col_y[i] = (pre ? __ldg(p.n.pre + i) : 1.f) * (scale ? 1.f + to_f32(sc[i]) : 1.f);
      if (post || gate) col_z[i] = (post ? __ldg(p.n.post + i) : 1.f) * (gate ? to_f32(g[i]) : 1.f);
    }
  };
  if constexpr (W && !MOD) fill_columns(0);

  const int tid = tpr <= 32 ? threadIdx.x & (tpr - 1) : threadIdx.x % tpr;
  const int group = threadIdx.x / tpr;
  const int lane = threadIdx.x & 31;
  int col[NV], left[NV];  // first element of each of this thread's vectors, elements from there on
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = ACCESS == VEC ? (v * tpr + tid) * 8 : v * 8 * tpr + tid;
    left[v] = d - col[v];
  }
  int turn = 0;
  auto reduce = [&](float (&a)[R][2]) { row_sums<SIZE, R>(a, tpr, group, scratch, turn); };
  F8 acc_mod[MOD ? 3 : 1][NV], acc_w[W && !MOD && !FAR ? 2 : 1][NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int k = 0; k < (MOD ? 3 : 1); ++k) acc_mod[k][v] = f8_zero();
#pragma unroll
    for (int k = 0; k < (W && !MOD && !FAR ? 2 : 1); ++k) acc_w[k][v] = f8_zero();
  }
  if constexpr (FAR) {
#pragma unroll
    for (int k = 0; k < 8 * NV; ++k) far_w[k * threads] = 0;
  }
  auto gain_sums = [&](int which, int v) {
    return p.partial_w + (cta * 2 + which) * static_cast<int64_t>(pitch) + col[v];
  };
  if constexpr (W && MOD) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (group != 0 || left[v] <= 0) continue;
      if (post) write8<ACCESS>(gain_sums(0, v), left[v], tpr, f8_zero());
      if (pre) write8<ACCESS>(gain_sums(1, v), left[v], tpr, f8_zero());
    }
  }
  // acc_w[which][v] += a b (0: post, 1: pre)
  auto add_w = [&](int which, int v, const F8& a, const F8& b) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (FAR) {
        uint64_t& x = far_w[((which * NV + v) * 4 + k) * threads];
        x = f2_fma(a.p[k], b.p[k], x);
      } else if constexpr (W && !MOD) {
        acc_w[which][v].p[k] = f2_fma(a.p[k], b.p[k], acc_w[which][v].p[k]);
      }
    }
  };
  // Adds a column sum over the CTA's row groups and hands group 0's threads
  // the total.
  auto across_groups = [&](F8(&acc)[NV]) {
    if (groups == 1) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k) exchange[(v * 4 + k) * threads + threadIdx.x] = acc[v].p[k];
    __syncthreads();
    if (group == 0) {
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[v].p[k] = f2_add(acc[v].p[k], exchange[(v * 4 + k) * threads + g * tpr + tid]);
    }
    __syncthreads();
  };

  int stage = 0;
  uint32_t phase = 0;
  // A warp whose wait gave up must not leave the other warps of its row, which
  // may have got their stage, at a barrier that has no time limit. It names the
  // step in its row's word and goes on to the step's reductions. Behind their
  // barrier the whole row finds the abort flag up, and that step named, and
  // leaves together at the next one. A row that is dead in a sample's last step
  // meets the CTA at the next sample's start. The CTA's barriers do not wait for
  // threads that have exited, and a step without reductions meets nobody. (At 32 x
  // 1024 x 2048 modulated and 8 x 1024 x 8192 with gains and modulation, us: this
  // 195 and 346; a vote at the reductions' barrier 200 and 373; a test behind it
  // 202 and 346; going on to the end without leaving 191 and 392.)
  bool leave = false;
  // The CTA's rows, sample by sample.
  for (int64_t seg0 = row0; seg0 < row1 && !leave;) {
    const int64_t sample = seg0 / p.sample_rows;
    const int64_t seg1 = min(row1, (sample + 1) * p.sample_rows);
    if constexpr (MOD) {
      // the sample before is done with its columns
      if constexpr (RING) leave = __syncthreads_or(abort_flag);
      else __syncthreads();
      if (leave) break;
      fill_columns(sample);
    }
    if constexpr (MOD || W) __syncthreads();
    const int count = static_cast<int>(seg1 - seg0);  // below 2^31: checked by the host
    // start of this group's first row of the step
    int64_t at0 = (seg0 + group * R) * d;
    for (int base = 0; base < count; base += step_rows, at0 += static_cast<int64_t>(step_rows) * d) {
      const int mine = count - base - group * R;  // rows of this step from this group's first one on
      if constexpr (RING) {
        if (threadIdx.x == 0 && seg0 + base != row0) refill();
        const bool aborted = abort_flag != 0;
        const bool got = wait_bounded(&full_bar[stage], phase, &abort_flag, p.err, NORM_WAIT_NS);
        if (!__all_sync(0xffffffffu, got && !aborted)) {
          const int first = stage == 0, p0 = static_cast<int>(phase);
          const int before = 2 * (first ? p.stages - 1 : stage - 1) + (p0 ^ first);  // the step before
          leave = (SIZE == 0 && tpr <= 32) || row_failed[group] == before;  // (or the row lies in this warp)
          if (leave) break;
          row_failed[group] = 2 * stage + p0;
        }
      }
      const uint8_t* src = smem + stage * stage_bytes;
      const int in_step = group * R * d;
      // A vector outside the row, or of a dead row, is skipped and adds
      // nothing; the warps of long rows that are all dead skip everything.
      if ((SIZE == 0 && tpr <= 32) || mine > 0) {
        bool live[R][NV];
        float4 st[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
          for (int v = 0; v < NV; ++v) live[i][v] = left[v] > 0 && i < mine;
          st[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (io.stats != nullptr && i < mine) {
            if constexpr (RING)
              st[i] = reinterpret_cast<const float4*>(src + by + bdr + br + bz)[group * R + i];
            else
              st[i] = __ldg(io.stats + seg0 + base + group * R + i);
          }
        }
        // Vector v of row i of array `a`, whose stage region starts at `off`.
        auto row8 = [&](auto* a, uint32_t off, int i, int v) -> F8 {
          using T = std::remove_const_t<std::remove_pointer_t<decltype(a)>>;
          if constexpr (ACCESS == VEC)
            return load_f8(reinterpret_cast<const T*>(src + off) + in_step + i * d + col[v]);
          else if constexpr (ACCESS == ELEM)
            return gather_f8(reinterpret_cast<const T*>(src + off + ring_offset(a + (seg0 + base) * d)) + in_step +
                                 i * d + col[v],
                             left[v], tpr);
          else
            return gather_f8(a + at0 + i * d + col[v], left[v], tpr);
        };
        // (r - m_r) s_r, and (z - m_z) s_z where z is normed
        auto normed_r = [&](int i, int v) -> F8 {
          F8 n = row8(io.r, by + bdr, i, v);
          const float s0 = -st[i].x * st[i].y;
          const uint64_t mul = f2_pack(st[i].y, st[i].y), add = f2_pack(s0, s0);
#pragma unroll
          for (int k = 0; k < 4; ++k) n.p[k] = f2_fma(n.p[k], mul, add);
          return n;
        };
        auto normed_z = [&](int i, int v) -> F8 {
          F8 q = row8(io.z, by + bdr + br, i, v);
          if (post) {
            const float s0 = -st[i].z * st[i].w;
            const uint64_t mul = f2_pack(st[i].w, st[i].w), add = f2_pack(s0, s0);
#pragma unroll
            for (int k = 0; k < 4; ++k) q.p[k] = f2_fma(q.p[k], mul, add);
          }
          return q;
        };
        F8 D[R][NV];
        float sums[R][2];
        uint64_t part[R][2];
        if (io.dy != nullptr) {
          F8 nn[AGAIN ? 1 : R][NV];
#pragma unroll
          for (int i = 0; i < R; ++i) part[i][0] = part[i][1] = 0;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            F8 w;
            if ((pre || scale) && left[v] > 0) w = read8<ACCESS>(col_y + col[v], left[v], tpr);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              if (!live[i][v]) continue;
              F8 x = row8(io.dy, 0, i, v);
              const F8 n = normed_r(i, v);
              if constexpr (MOD) {
                if (shift) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) acc_mod[SUM_SHIFT][v].p[k] = f2_add(acc_mod[SUM_SHIFT][v].p[k], x.p[k]);
                }
                if (scale || pre) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    acc_mod[SUM_SCALE][v].p[k] = f2_fma(x.p[k], n.p[k], acc_mod[SUM_SCALE][v].p[k]);
                }
              }
              if (pre || scale) {
                if constexpr (!MOD) add_w(1, v, x, n);
#pragma unroll
                for (int k = 0; k < 4; ++k) x.p[k] = f2_mul(x.p[k], w.p[k]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                part[i][0] = f2_fma(x.p[k], n.p[k], part[i][0]);
                part[i][1] = f2_add(part[i][1], x.p[k]);
              }
              D[i][v] = x;
              if constexpr (!AGAIN) nn[i][v] = n;
            }
          }
          join_halves(part, sums);
          reduce(sums);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float m1 = -sums[i][0] * p.n.inv_d * st[i].y;
            const float m2 = p.n.layer ? -sums[i][1] * p.n.inv_d * st[i].y : 0.f;
            const uint64_t M1 = f2_pack(m1, m1), M2 = f2_pack(m2, m2), S = f2_pack(st[i].y, st[i].y);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (!live[i][v]) continue;
              F8 x = f8_zero();
              if (io.dr != nullptr) x = row8(io.dr, by, i, v);
              F8 n;
              if constexpr (AGAIN) n = normed_r(i, v);
              else n = nn[i][v];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x.p[k] = f2_fma(n.p[k], M1, x.p[k]);
                if (p.n.layer) x.p[k] = f2_add(x.p[k], M2);
                D[i][v].p[k] = f2_fma(S, D[i][v].p[k], x.p[k]);
              }
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int v = 0; v < NV; ++v)
              if (live[i][v]) D[i][v] = row8(io.dr, by, i, v);
        }
        if (io.dx != nullptr) {
          const uint64_t alpha = f2_pack(p.n.alpha, p.n.alpha);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              if (!live[i][v]) continue;
              F8 o;
#pragma unroll
              for (int k = 0; k < 4; ++k) o.p[k] = f2_mul(alpha, D[i][v].p[k]);
              write8<ACCESS>(io.dx + at0 + i * d + col[v], left[v], tpr, o);
            }
        }
        if (io.z != nullptr) {
          F8 q[AGAIN ? 1 : R][NV];
          if (post || gate) {
#pragma unroll
            for (int i = 0; i < R; ++i) part[i][0] = part[i][1] = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              F8 w;
              if (left[v] > 0) w = read8<ACCESS>(col_z + col[v], left[v], tpr);
#pragma unroll
              for (int i = 0; i < R; ++i) {
                if (!live[i][v]) continue;
                const F8 x = normed_z(i, v);
                if constexpr (MOD) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    acc_mod[SUM_GATE][v].p[k] = f2_fma(D[i][v].p[k], x.p[k], acc_mod[SUM_GATE][v].p[k]);
                } else {
                  add_w(0, v, D[i][v], x);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  D[i][v].p[k] = f2_mul(D[i][v].p[k], w.p[k]);
                  part[i][0] = f2_fma(D[i][v].p[k], x.p[k], part[i][0]);
                  part[i][1] = f2_add(part[i][1], D[i][v].p[k]);
                }
                if constexpr (!AGAIN) q[i][v] = x;
              }
            }
          }
          if (post) {
            join_halves(part, sums);
            reduce(sums);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float m1 = -sums[i][0] * p.n.inv_d * st[i].w;
              const float m2 = p.n.layer ? -sums[i][1] * p.n.inv_d * st[i].w : 0.f;
              const uint64_t M1 = f2_pack(m1, m1), M2 = f2_pack(m2, m2), S = f2_pack(st[i].w, st[i].w);
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                if (!live[i][v]) continue;
                F8 x;
                if constexpr (AGAIN) x = normed_z(i, v);
                else x = q[i][v];
#pragma unroll
                for (int k = 0; k < 4; ++k) D[i][v].p[k] = f2_fma(S, D[i][v].p[k], f2_fma(x.p[k], M1, M2));
              }
            }
          }
          if (io.dz != nullptr) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
              for (int v = 0; v < NV; ++v)
                if (live[i][v]) write8<ACCESS>(io.dz + at0 + i * d + col[v], left[v], tpr, D[i][v]);
          }
        }
      }
      if constexpr (RING) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_bar[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (leave) break;
    if constexpr (MOD) {
      // the end of the sample, or of this CTA's part of it
      const bool before = sample * p.sample_rows < row0, after = (sample + 1) * p.sample_rows > row1;
      // what a sum is of a gain's gradient, and then the modulation's
      auto share = [&](int which, int v, F8& sum, const void* mods, int64_t ld, float plus, const float* gains) {
        const uint64_t add = f2_pack(plus, plus);
        F8 m = {{f2_pack(1.f, 1.f), f2_pack(1.f, 1.f), f2_pack(1.f, 1.f), f2_pack(1.f, 1.f)}};
        if (mods != nullptr) {
          m = read8<ACCESS>(static_cast<const BT*>(mods) + sample * ld + col[v], left[v], tpr);
#pragma unroll
          for (int k = 0; k < 4; ++k) m.p[k] = f2_add(m.p[k], add);
        }
        float* const at = gain_sums(which, v);
        F8 t = read8<ACCESS>(at, left[v], tpr);
        const F8 w = read8<ACCESS>(gains + col[v], left[v], tpr);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          t.p[k] = f2_fma(sum.p[k], m.p[k], t.p[k]);
          sum.p[k] = f2_mul(sum.p[k], w.p[k]);
        }
        write8<ACCESS>(at, left[v], tpr, t);
      };
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const bool gain = (k == SUM_GATE && post) || (k == SUM_SCALE && pre);
        if (!p.has[k] && !gain) continue;
        across_groups(acc_mod[k]);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (W && gain && group == 0 && left[v] > 0) {
            if (k == SUM_GATE) share(0, v, acc_mod[k][v], p.n.gate, p.n.gate_ld, 0.f, p.n.post);
            else share(1, v, acc_mod[k][v], p.n.scale, p.n.scale_ld, 1.f, p.n.pre);
          }
          if (p.has[k] && group == 0 && left[v] > 0) {
            if (before || after)
              write8<ACCESS>(
                  p.partial_mod + ((cta * 2 + (before ? 0 : 1)) * 3 + k) * static_cast<int64_t>(pitch) + col[v],
                  left[v], tpr, acc_mod[k][v]);
            else
              write8<ACCESS>(io.mod[k] + sample * d + col[v], left[v], tpr, acc_mod[k][v]);
          }
          acc_mod[k][v] = f8_zero();
        }
      }
    }
    seg0 = seg1;
  }
  if (RING && threadIdx.x == 0 && abort_flag) {
    // a wait gave up: let the copies in flight land before the CTA exits
    for (int s = 0; s < p.stages; ++s)
      if (fill.issued & (1u << s)) wait_drain(&full_bar[s], (fill.parity >> s) & 1u, 50000000ull);
  }
  if (leave) return;
  if constexpr (W && !MOD) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!p.has[SUM_POST + k]) continue;
      F8 total[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (FAR) {
#pragma unroll
          for (int j = 0; j < 4; ++j) total[v].p[j] = far_w[((k * NV + v) * 4 + j) * threads];
        } else {
          total[v] = acc_w[k][v];
        }
      }
      across_groups(total);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (group == 0 && left[v] > 0)
          write8<ACCESS>(gain_sums(k, v), left[v], tpr, total[v]);
    }
  }
}

// out[row][column] = sum of partial sums, in CTA order. The first
// (ctas - 1) x ceil(d / 256) blocks look after the samples that cross CTA
// ranges: the one for range c takes the sample, if any, that began in range
// c - 1 and goes on into c, and adds its partial sums, a thread per column
// (a sample inside one range is complete already). The others add the gains'
// partial sums of all CTAs, 32 columns a block: each of 8 warps adds every
// eighth, and warp 0 adds their totals.
template <typename BT>
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormGradParams p, BT* dgate, BT* dscale,
                                                        BT* dshift, float* dpost, float* dpre, int mod_blocks) {
  __shared__ float part[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t d = p.n.d, pitch = (d + 3) & ~int64_t(3);
  if (static_cast<int>(blockIdx.x) < mod_blocks) {
    const int wide = static_cast<int>((d + 255) / 256);
    const int64_t c = 1 + blockIdx.x / wide;
    const int64_t row = range_begin(p, c);
    const int64_t sample = row / p.sample_rows;
    const int64_t begin = sample * p.sample_rows, end = begin + p.sample_rows;
    const int64_t col = static_cast<int64_t>(blockIdx.x % wide) * 256 + threadIdx.x;
    if (row == begin || range_begin(p, c - 1) > begin || col >= d) return;
    BT* const out[3] = {dgate, dscale, dshift};
    float s[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = p.has[k] ? p.partial_mod[((c - 1) * 6 + 3 + k) * pitch + col] : 0.f;
    // the last range that holds a row of the sample: range i begins at floor(rows i / ctas)
    const int last = static_cast<int>((end * p.ctas - 1) / p.n.rows);
    const float* from = p.partial_mod + col;
#pragma unroll 8
    for (int i = static_cast<int>(c); i <= last; ++i) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (p.has[k]) s[k] += from[(i * 6 + k) * pitch];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (p.has[k]) out[k][sample * d + col] = from_f32<BT>(s[k]);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int job = static_cast<int>(blockIdx.x) - mod_blocks;
  const int tiles = static_cast<int>((d + 31) / 32);
  const int k = job / tiles;  // 0: post, 1: pre
  const int64_t col = static_cast<int64_t>(job - k * tiles) * 32 + lane;
  if (!p.has[SUM_POST + k]) return;
  const float* from = p.partial_w + k * pitch + col;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int64_t i = warp; i < p.ctas; i += 8) s += from[i * 2 * pitch];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= d) return;
  for (int w = 1; w < 8; ++w) s += part[w][lane];
  (k == 0 ? dpost : dpre)[col] = s;
}

struct NormGradArgs {
  const void *dy, *dr, *r, *z;
  const float* stats;
  void *dx, *dz;
  float* dpost;
  void* dgate;
  float* dpre;
  void *dscale, *dshift;
};

// Shared memory behind the ring of a kernel with these sums: the columns'
// arrays, the groups' exchange area, the gain sums that lie there.
inline NormShape grad_shape(int64_t d, size_t row_bytes, int arrays, bool vec, bool ring, bool w, bool mod) {
  return norm_shape(d, row_bytes, arrays, vec, ring, [&](int size, int threads, int groups, bool direct) {
    const bool ww = w || direct, mm = mod || direct;  // the direct kernel is compiled for every sum
    const int nv = norm_vectors(size);
    return (ww || mm ? 2 : 0) * ((d + 3) & ~int64_t(3)) * sizeof(float) +
           (groups > 1 ? static_cast<size_t>(threads) * 8 * nv * sizeof(float) : 0) +
           (grad_far(size, mm, ww) ? static_cast<size_t>(threads) * 16 * nv * sizeof(float) : 0);
  });
}

inline size_t row_bytes(const prm_block_norm_desc& c, bool dy, bool dr, bool z, bool stats) {
  const size_t rb = dtype_bytes(c.stream_dtype) * c.d, bb = dtype_bytes(c.block_dtype) * c.d;
  return (dy ? rb + bb : 0) + (dr ? rb : 0) + (z ? bb : 0) + (stats ? 16 : 0);
}

template <typename RT, typename BT, int SIZE, int R, int NV, int ACCESS, bool MOD, bool W>
cudaError_t launch_backward(NormGradParams& p, const NormShape& s, const NormGradArgs& a, cudaStream_t stream) {
  auto kernel = norm_backward_kernel<RT, BT, SIZE, R, NV, ACCESS, MOD, W>;
  static std::atomic<bool> set[64];
  cudaError_t e = norm_setup(kernel, set);
  if (e != cudaSuccess) return e;
  const NormGradIo<RT, BT> io{static_cast<const BT*>(a.dy), static_cast<const RT*>(a.dr), static_cast<const RT*>(a.r),
                              static_cast<const BT*>(a.z), reinterpret_cast<const float4*>(a.stats),
                              static_cast<RT*>(a.dx), static_cast<BT*>(a.dz),
                              {static_cast<BT*>(a.dgate), static_cast<BT*>(a.dscale), static_cast<BT*>(a.dshift)}};
  e = launch_dependent(kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(s.threads), s.smem, stream, p, io);
  if (e != cudaSuccess) return e;
  const bool mods = MOD && (p.has[SUM_GATE] || p.has[SUM_SCALE] || p.has[SUM_SHIFT]);
  const int d = p.n.d;
  const int mod_blocks = mods ? static_cast<int>(p.ctas - 1) * ((d + 255) / 256) : 0;
  const int w_blocks = W && (p.has[SUM_POST] || p.has[SUM_PRE]) ? 2 * ((d + 31) / 32) : 0;
  if (mod_blocks + w_blocks == 0) return cudaSuccess;
  return launch_dependent(norm_join_kernel<BT>, dim3(mod_blocks + w_blocks), dim3(256), 0, stream, p, io.mod[0],
                          io.mod[1], io.mod[2], a.dpost, a.dpre, mod_blocks);
}

template <typename RT, typename BT>
cudaError_t launch_shape(NormGradParams& p, const NormShape& s, const NormGradArgs& a, cudaStream_t stream) {
  const bool mod = p.has[SUM_GATE] || p.has[SUM_SCALE] || p.has[SUM_SHIFT];
  const bool w = p.has[SUM_POST] || p.has[SUM_PRE];
  using std::integral_constant;
  auto sums = [&](auto size, auto rows, auto access) {
    constexpr int S = decltype(size)::value, R = decltype(rows)::value, V = norm_vectors(S), A = decltype(access)::value;
    if (mod && w) return launch_backward<RT, BT, S, R, V, A, true, true>(p, s, a, stream);
    if (mod) return launch_backward<RT, BT, S, R, V, A, true, false>(p, s, a, stream);
    if (w) return launch_backward<RT, BT, S, R, V, A, false, true>(p, s, a, stream);
    return launch_backward<RT, BT, S, R, V, A, false, false>(p, s, a, stream);
  };
  const integral_constant<int, 0> small;
  const integral_constant<int, 1> one;  // (also the size of the rows in between)
  const integral_constant<int, 2> two;
  if (s.access == VEC) {
    const integral_constant<int, VEC> vec;
    if (s.size == 2) return sums(two, one, vec);
    if (s.size == 1) return s.rows == 2 ? sums(one, two, vec) : sums(one, one, vec);
    return s.rows == 2 ? sums(small, two, vec) : sums(small, one, vec);
  }
  if (s.access == ELEM) {
    const integral_constant<int, ELEM> elem;
    return s.size == 0 ? sums(small, one, elem) : s.size == 1 ? sums(one, one, elem) : sums(two, one, elem);
  }
  // DIRECT: compiled for every sum
  if (s.size == 0) return launch_backward<RT, BT, 0, 1, norm_vectors(0), DIRECT, true, true>(p, s, a, stream);
  if (s.size == 1) return launch_backward<RT, BT, 1, 1, norm_vectors(1), DIRECT, true, true>(p, s, a, stream);
  return launch_backward<RT, BT, 2, 1, norm_vectors(2), DIRECT, true, true>(p, s, a, stream);
}

// Defined per pair of types, each pair's kernels in a translation unit of a
// few (norm_grad_*.cu) to keep the build parallel.
template <typename RT, typename BT>
cudaError_t norm_grad_launch(NormGradParams& p, const NormShape& s, const NormGradArgs& a, cudaStream_t stream);

}  // namespace prm
