// Matrix product with bias, activation and residual on the tensor cores.
//
// y = act(x W + bias) + residual, x [M][K] bf16 (K-major), W [K][N] bf16 read
// as it lies (MN-major), fp32 accumulation in TMEM.
//
// A pair of CTAs on neighbouring SMs owns a 256 x 256 (or 256 x 128) tile (cta_group::2: the
// leader issues M = 256 MMAs; each CTA stages its 128 rows of x and 128 of the
// 256 columns of W, so an operand byte in shared memory feeds both tensor
// cores) and is persistent.  Per CTA: five stages of 32 KB (K = 64), and
//   warp 0     TMA producer; both CTAs' copies complete on the leader's barrier;
//   warp 1     (leader) MMA issuer; commits release the stage in both CTAs;
//   warps 2-9  epilogue, two 256-column accumulators in turn: TMEM -> bias,
//              activation, residual -> one 32-row, 64-byte-wide swizzled block
//              of the warp's four -> TMA store.  The residual's block comes
//              into the same buffers by TMA, four blocks at a time while the
//              MMAs fill the tile's accumulator; the accumulator and the bias
//              are read one block ahead.
// 16384 x 2048 x 8192 bf16 with bias and GELU: 338 us = 1.63 PFLOP/s, 93-95 % of
// the plain library product under the same power cap; a stage's MMAs take 515-525
// cycles of an ideal 512, tensor pipe 90 % active over the whole launch.  Smaller
// calls lose to the number of tiles: 16384 x 768 x 768 has 2.5 rounds of 76.
// Where y or the residual cannot be a TMA operand (row stride or address not on
// 16 bytes) the block leaves by coalesced element stores instead.
//
// fp32 inputs: x and W as three bf16 planes each (x = x0 + x1 + x2 exactly,
// 24 bits), six products x0 W0, x0 W1, x1 W0, x0 W2, x2 W0, x1 W1 into one
// accumulator; the dropped ones are below 2^-23 of the sum of |x W|.
#include <algorithm>
#include <type_traits>

#include "linear_common.cuh"
#include "tc2.cuh"

using layer::bf16;

namespace {

constexpr int BM = 256, BK = 64, EPI_WARPS = 8, NTHR = 64 + 32 * EPI_WARPS;
constexpr int BLK_BYTES = 32 * 64;                               // one epilogue block
constexpr int NBUF = 4;                                          // epilogue blocks per warp
template <int BN>
struct Cfg {
  static constexpr int A_BYTES = BM / 2 * BK * 2, B_BYTES = BN / 2 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 5 * 256 / (128 + BN / 2);        // 160 KB of stages: 5, or 6 for BN = 128
  static constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * NBUF * BLK_BYTES + 1024;
  static constexpr int HALF = BN / 2;                            // columns per epilogue warp
};
constexpr int BAND = 16;                                         // row tiles per band of the tile order

struct Params {
  int M, N, nk, kc, planes, kw;   // nk: blocks of 64 of K per plane, kc of them per pass; kw: W rows per plane
  int act;
  int kper, split_rows;     // K split: blocks of 64 per split (nk: no split), rows of y per split
  const float* bias;
  const void* residual;
  void* y;
  int tma_out;                // y (and the residual) go by TMA
  int* status;
};

// plane pairs of the six products, the smallest first
__device__ __forceinline__ void plane_pair(int i, int& a, int& b) {
  // (1,1) (0,2) (2,0) (0,1) (1,0) (0,0), one nibble each
  const uint32_t pa = 0x010201u, pb = 0x001021u;
  a = (pa >> (4 * i)) & 0xF;
  b = (pb >> (4 * i)) & 0xF;
}

struct Tile {
  int m0, n0;
};
template <int BN>
__device__ __forceinline__ Tile tile_at(int t, int ntm, int ntn) {
  const int width = BAND * ntn, first = t / width * BAND, h = min(BAND, ntm - first), r = t % width;
  return {(first + r % h) * BM, r / h * BN};
}

// SUM: K in passes, added up in the epilogue's registers (blocks_per_pass); else
// the whole of K (of a split) in one accumulator.
template <typename TO, int BN, bool SUM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHR, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_y, Params p) {
  using Q = Cfg<BN>;
  constexpr int STAGES = Q::STAGES, STAGE_BYTES = Q::STAGE_BYTES, A_BYTES = Q::A_BYTES, HALF = Q::HALF;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint8_t* blocks = sm + STAGES * STAGE_BYTES;
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], res_full[EPI_WARPS];
  __shared__ uint32_t tbase;
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = tc::cluster_rank();
  const int ntm = (p.M + BM - 1) / BM, ntn = (p.N + BN - 1) / BN, nmn = ntm * ntn;
  const int ntiles = nmn * ((p.nk + p.kper - 1) / p.kper);   // a split's tiles, then the next split's
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int pairs = p.planes == 1 ? 1 : 6;

  if (warp == 0) tc::tmem_alloc_pair(&tbase, 2 * BN);
  if (tid == 32) {
    tc::prefetch_map(&map_x);
    tc::prefetch_map(&map_w);
    if (p.tma_out) tc::prefetch_map(&map_y);
    if (p.tma_out && p.residual) tc::prefetch_map(&map_r);
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init_only(&full[s], 1);
      tc::mbar_init_only(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init_only(&acc_full[a], 1);
      tc::mbar_init_only(&acc_empty[a], 2 * EPI_WARPS);   // every epilogue warp of both CTAs
    }
    for (int w = 0; w < EPI_WARPS; ++w)
      tc::mbar_init_only(&res_full[w], 1);
    tc::mbar_init_fence();
    failed = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tacc = tbase;
  tc::grid_dependency_wait();   // nothing above touched global memory
  tc::grid_dependents_launch();

  // a ring slot: s counts through the stages, ph flips with every turn
  if (warp == 0) {
    const uint32_t ring = tc::smem_u32(sm), bfull = tc::smem_u32(full), bempty = tc::smem_u32(empty);
    const uint32_t lead = tc::map_rank(full, 0);   // the leader's barriers
    uint32_t s = 0, ph = 1;                                  // the first turn finds its slots free
    bool ok = true;
    for (int t = first; t < ntiles && ok; t += step) {
      const Tile tl = tile_at<BN>(t % nmn, ntm, ntn);
      const int m0 = tl.m0 + (int)rank * (BM / 2), n0 = tl.n0 + (int)rank * (BN / 2);
      const int k_lo = t / nmn * p.kper, k_hi = min(p.nk, k_lo + p.kper);
      for (int k0 = k_lo; k0 < k_hi && ok; k0 += p.kc) {
        const int k1 = min(k_hi, k0 + p.kc);
        for (int pr = 0; pr < pairs && ok; ++pr) {
          int row_x = m0, row_w = 0;
          if (pairs > 1) {
            int pa, pb;
            plane_pair(pr, pa, pb);
            row_x += pa * p.M;
            row_w = pb * p.kw;
          }
          for (int kt = k0; kt < k1; ++kt) {
            if (!(ok = __all_sync(0xffffffffu, tc::wait(bempty + 8 * s, ph)))) break;
            if (tc::elect()) {
              const uint32_t a = ring + s * STAGE_BYTES, b = a + A_BYTES, bar = lead + 8 * s;
              if (rank == 0) tc::expect_tx(bfull + 8 * s, 2 * STAGE_BYTES);
              tc::tma_load_2d_pair(a, &map_x, kt * BK, row_x, bar);
#pragma unroll
              for (int i = 0; i < HALF / 64; ++i)
                tc::tma_load_2d_pair(b + i * 8192, &map_w, n0 + 64 * i, row_w + kt * BK, bar);
            }
            __syncwarp();
            if (++s == STAGES) s = 0, ph ^= 1;
          }
        }
      }
    }
    // the commits behind the last stages arrive in both CTAs: none leaves before
    for (int i = 0; i < STAGES && ok; ++i) {
      ok = __all_sync(0xffffffffu, tc::wait(bempty + 8 * s, ph));
      if (++s == STAGES) s = 0, ph ^= 1;
    }
    if (!ok && lane == 0) atomicExch(&failed, 1);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = tc::idesc_f16(BM, BN, 1, 0, 1);
      const uint32_t bfull = tc::smem_u32(full), bempty = tc::smem_u32(empty);
      const uint64_t ad0 = tc::sdesc_sw128(tc::smem_u32(sm)), bd0 = tc::sdesc_sw128(tc::smem_u32(sm) + A_BYTES, 8192);
      uint32_t s = 0, ph = 0, n = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step) {
        const int k_lo = t / nmn * p.kper, k_hi = min(p.nk, k_lo + p.kper);
        for (int k0 = k_lo; k0 < k_hi && ok; k0 += p.kc, ++n) {
          const uint32_t a = n & 1;
          // the epilogues have read this accumulator's last contents
          if (!(ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&acc_empty[a]), ((n >> 1) & 1) ^ 1)))) break;
          tc::fence_after_sync();
          const int stages = (min(k_hi, k0 + p.kc) - k0) * pairs;
          for (int i = 0; i < stages; ++i) {
            if (!(ok = __all_sync(0xffffffffu, tc::wait(bfull + 8 * s, ph)))) break;
            if (tc::elect()) {
              const uint64_t ad = ad0 + s * (STAGE_BYTES >> 4), bd = bd0 + s * (STAGE_BYTES >> 4);
              // K steps: 16 values further inside the swizzled rows of x, 16 rows further in W
#pragma unroll
              for (int ks = 0; ks < BK / 16; ++ks)
                tc::mma_f16_pair(tacc + a * BN, ad + ks * (32 >> 4), bd + ks * ((16 * 128) >> 4), idesc,
                                 (i > 0 || ks > 0) ? 1u : 0u);
              tc::mma_commit_pair(bempty + 8 * s, 3);
            }
            __syncwarp();
            if (++s == STAGES) s = 0, ph ^= 1;
          }
          if (ok && tc::elect()) tc::mma_commit_pair(tc::smem_u32(&acc_full[a]), 3);
          __syncwarp();
        }
      }
      if (!ok && lane == 0) atomicExch(&failed, 1);
    }
  } else {
    constexpr int CW = 64 / (int)sizeof(TO);         // columns of a block on the TMA path
    const int e = warp - 2, q = warp & 3, half = e >> 2;
    constexpr int NBLK = HALF / CW;                  // blocks of a tile per warp
    uint8_t* buf = blocks + e * NBUF * BLK_BYTES;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const uint32_t release[2] = {tc::map_rank(&acc_empty[0], 0), tc::map_rank(&acc_empty[1], 0)};
    const TO* res = (const TO*)p.residual;
    TO* y = (TO*)p.y;
    const bool fetch = p.tma_out && res;
    uint32_t blk = 0, grp = 0, n = 0;   // blocks, groups of NBUF blocks and accumulators so far
    bool ok = true;
    // the warp's part of tile t: 32 rows from row m, HALF columns from column c
    auto part_of = [&](int t, int& m, int& c) {
      const Tile tl = tile_at<BN>(t % nmn, ntm, ntn);
      m = tl.m0 + (int)rank * 128 + 32 * q;
      c = tl.n0 + half * HALF;
    };
    // asks for the residual of the next group inside y, at or behind column ac
    // of tile at: NBUF blocks into the warp's buffers, all of them free
    auto ask = [&](int at, int ac) {
      int m, c;
      for (; at < ntiles; at += step, ac = 0) {
        part_of(at, m, c);
        if (m < p.M && ac < HALF && c + ac < p.N) break;
      }
      if (at < ntiles && tc::elect()) {
        const int cnt = min(min(NBUF, (HALF - ac) / CW), (p.N - c - ac + CW - 1) / CW);
        tc::mbar_expect_tx(&res_full[e], cnt * BLK_BYTES);
        for (int i = 0; i < cnt; ++i) tc::tma_load_2d(buf + i * BLK_BYTES, &map_r, c + ac + i * CW, m, &res_full[e]);
      }
      __syncwarp();
    };
    auto ask_next = [&](int at, int ac) {
      if (lane == 0) tc::bulk_wait_read<0>();   // the buffers' stores have been read
      __syncwarp();
      ask(at, ac);
    };
    if (fetch) ask(first, 0);
    // the sums of the passes before the tile's last
    constexpr int NSUM = SUM ? HALF : 1;
    float sums[NSUM];
    for (int t = first; t < ntiles; t += step, ++n) {
      int m, cbeg;
      part_of(t, m, cbeg);
      if constexpr (SUM) {
#pragma unroll
        for (int j = 0; j < NSUM; ++j) sums[j] = 0.f;
        const int k_lo = t / nmn * p.kper, passes = (min(p.kper, p.nk - k_lo) + p.kc - 1) / p.kc;
        for (int ps = 0; ps + 1 < passes; ++ps, ++n) {
          const int a = n & 1;
          ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&acc_full[a]), (n >> 1) & 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int j = 0; j < HALF; j += 32) {
            float v[32];
            tc::tmem_ld32(tacc + a * BN + lane_base + half * HALF + j, v);
            tc::tmem_ld_wait32(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sums[j + i] += v[i];
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_remote(release[a]);
        }
        if (!ok) break;
      }
      const int a = n & 1;
      ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&acc_full[a]), (n >> 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t col0 = tacc + a * BN + lane_base + half * HALF;
      if (m < p.M && p.tma_out) {
        // the next block's accumulator and bias are on their way while this one is
        // worked on; the sums leave no registers for that
        constexpr int AHEAD = SUM ? 0 : 1;
        float v[1 + AHEAD][CW], bias[AHEAD ? CW : 1];
        auto fetch_block = [&](int c, float* vv) {
          if constexpr (CW == 32)
            tc::tmem_ld32(col0 + c, vv);
          else
            tc::tmem_ld16(col0 + c, vv);
        };
        // four of the block's bias values (p.bias on a 16-byte boundary here)
        auto bias4 = [&](int c, float* bb) {
          if (cbeg + c + 4 <= p.N) {
            layer::load_vec<4>(p.bias + cbeg + c, bb);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) bb[j] = cbeg + c + j < p.N ? p.bias[cbeg + c + j] : 0.f;
          }
        };
        auto fetch_bias = [&](int c, float* bb) {
          if (p.bias)
#pragma unroll
            for (int j = 0; j < CW; j += 4) bias4(c + j, bb + j);
        };
        if constexpr (AHEAD == 1) {
          fetch_bias(0, bias);
          fetch_block(0, v[0]);
        }
#pragma unroll
        for (int i = 0; i < NBLK; ++i) {
          const int c = i * CW;
          if (cbeg + c >= p.N) break;
          float* vv = v[i & AHEAD];
          if constexpr (AHEAD == 0) fetch_block(c, vv);
          if constexpr (CW == 32)
            tc::tmem_ld_wait32(vv);
          else
            tc::tmem_ld_wait16(vv);
          if constexpr (AHEAD == 1) {
            if (i + 1 < NBLK) fetch_block(c + CW, v[(i + 1) & 1]);
          } else {
#pragma unroll
            for (int j = 0; j < CW; ++j) vv[j] += sums[c + j];
          }
          if constexpr (AHEAD == 1) {
            if (p.bias)
#pragma unroll
              for (int j = 0; j < CW; ++j) vv[j] += bias[j];
            if (i + 1 < NBLK) fetch_bias(c + CW, bias);
          } else if (p.bias) {
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
              float bb[4];
              bias4(c + j, bb);
#pragma unroll
              for (int k = 0; k < 4; ++k) vv[j + k] += bb[k];
            }
          }
          linear::act_run<TO, CW>(p.act, vv);
          const uint32_t b = fetch ? i % NBUF : blk % NBUF;
          if (fetch) {
            if (i % NBUF == 0) {
              if (i > 0) ask_next(t, c);
              if (!(ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&res_full[e]), grp & 1)))) break;
              ++grp;
            }
          } else {
            if (lane == 0) tc::bulk_wait_read<NBUF - 1>();
            __syncwarp();
          }
          uint8_t* row = buf + b * BLK_BYTES + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int PER = 16 / (int)sizeof(TO);
            TO* at = reinterpret_cast<TO*>(row + ((j ^ ((lane >> 1) & 3)) << 4));
            if (res) {
              float r[PER];
              layer::load_vec<PER>(at, r);
#pragma unroll
              for (int k = 0; k < PER; ++k) vv[j * PER + k] += r[k];
            }
            layer::store_vec<PER>(at, vv + j * PER);
          }
          tc::fence_smem_to_async();
          __syncwarp();
          if (lane == 0) {   // always lane 0: it waits for its own stores
            tc::tma_store_2d(&map_y, cbeg + c, m + t / nmn * p.split_rows, buf + b * BLK_BYTES);
            tc::bulk_commit();
          }
          ++blk;
        }
        tc::tmem_ld_wait();
        if (!ok) break;
      } else if (m < p.M) {
        float* st = reinterpret_cast<float*>(buf);   // 32 rows of 16 values, stride 17
        const int rows = min(32, p.M - m), r0 = lane / 16;
#pragma unroll
        for (int c = 0; c < HALF; c += 16) {
          if (cbeg + c >= p.N) break;
          const int col = cbeg + c + lane % 16;
          const size_t at = (size_t)(m + r0) * p.N + col;
          const bool in = col < p.N;
          const float bv = p.bias && in ? p.bias[col] : 0.f;
          float v[16], rv[16];
          tc::tmem_ld16(col0 + c, v);
          // all 16 rows of the residual in flight at once
#pragma unroll
          for (int i = 0; i < 16; ++i)
            rv[i] = res && in && r0 + 2 * i < rows ? layer::to_f32(res[at + (size_t)(2 * i) * p.N]) : 0.f;
          tc::tmem_ld_wait16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if constexpr (SUM) v[j] += sums[c + j];
            st[lane * 17 + j] = v[j];
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = st[(r0 + 2 * i) * 17 + lane % 16] + bv;
          linear::act_run<TO, 16>(p.act, v);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (in && r0 + 2 * i < rows) y[at + (size_t)(2 * i) * p.N] = layer::from_f32<TO>(v[i] + rv[i]);
          __syncwarp();
        }
      }
      // every TMEM read of this accumulator by this warp is done: hand it back
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(release[a]);
      if (fetch && m < p.M && cbeg < p.N) ask_next(t + step, 0);
    }
    if (!ok && lane == 0) atomicExch(&failed, 1);
    if (lane == 0) tc::bulk_wait_read<0>();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (failed && tid == 0) {
    tc::settle();
    atomicExch(p.status, ATLAS_ERR_TIMEOUT);
  }
  __syncthreads();
  tc::cluster_sync();
  if (warp == 0) tc::tmem_dealloc_pair(tbase, 2 * BN);
}

// y = act(sum of the splits + bias) + residual
template <typename TO>
__global__ void __launch_bounds__(256) k_linear_join(const float* __restrict__ part, int splits, int M, int N, int rows,
                                                     int cols, int act, const float* __restrict__ bias,
                                                     const TO* residual, TO* y) {
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const int per = cols / 4, m = (int)(i / per), c = (int)(i % per) * 4;
  if (m >= M) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    float p[4];
    layer::load_vec<4>(part + ((size_t)s * rows + m) * cols + c, p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += p[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] += bias && c + e < N ? bias[c + e] : 0.f;
  linear::act_run<TO, 4>(act, v);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < N) {
      const size_t at = (size_t)m * N + c + e;
      y[at] = layer::from_f32<TO>(residual ? v[e] + layer::to_f32(residual[at]) : v[e]);
    }
}

// rows and columns of a split's fp32 product in the workspace
int split_rows(int M) { return (M + BM - 1) / BM * BM; }
int split_cols(int N) { return (N + 3) / 4 * 4; }

// How many blocks of 64 of K go into one accumulator.  The tensor cores cut
// off, they do not round: an fp32 accumulator loses about 1.1e-9 of the result
// per value of K (measured: 4.8e-7 at K = 517, 9.1e-6 at 8192).  fp32 results
// take K in passes of 512, added up in registers; fp32 inputs, whatever the
// results' type, in passes of 256, each with its five small products first.
// bf16 inputs with bf16 results, rounded at 2^-8, take all of K at once.
// Only the kernel with SUM adds passes up: the host and the kernel's template
// have to agree on this.
template <bool SUM>
int blocks_per_pass(int planes, int nk) {
  return SUM ? std::min(nk, planes == 1 ? 8 : 4) : nk;
}

template <typename TO, int BN, bool SUM>
cudaError_t launch_pair(const linear::TcCall& c, cudaStream_t st) {
  CUtensorMap mx, mw, mr, my;
  if (!tc::tensor_map_2d(&mx, c.x, true, (uint64_t)c.planes * c.M, c.K, (uint64_t)c.ldx * 2, BM / 2) ||
      !tc::tensor_map_2d(&mw, c.W, true, (uint64_t)c.planes * c.K, c.N, (uint64_t)c.ldw * 2, BK))
    return cudaErrorInvalidValue;
  const int nk = (c.K + BK - 1) / BK, kper = (nk + c.splits - 1) / c.splits;
  Params p{c.M, c.N, nk, blocks_per_pass<SUM>(c.planes, nk), c.planes, c.K, c.act, kper, 0, c.bias, c.residual, c.y, 0, c.status};
  uint64_t rows = c.M;
  if (c.splits > 1) {
    p.split_rows = split_rows(c.M);
    rows = (uint64_t)c.splits * p.split_rows;
  }
  const uint64_t row = (uint64_t)(c.splits > 1 ? split_cols(c.N) : c.N) * sizeof(TO);
  p.tma_out = row % 16 == 0 && layer::aligned16(c.y) && layer::aligned16(c.residual) && layer::aligned16(c.bias) &&
              tc::tensor_map_2d(&my, c.y, sizeof(TO) == 2, rows, c.N, row, 32, 64) &&
              tc::tensor_map_2d(&mr, c.residual ? c.residual : c.y, sizeof(TO) == 2, c.M, c.N, row, 32, 64);
  if (c.splits > 1 && !p.tma_out) return cudaErrorInvalidValue;
  if (!p.tma_out) mr = my = mx;   // not used
  auto kern = k_linear_pair<TO, BN, SUM>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((c.M + BM - 1) / BM) * ((c.N + BN - 1) / BN) * c.splits;
  const int grid = (int)std::min<long long>(tiles, layer::sm_count() / 2) * 2;
  return tc::launch_overlapped(kern, dim3(grid), dim3(NTHR), Cfg<BN>::SMEM, st, mx, mw, mr, my, p);
}

}  // namespace

namespace linear {

// K is split over idle pairs where a tile takes 32 stages or more on its own and
// at least half of the pairs have none: down to 8 stages each.  The splits' fp32
// products go through the workspace and are added in order.  bf16, without the
// split / with it: 30 x 4864 x 108 (76 stages) 27 / 15 us, 145 x 4864 x 605 31 / 20,
// 64 x 8192 x 1024 37 / 21, 40 x 16384 x 136 64 / 19, 5 x 2048 x 2048 (32 stages)
// 16 / 14; fp32 128 x 4096 x 256: 94 / 24, 300 x 1024 x 512 33 / 22.  Splitting
// where fewer pairs are idle loses: 300 x 4096 x 4096 25 / 35.
int tc_splits(int M, int N, int K, int planes) {
  const long long pairs = layer::sm_count() / 2, tiles = (long long)((M + BM - 1) / BM) * ((N + 127) / 128);
  const long long nk = (K + BK - 1) / BK, stages = nk * (planes == 1 ? 1 : 6);
  if (stages < 32 || 2 * tiles > pairs) return 1;
  const long long s = std::min(std::min(pairs / tiles, stages / 8), std::min(nk, 32LL)), per = (nk + s - 1) / s;
  return (int)((nk + per - 1) / per);   // no empty split
}
size_t tc_split_bytes(int M, int N, int splits) {
  return splits > 1 ? (size_t)splits * split_rows(M) * split_cols(N) * sizeof(float) : 0;
}

cudaError_t tc_big(const TcCall& c, cudaStream_t st) {
  if (c.splits > 1) {
    TcCall part = c;
    part.bias = nullptr, part.residual = nullptr, part.y = c.split_ws, part.act = ATLAS_ACT_NONE, part.out_bf16 = 0;
    cudaError_t e = launch_pair<float, 128, true>(part, st);
    if (e != cudaSuccess) return e;
    const int cols = split_cols(c.N);
    const unsigned grid = (unsigned)(((size_t)c.M * (cols / 4) + 255) / 256);
    auto join = [&](auto kern, auto* y) {
      using T = std::remove_pointer_t<decltype(y)>;
      return tc::launch_overlapped(kern, dim3(grid), dim3(256), 0, st, (const float*)c.split_ws, c.splits, c.M, c.N,
                                   split_rows(c.M), cols, c.act, c.bias, (const T*)c.residual, (T*)c.y);
    };
    return c.out_bf16 ? join(k_linear_join<bf16>, (bf16*)nullptr) : join(k_linear_join<float>, (float*)nullptr);
  }
  // 128 columns per tile where the last round of tiles then wastes less: time in
  // units of 128 columns, the narrow tiles 1.3 times as long per column (they
  // fetch 1.5 times as much: 8192^3 took 816 us with them, 665 with wide ones)
  const long long pairs = layer::sm_count() / 2, tm = (c.M + BM - 1) / BM;
  const long long wide = (tm * ((c.N + 255) / 256) + pairs - 1) / pairs * 2,
                  narrow = (tm * ((c.N + 127) / 128) + pairs - 1) / pairs;
  auto go = [&](auto bn) {
    constexpr int BN = decltype(bn)::value;
    if (!c.out_bf16) return launch_pair<float, BN, true>(c, st);
    return c.planes > 1 ? launch_pair<bf16, BN, true>(c, st) : launch_pair<bf16, BN, false>(c, st);
  };
  return 13 * narrow < 10 * wide ? go(std::integral_constant<int, 128>()) : go(std::integral_constant<int, 256>());
}

}  // namespace linear
