// Matrix product with bias, activation and residual on the tensor cores.
//
// y = act(x W + bias) + residual, x [M][K] bf16 (K-major), W [K][N] bf16 read
// as it lies (MN-major), fp32 accumulation in TMEM.
//
// A pair of CTAs on neighbouring SMs owns a 256 x 256 tile (cta_group::2: the
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

constexpr int BM = 256, BN = 256, BK = 64, STAGES = 5, EPI_WARPS = 8, NTHR = 64 + 32 * EPI_WARPS;
constexpr int A_BYTES = BM / 2 * BK * 2, B_BYTES = BN / 2 * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BLK_BYTES = 32 * 64;                               // one epilogue block
constexpr int NBUF = 4;                                          // epilogue blocks per warp
constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * NBUF * BLK_BYTES + 1024;
constexpr int BAND = 16;                                         // row tiles per band of the tile order

struct Params {
  int M, N, nk, planes, kw;   // nk: blocks of 64 of K per plane; kw: W rows per plane
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
__device__ __forceinline__ Tile tile_at(int t, int ntm, int ntn) {
  const int width = BAND * ntn, first = t / width * BAND, h = min(BAND, ntm - first), r = t % width;
  return {(first + r % h) * BM, r / h * BN};
}

template <int ACT, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHR, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_y, Params p) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint8_t* blocks = sm + STAGES * STAGE_BYTES;
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], res_full[EPI_WARPS];
  __shared__ uint32_t tbase;
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = tc::cluster_rank();
  const int ntm = (p.M + BM - 1) / BM, ntn = (p.N + BN - 1) / BN, ntiles = ntm * ntn;
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
      const Tile tl = tile_at(t, ntm, ntn);
      const int m0 = tl.m0 + (int)rank * (BM / 2), n0 = tl.n0 + (int)rank * (BN / 2);
      for (int kt = 0; kt < p.nk && ok; ++kt) {
        for (int pr = 0; pr < pairs; ++pr) {
          int row_x = m0, row_w = kt * BK;
          if (pairs > 1) {
            int pa, pb;
            plane_pair(pr, pa, pb);
            row_x += pa * p.M;
            row_w += pb * p.kw;
          }
          if (!(ok = __all_sync(0xffffffffu, tc::wait(bempty + 8 * s, ph)))) break;
          if (tc::elect()) {
            const uint32_t a = ring + s * STAGE_BYTES, b = a + A_BYTES, bar = lead + 8 * s;
            if (rank == 0) tc::expect_tx(bfull + 8 * s, 2 * STAGE_BYTES);
            tc::tma_load_2d_pair(a, &map_x, kt * BK, row_x, bar);
            tc::tma_load_2d_pair(b, &map_w, n0, row_w, bar);
            tc::tma_load_2d_pair(b + B_BYTES / 2, &map_w, n0 + 64, row_w, bar);
          }
          __syncwarp();
          if (++s == STAGES) s = 0, ph ^= 1;
        }
      }
    }
    if (!ok && lane == 0) atomicExch(&failed, 1);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = tc::idesc_f16(BM, BN, 1, 0, 1);
      const uint32_t bfull = tc::smem_u32(full), bempty = tc::smem_u32(empty);
      const uint64_t ad0 = tc::sdesc_sw128(tc::smem_u32(sm)), bd0 = tc::sdesc_sw128(tc::smem_u32(sm) + A_BYTES, B_BYTES / 2);
      uint32_t s = 0, ph = 0, n = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step, ++n) {
        const uint32_t a = n & 1;
        // the epilogues have read this accumulator's previous tile
        if (!(ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&acc_empty[a]), ((n >> 1) & 1) ^ 1)))) break;
        tc::fence_after_sync();
        for (int kt = 0; kt < p.nk && ok; ++kt) {
          for (int pr = 0; pr < pairs; ++pr) {
            if (!(ok = __all_sync(0xffffffffu, tc::wait(bfull + 8 * s, ph)))) break;
            if (tc::elect()) {
              const uint64_t ad = ad0 + s * (STAGE_BYTES >> 4), bd = bd0 + s * (STAGE_BYTES >> 4);
              // K steps: 16 values further inside the swizzled rows of x, 16 rows further in W
#pragma unroll
              for (int ks = 0; ks < BK / 16; ++ks)
                tc::mma_f16_pair(tacc + a * BN, ad + ks * (32 >> 4), bd + ks * ((16 * 128) >> 4), idesc,
                                 (kt > 0 || pr > 0 || ks > 0) ? 1u : 0u);
              tc::mma_commit_pair(bempty + 8 * s, 3);
            }
            __syncwarp();
            if (++s == STAGES) s = 0, ph ^= 1;
          }
        }
        if (ok && tc::elect()) tc::mma_commit_pair(tc::smem_u32(&acc_full[a]), 3);
        __syncwarp();
      }
      if (!ok && lane == 0) atomicExch(&failed, 1);
    }
  } else {
    constexpr int CW = 64 / (int)sizeof(TO);         // columns of a block on the TMA path
    const int e = warp - 2, q = warp & 3, half = e >> 2;
    constexpr int NBLK = 128 / CW;                   // blocks of a tile per warp
    uint8_t* buf = blocks + e * NBUF * BLK_BYTES;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const uint32_t release[2] = {tc::map_rank(&acc_empty[0], 0), tc::map_rank(&acc_empty[1], 0)};
    const TO* res = (const TO*)p.residual;
    TO* y = (TO*)p.y;
    const bool fetch = p.tma_out && res;
    uint32_t blk = 0, grp = 0, n = 0;   // blocks, groups of NBUF blocks and tiles so far
    bool ok = true;
    // the warp's part of tile t: 32 rows from row m, 128 columns from column c
    auto part_of = [&](int t, int& m, int& c) {
      const Tile tl = tile_at(t, ntm, ntn);
      m = tl.m0 + (int)rank * 128 + 32 * q;
      c = tl.n0 + half * 128;
    };
    // asks for the residual of the next group inside y, at or behind column ac
    // of tile at: NBUF blocks into the warp's buffers, all of them free
    auto ask = [&](int at, int ac) {
      int m, c;
      for (; at < ntiles; at += step, ac = 0) {
        part_of(at, m, c);
        if (m < p.M && ac < 128 && c + ac < p.N) break;
      }
      if (at < ntiles && tc::elect()) {
        const int cnt = min(NBUF, (p.N - c - ac + CW - 1) / CW);
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
    for (int t = first; t < ntiles; t += step, ++n) {
      const int a = n & 1;
      ok = __all_sync(0xffffffffu, tc::wait(tc::smem_u32(&acc_full[a]), (n >> 1) & 1));
      if (!ok) break;
      tc::fence_after_sync();
      int m, cbeg;
      part_of(t, m, cbeg);
      const uint32_t col0 = tacc + a * BN + lane_base + half * 128;
      if (m < p.M && p.tma_out) {
        float v[2][CW], bias[2][CW];
        auto fetch_block = [&](int c, float* vv, float* bb) {
          if constexpr (CW == 32)
            tc::tmem_ld32(col0 + c, vv);
          else
            tc::tmem_ld16(col0 + c, vv);
          if (p.bias) {
            const float* bp = p.bias + cbeg + c;
            if (cbeg + c + CW <= p.N) {
#pragma unroll
              for (int j = 0; j < CW; j += 4) layer::load_vec<4>(bp + j, bb + j);
            } else {
#pragma unroll
              for (int j = 0; j < CW; ++j) bb[j] = cbeg + c + j < p.N ? bp[j] : 0.f;
            }
          }
        };
        fetch_block(0, v[0], bias[0]);
#pragma unroll
        for (int i = 0; i < NBLK; ++i) {
          const int c = i * CW;
          if (cbeg + c >= p.N) break;
          float* vv = v[i & 1];
          float* bb = bias[i & 1];
          if constexpr (CW == 32)
            tc::tmem_ld_wait32(vv);
          else
            tc::tmem_ld_wait16(vv);
          if (i + 1 < NBLK) fetch_block(c + CW, v[(i + 1) & 1], bias[(i + 1) & 1]);
          if (p.bias)
#pragma unroll
            for (int j = 0; j < CW; ++j) vv[j] += bb[j];
          linear::act_all<ACT, TO, CW>(vv);
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
            tc::tma_store_2d(&map_y, cbeg + c, m, buf + b * BLK_BYTES);
            tc::bulk_commit();
          }
          ++blk;
        }
        tc::tmem_ld_wait();
        if (!ok) break;
      } else if (m < p.M) {
        float* st = reinterpret_cast<float*>(buf);   // 32 rows of 16 values, stride 17
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          if (cbeg + c >= p.N) break;
          float v[16];
          tc::tmem_ld16(col0 + c, v);
          tc::tmem_ld_wait16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) st[lane * 17 + j] = v[j];
          __syncwarp();
          const int col = cbeg + c + lane % 16;
          if (col < p.N) {
            const float bv = p.bias ? p.bias[col] : 0.f;
            const int rows = min(32, p.M - m);
#pragma unroll 4
            for (int r = lane / 16; r < rows; r += 2) {
              const size_t at = (size_t)(m + r) * p.N + col;
              float o = linear::act_for<ACT, TO>(st[r * 17 + lane % 16] + bv);
              if (res) o += layer::to_f32(res[at]);
              y[at] = layer::from_f32<TO>(o);
            }
          }
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
    // let every copy this CTA issued land before its memory is freed
    for (int s = 0; s < STAGES; ++s) tc::mbar_wait(&full[s], 0, tc::kWaitCycles / 16);
    atomicExch(p.status, ATLAS_ERR_TIMEOUT);
  }
  __syncthreads();
  tc::cluster_sync();
  if (warp == 0) tc::tmem_dealloc_pair(tbase, 2 * BN);
}

template <int ACT, typename TO>
cudaError_t launch_pair(const linear::TcCall& c, cudaStream_t st) {
  CUtensorMap mx, mw, mr, my;
  if (!tc::tensor_map_2d(&mx, c.x, true, (uint64_t)c.planes * c.M, c.K, (uint64_t)c.ldx * 2, BM / 2) ||
      !tc::tensor_map_2d(&mw, c.W, true, (uint64_t)c.planes * c.K, c.N, (uint64_t)c.ldw * 2, BK))
    return cudaErrorInvalidValue;
  Params p{c.M, c.N, (c.K + BK - 1) / BK, c.planes, c.K, c.bias, c.residual, c.y, 0, c.status};
  const uint64_t row = (uint64_t)c.N * sizeof(TO);
  p.tma_out = row % 16 == 0 && layer::aligned16(c.y) && layer::aligned16(c.residual) && layer::aligned16(c.bias) &&
              tc::tensor_map_2d(&my, c.y, sizeof(TO) == 2, c.M, c.N, row, 32, 64) &&
              tc::tensor_map_2d(&mr, c.residual ? c.residual : c.y, sizeof(TO) == 2, c.M, c.N, row, 32, 64);
  if (!p.tma_out) mr = my = mx;   // not used
  auto kern = k_linear_pair<ACT, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((c.M + BM - 1) / BM) * ((c.N + BN - 1) / BN);
  const int grid = (int)std::min<long long>(tiles, layer::sm_count() / 2) * 2;
  return tc::launch_overlapped(kern, dim3(grid), dim3(NTHR), SMEM, st, mx, mw, mr, my, p);
}

}  // namespace

namespace linear {

cudaError_t tc_big(const TcCall& c, cudaStream_t st) {
  auto by_type = [&](auto act) {
    constexpr int A = decltype(act)::value;
    return c.out_bf16 ? launch_pair<A, bf16>(c, st) : launch_pair<A, float>(c, st);
  };
  if (c.act == ATLAS_ACT_SILU) return by_type(std::integral_constant<int, ATLAS_ACT_SILU>());
  if (c.act == ATLAS_ACT_GELU) return by_type(std::integral_constant<int, ATLAS_ACT_GELU>());
  return by_type(std::integral_constant<int, ATLAS_ACT_NONE>());
}

}  // namespace linear
