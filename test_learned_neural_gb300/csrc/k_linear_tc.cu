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
//              activation, residual -> one 32-row, 128-byte-wide swizzled block
//              per warp (two of them alternate) -> TMA store.  The residual's
//              block comes into the same buffer by TMA one block ahead.
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
constexpr int A_BYTES = BM / 2 * BK * 2, B_BYTES = BN / 2 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BLK_BYTES = 32 * 128;                              // one epilogue block
constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * 2 * BLK_BYTES + 1024;
constexpr int BAND = 16;                                         // row tiles per band of the tile order

struct Params {
  int M, N, nk, planes, kw;   // nk: stages of K per plane; kw: W rows per plane
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
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], res_full[EPI_WARPS][2];
  __shared__ uint32_t tbase;
  __shared__ int failed;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = tc::cluster_rank();
  const int ntm = (p.M + BM - 1) / BM, ntn = (p.N + BN - 1) / BN, ntiles = ntm * ntn;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int pairs = p.planes == 1 ? 1 : 6, iters = p.nk * pairs;

  if (warp == 0) tc::tmem_alloc_pair(&tbase, 2 * BN);
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&acc_full[a], 1);
      tc::mbar_init(&acc_empty[a], 2 * EPI_WARPS);   // every epilogue warp of both CTAs
    }
    for (int w = 0; w < EPI_WARPS; ++w)
      for (int b = 0; b < 2; ++b) tc::mbar_init(&res_full[w][b], 1);
    failed = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tacc = tbase;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step) {
        const Tile tl = tile_at(t, ntm, ntn);
        const int m0 = tl.m0 + (int)rank * (BM / 2), n0 = tl.n0 + (int)rank * (BN / 2);
        for (int i = 0; i < iters; ++i, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES && !(ok = tc::mbar_wait_cluster(&empty[s], ((it / STAGES) - 1) & 1, tc::kWaitCycles))) break;
          int pa = 0, pb = 0, kt = i;
          if (pairs > 1) {
            kt = i / 6;
            plane_pair(i % 6, pa, pb);
          }
          uint8_t* a = sm + s * STAGE_BYTES;
          const uint32_t bar = tc::map_rank(&full[s], 0);
          if (rank == 0) tc::mbar_expect_tx(&full[s], 2 * STAGE_BYTES);
          tc::tma_load_2d_pair(a, &map_x, kt * BK, pa * p.M + m0, bar);
          tc::tma_load_2d_pair(a + A_BYTES, &map_w, n0, pb * p.kw + kt * BK, bar);
          tc::tma_load_2d_pair(a + A_BYTES + B_BYTES / 2, &map_w, n0 + 64, pb * p.kw + kt * BK, bar);
        }
      }
      if (!ok) atomicExch(&failed, 1);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = tc::idesc_f16(BM, BN, 1, 0, 1);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok; t += step, ++n) {
        const int a = n & 1;
        if (n >= 2 && !(ok = tc::mbar_wait_cluster(&acc_empty[a], ((n >> 1) - 1) & 1, tc::kWaitCycles))) break;
        tc::fence_after_sync();
        for (int i = 0; i < iters; ++i, ++it) {
          const int s = it % STAGES;
          if (!(ok = tc::mbar_wait_cluster(&full[s], (it / STAGES) & 1, tc::kWaitCycles))) break;
          tc::fence_after_sync();
          const uint32_t sa = tc::smem_u32(sm + s * STAGE_BYTES);
          uint64_t ad = tc::sdesc_sw128(sa), bd = tc::sdesc_sw128(sa + A_BYTES, B_BYTES / 2);
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks) {
            tc::mma_f16_pair(tacc + a * BN, ad, bd, idesc, (i > 0 || ks > 0) ? 1u : 0u);
            ad += 32 >> 4;           // 16 values further along K inside the swizzled row
            bd += (16 * 128) >> 4;   // 16 rows of K further
          }
          tc::mma_commit_pair(&empty[s]);
        }
        if (ok) tc::mma_commit_pair(&acc_full[a]);
      }
      if (!ok) atomicExch(&failed, 1);
    }
  } else {
    constexpr int CW = 128 / (int)sizeof(TO);        // columns of a block on the TMA path
    const int e = warp - 2, q = warp & 3, half = e >> 2;
    uint8_t* buf = blocks + e * 2 * BLK_BYTES;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const uint32_t release[2] = {tc::map_rank(&acc_empty[0], 0), tc::map_rank(&acc_empty[1], 0)};
    const TO* res = (const TO*)p.residual;
    TO* y = (TO*)p.y;
    const bool fetch = p.tma_out && res;
    int blk = 0, n = 0;
    bool ok = true;
    // asks for the residual's block of (tile, column); the buffer's last store has been read
    auto ask = [&](int b, int m, int c) {
      if (lane == 0) {
        tc::mbar_expect_tx(&res_full[e][b], BLK_BYTES);
        tc::tma_load_2d(buf + b * BLK_BYTES, &map_r, c, m, &res_full[e][b]);
      }
    };
    // the first block of this warp at or behind tile t that lies inside y, if any
    auto ask_first = [&](int b, int t) {
      for (; t < ntiles; t += step) {
        const Tile tl = tile_at(t, ntm, ntn);
        const int m = tl.m0 + (int)rank * 128 + 32 * q, c = tl.n0 + half * 128;
        if (m < p.M && c < p.N) {
          ask(b, m, c);
          return;
        }
      }
    };
    if (fetch) ask_first(0, first);
    for (int t = first; t < ntiles; t += step, ++n) {
      const int a = n & 1;
      ok = __all_sync(0xffffffffu, tc::mbar_wait_cluster(&acc_full[a], (n >> 1) & 1, tc::kWaitCycles));
      if (!ok) break;
      tc::fence_after_sync();
      const Tile tl = tile_at(t, ntm, ntn);
      const int m = tl.m0 + (int)rank * 128 + 32 * q, cbeg = tl.n0 + half * 128;
      const uint32_t col0 = tacc + a * BN + lane_base + half * 128;
      if (m < p.M && p.tma_out) {
#pragma unroll 1
        for (int c = 0; c < 128; c += CW) {
          if (cbeg + c >= p.N) break;
          const int b = blk & 1;
          float v[CW];
#pragma unroll
          for (int j = 0; j < CW; j += 32) tc::tmem_ld32(col0 + c + j, v + j);
#pragma unroll
          for (int j = 0; j < CW; j += 32) tc::tmem_ld_wait32(v + j);
          if (p.bias) {
            const float* bp = p.bias + cbeg + c;
            const bool whole = cbeg + c + CW <= p.N;
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
              float bv[4];
              if (whole) {
                layer::load_vec<4>(bp + j, bv);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) bv[i] = cbeg + c + j + i < p.N ? bp[j + i] : 0.f;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) v[j + i] += bv[i];
            }
          }
#pragma unroll
          for (int j = 0; j < CW; ++j) v[j] = linear::act_for<ACT, TO>(v[j]);
          // the other buffer's store has been read: ask for its next block
          if (lane == 0) tc::bulk_wait_read<0>();
          if (fetch) {
            if (c + CW < 128 && cbeg + c + CW < p.N)
              ask(b ^ 1, m, cbeg + c + CW);
            else
              ask_first(b ^ 1, t + step);
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&res_full[e][b], (blk >> 1) & 1, tc::kWaitCycles));
            if (!ok) break;
          }
          __syncwarp();
          uint8_t* row = buf + b * BLK_BYTES + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            constexpr int PER = 16 / (int)sizeof(TO);
            TO* at = reinterpret_cast<TO*>(row + ((j ^ (lane & 7)) << 4));
            if (res) {
              float r[PER];
              layer::load_vec<PER>(at, r);
#pragma unroll
              for (int i = 0; i < PER; ++i) v[j * PER + i] += r[i];
            }
            layer::store_vec<PER>(at, v + j * PER);
          }
          tc::fence_smem_to_async();
          __syncwarp();
          if (lane == 0) {
            tc::tma_store_2d(&map_y, cbeg + c, m, buf + b * BLK_BYTES);
            tc::bulk_commit();
          }
          ++blk;
        }
        if (!ok) break;
      } else if (m < p.M) {
        float* st = reinterpret_cast<float*>(buf);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          if (cbeg + c >= p.N) break;
          float v[32];
          tc::tmem_ld32(col0 + c, v);
          tc::tmem_ld_wait32(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) st[lane * 33 + j] = v[j];
          __syncwarp();
          const int col = cbeg + c + lane;
          if (col < p.N) {
            const float bv = p.bias ? p.bias[col] : 0.f;
            const int rows = min(32, p.M - m);
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
              const size_t at = (size_t)(m + r) * p.N + col;
              float o = linear::act_for<ACT, TO>(st[r * 33 + lane] + bv);
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
    }
    if (!ok && lane == 0) atomicExch(&failed, 1);
    if (lane == 0) tc::bulk_wait_all();
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
              tc::tensor_map_2d(&my, c.y, sizeof(TO) == 2, c.M, c.N, row, 32) &&
              tc::tensor_map_2d(&mr, c.residual ? c.residual : c.y, sizeof(TO) == 2, c.M, c.N, row, 32);
  if (!p.tma_out) mr = my = mx;   // not used
  auto kern = k_linear_pair<ACT, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((c.M + BM - 1) / BM) * ((c.N + BN - 1) / BN);
  const int grid = (int)std::min<long long>(tiles, layer::sm_count() / 2) * 2;
  kern<<<grid, NTHR, SMEM, st>>>(mx, mw, mr, my, p);
  return cudaGetLastError();
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
