// Decay attention on the tensor cores for 64 < d_k <= 128: bf16 q, k, v, any
// d_v in slices of 64 columns, chunks of 128 tokens (decay_common.cuh has the
// formulas).  Two 64-wide tiles of q and k and their three terms leave no room
// for k_decay_ws.cu's ring, so every warp does each stage in turn.
//
// k_decay_tc, one CTA per (segment, slice, unit), chunks in order.  Per chunk:
//   scores  Q K^T                      M = 128 tokens, N = 128
//   inter   Q S                        N = 64, S split into bf16 terms
//   intra   P V, P = scores * decays   P from TMEM, split into NT terms
//   state   (w K)^T V, w_j = g^{n-1-j} w K split into three bf16 terms (24
//           bits), V exact, so the fp32 state keeps fp32 accuracy
// The decays are applied in fp32 registers; the state lives there too, fp32,
// for the whole segment.  NT = 2 for bf16 read-outs: P and S are kept to 16 bits
// each (2^-16 of a term against the read-out's own rounding of 2^-8; with P in
// one term, 2^-8 of every term, the read-outs were 1.2 times as far from the
// exact ones as their rounding alone).  NT = 3 for fp32 read-outs: 24 bits.
//
// TMEM (256 columns): scores, then P in place, then the state's product, in 128
// columns; inter and intra read-outs 64 columns each.
//
// k_decay_tc_state: a segment's own contribution to the state at its end, the
// same product with weights counted to the segment's end, accumulated in TMEM
// over the whole segment.
#include "decay_tc_dev.cuh"

using namespace decay;
using layer::bf16;

namespace {

constexpr int NTHR = 256;
constexpr int KB = 2;   // 64-wide tiles of d_k

// Rows n .. 127 of a tile become zero (a row's tokens past its length: 0 * NaN
// must not reach the sums).
__device__ __forceinline__ void zero_rows(uint32_t tile, int n, int tid) {
  for (int i = tid; i < (C - n) * 8; i += NTHR) sts128(tile + (n + i / 8) * 128 + (i % 8) * 16, 0, 0, 0, 0);
}

// Token tid % 128's 32 keys of half tid / 128 of a 64-wide tile, times w, in
// three bf16 terms: term 0 stays packed in k0, terms 1 and 2 go to their tiles.
__device__ __forceinline__ void scale_keys(uint32_t ktile, uint32_t t1, uint32_t t2, float w, bool live, int tid,
                                           uint32_t* k0) {
  const int r = tid & (C - 1), j0 = (tid >> 7) * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t x[4], y[4][3];
    lds128(ktile + swz(r, j0 + j), x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!live) x[i] = 0u;
      split2<3>(__uint_as_float(x[i] << 16) * w, __uint_as_float(x[i] & 0xffff0000u) * w, y[i]);
      k0[4 * j + i] = y[i][0];
    }
    sts128(t1 + swz(r, j0 + j), y[0][1], y[1][1], y[2][1], y[3][1]);
    sts128(t2 + swz(r, j0 + j), y[0][2], y[1][2], y[2][2], y[3][2]);
  }
}
__device__ __forceinline__ void store_keys(uint32_t tile, int tid, const uint32_t* k0) {
  const int r = tid & (C - 1), j0 = (tid >> 7) * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) sts128(tile + swz(r, j0 + j), k0[4 * j], k0[4 * j + 1], k0[4 * j + 2], k0[4 * j + 3]);
}

// (w K)^T V into TMEM at d, M = 128: three terms of two 64-wide key tiles, one
// instruction per 16 tokens, the smallest term first; terms at t0, t1, t2
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t t0, uint32_t t1, uint32_t t2, uint32_t vtile,
                                          bool accumulate) {
  const uint32_t idesc = tc::idesc_f16(128, SL, 1, 1, 1);
  const uint64_t vd = tc::sdesc_sw128(vtile, TILE);
  const uint64_t kd[3] = {tc::sdesc_sw128(t0, TILE), tc::sdesc_sw128(t1, TILE), tc::sdesc_sw128(t2, TILE)};
#pragma unroll
  for (int i = 2; i >= 0; --i)
#pragma unroll
    for (int s = 0; s < C / 16; ++s)
      tc::mma_f16(d, kd[i] + s * (2048 >> 4), vd + s * (2048 >> 4), idesc, (accumulate || i < 2 || s > 0) ? 1u : 0u);
}

// The state's product as the threads hold it (warp = q + 4 h): row 32 q + lane
// of d_k, 32 columns from 32 h.
struct StatePart {
  static constexpr int N = 32;
  int row, col;
  __device__ StatePart(int warp, int lane) : row(32 * (warp & 3) + lane), col(32 * (warp >> 2)) {}
  __device__ __forceinline__ void load(uint32_t tmem, int warp, float* v) const {
    tc::tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32 * (warp >> 2), v);
    tc::tmem_ld_wait32(v);
  }
};

template <int NT>
struct Smem {   // byte offsets from a 1024-byte aligned base
  static constexpr int q = 0, k = q + KB * TILE, v = k + KB * TILE, k1 = v + TILE, k2 = k1 + KB * TILE,
                       s = k2 + KB * TILE, NS = NT == 2 ? 2 : 3, s_tile = KB * 64 * 128,
                       y = NT == 2 ? s + NS * s_tile : q,   // read-outs: a tile of their own, or q's once it is read
                       pw = NT == 2 ? y + TILE : s + NS * s_tile, bars = pw + (C + 4) * 4, end = bars + 64;
};

template <int NT, typename TO>
__global__ void __launch_bounds__(NTHR, 1)
    k_decay_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap my, Geom g, Ptrs p,
               int* status) {
  using L = Smem<NT>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  float* pw = reinterpret_cast<float*>(sm + L::pw);   // g^0 .. g^128
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
  // full_q, full_kv, scores, intra, state, tmem base, failed
  uint32_t* tbase = reinterpret_cast<uint32_t*>(bars + 6);
  int* failed = reinterpret_cast<int*>(bars + 7);
  const int s = blockIdx.x, sl = blockIdx.y, unit = blockIdx.z;
  const int b = unit / g.H, h = unit % g.H, hq = h / g.share;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, wq = warp & 3, wh = warp >> 2;
  const uint32_t bq = tc::smem_u32(bars), bkv = bq + 8, bsc = bq + 16, bin = bq + 24, bst = bq + 32;
  if (warp == 0) tc::tmem_alloc(tbase, 256);
  if (tid == 32) {
    for (int i = 0; i < 5; ++i) tc::mbar_init_only(bars + i, 1);
    tc::mbar_init_fence();
    *failed = (base & 1023u) ? 1 : 0;   // the swizzled tiles need it; never seen otherwise
    tc::prefetch_map(&mq);
    tc::prefetch_map(&mk);
    tc::prefetch_map(&mv);
    tc::prefetch_map(&my);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tbase;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();

  const int live = decay::live_tokens(g, p, b);
  const int t_lo = s * g.seg, t_hi = min(g.T, t_lo + g.seg), t_live = min(t_hi, max(live, t_lo));
  const int c0 = sl * SL, cols = min(SL, g.d_v - c0);
  const size_t sq = (size_t)g.d_k * g.d_v;
  bool ok = *failed == 0;

  auto load_q = [&](int t0) {
    tc::expect_tx(bq, KB * TILE);
    for (int i = 0; i < KB; ++i) load_4d(base + L::q + i * TILE, &mq, 64 * i, t0, hq, b, bq);
  };
  auto load_kv = [&](int t0) {
    tc::expect_tx(bkv, (KB + 1) * TILE);
    for (int i = 0; i < KB; ++i) load_4d(base + L::k + i * TILE, &mk, 64 * i, t0, hq, b, bkv);
    load_4d(base + L::v, &mv, c0, t0, h, b, bkv);
  };
  if (ok && t_lo < t_live && warp == 0) {
    if (tc::elect()) {
      load_q(t_lo);
      load_kv(t_lo);
    }
    __syncwarp();
  }
  const float l2g = log2f(p.decay[h]);
  for (int i = tid; i <= C; i += NTHR) pw[i] = decay::power(l2g, i);

  // the state, fp32, and its bf16 terms as the operand of Q S: rows d_k, 64
  // values of d_v
  const StatePart part(warp, lane);
  float S[StatePart::N];
  {
    const float* start = g.nseg > 1 ? p.seg + ((size_t)unit * g.nseg + s) * sq : p.S0 ? p.S0 + unit * sq : nullptr;
#pragma unroll
    for (int i = 0; i < StatePart::N; ++i)
      S[i] = start && part.row < g.d_k && part.col + i < cols ? start[(size_t)part.row * g.d_v + c0 + part.col + i] : 0.f;
  }
  auto state_tiles = [&]() {
#pragma unroll
    for (int i = 0; i < StatePart::N; i += 8) {
      uint32_t w[4][L::NS];
#pragma unroll
      for (int j = 0; j < 4; ++j) split2<L::NS>(S[i + 2 * j], S[i + 2 * j + 1], w[j]);
#pragma unroll
      for (int n = 0; n < L::NS; ++n)
        sts128(base + L::s + n * L::s_tile + swz(part.row, (part.col + i) / 8), w[0][n], w[1][n], w[2][n], w[3][n]);
    }
  };
  state_tiles();
  tc::fence_smem_to_async();
  __syncthreads();

  const uint32_t lanes = (uint32_t)(32 * wq) << 16;
  const int row = 32 * wq + lane;   // token of this thread in the chunk's scores and read-outs
  uint32_t ph = 0;
  for (int t0 = t_lo; ok && t0 < t_live; t0 += C, ph ^= 1) {
    const int n = min(C, t_live - t0);
    ok &= tc::wait(bq, ph);
    ok &= tc::wait(bkv, ph);
    auto mma_inter = [&]() {   // Q S, the smallest terms first
      const uint32_t idesc = tc::idesc_f16(C, SL, 1, 0, 1);
#pragma unroll
      for (int i = L::NS - 1; i >= 0; --i)
#pragma unroll
        for (int ks = 0; ks < 4 * KB; ++ks)
          tc::mma_f16(tm + 128, tc::sdesc_sw128(base + L::q + (ks / 4) * TILE) + (ks % 4) * (32 >> 4),
                      tc::sdesc_sw128(base + L::s + i * L::s_tile, 8192) + ks * (2048 >> 4), idesc,
                      (i < L::NS - 1 || ks > 0) ? 1u : 0u);
    };
    if (warp == 0) {
      if (tc::elect()) {
        const uint32_t idesc = tc::idesc_f16(C, C, 1, 0, 0);
#pragma unroll
        for (int ks = 0; ks < 4 * KB; ++ks)
          tc::mma_f16(tm, tc::sdesc_sw128(base + L::q + (ks / 4) * TILE) + (ks % 4) * (32 >> 4),
                      tc::sdesc_sw128(base + L::k + (ks / 4) * TILE) + (ks % 4) * (32 >> 4), idesc, ks > 0 ? 1u : 0u);
        if constexpr (NT == 2) mma_inter();
        tc::mma_commit(bars + 2);
      }
      __syncwarp();
    }
    // keys times decays; the first term waits in registers until the scores have read the keys
    uint32_t k0[KB][16];
    {
      const int r = tid & (C - 1);
      const float w = r < n ? pw[n - 1 - r] : 0.f;
#pragma unroll
      for (int i = 0; i < KB; ++i)
        scale_keys(base + L::k + i * TILE, base + L::k1 + i * TILE, base + L::k2 + i * TILE, w, r < n, tid, k0[i]);
      if (n < C) zero_rows(base + L::v, n, tid);
    }
    ok &= tc::wait(bsc, ph);
    tc::fence_after_sync();
#pragma unroll
    for (int i = 0; i < KB; ++i) store_keys(base + L::k + i * TILE, tid, k0[i]);
    // P: 32 x 32 blocks, two per warp; full ones below the diagonal
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int blk = wh == 0 ? 3 * u : 1 + u;   // columns 32 blk ..
      uint32_t w[16][NT];
      if (blk > wq) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int k = 0; k < NT; ++k) w[i][k] = 0u;
      } else {
        float v[32];
        tc::tmem_ld32(tm + lanes + 32 * blk, v);
        tc::tmem_ld_wait32(v);
        if (blk < wq) {
          const float f = pw[row - 32 * blk - 31];   // times g^{31 - c}
#pragma unroll
          for (int i = 0; i < 16; ++i)
            split2<NT>(v[2 * i] * (f * pw[31 - 2 * i]), v[2 * i + 1] * (f * pw[30 - 2 * i]), w[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float a = lane >= 2 * i ? v[2 * i] * pw[max(0, lane - 2 * i)] : 0.f;
            const float c = lane >= 2 * i + 1 ? v[2 * i + 1] * pw[max(0, lane - 2 * i - 1)] : 0.f;
            split2<NT>(a, c, w[i]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = w[i][k];
        // terms 0 and 1 inside the block's own columns, term 2 where Q S goes later
        tmem_st16u(tm + lanes + (k < 2 ? 32 * blk + 16 * k : 128 + 16 * blk), x);
      }
    }
    tc::tmem_st_wait();
    tc::fence_smem_to_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) {
      if (tc::elect()) {
        if constexpr (NT == 2)
          if (t0 + C < t_live) load_q(t0 + C);   // scores and Q S have read q
        const uint32_t idesc = tc::idesc_f16(C, SL, 1, 0, 1);
        const uint64_t vd = tc::sdesc_sw128(base + L::v, TILE);
#pragma unroll
        for (int k = NT - 1; k >= 0; --k)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(tm + 192, tm + (k < 2 ? 32 * (ks / 2) + 16 * k : 128 + 16 * (ks / 2)) + 8 * (ks % 2),
                   vd + ks * (2048 >> 4), idesc, (k < NT - 1 || ks > 0) ? 1u : 0u);
        tc::mma_commit(bars + 3);
      }
      __syncwarp();
    }
    ok &= tc::wait(bin, NT == 3 ? 0 : ph);   // P V done: its columns are free (NT = 3: two phases per chunk)
    tc::fence_after_sync();
    if (NT == 3) {
      if (warp == 0) {
        if (tc::elect()) {
          mma_inter();
          tc::mma_commit(bars + 3);
        }
        __syncwarp();
      }
    }
    if (warp == 0) {
      if (tc::elect()) {
        mma_state(tm, base + L::k, base + L::k1, base + L::k2, base + L::v, false);
        tc::mma_commit(bars + 4);
      }
      __syncwarp();
    }
    // the read-outs, 32 columns per thread
    {
      float yi[32], ya[32];
      if (NT == 3) {
        ok &= tc::wait(bin, 1);
        tc::fence_after_sync();
      }
      tc::tmem_ld32(tm + 128 + lanes + 32 * wh, yi);
      tc::tmem_ld32(tm + 192 + lanes + 32 * wh, ya);
      tc::tmem_ld_wait32(yi);
      tc::tmem_ld_wait32(ya);
      const float f = pw[row + 1] * g.scale;
#pragma unroll
      for (int i = 0; i < 32; ++i) ya[i] = row < n ? fmaf(f, yi[i], g.scale * ya[i]) : 0.f;
      if constexpr (sizeof(TO) == 2) {
        if (lane == 0 && warp == 0) tc::bulk_wait_read<0>();   // the last chunk's store has been read
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sts128(base + L::y + swz(row, 4 * wh + j), layer::pack_bf16(ya[8 * j], ya[8 * j + 1]),
                 layer::pack_bf16(ya[8 * j + 2], ya[8 * j + 3]), layer::pack_bf16(ya[8 * j + 4], ya[8 * j + 5]),
                 layer::pack_bf16(ya[8 * j + 6], ya[8 * j + 7]));
        tc::fence_smem_to_async();
        __syncthreads();
        if (tid == 0) {
          store_4d(&my, c0, t0, h, b, base + L::y);
          tc::bulk_commit();
        }
      } else {
        // 32 columns at a time through one tile
        for (int half = 0; half < 2; ++half) {
          if (half == 1 && cols <= 32) break;
          if (wh == half)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sts128(base + L::y + swz(row, j), __float_as_uint(ya[4 * j]), __float_as_uint(ya[4 * j + 1]),
                     __float_as_uint(ya[4 * j + 2]), __float_as_uint(ya[4 * j + 3]));
          tc::fence_smem_to_async();
          __syncthreads();
          if (tid == 0) {
            store_4d(&my, c0 + 32 * half, t0, h, b, base + L::y);
            tc::bulk_commit();
            tc::bulk_wait_read<0>();
          }
          __syncthreads();
        }
      }
    }
    // the state behind this chunk
    ok &= tc::wait(bst, ph);
    tc::fence_after_sync();
    if (warp == 0 && t0 + C < t_live) {
      if (tc::elect()) {
        if constexpr (NT == 3) load_q(t0 + C);
        load_kv(t0 + C);   // the state's product has read k and v
      }
      __syncwarp();
    }
    {
      float d[StatePart::N];
      part.load(tm, warp, d);
      const float f = pw[n];
#pragma unroll
      for (int i = 0; i < StatePart::N; ++i) S[i] = fmaf(f, S[i], d[i]);
    }
    if (t0 + C < t_live) state_tiles();
    tc::fence_smem_to_async();
    tc::fence_before_sync();
    ok = __syncthreads_and(ok);
    tc::fence_after_sync();
  }
  if (ok) {
    // read-outs past the row's length: whole chunks (the last live chunk wrote its own)
    TO* y = (TO*)p.y + b * g.y_b + h * g.y_h + c0;
    const int z0 = t_lo + (t_live - t_lo + C - 1) / C * C;
    for (int t = z0 + tid / 64; t < t_hi; t += NTHR / 64)
      if (tid % 64 < cols) y[t * g.y_t + tid % 64] = layer::from_f32<TO>(0.f);
    if (s == g.nseg - 1 && p.S_out) {
#pragma unroll
      for (int i = 0; i < StatePart::N; ++i)
        if (part.row < g.d_k && part.col + i < cols)
          p.S_out[unit * sq + (size_t)part.row * g.d_v + c0 + part.col + i] = S[i];
    }
  } else if (tid == 0) {
    tc::settle();
    atomicExch(status, ATLAS_ERR_TIMEOUT);
  }
  if (tid == 0) tc::bulk_wait_read<0>();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tm, 256);
}

// shared memory of k_decay_tc_state: two (k, v) buffers, three terms
struct SmemState {
  static constexpr int kv_bytes = (KB + 1) * TILE, t0 = 2 * kv_bytes, bars = t0 + 3 * KB * TILE, end = bars + 64;
};

__global__ void __launch_bounds__(NTHR, 1)
    k_decay_tc_state(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, Geom g, Ptrs p,
                     int* status) {
  using L = SmemState;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);   // full[2], done, tmem base, failed
  uint32_t* tbase = reinterpret_cast<uint32_t*>(bars + 3);
  int* failed = reinterpret_cast<int*>(bars + 4);
  const int s = blockIdx.x, sl = blockIdx.y, unit = blockIdx.z;
  const int b = unit / g.H, h = unit % g.H, hq = h / g.share;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t bfull = tc::smem_u32(bars), bdone = bfull + 16;
  if (warp == 0) tc::tmem_alloc(tbase, 64);
  if (tid == 32) {
    for (int i = 0; i < 3; ++i) tc::mbar_init_only(bars + i, 1);
    tc::mbar_init_fence();
    *failed = (base & 1023u) ? 1 : 0;
    tc::prefetch_map(&mk);
    tc::prefetch_map(&mv);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tbase;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();

  const int live = decay::live_tokens(g, p, b);
  const int t_lo = s * g.seg, t_hi = min(g.T, t_lo + g.seg), t_live = min(t_hi, max(live, t_lo));
  const int c0 = sl * SL, cols = min(SL, g.d_v - c0), chunks = (t_live - t_lo + C - 1) / C;
  bool ok = *failed == 0;
  auto load = [&](int c) {
    const uint32_t at = base + (c & 1) * L::kv_bytes, bar = bfull + 8 * (c & 1);
    const int t0 = t_lo + c * C;
    tc::expect_tx(bar, (KB + 1) * TILE);
    for (int i = 0; i < KB; ++i) load_4d(at + i * TILE, &mk, 64 * i, t0, hq, b, bar);
    load_4d(at + KB * TILE, &mv, c0, t0, h, b, bar);
  };
  if (ok && warp == 0) {
    if (tc::elect())
      for (int c = 0; c < min(2, chunks); ++c) load(c);
    __syncwarp();
  }
  const float l2g = log2f(p.decay[h]);
  for (int c = 0; ok && c < chunks; ++c) {
    const int t0 = t_lo + c * C, n = min(C, t_live - t0);
    const uint32_t kt = base + (c & 1) * L::kv_bytes, vt = kt + KB * TILE;
    ok &= tc::wait(bfull + 8 * (c & 1), (c >> 1) & 1);
    if (c > 0) ok &= tc::wait(bdone, (c - 1) & 1);   // the last product has read the terms
    const int r = tid & (C - 1);
    const float w = r < n ? decay::power(l2g, t_live - 1 - t0 - r) : 0.f;
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      uint32_t k0[16];
      scale_keys(kt + i * TILE, base + L::t0 + (KB + i) * TILE, base + L::t0 + (2 * KB + i) * TILE, w, r < n, tid, k0);
      store_keys(base + L::t0 + i * TILE, tid, k0);
    }
    if (n < C) zero_rows(vt, n, tid);
    tc::fence_smem_to_async();
    tc::fence_before_sync();
    ok = __syncthreads_and(ok);
    tc::fence_after_sync();
    if (warp == 0 && ok) {
      // the buffer of the chunk behind the next: free once its product is done
      if (c >= 1 && c + 1 < chunks) {
        if (tc::elect()) load(c + 1);
        __syncwarp();
      }
      if (tc::elect()) {
        mma_state(tm, base + L::t0, base + L::t0 + KB * TILE, base + L::t0 + 2 * KB * TILE, vt, c > 0);
        tc::mma_commit(bars + 2);
      }
      __syncwarp();
    }
  }
  if (ok && chunks > 0) ok = tc::wait(bdone, (chunks - 1) & 1);
  tc::fence_after_sync();
  ok = __syncthreads_and(ok);
  if (ok) {
    const StatePart part(warp, lane);
    float d[StatePart::N];
    if (chunks > 0) {
      part.load(tm, warp, d);
    } else {
#pragma unroll
      for (int i = 0; i < StatePart::N; ++i) d[i] = 0.f;
    }
    float* dst = p.seg + ((size_t)unit * g.nseg + s + 1) * ((size_t)g.d_k * g.d_v);
#pragma unroll
    for (int i = 0; i < StatePart::N; ++i)
      if (part.row < g.d_k && part.col + i < cols) dst[(size_t)part.row * g.d_v + c0 + part.col + i] = d[i];
  } else if (tid == 0) {
    tc::settle();
    atomicExch(status, ATLAS_ERR_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tm, 64);
}

template <int NT, typename TO>
cudaError_t launch_out(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& my,
                       const Geom& g, const Ptrs& p, int* status, cudaStream_t st) {
  auto kern = k_decay_tc<NT, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<NT>::end);
  if (e != cudaSuccess) return e;
  return tc::launch_overlapped(kern, dim3(g.nseg, g.slices, g.B * g.H), dim3(NTHR), Smem<NT>::end, st, mq, mk, mv,
                               my, g, p, status);
}
cudaError_t launch_state(const CUtensorMap& mk, const CUtensorMap& mv, const Geom& g, const Ptrs& p, int* status,
                         cudaStream_t st) {
  auto kern = k_decay_tc_state;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemState::end);
  if (e != cudaSuccess) return e;
  return tc::launch_overlapped(kern, dim3(g.nseg - 1, g.slices, g.B * g.H), dim3(NTHR), SmemState::end, st, mk, mv,
                               g, p, status);
}

}  // namespace

namespace decay {

cudaError_t tc_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st) {
  if (g.d_k <= 64) return ws_launch(g, p, y_bf16, status, st);
  CUtensorMap mq, mk, mv, my;
  const int hq = g.H / g.share;
  if (!map_4d(&mq, p.q, true, g.dk_row, g.T, hq, g.B, g.qk_t, g.qk_h, g.qk_b) ||
      !map_4d(&mk, p.k, true, g.dk_row, g.T, hq, g.B, g.qk_t, g.qk_h, g.qk_b) ||
      !map_4d(&mv, p.v, true, g.dv_row, g.T, g.H, g.B, g.v_t, g.v_h, g.v_b) ||
      !map_4d(&my, p.y, y_bf16, g.dv_row, g.T, g.H, g.B, g.y_t, g.y_h, g.y_b))
    return cudaErrorInvalidValue;
  if (g.nseg > 1) {
    cudaError_t e = launch_state(mk, mv, g, p, status, st);
    if (e != cudaSuccess) return e;
    e = scan_launch(g, p, st);
    if (e != cudaSuccess) return e;
  }
  return y_bf16 ? launch_out<2, bf16>(mq, mk, mv, my, g, p, status, st)
                : launch_out<3, float>(mq, mk, mv, my, g, p, status, st);
}

}  // namespace decay
