// Decay attention on the tensor cores for d_k <= 64: the same products per
// chunk as k_decay_tc.cu, as a pipeline of specialised warps, one CTA per SM.
//
//   warp 0       TMA: q, k, v of a chunk (48 KB) into a ring of three stages; a
//                chunk's read-outs out of its stage before the next load into it
//   warp 1       MMAs, per chunk c: state product c, scores c + 1, P V c, Q S c
//   keys  (4)    K tile times decays -> three bf16 terms (w K)
//   probs (8)    scores of chunk c -> decays -> bf16 terms in TMEM; then the
//                read-outs of chunk c - 1: TMEM -> the stage's own q and k tiles
//   state (4)    the state in fp32 registers; its terms as the operand of Q S
//
// Only the state warps carry anything from chunk to chunk, so the others run
// ahead: the scores and keys of chunk c + 1 are formed while chunk c's products
// run.  TMEM: two score buffers (P's first two terms in place), inter and intra
// read-outs, the state's product (transposed, V^T (w K), in as many blocks of
// columns as there is room for: an MMA of N = 64 takes as long as one of 96),
// and the third term of P for fp32 read-outs.
// Measured, cycles per chunk and SM: 3900 for bf16 read-outs, 5200 for fp32 ones
// (MMAs 3300 of them), against 6300 in lock step (every warp doing each stage in
// turn, two CTAs per SM).  What is left is the chain of a chunk's products: the
// scores have to leave TMEM, be weighted and split before P V can start, and the
// stage is free only when its read-outs, formed in the q and k tiles, have left.
// 16 x 131072 tokens, d 64, fp32 y: 390 us (state pass 102, scan 7, read-outs
// 290); 4 x 8 x 4096, bf16: 34 us (33 with P in one term).
#include <algorithm>

#include "decay_tc_dev.cuh"

using namespace decay;
using layer::bf16;

namespace {

constexpr int NTHR = 18 * 32, STAGES = 3, STAGE = 3 * TILE;
// Most segments whose starts the read-out pass adds up itself.  It saves a launch,
// but a block waits for the sums of every segment before its own, one after the
// other: 3 segments (3 x 16 rows and heads, 8192 tokens) 78 us so, 82 with the
// scan as a launch; 4 segments (4 x 8, 4096 tokens) 33 / 34; 8 segments (1 x 16,
// 4096 tokens) 35 / 28.
constexpr int kInlineScan = 4;

template <int NT>
struct Smem {
  static constexpr int k0 = STAGES * STAGE, s = k0 + 3 * TILE, NS = NT == 2 ? 2 : 3, s_tile = 64 * 128,
                       pw = s + NS * s_tile, rev = pw + (C + 4) * 4, bars = rev + 32 * 4, end = bars + 24 * 8;
};

enum Bar { FULL = 0, SC = 3, P = 5, K = 7, DS, DSFREE, S, PV, Y, YFREE, OUT, NBARS };

// 8 of a token's keys (16-byte chunk j of row r), times w, in three terms
__device__ __forceinline__ void scale_chunk(uint32_t src, uint32_t dst, int r, int j, float w, bool live) {
  uint32_t x[4], y[4][3];
  lds128(src + swz(r, j), x);
#pragma unroll
  for (int i = 0; i < 4; ++i) split_pair<3>(mul_pair(widen(live ? x[i] : 0u), pair(w, w)), y[i]);
#pragma unroll
  for (int t = 0; t < 3; ++t) sts128(dst + t * TILE + swz(r, j), y[0][t], y[1][t], y[2][t], y[3][t]);
}
// V^T (w K) into TMEM at d, rows d_v, columns d_k, in BLOCKS blocks of 64
// columns: 3: a block per term, one MMA of N = 192 per 16 tokens; 2: term 0,
// then terms 1 and 2; 1: all three.  The sum of the blocks is the product.
template <int BLOCKS>
__device__ __forceinline__ void mma_state_t(uint32_t d, uint32_t keys, uint32_t vtile, bool accumulate) {
  const uint64_t vd = tc::sdesc_sw128(vtile, TILE), kd = tc::sdesc_sw128(keys, TILE);
  const uint32_t wide = tc::idesc_f16(64, 64 * BLOCKS, 1, 1, 1), one = tc::idesc_f16(64, 64, 1, 1, 1);
  auto term = [&](int t, uint32_t at, uint32_t idesc, bool acc) {
#pragma unroll
    for (int s = 0; s < C / 16; ++s)
      tc::mma_f16(at, vd + s * (2048 >> 4), kd + (t * TILE >> 4) + s * (2048 >> 4), idesc, (acc || s > 0) ? 1u : 0u);
  };
  if constexpr (BLOCKS == 3) {
    term(0, d, wide, accumulate);
  } else if constexpr (BLOCKS == 2) {
    term(0, d, wide, accumulate);
    term(2, d + 64, one, true);
  } else {
    term(2, d, one, accumulate);
    term(1, d, one, true);
    term(0, d, one, true);
  }
}
__device__ __forceinline__ void zero_row(uint32_t tile, int r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) sts128(tile + r * 128 + 16 * j, 0, 0, 0, 0);
}

template <int NT, typename TO>
__global__ void __launch_bounds__(NTHR, 1)
    k_decay_ws(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap my, Geom g, Ptrs p,
               int inline_scan, int* status) {
  using L = Smem<NT>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  float* pw = reinterpret_cast<float*>(sm + L::pw);      // g^0 .. g^128
  float* rev = reinterpret_cast<float*>(sm + L::rev);    // g^31 .. g^0
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint32_t* tbase = reinterpret_cast<uint32_t*>(bars + NBARS);
  int* failed = reinterpret_cast<int*>(bars + NBARS + 1);
  const uint32_t bar0 = tc::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };
  const int s = blockIdx.x, sl = blockIdx.y, unit = blockIdx.z;
  const int b = unit / g.H, h = unit % g.H, hq = h / g.share;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, quarter = warp & 3, group = (warp - 2) >> 2;
  if (warp == 0) tc::tmem_alloc(tbase, 512);
  if (tid == 32) {
    for (int i = 0; i < NBARS; ++i) {
      const bool four = i == K || i == DSFREE || i == S, eight = i == P || i == P + 1 || i == YFREE || i == OUT;
      tc::mbar_init_only(bars + i, eight ? 8 : four ? 4 : 1);
    }
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
  // All 512 columns: they start at 0.  As a constant (and not as read back) the
  // MMAs' operands stay in uniform registers.
  constexpr uint32_t tm = 0;
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();

  const int live = live_tokens(g, p, b);
  const int t_lo = s * g.seg, t_hi = min(g.T, t_lo + g.seg), t_live = min(t_hi, max(live, t_lo));
  const int chunks = (t_live - t_lo + C - 1) / C;
  const int c0 = sl * SL, cols = min(SL, g.d_v - c0);
  const size_t sq = (size_t)g.d_k * g.d_v;
  const float l2g = log2f(p.decay[h]);
  for (int i = tid; i <= C; i += NTHR) pw[i] = power(l2g, i);
  if (tid < 32) rev[tid] = power(l2g, 31 - tid);
  __syncthreads();
  bool ok = *failed == 0 && *tbase == tm;
  constexpr uint32_t tSC = tm, tY1 = tm + 256, tY2 = tm + 320, tDS = tm + 384, tP2 = tm + 448;   // tP2: NT = 3
  auto all_wait = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, tc::wait(bar(i), parity)); };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + i);
  };
  auto tokens = [&](int c) { return min(C, t_live - t_lo - c * C); };

  if (warp == 0) {
    auto load = [&](int c) {
      const uint32_t at = base + (c % STAGES) * STAGE, full = bar(FULL + c % STAGES);
      const int t0 = t_lo + c * C;
      tc::expect_tx(full, STAGE);
      load_4d(at, &mq, 0, t0, hq, b, full);
      load_4d(at + TILE, &mk, 0, t0, hq, b, full);
      load_4d(at + 2 * TILE, &mv, c0, t0, h, b, full);
    };
    if (ok && tc::elect())
      for (int c = 0; c < min(chunks, STAGES); ++c) load(c);
    __syncwarp();
    for (int c = 0; c < chunks && ok; ++c) {
      if (!(ok = all_wait(OUT, c & 1))) break;
      if (tc::elect()) {
        const uint32_t at = base + (c % STAGES) * STAGE;
        store_4d(&my, c0, t_lo + c * C, h, b, at);
        if (sizeof(TO) == 4 && cols > 32) store_4d(&my, c0 + 32, t_lo + c * C, h, b, at + TILE);
        tc::bulk_commit();
        tc::bulk_wait_read<0>();
        if (c + STAGES < chunks) load(c + STAGES);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    auto scores = [&](int c) {
      if (!(ok = all_wait(FULL + c % STAGES, (c / STAGES) & 1))) return;
      if (tc::elect()) {
        const uint32_t at = base + (c % STAGES) * STAGE, idesc = tc::idesc_f16(C, C, 1, 0, 0);
        const uint64_t qd = tc::sdesc_sw128(at), kd = tc::sdesc_sw128(at + TILE);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc::mma_f16(tSC + 128 * (c & 1), qd + ks * (32 >> 4), kd + ks * (32 >> 4), idesc, ks > 0 ? 1u : 0u);
        tc::mma_commit(bars + SC + (c & 1));
      }
      __syncwarp();
    };
    if (ok && chunks > 0) scores(0);
    for (int c = 0; c < chunks && ok; ++c) {
      const uint32_t at = base + (c % STAGES) * STAGE, vt = at + 2 * TILE;
      // scores of the next chunk, where P of the one before was
      auto next_scores = [&]() {
        if (c + 1 >= chunks) return;
        if (c > 0 && !(ok = all_wait(PV, (c - 1) & 1))) return;
        tc::fence_after_sync();
        scores(c + 1);
      };
      // state product: the keys' terms are there, the last product has been taken
      auto state_product = [&]() {
        if (!(ok = all_wait(K, c & 1) && (c == 0 || all_wait(DSFREE, (c - 1) & 1)))) return;
        tc::fence_after_sync();
        if (tc::elect()) {
          mma_state_t<NT == 2 ? 2 : 1>(tDS, base + L::k0, vt, false);
          tc::mma_commit(bars + DS);
        }
        __syncwarp();
      };
      // NT = 3 holds its stages longer, so the next chunk's copies come later:
      // scores first cost it 3 % (417 against 405 us at 16 x 131072 tokens); NT = 2
      // waits for the keys instead (36 against 34 us at 32 x 4096 tokens)
      if constexpr (NT == 2) {
        next_scores();
        if (ok) state_product();
      } else {
        state_product();
        if (ok) next_scores();
      }
      if (!ok) break;
      if (!(ok = all_wait(P + (c & 1), (c >> 1) & 1) && (c == 0 || all_wait(YFREE, (c - 1) & 1)))) break;
      tc::fence_after_sync();
      const uint32_t idesc = tc::idesc_f16(C, SL, 1, 0, 1), idesc_s = tc::idesc_f16(C, SL, 1, 0, 0);
      if (tc::elect()) {
        const uint64_t vd = tc::sdesc_sw128(vt, TILE);
#pragma unroll
        for (int k = NT - 1; k >= 0; --k)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(tY2, k < 2 ? tSC + 128 * (c & 1) + 16 * ks + 8 * k : tP2 + 8 * ks, vd + ks * (2048 >> 4), idesc,
                   (k < NT - 1 || ks > 0) ? 1u : 0u);
        tc::mma_commit(bars + PV);
      }
      __syncwarp();
      if (!(ok = all_wait(S, c & 1))) break;
      tc::fence_after_sync();
      if (tc::elect()) {
        const uint64_t qd = tc::sdesc_sw128(at);
#pragma unroll
        for (int i = L::NS - 1; i >= 0; --i) {   // the smallest terms first
          const uint64_t sd = tc::sdesc_sw128(base + L::s + i * L::s_tile);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_f16(tY1, qd + ks * (32 >> 4), sd + ks * (32 >> 4), idesc_s, (i < L::NS - 1 || ks > 0) ? 1u : 0u);
        }
        tc::mma_commit(bars + Y);
      }
      __syncwarp();
    }
  } else if (group == 0) {
    // keys: one token per thread
    const int r = 32 * quarter + lane;
    for (int c = 0; c < chunks; ++c) {
      const uint32_t at = base + (c % STAGES) * STAGE;
      const int n = tokens(c);
      const float w = r < n ? pw[n - 1 - r] : 0.f;
      if (!(ok = all_wait(FULL + c % STAGES, (c / STAGES) & 1) && (c == 0 || all_wait(DS, (c - 1) & 1)))) break;
#pragma unroll 2
      for (int j = 0; j < 8; ++j) scale_chunk(at + TILE, base + L::k0, r, j, w, r < n);
      // a token past the row's length: 0 * NaN must not reach the sums
      if (r >= n) zero_row(at + 2 * TILE, r);
      tc::fence_smem_to_async();
      arrive(K);
    }
  } else if (group <= 2) {
    // probs: 32 x 32 blocks of a warp's 32 rows, 0 and 3 or 1 and 2 of the four
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int row = 32 * quarter + lane, side = group - 1;
    // the read-outs of chunk c, this warp's 32 tokens and half of the columns
    auto reads = [&](int c) {
      if (!(ok = all_wait(Y, c & 1))) return;
      tc::fence_after_sync();
      const float f = pw[row + 1] * g.scale, sc = g.scale;
      const bool dead = row >= tokens(c);
      const uint32_t out = base + (c % STAGES) * STAGE;
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {   // 16 columns at a time
        float yi[16], ya[16];
        tc::tmem_ld16(tY1 + lanes + 32 * side + 16 * part, yi);
        tc::tmem_ld16(tY2 + lanes + 32 * side + 16 * part, ya);
        tc::tmem_ld_wait16(yi);
        tc::tmem_ld_wait16(ya);
        if (part == 1) {
          tc::fence_before_sync();
          arrive(YFREE);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2)
          unpair(fma_pair(pair(yi[i], yi[i + 1]), pair(f, f), mul_pair(pair(ya[i], ya[i + 1]), pair(sc, sc))), ya[i],
                 ya[i + 1]);
        if (dead) {
#pragma unroll
          for (int i = 0; i < 16; ++i) ya[i] = 0.f;
        }
        if constexpr (sizeof(TO) == 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            sts128(out + swz(row, 4 * side + 2 * part + j), layer::pack_bf16(ya[8 * j], ya[8 * j + 1]),
                   layer::pack_bf16(ya[8 * j + 2], ya[8 * j + 3]), layer::pack_bf16(ya[8 * j + 4], ya[8 * j + 5]),
                   layer::pack_bf16(ya[8 * j + 6], ya[8 * j + 7]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sts128(out + side * TILE + swz(row, 4 * part + j), __float_as_uint(ya[4 * j]),
                   __float_as_uint(ya[4 * j + 1]), __float_as_uint(ya[4 * j + 2]), __float_as_uint(ya[4 * j + 3]));
        }
      }
      tc::fence_smem_to_async();
      arrive(OUT);
    };
    for (int c = 0; c < chunks; ++c) {
      const uint32_t sc = tSC + 128 * (c & 1) + lanes;
      // the scores; the third term's columns are the last chunk's until its P V is done
      if (!(ok = all_wait(SC + (c & 1), (c >> 1) & 1) && (NT == 2 || c == 0 || all_wait(PV, (c - 1) & 1)))) break;
      tc::fence_after_sync();
      // 16 columns a turn: with everything unrolled the kernel's code overran the
      // instruction caches (4.6 of 11 cycles per instruction were spent on that)
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {
        const int blk = side == 0 ? 3 * (u >> 1) : 1 + (u >> 1), h0 = 16 * (u & 1);   // columns 32 blk + h0 ..
        uint32_t w[8][NT];
        if (blk > quarter) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < NT; ++k) w[i][k] = 0u;
        } else {
          float v[16];
          tc::tmem_ld16(sc + 32 * blk + h0, v);
          tc::tmem_ld_wait16(v);
          if (blk < quarter) {
            const float f = pw[row - 32 * blk - 31];   // times g^{31 - column}
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float4 d = *reinterpret_cast<const float4*>(rev + h0 + 2 * i);
              split_pair<NT>(mul_pair(pair(v[2 * i], v[2 * i + 1]), mul_pair(pair(d.x, d.y), pair(f, f))), w[i]);
              split_pair<NT>(mul_pair(pair(v[2 * i + 2], v[2 * i + 3]), mul_pair(pair(d.z, d.w), pair(f, f))), w[i + 1]);
            }
          } else {
            const int gap = lane - h0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = gap >= 2 * i ? v[2 * i] * pw[max(0, gap - 2 * i)] : 0.f;
              const float y = gap >= 2 * i + 1 ? v[2 * i + 1] * pw[max(0, gap - 2 * i - 1)] : 0.f;
              split2<NT>(x, y, w[i]);
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = w[i][k];
          // terms 0 and 1 over the halves of the 16 columns just read
          tmem_st8u(k < 2 ? sc + 32 * blk + h0 + 8 * k : tP2 + lanes + 16 * blk + h0 / 2, x);
        }
      }
      if (!ok) break;
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(P + (c & 1));
      if (c > 0) {
        reads(c - 1);
        if (!ok) break;
      }
    }
    if (ok && chunks > 0) reads(chunks - 1);
    if (ok) {
      // read-outs past the row's length: whole chunks (the last live chunk wrote its own)
      TO* y = (TO*)p.y + b * g.y_b + h * g.y_h + c0 + 32 * side;
      for (int t = t_lo + chunks * C + row / 32; t < t_hi; t += 4)
        if (32 * side + lane < cols) y[t * g.y_t + lane] = layer::from_f32<TO>(0.f);
    }
  } else {
    // state, transposed: column 16 quarter + lane % 16 of d_v, rows 16 (lane /
    // 16) + 32 i of d_k
    const int row = 16 * quarter + lane % 16, col = 16 * (lane / 16);
    const uint32_t at = tDS + ((uint32_t)(32 * quarter) << 16);
    float st[32];
    auto element = [&](int i) { return (size_t)(col + 32 * (i / 16) + i % 16) * g.d_v + c0 + row; };
    auto inside = [&](int i) { return row < cols && col + 32 * (i / 16) + i % 16 < g.d_k; };
    {
      // start = S0 carried over the segments before this one; S0 from its copy in
      // the workspace, since the last segment's block may have written S_out, the
      // same array, by now
      const bool add = g.nseg > 1 && inline_scan;
      const float* d = g.nseg == 1 ? (p.S0 ? p.S0 + unit * sq : nullptr)
                       : add && !p.S0 ? nullptr : p.seg + ((size_t)unit * g.nseg + (add ? 0 : s)) * sq;
#pragma unroll
      for (int i = 0; i < 32; ++i) st[i] = d && inside(i) ? d[element(i)] : 0.f;
      for (int e = 0; add && e < s; ++e) {
        const float f = power(l2g, min(g.seg, max(0, live - e * g.seg)));
        const float* x = p.seg + ((size_t)unit * g.nseg + e + 1) * sq;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = inside(i) ? x[element(i)] : 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) st[i] = fmaf(f, st[i], v[i]);
      }
    }
    auto tiles = [&]() {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t w[4][L::NS];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2<L::NS>(st[i + 2 * j], st[i + 2 * j + 1], w[j]);
#pragma unroll
        for (int n = 0; n < L::NS; ++n)
          sts128(base + L::s + n * L::s_tile + swz(row, (col + 32 * (i / 16) + i % 16) / 8), w[0][n], w[1][n], w[2][n],
                 w[3][n]);
      }
      tc::fence_smem_to_async();
      arrive(S);
    };
    if (chunks > 0) tiles();
    for (int c = 0; c < chunks; ++c) {
      if (!(ok = all_wait(DS, c & 1))) break;
      tc::fence_after_sync();
      {
        const float f = pw[tokens(c)];
#pragma unroll
        for (int t = (NT == 2 ? 1 : 0); t >= 0; --t) {   // the product's blocks
          float d[32];
          tc::tmem_ld16_x2(at + 64 * t, d);
          tc::tmem_ld16_x2(at + 64 * t + 32, d + 16);
          tc::tmem_ld_wait32(d);
          if (t == (NT == 2 ? 1 : 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) st[i] = fmaf(f, st[i], d[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) st[i] += d[i];
          }
        }
        tc::fence_before_sync();
        arrive(DSFREE);
      }
      if (c + 1 < chunks) {
        if (!(ok = all_wait(Y, c & 1))) break;   // Q S has read the last terms
        tiles();
      }
    }
    if (ok && s == g.nseg - 1 && p.S_out) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (inside(i)) p.S_out[unit * sq + element(i)] = st[i];
    }
  }
  if (!ok && lane == 0) atomicExch(failed, 1);
  tc::fence_before_sync();
  __syncthreads();
  if (*failed && tid == 0) {
    tc::settle();
    atomicExch(status, ATLAS_ERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tm, 512);
}

// A segment's own contribution to the state at its end: weights counted to
// that end, the product accumulated in TMEM over the whole segment.  Two groups
// of four key warps take chunks in turn, each with its own terms.
struct SmemState {
  static constexpr int stage = 2 * TILE, k0 = STAGES * stage, bars = k0 + 6 * TILE, end = bars + 16 * 8;
};
constexpr int NTHR_STATE = 10 * 32;
enum BarState { SFULL = 0, SEMPTY = 3, SK = 6, SFREE = 8, NSBARS = 10 };

__global__ void __launch_bounds__(NTHR_STATE, 1)
    k_decay_ws_state(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, Geom g, Ptrs p,
                     int* status) {
  using L = SmemState;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint32_t* tbase = reinterpret_cast<uint32_t*>(bars + NSBARS);
  int* failed = reinterpret_cast<int*>(bars + NSBARS + 1);
  const uint32_t bar0 = tc::smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };
  const int s = blockIdx.x, sl = blockIdx.y, unit = blockIdx.z;
  const int b = unit / g.H, h = unit % g.H, hq = h / g.share;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, quarter = warp & 3, group = (warp - 2) >> 2;
  if (warp == 0) tc::tmem_alloc(tbase, 256);
  if (tid == 32) {
    for (int i = 0; i < NSBARS; ++i) tc::mbar_init_only(bars + i, i == SK || i == SK + 1 ? 4 : 1);
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

  const int live = live_tokens(g, p, b);
  const int t_lo = s * g.seg, t_hi = min(g.T, t_lo + g.seg), t_live = min(t_hi, max(live, t_lo));
  const int c0 = sl * SL, cols = min(SL, g.d_v - c0), chunks = (t_live - t_lo + C - 1) / C;
  bool ok = *failed == 0;
  auto all_wait = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, tc::wait(bar(i), parity)); };
  if (warp == 0) {
    for (int c = 0; c < chunks && ok; ++c) {
      const int st = c % STAGES;
      if (c >= STAGES && !(ok = all_wait(SEMPTY + st, (c / STAGES - 1) & 1))) break;
      if (tc::elect()) {
        const uint32_t at = base + st * L::stage, full = bar(SFULL + st);
        tc::expect_tx(full, L::stage);
        load_4d(at, &mk, 0, t_lo + c * C, hq, b, full);
        load_4d(at + TILE, &mv, c0, t_lo + c * C, h, b, full);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    for (int c = 0; c < chunks; ++c) {
      if (!(ok = all_wait(SK + (c & 1), (c >> 1) & 1))) break;
      tc::fence_after_sync();
      if (tc::elect()) {
        const uint32_t k0 = base + L::k0 + (c & 1) * 3 * TILE;
        mma_state_t<3>(tm, k0, base + (c % STAGES) * L::stage + TILE, c > 0);
        tc::mma_commit(bars + SFREE + (c & 1));
        tc::mma_commit(bars + SEMPTY + c % STAGES);
      }
      __syncwarp();
    }
  } else {
    const int r = 32 * quarter + lane;
    const int row = 16 * quarter + lane % 16, col = 16 * (lane / 16);   // a thread's column of d_v, rows of d_k
    auto element = [&](int i) { return col + 32 * (i / 16) + i % 16; };
    auto inside = [&](int i) { return row < cols && element(i) < g.d_k; };
    const size_t sq = (size_t)g.d_k * g.d_v;
    const float l2g = log2f(p.decay[h]);
    for (int c = group; c < chunks; c += 2) {
      const int t0 = t_lo + c * C, n = min(C, t_live - t0);
      const uint32_t at = base + (c % STAGES) * L::stage, k0 = base + L::k0 + (c & 1) * 3 * TILE;
      const float w = r < n ? power(l2g, t_live - 1 - t0 - r) : 0.f;
      // the terms' buffer first: chunk c - 2's product done means that the loads
      // up to chunk c - 2 have landed, so the stage's parity below is the one of
      // this chunk's load or the one before it
      if (!(ok = (c < 2 || all_wait(SFREE + (c & 1), ((c >> 1) - 1) & 1)) && all_wait(SFULL + c % STAGES, (c / STAGES) & 1)))
        break;
#pragma unroll 2
      for (int j = 0; j < 8; ++j) scale_chunk(at, k0, r, j, w, r < n);
      if (r >= n) zero_row(at + TILE, r);
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + SK + (c & 1));
    }
    // the sums, by the group of the last chunk
    if (ok && chunks > 0 && group == ((chunks - 1) & 1)) {
      ok = all_wait(SFREE + ((chunks - 1) & 1), ((chunks - 1) >> 1) & 1);
      tc::fence_after_sync();
    }
    if (ok && group == (chunks > 0 ? (chunks - 1) & 1 : 0)) {
      float sum[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[i] = 0.f;
      if (chunks > 0) {
        const uint32_t ta = tm + ((uint32_t)(32 * quarter) << 16);
#pragma unroll
        for (int t = 2; t >= 0; --t) {
          float d[32];
          tc::tmem_ld16_x2(ta + 64 * t, d);
          tc::tmem_ld16_x2(ta + 64 * t + 32, d + 16);
          tc::tmem_ld_wait32(d);
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[i] += d[i];
        }
      }
      float* dst = p.seg + ((size_t)unit * g.nseg + s + 1) * sq + c0 + row;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (inside(i)) dst[(size_t)element(i) * g.d_v] = sum[i];
    } else if (ok && s == 0 && p.S0 && g.nseg <= kInlineScan) {   // S0 to slot 0, by the other group
      const float* src = p.S0 + unit * sq + c0 + row;
      float* dst = p.seg + (size_t)unit * g.nseg * sq + c0 + row;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = inside(i) ? src[(size_t)element(i) * g.d_v] : 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (inside(i)) dst[(size_t)element(i) * g.d_v] = v[i];
    }
  }
  if (!ok && lane == 0) atomicExch(failed, 1);
  tc::fence_before_sync();
  __syncthreads();
  if (*failed && tid == 0) {
    tc::settle();
    atomicExch(status, ATLAS_ERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tm, 256);
}

template <int NT, typename TO>
cudaError_t launch_out(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& my,
                       const Geom& g, const Ptrs& p, int inline_scan, int* status, cudaStream_t st) {
  auto kern = k_decay_ws<NT, TO>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<NT>::end);
  if (e != cudaSuccess) return e;
  return tc::launch_overlapped(kern, dim3(g.nseg, g.slices, g.B * g.H), dim3(NTHR), Smem<NT>::end, st, mq, mk, mv, my,
                               g, p, inline_scan, status);
}

}  // namespace

namespace decay {

cudaError_t ws_launch(const Geom& g, const Ptrs& p, bool y_bf16, int* status, cudaStream_t st) {
  CUtensorMap mq, mk, mv, my;
  const int hq = g.H / g.share;
  if (!map_4d(&mq, p.q, true, g.dk_row, g.T, hq, g.B, g.qk_t, g.qk_h, g.qk_b) ||
      !map_4d(&mk, p.k, true, g.dk_row, g.T, hq, g.B, g.qk_t, g.qk_h, g.qk_b) ||
      !map_4d(&mv, p.v, true, g.dv_row, g.T, g.H, g.B, g.v_t, g.v_h, g.v_b) ||
      !map_4d(&my, p.y, y_bf16, g.dv_row, g.T, g.H, g.B, g.y_t, g.y_h, g.y_b))
    return cudaErrorInvalidValue;
  int inline_scan = 1;
  if (g.nseg > 1) {
    cudaError_t e = cudaFuncSetAttribute(k_decay_ws_state, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemState::end);
    if (e != cudaSuccess) return e;
    e = tc::launch_overlapped(k_decay_ws_state, dim3(g.nseg - 1, g.slices, g.B * g.H), dim3(NTHR_STATE), SmemState::end,
                              st, mk, mv, g, p, status);
    if (e != cudaSuccess) return e;
    if (g.nseg > kInlineScan) {
      inline_scan = 0;
      e = scan_launch(g, p, st);
      if (e != cudaSuccess) return e;
    }
  }
  return y_bf16 ? launch_out<2, bf16>(mq, mk, mv, my, g, p, inline_scan, status, st)
                : launch_out<3, float>(mq, mk, mv, my, g, p, inline_scan, status, st);
}

}  // namespace decay
