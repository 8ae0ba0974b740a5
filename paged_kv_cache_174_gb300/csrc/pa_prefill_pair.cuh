// pa_prefill_pair.cuh -- the products and the softmax of a unit of two query
// tiles (the sliding-window prefill with many query tiles); included by
// pa_prefill_kernel.cuh, whose producers load the pair's queries, keys and
// values.
//
// A unit of one query tile is paced by bringing each key tile to the SM (64 KB
// for 2 x 128 x 128 x head_dim multiply-adds) and by one tile at a time in the
// softmax, whose eight warps wait for one another.  Here two query tiles of
// consecutive tokens share every K and V tile, half the bytes for the same
// products, and each has four softmax warps of its own, a row to a thread, so
// neither tile's softmax waits for the other's and no row is split.  A key tile
// is taken in halves of 64 keys: TMEM then holds two S / P buffers for each
// query tile beside its O accumulator (4 x 64 + 2 x head_dim columns), so the
// scores of the next half are ready when a softmax warp comes for them.  The S
// product pays for it, 48 cycles per 64 columns against 64 per 128 (it is bound
// by its shared-memory operand there).
//
// What it measured on the way (an 8192-token prompt, a 4096-token window, 32 q /
// 8 kv heads of 128, bf16; single tiles take 538 us):
//  * both halves' code unrolled, 781 us: the loop did not fit the instruction
//    cache, and every phase of the softmax took half as long again;
//  * one thread issuing S for both query tiles and one issuing P V, 562 us: a
//    thread spends as long on the wait before and the commit after a product
//    as on its issue, so the four products of a step now have an issuer for
//    each query tile, 492 us;
//  * no key bits where a whole step is seen by every row, 477 us (without any
//    exponential it would then have taken 452 us, so the products' hand-offs
//    pace it more than the softmax's arithmetic);
//  * output rows through shared memory, and the unit's place found with 32-bit
//    divisions: 451 us, 1143 TFLOP/s.
// With the 8-bit cache the producers' conversion paces it.
//
// Buffer b = 2 * half + query tile.  A half is one "step"; with one query tile
// in the unit (an odd number of them) the other's buffers rest.
#pragma once

namespace pa {
namespace {

constexpr int kHalfKeys = kKeysPerTile / 2;
constexpr int kPairOCol = 4 * kHalfKeys;  // O of query tile q at kPairOCol + q * D

// Waits until *count, which only grows, has reached n (bounded as mbar_wait).
__device__ __forceinline__ void wait_count(const uint32_t* count, uint32_t n, unsigned* err,
                                           volatile int* abort) {
  const uint32_t at = smem_addr(count);
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t c;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(c) : "r"(at) : "memory");
    if (c >= n) return;
    if ((it & 63u) == 0) {
      if (*abort) return;
      const unsigned long long t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *abort = 1;
        flag_error(err, DEVERR_TIMEOUT);
        return;
      }
    }
  }
}

// Steps of key tile kt: halves that hold a page.
__device__ __forceinline__ int pair_steps(const Unit& U, int kt) {
  return U.pages - kt * kPagesPerTile > kPagesPerTile / 2 ? 2 : 1;
}

// Issues S = Q K^T of every step of query tile q (one thread).
template <int D, int TM, bool F8, class Cursor>
__device__ __forceinline__ void pair_issue_s(const PrefillParams& p, PrefillShared& B, Cursor& cur,
                                             long long total_units, uint32_t tmem, uint32_t q_s,
                                             uint32_t k_s, int q) {
  constexpr int NH = D / 64;
  constexpr uint32_t HALF = kRows * 128;
  constexpr uint32_t TILE = NH * HALF;
  constexpr uint32_t IDESC = F8 ? tc::idesc_f16_f32(kRows, kHalfKeys, 0, 0)
                                : tc::idesc_bf16_f32(kRows, kHalfKeys, 0, 0);
  volatile int* abort_flag = &B.abort_flag;
  const tc::Desc qd = tc::sw128_desc_pair(q_s + q * TILE, 16, 1024);
  const tc::Desc kd = tc::sw128_desc_pair(k_s, 16, 1024);
  Ring kv;
  uint32_t used0 = 0, used1 = 0;  // products issued into this tile's two buffers
  int n_out = 0;
  for (long long u = blockIdx.x; u < total_units; u += gridDim.x) {
    Unit U;
    if (!cur.locate(p, u, U)) break;
    const bool on = q == 0 || U.ntok > TM;
    // this unit's Q: the last unit's load was waited for here, and the next
    // load waits for q_empty, which this thread arrives on
    mbar_wait_spin(smem_addr(&B.q_full), n_out & 1, p.err, abort_flag);
    for (int kt = U.kt0; kt < U.kt1; ++kt) {
      // K tile kt: this thread waited for the stage's last use, and the
      // stage's next copy waits for k_empty, arrived on below
      mbar_wait_spin(smem_addr(&B.k_full[kv.stage]), kv.phase, p.err, abort_flag);
      if (!on) {  // no second query tile: only release the stage
        mbar_arrive(smem_addr(&B.k_empty[kv.stage]));
        kv.next(2);
        continue;
      }
      const int steps = pair_steps(U, kt);
#pragma unroll 1
      for (int half = 0; half < steps; ++half) {
        const int b = 2 * half + q;
        // P V of the step that last used this buffer: the one before on the
        // buffer was waited for here, and the next needs the P of the S
        // about to be issued into it
        const uint32_t used = half ? used1 : used0;
        if (used > 0)
          mbar_wait_spin(smem_addr(&B.pv_done[b]), (used - 1) & 1, p.err, abort_flag);
        tc::fence_after_sync();
        const uint32_t d = tmem + b * kHalfKeys;
        const uint32_t b_at = kv.stage * (TILE >> 4) + ((half * kHalfKeys * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
          if (kk == 0)
            tc::mma_bf16_pair<false>(d, qd, off, kd, b_at + off, IDESC);
          else
            tc::mma_bf16_pair<true>(d, qd, off, kd, b_at + off, IDESC);
        }
        tc::commit(smem_addr(&B.s_full[b]));
        if (half)
          ++used1;
        else
          ++used0;
      }
      tc::commit(smem_addr(&B.k_empty[kv.stage]));
      kv.next(2);
    }
    if (on)
      tc::commit(smem_addr(&B.q_empty));
    else
      mbar_arrive(smem_addr(&B.q_empty));
    ++n_out;
  }
  if (n_out > 0) {
    tc::commit(smem_addr(&B.s_done[q]));  // its only use: phase 0
    mbar_wait_spin(smem_addr(&B.s_done[q]), 0, p.err, abort_flag);
  }
}

// Issues O += P V of every step of query tile q (one thread).
template <int D, int TM, bool F8, class Cursor>
__device__ __forceinline__ void pair_issue_pv(const PrefillParams& p, PrefillShared& B,
                                              Cursor& cur, long long total_units, uint32_t tmem,
                                              uint32_t v_s, int q) {
  constexpr uint32_t V_PAGE = (D / 64) * kBlock * 128;
  constexpr uint32_t TILE = kPagesPerTile * V_PAGE;
  constexpr uint32_t IDESC =
      F8 ? tc::idesc_f16_f32(kRows, D, 0, 1) : tc::idesc_bf16_f32(kRows, D, 0, 1);
  volatile int* abort_flag = &B.abort_flag;
  const tc::Desc vd = tc::sw128_desc_pair(v_s, kBlock * 128, 1024);
  const uint32_t o = tmem + kPairOCol + q * D;
  Ring kv;
  uint32_t used0 = 0, used1 = 0;  // products issued from this tile's two buffers
  uint32_t outs = 0;              // O tiles finished
  uint32_t landed = 0;            // V tiles waited for
  for (long long u = blockIdx.x; u < total_units; u += gridDim.x) {
    Unit U;
    if (!cur.locate(p, u, U)) break;
    const bool on = q == 0 || U.ntok > TM;
    for (int kt = U.kt0; kt < U.kt1; ++kt) {
      // V tile kt: the stage's last use was waited for here, and its next copy
      // waits for v_empty, arrived on below
      mbar_wait_spin(smem_addr(&B.v_full[kv.stage]), kv.phase, p.err, abort_flag);
      ++landed;
      asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_addr(&B.v_landed[q])),
                   "r"(landed)
                   : "memory");
      if (!on) {  // no second query tile: only release the stage
        mbar_arrive(smem_addr(&B.v_empty[kv.stage]));
        kv.next(2);
        continue;
      }
      const int steps = pair_steps(U, kt);
#pragma unroll 1
      for (int half = 0; half < steps; ++half) {
        const int b = 2 * half + q;
        const bool first = kt == U.kt0 && half == 0;
        // P of this step: the buffer's last P was waited for here, and its
        // next P needs an S that waits for this P V (pv_done)
        mbar_wait_spin(smem_addr(&B.p_full[b]), (half ? used1 : used0) & 1, p.err, abort_flag);
        // the query tile's last O read out: the release before was waited for
        // here, and the next needs this unit's O (o_full)
        if (first && outs > 0)
          mbar_wait_spin(smem_addr(&B.o_empty[q]), (outs - 1) & 1, p.err, abort_flag);
        tc::fence_after_sync();
        const uint32_t pp = tmem + b * kHalfKeys;
        const uint32_t v_at = (kv.stage * TILE + half * (kPagesPerTile / 2) * V_PAGE) >> 4;
        if (first)
          tc::mma_bf16_tmem_a_pair<false>(o, pp, vd, v_at, IDESC);
        else
          tc::mma_bf16_tmem_a_pair<true>(o, pp, vd, v_at, IDESC);
#pragma unroll
        for (int kk = 1; kk < kPagesPerTile / 2; ++kk)
          tc::mma_bf16_tmem_a_pair<true>(o, pp + kk * 8, vd, v_at + ((kk * V_PAGE) >> 4), IDESC);
        tc::commit(smem_addr(&B.pv_done[b]));
        if (half)
          ++used1;
        else
          ++used0;
      }
      tc::commit(smem_addr(&B.v_empty[kv.stage]));
      kv.next(2);
    }
    if (on) {
      tc::commit(smem_addr(&B.o_full[q]));
      ++outs;
    }
  }
  if (outs > 0) {
    tc::commit(smem_addr(&B.pv_done_all[q]));  // its only use: phase 0
    mbar_wait_spin(smem_addr(&B.pv_done_all[q]), 0, p.err, abort_flag);
  }
}

// Softmax and output: warps 2-5 for the first query tile, 6-9 for the second,
// a row to a thread.
template <int D, int G, bool F8, class Cursor>
__device__ __forceinline__ void pair_softmax(const PrefillParams& p, PrefillShared& B, Cursor& cur,
                                             long long total_units, uint32_t tmem,
                                             unsigned char* v_s, unsigned char* out_s, int warp,
                                             int lane) {
  constexpr int TM = kRows / G;
  constexpr int NH = D / 64;
  constexpr uint32_t V_PAGE = NH * kBlock * 128;
  constexpr uint32_t TILE = kPagesPerTile * V_PAGE;
  volatile int* abort_flag = &B.abort_flag;
  const int q = (warp - 2) >> 2;
  const int quarter = warp & 3;  // TMEM lanes 32*quarter .. +31
  const int r = quarter * 32 + lane;
  const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
  const int tl = q * TM + r / G, hl = r % G;  // the row's token in the unit, its head
  const float sl2 = p.scale_log2;
  // with a positive scale the max of the raw scores gives the max of the
  // scaled ones and the scale folds into the exponent's FMA; otherwise the
  // scores are scaled first
  const bool pos_scale = sl2 > 0.f;
  const float mul = pos_scale ? 1.f : sl2;
  const float emul = pos_scale ? sl2 : 1.f;
  const uint32_t o_cols = tmem + lane_addr + kPairOCol + q * D;
  uint32_t vt = 0;  // key tiles of all units so far
  uint32_t used0 = 0, used1 = 0;  // steps done in this tile's two buffers
  uint32_t n_out = 0;
  for (long long u = blockIdx.x; u < total_units; u += gridDim.x) {
    Unit U;
    if (!cur.locate(p, u, U)) break;
    if (q && U.ntok <= TM) {  // no second query tile in this unit
      vt += U.kt1 - U.kt0;
      continue;
    }
    const bool row_valid = tl < U.ntok;
    const int p_row = row_valid ? U.p_first + tl : U.kv_end - 1;
    const int p_tile = U.p_first + q * TM;  // position of the tile's first row
    float m_ref = kNegInf, l = 0.f;
    for (int kt = U.kt0; kt < U.kt1; ++kt) {
      const int steps = pair_steps(U, kt);
#pragma unroll 1  // (both halves unrolled would not fit the instruction cache)
      for (int half = 0; half < steps; ++half) {
        const int b = 2 * half + q;
        const uint32_t s_cols = tmem + lane_addr + b * kHalfKeys;
        // S of this step: the buffer's last S was waited for here, and its
        // next S waits for the P V of this step, which needs this P
        mbar_wait(smem_addr(&B.s_full[b]), (half ? used1 : used0) & 1, p.err, abort_flag);
        tc::fence_after_sync();
        uint32_t sr[64];
        tc::tmem_ld32(s_cols, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tc::tmem_ld32(s_cols + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        // Does every row of this query tile see every key of the step?  Then
        // there is nothing to mask, and no V row to clear.
        const int e0 = kt * kPagesPerTile + half * (kPagesPerTile / 2);
        const int pos0 = U.template page<true>(e0) * kBlock;
        const int pos1 = U.template page<true>(e0 + kPagesPerTile / 2 - 1) * kBlock + kBlock - 1;
        const bool plain =
            pos1 <= p_tile && (pos0 > p_tile + TM - 1 - p.window || pos1 < p.num_sinks);
        tc::tmem_wait_ld();
        if (!plain || !pos_scale) {
          // which keys the row sees, one bit each (an entry past the pages read
          // lies past the unit's keys)
          uint32_t seen[2];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t bits =
                window_bits(U.template page<true>(e0 + g) * kBlock, p_row, p.window, p.num_sinks);
            if (g & 1)
              seen[g >> 1] |= bits << 16;
            else
              seen[g >> 1] = bits;
          }
#pragma unroll
          for (int c = 0; c < 64; ++c)
            sr[c] = __float_as_uint(
                (seen[c >> 5] >> (c & 31)) & 1u ? __uint_as_float(sr[c]) * mul : kNegInf);
        }
        float m4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          const int i = (c >> 3) & 3;
          m4[i] = fmax3(m4[i], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          m4[i] = fmax3(m4[i], __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          m4[i] = fmax3(m4[i], __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          m4[i] = fmax3(m4[i], __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        mx = (mx == kNegInf) ? kNegInf : mx * emul;  // now in scaled base-2 units
        float alpha = 1.f;
        if (m_ref == kNegInf) {
          m_ref = mx;  // first step with a visible key: O holds zeros so far
        } else if (mx > m_ref + kRescaleThreshold) {
          alpha = fast_exp2(m_ref - mx);
          l *= alpha;
          m_ref = mx;
        }
        // p = 2^(emul * s - m_ref), rounded to 16 bits for the product, the
        // sum over the rounded values (as in the single tile's softmax)
        const float mu = (m_ref == kNegInf) ? 0.f : m_ref;
        const float2 e2 = make_float2(emul, emul);
        const float2 nm2 = make_float2(-mu, -mu);
        float2 l4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) l4[j] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(sr[2 * j]), __uint_as_float(sr[2 * j + 1])), e2, nm2);
          if constexpr (F8) {
            sr[j] = f16x2_from_floats(fast_exp2(x.x), fast_exp2(x.y));
            add_f16x2_to(l4[j & 3], sr[j]);
          } else {
            sr[j] = pack_bf16x2(fast_exp2(x.x), fast_exp2(x.y));
            add_bf16x2_to(l4[j & 3], sr[j]);
          }
        }
        tc::tmem_st32(s_cols, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        l += ((l4[0].x + l4[0].y) + (l4[1].x + l4[1].y)) +
             ((l4[2].x + l4[2].y) + (l4[3].x + l4[3].y));
        // rescale the running output when the reference max moved (rare); the
        // P V product of this tile's last step must have landed first
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          // this tile's last step used its other buffer, or (an odd key tile
          // of one step before) this one, whose P V the S of this step waited
          // for: the buffer's use before was waited for by the S issued into
          // it, which these warps waited for, and its next needs a later P
          const uint32_t last = half ? used0 : used1;
          if (last > 0)
            mbar_wait(smem_addr(&B.pv_done[b ^ 2]), (last - 1) & 1, p.err, abort_flag);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(o_cols + c * 32, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tc::tmem_st32(o_cols + c * 32, o);
          }
        }
        // V rows that no row of the unit sees (past its keys, or before its
        // window and no sinks) may hold anything: zero them, so that P = 0
        // times V stays 0.  Thread r clears half of V row r / 2; both query
        // tiles' warps do, each before its own product.
        const int key = half * kHalfKeys + (r >> 1);
        const int pos =
            U.template page<true>(kt * kPagesPerTile + (key >> 4)) * kBlock + (key & 15);
        const bool unseen = pos >= U.kv_end || (pos >= p.num_sinks && pos < U.w0);
        if (!plain && __any_sync(0xffffffffu, unseen)) {
          // V tile kt must have landed.  These warps may have left out the tiles
          // of units without their query tile, so a parity wait on the stage
          // could not tell its uses apart; the issuer of this query tile's
          // products waits for every V tile in turn and counts them.
          wait_count(&B.v_landed[q], vt + 1, p.err, abort_flag);
          if (unseen) {
            unsigned char* vpage = v_s + (vt & 1) * TILE + (key >> 4) * V_PAGE;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int c8 = 4 * (r & 1); c8 < 4 * (r & 1) + 4; ++c8)
                *reinterpret_cast<uint4*>(vpage + h * (kBlock * 128) + sw128_chunk(key & 15, c8)) =
                    make_uint4(0, 0, 0, 0);
          }
        }
        tc::tmem_wait_st();
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&B.p_full[b]));
        if (half)
          ++used1;
        else
          ++used0;
      }
      ++vt;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    // this tile's O: the last unit's was waited for here, and the next unit's
    // first P V waits for o_empty, which these warps arrive on
    mbar_wait(smem_addr(&B.o_full[q]), n_out & 1, p.err, abort_flag);
    tc::fence_after_sync();
    const int64_t row = row_valid ? (int64_t)(U.q0 + tl) * p.n_q + U.g * G + hl : -1;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      tc::tmem_ld32(o_cols + c * 32, o);
      tc::tmem_wait_ld();
      store_rows<D>(p.out, row, c * 32, out_s, o, inv, lane);
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&B.o_empty[q]));
    ++n_out;
  }
}

}  // namespace
}  // namespace pa
