// prefix_tc.cu -- the shared prefix of prefix_attn.cu for many query rows, on the 5th-generation tensor
// cores.
//
// When hundreds of rows of one key head attend to one prefix (requests behind a prompt, drafts of many
// beams), the work is two matrix products per key tile and the bytes of K and V are small. A persistent
// kernel, one CTA per SM, walks work items of (group, key head, two tiles of query rows, share of the
// prefix) in the manner of attn.cu: TMA-fed K and V rings, S = Q K^T and O += P V by tcgen05.mma into
// TMEM, P written back to TMEM as the A operand of the second product, one softmax thread per query row,
// and the two row tiles taking turns on the exponentials through named barriers. What differs:
//  - a row tile holds 128 / r tokens of all r query heads of the key head (a TMA box of 64 x r x tokens
//    over the strided queries), so grouped heads fill the tile's 128 rows and share K and V;
//  - the number of keys and the group's rows are read on the device, and every role derives the same
//    items from them; shares without keys write (-inf, 0);
//  - keys behind the prefix's length may hold anything: their scores are masked, and the rows of V
//    behind the last key are zeroed in shared memory before the product (0 x NaN would not be 0);
//  - every item writes partial results (m, l, O), which prefix_join_kernel joins with those of the
//    sequences' own keys.
// P enters the second product as two bf16 numbers (it is off by 2^-16 then), as in the one-launch form, so that a
// row's result does not depend on how many others share its prefix. The large part is the A operand in TMEM, as in
// attn.cu; the small one, for which TMEM has no columns left beside S and O, is one in shared memory. With the large
// part alone the error of long prompts was 1.4 times that of rounding the output.
// What bounds it: the softmax warps' instructions (the exponentials, 256 x 128 a key tile or 1.1 us of an SM, and
// five for every two probabilities to cut them in two), and at this length the ends of a CTA's work: 1280 rows of
// each of 4 key heads over 8191 keys, 10.7 GFLOP, take 29.5 us cold (144 CTAs of 11 key tiles), with one part 22.7,
// and with the join 28.5 in a captured graph. Of the difference the second product is 1 us: without it as many
// instructions remain. Subtractions by scalar (56.0 us for the call, as it is 51.6) or fp32 += bf16 FMAs (55.8),
// parts cut off instead of rounded (52.0), and the parts formed behind the exponentials (56.6) cost more. On
// mma.sync, with 64 rows a CTA, the same part took about 80 us.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <atomic>

#include "launch.h"
#include "ptx.cuh"

namespace {

using namespace wenc_dev;

constexpr int BQ = 128;    // query rows per tile (two tiles per CTA)
constexpr int BKV = 128;  // keys per tile
constexpr int HD = 64;
constexpr int NK = 3;                     // K ring depth
constexpr int NV = 3;                     // V ring depth
constexpr int kThreads = 384;             // producer, 3 MMA issuers, 2 softmax warpgroups
// Registers per thread after the start-up reallocation (setmaxnreg): the control warpgroup
// (producer and MMA issuers) gives up registers that the two softmax warpgroups take, which keeps
// a row's 128 scores and the exponential pipeline out of local memory. The sum must fit in what
// the CTA is launched with (checked on the host before the first launch).
constexpr int kCtrlRegs = 72;
constexpr int kSoftmaxRegs = 216;
constexpr int kRegsNeeded = kCtrlRegs * 128 + kSoftmaxRegs * 256;
static_assert(kRegsNeeded <= (65536 / kThreads) / 8 * 8 * kThreads, "register split exceeds the launch budget");

constexpr uint32_t Q_BYTES = BQ * HD * 2;           // 16 KB per query tile
constexpr uint32_t KV_BYTES = BKV * HD * 2;         // 16 KB per K or V tile
constexpr uint32_t OFF_Q = 0;                       // two buffers of (Q_A, Q_B): this item's and the next's
constexpr uint32_t OFF_K = OFF_Q + 4 * Q_BYTES;
constexpr uint32_t OFF_V = OFF_K + NK * KV_BYTES;
constexpr uint32_t P_BYTES = BQ * BKV * 2;          // 32 KB: the small part of a tile's P, two blocks of 64 keys
constexpr uint32_t OFF_P = OFF_V + NV * KV_BYTES;
constexpr uint32_t OFF_BARS = OFF_P + 2 * P_BYTES;
// bars: q_full[2], q_empty[2], k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], and per query
// tile t: s_full[t], s_free[t], p_full[t], pv_done[t]; drain. (The exponential turn uses the
// hardware named barriers 1 and 2.)
constexpr int NUM_BARS = 4 + 2 * NK + 2 * NV + 8 + 1;
constexpr size_t SMEM = 1024 + OFF_BARS + NUM_BARS * 8 + 16;
static_assert(SMEM <= 232448, "shared memory of the bf16 prefix kernel");
constexpr uint32_t TMEM_COLS = 512;  // S_A 0..127, S_B 128..255, O_A 256..319, O_B 320..383, P_A 384..447, P_B 448..511
// Grow the running maximum only when a tile's maximum exceeds it by more than this (log2
// units); otherwise keep it, so p <= 2^8 and O is rescaled rarely. The result is unchanged:
// numerator and denominator always use the same reference maximum.
constexpr float kRescaleThreshold = 8.0f;

__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const wenc_host::PrefixTcArgs p, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem);
  const uint32_t sQ = s0 + OFF_Q, sK = s0 + OFF_K, sV = s0 + OFF_V, sP = s0 + OFF_P;
  const uint32_t bar0 = s0 + OFF_BARS;
  auto q_full = [&](int u) { return bar0 + 8u * u; };
  auto q_empty = [&](int u) { return bar0 + 8u * (2 + u); };
  auto k_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto k_empty = [&](int s) { return bar0 + 8u * (4 + NK + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + 2 * NK + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (4 + 2 * NK + NV + s); };
  const uint32_t tb0 = bar0 + 8u * (4 + 2 * NK + 2 * NV);
  auto s_full = [&](int t) { return tb0 + 8u * t; };
  auto s_free = [&](int t) { return tb0 + 16u + 8u * t; };
  auto p_full = [&](int t) { return tb0 + 32u + 8u * t; };
  auto pv_done = [&](int t) { return tb0 + 48u + 8u * t; };
  const uint32_t drain = tb0 + 64u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BARS + NUM_BARS * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, err};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // Work item w (this CTA takes w = blockIdx.x, blockIdx.x + gridDim.x, ...), from lengths and offsets in
  // device memory: every role derives the same items. n_kv == 0: no rows, or no keys in this share.
  struct Item {
    int grp, hk, split, token0, n_tokens, len, kv0, n_kv;
  };
  auto decode = [&](int w) {
    Item it;
    it.split = w % p.np;
    w /= p.np;
    const int x = w % p.n_x;
    w /= p.n_x;
    it.hk = w % p.Hkv;
    it.grp = w / p.Hkv;
    int begin = it.grp * p.max_group, count = p.max_group;
    if (p.group_start) {
      begin = p.group_start[it.grp];
      count = p.group_start[it.grp + 1] - begin;
      if (begin < 0 || count < 0 || begin > p.n_seqs - count || count > p.max_group) {
        *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
        begin = count = 0;
      }
    }
    it.len = p.prefix_lens ? p.prefix_lens[it.grp] : p.prefix_max;
    if (it.len < 0 || it.len > p.prefix_max) {
      *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
      it.len = 0;
    }
    // the pair's first token, and how many tokens of the group are left from there
    it.token0 = begin * p.q_len + x * 2 * p.tokens;
    it.n_tokens = count * p.q_len - x * 2 * p.tokens;
    const int n_kv_all = (it.len + BKV - 1) / BKV, per = (n_kv_all + p.np - 1) / p.np;
    it.kv0 = it.split * per;
    it.n_kv = it.n_tokens > 0 ? max(0, min(per, n_kv_all - it.kv0)) : 0;
    return it;
  };

  if (threadIdx.x == 0) {
    for (int u = 0; u < 2; ++u) {
      mbar_init(q_full(u), 1);
      mbar_init(q_empty(u), 1);  // released by the S issuer's commit after an item's last S
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 2);  // released by both PV issuers
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(s_free(t), 4);  // one arrival per softmax warp of the tile
      mbar_init(p_full(t), 4);
      mbar_init(pv_done(t), 1);
    }
    mbar_init(drain, 3);  // one commit per MMA-issuing thread
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();  // TMEM is held: the next kernel may be scheduled
  pdl_wait();     // queries, prefix and lengths from the previous kernels are complete from here on
  auto tS = [&](int t) { return tmem_base + 128u * t; };
  auto tO = [&](int t) { return tmem_base + 256u + 64u * t; };
  auto tP = [&](int t) { return tmem_base + 384u + 64u * t; };  // P as bf16 pairs: 64 columns per tile

  // Every role walks the same items in the same order and counts K/V tiles across them (kc,
  // vc, g below), so ring slots and barrier parities continue from one item to the next.
  if (warp < 4) {
    // control warpgroup: registers to the softmax warpgroups first
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kCtrlRegs) : "memory");
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer, per item: Q_A, Q_B into the item's Q buffer (free once the
      // S products of the item two back are done), then K0, then (K[j], V[j-1]) for j >= 1, then
      // V[n-1]; the next item's Q and first K tiles load while this item's last tiles run.
      int kc = 0, vc = 0, qi = 0;  // K tiles, V tiles and items issued
      auto load_k = [&](const Item& it, int j) -> bool {
        const int st = kc % NK;
        if (!mbar_wait(k_empty(st), ((kc / NK) & 1) ^ 1u, wc, 11)) return false;
        mbar_arrive_expect_tx(k_full(st), KV_BYTES);
        tma_load_3d(sK + st * KV_BYTES, &tk, k_full(st), it.hk * HD, (it.kv0 + j) * BKV, it.grp);
        ++kc;
        return true;
      };
      auto load_v = [&](const Item& it, int j) -> bool {
        const int st = vc % NV;
        if (!mbar_wait(v_empty(st), ((vc / NV) & 1) ^ 1u, wc, 10)) return false;
        mbar_arrive_expect_tx(v_full(st), KV_BYTES);
        tma_load_3d(sV + st * KV_BYTES, &tv, v_full(st), it.hk * HD, (it.kv0 + j) * BKV, it.grp);
        ++vc;
        return true;
      };
      const uint32_t q_bytes = static_cast<uint32_t>(p.r * p.tokens) * HD * 2;  // of one box
      bool ok = true;
      for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
        const Item it = decode(w);
        if (it.n_kv == 0) continue;
        const int qb = qi & 1;
        if (!in_bounds(it.token0 >= 0 && it.token0 < p.n_seqs * p.q_len && it.hk < p.Hkv && it.split < p.np &&
                           (it.kv0 + it.n_kv - 1) * BKV < it.len && it.len <= p.prefix_max,
                       err, 93)) {
          *abort_flag = 1u;  // an item outside the problem: stop as a failed wait would
          break;
        }
        if (!mbar_wait(q_empty(qb), ((qi >> 1) & 1) ^ 1u, wc, 9)) break;
        mbar_arrive_expect_tx(q_full(qb), 2 * q_bytes);
        tma_load_3d(sQ + qb * 2 * Q_BYTES, &tq, q_full(qb), 0, it.hk * p.r, it.token0);
        tma_load_3d(sQ + qb * 2 * Q_BYTES + Q_BYTES, &tq, q_full(qb), 0, it.hk * p.r, it.token0 + p.tokens);
        ++qi;
        for (int j = 0; ok && j <= it.n_kv; ++j) {
          if (j < it.n_kv) ok = load_k(it, j);
          if (ok && j >= 1) ok = load_v(it, j - 1);
        }
      }
      if (*abort_flag) {
        // Error path: let the copies already issued land before the CTA exits.
        for (int u = (qi > 2 ? qi - 2 : 0); u < qi; ++u) mbar_wait_drain(q_full(u & 1), (u >> 1) & 1);
        for (int j = (kc > NK ? kc - NK : 0); j < kc; ++j) mbar_wait_drain(k_full(j % NK), (j / NK) & 1);
        for (int j = (vc > NV ? vc - NV : 0); j < vc; ++j) mbar_wait_drain(v_full(j % NV), (j / NV) & 1);
      }
    } else if (warp >= 1 && warp <= 3) {
      // ---------------- UMMA issuers (one thread each of three warps: see attn.cu): warp 1 S_A and S_B,
      // warps 2 and 3 O_A and O_B. The whole warp waits; lane 0 issues.
      bool ok = true;
      if (warp == 1) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(BQ, BKV, false);  // B = K tile, K-major, N = 128
        int kc = 0, i = 0;  // K tiles and items consumed
        for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
          const int n_kv = decode(w).n_kv;
          if (n_kv == 0) continue;
          const int qb = i & 1;
          if (!mbar_wait_warp(q_full(qb), (i >> 1) & 1, wc, 12)) { ok = false; break; }
          ++i;
          for (int j = 0; ok && j < n_kv; ++j, ++kc) {
            const int st = kc % NK;
            if (!mbar_wait_warp(k_full(st), (kc / NK) & 1, wc, 13)) { ok = false; break; }
            const uint64_t kdesc = sdesc_sw128(sK + st * KV_BYTES, 16, 1024);
            for (int t = 0; t < 2 && ok; ++t) {
              if (kc >= 1 && !mbar_wait_warp(s_free(t), (kc - 1) & 1, wc, 14)) { ok = false; break; }
              tc_fence_after();
              if (lane == 0) {
                const uint64_t qdesc = sdesc_sw128(sQ + qb * 2 * Q_BYTES + t * Q_BYTES, 16, 1024);
#pragma unroll
                for (int k = 0; k < HD / 16; ++k) umma_bf16_ss(tS(t), qdesc + k * 2, kdesc + k * 2, idesc_s, k > 0);
                umma_commit(s_full(t));
              }
              __syncwarp();
            }
            if (ok && lane == 0) umma_commit(k_empty(st));
          }
          if (ok && lane == 0) umma_commit(q_empty(qb));  // the item's Q buffer is free once its S products are done
        }
      } else {
        constexpr uint32_t idesc_o = idesc_bf16_f32(BQ, HD, true);  // B = V tile, MN-major, N = 64
        const int t = warp - 2;
        int vc = 0;  // V tiles consumed, across items
        for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
          const Item it = decode(w);
          for (int j = 0; j < it.n_kv; ++j, ++vc) {
            const int st = vc % NV;
            if (!mbar_wait_warp(v_full(st), (vc / NV) & 1, wc, 15)) { ok = false; break; }
            const int valid = it.len - (it.kv0 + j) * BKV;
            if (valid < BKV) {  // rows of V behind the last key (both issuers write the same zeros)
              for (int c = valid * 8 + lane; c < BKV * 8; c += 32)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sV + st * KV_BYTES + c * 16), "r"(0) : "memory");
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (!mbar_wait_warp(p_full(t), vc & 1, wc, 16)) { ok = false; break; }
            tc_fence_after();
            if (lane == 0) {
              const uint64_t vdesc = sdesc_sw128(sV + st * KV_BYTES, 1024, 1024);
              const uint64_t pdesc = sdesc_sw128(sP + t * P_BYTES, 16, 1024);
#pragma unroll
              for (int k = 0; k < BKV / 16; ++k)  // (64 keys a block of 128-byte rows)
                umma_bf16_ss(tO(t), pdesc + (k >> 2) * (P_BYTES / 2 >> 4) + (k & 3) * 2, vdesc + k * 128, idesc_o,
                             (j > 0 || k > 0) ? 1u : 0u);
#pragma unroll
              for (int k = 0; k < BKV / 16; ++k) umma_bf16_ts(tO(t), tP(t) + 8 * k, vdesc + k * 128, idesc_o, 1u);
              umma_commit(pv_done(t));
              umma_commit(v_empty(st));
            }
            __syncwarp();
          }
        }
      }
      // Every MMA this thread issued completes before TMEM is released.
      if (lane == 0) {
        umma_commit(drain);
        mbar_wait_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs) : "memory");
    // ---------------- softmax / correction / output: one query row per thread
    const int t = (warp - 4) >> 2;  // query tile of this warpgroup
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    // The turn passes through two hardware named barriers of 256 threads: barrier 1 is tile A's
    // turn, barrier 2 tile B's. The four warps taking the turn sync, the four passing it arrive.
    // Per key tile, tile B syncs on 2 and arrives on 1; tile A syncs on 1 (from its second tile)
    // and arrives on 2; tile A closes with one more sync on 1. Both tiles walk the same key tiles,
    // so every phase completes. After a failed wait a warp runs the turn operations of the key
    // tiles it has not walked yet before it stops, so the other tile never waits for it in vain.
    bool ok = true;
    int g = 0;       // key tiles processed, across items
    int g_turn = 0;  // the first key tile whose turn operations have not run
    const int tok = row / p.r, hr = row - tok * p.r;  // token of the tile and head of the group this row holds
    const float scale_log2 = p.scale_log2;
    const size_t n_parts = static_cast<size_t>(p.n_seqs) * p.q_len * p.H * p.n_slots;  // (for the index checks)
    for (int w = blockIdx.x; ok && w < p.n_items; w += gridDim.x) {
      const Item it = decode(w);
      const int n_kv = it.n_kv;
      const bool mine = tok < p.tokens && t * p.tokens + tok < it.n_tokens;
      // (size_t: rows x slots x 64 floats pass 2^32 bytes)
      const size_t pi = (static_cast<size_t>(it.token0 + t * p.tokens + tok) * p.H + it.hk * p.r + hr) * p.n_slots + it.split;
      if (n_kv == 0) {
        if (mine && in_bounds(pi < n_parts, err, 92)) p.part_ml[pi] = make_float2(-CUDART_INF_F, 0.0f);
        continue;
      }
      float m = -CUDART_INF_F;  // running maximum, in units of scale_log2
      float l = 0.0f;           // running denominator
      for (int j = 0; j < n_kv; ++j, ++g) {
        if (!mbar_wait_warp(s_full(t), g & 1, wc, 17)) { ok = false; break; }
        tc_fence_after();
        float sv[128];
        {
          // the row's 128 scores: four loads in flight, one wait
          uint32_t r[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tS(t) + lane_off + c * 32, r[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[c * 32 + e] = __uint_as_float(r[c][e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(t));  // the MMA may overwrite S with the next tile

        const int valid = it.len - (it.kv0 + j) * BKV;  // keys of this tile inside the prefix
        if (valid < BKV) {              // only a prefix's last tile can be partial (warp-uniform)
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = (c < valid) ? sv[c] : -CUDART_INF_F;
        }
        // Row maximum: eight independent chains of three-input max.
        float mc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float a = fmax3(sv[16 * k], sv[16 * k + 1], sv[16 * k + 2]);
#pragma unroll
          for (int e = 3; e < 15; e += 2) a = fmax3(a, sv[16 * k + e], sv[16 * k + e + 1]);
          mc[k] = fmaxf(a, sv[16 * k + 15]);
        }
        const float mx = fmaxf(fmax3(mc[0], mc[1], mc[2]), fmax3(fmax3(mc[3], mc[4], mc[5]), mc[6], mc[7]));
        const float mx_s = mx * scale_log2;
        const float m_new = (mx_s > m + kRescaleThreshold) ? mx_s : m;
        const float ref = m_new == -CUDART_INF_F ? 0.0f : m_new;  // (scores of -inf alone so far: weights of 0)
        const float alpha = ex2_approx(m - ref);  // 0 on the first tile (m = -inf)

        // Ping-pong: the two tiles take turns on the exponentials (MUFU), so that one tile's
        // exponentials overlap the other tile's loads, stores and waits instead of contending.
        // Tile A's turn j follows tile B's exponentials of tile j-1; tile B's follows A's of j.
        if (t == 1 || g > 0) named_sync(1 + t, 256);

        // p = 2^(s * scale_log2 - m_new): packed fp32x2 FMA for the argument, packed adds for the
        // row sum; P is cut into its two bf16 parts before waiting on the previous PV product.
        const uint64_t c2 = pack_f32x2(scale_log2, scale_log2);
        const uint64_t nm2 = pack_f32x2(-ref, -ref);
        uint64_t sum2a = pack_f32x2(0.0f, 0.0f), sum2b = sum2a;
        const uint64_t minus1 = pack_f32x2(-1.0f, -1.0f);
        uint32_t pk[64], pl[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float a0, a1;
          unpack_f32x2(fma_f32x2(pack_f32x2(sv[2 * i], sv[2 * i + 1]), c2, nm2), a0, a1);
          const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
          const uint64_t pp = pack_f32x2(p0, p1);
          if (i & 1) sum2b = add_f32x2(sum2b, pp);
          else sum2a = add_f32x2(sum2a, pp);
          pk[i] = pack_bf16x2(p0, p1);
          float l0, l1;  // what the large part leaves (exact)
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xffff0000u)), minus1, pp), l0, l1);
          pl[i] = pack_bf16x2(l0, l1);
        }
        float sa0, sa1, sb0, sb1;
        unpack_f32x2(sum2a, sa0, sa1);
        unpack_f32x2(sum2b, sb0, sb1);
        const float sum = (sa0 + sa1) + (sb0 + sb1);
        __syncwarp();
        named_arrive(2 - t, 256);  // the other tile's turn
        g_turn = g + 1;

        if (j > 0) {
          // PV[j-1] must be complete: P is overwritten below and O may be rescaled.
          if (!mbar_wait_warp(pv_done(t), (g - 1) & 1, wc, 18)) { ok = false; break; }
          tc_fence_after();
          if (__any_sync(0xffffffffu, m_new != m)) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tO(t) + lane_off + half * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st_32x32b_x32(tO(t) + lane_off + half * 32, o);
            }
            tmem_st_wait();
          }
        }

        // P row (128 keys as 64 bf16 pairs): the large part into the tile's P columns of TMEM, the small one into
        // its swizzled rows of shared memory (16 bytes are 8 keys).
        {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            sts_v4(sP + t * P_BYTES + (c >> 3) * (P_BYTES / 2) + row * 128u + (((c & 7) ^ (row & 7)) << 4), pl[4 * c], pl[4 * c + 1],
                   pl[4 * c + 2], pl[4 * c + 3]);
          fence_proxy_async_smem();
          uint32_t p0[32], p1[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            p0[e] = pk[e];
            p1[e] = pk[32 + e];
          }
          tmem_st_32x32b_x32(tP(t) + lane_off, p0);
          tmem_st_32x32b_x32(tP(t) + lane_off + 32, p1);
          tmem_st_wait();
        }
        l = l * alpha + sum;
        m = m_new;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
      }
      if (!ok) break;
      if (!mbar_wait_warp(pv_done(t), (g - 1) & 1, wc, 19)) { ok = false; break; }
      {
        // The item's partial result, from O in TMEM once the PV product of its last key tile is done;
        // the next item's first PV product (which overwrites O) waits for P that this warp
        // writes only after these reads.
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO(t) + lane_off + half * 32, o);
          tmem_ld_wait();
          if (mine && in_bounds(pi < n_parts, err, 92)) {
            float4* d4 = reinterpret_cast<float4*>(p.part_o + pi * HD + half * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              d4[q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                  __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
          }
        }
        if (mine && in_bounds(pi < n_parts, err, 92)) p.part_ml[pi] = make_float2(m, l);
        tc_fence_before();
      }
    }
    int turns = g;  // key tiles whose turns this warp has taken part in
    if (!ok) {
      int n_tiles = 0;
      for (int w = blockIdx.x; w < p.n_items; w += gridDim.x) n_tiles += decode(w).n_kv;
      for (int gg = g_turn; gg < n_tiles; ++gg) {
        if (t == 1 || gg > 0) named_sync(1 + t, 256);
        named_arrive(2 - t, 256);
      }
      turns = n_tiles;
    }
    // tile B's last hand-over (there is none from a CTA without a key tile)
    if (t == 0 && turns > 0) named_sync(1, 256);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace

namespace wenc_host {

cudaError_t launch_prefix_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefixTcArgs& p,
                             uint32_t* err, int num_sms, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured{-1};
  e = opt_in_smem(prefix_tc_kernel, SMEM, dev, configured);
  if (e != cudaSuccess) return e;
  // The softmax warpgroups' register increase is met only from the registers the CTA was launched with: refuse to
  // launch a build that was given fewer (a property of the build).
  static const int launch_regs = registers_of(prefix_tc_kernel);
  if (launch_regs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  const int grid = p.n_items < num_sms ? p.n_items : num_sms;
  return launch_pdl(prefix_tc_kernel, dim3(grid), dim3(kThreads), SMEM, stream, tq, tk, tv, p, err);
}

}  // namespace wenc_host
