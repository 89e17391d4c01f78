// prefix_tc32.cu -- the shared prefix of prefix_attn.cu for many float32 query rows, on the 5th-generation
// tensor cores.
//
// A float32 is the sum of three bf16 numbers, exactly: its 24 significant bits cut into eight, eight and eight
// (x = x0 + x1 + x2, each part what is left of x cut off after eight bits). A product of two is
//   x y = x0 y0 + (x0 y1 + x1 y0) + (x0 y2 + x1 y1 + x2 y0) + at most 2^-21 |x y|,
// six bf16 products, exact in the accumulator. bf16 runs at twice the rate of TF32 on tcgen05, so the six cost what
// the three products of TF32's two-part form cost, and bf16 (unlike TF32) can read V as it lies, keys
// along K. The small products go into the accumulator first: the tensor core's sums truncate, and what they lose
// is relative to the sum so far. For the same reason every key tile's O is a product of its own, and is added to
// the row's sum in registers. (An infinite key or value makes its rows NaN: its second part is inf - inf.)
//
// One CTA attends one item of (group, key head, tile of query rows, share of the prefix), in four warpgroups:
//  - two of softmax warps, which take the tiles of 64 keys in turn, a query row a thread: the scores from TMEM, the running
//    maximum and sum, the probabilities in parts to TMEM, and the O of their tile before added to 64
//    registers; each keeps a state of its own, joined at the end through shared memory;
//  - one of converting warps: rows of K and V from global memory to registers, split, and stored to the swizzled
//    stage (four stages of 48 KB; the next tile's loads are under way meanwhile);
//  - one of issuing warps, for S = Q K^T and for O = P V of each softmax warpgroup (a thread takes some 80 cycles for
//    an MMA, the tensor core 45). Both products read their A operand (P, and Q's first two parts) from TMEM: with
//    N = 64 a shared A would ask shared memory for more than its 128 bytes a cycle.
// A row tile holds 128 / r tokens of all r query heads of the key head, as in prefix_tc.cu; the item's partial
// result (m, l, O) goes to the workspace and prefix_join_kernel joins it with the others.
//
// Measured (us on the device; the mma.sync form of prefix_attn.cu in brackets): 2 groups x 410 rows of each of 8 key heads
// over 5848 keys 80 (181), 59 GFLOP of bf16 products at 740 TFLOP/s; 2352 rows of each of 2 over 5101 40 (121); 64
// sequences x 5 rows of 4 over 4000 26 (39). What bounds it: the converting warps (some 2500 cycles a key tile beside the
// two softmax warps of their schedulers) and the 48 MMAs of a tile (2150 cycles alone; with N larger 1540). Steps on the first
// case: one warpgroup of softmax 116; two, one issuing warp 129; two issuing warps 94, four 89; packed subtractions
// 80. Not kept: K and V in rings of their own, V two tiles behind K, 108; sixteen lanes a row in the conversion 99 (of
// 94); the six products of one k together 95 (of 94); a branch for whole tiles in place of predicated loads 125 (of 80).
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "launch.h"
#include "ptx.cuh"

namespace {

using namespace wenc_dev;

constexpr int HD = 64;
constexpr int BQ = 128;       // query rows
constexpr int BKV = 64;       // keys per tile
constexpr int kStages = 4;
constexpr int kThreads = 512;  // two warpgroups of softmax, one that converts, one that issues
// Registers per thread after the start-up reallocation (setmaxnreg), and their sum, which has to be there at launch
// (checked on the host before the first one).
constexpr int kSoftmaxRegs = 184, kConvertRegs = 96, kIssueRegs = 48;
constexpr int kRegsNeeded = 128 * (2 * kSoftmaxRegs + kConvertRegs + kIssueRegs);
static_assert(kRegsNeeded <= 65536, "register split exceeds the launch budget");
constexpr uint32_t kPart = BKV * HD * 2;      // one part of K or V: 8 KB
constexpr uint32_t kStageBytes = 6 * kPart;   // K in three parts, V in three parts
constexpr uint32_t OFF_Q = kStages * kStageBytes;  // the queries' third part, 16 KB
constexpr uint32_t OFF_BARS = OFF_Q + BQ * HD * 2;
// full[4], empty[4], and per softmax warpgroup s_full, s_free, p_full, o_full; q_full, drain[4]
constexpr int NUM_BARS = 2 * kStages + 8 + 5;
constexpr size_t SMEM = 1024 + OFF_BARS + NUM_BARS * 8 + 16;
static_assert(SMEM <= 232448, "shared memory of the fp32 prefix kernel");
constexpr uint32_t TMEM_COLS = 512;  // per softmax warpgroup S (64), O (64) and P (3 parts of 32); Q's first two parts (32 each)
constexpr float kRescaleThreshold = 8.0f;  // as in attn.cu: p <= 2^8, and rows are rescaled rarely

// The leading eight bits of x and y as a pair of bf16 numbers; x and y keep the rest (exact).
__device__ __forceinline__ uint32_t cut_pair(float& x, float& y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  x -= __uint_as_float(a & 0xffff0000u);
  y -= __uint_as_float(b & 0xffff0000u);
  return __byte_perm(a, b, 0x7632);
}
// The same with one packed subtraction (the softmax has no registers left for its aligned pairs).
__device__ __forceinline__ uint32_t cut_pair_packed(float& x, float& y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  const float cx = __uint_as_float((a & 0xffff0000u) ^ 0x80000000u), cy = __uint_as_float((b & 0xffff0000u) ^ 0x80000000u);
  unpack_f32x2(add_f32x2(pack_f32x2(x, y), pack_f32x2(cx, cy)), x, y);
  return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t top_pair(float x, float y) {
  return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}

// 32 TMEM lanes x 16 columns, a lane a thread.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A 128-row, 64-deep operand in TMEM, N parts of 32 columns: this thread's row of 64 floats, which keeps the rest.
template <int N>
__device__ __forceinline__ void store_parts(uint32_t taddr, float (&x)[64]) {
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int part = 0; part < N; ++part) {
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float &a = x[32 * half + 2 * i], &b = x[32 * half + 2 * i + 1];
        r[i] = part < 2 ? cut_pair(a, b) : top_pair(a, b);
      }
      tmem_st_32x32b_x16(taddr + 32 * part + 16 * half, r);
    }
  tmem_st_wait();
}
// The products' order: (part of A, part of B), small ones first.
__device__ constexpr int kPartA[6] = {2, 1, 0, 1, 0, 0}, kPartB[6] = {0, 1, 2, 0, 1, 0};

__global__ void __launch_bounds__(kThreads, 1) prefix_tc32_kernel(const wenc_host::PrefixTc32Args p, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem), bar0 = s0 + OFF_BARS;
  auto full = [&](int st) { return bar0 + 8u * st; };
  auto empty = [&](int st) { return bar0 + 8u * (kStages + st); };
  const uint32_t tb0 = bar0 + 8u * (2 * kStages);
  auto s_full = [&](int b) { return tb0 + 8u * b; };
  auto s_free = [&](int b) { return tb0 + 16u + 8u * b; };
  auto p_full = [&](int b) { return tb0 + 32u + 8u * b; };
  auto o_full = [&](int b) { return tb0 + 48u + 8u * b; };
  const uint32_t q_full = tb0 + 64u, drain = tb0 + 72u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BARS + NUM_BARS * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full(st), 4);   // the converting warps
      mbar_init(empty(st), 1);  // the commit behind the tile's O
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_free(b), 4);  // a softmax warpgroup's warps
      mbar_init(p_full(b), 4);
      mbar_init(o_full(b), 1);
    }
    mbar_init(q_full, 4);
    for (int i = 0; i < 4; ++i) mbar_init(drain + 8u * i, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();  // TMEM is held: the next kernel may be scheduled
  pdl_wait();
  auto tS = [&](int b) { return tmem + 64u * b; };
  auto tO = [&](int b) { return tmem + 128u + 64u * b; };
  auto tP = [&](int b, int part) { return tmem + 256u + 96u * b + 32u * part; };
  auto tQ = [&](int part) { return tmem + 448u + 32u * part; };

  // ---- the item
  int w = blockIdx.x;
  const int split = w % p.np;
  w /= p.np;
  const int x = w % p.n_x;
  w /= p.n_x;
  const int hk = w % p.Hkv, grp = w / p.Hkv;
  int begin = grp * p.max_group, count = p.max_group;
  if (p.group_start) {
    begin = p.group_start[grp];
    count = p.group_start[grp + 1] - begin;
    if (begin < 0 || count < 0 || begin > p.n_seqs - count || count > p.max_group) {
      *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
      begin = count = 0;
    }
  }
  int len = p.prefix_lens ? p.prefix_lens[grp] : p.prefix_max;
  if (len < 0 || len > p.prefix_max) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
    len = 0;
  }
  const long long token0 = static_cast<long long>(begin) * p.q_len + static_cast<long long>(x) * p.tokens;
  const int n_tokens = count * p.q_len - x * p.tokens;  // tokens of the group from there on
  const int n_all = (len + BKV - 1) / BKV, per = (n_all + p.np - 1) / p.np, tile0 = split * per;
  const int n_kv = n_tokens > 0 ? max(0, min(per, n_all - tile0)) : 0;  // key tiles of this item

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs) : "memory");
    // ---------------- softmax: one query row per thread, tiles b, b + 2, ... of the item
    const int b = warp >> 2, row = (warp & 3) * 32 + lane, tok = row / p.r, hr = row - tok * p.r;
    const bool mine = tok < p.tokens && tok < n_tokens;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float o[64], m = -CUDART_INF_F, l = 0.0f;
    bool ok = true;
    if (n_kv > 0 && b == 0) {
      float (&q)[64] = o;
      const float4* src = reinterpret_cast<const float4*>(p.q + (token0 + tok) * p.q_stride + (hk * p.r + hr) * (HD * 4));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 v = mine && in_bounds(token0 + tok < static_cast<long long>(p.n_seqs) * p.q_len && hk * p.r + hr < p.H, err, 94)
                             ? src[i]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) q[4 * i + e] = __uint_as_float((__float_as_uint(f[e]) & p.q_keep) ^ p.q_flip);
      }
      store_parts<2>(tQ(0) + lane_off, q);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        sts_v4(s0 + OFF_Q + row * 128u + ((c ^ (row & 7)) << 4), top_pair(q[8 * c], q[8 * c + 1]), top_pair(q[8 * c + 2], q[8 * c + 3]),
               top_pair(q[8 * c + 4], q[8 * c + 5]), top_pair(q[8 * c + 6], q[8 * c + 7]));
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) o[i] = 0.0f;
    // O of this warpgroup's last product added to the row's sum
    auto add_o = [&]() {
      uint32_t t[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        tmem_ld_32x32b_x32(tO(b) + lane_off + 32 * half, t);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[32 * half + i] += __uint_as_float(t[i]);
      }
    };
    int k = 0;  // tiles of this warpgroup done
    for (int j = b; j < n_kv; j += 2, ++k) {
      if (!mbar_wait_warp(s_full(b), k & 1, wc, 50)) { ok = false; break; }
      tc_fence_after();
      float s[64];
      {
        uint32_t t[2][32];
        tmem_ld_32x32b_x32(tS(b) + lane_off, t[0]);
        tmem_ld_32x32b_x32(tS(b) + lane_off + 32, t[1]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(t[i / 32][i % 32]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(b));
      const int valid = len - (tile0 + j) * BKV;
      if (valid < BKV) {  // only a prefix's last tile can be partial (warp-uniform)
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = i < valid ? s[i] : -CUDART_INF_F;
      }
      float mc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mc[c] = fmaxf(s[16 * c], s[16 * c + 1]);
#pragma unroll
        for (int e = 2; e < 16; e += 2) mc[c] = fmax3(mc[c], s[16 * c + e], s[16 * c + e + 1]);
      }
      const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * p.scale_log2;
      const float m_new = mx > m + kRescaleThreshold ? mx : m;
      const float ref = m_new == -CUDART_INF_F ? 0.0f : m_new;  // (scores of -inf alone so far: weights of 0)
      const float alpha = ex2_approx(m - ref);
      const uint64_t c2 = pack_f32x2(p.scale_log2, p.scale_log2), nm2 = pack_f32x2(-ref, -ref);
      uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float a0, a1;
        unpack_f32x2(fma_f32x2(pack_f32x2(s[2 * i], s[2 * i + 1]), c2, nm2), a0, a1);
        s[2 * i] = ex2_approx(a0);
        s[2 * i + 1] = ex2_approx(a1);
        sum[i & 1] = add_f32x2(sum[i & 1], pack_f32x2(s[2 * i], s[2 * i + 1]));
      }
      float sa0, sa1, sb0, sb1;
      unpack_f32x2(sum[0], sa0, sa1);
      unpack_f32x2(sum[1], sb0, sb1);
      l = l * alpha + ((sa0 + sa1) + (sb0 + sb1));
      if (k > 0) {  // the product before is complete: P may be overwritten, and O is read before the next one
        if (!mbar_wait_warp(o_full(b), (k - 1) & 1, wc, 51)) { ok = false; break; }
        tc_fence_after();
        add_o();  // (in the units of the maximum before this tile's)
      }
      store_parts<3>(tP(b, 0) + lane_off, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(b));
      if (__any_sync(0xffffffffu, m_new != m)) {
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] *= alpha;
      }
      m = m_new;
    }
    if (ok && k > 0) {
      ok = mbar_wait_warp(o_full(b), (k - 1) & 1, wc, 52);
      tc_fence_after();
      if (ok) add_o();
    }
    // ---- the two states of a row, joined: each warpgroup hands over half of its O and finishes the other half
    named_sync(1, 256);  // (every product is complete: the stages are free)
    float* part = reinterpret_cast<float*>(smem);  // [warpgroup][32 elements and m, l][row]
    float *give = part + b * (34 * BQ) + row, *take = part + (1 - b) * (34 * BQ) + row;
#pragma unroll
    for (int i = 0; i < 32; ++i) give[i * BQ] = b ? o[i] : o[32 + i];
    give[32 * BQ] = m;
    give[33 * BQ] = l;
    named_sync(1, 256);
    const float m1 = take[32 * BQ], l1 = take[33 * BQ], mm = fmaxf(m, m1), u = mm == -CUDART_INF_F ? 0.0f : mm;
    const float f0 = ex2_approx(m - u), f1 = ex2_approx(m1 - u);
    const size_t at = (static_cast<size_t>(token0 + tok) * p.H + hk * p.r + hr) * p.n_slots + split;
    if (ok && mine && !*abort_flag && in_bounds(at < static_cast<size_t>(p.n_seqs) * p.q_len * p.H * p.n_slots, err, 95)) {
      if (n_kv > 0) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + at * HD + 32 * b);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = f0 * (b ? o[32 + i + e] : o[i + e]) + f1 * take[(i + e) * BQ];
          dst[i / 4] = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      if (b == 0) p.part_ml[at] = make_float2(mm, f0 * l + f1 * l1);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kConvertRegs) : "memory");
    // ---------------- K and V, split: rows 16 (warp - 8) .. + 15 of a tile, eight lanes a row, eight elements a lane
    const int row0 = 16 * (warp - 8) + (lane >> 3), c = lane & 7;
    int key = tile0 * BKV + row0;  // of the first row to load
    const uint8_t* kp = p.kp + grp * p.k_group + hk * (HD * 4) + c * 32 + key * p.k_token;
    const uint8_t* vp = p.vp + grp * p.v_group + hk * (HD * 4) + c * 32 + key * p.v_token;
    float4 v[8][2];  // four rows of K, four of V
    auto load = [&](int i) {
      const bool in = key + 4 * (i & 3) < len && in_bounds(key >= 0 && key + 4 * (i & 3) < p.prefix_max && hk < p.Hkv, err, 96);  // rows behind the prefix are zeros, whatever memory holds there
      const float4* src = reinterpret_cast<const float4*>(i < 4 ? kp + 4 * i * p.k_token : vp + 4 * (i - 4) * p.v_token);
#pragma unroll
      for (int h = 0; h < 2; ++h) v[i][h] = in ? __ldg(src + h) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto advance = [&]() {
      key += BKV;
      kp += BKV * p.k_token;
      vp += BKV * p.v_token;
    };
    const uint32_t at0 = s0 + row0 * 128u + ((c ^ (row0 & 7)) << 4);  // (rows 4 apart: the swizzle's bit 2 turns)
    if (n_kv > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) load(i);
      advance();
    }
    for (int j = 0; j < n_kv; ++j) {
      const int st = j % kStages;
      if (!mbar_wait_warp(empty(st), ((j / kStages) & 1) ^ 1u, wc, 53)) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = (at0 ^ ((i & 1) << 6)) + st * kStageBytes + (i < 4 ? 0u : 3 * kPart) + (i & 3) * 512u;
        float f[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
        if (j + 1 < n_kv) load(i);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t a = cut_pair_packed(f[0], f[1]), b = cut_pair_packed(f[2], f[3]);
          const uint32_t d = cut_pair_packed(f[4], f[5]), e = cut_pair_packed(f[6], f[7]);
          sts_v4(at + part * kPart, a, b, d, e);
        }
        sts_v4(at + 2 * kPart, top_pair(f[0], f[1]), top_pair(f[2], f[3]), top_pair(f[4], f[5]), top_pair(f[6], f[7]));
      }
      advance();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(st));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kIssueRegs) : "memory");
    // ---------------- the issuing warps, two for S and two for O: all of a warp waits, lane 0 issues
    const int odd = warp & 1;  // the tiles a warp issues for: those of one softmax warpgroup
    if (warp < 14 && n_kv > 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(BQ, BKV, false);  // B = K tile, K-major
      const uint64_t qdesc = sdesc_sw128(s0 + OFF_Q, 16, 1024);
      bool ok = mbar_wait_warp(q_full, 0, wc, 54);
      for (int j = odd; ok && j < n_kv; j += 2) {
        const int st = j % kStages, b = odd;
        if (!mbar_wait_warp(full(st), (j / kStages) & 1, wc, 55)) break;
        if (j >= 2 && !mbar_wait_warp(s_free(b), ((j >> 1) - 1) & 1, wc, 56)) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t kdesc = sdesc_sw128(s0 + st * kStageBytes, 16, 1024);
#pragma unroll
          for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint64_t kd = kdesc + kPartB[i] * (kPart >> 4) + 2 * k;
              if (kPartA[i] == 2) umma_bf16_ss(tS(b), qdesc + 2 * k, kd, idesc, (i | k) != 0 ? 1u : 0u);
              else umma_bf16_ts(tS(b), tQ(kPartA[i]) + 8 * k, kd, idesc, (i | k) != 0 ? 1u : 0u);
            }
          umma_commit(s_full(b));
        }
        __syncwarp();
      }
    } else if (n_kv > 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(BQ, HD, true);  // B = V tile, MN-major
      for (int j = odd; j < n_kv; j += 2) {
        const int st = j % kStages, b = odd;
        if (!mbar_wait_warp(p_full(b), (j >> 1) & 1, wc, 57)) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t vdesc = sdesc_sw128(s0 + st * kStageBytes + 3 * kPart, 1024, 1024);
#pragma unroll
          for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int k = 0; k < BKV / 16; ++k)
              umma_bf16_ts(tO(b), tP(b, kPartA[i]) + 8 * k, vdesc + kPartB[i] * (kPart >> 4) + 128 * k, idesc, (i | k) != 0 ? 1u : 0u);
          umma_commit(o_full(b));
          umma_commit(empty(st));  // (its S is long done)
        }
        __syncwarp();
      }
    }
    // every MMA issued completes before TMEM is released
    if (n_kv > 0) {
      if (lane == 0) {
        umma_commit(drain + 8u * (warp - 12));
        mbar_wait_drain(drain + 8u * (warp - 12), 0);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

namespace wenc_host {

cudaError_t launch_prefix_tc32(const PrefixTc32Args& p, uint32_t* err, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured{-1};
  e = opt_in_smem(prefix_tc32_kernel, SMEM, dev, configured);
  if (e != cudaSuccess) return e;
  // The softmax warpgroups' register increase is met only from the registers the CTA was launched with: refuse to
  // launch a build that was given fewer (a property of the build).
  static const int launch_regs = registers_of(prefix_tc32_kernel);
  if (launch_regs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  return launch_pdl(prefix_tc32_kernel, dim3(p.n_items), dim3(kThreads), SMEM, stream, p, err);
}

}  // namespace wenc_host
