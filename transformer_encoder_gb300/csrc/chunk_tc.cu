// chunk_tc.cu -- the chunks of chunk_attn.cu that bring many bf16 query rows (prompts and their parts), on the 5th-generation
// tensor cores.
//
// Of a sequence with more rows per key head than the few of chunk_attn.cu, a unit of work is 2 x 128 / r tokens of one key head
// (r query heads share it; two row tiles of 128) against the keys that these tokens see, in steps of 128. Units differ in
// length: a prompt's later tokens see more keys, sequences bring what they bring. So all units' steps are laid end to end, each
// with kStart more for its beginning and end, and every CTA (one per SM) takes an equal run of them, which it finds itself from
// the lengths: there is no plan to build and read, and no CTA idles while another works on a long unit. A unit that is whole
// within a run goes straight to the output; of one that is cut, the pieces (at most one at either end of a run) go to the
// workspace, and chunk_join_kernel joins them, in order.
//
// Within a CTA, in the manner of prefix_tc.cu: S = Q K^T and O += P V by tcgen05.mma into TMEM, one softmax thread per query row,
// P as two bf16 parts (2^-16), the A operands of the second product. What differs:
//  - two warps gather K and V by cp.async, 128 bytes a row from wherever its page lies, so pages may have any size; keys that no
//    token of the unit sees are zero-filled and not read, and steps at the borders of what the rows see are masked;
//  - three score buffers go round the two row tiles, and both parts of P lie in the 32 columns of the 32 scores they come from: no
//    shared memory for P, and the next scores are there before this step's P has been used;
//  - a row's reference is the maximum of its first step, moved only when weights pass 2^20, so no step forms a maximum; it is a
//    whole number (of log2), so moving it is exact;
//  - rows that come out as no numbers are formed again behind this kernel, by chunk_join_kernel: that takes as long as the cache is
//    long, and the other roles' waits have a limit.
// What bounds it: the two softmax warps of a scheduler (all warps together issue 1970 instructions a scheduler and step of 256
// x 128, in 58% of the cycles; what they wait for are TMEM loads and results of their own, and more warps find no registers).
// The tensor pipe is busy for 47%. 2048 tokens of 20 heads over 4 behind 14000 keys take 228 us, 687 TFLOP/s of the two
// products, a step some 3400 cycles; its MMAs alone, in straight lines, would take 1650, its exponentials (16 an SM and cycle)
// 2048. (These are 7.7 instructions a score; the arithmetic as it is written here counts some 4.5.) On the way there (us):
// first form 567 (every role walked, loops unrolled: warps waited for instructions), 442 walked by one warp, 313 with rolled
// loops, 270 with the pages looked up a step ahead and three score buffers, 257 with P in TMEM alone, 245 with tiles handed
// over by their copies' own arrival and P's barriers in pairs, 228 with a piece's queries addressed without divisions. Not
// kept: taking turns on the exponentials, unrolled exponentials (331), the next 32 scores loaded ahead (256 against 245), four
// gathering warps (252); a polynomial on the FMA pipe for one pair of exponentials in 8, 4 or 2 (238, 249, 293 against 230): it
// is instructions that count.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <atomic>

#include "chunk.cuh"
#include "decode_index.cuh"
#include "launch.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace {

using namespace wenc_dev;

constexpr int BQ = 128;    // query rows per tile (two tiles per unit)
constexpr int BKV = 128;   // keys per step
constexpr int HD = 64;
constexpr int NK = 4;      // K ring depth
constexpr int NV = 4;      // V ring depth
constexpr int NP = 4;      // ring of pieces
constexpr int kThreads = 384;  // K and V producers, 2 MMA issuers, 2 softmax warpgroups
constexpr int kWarps = kThreads / 32;
constexpr int kStart = 1;  // what a unit's beginning and end cost, in steps
constexpr int kLeast = 4;  // no CTA takes fewer steps
// Registers per thread after the start-up reallocation (setmaxnreg), as in prefix_tc.cu; the sum must fit in what the CTA is
// launched with (checked on the host before the first launch).
constexpr int kCtrlRegs = 104;
constexpr int kSoftmaxRegs = 200;
constexpr int kRegsNeeded = kCtrlRegs * 128 + kSoftmaxRegs * 256;
static_assert(kRegsNeeded <= (65536 / kThreads) / 8 * 8 * kThreads, "register split exceeds the launch budget");

constexpr uint32_t Q_BYTES = BQ * HD * 2;    // 16 KB per query tile
constexpr uint32_t KV_BYTES = BKV * HD * 2;  // 16 KB per K or V tile
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_K = OFF_Q + 2 * Q_BYTES;
constexpr uint32_t OFF_V = OFF_K + NK * KV_BYTES;
constexpr uint32_t OFF_BARS = OFF_V + NV * KV_BYTES;
// bars: q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], and per query tile t: s_full[t][2], p_full[t][2] and
// pv_done[t][2]; drain; piece_full[NP], piece_empty[NP]. (Pairs, of even and odd steps: a wait tells a phase from the next one
// only, and an S may be a step ahead of its softmax, a P one ahead of the PV issuer, which may wait for V, a PV one ahead of
// the S issuer's wait for the last.)
constexpr int NUM_BARS = 2 + 2 * NK + 2 * NV + 12 + 1 + 2 * NP;
constexpr int kTakers = 11;  // warps that take pieces from the ring: all but the one that walks
constexpr size_t SMEM = 1024 + OFF_BARS + NUM_BARS * 8 + 16;
static_assert(SMEM + 2600 <= 232448, "shared memory of the chunk kernel");
// TMEM: three buffers of S at 0, 128 and 256, O_A 384..447, O_B 448..511. Step g of tile t is S number 2 g + t, in buffer number
// modulo three, and its P overwrites the scores that have been read: so the next step's S is there before this one's P has
// been used, and no softmax waits for an S.
constexpr uint32_t TMEM_COLS = 512;
// The sum of a row's weights of 32 keys above which its reference moves.
constexpr float kTooMuch = 0x1p20f;

// The largest of 32 scores, in independent chains of three-input max.
__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
  float mc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    auto at = [&](int e) { return __uint_as_float(r[8 * k + e]); };
    mc[k] = fmaxf(fmax3(fmax3(at(0), at(1), at(2)), at(3), at(4)), fmax3(at(5), at(6), at(7)));
  }
  return fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
}

using wenc_host::ChunkCut;
using wenc_host::ChunkRun;
using wenc_host::ChunkTcArgs;
using wenc_host::kChunkMark;

// Unit x of a sequence: its tokens i0 .. i1 (of the sequence's) and their keys.
struct Unit {
  int i0, i1;
  KeySteps ks;
  Unit() = default;
  __device__ __forceinline__ Unit(const ChunkParams& p, int m, int len, int per_unit, int x)
      : i0(x * per_unit), i1(min(m, (x + 1) * per_unit) - 1), ks(len - m + i0, len - m + i1, p.window, p.sinks, BKV, 1) {}
  // (at least one, of which nothing is seen: tokens in front of the cache have rows of zeros)
  __device__ __forceinline__ int steps() const { return max(1, ks.n); }
};

// The sequence's tokens where its units are this kernel's, else 0; and its length.
__device__ __forceinline__ int long_tokens(const ChunkParams& p, int few, int s, int& len, uint32_t* err) {
  const ChunkSeq q = chunk_seq(p, s, err);
  len = q.len;
  return q.m * p.r > few ? q.m : 0;
}

// Steps k0 .. k1 - 1 of a unit's n, and where the unit's last one ends among all.
struct Piece {
  Unit u;
  int hk, seq, x, row0, pos0, k0, k1, n;  // row0, pos0: of the sequence's first token
  long long end;
};

// The way through a CTA's run of steps. One warp walks; it hands the pieces to the other roles through a ring in shared memory
// (walking in every role made the kernel's code 164 KB, and 4.4 of the 5.6 warps that waited on average waited for instructions).
struct Walk {
  Piece pc;                           // the piece in hand
  int hk, seq, x, row0, m, len, skip;  // where the run goes on: step `skip` (of n + kStart) of that unit
  long long left, at;                 // steps left, and the number of the unit's first step among all

  Walk() = default;
  __device__ __forceinline__ explicit Walk(const ChunkRun& r)
      : hk(r.hk), seq(r.seq), x(r.x), row0(r.row0), m(r.m), len(r.len), skip(r.skip), left(r.left), at(r.at) {}

  // The next piece; false at the end of the run. All lanes of a warp call.
  __device__ __forceinline__ bool next(const ChunkParams& p, const ChunkTcArgs& a, uint32_t* err) {
    while (left > 0) {
      const Unit u(p, m, len, a.per_unit, x);
      const int n = u.steps(), all = n + kStart, take = static_cast<int>(min(left, static_cast<long long>(all - skip)));
      pc = Piece{u, hk, seq, x, row0, len - m, max(0, skip - kStart), max(0, skip + take - kStart), n, at + all};
      left -= take;
      skip += take;
      if (skip == all && left > 0) {  // on to the next unit
        at += all;
        skip = 0;
        if ((x + 1) * a.per_unit < m) {
          ++x;
        } else {
          x = 0;
          find(p, a, seq + 1, err);
        }
      }
      if (pc.k1 > pc.k0) return true;
    }
    return false;
  }

  // The first sequence with units from s on (of the next key head behind the last).
  __device__ __forceinline__ void find(const ChunkParams& p, const ChunkTcArgs& a, int s, uint32_t* err) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
#pragma unroll 1
      for (; s < p.n_seqs; s += 32) {
        int l = 0;
        const int mine = s + lane < p.n_seqs ? long_tokens(p, a.few, s + lane, l, err) : 0;
        const uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
        if (some) {
          const int i = __ffs(some) - 1;
          seq = s + i;
          m = __shfl_sync(0xffffffffu, mine, i);
          len = __shfl_sync(0xffffffffu, l, i);
          row0 = p.seq_start ? p.seq_start[seq] : seq * p.per_seq;
          return;
        }
      }
      ++hk;
      s = 0;
    }
    left = 0;  // (not reached: a run ends within the units)
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkTcArgs a, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long sums[kWarps];
  __shared__ ChunkRun start;  // of this CTA's run
  __shared__ Piece pieces[NP];
  __shared__ uint64_t places[2][BKV];
  __shared__ long long of_run[2];  // all steps, and the CTAs that share them
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem);
  const uint32_t sQ = s0 + OFF_Q, sK = s0 + OFF_K, sV = s0 + OFF_V;
  const uint32_t bar0 = s0 + OFF_BARS;
  const uint32_t q_full = bar0, q_empty = bar0 + 8u;
  auto k_full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto k_empty = [&](int s) { return bar0 + 8u * (2 + NK + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (2 + 2 * NK + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (2 + 2 * NK + NV + s); };
  const uint32_t tb0 = bar0 + 8u * (2 + 2 * NK + 2 * NV);
  auto s_full = [&](int t, int g) { return tb0 + 16u * t + 8u * (g & 1); };
  auto p_full = [&](int t, int g) { return tb0 + 32u + 16u * t + 8u * (g & 1); };
  auto pv_done = [&](int t, int g) { return tb0 + 64u + 16u * t + 8u * (g & 1); };
  const uint32_t drain = tb0 + 96u;
  auto piece_full = [&](int i) { return tb0 + 104u + 8u * i; };
  auto piece_empty = [&](int i) { return tb0 + 104u + 8u * (NP + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BARS + NUM_BARS * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, err};
  // (from lane 0, so that the compiler knows it for the whole warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 64);  // the lanes of the two warps that copy
    mbar_init(q_empty, 1);  // released by the S issuer's commit after a piece's last S
    for (int s = 0; s < NK; ++s) {
      mbar_init(k_full(s), 32);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(v_full(s), 32);
      mbar_init(v_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int g = 0; g < 2; ++g) {
        mbar_init(s_full(t, g), 1);
        mbar_init(p_full(t, g), 4);  // one arrival per softmax warp of the tile
        mbar_init(pv_done(t, g), 1);
      }
    }
    mbar_init(drain, 2);  // one commit per MMA-issuing thread
    for (int i = 0; i < NP; ++i) {
      mbar_init(piece_full(i), 1);
      mbar_init(piece_empty(i), kTakers);
    }
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // TMEM is held: the next kernel may be scheduled
  pdl_wait();     // queries, cache and lengths from the previous kernels are complete from here on

  // ---- the CTA's run of steps: the warps sum the steps of a share of the sequences each (lanes over a sequence's units) ...
  const int per_warp = (p.n_seqs + kWarps - 1) / kWarps;
  const int seq_a = min(p.n_seqs, warp * per_warp), seq_b = min(p.n_seqs, seq_a + per_warp);
  auto weigh = [&](int m, int len, int x) { return x * a.per_unit < m ? Unit(p, m, len, a.per_unit, x).steps() + kStart : 0; };
  // f(sequence, its tokens, its length) for the warp's sequences with units, until it returns true
  auto each_seq = [&](auto&& f) {
#pragma unroll 1
    for (int s = seq_a; s < seq_b; s += 32) {
      int l = 0;
      const int mine = s + lane < seq_b ? long_tokens(p, a.few, s + lane, l, err) : 0;
#pragma unroll 1
      for (uint32_t some = __ballot_sync(0xffffffffu, mine > 0); some; some &= some - 1) {
        const int i = __ffs(some) - 1;
        if (f(s + i, __shfl_sync(0xffffffffu, mine, i), __shfl_sync(0xffffffffu, l, i))) return;
      }
    }
  };
  auto warp_sum = [&](long long v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  {
    long long sum = 0;
    each_seq([&](int, int m, int len) {
#pragma unroll 1
      for (int x = lane; x * a.per_unit < m; x += 32) sum += weigh(m, len, x);
      return false;
    });
    sum = warp_sum(sum);
    if (lane == 0) sums[warp] = sum;
  }
  __syncthreads();
  long long of_head = 0, before = 0;  // steps of one key head, and of the sequences before this warp's
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    of_head += sums[w];
  }
  // ... and the run's beginning is found by the warp whose share holds it.
  const long long total = of_head * p.Hkv;
  const long long ctas = max(1ll, min(static_cast<long long>(gridDim.x), total / kLeast));
  const long long b0 = min(total, total * blockIdx.x / ctas), b1 = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : b0;
  const bool busy = b1 > b0 && blockIdx.x < ctas;
  if (busy) {
    const long long t = b0 % of_head;
    if (t >= before && t < before + sums[warp]) {
      long long at = before;
      each_seq([&](int s, int m, int len) {
#pragma unroll 1
        for (int x0 = 0; x0 * a.per_unit < m; x0 += 32) {
          const int w = weigh(m, len, x0 + lane);
          int sum = w;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += up;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, t < at + sum);
          if (past) {
            if (lane == __ffs(past) - 1) {
              const int skip = static_cast<int>(t - (at + sum - w));
              start = ChunkRun{0, static_cast<int>(b0 / of_head), s, x0 + lane, skip, m, len,
                               p.seq_start ? p.seq_start[s] : s * p.per_seq, b1 - b0, b0 - skip};
            }
            return true;
          }
          at += __shfl_sync(0xffffffffu, sum, 31);
        }
        return false;
      });
    }
  }
  __syncthreads();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (threadIdx.x == 0) {
    if (!busy) start = ChunkRun{};
    a.cuts[blockIdx.x].pieces = 0;
    a.runs[blockIdx.x] = start;
    of_run[0] = total;
    of_run[1] = ctas;
  }
  __syncthreads();  // (a piece that is cut at the run's end writes into `cuts`, a whole one without numbers into `runs`)

  auto tS = [&](int buf) { return tmem_base + 128u * buf; };  // (and the P that follows)
  auto tO = [&](int t) { return tmem_base + 384u + 64u * t; };

  // Every role takes the same pieces in the same order and counts K/V tiles across them, so ring slots and barrier parities
  // continue from one piece to the next. take(i): piece i, false behind the last (or after a failed wait); give(i): it is done
  // with.
  auto take = [&](int i) { return mbar_wait_warp(piece_full(i % NP), (i / NP) & 1, wc, 8) && pieces[i % NP].k1 > 0; };
  auto give = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty(i % NP));
  };
  if (warp < 4) {
    // control warpgroup: registers to the softmax warpgroups first
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kCtrlRegs) : "memory");
    if (warp < 2) {
      // ---------------- gathering: warp 0 K, warp 1 V, and a tile of the queries each.
      const bool is_k = warp == 0;
      const uint8_t* pages = is_k ? p.k_pages : p.v_pages;
      const uint32_t page16 = is_k ? p.k_page16 : p.v_page16;
      const uint32_t ring = is_k ? sK : sV;
      const int c = lane & 7, r4 = lane >> 3;  // 16-byte piece of a row, and row of the four that an instruction copies
      const uint32_t even = r4 * 128u + ((c ^ r4) << 4), odd = (r4 + 4) * 128u + ((c ^ (r4 + 4)) << 4);
      // (all 32 lanes arrive, each when its own copies have landed: nobody waits here, and nothing is fenced here, which would wait
      // for the copies just issued; the thread that issues the MMAs fences)
      auto hand_over = [&](uint32_t bar) {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      };
      Walk run;
      if (is_k) run = Walk(start);
      int kc = 0;  // tiles
      bool ok = true;
#pragma unroll 1
      for (int np = 0; ok; ++np) {
        const Piece& pc = pieces[np % NP];
        if (is_k) {
          const bool more = run.next(p, a, err);
          if (!more) run.pc.k0 = run.pc.k1 = 0;
          if (!mbar_wait_warp(piece_empty(np % NP), ((np / NP) & 1) ^ 1u, wc, 8)) break;
          if (lane == 0) {
            pieces[np % NP] = run.pc;
            mbar_arrive(piece_full(np % NP));
          }
          __syncwarp();
          if (!more) break;
        } else if (!take(np)) {
          break;
        }
        const Unit u = pc.u;
        if (!mbar_wait_warp(q_empty, (np & 1) ^ 1u, wc, 9)) break;
        {
          // the queries: a row tile a warp. Token and head of a row run along (divided for each of them, a piece's queries took
          // 15000 cycles, 8 us).
          int tok = r4 / p.r, hr = r4 - tok * p.r;
          const int d_tok = 4 / p.r, d_hr = 4 - d_tok * p.r, at0 = u.i0 + warp * a.tokens;
          const uint8_t* src = p.q + static_cast<long long>(pc.row0) * p.q_stride + pc.hk * p.r * (HD * 2) + c * 16;
          const uint32_t dst = sQ + warp * Q_BYTES;
#pragma unroll 4
          for (int i = 0; i < BQ / 4; ++i) {
            const bool in = tok < a.tokens && at0 + tok <= u.i1 &&
                            in_bounds(pc.row0 + at0 + tok < p.n_tokens && pc.hk * p.r + hr < p.H, err, 121);
            cp_async16(dst + (i >> 1) * 1024 + (i & 1 ? odd : even), in ? src + (at0 + tok) * p.q_stride + hr * (HD * 2) : p.q, in);
            tok += d_tok;
            hr += d_hr;
            if (hr >= p.r) {
              hr -= p.r;
              ++tok;
            }
          }
          hand_over(q_full);
        }
        // A step's keys, four a lane: their pages are read a step ahead, and their rows' addresses go through shared memory to
        // the lanes that copy them (0: not there). With both in one chain, a step took its producers 4300 cycles.
        const int32_t* row = p.table + pc.seq * p.table_stride;
        const int seq = pc.seq, k1 = pc.k1;
        const uint8_t* head = pages + pc.hk * (HD * 2);
        int page[4];
        auto look = [&](int j) {
          const int key0 = u.ks.key0(j, BKV) + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 32 * i, pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
            page[i] = -1;
            // (volatile: else the compiler moves the load down to its use)
            if (u.ks.seen(key) && in_bounds(seq < p.n_seqs && pi >= 0 && pi < p.max_pages, err, 122))
              asm volatile("ld.global.b32 %0, [%1];" : "=r"(page[i]) : "l"(row + pi) : "memory");
          }
        };
        look(pc.k0);
#pragma unroll 1
        for (int j = pc.k0; j < k1; ++j, ++kc) {
          const int st = kc % NK;
          static_assert(NK == NV, "one ring arithmetic for both");
          const int key0 = u.ks.key0(j, BKV) + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 32 * i, pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
            uint64_t at = 0;
            if (u.ks.seen(key)) {
              if (static_cast<uint32_t>(page[i]) < static_cast<uint32_t>(p.n_pages))
                at = reinterpret_cast<uint64_t>(head) + ((static_cast<uint64_t>(page[i]) * page16 + static_cast<uint32_t>(key - pi * p.page_size) * p.row16) << 4);
              else
                *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
            }
            places[warp][32 * i + lane] = at;
          }
          if (j + 1 < k1) look(j + 1);
          __syncwarp();
          if (!mbar_wait_warp(is_k ? k_empty(st) : v_empty(st), ((kc / NK) & 1) ^ 1u, wc, is_k ? 11 : 10)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + st * KV_BYTES;
#pragma unroll 1
          for (int i8 = 0; i8 < BKV / 8; i8 += 4) {
            uint64_t at[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) at[i] = places[warp][8 * i8 + 4 * i + r4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              cp_async16(dst + (i8 + (i >> 1)) * 1024 + (i & 1 ? odd : even), reinterpret_cast<const uint8_t*>(at[i] != 0 ? at[i] + c * 16 : reinterpret_cast<uint64_t>(pages)), at[i] != 0);
          }
          __syncwarp();  // (before the places of the next step)
          hand_over(is_k ? k_full(st) : v_full(st));
        }
        if (!is_k) give(np);
      }
      cp_async_commit();
      cp_async_wait<0>();  // (also on the error path: the copies land before the CTA exits)
    } else {
      // ---------------- UMMA issuers: warp 2 S_A and S_B, warp 3 O_A and O_B. The whole warp waits; one thread issues.
      bool ok = true;
      if (warp == 2) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(BQ, BKV, false);  // B = K tile, K-major, N = 128
        int kc = 0, buf = 0;  // K tiles consumed, across pieces, and the buffer of the next S
        for (int np = 0; ok && take(np); ++np) {
          if (!mbar_wait_warp(q_full, np & 1, wc, 12)) break;
#pragma unroll 1
          for (int j = pieces[np % NP].k0, j1 = pieces[np % NP].k1; j < j1; ++j, ++kc) {
            const int st = kc % NK;
            if (!mbar_wait_warp(k_full(st), (kc / NK) & 1, wc, 13)) { ok = false; break; }
            fence_proxy_async_smem();  // (K's rows, and before a piece's first product the queries, were written by cp.async)
            const uint64_t kdesc = sdesc_sw128(sK + st * KV_BYTES, 16, 1024);
#pragma unroll
            for (int t = 0; t < 2 && ok; ++t) {
              // the buffer's last P, of the S three before, has to have been used
              if (t == 0 ? kc >= 2 : kc >= 1) ok = mbar_wait_warp(pv_done(1 - t, kc + t), ((kc - 2 + t) >> 1) & 1, wc, 14);
              if (!ok) break;
              tc_fence_after();
              const uint64_t qdesc = sdesc_sw128(sQ + t * Q_BYTES, 16, 1024);
              const uint32_t to = tS(buf), bar = s_full(t, kc);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < HD / 16; ++k) umma_bf16_ss(to, qdesc + k * 2, kdesc + k * 2, idesc_s, k > 0);
                umma_commit(bar);
                if (t == 1) umma_commit(k_empty(st));
                if (t == 1 && j + 1 == j1) umma_commit(q_empty);  // the Q tiles are free once the piece's S products are done
              }
              __syncwarp();
              buf = buf == 2 ? 0 : buf + 1;
            }
            if (!ok) break;
          }
          give(np);
        }
      } else {
        constexpr uint32_t idesc_o = idesc_bf16_f32(BQ, HD, true);  // B = V tile, MN-major, N = 64
        int vc = 0, buf = 0;  // V tiles consumed, across pieces, and the buffer of the next P
        for (int np = 0; ok && take(np); ++np) {
          const int k0 = pieces[np % NP].k0, k1 = pieces[np % NP].k1;
#pragma unroll 1
          for (int j = k0; ok && j < k1; ++j, ++vc) {
            const int st = vc % NV;
            if (!mbar_wait_warp(v_full(st), (vc / NV) & 1, wc, 15)) { ok = false; break; }
            fence_proxy_async_smem();
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
              if (!mbar_wait_warp(p_full(t, vc), (vc >> 1) & 1, wc, 16)) { ok = false; break; }
              tc_fence_after();
              const uint64_t vdesc = sdesc_sw128(sV + st * KV_BYTES, 1024, 1024);
              const uint32_t to = tO(t), from = tS(buf), bar = pv_done(t, vc), v_bar = v_empty(st), more = j > k0;
              if (elect_one()) {
#pragma unroll
                for (int part = 1; part >= 0; --part)  // (the small parts first: the tensor core's sums truncate)
#pragma unroll
                  for (int k = 0; k < BKV / 16; ++k)
                    umma_bf16_ts(to, from + 32 * (k >> 1) + 16 * part + 8 * (k & 1), vdesc + k * 128, idesc_o, part == 0 || k > 0 ? 1u : more);
                umma_commit(bar);
                if (t == 1) umma_commit(v_bar);
              }
              __syncwarp();
              buf = buf == 2 ? 0 : buf + 1;
            }
          }
          give(np);
        }
      }
      // Every MMA this thread issued completes before TMEM is released.
      if (elect_one()) {  // (the thread that issued them)
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
    bool ok = true;
    int g = 0;    // steps processed, across pieces
    int buf = t;  // of the step's S: two further, modulo three, each step
    const int tok = row / p.r, hr = row - tok * p.r;  // token of the tile and head of the group this row holds
    const float scale_log2 = p.scale_log2;
    for (int np = 0; ok && take(np); ++np) {
      const Piece& pc = pieces[np % NP];
      // (what concerns the piece stays in shared memory until it is needed: the registers hold scores)
      float m = -CUDART_INF_F;  // running maximum, in units of scale_log2
      float l = 0.0f;           // running denominator
#pragma unroll 1
      for (int j = pc.k0; j < pc.k1; ++j, ++g, buf = buf == 0 ? 2 : buf - 1) {
        if (!mbar_wait_warp(s_full(t, g), (g >> 1) & 1, wc, 17)) { ok = false; break; }
        tc_fence_after();
        const int key0 = pc.u.ks.key0(j, BKV);
        const int first = pc.pos0 + pc.u.i0 + t * a.tokens, last = pc.pos0 + pc.u.i1;  // (of the tile's tokens, and of all)
        // visible: key <= hi and (key > hi - window or key < sinks); rows without a token see what the unit's last one does
        const bool border = key0 + BKV - 1 > first || (key0 <= last - p.window && key0 + BKV > p.sinks);
        const int ca = min(first + tok, last) - key0 + 1, cb = ca - p.window, cd = p.sinks - key0;  // keys [cb, ca), and [0, cd) below ca
        auto hide = [&](uint32_t (&r)[32], int c0) {  // scores of keys c0 .. c0 + 31 of the step
          auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
          const uint32_t sees = below(ca - c0) & (~below(cb - c0) | below(cd - c0));
#pragma unroll
          for (int c = 0; c < 32; ++c) r[c] = (sees >> c) & 1u ? r[c] : 0xff800000u;
        };
        // The row's reference is the maximum (rounded up to a whole number, so that references differ by powers of two) of the
        // first step of which it sees a key, and stays as long as the weights stay below 2^20. The maximum of every step,
        // formed first, costs a quarter of the instructions.
        float m_new = m;
        if (__any_sync(0xffffffffu, m == -CUDART_INF_F)) {
          float mx = -CUDART_INF_F;
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tS(buf) + lane_off + 32 * b, r);
            tmem_ld_wait();
            if (border) hide(r, 32 * b);
            mx = fmaxf(mx, max32(r));
          }
          if (m == -CUDART_INF_F) m_new = ceilf(mx * scale_log2);
        }
        // p = 2^(s * scale_log2 - m_new): packed fp32x2 FMA for the argument, packed adds for the row sum; P is cut into its
        // two bf16 parts, 32 keys at a time, which go over these keys' scores: 16 columns of the large parts, 16 of the small ones.
        const uint64_t c2 = pack_f32x2(scale_log2, scale_log2);
        const uint64_t minus1 = pack_f32x2(-1.0f, -1.0f);
        float sum = 0.0f;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t r[32], pp16[32];  // (the large parts of the 32 keys' weights, two to a column, then the small ones)
          tmem_ld_32x32b_x32(tS(buf) + lane_off + 32 * b, r);
          tmem_ld_wait();
          if (border) hide(r, 32 * b);
          float part;
#pragma unroll 1
          for (bool again = false;; again = true) {
            const float ref = m_new == -CUDART_INF_F ? 0.0f : m_new;  // (nothing visible so far: weights of 0)
            const uint64_t nm2 = pack_f32x2(-ref, -ref);
            uint64_t sum2a = pack_f32x2(0.0f, 0.0f), sum2b = sum2a;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a0, a1;
              unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), c2, nm2), a0, a1);
              const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
              const uint64_t pp = pack_f32x2(p0, p1);
              if (i & 1) sum2b = add_f32x2(sum2b, pp);
              else sum2a = add_f32x2(sum2a, pp);
              const uint32_t large = pack_bf16x2(p0, p1);
              float l0, l1;  // what the large part leaves (exact)
              unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(large << 16), __uint_as_float(large & 0xffff0000u)), minus1, pp), l0, l1);
              pp16[i] = large;
              pp16[16 + i] = pack_bf16x2(l0, l1);
            }
            float sa0, sa1, sb0, sb1;
            unpack_f32x2(sum2a, sa0, sa1);
            unpack_f32x2(sum2b, sb0, sb1);
            part = (sa0 + sa1) + (sb0 + sb1);
            const bool much = !(part <= kTooMuch);
            if (again || !__any_sync(0xffffffffu, much)) break;
            // Rare: scores far above the reference (or none at all). It moves, by a power of two, and the step's weights that are
            // written already move with it.
            const float moved = much ? fmaxf(m_new, ceilf(max32(r) * scale_log2)) : m_new;
            const float down = m_new - moved;  // (a whole number)
            const float f = m_new == moved ? 1.0f : down > -126.5f ? __int_as_float((127 + static_cast<int>(down)) << 23) : 0.0f;
            sum *= f;
            m_new = moved;
            auto scaled = [&](uint32_t x) { return pack_bf16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
            tmem_st_wait();
#pragma unroll 1
            for (int c = 0; c < b; ++c) {
              uint32_t x[32];
              tmem_ld_32x32b_x32(tS(buf) + lane_off + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = scaled(x[e]);
              tmem_st_32x32b_x32(tS(buf) + lane_off + 32 * c, x);
            }
          }
          sum += part;
          tmem_st_32x32b_x32(tS(buf) + lane_off + 32 * b, pp16);  // (over the 32 scores)
        }
        const float alpha = ex2_approx(m - (m_new == -CUDART_INF_F ? 0.0f : m_new));  // 0 on the first step (m = -inf)
        if (j > pc.k0 && __any_sync(0xffffffffu, m_new != m)) {  // O moves with the reference, once PV[j-1] is complete
          if (!mbar_wait_warp(pv_done(t, g - 1), ((g - 1) >> 1) & 1, wc, 18)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO(t) + lane_off + half * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st_32x32b_x32(tO(t) + lane_off + half * 32, o);
          }
        }
        tmem_st_wait();
        l = l * alpha + sum;
        m = m_new;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t, g));
      }
      if (!ok || !mbar_wait_warp(pv_done(t, g - 1), ((g - 1) >> 1) & 1, wc, 19)) break;
      // The piece's result, from O in TMEM once the PV product of its last step is done; the next piece's first PV product
      // (which overwrites O) waits for P that this warp writes only after these reads.
      tc_fence_after();
      const bool whole = pc.k0 == 0 && pc.k1 == pc.n;
      const int i = pc.u.i0 + t * a.tokens + tok;  // the row's token of the sequence
      const bool mine = tok < a.tokens && i <= pc.u.i1;
      const int token = pc.row0 + i, head = pc.hk * p.r + hr;
      const bool put = mine && in_bounds(token >= 0 && token < p.n_tokens && head < p.H, err, 123);
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (pc.k0 == 0 ? 1 : 0);
      float zero = l * 0.0f;  // a number, as long as all of the row's are
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO(t) + lane_off + half * 32, o);
        tmem_ld_wait();
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<long long>(token) * p.out_stride + head * (HD * 2) + half * 64);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = __uint_as_float(o[8 * q + e]);
              zero = fmaf(f[e], 0.0f, zero);
            }
            if (put)
              dst[q] = make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                                  pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
          }
        } else if (put) {
          float4* d4 = reinterpret_cast<float4*>(a.part_o + (slot * 2 * BQ + t * BQ + row) * HD + half * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            d4[q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]), __uint_as_float(o[4 * q + 2]),
                                __uint_as_float(o[4 * q + 3]));
        }
      }
      tc_fence_before();
      if (!whole) {
        if (put) a.part_ml[slot * 2 * BQ + t * BQ + row] = make_float2(m, l);
        if (warp == 4 && lane == 0 && pc.k0 == 0) {  // the first piece of a unit that is cut: how many follow
          long long c = blockIdx.x + 1;
          while (c < of_run[1] && of_run[0] * c / of_run[1] < pc.end) ++c;
          a.cuts[blockIdx.x] = ChunkCut{pc.seq, pc.hk, pc.x, static_cast<int>(c - blockIdx.x)};
        }
      } else if (put && (!(zero == 0.0f) || (l == 0.0f && pc.pos0 + i >= 0))) {  // (rare: see chunk_redo)
        *reinterpret_cast<uint4*>(p.out + static_cast<long long>(token) * p.out_stride + head * (HD * 2)) =
            make_uint4(kChunkMark, kChunkMark, kChunkMark, kChunkMark);
        a.runs[blockIdx.x].redo = 1;
      }
      give(np);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// The marked rows of the units that were whole within CTA blockIdx.x's run: block (c, y) forms rows 32 y .. of each again, four
// rows a warp. All warps walk the run. Measured: 2048 tokens behind 14000 keys, a fourth of whose rows see a NaN, 39 ms instead
// of 0.23 (a key takes some 1.2 us, from dependent loads); three tokens of 128 heads behind 59000 keys 138 ms.
__device__ __noinline__ void redo_run(const ChunkParams& p, const ChunkTcArgs& a, uint32_t* err) {
  const int row = 32 * blockIdx.y + (threadIdx.x >> 3), c8 = (threadIdx.x & 7) * 8;  // 8 threads a row
  const int t = row / BQ, tok = row % BQ / p.r, hr = row % BQ - tok * p.r;
  Walk run(a.runs[blockIdx.x]);
  while (run.next(p, a, err)) {
    const Piece& pc = run.pc;
    if (pc.k0 != 0 || pc.k1 != pc.n) continue;
    const int i = pc.u.i0 + t * a.tokens + tok, token = pc.row0 + i, head = pc.hk * p.r + hr;
    bool mine = tok < a.tokens && i <= pc.u.i1 && in_bounds(token >= 0 && token < p.n_tokens && head < p.H, err, 126);
    if (mine) {
      const uint8_t* at = p.out + static_cast<long long>(token) * p.out_stride + head * (HD * 2);
      mine = *reinterpret_cast<const uint32_t*>(at) == kChunkMark;
    }
    if (!__any_sync(0xffffffffu, mine)) continue;
    const int tt = mine ? token : pc.row0, hh = mine ? head : 0;
    float v[8], l = CUDART_NAN_F;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = CUDART_NAN_F;
    chunk_redo<__nv_bfloat16>(p, pc.seq, pc.hk, p.q + static_cast<long long>(tt) * p.q_stride + hh * (HD * 2), pc.pos0 + i, mine,
                              pc.u.ks.lo, pc.u.ks.hi, pc.u.ks.first, c8, v, &l, err);
    if (mine) chunk_write8<__nv_bfloat16>(p, token, head, c8, v, l, err);
  }
}

// Units that were cut: block (c, y) joins rows 32 y .. of the unit whose first piece CTA c wrote with those of the CTAs behind it.
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkTcArgs a,
                                                         uint32_t* err) {
  pdl_trigger();
  pdl_wait();
  if (a.runs[blockIdx.x].redo) redo_run(p, a, err);
  const ChunkCut cut = a.cuts[blockIdx.x];
  if (cut.pieces == 0) return;
  const ChunkSeq sq = chunk_seq(p, cut.seq, err);
  const Unit u(p, sq.m, sq.len, a.per_unit, cut.x);
  const int row = 32 * blockIdx.y + (threadIdx.x >> 3), c8 = (threadIdx.x & 7) * 8;  // 8 threads a row
  const int t = row / BQ, tok = row % BQ / p.r, hr = row % BQ - tok * p.r;
  const int i = u.i0 + t * a.tokens + tok, token = sq.row0 + i, head = cut.hk * p.r + hr;
  const bool in = tok < a.tokens && i <= u.i1 && in_bounds(token < p.n_tokens && head < p.H, err, 124);
  // piece k: the first CTA's second slot, then the first slots of the CTAs behind it
  auto slot = [&](int k) { return (2 * static_cast<size_t>(blockIdx.x + k) + (k == 0 ? 1 : 0)) * 2 * BQ + row; };
  float v[8] = {}, m = -CUDART_INF_F, l = 0.0f;
  if (in) {
    for (int k = 0; k < cut.pieces; ++k) m = fmaxf(m, a.part_ml[slot(k)].x);
    const float ref = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll 2
    for (int k = 0; k < cut.pieces; ++k) {
      const float2 ml = a.part_ml[slot(k)];
      const float4* o = reinterpret_cast<const float4*>(a.part_o + slot(k) * HD + c8);
      const float4 o0 = o[0], o1 = o[1];
      const float f = ex2_approx(ml.x - ref);
      l += f * ml.y;
      v[0] += f * o0.x; v[1] += f * o0.y; v[2] += f * o0.z; v[3] += f * o0.w;
      v[4] += f * o1.x; v[5] += f * o1.y; v[6] += f * o1.z; v[7] += f * o1.w;
    }
  }
  if (__any_sync(0xffffffffu, in && !chunk_numbers(v, l, sq.len - sq.m + i))) {
    const int tt = in ? token : sq.row0, hh = in ? head : 0;
    chunk_redo<__nv_bfloat16>(p, cut.seq, cut.hk, p.q + static_cast<long long>(tt) * p.q_stride + hh * (HD * 2), sq.len - sq.m + i, in,
                              u.ks.lo, u.ks.hi, u.ks.first, c8, v, &l, err);
  }
  if (in) chunk_write8<__nv_bfloat16>(p, token, head, c8, v, l, err);
}

}  // namespace

namespace wenc_host {

namespace {
// The workspace's parts, and its size in `end`.
struct Room {
  size_t runs, part_o, part_ml, end;
  explicit Room(int sms) {
    const size_t n = static_cast<size_t>(sms);
    runs = (n * sizeof(ChunkCut) + 255) / 256 * 256;
    part_o = runs + (n * sizeof(ChunkRun) + 255) / 256 * 256;
    part_ml = part_o + n * 2 * 2 * BQ * HD * sizeof(float);
    end = part_ml + n * 2 * 2 * BQ * sizeof(float2);
  }
};
}  // namespace

size_t chunk_tc_workspace(int sms) { return Room(sms).end; }

cudaError_t launch_chunk_tc(const ChunkParams& p, int few, void* workspace, uint32_t* err, int sms, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured{-1};
  e = opt_in_smem(chunk_tc_kernel, SMEM, dev, configured);
  if (e != cudaSuccess) return e;
  // The softmax warpgroups' register increase is met only from the registers the CTA was launched with: refuse to
  // launch a build that was given fewer (a property of the build).
  static const int launch_regs = registers_of(chunk_tc_kernel);
  if (launch_regs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  ChunkTcArgs a;
  a.few = few;
  a.tokens = BQ / p.r;
  a.per_unit = 2 * a.tokens;
  uint8_t* room = static_cast<uint8_t*>(workspace);
  const Room at(sms);
  a.cuts = reinterpret_cast<ChunkCut*>(room);
  a.runs = reinterpret_cast<ChunkRun*>(room + at.runs);
  a.part_o = reinterpret_cast<float*>(room + at.part_o);
  a.part_ml = reinterpret_cast<float2*>(room + at.part_ml);
  e = launch_pdl(chunk_tc_kernel, dim3(sms), dim3(kThreads), SMEM, stream, p, a, err);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_join_kernel, dim3(sms, 2 * BQ / 32), dim3(256), 0, stream, p, a, err);
}

}  // namespace wenc_host
