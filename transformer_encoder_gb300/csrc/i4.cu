// i4.cu -- the matrix product with 4-bit weights that have a scale for each group of inputs.
//
//   out_mn = epilogue(sum_g scale_ng sum_{k in g} (u_nk - 8) x_mk + bias_n),   groups of 32, 64 or 128
// (oxinfer 0.0.5 src/whisper/model.rs, make_lin: quantised weights; here with groups of inputs).
//
// u - 8 is exact in bf16, a bf16 x times it is exact in fp32, so a group's product runs on the bf16 tensor cores without a
// rounding of either operand, and the scale, which would not fit into the weight exactly, multiplies the group's fp32 sum.
// float32 x is cut into three bf16 parts (8 + 8 + 8 significant bits: exact together), the products of which share a group's
// sum.
//
// Two forms, on the device in us: up to 16 tokens on mma.sync, where a token costs little beside the weights' bytes and latency
// (tokens x N x K: 1 x 1152 x 384 3.7, 16 x 5120 x 1280 6.3, 1 x 7680 x 5120 14.4, where 1.4 TB/s of weights wait for loads of
// four bytes a lane, one piece ahead), more on tcgen05 (24 x 5120 x 1280 8.0, 80 x 5120 x 1280 11.4, 2240 x 1280 x 5120 33.4,
// 880 TFLOP/s; float32 300 x 1280 x 1280 15).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <string>

#include "launch.h"
#include "mma.cuh"
#include "ptx.cuh"
#include "wenc.h"

wenc_status wenc_internal_fail(wenc_status s, const char* msg);
void wenc_internal_clear_error();
int wenc_internal_sm_count();
wenc_status wenc_internal_device(int* sms, uint32_t** err);

namespace {

using namespace wenc_dev;
using wenc_host::Range;
using wenc_host::share;

struct I4Params {
  const void* x;
  const uint8_t* w;
  const void* scale;
  const float *bias, *resid;
  void* out;
  int M, N, K, group, groups;  // groups: K / group
  int scale_f32, out_f32, epilogue, ksplit;
};

// Four of a word's eight weights' pairs: pair s holds weights s and s + 4 as bf16. As the low bits of 128's pattern a
// weight reads 128 + u, exact to subtract 136 from (bf16 has 8 significant bits).
__device__ __forceinline__ uint32_t widen_pair(uint32_t w, int s) {
  uint32_t v = ((w >> (4 * s)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 base = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
  const __nv_bfloat162 y = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), base);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Weights 2 i and 2 i + 1 of a word as bf16 (hi: the word shifted right by 4), likewise.
__device__ __forceinline__ uint32_t widen_byte(uint32_t w, uint32_t hi, int i) {
  // (bytes i of both: the low one's low half in bits 0 .. 3, the high one's in bits 16 .. 19)
  uint32_t v = (__byte_perm(w, hi, i | i << 4 | (4 + i) << 8 | (4 + i) << 12) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 base = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
  const __nv_bfloat162 y = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), base);
  return *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ float scale_at(const I4Params& p, size_t i) {
  return p.scale_f32 ? __ldg(static_cast<const float*>(p.scale) + i)
                     : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.scale) + i)) << 16);
}

// x = a + b + c, each the upper 16 bits of a float: the leading 8 significant bits, the next 8 and the last 8, cut off, not
// rounded (so that nothing next to the largest float leaves the range). An infinity or a NaN is its own first part.
__device__ __forceinline__ void split3(float x, uint32_t& a, uint32_t& b, uint32_t& c) {
  const bool finite = fabsf(x) < __uint_as_float(0x7f800000u);
  a = __float_as_uint(x) & 0xffff0000u;
  if (x != x) a = 0x7fc00000u;
  const float r = finite ? x - __uint_as_float(a) : 0.0f;
  b = __float_as_uint(r) & 0xffff0000u;
  c = __float_as_uint(r - __uint_as_float(b));
}

// The value that an output element takes, from the sum of its products.
__device__ __forceinline__ float gelu_erf(float z) { return 0.5f * z * erfcf(-0.70710678118654752f * z); }

__device__ __forceinline__ void put(const I4Params& p, size_t at, float v) {
  if (p.epilogue == WENC_EPI_BIAS_RESID_F32) {
    static_cast<float*>(p.out)[at] = p.resid[at] + v;
    return;
  }
  if (p.epilogue == WENC_EPI_BIAS_GELU_BF16) v = gelu_erf(v);
  if (p.out_f32) static_cast<float*>(p.out)[at] = v;
  else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// Four neighbours; res: the residual's.
__device__ __forceinline__ void put4(const I4Params& p, size_t at, float4 v, const float4& res) {
  if (p.epilogue == WENC_EPI_BIAS_RESID_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(res.x + v.x, res.y + v.y, res.z + v.z, res.w + v.w);
  } else if (p.out_f32) {
    if (p.epilogue == WENC_EPI_BIAS_GELU_BF16) v = make_float4(gelu_erf(v.x), gelu_erf(v.y), gelu_erf(v.z), gelu_erf(v.w));
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
  } else {
    if (p.epilogue == WENC_EPI_BIAS_GELU_BF16) {
      gelu_erf_x2(v.x, v.y);
      gelu_erf_x2(v.z, v.w);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// ---------------------------------------------------------------- few tokens
// out^T = W x^T for up to 8 NT tokens: a CTA takes 16 channels (the MMA's M), its warps share K in pieces of 128, and the CTAs
// of a cluster share it further; they are joined through shared memory, in the order of the warps. Weights go from global
// memory to registers: a lane takes the word (8 weights) that its MMA rows need of each 32 inputs, so a group's products stay
// together for every group size, and x comes in the same order of k from L1 or L2.
constexpr int kRowsWarps = 8;
constexpr int kPiece = 128;  // inputs of a warp's piece

template <typename T, int NT>
__global__ void __launch_bounds__(32 * kRowsWarps) i4_rows_kernel(const __grid_constant__ I4Params p, uint32_t* err) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int TOK = 8 * NT, PARTS = F32 ? 3 : 1;
  __shared__ float red[kRowsWarps][16][TOK + 1];
  __shared__ float sum[TOK][16];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int rank = blockIdx.x % p.ksplit, n0 = blockIdx.x / p.ksplit * 16, m0 = blockIdx.y * TOK;
  const int pieces = p.K / kPiece, step = kRowsWarps * p.ksplit;
  const uint8_t* wrow = p.w + static_cast<size_t>(n0 + g) * (p.K / 2) + 4 * tq;
  const size_t row8 = static_cast<size_t>(8) * (p.K / 2);
  const bool fits = in_bounds(n0 + 16 <= p.N, err, 113);
  float tot[NT][4], acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) tot[n][e] = acc[n][e] = 0.0f;
  uint32_t w[2][4];
  auto fetch = [&](uint32_t (&v)[2][4], int piece) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = wrow + piece * (kPiece / 2) + 16 * i;
      v[0][i] = __ldg(reinterpret_cast<const uint32_t*>(at));
      v[1][i] = __ldg(reinterpret_cast<const uint32_t*>(at + row8));
    }
  };
  int piece = rank * kRowsWarps + warp;
  if (piece < pieces && fits) fetch(w, piece);
  for (; piece < pieces && fits; piece += step) {
    uint32_t next[2][4] = {};
    if (piece + step < pieces) fetch(next, piece + step);
    const size_t s0 = static_cast<size_t>(n0 + g) * p.groups, s1 = s0 + static_cast<size_t>(8) * p.groups;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[2][4];  // two MMAs' weights
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[j][e] = widen_pair(w[e & 1][i], 2 * j + (e >> 1));
      const int k = piece * kPiece + 32 * i + 8 * tq;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = m0 + 8 * n + g;
        const bool in = m < p.M && in_bounds(k + 8 <= p.K, err, 114);
        const T* src = static_cast<const T*>(p.x) + static_cast<size_t>(in ? m : 0) * p.K + k;
        // the lane's eight inputs as parts of bf16 pairs (j, j + 4)
        uint32_t b[PARTS][4];
        if constexpr (F32) {
          const float4 lo = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 hi = in ? *reinterpret_cast<const float4*>(src + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t c[3], d[3];
            split3(l[e], c[0], c[1], c[2]);
            split3(h[e], d[0], d[1], d[2]);
#pragma unroll
            for (int q = 0; q < 3; ++q) b[q][e] = __byte_perm(c[q], d[q], 0x7632);
          }
        } else {
          const uint4 u = in ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
          b[0][0] = __byte_perm(u.x, u.z, 0x5410);
          b[0][1] = __byte_perm(u.x, u.z, 0x7632);
          b[0][2] = __byte_perm(u.y, u.w, 0x5410);
          b[0][3] = __byte_perm(u.y, u.w, 0x7632);
        }
        // (the small parts first: the tensor core's sums truncate)
#pragma unroll
        for (int q = PARTS - 1; q >= 0; --q)
#pragma unroll
          for (int j = 0; j < 2; ++j) mma_bf16(acc[n], a[j], b[q][2 * j], b[q][2 * j + 1]);
      }
      if ((32 * (i + 1)) % p.group == 0) {  // the group is complete
        const int grp = (piece * kPiece + 32 * i) / p.group;
        const float f0 = scale_at(p, s0 + grp), f1 = scale_at(p, s1 + grp);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            tot[n][e] = fmaf(e < 2 ? f0 : f1, acc[n][e], tot[n][e]);
            acc[n][e] = 0.0f;
          }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[r][i] = next[r][i];
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][g + 8 * (e >> 1)][8 * n + 2 * tq + (e & 1)] = tot[n][e];
  __syncthreads();
  const int m_here = min(TOK, p.M - m0);
  for (int i = threadIdx.x; i < 16 * m_here; i += 32 * kRowsWarps) {
    const int c = i & 15, t = i >> 4;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kRowsWarps; ++q) v += red[q][c][t];
    if (p.ksplit > 1) sum[t][c] = v;
    else if (in_bounds(m0 + t < p.M, err, 115)) put(p, static_cast<size_t>(m0 + t) * p.N + n0 + c, v + __ldg(p.bias + n0 + c));
  }
  if (p.ksplit > 1) {
    cluster_arrive_wait();
    const uint32_t part = smem_u32(sum);
    for (int i = threadIdx.x + 32 * kRowsWarps * rank; i < 16 * m_here; i += 32 * kRowsWarps * p.ksplit) {
      const int c = i & 15, t = i >> 4;
      float v = 0.0f;
      for (int q = 0; q < p.ksplit; ++q) {
        float y;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(rank_addr(part + i * 4, q)) : "memory");
        v += y;
      }
      if (in_bounds(m0 + t < p.M, err, 115)) put(p, static_cast<size_t>(m0 + t) * p.N + n0 + c, v + __ldg(p.bias + n0 + c));
    }
    cluster_arrive_wait();  // no CTA leaves while another reads its sums
  }
}

// ---------------------------------------------------------------- many tokens
// out^T = W x^T on tcgen05: a CTA takes 128 channels (the MMA's M, TMEM's lanes) and up to 160 tokens (its N), and the CTAs of
// a cluster share K where there are few tiles. Four warps widen the weights from global memory straight into TMEM, a channel a
// thread: the A operand. x comes by TMA as it lies (float32: its three parts, cut apart by i4_split_kernel first). A group's
// products make an accumulator of their own, one of two in TMEM; eight warps, a channel a thread again, add it times the
// group's scale to their sums in registers while the MMAs fill the other. So a scale is one number a thread and group, and no
// weight is rounded.
// What bounds it: the MMAs (80 cycles for each 16 inputs of 160 tokens; busy 41% of the cycles at 2240 x
// 1280 x 5120, whose 140 CTAs begin and end together), and with groups of 32 the reading of accumulators. At 80 x 5120 x 1280,
// two CTAs to a K, five pieces in a row of some 0.8 us each, and some 7 us of a CTA's beginning, join and end. Not kept: four
// pieces unrolled in the issuers (41.6 us against 35 for the large one: code past the instruction cache), four accumulators of
// 80 tokens (no gain), the output unrolled (12.5 us against 11.4 for the small one).
constexpr int kTcMost = 160;                // tokens of a tile
constexpr int kTcThreads = 512;             // 4 widening warps, 2 MMA issuers, TMA producer, a warp for the scales, 8 summing warps
constexpr int kAStages = 2, kXStages = 4;   // of 128 inputs
constexpr uint32_t kXHalf = kTcMost * 128;  // 64 inputs of a tile's tokens
constexpr uint32_t kXBytes = 2 * kXHalf;
constexpr int kSStages = 3, kSGroups = 8;   // scales: stages of eight groups, [group][128 channels] as fp32
constexpr uint32_t kSBytes = kSGroups * 128 * 4;
constexpr uint32_t kTcScales = kXStages * kXBytes;
constexpr uint32_t kTcBars = kTcScales + kSStages * kSBytes;
constexpr int kTcNumBars = 2 * kAStages + 2 * kXStages + 4 + 1 + 2 * kSStages + 2;
constexpr size_t kTcSmem = 1024 + kTcBars + kTcNumBars * 8 + 16;
constexpr uint32_t kTcColumns = 512;        // sums 0..159, 160..319; A stages from 384 on, 64 each
static_assert(kTcSmem <= 232448 && kTcMost * 128 * 4 <= static_cast<int>(kTcScales), "the sums of the output lie over the stages");

struct I4Tc {
  int tok, n_tiles;  // tokens of a tile; channel tiles
};

// PARTS of x: 1, or 3 (planes of M rows); groups of GROUP inputs.
template <int PARTS, int GROUP>
__global__ void __launch_bounds__(kTcThreads, 1)
    i4_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ I4Params p, const I4Tc c, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem), bar0 = s0 + kTcBars;
  auto a_full = [&](int i) { return bar0 + 8u * i; };
  auto a_empty = [&](int i) { return bar0 + 8u * (kAStages + i); };
  auto x_full = [&](int i) { return bar0 + 8u * (2 * kAStages + i); };
  auto x_empty = [&](int i) { return bar0 + 8u * (2 * kAStages + kXStages + i); };
  auto d_full = [&](int i) { return bar0 + 8u * (2 * kAStages + 2 * kXStages + i); };
  auto d_empty = [&](int i) { return bar0 + 8u * (2 * kAStages + 2 * kXStages + 2 + i); };
  const uint32_t drain = bar0 + 8u * (2 * kAStages + 2 * kXStages + 4);
  auto s_full = [&](int i) { return drain + 8u * (1 + i); };
  auto s_empty = [&](int i) { return drain + 8u * (1 + kSStages + i); };
  auto turn = [&](int i) { return drain + 8u * (1 + 2 * kSStages + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTcBars + kTcNumBars * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, err};
  // (numbers of the whole warp come from lane 0, so that the compiler knows them for such: operands of an MMA that it takes
  // for a lane's own are moved for every MMA)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.ksplit, tile = blockIdx.x / p.ksplit;
  const int n0 = tile % c.n_tiles * 128, m0 = tile / c.n_tiles * c.tok, m_here = min(c.tok, p.M - m0);
  // this CTA's share of K, in pieces of 128 (whole groups)
  const int pieces = p.K / kPiece, per = (pieces + p.ksplit - 1) / p.ksplit;
  const int first = min(rank * per, pieces), n_pieces = min(per, pieces - first);
  const int k_begin = first * kPiece, n_groups = n_pieces * kPiece / GROUP;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kAStages; ++i) {
      mbar_init(a_full(i), 4);   // the widening warps
      mbar_init(a_empty(i), 1);  // the MMAs' commit
    }
    for (int i = 0; i < kXStages; ++i) {
      mbar_init(x_full(i), 1);
      mbar_init(x_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(d_full(i), 1);
      mbar_init(d_empty(i), 8);  // the summing warps
    }
    mbar_init(drain, 2);
    mbar_init(turn(0), 1);       // the issuers take turns
    mbar_init(turn(1), 1);
    for (int i = 0; i < kSStages; ++i) {
      mbar_init(s_full(i), 1);   // the warp that fetches scales
      mbar_init(s_empty(i), 8);  // the summing warps
    }
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tx);
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_slot), kTcColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_trigger();  // TMEM is held: the next kernel may be scheduled
  pdl_wait();
  auto tD = [&](int i) { return tmem + kTcMost * i; };
  auto tA = [&](int i) { return tmem + 384u + 64u * i; };
  const bool fits = in_bounds(n0 + 128 <= p.N && k_begin + n_pieces * kPiece <= p.K && m0 < p.M, err, 125);

  bool ok = fits;
  if (warp < 4) {
    // ---------------- widening: thread = channel; the next piece's weights are under way
    const uint4* row = reinterpret_cast<const uint4*>(p.w + static_cast<size_t>(n0 + threadIdx.x) * (p.K / 2) + k_begin / 2);
    uint4 w[4];
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(row + 4 * j + i);
    };
    if (ok && n_pieces > 0) fetch(0);
#pragma unroll 1
    for (int j = 0; ok && j < n_pieces; ++j) {
      const int st = j % kAStages;
      uint32_t r[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v[8] = {w[2 * h].x, w[2 * h].y, w[2 * h].z, w[2 * h].w, w[2 * h + 1].x, w[2 * h + 1].y, w[2 * h + 1].z, w[2 * h + 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) r[h][4 * i + e] = widen_byte(v[i], v[i] >> 4, e);
      }
      if (j + 1 < n_pieces) fetch(j + 1);
      if (!mbar_wait_warp(a_empty(st), ((j / kAStages) & 1) ^ 1u, wc, 60)) break;
      tc_fence_after();
      tmem_st_32x32b_x32(tA(st) + (static_cast<uint32_t>(32 * warp) << 16), r[0]);
      tmem_st_32x32b_x32(tA(st) + 32u + (static_cast<uint32_t>(32 * warp) << 16), r[1]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full(st));
    }
  } else if (warp == 4 || warp == 6) {
    // ---------------- MMA issuers, two for every other piece: the whole warp waits, one thread issues.
    // A group's MMAs are straight lines behind one election (44 cycles each, or their own time; with a branch between them 110 to 130). What lies between the lines,
    // waits that are over and a descriptor, is some 700 cycles a piece, more than its MMAs take: so the other issuer's run
    // meanwhile. They go in turn: a wait tells one phase of a barrier from the next, not from the one after.
    constexpr int kLine = GROUP < 64 ? GROUP : 64, kSteps = kLine / 16, kLines = kPiece / kLine;  // (a group of 128 in two)
    static_assert(kXStages == 4 && kAStages == 2, "slots and parities by masks");
    const uint32_t idesc = idesc_bf16_f32(128, (m_here + 15) / 16 * 16, false);
#pragma unroll 1
    for (int j = warp == 6; ok && j < n_pieces; j += 2) {
      const uint32_t a_slot = j & 1;
      uint64_t desc[PARTS];
      uint32_t x_bar[PARTS];
      ok = mbar_wait_warp(a_full(a_slot), j >> 1 & 1, wc, 61);
      auto tiles = [&]() {
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          const uint32_t xi = j * PARTS + q;
          ok = ok && mbar_wait_warp(x_full(xi & 3), xi >> 2 & 1, wc, 62);
          desc[q] = sdesc_sw128(s0 + (xi & 3) * kXBytes, 16, 1024);
          x_bar[q] = x_empty(xi & 3);
        }
      };
      // (one tile a piece: an issuer's slots are its own; three: the other issuer's tiles come between, so its turn comes first)
      if (PARTS == 1) tiles();
      const uint32_t a_at = tA(a_slot), a_bar = a_empty(a_slot), other = turn(a_slot ^ 1);
      if (j > 0) ok = ok && mbar_wait_warp(turn(a_slot), (j - 1) >> 1 & 1, wc, 68);
      if (PARTS > 1) tiles();
#pragma unroll
      for (int i = 0; i < kLines; ++i) {
        const bool begins = i * kLine % GROUP == 0, ends = (i + 1) * kLine % GROUP == 0;
        const uint32_t grp = j * (kPiece / GROUP) + i * kLine / GROUP, buf = grp & 1;
        if (begins) ok = ok && mbar_wait_warp(d_empty(buf), (grp >> 1 & 1) ^ 1u, wc, 63);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_at = tmem + (buf ? static_cast<uint32_t>(kTcMost) : 0u), d_bar = d_full(buf);
        if (elect_one()) {
#pragma unroll
          for (int k = i * kSteps; k < (i + 1) * kSteps; ++k)
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
              umma_bf16_ts(d_at, a_at + 8 * k, desc[q] + (k >> 2) * (kXHalf >> 4) + 2 * (k & 3), idesc,
                           !begins || k > i * kSteps || q > 0 ? 1u : 0u);
          if (ends) umma_commit(d_bar);
          if (i == kLines - 1) {
            umma_commit(a_bar);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) umma_commit(x_bar[q]);
            mbar_arrive(other);
          }
        }
        __syncwarp();
      }
    }
    // every MMA issued completes before anything is freed
    if (elect_one()) {  // (the thread that issued them)
      umma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------- x by TMA, its small parts first (the tensor core's sums truncate)
    if (lane == 0) {
      int xi = 0;
      for (int j = 0; ok && j < n_pieces; ++j)
        for (int q = PARTS - 1; q >= 0; --q, ++xi) {
          const int st = xi % kXStages;
          if (!mbar_wait(x_empty(st), ((xi / kXStages) & 1) ^ 1u, wc, 64)) { ok = false; break; }
          mbar_arrive_expect_tx(x_full(st), static_cast<uint32_t>(c.tok) * 256u);
          tma_load_2d(s0 + st * kXBytes, &tx, x_full(st), k_begin + kPiece * j, q * p.M + m0);
          tma_load_2d(s0 + st * kXBytes + kXHalf, &tx, x_full(st), k_begin + kPiece * j + 64, q * p.M + m0);
        }
      if (*abort_flag)  // error path: let the copies already issued land before the CTA exits
        for (int i = (xi > kXStages ? xi - kXStages : 0); i < xi; ++i) mbar_wait_drain(x_full(i % kXStages), (i / kXStages) & 1);
    }
    __syncwarp();
  } else if (warp == 7) {
    // ---------------- the scales of eight groups at a time, four channels a lane, two stages ahead of what is stored: their
    // latency would be the summing warps' otherwise
    const size_t row = static_cast<size_t>(n0 + lane) * p.groups + k_begin / GROUP, step = static_cast<size_t>(32) * p.groups;
    uint32_t raw[2][4][kSGroups];
    auto fetch = [&](uint32_t (&r)[4][kSGroups], int g0) {  // (as they lie: nothing waits for a load before it is widened)
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < kSGroups; ++i) {
          r[h][i] = 0;
          if (fits && g0 + i < n_groups) {
            if (p.scale_f32) asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r[h][i]) : "l"(static_cast<const uint32_t*>(p.scale) + row + h * step + g0 + i));
            else asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(r[h][i]) : "l"(static_cast<const uint16_t*>(p.scale) + row + h * step + g0 + i));
          }
        }
    };
    fetch(raw[0], 0);
    fetch(raw[1], kSGroups);
    const int shift = p.scale_f32 ? 0 : 16;
#pragma unroll 1
    for (int g0 = 0, b = 0; ok && g0 < n_groups; g0 += 2 * kSGroups) {
#pragma unroll
      for (int d = 0; d < 2; ++d, ++b) {
        if (!ok || g0 + d * kSGroups >= n_groups) break;
        const int st = b % kSStages;
        if (!mbar_wait_warp(s_empty(st), ((b / kSStages) & 1) ^ 1u, wc, 66)) { ok = false; break; }
        float* to = reinterpret_cast<float*>(smem + kTcScales + st * kSBytes) + lane;
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int i = 0; i < kSGroups; ++i) to[i * 128 + 32 * h] = __uint_as_float(raw[d][h][i] << shift);
        __syncwarp();
        if (lane == 0) mbar_arrive(s_full(st));
        fetch(raw[d], g0 + (d + 2) * kSGroups);
      }
    }
  }
  // ---------------- summing: thread = channel; warps 8 .. 11 the first half of the tokens, 12 .. 15 the second
  const int ch = 32 * (warp & 3) + lane, half = c.tok / 2, t0 = warp >= 12 ? half : 0;  // (tok is a multiple of 16)
  float acc[kTcMost / 2];
  if (warp >= 8) {
#pragma unroll
    for (int i = 0; i < kTcMost / 2; ++i) acc[i] = 0.0f;
    for (int g0 = 0, b = 0; ok && g0 < n_groups; g0 += kSGroups, ++b) {
      const int st = b % kSStages;
      if (!mbar_wait_warp(s_full(st), (b / kSStages) & 1, wc, 67)) { ok = false; break; }
      const float* scales = reinterpret_cast<const float*>(smem + kTcScales + st * kSBytes) + ch;
#pragma unroll 1
      for (int i = 0; i < kSGroups && g0 + i < n_groups; ++i) {
        const int g = g0 + i, buf = g & 1;
        const float s = scales[i * 128];
        if (!mbar_wait_warp(d_full(buf), (g >> 1) & 1, wc, 65)) { ok = false; break; }
        tc_fence_after();
        const uint64_t s2 = pack_f32x2(s, s);
        const uint32_t from = tD(buf) + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t0;
        // (columns of the other half or behind the tokens add what nobody reads)
        auto add = [&](const uint32_t* r, int b, int n) {
#pragma unroll
          for (int e = 0; e < n; e += 2) {
            float x, y;
            unpack_f32x2(fma_f32x2(s2, pack_f32x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), pack_f32x2(acc[b + e], acc[b + e + 1])), x, y);
            acc[b + e] = x;
            acc[b + e + 1] = y;
          }
        };
        static_assert(kTcMost / 2 == 80, "two loads of 32 and one of 16");
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
          if (b >= half) break;  // (uniform)
          uint32_t r[32];
          tmem_ld_32x32b_x32(from + b, r);
          tmem_ld_wait();
          add(r, b, 32);
        }
        if (half > 64) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(from + 64, r);
          tmem_ld_wait();
          add(r, 64, 16);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(buf));
      }
      if (lane == 0) mbar_arrive(s_empty(st));  // (behind the last group's __syncwarp)
    }
  }
  // ---------------- output. The sums go over the stages as [token][channel] (every MMA and copy is done: the sums waited for the
  // last group, and the last MMA read the last tile); then the warps of the cluster's CTAs share the tokens out, four channels a
  // lane, in a loop that is small: the epilogue unrolled over 80 sums a thread was 150 KB of code, and 30 us of a cold call.
  __syncthreads();
  if (warp >= 8) {
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < kTcMost / 2; ++i)
      if (i < half && t0 + i < m_here) part[(t0 + i) * 128 + ch] = acc[i];
  }
  __syncwarp();
  if (p.ksplit > 1) cluster_arrive_wait();
  else __syncthreads();
  if (fits && !*abort_flag) {
    constexpr int kAhead = 4;  // tokens whose residual is on its way before the first store (`out` may be `resid`)
    const int stride = p.ksplit * (kTcThreads / 32);
    const float4 bn = __ldg(reinterpret_cast<const float4*>(p.bias + n0) + lane);
#pragma unroll 1
    for (int t = rank + p.ksplit * warp; t < m_here; t += kAhead * stride) {
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.epilogue == WENC_EPI_BIAS_RESID_F32 && t + i * stride < m_here)
          v[i] = *(reinterpret_cast<const float4*>(p.resid + static_cast<size_t>(m0 + t + i * stride) * p.N + n0) + lane);
      }
#pragma unroll 1
      for (int i = 0; i < kAhead && t + i * stride < m_here; ++i) {
        const int tt = t + i * stride;
        float4 y = bn;
        if (p.ksplit == 1) {
          const float4 z = *reinterpret_cast<const float4*>(smem + tt * 512 + lane * 16);
          y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        } else {
          for (int r = 0; r < p.ksplit; ++r) {
            const float4 z = ld_cluster_f4(rank_addr(s0 + tt * 512 + lane * 16, r));
            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
          }
        }
        const float4 res = i < 2 ? (i == 0 ? v[0] : v[1]) : (i == 2 ? v[2] : v[3]);
        put4(p, static_cast<size_t>(m0 + tt) * p.N + n0 + 4 * lane, y, res);
      }
    }
  }
  __syncwarp();
  if (p.ksplit > 1) cluster_arrive_wait();  // no CTA leaves while another reads its sums
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcColumns);
  }
}

// float32 rows as three planes of bf16 parts.
__global__ void __launch_bounds__(256) i4_split_kernel(const float4* __restrict__ x, uint2* __restrict__ planes, long long n4, uint32_t* err) {
  pdl_trigger();
  pdl_wait();
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
    const float4 v = x[i];
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t part[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(f[e], part[e][0], part[e][1], part[e][2]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      planes[q * n4 + i] = make_uint2(__byte_perm(part[0][q], part[1][q], 0x7632), __byte_perm(part[2][q], part[3][q], 0x7632));
  }
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

wenc_status launch_failed(cudaError_t e) {
  char buf[200];
  snprintf(buf, sizeof(buf), "linear_i4 launch: %s", cudaGetErrorString(e));
  return wenc_internal_fail(WENC_ERR_CUDA, buf);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs that share K: as long as there are SMs without one, and every warp of theirs has a piece.
int pick_ksplit(long long tiles, int pieces, int sms) {
  int n = 1;
  while (n < 8 && tiles * n <= sms && pieces >= 2 * n * kRowsWarps) n *= 2;
  return n;
}

template <typename T, int NT>
cudaError_t launch_rows(I4Params p, int sms, uint32_t* err, cudaStream_t stream) {
  const int m_tiles = (p.M + 8 * NT - 1) / (8 * NT);
  p.ksplit = pick_ksplit(static_cast<long long>(p.N / 16) * m_tiles, p.K / kPiece, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.N / 16 * p.ksplit), static_cast<unsigned>(m_tiles));
  cfg.blockDim = dim3(32 * kRowsWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.ksplit);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ksplit > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, i4_rows_kernel<T, NT>, p, err);
}

constexpr int kRowsMost = 16;  // tokens up to which the product runs on mma.sync

size_t split_bytes(int M, int K, int x_dtype) {
  return M > kRowsMost && x_dtype == WENC_DTYPE_F32 ? (static_cast<size_t>(M) * K * 6 + 255) / 256 * 256 : 0;
}

// Tokens of a tile and CTAs that share K: the division whose rounds of the machine take least, in cycles of a piece of 128
// inputs (the MMAs' 4 a token, but no less than widening and, of every group, summing take) and of a CTA's beginning and end. The
// constants put divisions that were measured in their order; they foretell no times (some half of the measured cycles at 2240 x
// 1280 x 5120, and 24 and 80 tokens x 5120 x 1280 come out alike, which take 8.0 and 11.4 us). Where K is shared, an end adds
// the joining. 80 x 5120 x 1280, on 152 SMs: one CTA to a K (ten pieces) 15.4 us, two 11.4, three 10.9 (only powers of two are
// tried), four 17.6 (160 CTAs: a second round).
constexpr long long kWidenCycles = 600, kSumCycles = 350, kEndCycles = 5000, kJoinCycles = 1500;
void pick_tiles(int M, int n_tiles, int K, int group, int parts, int sms, int& tok, int& ksplit) {
  const int least = (M + kTcMost - 1) / kTcMost, pieces = K / kPiece;
  long long best = -1;
  for (int tiles = least; tiles <= least + 16 && tiles <= (M + 15) / 16; ++tiles) {
    const int t = ((M + tiles - 1) / tiles + 15) / 16 * 16;
    long long piece = 4ll * parts * t;
    if (piece < kWidenCycles) piece = kWidenCycles;
    if (piece < kPiece / group * kSumCycles) piece = kPiece / group * kSumCycles;
    for (int ks = 1; ks <= 8 && pieces >= ks; ks *= 2) {
      const long long ctas = static_cast<long long>(n_tiles) * ((M + t - 1) / t) * ks, rounds = (ctas + sms - 1) / sms;
      const long long cost = rounds * ((pieces + ks - 1) / ks * piece + kEndCycles + (ks > 1 ? kJoinCycles : 0));
      if (best < 0 || cost < best) {
        best = cost;
        tok = t;
        ksplit = ks;
      }
    }
  }
}

wenc_status launch_tc(I4Params p, bool f32, void* workspace, int sms, uint32_t* err, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  using Kernel = void (*)(const CUtensorMap, const I4Params, const I4Tc, uint32_t*);
  static const Kernel kernels[6] = {i4_tc_kernel<1, 32>, i4_tc_kernel<1, 64>, i4_tc_kernel<1, 128>,
                                    i4_tc_kernel<3, 32>, i4_tc_kernel<3, 64>, i4_tc_kernel<3, 128>};
  static std::atomic<int> configured[6] = {{-1}, {-1}, {-1}, {-1}, {-1}, {-1}};
  const int which = (f32 ? 3 : 0) + (p.group == 32 ? 0 : p.group == 64 ? 1 : 2);
  const Kernel kern = kernels[which];
  if (e == cudaSuccess) e = wenc_host::opt_in_smem(kern, kTcSmem, dev, configured[which]);
  const void* x = p.x;
  if (e == cudaSuccess && f32) {
    const long long n4 = static_cast<long long>(p.M) * p.K / 4;
    long long blocks = (n4 + 255) / 256;
    if (blocks > 16ll * sms) blocks = 16ll * sms;
    e = wenc_host::launch_pdl(i4_split_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, static_cast<const float4*>(x),
                              static_cast<uint2*>(workspace), n4, err);
    x = workspace;
  }
  if (e == cudaSuccess) {
    I4Tc c;
    c.n_tiles = p.N / 128;
    const int parts = f32 ? 3 : 1;
    pick_tiles(p.M, c.n_tiles, p.K, p.group, parts, sms, c.tok, p.ksplit);
    const long long tiles = static_cast<long long>(c.n_tiles) * ((p.M + c.tok - 1) / c.tok);
    if (tiles * p.ksplit > 0x7fffffffll) return bad(WENC_ERR_UNSUPPORTED, "linear_i4: %lld tiles pass 2^31 - 1", tiles);
    CUtensorMap tx;
    std::string why;
    if (!wenc_host::make_tmap_2d_bf16(&tx, x, p.K, static_cast<uint64_t>(p.M) * parts, static_cast<uint64_t>(p.K) * 2, 64, c.tok, &why))
      return wenc_internal_fail(WENC_ERR_INVALID_ARG, why.c_str());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.ksplit));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kTcSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.ksplit);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ksplit > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, tx, p, c, err);
  }
  return e == cudaSuccess ? WENC_OK : launch_failed(e);
}

}  // namespace

extern "C" size_t wenc_linear_i4_workspace(int M, int N, int K, int x_dtype, int group) {
  wenc_internal_clear_error();
  if (M < 1 || N < 1 || K < 1 || group < 1) return 0;
  return split_bytes(M, K, x_dtype);
}

extern "C" wenc_status wenc_linear_i4(const void* x, int x_dtype, const uint8_t* w, const void* w_scale, int scale_dtype,
                                      const float* bias, const float* resid, void* out, int M, int N, int K, int group,
                                      int epilogue, void* workspace, size_t workspace_bytes, wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!x || !w || !w_scale || !bias || !out) return bad(WENC_ERR_INVALID_ARG, "linear_i4: x/w/w_scale/bias/out is NULL");
  if ((x_dtype != WENC_DTYPE_F32 && x_dtype != WENC_DTYPE_BF16) || (scale_dtype != WENC_DTYPE_F32 && scale_dtype != WENC_DTYPE_BF16))
    return bad(WENC_ERR_INVALID_ARG, "linear_i4: x_dtype %lld or scale_dtype %lld unknown", x_dtype, scale_dtype);
  if (epilogue < 0 || epilogue > 2) return bad(WENC_ERR_INVALID_ARG, "epilogue %lld unknown", epilogue);
  if (epilogue == WENC_EPI_BIAS_RESID_F32 && !resid) return bad(WENC_ERR_INVALID_ARG, "resid is NULL");
  if (M < 1) return bad(WENC_ERR_INVALID_ARG, "M must be >= 1");
  if (M > (1 << 28)) return bad(WENC_ERR_UNSUPPORTED, "M %lld: at most 2^28", M);
  if (N < 128 || N % 128 != 0) return bad(WENC_ERR_UNSUPPORTED, "N %lld: must be a positive multiple of 128", N);
  if (K < 128 || K % 128 != 0) return bad(WENC_ERR_UNSUPPORTED, "K %lld: must be a positive multiple of 128", K);
  if (group != 32 && group != 64 && group != 128) return bad(WENC_ERR_UNSUPPORTED, "group %lld: 32, 64 or 128", group);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(w_scale, 16) || !aligned(bias, 16) || !aligned(resid, 16) || !aligned(out, 16))
    return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  // (inputs are read while others' results are written; a residual is read by the threads that write over it)
  const bool joins = epilogue == WENC_EPI_BIAS_RESID_F32;
  const long long es = x_dtype == WENC_DTYPE_F32 ? 4 : 2, ss = scale_dtype == WENC_DTYPE_F32 ? 4 : 2, rows = M;
  const Range out_at[] = {{out, rows * N * (joins ? 4 : es)}};
  const Range room_at[] = {{workspace, static_cast<long long>(split_bytes(M, K, x_dtype))}};
  const Range resid_at[] = {{joins ? resid : nullptr, rows * N * 4}};
  const Range in[] = {{x, rows * K * es}, {w, static_cast<long long>(N) * (K / 2)},
                      {w_scale, static_cast<long long>(N) * (K / group) * ss}, {bias, 4ll * N}};
  if (share(in, out_at)) return bad(WENC_ERR_INVALID_ARG, "linear_i4: out must lie apart from x, w, w_scale and bias");
  if (resid != out && share(resid_at, out_at))
    return bad(WENC_ERR_INVALID_ARG, "linear_i4: out must be resid or lie apart from it");
  if (share(in, room_at) || share(resid_at, room_at) || share(out_at, room_at))
    return bad(WENC_ERR_INVALID_ARG, "linear_i4: the workspace must lie apart from the other arguments");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  I4Params p = {};
  p.x = x;
  p.w = w;
  p.scale = w_scale;
  p.bias = bias;
  p.resid = resid;
  p.out = out;
  p.M = M;
  p.N = N;
  p.K = K;
  p.group = group;
  p.groups = K / group;
  p.scale_f32 = scale_dtype == WENC_DTYPE_F32;
  p.out_f32 = x_dtype == WENC_DTYPE_F32;
  p.epilogue = epilogue;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = x_dtype == WENC_DTYPE_F32;
  if (M > kRowsMost) {
    const size_t need = split_bytes(M, K, x_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return bad(WENC_ERR_INVALID_ARG, "linear_i4: workspace of %lld bytes needed, %lld given", static_cast<long long>(need),
                 workspace ? static_cast<long long>(workspace_bytes) : 0ll);
    if (need > 0 && !aligned(workspace, 256)) return bad(WENC_ERR_INVALID_ARG, "linear_i4: the workspace must be 256-byte aligned");
    return launch_tc(p, f32, workspace, sms, err, s);
  }
  cudaError_t e;
  if (M <= 8) e = f32 ? launch_rows<float, 1>(p, sms, err, s) : launch_rows<__nv_bfloat16, 1>(p, sms, err, s);
  else e = f32 ? launch_rows<float, 2>(p, sms, err, s) : launch_rows<__nv_bfloat16, 2>(p, sms, err, s);
  return e == cudaSuccess ? WENC_OK : launch_failed(e);
}
