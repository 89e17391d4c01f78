// i8.cu -- the matrix product in 8-bit integers with a scale for each token and each channel, and
// the rows of integers it takes.
//
//   scale_m = max_k |x_mk| (1 / 127),  xq_mk = round(x_mk / scale_m)                   (quantize)
//   out_mn = epilogue((sum_k xq_mk wq_nk) scale_m wscale_n + bias_n)                   (product)
// (oxinfer 0.0.5 src/whisper/model.rs, make_lin Q8: 8-bit weights; here one scale spans a whole row,
// so that it leaves the sum).
//
// sm_103a has no integer form of the fifth-generation MMA, and GB300's older integer units are far
// slower than its 16-bit ones. Integers up to 128 are exact in bf16 (8 significant bits) and in fp16, a
// product (at most 2^14) is exact in the fp32 accumulator, and so is every sum below 2^24; longer sums
// round as any fp32 sum does. So the product runs on the 16-bit tensor cores, in three forms:
//  - up to 16 tokens (a decode step of few beams): mma.sync on weights that go from global memory to
//    registers (i8_rows_kernel): a 128-row tcgen05 tile would give too few CTAs to keep the weights' bytes
//    coming;
//  - up to an output tile of 128 x 128 per SM, or few tokens and many channels: tcgen05 on operands widened on the
//    chip (i8_tc_kernel), no workspace;
//  - more: the operands are widened to bf16 in the workspace and multiplied by the GEMM of gemm.cu, whose
//    epilogue applies the scales. On-chip widening repeats itself in every tile, and its loads and stores then
//    bind the shared-memory pipe (24000 x 1280 x 5120: 399 us against 266 us for both passes; at 1024 x 1280
//    x 5120 both take 34 us, at 256 x 1280 x 5120 it is 16 against 32 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstdio>
#include <string>

#include "launch.h"
#include "ptx.cuh"
#include "wenc.h"

wenc_status wenc_internal_fail(wenc_status s, const char* msg);
void wenc_internal_clear_error();
int wenc_internal_sm_count();
wenc_status wenc_internal_device(int* sms, uint32_t** err);

namespace {

using namespace wenc_dev;

// x / s rounded to the nearest integer, ties to even, as of the exact quotient: n = rint(x * inv) is
// within one of it; the remainder x - n s (one FMA, exact for the n that matter) says which way.
__device__ __forceinline__ int quantum(float x, float s, float inv, float half) {
  float n = rintf(x * inv);
  const float e = fmaf(-n, s, x);
  if (fabsf(e) > half) n += copysignf(1.0f, e);
  else if (fabsf(e) == half && (static_cast<int>(n) & 1)) n += copysignf(1.0f, e);
  n = fminf(fmaxf(n, -127.0f), 127.0f);
  return static_cast<int>(n);
}

// ---------------------------------------------------------------- quantize_rows
// One 16-byte vector of a row as fp32, and the largest magnitude in it, as the bits of a non-negative
// float (ordered as integers; an infinity or a NaN is 0x7f800000 or more).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ uint32_t amax(const uint4& u) {
    return max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ uint32_t amax(const uint4& u) {
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// A row's scale and what dividing by it takes.
struct RowScale {
  float scale, up, s, inv, half;  // s = scale * up; half = s / 2
  bool zero;                      // all integers are 0
  __device__ __forceinline__ explicit RowScale(uint32_t amax) {
    const bool bad = amax >= 0x7f800000u;
    scale = bad ? CUDART_NAN_F : __uint_as_float(amax) * (1.0f / 127.0f);
    zero = bad || scale == 0.0f;
    // rows of tiny values are scaled up (exactly) first: neither 1 / s nor s / 2 leaves the range then
    up = scale < 0x1p-100f ? 0x1p64f : 1.0f;
    s = scale * up;
    inv = zero ? 0.0f : __frcp_rn(s);
    half = 0.5f * s;
  }
};

// The integers of a vector, packed: n = x * inv rounded by adding 1.5 * 2^23, whose low byte then is n.
// The remainder x - n s (one FMA, exact) proves n the nearest unless it reaches s / 2 in magnitude: then, or
// in a row of tiny values (whose scale may be too coarse for 127), quantum() decides each element.
template <int E>
__device__ __forceinline__ void quantize_vec(const float (&f)[E], const RowScale& r, uint32_t (&q)[E / 4]) {
  const float magic = 12582912.0f;
  uint32_t b[E];
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float t = fmaf(f[i], r.inv, magic);
    worst = fmaxf(worst, fabsf(fmaf(magic - t, r.s, f[i])));
    b[i] = __float_as_uint(t);
  }
  if (r.zero || r.up != 1.0f || worst >= r.half) {
#pragma unroll
    for (int i = 0; i < E; ++i) b[i] = r.zero ? 0u : static_cast<uint32_t>(quantum(f[i] * r.up, r.s, r.inv, r.half));
  }
#pragma unroll
  for (int i = 0; i < E / 4; ++i)
    q[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
}

// (24000 rows of 5120 bf16: 57 us, 6.5 TB/s, 95% of the measured copy rate; with the row read twice and every integer
// formed by compares, 109 us. 80 rows of 1280: 2.3 us.)
// One pass: a row's vectors stay in the registers of its threads (a warp, or the block: WARP) between the
// maximum and the division. What bounds it: bytes (x once, the integers once).
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) quantize_rows_kernel(const T* __restrict__ x, int8_t* __restrict__ xq,
                                                             float* __restrict__ scale, int rows, int nv,
                                                             uint32_t* err) {
  using V = Vec<T>;
  __shared__ uint32_t part[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (row >= rows) return;  // (a whole warp; the block form has a block for each row)
  // (the threads' vectors cover the row, and each is checked against its end)
  if (!in_bounds(VPT * (WARP ? 32 : static_cast<int>(blockDim.x)) >= nv, err, 99)) return;
  const int first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x) + row * nv;
  uint4 v[VPT];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < VPT; ++i) v[i] = first + i * step < nv ? xr[first + i * step] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < VPT; ++i) m = max(m, V::amax(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (!WARP) {
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, part[lane < (blockDim.x >> 5) ? lane : 0]);
  }
  const RowScale r(m);
  if (first == 0) scale[row] = r.scale;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (first + i * step >= nv) continue;
    float f[V::E];
    uint32_t q[V::E / 4];
    V::unpack(v[i], f);
    quantize_vec<V::E>(f, r, q);
    uint32_t* dst = reinterpret_cast<uint32_t*>(xq) + (row * nv + first + i * step) * (V::E / 4);
    if constexpr (V::E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
    else *dst = q[0];
  }
}

// Rows longer than the registers of a block hold (131072 bytes): read twice.
template <typename T>
__global__ void __launch_bounds__(1024) quantize_long_rows_kernel(const T* __restrict__ x, int8_t* __restrict__ xq,
                                                                  float* __restrict__ scale, int nv) {
  using V = Vec<T>;
  __shared__ uint32_t part[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x) + row * nv;
  uint32_t m = 0u;
  for (int i = threadIdx.x; i < nv; i += 1024) m = max(m, V::amax(xr[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) part[warp] = m;
  __syncthreads();
  const RowScale r(__reduce_max_sync(0xffffffffu, part[lane]));
  if (threadIdx.x == 0) scale[row] = r.scale;
  for (int i = threadIdx.x; i < nv; i += 1024) {
    float f[V::E];
    uint32_t q[V::E / 4];
    V::unpack(xr[i], f);
    quantize_vec<V::E>(f, r, q);
    uint32_t* dst = reinterpret_cast<uint32_t*>(xq) + (row * nv + i) * (V::E / 4);
    if constexpr (V::E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
    else *dst = q[0];
  }
}

template <typename T, int VPT>
cudaError_t launch_quantize(const T* x, int8_t* xq, float* scale, int rows, int nv, int threads, uint32_t* err, cudaStream_t s) {
  if (threads == 32)  // a warp per row, four rows a block
    return wenc_host::launch_pdl(quantize_rows_kernel<T, VPT, true>, dim3((rows - 1) / 4 + 1), dim3(128), 0, s, x, xq, scale, rows, nv, err);
  return wenc_host::launch_pdl(quantize_rows_kernel<T, VPT, false>, dim3(rows), dim3(threads), 0, s, x, xq, scale, rows, nv, err);
}

// Threads per row: a warp up to 64 vectors (two a lane); else the fewest, from 128, that keep a row within
// eight vectors a thread.
template <typename T>
cudaError_t quantize(const T* x, int8_t* xq, float* scale, int rows, int d, uint32_t* err, cudaStream_t s) {
  const int nv = d / Vec<T>::E;
  if (nv > 8 * 1024)
    return wenc_host::launch_pdl(quantize_long_rows_kernel<T>, dim3(rows), dim3(1024), 0, s, x, xq, scale, nv);
  int threads = 32;
  if (nv > 64) {
    threads = 128;
    while (threads * 8 < nv) threads *= 2;
  }
  const int vpt = (nv + threads - 1) / threads;
  if (vpt <= 2) return launch_quantize<T, 2>(x, xq, scale, rows, nv, threads, err, s);
  if (vpt <= 4) return launch_quantize<T, 4>(x, xq, scale, rows, nv, threads, err, s);
  if (vpt <= 6) return launch_quantize<T, 6>(x, xq, scale, rows, nv, threads, err, s);
  return launch_quantize<T, 8>(x, xq, scale, rows, nv, threads, err, s);
}

// ---------------------------------------------------------------- few tokens
// Four int8 to four fp16, two to a register: with its sign bit flipped a byte is b + 128; as the low byte
// of 1024's pattern it reads 1024 + 128 + b, exact to subtract from (fp16 has 11 significant bits).
__device__ __forceinline__ void widen_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 base = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), base), y = __hsub2(*reinterpret_cast<__half2*>(&b), base);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_rank_f32(uint32_t saddr, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(rank_addr(saddr, rank)) : "memory");
  return v;
}

// out^T = W x^T for up to 8 NT tokens: a CTA takes 32 channels and a share of K (the CTAs of a cluster split
// K between them and join through distributed shared memory). Its eight warps are two groups of 16 channels
// (the MMA's M) times four quarters of a round: per round of 256 k, warp (c, q) multiplies channels 16 c .. + 15
// by the 64 k of quarter q. The order of k within those 64 is free as long as both operands agree: a lane
// takes 16 consecutive bytes of a weight row, which are four MMAs' worth of its fragments, so weights go from
// global memory to registers in full 64-byte pieces and are widened there; the tokens are widened once
// per CTA and round into shared memory, in the same order, rows 16 bytes past a multiple of 128 apart so
// that the fragment loads touch all banks. Weights and tokens of the next rounds are on their way meanwhile, and the
// tokens' two buffers leave one barrier a round.
// What bounds it: at a decode step's sizes, latency; the weights' bytes beyond. 1 x 1536 x 384 with its quantize_rows:
// 3.2 us (10.0 in the two-pass form); 8 x 5120 x 1280: 3.7 us for 6.6 MB of weights (4.5 with one round under way); 1 x
// 51968 x 1280: 15.6 us, 4.3 TB/s; 1 x 20480 x 5120: 27 us, 3.9 TB/s (35.6). Against the tcgen05 form below, with one round
// under way: at 16 tokens 5.5 us (5120 x 1280; now 4.6), 3.9 (1536 x 512), 7.7 (1280 x 5120; now 6.4); at 32, 6.9 / 7.0, 5.5 / 4.5 and 10.7 / 9.4; at 80, 13.9
// / 9.1, 9.5 / 5.9 and 21.3 / 12.1.
constexpr int kRowsChannels = 32;
constexpr int kRowsK = 256;  // k per round

template <int NT>
struct RowsCfg {
  static constexpr int TOK = 8 * NT;
  static constexpr int XROW = kRowsK * 2 + 16;            // bytes of a token's round in shared memory
  static constexpr int XN = (TOK * (kRowsK / 16) + 255) / 256;  // 16-byte pieces of x per thread and round
  static constexpr int RED = 8 * 16 * (TOK + 1) * 4;      // the warps' sums
  static constexpr int XBUF = TOK * XROW;                 // two of them
  static constexpr int SMEM = 2 * XBUF > RED ? 2 * XBUF : RED;
};

// AHEAD rounds of weights are under way (even: the tokens' buffers alternate), and the registers are for CTAS per SM.
template <int NT, int AHEAD, int CTAS>
__global__ void __launch_bounds__(256, CTAS) i8_rows_kernel(const int8_t* __restrict__ xq, const float* __restrict__ x_scale,
                                                         const int8_t* __restrict__ wq, const float* __restrict__ w_scale,
                                                         const float* __restrict__ bias, const float* resid, void* out, int M,
                                                         int N, int K, int ksplit, int epilogue, uint32_t* err) {
  using C = RowsCfg<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int c16 = warp & 1, quarter = warp >> 1;
  const int rank = blockIdx.x % ksplit;
  const int n0 = blockIdx.x / ksplit * kRowsChannels;
  // this CTA's k: whole pieces of 64, as equal as they divide
  const int pieces = K / 64, per = (pieces + ksplit - 1) / ksplit;
  const int k_begin = min(rank * per, pieces) * 64, k_end = min((rank + 1) * per, pieces) * 64;

  const int8_t* wa = wq + static_cast<size_t>(n0 + 16 * c16 + g) * K + 16 * tq;
  const int8_t* wb = wa + static_cast<size_t>(8) * K;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 w[AHEAD][2], xv[2][C::XN];
  // weights and tokens of the round that starts at k0, as far as it lies before k_end
  auto fetch_w = [&](uint4 (&w)[2], int k0) {
    const int k = k0 + 64 * quarter;
    const bool in = k < k_end && in_bounds(n0 + kRowsChannels <= N && k >= 0 && k + 64 <= K, err, 100);
    w[0] = in ? __ldg(reinterpret_cast<const uint4*>(wa + k)) : zero;
    w[1] = in ? __ldg(reinterpret_cast<const uint4*>(wb + k)) : zero;
  };
  auto fetch_x = [&](uint4 (&x)[C::XN], int k0) {
#pragma unroll
    for (int i = 0; i < C::XN; ++i) {
      const int at = threadIdx.x + 256 * i, tok = at / (kRowsK / 16), kk = k0 + at % (kRowsK / 16) * 16;
      x[i] = tok < M && kk < k_end && in_bounds(kk >= 0 && kk + 16 <= K, err, 101) ? *reinterpret_cast<const uint4*>(xq + static_cast<size_t>(tok) * K + kk) : zero;
    }
  };
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) fetch_w(w[d], k_begin + d * kRowsK);
  fetch_x(xv[0], k_begin);
  fetch_x(xv[1], k_begin + kRowsK);
  for (int k00 = k_begin; k00 < k_end; k00 += AHEAD * kRowsK) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      const int k0 = k00 + d * kRowsK;
      if (k0 >= k_end) break;
      uint8_t* buf = smem + (d & 1) * C::XBUF;
      // tokens of this round into shared memory as fp16, each 16-byte piece as 32 bytes
#pragma unroll
      for (int i = 0; i < C::XN; ++i) {
        const int at = threadIdx.x + 256 * i, tok = at / (kRowsK / 16), piece = at % (kRowsK / 16);
        const uint4 x = xv[d & 1][i];
        if (tok < C::TOK) {
          uint4 a, b;
          widen_half(x.x, a.x, a.y);
          widen_half(x.y, a.z, a.w);
          widen_half(x.z, b.x, b.y);
          widen_half(x.w, b.z, b.w);
          uint4* dst = reinterpret_cast<uint4*>(buf + tok * C::XROW + piece * 32);
          dst[0] = a;
          dst[1] = b;
        }
      }
      fetch_x(xv[d & 1], k0 + 2 * kRowsK);
      uint32_t wf[4][4];  // the fragments of four MMAs
      const uint4 w0 = w[d][0], w1 = w[d][1];
      widen_half(w0.x, wf[0][0], wf[0][2]);
      widen_half(w1.x, wf[0][1], wf[0][3]);
      widen_half(w0.y, wf[1][0], wf[1][2]);
      widen_half(w1.y, wf[1][1], wf[1][3]);
      widen_half(w0.z, wf[2][0], wf[2][2]);
      widen_half(w1.z, wf[2][1], wf[2][3]);
      widen_half(w0.w, wf[3][0], wf[3][2]);
      widen_half(w1.w, wf[3][1], wf[3][3]);
      fetch_w(w[d], k0 + AHEAD * kRowsK);
      __syncthreads();  // (the next round writes the other buffer, which the last one's products have left)
      const uint8_t* xs = buf + g * C::XROW + quarter * 128 + tq * 32;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b0 = *reinterpret_cast<const uint4*>(xs + n * 8 * C::XROW);
        const uint4 b1 = *reinterpret_cast<const uint4*>(xs + n * 8 * C::XROW + 16);
        mma_f16(acc[n], wf[0], b0.x, b0.y);
        mma_f16(acc[n], wf[1], b0.z, b0.w);
        mma_f16(acc[n], wf[2], b1.x, b1.y);
        mma_f16(acc[n], wf[3], b1.z, b1.w);
      }
    }
  }
  __syncthreads();  // the sums go over the tokens
  // sums of the four quarters through shared memory: [warp][channel][token]
  float* red = reinterpret_cast<float*>(smem);
  constexpr int RS = C::TOK + 1;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[(warp * 16 + g + 8 * (e >> 1)) * RS + 8 * n + 2 * tq + (e & 1)] = acc[n][e];
  __syncthreads();
  // this CTA's sum of (channel, token), in warp c16 = channel / 16's place; a lane per channel
  auto sum4 = [&](int ch, int tok) {
    const float* r = red + (((ch >> 4) * 16) + (ch & 15)) * RS + tok;
    return (r[0] + r[2 * 16 * RS]) + (r[4 * 16 * RS] + r[6 * 16 * RS]);
  };
  if (ksplit > 1) {
    for (int at = threadIdx.x; at < kRowsChannels * C::TOK; at += 256) {
      const int ch = at & 31, tok = at >> 5;
      if (tok < M) red[((ch >> 4) * 16 + (ch & 15)) * RS + tok] = sum4(ch, tok);
    }
    cluster_arrive_wait();
  }
  const uint32_t red_addr = smem_u32(red);
  const int ch = lane, n = n0 + ch;
  const float ws = __ldg(w_scale + n), bn = __ldg(bias + n);
  for (int tok = warp * ksplit + rank; tok < M; tok += 8 * ksplit) {
    float a = 0.0f;
    if (ksplit > 1) {
      for (int r = 0; r < ksplit; ++r) a += ld_rank_f32(red_addr + (((ch >> 4) * 16 + (ch & 15)) * RS + tok) * 4, r);
    } else {
      a = sum4(ch, tok);
    }
    float v = fmaf(a, __ldg(x_scale + tok) * ws, bn), unused = 0.0f;
    const size_t at = static_cast<size_t>(tok) * N + n;
    if (!in_bounds(n < N, err, 102)) continue;
    if (epilogue == WENC_EPI_BIAS_RESID_F32) {
      static_cast<float*>(out)[at] = resid[at] + v;
    } else {
      if (epilogue == WENC_EPI_BIAS_GELU_BF16) gelu_erf_x2(v, unused);
      static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    }
  }
  if (ksplit > 1) cluster_arrive_wait();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------- a few tiles
// D[128 channels][up to 128 tokens] += W x^T on tcgen05, the weights as the A operand in TMEM, the tokens as
// the B operand in shared memory. Per 64 k (a stage): four warps load 16 bytes of weight rows a lane, widen
// them and store them to TMEM in the 16x256b shape, whose rows and columns are those of the loads
// (lane / 4 and 2 (lane % 4) + 0, 1 of every 8); four warps load 32 bytes of a token a lane, widen them and
// store them to the swizzled stage; one thread issues the MMAs. That order of the k is not the memory's:
// TMEM column 8 b + 2 t + e (k pair of the MMA) holds k = 16 t + 4 b + 2 e and the next, and the tokens are
// stored in the same order, which leaves the sum as it is. With A in TMEM the shared memory is written
// and read once per stage for the tokens alone (2 x 16 KB in the 256 cycles of the stage's MMAs, which is its
// bandwidth); both operands there would need twice that. Two CTAs share an SM (256 TMEM columns and 66 KB
// each), so that one's MMAs run under the other's first loads and epilogue. The channels are D's lanes: every
// store of a warp writes 32 neighbouring channels of one token. Few tiles: a cluster splits K and joins its sums
// through distributed shared memory.
// What bounds it: few tiles, latency (80 x 5120 x 1280, four CTAs to a cluster: 9.1 us, as 5 stages of loads, the
// join and the launch); many, the pipe that shared-memory and global accesses share (85% busy at 4096 x 1280 x 5120: a
// load instruction covers 8 or 16 rows of 64 bytes, a line each), which is why more tiles take the other form.
constexpr int kTcTok = 128;
constexpr int kTcStages = 4;
constexpr int kTcThreads = 288;  // 4 weight warps, 4 token warps, the issuing warp
constexpr uint32_t kTcStageBytes = kTcTok * 128;
constexpr uint32_t kTcBars = kTcStages * kTcStageBytes;
constexpr uint32_t kTcColumns = 256;  // D 0..127, A stages of 32 columns from 128
// More shared memory than the stages take, so that a third CTA never shares an SM with two of these, nor does a CTA
// of another TMEM kernel (they take 160 KB and more): it would wait in its TMEM allocation for one of the two to
// end, and these wait for the others of their cluster, which could be waiting in the same way elsewhere.
constexpr uint32_t kTcSmem = 77 * 1024;
static_assert(kTcSmem >= 1024 + kTcBars + (2 * kTcStages + 2) * 8 + 16 && 3 * (kTcSmem + 1024) > 228 * 1024,
              "shared memory of the on-chip form");

// kind::f16 with fp16 operands, both K-major, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 TMEM lanes x 32 columns: register 4 b + h of a lane is lane (thread / 4 + 8 (h / 2)), column
// 8 b + 2 (thread % 4) + h % 2.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__global__ void __launch_bounds__(kTcThreads, 2)
    i8_tc_kernel(const int8_t* __restrict__ xq, const float* __restrict__ x_scale, const int8_t* __restrict__ wq,
                 const float* __restrict__ w_scale, const float* __restrict__ bias, const float* resid, void* out, int M, int N,
                 int K, int ksplit, int epilogue, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem), bar0 = s0 + kTcBars;
  auto full = [&](int st) { return bar0 + 8u * st; };
  auto empty = [&](int st) { return bar0 + 8u * (kTcStages + st); };
  const uint32_t done = bar0 + 8u * (2 * kTcStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTcBars + (2 * kTcStages + 2) * 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int rank = blockIdx.x % ksplit;
  const int n0 = blockIdx.x / ksplit * 128, m0 = blockIdx.y * kTcTok, m_here = min(kTcTok, M - m0);
  const int pieces = K / 64, per = (pieces + ksplit - 1) / ksplit;
  const int first = min(rank * per, pieces), n_chunks = min(per, pieces - first);

  if (threadIdx.x == 0) {
    for (int st = 0; st < kTcStages; ++st) {
      mbar_init(full(st), 8);   // the eight converting warps
      mbar_init(empty(st), 1);  // the MMAs' commit
    }
    mbar_init(done, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), kTcColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, a_tmem = tmem + 128;
  pdl_trigger();  // TMEM is held: the next kernel may be scheduled
  pdl_wait();

  if (warp < 8) {
    // ---------------- load and widen: two stages' loads are kept in flight, and the loop is unrolled over the
    // ring, so that a stage costs little more than its widening.
    // Weight warps: rows 8 i + g of the warp's 32, bytes 16 tq ..; token warps: rows tok and 16 + tok of the
    // warp's 32, 32 bytes from 32 u (tok spreads the eight lanes of a store's quarter over all banks).
    const bool is_w = warp < 4;
    const int u = lane & 1, ti = lane >> 1, tok = ((ti & 3) << 1) | ((ti >> 2) & 1) | (ti & 8);
    const int8_t* src[4];
    bool there[2] = {true, true};
    if (is_w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) src[i] = wq + static_cast<size_t>(n0 + 32 * warp + 8 * i + g) * K + first * 64 + 16 * tq;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 32 * (warp & 3) + 16 * h + tok;
        there[h] = row < m_here;  // rows past the last token read as zeros (its own row stands in for the address)
        src[2 * h] = xq + static_cast<size_t>(m0 + (there[h] ? row : 0)) * K + first * 64 + 32 * u;
        src[2 * h + 1] = src[2 * h] + 16;
      }
    }
    auto load = [&](uint4 (&b)[4], int ahead) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = there[i >> 1] && in_bounds(src[i] + ahead * 64 >= (is_w ? wq : xq) &&
                                              src[i] + ahead * 64 + 16 <= (is_w ? wq + static_cast<size_t>(N) * K : xq + static_cast<size_t>(M) * K),
                                          err, 103)
                   ? __ldg(reinterpret_cast<const uint4*>(src[i] + ahead * 64))
                   : make_uint4(0u, 0u, 0u, 0u);
    };
    const uint32_t row0 = s0 + (32 * (warp & 3) + tok) * 128, a0 = a_tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    uint32_t at[4];  // where the four 16-byte pieces of a token's 32 bytes go (swizzled)
#pragma unroll
    for (int c = 0; c < 4; ++c) at[c] = row0 + (((2 * c + u) ^ (tok & 7)) << 4);
    auto convert = [&](const uint4 (&b)[4], int st, uint32_t parity) {
      if (!mbar_wait_warp(empty(st), parity, wc, 40)) return false;
      if (is_w) {
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // rows 16 h .. 16 h + 15 of the warp's lanes
          const uint4 lo = b[2 * h], hi = b[2 * h + 1];
          uint32_t r[16];
          widen_half(lo.x, r[0], r[1]);
          widen_half(hi.x, r[2], r[3]);
          widen_half(lo.y, r[4], r[5]);
          widen_half(hi.y, r[6], r[7]);
          widen_half(lo.z, r[8], r[9]);
          widen_half(hi.z, r[10], r[11]);
          widen_half(lo.w, r[12], r[13]);
          widen_half(hi.w, r[14], r[15]);
          tmem_st_16x256b_x4(a0 + 32 * st + (static_cast<uint32_t>(16 * h) << 16), r);
        }
        tmem_st_wait();
        tc_fence_before();
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t wa[4] = {b[2 * h].x, b[2 * h].y, b[2 * h].z, b[2 * h].w};
          const uint32_t wb[4] = {b[2 * h + 1].x, b[2 * h + 1].y, b[2 * h + 1].z, b[2 * h + 1].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t a0, a1, b0, b1;
            widen_half(wa[c], a0, a1);
            widen_half(wb[c], b0, b1);
            sts_v4(at[c] + st * kTcStageBytes + h * 16 * 128, a0, a1, b0, b1);
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full(st));
      return true;
    };
    static_assert(kTcStages == 4, "the loop below is unrolled over four stages");
    uint4 b0[4], b1[4];
    if (n_chunks > 0) load(b0, 0);
    if (n_chunks > 1) load(b1, 1);
    bool ok = true;
    uint32_t parity = 1;
    for (int j = 0; ok && j < n_chunks; j += 4, parity ^= 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (!ok || j + q >= n_chunks) break;
        ok = convert(q & 1 ? b1 : b0, q, parity);
        if (j + q + 2 < n_chunks) load(q & 1 ? b1 : b0, q + 2);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) src[i] += 4 * 64;
    }
    // ---------------- epilogue: warp w reads the channels of TMEM lane quadrant w % 4, tokens 64 (w / 4) ..
    if (ok && n_chunks > 0) ok = mbar_wait_warp(done, 0, wc, 41);
    tc_fence_after();
    const int ch = 32 * (warp & 3) + lane, tok0 = 64 * (warp >> 2);
    const float ws = __ldg(w_scale + n0 + ch), bn = __ldg(bias + n0 + ch);
    float* part = reinterpret_cast<float*>(smem);  // [token][128 channels], over the stages
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int t0 = tok0 + 32 * c;
      if (!ok || t0 >= m_here) break;  // warp-uniform
      uint32_t acc[32];
      if (n_chunks > 0) {
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t0, acc);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = 0u;
      }
      if (ksplit > 1) {
#pragma unroll
        for (int e = 0; e < 32; ++e) part[(t0 + e) * 128 + ch] = __uint_as_float(acc[e]);
        continue;
      }
      // (residual rows are all on their way before the first store: `out` may be `resid`, so the compiler cannot
      // move a load up over a store)
#pragma unroll
      for (int e0 = 0; e0 < 32; e0 += 16) {
        const size_t at0 = static_cast<size_t>(m0 + t0 + e0) * N + n0 + ch;
        float rr[16];
        if (epilogue == WENC_EPI_BIAS_RESID_F32) {
#pragma unroll
          for (int e = 0; e < 16; ++e) rr[e] = t0 + e0 + e < m_here ? resid[at0 + static_cast<size_t>(e) * N] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const int t = t0 + e0 + e;
          const bool in0 = t < m_here && in_bounds(m0 + t < M && n0 + ch < N, err, 104);
          const bool in1 = t + 1 < m_here && in_bounds(m0 + t + 1 < M && n0 + ch < N, err, 104);
          float v0 = fmaf(__uint_as_float(acc[e0 + e]), (in0 ? __ldg(x_scale + m0 + t) : 0.0f) * ws, bn);
          float v1 = fmaf(__uint_as_float(acc[e0 + e + 1]), (in1 ? __ldg(x_scale + m0 + t + 1) : 0.0f) * ws, bn);
          const size_t at = at0 + static_cast<size_t>(e) * N;
          if (epilogue == WENC_EPI_BIAS_RESID_F32) {
            float* o = static_cast<float*>(out);
            if (in0) o[at] = rr[e] + v0;
            if (in1) o[at + N] = rr[e + 1] + v1;
          } else {
            if (epilogue == WENC_EPI_BIAS_GELU_BF16) gelu_erf_x2(v0, v1);
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
            if (in0) o[at] = __float2bfloat16_rn(v0);
            if (in1) o[at + N] = __float2bfloat16_rn(v1);
          }
        }
      }
    }
  } else {
    // ---------------- MMA issuer: the whole warp waits, lane 0 issues
    const uint32_t idesc = idesc_f16_f32(128, (m_here + 15) / 16 * 16);
    for (int j = 0; j < n_chunks; ++j) {
      const int st = j % kTcStages;
      if (!mbar_wait_warp(full(st), (j / kTcStages) & 1, wc, 42)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t bd = sdesc_sw128(s0 + st * kTcStageBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(tmem, a_tmem + 32 * st + 8 * k, bd + 2 * k, idesc, (j | k) != 0 ? 1u : 0u);
        umma_commit(empty(st));
      }
      __syncwarp();
    }
    // every MMA issued completes before anything is read or freed
    if (lane == 0) {
      umma_commit(done);
      mbar_wait_drain(done, 0);
    }
    __syncwarp();
  }
  if (ksplit > 1) {
    // the CTAs' sums: the ranks share the tokens out, a warp a token, four channels a lane
    __syncwarp();
    cluster_arrive_wait();
    if (warp < 8) {
      const uint32_t part = s0 + lane * 16;
      const float4 ws = __ldg(reinterpret_cast<const float4*>(w_scale + n0) + lane), bn = __ldg(reinterpret_cast<const float4*>(bias + n0) + lane);
      for (int t = rank + ksplit * warp; t < m_here && !*abort_flag; t += ksplit * 8) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < ksplit; ++r) {
          const float4 v = ld_cluster_f4(rank_addr(part + t * 512, r));
          a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
        }
        const float xs = __ldg(x_scale + m0 + t);
        float4 v = make_float4(fmaf(a.x, xs * ws.x, bn.x), fmaf(a.y, xs * ws.y, bn.y), fmaf(a.z, xs * ws.z, bn.z), fmaf(a.w, xs * ws.w, bn.w));
        const size_t at = static_cast<size_t>(m0 + t) * N + n0 + 4 * lane;
        if (!in_bounds(m0 + t < M && n0 + 128 <= N, err, 104)) break;
        if (epilogue == WENC_EPI_BIAS_RESID_F32) {
          const float4 r = *reinterpret_cast<const float4*>(resid + at);
          *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(r.x + v.x, r.y + v.y, r.z + v.z, r.w + v.w);
        } else {
          if (epilogue == WENC_EPI_BIAS_GELU_BF16) {
            gelu_erf_x2(v.x, v.y);
            gelu_erf_x2(v.z, v.w);
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
      }
    }
    __syncwarp();
    cluster_arrive_wait();  // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcColumns);
  }
}

// ---------------------------------------------------------------- many tokens
// Four int8 (bytes of w) to four bf16. A byte b with its sign bit flipped is b + 128 = 0..255; set
// as the low byte of 2^23's pattern it reads 2^23 + b + 128 in fp32, exact to subtract from.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const float base = 8388608.0f + 128.0f;
  const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - base;
  const float b = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - base;
  const float c = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - base;
  const float d = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - base;
  return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// int8 -> bf16, 16 a thread: both operands in one launch. Bytes bind it: 123 MB + 246 MB in 74 us, 5.0 TB/s (four pieces
// in flight a thread, or the rows in reverse so that the newest come from L2, changed nothing). The GEMM behind it takes
// 192 us for 24000 x 1280 x 5120, 1640 TFLOP/s. Passes of rows whose widened copy stays in L2 cost more in the GEMM's
// last waves than they saved (279 against 249 us for both).
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* __restrict__ a, uint16_t* __restrict__ ab, size_t na,
                                                    const int8_t* __restrict__ w, uint16_t* __restrict__ wb, size_t nw) {
  pdl_trigger();
  pdl_wait();
  const size_t split = na / 16, total = split + nw / 16;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const bool is_a = i < split;
    const size_t j = is_a ? i : i - split;
    const uint4 v = reinterpret_cast<const uint4*>(is_a ? a : w)[j];
    const uint2 p0 = widen4(v.x), p1 = widen4(v.y), p2 = widen4(v.z), p3 = widen4(v.w);
    uint4* dst = reinterpret_cast<uint4*>(is_a ? ab : wb) + 2 * j;
    dst[0] = make_uint4(p0.x, p0.y, p1.x, p1.y);
    dst[1] = make_uint4(p2.x, p2.y, p3.x, p3.y);
  }
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

wenc_status launch_failed(const char* what, cudaError_t e) {
  char buf[200];
  snprintf(buf, sizeof(buf), "%s: %s", what, cudaGetErrorString(e));
  return wenc_internal_fail(WENC_ERR_CUDA, buf);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// The few-token form up to this many tokens.
constexpr int kRowsMost = 16;

// Whether the operands are widened on the chip: up to one output tile (128 x 128) per SM, and with more tiles where
// the weights are most of the bytes: one row of tiles, or two of long rows. Measured around it (us on the device, on the chip / two passes): 1536 x 512 at 128 tokens (12 tiles) 6.6 / 8.0, at 512 (48) 9.1 / 8.4, at
// 1024 (96) 11.1 / 9.5; 5120 x 1280 at 256 (80) 14.9 / 14.8, at 512 (160) 19.7 / 15.7; 1280 x 5120 at 256 (20) 15.6 /
// 31.7, at 1024 (80) 34.0 / 34.2; 51968 x 1280 at 80 (406 tiles) 40 / 69, at 256 62 / 71, at 384 96 / 96; 20480 x 512 at 80
// (160) 10.8 / 16.4, at 256 20.8 / 16.4; 51968 x 384 at 80 18.6 / 25.2, at 256 31.9 / 27.3. The second form's workspace, second launch and tensor maps cost its caller about 7 us
// more on the host, which is what an eager call of these sizes waits for.
bool on_chip(int M, int N, int K, int sms) {
  const int m_tiles = (M + kTcTok - 1) / kTcTok;
  return m_tiles == 1 || (m_tiles == 2 && K >= 1024) || static_cast<long long>(m_tiles) * (N / 128) <= sms;
}

// CTAs of a cluster that split K, for `tiles` output tiles: until the machine has a CTA per SM, none with
// fewer than `least` of the `pieces` of 64 k.
int pick_ksplit(long long tiles, int pieces, int least, int sms) {
  int n = 1;
  while (n < 8 && tiles * n <= sms && pieces >= 2 * n * least) n *= 2;
  return n;
}

void cluster_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], dim3 grid, int threads, size_t smem, int cluster,
                    cudaStream_t stream) {
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
}

cudaError_t launch_tc(int epilogue, const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale, const float* bias,
                      const float* resid, void* out, int M, int N, int K, int sms, uint32_t* err, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured{-1};
  e = wenc_host::opt_in_smem(i8_tc_kernel, kTcSmem, dev, configured);
  if (e != cudaSuccess) return e;
  const int m_tiles = (M + kTcTok - 1) / kTcTok;
  const int ksplit = pick_ksplit(static_cast<long long>(N / 128) * m_tiles, K / 64, 2, sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, dim3(N / 128 * ksplit, m_tiles), kTcThreads, kTcSmem, ksplit, stream);
  return cudaLaunchKernelEx(&cfg, i8_tc_kernel, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, ksplit, epilogue, err);
}

template <int NT, int AHEAD, int CTAS>
cudaError_t launch_rows_as(int ksplit, int epilogue, const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                           const float* bias, const float* resid, void* out, int M, int N, int K, uint32_t* err, cudaStream_t stream) {
  using C = RowsCfg<NT>;
  static_assert(C::SMEM <= 48 * 1024, "no opt-in for more shared memory");
  static_assert(AHEAD % 2 == 0, "the tokens' buffers alternate with the rounds");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, dim3(N / kRowsChannels * ksplit), 256, C::SMEM, ksplit, stream);
  return cudaLaunchKernelEx(&cfg, i8_rows_kernel<NT, AHEAD, CTAS>, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, ksplit, epilogue, err);
}

template <int NT>
cudaError_t launch_rows(int epilogue, const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale, const float* bias,
                        const float* resid, void* out, int M, int N, int K, int sms, uint32_t* err, cudaStream_t stream) {
  const int tiles = N / kRowsChannels;
  const int ksplit = pick_ksplit(tiles, K / 64, kRowsK / 64, sms);
  // More CTAs than two an SM: three are resident, and cover each other's latency. Else the loads under way have to: two
  // rounds, or four for up to 8 tokens (16 leave no registers) and rows of so many rounds. Measured (us, 1 and 16
  // tokens; three CTAs / two rounds / four): 51968 x 1280 15.6 17.8 23.8 and 22.2 27.4 27.9; 5120 x 5120 14.3 13.5 12.8
  // and 16.7 14.0 15.0; 5120 x 1280 4.5 4.1 3.7 and 5.6 4.7 4.8; 1536 x 384 2.07 2.07 2.23 and 2.6 2.75 2.7.
  if (tiles * ksplit > 2 * sms)
    return launch_rows_as<NT, 2, 3>(ksplit, epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, err, stream);
  if constexpr (NT == 1)
    if (K / ksplit >= 4 * kRowsK)
      return launch_rows_as<NT, 4, 2>(ksplit, epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, err, stream);
  return launch_rows_as<NT, 2, 2>(ksplit, epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, err, stream);
}

}  // namespace

extern "C" wenc_status wenc_quantize_rows(const void* x, int x_dtype, int8_t* xq, float* scale, int rows, int d,
                                          wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!x || !xq || !scale) return bad(WENC_ERR_INVALID_ARG, "quantize_rows: x/xq/scale is NULL");
  if (x_dtype != WENC_DTYPE_F32 && x_dtype != WENC_DTYPE_BF16)
    return bad(WENC_ERR_INVALID_ARG, "quantize_rows: x_dtype %lld unknown", x_dtype);
  if (rows < 1) return bad(WENC_ERR_INVALID_ARG, "rows must be >= 1");
  if (d < 16 || d % 16 != 0) return bad(WENC_ERR_UNSUPPORTED, "d %lld: must be a positive multiple of 16", d);
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(scale, 4))
    return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned (scale: 4)");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = x_dtype == WENC_DTYPE_F32 ? quantize(static_cast<const float*>(x), xq, scale, rows, d, err, s)
                                                  : quantize(static_cast<const __nv_bfloat16*>(x), xq, scale, rows, d, err, s);
  if (e != cudaSuccess) return launch_failed("quantize_rows launch", e);
  return WENC_OK;
}

extern "C" size_t wenc_linear_i8_workspace(int M, int N, int K) {
  wenc_internal_clear_error();
  if (M <= kRowsMost || N < 1 || K < 1 || on_chip(M, N, K, wenc_internal_sm_count())) return 0;
  return up256(size_t(M) * K * 2) + up256(size_t(N) * K * 2);
}

extern "C" wenc_status wenc_linear_i8(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                                      const float* bias, const float* resid, void* out, int M, int N, int K,
                                      int epilogue, void* workspace, size_t workspace_bytes, wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!xq || !x_scale || !wq || !w_scale || !bias || !out)
    return bad(WENC_ERR_INVALID_ARG, "linear_i8: xq/x_scale/wq/w_scale/bias/out is NULL");
  if (epilogue < 0 || epilogue > 2) return bad(WENC_ERR_INVALID_ARG, "epilogue %lld unknown", epilogue);
  if (epilogue == WENC_EPI_BIAS_RESID_F32 && !resid) return bad(WENC_ERR_INVALID_ARG, "resid is NULL");
  if (M < 1) return bad(WENC_ERR_INVALID_ARG, "M must be >= 1");
  if (M > (1 << 28)) return bad(WENC_ERR_UNSUPPORTED, "M %lld: at most 2^28", M);
  if (N < 128 || N % 128 != 0) return bad(WENC_ERR_UNSUPPORTED, "N %lld: must be a positive multiple of 128", N);
  if (K < 64 || K % 64 != 0) return bad(WENC_ERR_UNSUPPORTED, "K %lld: must be a positive multiple of 64", K);
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(bias, 16) || !aligned(w_scale, 16) || !aligned(out, 16) ||
      !aligned(resid, 16) || !aligned(x_scale, 4))
    return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned (x_scale: 4)");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (M <= kRowsMost || on_chip(M, N, K, sms)) {
    e = M <= 8           ? launch_rows<1>(epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, err, s)
        : M <= kRowsMost ? launch_rows<2>(epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, err, s)
                         : launch_tc(epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, err, s);
    if (e != cudaSuccess) return launch_failed("linear_i8 launch", e);
    return WENC_OK;
  }
  const int bn = wenc_host::gemm_pick_bn(N);
  const size_t na = size_t(M) * K, nw = size_t(N) * K, a_bytes = up256(na * 2), need = a_bytes + up256(nw * 2);
  if (!workspace || workspace_bytes < need)
    return bad(WENC_ERR_INVALID_ARG, "linear_i8: workspace of %lld bytes needed, %lld given", static_cast<long long>(need),
               workspace ? static_cast<long long>(workspace_bytes) : 0ll);
  if (!aligned(workspace, 256)) return bad(WENC_ERR_INVALID_ARG, "linear_i8: the workspace must be 256-byte aligned");
  uint16_t* ab = static_cast<uint16_t*>(workspace);
  uint16_t* wb = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + a_bytes);
  std::string why;
  CUtensorMap ta, tw, tw_h;
  if (!wenc_host::make_tmap_2d_bf16(&ta, ab, K, M, size_t(K) * 2, 64, wenc_host::kGemmBM, &why) ||
      !wenc_host::make_tmap_2d_bf16(&tw, wb, K, N, size_t(K) * 2, 64, bn, &why) ||
      !wenc_host::make_tmap_2d_bf16(&tw_h, wb, K, N, size_t(K) * 2, 64, bn / 2, &why))
    return wenc_internal_fail(WENC_ERR_INVALID_ARG, why.c_str());
  size_t blocks = ((na + nw) / 16 + 255) / 256;
  if (blocks > size_t(16) * sms) blocks = size_t(16) * sms;
  e = wenc_host::launch_pdl(widen_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, xq, ab, na, wq, wb, nw);
  if (e != cudaSuccess) return launch_failed("linear_i8 widening", e);
  wenc_host::GemmExtra ex;
  ex.colsum = w_scale;
  ex.row_scale = x_scale;
  e = wenc_host::launch_gemm(ta, tw, M, N, K, bn, wenc_host::kEpiScaled + epilogue, bias, resid, out, err, sms, s, false, 0, ex,
                             &tw_h);
  if (e != cudaSuccess) return launch_failed("linear_i8 launch", e);
  return WENC_OK;
}
