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
// round as any fp32 sum does. So the product runs on 16-bit tensor cores, in two forms:
//  - many tokens: both operands are widened to bf16 in the workspace and multiplied by the tcgen05 GEMM
//    of gemm.cu, whose epilogue applies the scales. What bounds it: the tensor pipe, plus the
//    widening's bytes;
//  - few tokens (a decode step): the weights are what there is to read, once, as bytes; they are widened
//    in registers and multiplied by mma.sync, no workspace (i8_rows_kernel below).
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

// One pass: a row's vectors stay in the registers of its threads (a warp, or the block: WARP) between the
// maximum and the division. What bounds it: bytes (x once, the integers once).
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) quantize_rows_kernel(const T* __restrict__ x, int8_t* __restrict__ xq,
                                                             float* __restrict__ scale, int rows, int nv) {
  using V = Vec<T>;
  __shared__ uint32_t part[32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (row >= rows) return;  // (a whole warp; the block form has a block for each row)
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
cudaError_t launch_quantize(const T* x, int8_t* xq, float* scale, int rows, int nv, int threads, cudaStream_t s) {
  if (threads == 32)  // a warp per row, four rows a block
    return wenc_host::launch_pdl(quantize_rows_kernel<T, VPT, true>, dim3((rows + 3) / 4), dim3(128), 0, s, x, xq, scale, rows, nv);
  return wenc_host::launch_pdl(quantize_rows_kernel<T, VPT, false>, dim3(rows), dim3(threads), 0, s, x, xq, scale, rows, nv);
}

// Threads per row: a warp up to 64 vectors (two a lane); else the fewest, from 128, that keep a row within
// eight vectors a thread.
template <typename T>
cudaError_t quantize(const T* x, int8_t* xq, float* scale, int rows, int d, cudaStream_t s) {
  const int nv = d / Vec<T>::E;
  if (nv > 8 * 1024)
    return wenc_host::launch_pdl(quantize_long_rows_kernel<T>, dim3(rows), dim3(1024), 0, s, x, xq, scale, nv);
  int threads = 32;
  if (nv > 64) {
    threads = 128;
    while (threads * 8 < nv) threads *= 2;
  }
  const int vpt = (nv + threads - 1) / threads;
  if (vpt <= 2) return launch_quantize<T, 2>(x, xq, scale, rows, nv, threads, s);
  if (vpt <= 4) return launch_quantize<T, 4>(x, xq, scale, rows, nv, threads, s);
  if (vpt <= 6) return launch_quantize<T, 6>(x, xq, scale, rows, nv, threads, s);
  return launch_quantize<T, 8>(x, xq, scale, rows, nv, threads, s);
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
__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_rank_f32(uint32_t saddr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// out^T = W x^T for up to 8 NT tokens: a CTA takes 32 channels and a share of K (the CTAs of a cluster split
// K between them and join through distributed shared memory). Its eight warps are two groups of 16 channels
// (the MMA's M) times four quarters of a round: per round of 256 k, warp (c, q) multiplies channels 16 c .. + 15
// by the 64 k of quarter q. The order of k within those 64 is free as long as both operands agree: a lane
// takes 16 consecutive bytes of a weight row, which are four MMAs' worth of its fragments, so weights go from
// global memory to registers in full 64-byte pieces and are widened there; the tokens are widened once
// per CTA and round into shared memory, in the same order, rows 16 bytes past a multiple of 128 apart so
// that the fragment loads touch all banks. Weights and tokens of the next round are on their way meanwhile.
// What bounds it: at a decode step's sizes, latency; the weights' bytes beyond.
constexpr int kRowsChannels = 32;
constexpr int kRowsK = 256;  // k per round

template <int NT>
struct RowsCfg {
  static constexpr int TOK = 8 * NT;
  static constexpr int XROW = kRowsK * 2 + 16;            // bytes of a token's round in shared memory
  static constexpr int XV = TOK * (kRowsK / 16) / 256;    // 16-byte pieces of x per thread and round
  static constexpr int XN = XV < 1 ? 1 : XV;
  static constexpr int RED = 8 * 16 * (TOK + 1) * 4;      // the warps' sums
  static constexpr int SMEM = TOK * XROW > RED ? TOK * XROW : RED;
};

template <int NT, int EPI>
__global__ void __launch_bounds__(256) i8_rows_kernel(const int8_t* __restrict__ xq, const float* __restrict__ x_scale,
                                                      const int8_t* __restrict__ wq, const float* __restrict__ w_scale,
                                                      const float* __restrict__ bias, const float* resid, void* out, int M,
                                                      int N, int K, int ksplit) {
  using C = RowsCfg<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int c16 = warp & 1, quarter = warp >> 1;
  const int rank = blockIdx.x % ksplit;
  const int n0 = blockIdx.x / ksplit * kRowsChannels, m0 = blockIdx.y * C::TOK;
  const int m_here = min(C::TOK, M - m0);
  // this CTA's k: whole pieces of 64, as equal as they divide
  const int pieces = K / 64, per = (pieces + ksplit - 1) / ksplit;
  const int k_begin = min(rank * per, pieces) * 64, k_end = min((rank + 1) * per, pieces) * 64;

  const int8_t* wa = wq + static_cast<size_t>(n0 + 16 * c16 + g) * K + 16 * tq;
  const int8_t* wb = wa + static_cast<size_t>(8) * K;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 w0 = zero, w1 = zero, xv[C::XN];
  auto fetch = [&](int k0) {  // the round that starts at k0, as far as it lies before k_end
    const int k = k0 + 64 * quarter;
    w0 = k < k_end ? __ldg(reinterpret_cast<const uint4*>(wa + k)) : zero;
    w1 = k < k_end ? __ldg(reinterpret_cast<const uint4*>(wb + k)) : zero;
#pragma unroll
    for (int i = 0; i < C::XN; ++i) {
      const int at = threadIdx.x + 256 * i, tok = at / (kRowsK / 16), kk = k0 + at % (kRowsK / 16) * 16;
      xv[i] = tok < m_here && kk < k_end ? *reinterpret_cast<const uint4*>(xq + static_cast<size_t>(m0 + tok) * K + kk) : zero;
    }
  };
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
  fetch(k_begin);
  for (int k0 = k_begin; k0 < k_end; k0 += kRowsK) {
    // tokens of this round into shared memory as fp16, each 16-byte piece as 32 bytes
#pragma unroll
    for (int i = 0; i < C::XN; ++i) {
      const int at = threadIdx.x + 256 * i, tok = at / (kRowsK / 16), piece = at % (kRowsK / 16);
      if (tok < C::TOK) {
        uint4 a, b;
        widen_half(xv[i].x, a.x, a.y);
        widen_half(xv[i].y, a.z, a.w);
        widen_half(xv[i].z, b.x, b.y);
        widen_half(xv[i].w, b.z, b.w);
        uint4* dst = reinterpret_cast<uint4*>(smem + tok * C::XROW + piece * 32);
        dst[0] = a;
        dst[1] = b;
      }
    }
    uint32_t wf[4][4];  // the fragments of four MMAs
    widen_half(w0.x, wf[0][0], wf[0][2]);
    widen_half(w1.x, wf[0][1], wf[0][3]);
    widen_half(w0.y, wf[1][0], wf[1][2]);
    widen_half(w1.y, wf[1][1], wf[1][3]);
    widen_half(w0.z, wf[2][0], wf[2][2]);
    widen_half(w1.z, wf[2][1], wf[2][3]);
    widen_half(w0.w, wf[3][0], wf[3][2]);
    widen_half(w1.w, wf[3][1], wf[3][3]);
    __syncthreads();
    if (k0 + kRowsK < k_end) fetch(k0 + kRowsK);
    const uint8_t* xs = smem + g * C::XROW + quarter * 128 + tq * 32;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= m_here) break;
      const uint4 b0 = *reinterpret_cast<const uint4*>(xs + n * 8 * C::XROW);
      const uint4 b1 = *reinterpret_cast<const uint4*>(xs + n * 8 * C::XROW + 16);
      mma_f16(acc[n], wf[0], b0.x, b0.y);
      mma_f16(acc[n], wf[1], b0.z, b0.w);
      mma_f16(acc[n], wf[2], b1.x, b1.y);
      mma_f16(acc[n], wf[3], b1.z, b1.w);
    }
    __syncthreads();  // the next round overwrites the tokens
  }
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
      if (tok < m_here) red[((ch >> 4) * 16 + (ch & 15)) * RS + tok] = sum4(ch, tok);
    }
    cluster_arrive_wait();
  }
  const uint32_t red_addr = smem_u32(red);
  const int ch = lane, n = n0 + ch;
  const float ws = __ldg(w_scale + n), bn = __ldg(bias + n);
  for (int tok = warp * ksplit + rank; tok < m_here; tok += 8 * ksplit) {
    float a = 0.0f;
    if (ksplit > 1) {
      for (int r = 0; r < ksplit; ++r) a += ld_rank_f32(red_addr + (((ch >> 4) * 16 + (ch & 15)) * RS + tok) * 4, r);
    } else {
      a = sum4(ch, tok);
    }
    const int m = m0 + tok;
    float v = fmaf(a, __ldg(x_scale + m) * ws, bn), unused = 0.0f;
    const size_t at = static_cast<size_t>(m) * N + n;
    if constexpr (EPI == WENC_EPI_BIAS_RESID_F32) {
      static_cast<float*>(out)[at] = resid[at] + v;
    } else {
      if constexpr (EPI == WENC_EPI_BIAS_GELU_BF16) gelu_erf_x2(v, unused);
      static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    }
  }
  if (ksplit > 1) cluster_arrive_wait();  // no CTA leaves while another reads its sums
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

// int8 -> bf16, 16 a thread: both operands in one launch.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* __restrict__ a, uint16_t* __restrict__ ab, size_t na,
                                                    const int8_t* __restrict__ w, uint16_t* __restrict__ wb, size_t nw) {
  pdl_trigger();
  pdl_wait();
  const size_t total = (na + nw) / 16;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const bool is_a = i < na / 16;
    const size_t j = is_a ? i : i - na / 16;
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

// The few-token form up to this many tokens (in tiles of at most 128).
constexpr int kRowsMost = 128;

template <int NT, int EPI>
cudaError_t launch_rows(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale, const float* bias,
                        const float* resid, void* out, int M, int N, int K, int sms, cudaStream_t stream) {
  using C = RowsCfg<NT>;
  auto kern = i8_rows_kernel<NT, EPI>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // Shared-memory opt-in, once per device and instantiation (a repeat by a racing host thread is harmless).
  static std::atomic<int> configured_device{-1};
  if (C::SMEM > 48 * 1024 && configured_device.load(std::memory_order_acquire) != dev) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    configured_device.store(dev, std::memory_order_release);
  }
  // clusters along K until the machine has a CTA per SM, none with less than one round
  const int tiles = N / kRowsChannels, m_tiles = (M + C::TOK - 1) / C::TOK;
  int ksplit = 1;
  while (ksplit < 8 && static_cast<long long>(tiles) * m_tiles * ksplit * 2 <= 2ll * sms && K >= 2 * ksplit * kRowsK) ksplit *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * ksplit, m_tiles);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ksplit;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ksplit > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, ksplit);
}

template <int NT>
cudaError_t launch_rows_epi(int epilogue, const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                            const float* bias, const float* resid, void* out, int M, int N, int K, int sms, cudaStream_t s) {
  if (epilogue == WENC_EPI_BIAS_BF16) return launch_rows<NT, WENC_EPI_BIAS_BF16>(xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, s);
  if (epilogue == WENC_EPI_BIAS_GELU_BF16)
    return launch_rows<NT, WENC_EPI_BIAS_GELU_BF16>(xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, s);
  return launch_rows<NT, WENC_EPI_BIAS_RESID_F32>(xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, s);
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
  const cudaError_t e = x_dtype == WENC_DTYPE_F32 ? quantize(static_cast<const float*>(x), xq, scale, rows, d, s)
                                                  : quantize(static_cast<const __nv_bfloat16*>(x), xq, scale, rows, d, s);
  if (e != cudaSuccess) return launch_failed("quantize_rows launch", e);
  return WENC_OK;
}

extern "C" size_t wenc_linear_i8_workspace(int M, int N, int K) {
  wenc_internal_clear_error();
  if (M <= kRowsMost || N < 1 || K < 1) return 0;
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
  const int bn = wenc_host::gemm_pick_bn(N);
  if (N < 1 || bn == 0) return bad(WENC_ERR_UNSUPPORTED, "N %lld: must be a multiple of 128", N);
  if (K < 64 || K % 64 != 0) return bad(WENC_ERR_UNSUPPORTED, "K %lld: must be a positive multiple of 64", K);
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(bias, 16) || !aligned(w_scale, 16) || !aligned(out, 16) ||
      !aligned(resid, 16) || !aligned(x_scale, 4))
    return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned (x_scale: 4)");
  const size_t need = wenc_linear_i8_workspace(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return bad(WENC_ERR_INVALID_ARG, "linear_i8: workspace of %lld bytes needed, %lld given", static_cast<long long>(need),
               workspace ? static_cast<long long>(workspace_bytes) : 0ll);
  if (need > 0 && !aligned(workspace, 256))
    return bad(WENC_ERR_INVALID_ARG, "linear_i8: the workspace must be 256-byte aligned");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M <= kRowsMost) {
    auto rows = M <= 8 ? launch_rows_epi<1> : M <= 16 ? launch_rows_epi<2> : M <= 32 ? launch_rows_epi<4> : M <= 64 ? launch_rows_epi<8> : launch_rows_epi<16>;
    const cudaError_t e = rows(epilogue, xq, x_scale, wq, w_scale, bias, resid, out, M, N, K, sms, s);
    if (e != cudaSuccess) return launch_failed("linear_i8 launch", e);
    return WENC_OK;
  }
  const size_t na = size_t(M) * K, nw = size_t(N) * K;
  uint16_t* ab = static_cast<uint16_t*>(workspace);
  uint16_t* wb = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + up256(na * 2));
  std::string why;
  CUtensorMap ta, tw, tw_h;
  const bool ok = wenc_host::make_tmap_2d_bf16(&ta, ab, K, M, size_t(K) * 2, 64, wenc_host::kGemmBM, &why) &&
                  wenc_host::make_tmap_2d_bf16(&tw, wb, K, N, size_t(K) * 2, 64, bn, &why) &&
                  wenc_host::make_tmap_2d_bf16(&tw_h, wb, K, N, size_t(K) * 2, 64, bn / 2, &why);
  if (!ok) return wenc_internal_fail(WENC_ERR_INVALID_ARG, why.c_str());
  size_t blocks = ((na + nw) / 16 + 255) / 256;
  if (blocks > size_t(16) * sms) blocks = size_t(16) * sms;
  cudaError_t e = wenc_host::launch_pdl(widen_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, xq, ab, na, wq,
                                        wb, nw);
  if (e != cudaSuccess) return launch_failed("linear_i8 widening", e);
  wenc_host::GemmExtra ex;
  ex.colsum = w_scale;
  ex.row_scale = x_scale;
  e = wenc_host::launch_gemm(ta, tw, M, N, K, bn, wenc_host::kEpiScaled + epilogue, bias, resid, out, err, sms, s, false,
                             0, ex, &tw_h);
  if (e != cudaSuccess) return launch_failed("linear_i8 launch", e);
  return WENC_OK;
}
