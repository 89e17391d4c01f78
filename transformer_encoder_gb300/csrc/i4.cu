// i4.cu -- the matrix product with 4-bit weights that have a scale for each group of inputs.
//
//   out_mn = epilogue(sum_g scale_ng sum_{k in g} (u_nk - 8) x_mk + bias_n),   groups of 32, 64 or 128
// (oxinfer 0.0.5 src/whisper/model.rs, make_lin: quantised weights; here with groups of inputs).
//
// u - 8 is exact in bf16, a bf16 x times it is exact in fp32, so a group's product runs on the bf16 tensor cores without a
// rounding of either operand, and the scale, which would not fit into the weight exactly, multiplies the group's fp32 sum. float32 x is
// cut into three bf16 parts (8 + 8 + 8 significant bits: exact together), the products of which share a group's sum.
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

// ---------------------------------------------------------------- few tokens
// out^T = W x^T for up to 8 NT tokens: a CTA takes 16 channels (the MMA's M), its warps share K in pieces of 128, and the CTAs
// of a cluster share it further; they are joined through shared memory, in the order of the warps. Weights go from global memory to registers: a
// lane takes the word (8 weights) that its MMA rows need of each 32 inputs, so a group's products stay together for
// every group size, and x comes in the same order of k from L1 or L2.
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

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
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

}  // namespace

extern "C" size_t wenc_linear_i4_workspace(int M, int N, int K, int x_dtype, int group) {
  wenc_internal_clear_error();
  return 0;
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
  cudaError_t e;
  if (M <= 8) e = f32 ? launch_rows<float, 1>(p, sms, err, s) : launch_rows<__nv_bfloat16, 1>(p, sms, err, s);
  else if (M <= 16) e = f32 ? launch_rows<float, 2>(p, sms, err, s) : launch_rows<__nv_bfloat16, 2>(p, sms, err, s);
  else e = f32 ? launch_rows<float, 4>(p, sms, err, s) : launch_rows<__nv_bfloat16, 4>(p, sms, err, s);
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "linear_i4 launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}
