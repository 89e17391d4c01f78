// i8.cu -- the matrix product in 8-bit integers with a scale for each token and each channel, and
// the rows of integers it takes.
//
//   scale_m = max_k |x_mk| (1 / 127),  xq_mk = round(x_mk / scale_m)                       (quantize)
//   out_mn = epilogue((sum_k xq_mk wq_nk) scale_m wscale_n + bias_n)                   (product)
// (oxinfer 0.0.5 src/whisper/model.rs, make_lin Q8: 8-bit weights; here one scale spans a whole row,
// so that it leaves the sum).
//
// sm_103a has no integer form of the fifth-generation MMA, and GB300's older integer units are far
// slower than its bf16 ones. Integers up to 127 are exact in bf16 (8 significant bits), a product
// (at most 2^14) is exact in the fp32 accumulator, and so is every sum below 2^24; longer sums round
// as any fp32 sum does. So the product runs on the bf16 tensor cores.
// The operands are widened to bf16 in the workspace and multiplied by the GEMM of gemm.cu, whose
// epilogue applies the scales.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdio>
#include <string>

#include "launch.h"
#include "ptx.cuh"
#include "wenc.h"

wenc_status wenc_internal_fail(wenc_status s, const char* msg);
void wenc_internal_clear_error();
uint32_t* wenc_internal_error_word(std::string* why);
bool wenc_internal_is_sm103(std::string* why);
int wenc_internal_sm_count();

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

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (a & 0xff) | (b & 0xff) << 8 | (c & 0xff) << 16 | static_cast<uint32_t>(d) << 24;
}

// The 16 elements [16 c, 16 c + 16) of a row.
__device__ __forceinline__ void load16(const float* x, int c, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(x)[4 * c + i];
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* x, int c, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(x)[2 * c + i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      f[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
}

// One block per row.
template <typename T>
__global__ void __launch_bounds__(128) quantize_rows_kernel(const T* __restrict__ x, int8_t* __restrict__ xq,
                                                            float* __restrict__ scale, int d) {
  __shared__ float part[4];
  __shared__ int bad_part[4];
  pdl_trigger();
  pdl_wait();
  const size_t row = blockIdx.x;
  const T* xr = x + row * d;
  const int n16 = d / 16;
  float amax = 0.0f;
  int finite = 1;
  for (int c = threadIdx.x; c < n16; c += 128) {
    float f[16];
    load16(xr, c, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      amax = fmaxf(amax, fabsf(f[i]));  // fmaxf passes over a NaN: kept apart
      finite &= fabsf(f[i]) < CUDART_INF_F;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  finite = __all_sync(0xffffffffu, finite);
  if ((threadIdx.x & 31) == 0) {
    part[threadIdx.x >> 5] = amax;
    bad_part[threadIdx.x >> 5] = !finite;
  }
  __syncthreads();
  amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const bool bad = bad_part[0] | bad_part[1] | bad_part[2] | bad_part[3];
  const float s = bad ? CUDART_NAN_F : amax * (1.0f / 127.0f);
  if (threadIdx.x == 0) scale[row] = s;
  const bool zero = bad || s == 0.0f;
  // rows of tiny values are scaled up (exactly) first: neither 1 / s nor s / 2 leaves the range then
  const float up = s < 0x1p-100f ? 0x1p64f : 1.0f, su = s * up;
  const float inv = zero ? 0.0f : __frcp_rn(su), half = 0.5f * su;
  uint4* dst = reinterpret_cast<uint4*>(xq + row * d);
  for (int c = threadIdx.x; c < n16; c += 128) {
    float f[16];
    load16(xr, c, f);
    int q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = zero ? 0 : quantum(f[i] * up, su, inv, half);
    dst[c] = make_uint4(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]), pack4(q[8], q[9], q[10], q[11]),
                        pack4(q[12], q[13], q[14], q[15]));
  }
}

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
  std::string why;
  if (!wenc_internal_is_sm103(&why)) return wenc_internal_fail(WENC_ERR_UNSUPPORTED, why.c_str());
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      x_dtype == WENC_DTYPE_F32
          ? wenc_host::launch_pdl(quantize_rows_kernel<float>, dim3(rows), dim3(128), 0, s, static_cast<const float*>(x),
                                  xq, scale, d)
          : wenc_host::launch_pdl(quantize_rows_kernel<__nv_bfloat16>, dim3(rows), dim3(128), 0, s,
                                  static_cast<const __nv_bfloat16*>(x), xq, scale, d);
  if (e != cudaSuccess) return launch_failed("quantize_rows launch", e);
  return WENC_OK;
}

extern "C" size_t wenc_linear_i8_workspace(int M, int N, int K) {
  wenc_internal_clear_error();
  if (M < 1 || N < 1 || K < 1) return 0;
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
  std::string why;
  if (!wenc_internal_is_sm103(&why)) return wenc_internal_fail(WENC_ERR_UNSUPPORTED, why.c_str());
  uint32_t* err = wenc_internal_error_word(&why);
  if (!err) return wenc_internal_fail(WENC_ERR_CUDA, why.c_str());
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = wenc_internal_sm_count();
  const size_t na = size_t(M) * K, nw = size_t(N) * K;
  uint16_t* ab = static_cast<uint16_t*>(workspace);
  uint16_t* wb = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + up256(na * 2));
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
