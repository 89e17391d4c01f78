// append.cu -- new keys and values into a paged cache, with the position rotation on the way.
//
// The decoder's self-attention keeps the keys and values of the tokens it has seen
// (inferencelayer 0.2.4 src/whisper_gpu.rs, DEC_WRITE; oxinfer 0.0.5 src/whisper/model.rs,
// LayerCache). Here the cache is a pool of pages of page_size tokens, [n_pages][page_size][Hkv][64],
// and a table that names the pages of each sequence, so that beams and requests of any length share
// one allocation. Token t of the call belongs to the sequence s with
// seq_start[s] <= t < seq_start[s+1] and goes to cache position
//   pos = lens[s] - (seq_start[s+1] - t)          (lens counts the call's tokens)
// that is slot pos % page_size of page table[s][pos / page_size]. Rows behind the last sequence's
// (the padding of a captured graph) are left alone.
//
// Rotation: pairs (x_a, x_b) of the first rot_dim elements of every query and key head turn by the
// angle P * inv_freq[i], P the token's position, to (x_a cos - x_b sin, x_b cos + x_a sin), with
// (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved. Products are fp32, with one
// rounding to the stored type. The angle is formed in turns as a 64-bit fraction: inv_freq / 2 pi is
// held to 2^-64 turns and multiplied by the integer position modulo 2^64, which is exact, so the
// angle of position 2^31 is as good as that of position 1, with one integer product a token instead
// of double-precision trigonometry (GB300 runs two double FMAs a clock and SM).
//
// What bounds it: bytes. Each row of 64 elements is read once and written once, 16 bytes a lane.
// A warp owns whole tokens (or a share of one token's rows, when there are few tokens): its 32
// lanes form the 32 angles at once, and every lane then keeps the angles of its own 16-byte piece
// in registers for all of the token's heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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

constexpr int HD = 64;
constexpr int kWarps = 8;    // per block
constexpr int kUnroll = 8;   // 16-byte loads a lane keeps in flight

struct AppendParams {
  const uint8_t *q, *k, *v;             // rows of 64 elements, heads contiguous
  uint8_t *q_out, *k_pages, *v_pages;
  long long q_stride, q_out_stride, k_stride, v_stride;  // bytes between tokens
  long long k_page_stride, v_page_stride;                // bytes between pages
  const int32_t *table, *lens, *seq_start, *positions;
  const float* inv_freq;
  long long table_stride;
  int n_tokens, n_seqs, per_seq, H, Hkv, n_pages, page_size, max_pages, half, interleaved;
};

// 2^64 * frac(f / 2 pi): the turns a position advances the angle by, as a 64-bit fraction.
// 1 / 2 pi = c1 + c2 with c1 of 29 bits, so f * c1 is exact in double.
__device__ __forceinline__ unsigned long long turns64(float f) {
  const double c1 = 0x1.45f306dp-3, c2 = 0x1.9391054a7f09dp-32;
  double hi = static_cast<double>(f) * c1, lo = static_cast<double>(f) * c2;
  hi -= floor(hi);
  // hi in [0, 1): in two 32-bit parts (a conversion of hi * 2^64 could reach 2^64)
  const double h32 = hi * 4294967296.0;
  const unsigned long long top = static_cast<unsigned long long>(h32);
  const unsigned long long low = static_cast<unsigned long long>((h32 - static_cast<double>(top)) * 4294967296.0);
  lo -= floor(lo);
  const double l32 = lo * 4294967296.0;
  const unsigned long long ltop = static_cast<unsigned long long>(l32);
  const unsigned long long llow = static_cast<unsigned long long>((l32 - static_cast<double>(ltop)) * 4294967296.0);
  return (top << 32) + low + (ltop << 32) + llow;
}

// The last sequence s with seq_start[s] <= t among 0 .. n-1 (-1: none), by all lanes of a warp: 32
// probes a step.
__device__ __forceinline__ int find_seq(const int32_t* start, int n, int t, int lane) {
  int lo = 0, len = n;  // the answer + 1 lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < len && start[at] <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, le));
    if (hits == 0) return lo - 1;
    const int base = (hits - 1) * step;  // start[lo + base] <= t, and the next probe is not
    const int rest = min(step, len - base) - 1;
    lo += base + 1;
    len = rest;
  }
  return lo - 1;
}

// One 16-byte piece of a row: E elements as fp32.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// wpt warps share a token's rows (1, 2, 4 or 8); a group of wpt warps takes `chunk` tokens in a row.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const AppendParams p, int wpt, int chunk,
                                                                uint32_t* err) {
  using P = Piece<T>;
  constexpr int E = P::E;
  constexpr int LPR = HD / E;        // lanes per row: 8 (bf16) or 16 (fp32)
  constexpr int RPW = 32 / LPR;      // rows a warp moves at once
  __shared__ float2 cs_all[kWarps][HD / 2];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = lane % LPR, sub = lane / LPR;
  const int per_block = kWarps / wpt;
  const int share = warp % wpt;  // which of the token's row sets
  const long long group = static_cast<long long>(blockIdx.x) * per_block + warp / wpt;
  const long long t0 = group * chunk;
  if (t0 >= p.n_tokens) return;
  const int t1 = static_cast<int>(min(t0 + chunk, static_cast<long long>(p.n_tokens)));
  float2* cs = cs_all[warp];

  const bool rotate = p.half > 0;
  const unsigned long long step = rotate && lane < p.half ? turns64(p.inv_freq[lane]) : 0ull;
  // this lane's piece: its first element, and which angles and partner it turns with
  const int e0 = piece * E;
  const bool turned = rotate && e0 < 2 * p.half;
  const bool upper = e0 >= p.half;                 // half-split: the b of its pairs
  const int partner = p.half / E;                  // half-split: pieces between a and b
  const int n_q = p.q ? p.H : 0;
  const int rows = n_q + 2 * p.Hkv;

  int s = -1, begin = 0, end = 0;
  for (int t = static_cast<int>(t0); t < t1; ++t) {
    // ---- its first rows (queries, keys, values) are on their way while its place and angles are found
    uint4 x[kUnroll];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * wpt * RPW + sub;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= rows) continue;
        const uint8_t* src = r < n_q ? p.q + t * p.q_stride + r * static_cast<int>(HD * sizeof(T))
                             : r < n_q + p.Hkv
                                 ? p.k + t * p.k_stride + (r - n_q) * static_cast<int>(HD * sizeof(T))
                                 : p.v + t * p.v_stride + (r - n_q - p.Hkv) * static_cast<int>(HD * sizeof(T));
        x[u] = *reinterpret_cast<const uint4*>(src + piece * 16);
      }
    };
    fetch(share * RPW);
    // ---- the token's sequence, cache position and page
    if (p.seq_start) {
      if (t >= end) {
        s = find_seq(p.seq_start, p.n_seqs + 1, t, lane);
        if (s >= p.n_seqs) return;  // behind the last sequence: padding rows, as are all that follow
        begin = s < 0 ? 0 : p.seq_start[s];
        end = s < 0 ? 0 : p.seq_start[s + 1];
      }
    } else {
      s = t / p.per_seq;
      begin = s * p.per_seq;
      end = begin + p.per_seq;
    }
    if (s < 0 || t < begin || t >= end) {  // offsets that do not start at 0 or do not ascend
      if (lane == 0) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
      end = 0;
      continue;
    }
    const long long pos_l = static_cast<long long>(p.lens[s]) - (end - t);
    const int pos = static_cast<int>(pos_l);
    const int page_i = pos / p.page_size;
    if (pos_l < 0 || page_i >= p.max_pages) {
      if (lane == 0) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
      continue;
    }
    const int page = p.table[s * p.table_stride + page_i];
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
      continue;
    }
    const long long slot = static_cast<long long>(pos - page_i * p.page_size) * p.Hkv * (HD * sizeof(T));
    uint8_t* k_dst = p.k_pages + page * p.k_page_stride + slot;
    uint8_t* v_dst = p.v_pages + page * p.v_page_stride + slot;

    // ---- its angles: one per lane, then the E (or E / 2) of this lane's piece
    float c[E], sn[E];
    if (rotate) {
      const int at = p.positions ? p.positions[t] : pos;
      if (lane < p.half) {
        const long long turn = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(at)) * step);
        float sv, cv;
        sincospif(static_cast<float>(turn >> 32) * 0x1p-31f, &sv, &cv);  // turn * 2 pi = pi * (turn / 2^63)
        cs[lane] = make_float2(cv, sv);
      }
      __syncwarp();
      if (turned) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float2 a = cs[p.interleaved ? (e0 + i) >> 1 : (upper ? e0 - p.half : e0) + i];
          c[i] = a.x;
          sn[i] = a.y;
        }
      }
      __syncwarp();
    }

    // ---- turned and stored
    for (int r0 = share * RPW; r0 < rows; r0 += wpt * RPW * kUnroll) {
      if (r0 != share * RPW) fetch(r0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * wpt * RPW + sub;
        uint4 y = x[u];
        if (rotate) {
          // every lane of the warp takes part in the exchange; values and rows past the end pass through
          uint4 o = x[u];
          if (!p.interleaved) {
            const int from = upper ? lane - partner : lane + partner;
            o.x = __shfl_sync(0xffffffffu, x[u].x, from & 31);
            o.y = __shfl_sync(0xffffffffu, x[u].y, from & 31);
            o.z = __shfl_sync(0xffffffffu, x[u].z, from & 31);
            o.w = __shfl_sync(0xffffffffu, x[u].w, from & 31);
          }
          if (turned && r < n_q + p.Hkv) {
            float f[E], g[E];
            P::unpack(x[u], f);
            if (p.interleaved) {
#pragma unroll
              for (int i = 0; i < E; i += 2) {
                const float a = f[i], b = f[i + 1];
                f[i] = a * c[i] - b * sn[i];
                f[i + 1] = b * c[i] + a * sn[i];
              }
            } else {
              P::unpack(o, g);
#pragma unroll
              for (int i = 0; i < E; ++i) f[i] = upper ? f[i] * c[i] + g[i] * sn[i] : f[i] * c[i] - g[i] * sn[i];
            }
            y = P::pack(f);
          }
        }
        if (r < rows) {
          uint8_t* dst = r < n_q ? p.q_out + t * p.q_out_stride + r * static_cast<int>(HD * sizeof(T))
                         : r < n_q + p.Hkv ? k_dst + (r - n_q) * static_cast<int>(HD * sizeof(T))
                                           : v_dst + (r - n_q - p.Hkv) * static_cast<int>(HD * sizeof(T));
          *reinterpret_cast<uint4*>(dst + piece * 16) = y;
        }
      }
    }
  }
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

}  // namespace

extern "C" wenc_status wenc_kv_append(const wenc_kv_append_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!a) return bad(WENC_ERR_INVALID_ARG, "kv_append: args is NULL");
  if (!a->k || !a->v || !a->k_pages || !a->v_pages || !a->block_table || !a->lens)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: k, v, the pages, the block table or lens is NULL");
  if ((a->q == nullptr) != (a->q_out == nullptr)) return bad(WENC_ERR_INVALID_ARG, "kv_append: q and q_out come together");
  if (a->dtype != WENC_DTYPE_F32 && a->dtype != WENC_DTYPE_BF16)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: dtype %lld unknown", a->dtype);
  if (a->head_dim != HD) return bad(WENC_ERR_UNSUPPORTED, "head_dim %lld: only 64 is implemented", a->head_dim);
  if (a->n_seqs < 1 || a->n_kv_heads < 1 || a->n_pages < 1 || a->page_size < 1 || a->max_pages < 1 || a->n_tokens < 0)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: sizes must be positive (n_tokens may be 0)");
  if (a->q && a->n_heads < 1) return bad(WENC_ERR_INVALID_ARG, "kv_append: n_heads must be >= 1");
  if (a->n_heads > 4096 || a->n_kv_heads > 4096) return bad(WENC_ERR_UNSUPPORTED, "kv_append: more than 4096 heads");
  if (static_cast<long long>(a->max_pages) * a->page_size > 0x7fffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "kv_append: max_pages %lld x page_size %lld passes 2^31 - 1", a->max_pages, a->page_size);
  if (!a->seq_start && a->n_tokens % a->n_seqs != 0)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: %lld tokens are no multiple of %lld sequences (pass seq_start)", a->n_tokens,
               a->n_seqs);
  const int rot = a->inv_freq ? a->rot_dim : 0;
  if (a->inv_freq && (rot < 16 || rot > HD || rot % 16 != 0))
    return bad(WENC_ERR_UNSUPPORTED, "kv_append: rot_dim %lld: a multiple of 16, 16..64", rot);
  const long long es = a->dtype == WENC_DTYPE_F32 ? 4 : 2, per16 = 16 / es;
  const long long kv_row = static_cast<long long>(a->n_kv_heads) * HD, page_row = kv_row * a->page_size;
  if (a->k_stride < kv_row || a->v_stride < kv_row ||
      (a->q && (a->q_stride < static_cast<long long>(a->n_heads) * HD || a->q_out_stride < static_cast<long long>(a->n_heads) * HD)))
    return bad(WENC_ERR_INVALID_ARG, "kv_append: a token stride is smaller than its heads");
  if (a->k_page_stride < page_row || a->v_page_stride < page_row)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: a page stride is smaller than a page (%lld elements)", page_row);
  if (a->block_table_stride < a->max_pages && a->n_seqs > 1)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: block_table_stride %lld < max_pages %lld", a->block_table_stride, a->max_pages);
  const void* ptrs[] = {a->q, a->q_out, a->k, a->v, a->k_pages, a->v_pages};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  const long long strides[] = {a->q ? a->q_stride : 0, a->q ? a->q_out_stride : 0, a->k_stride, a->v_stride,
                               a->k_page_stride, a->v_page_stride};
  for (long long x : strides)
    if (x % per16 != 0) return bad(WENC_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
  if (a->n_tokens == 0) return WENC_OK;
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;

  AppendParams p;
  p.q = static_cast<const uint8_t*>(a->q);
  p.k = static_cast<const uint8_t*>(a->k);
  p.v = static_cast<const uint8_t*>(a->v);
  p.q_out = static_cast<uint8_t*>(a->q_out);
  p.k_pages = static_cast<uint8_t*>(a->k_pages);
  p.v_pages = static_cast<uint8_t*>(a->v_pages);
  p.q_stride = a->q_stride * es;
  p.q_out_stride = a->q_out_stride * es;
  p.k_stride = a->k_stride * es;
  p.v_stride = a->v_stride * es;
  p.k_page_stride = a->k_page_stride * es;
  p.v_page_stride = a->v_page_stride * es;
  p.table = a->block_table;
  p.table_stride = a->block_table_stride;
  p.lens = a->lens;
  p.seq_start = a->seq_start;
  p.positions = a->positions;
  p.inv_freq = a->inv_freq;
  p.n_tokens = a->n_tokens;
  p.n_seqs = a->n_seqs;
  p.per_seq = a->seq_start ? 1 : a->n_tokens / a->n_seqs;
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.n_pages = a->n_pages;
  p.page_size = a->page_size;
  p.max_pages = a->max_pages;
  p.half = rot / 2;
  p.interleaved = a->interleaved;
  // queries that neither turn nor move need no pass
  if (p.half == 0 && p.q == p.q_out) p.q = nullptr;

  const int rpw = a->dtype == WENC_DTYPE_F32 ? 2 : 4;
  const int rows = (p.q ? p.H : 0) + 2 * p.Hkv;
  // Few tokens: several warps share one token's rows, so that the rows' loads go out together.
  // Many: a warp takes a run of tokens and finds its sequence and angle steps once.
  int wpt = 1;
  while (wpt < kWarps && wpt * rpw < rows && static_cast<long long>(a->n_tokens) * wpt < 16ll * sms) wpt *= 2;
  const long long warps = static_cast<long long>(a->n_tokens) * wpt;
  int chunk = static_cast<int>((warps + 64ll * sms - 1) / (64ll * sms));
  if (chunk > 8) chunk = 8;
  if (wpt > 1) chunk = 1;
  const long long groups = (a->n_tokens + chunk - 1) / chunk;
  const long long blocks = (groups + kWarps / wpt - 1) / (kWarps / wpt);
  auto kern = a->dtype == WENC_DTYPE_F32 ? kv_append_kernel<float> : kv_append_kernel<__nv_bfloat16>;
  const cudaError_t e = wenc_host::launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0,
                                              reinterpret_cast<cudaStream_t>(stream), p, wpt, chunk, err);
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "kv_append launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}
