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
// A warp owns a run of tokens (or a share of one token's rows, when there are few tokens). What would be
// a chain of dependent loads per token (its sequence, length, page) is done for the whole run at once, a
// lane a token, and so are the run's angles; then the rows stream, and every lane keeps the angles of its
// own 16-byte piece in registers for all of a token's heads.
// Measured (us on the device in a captured graph; bytes at the measured copy rate in brackets): 27465 tokens of 16
// prompts, 20 + 2 x 4 heads, bf16, rotated: 39.1 [29.0], 5.0 TB/s of reads and writes, where a library copy of the
// same 98 MB takes 66 and the call without rotation 38; 1300 tokens of 80 sequences, fp32: 7.9 [2.6]; one token 3.4, of
// which a launch is most. One token at a time with its lookups in a chain, and pairs exchanged by shuffles: 50.5,
// 9.9 and 4.1. Three blocks an SM beat four (43.6: the two pieces of two rows spill) and two (47.7).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <string>

#include "decode_index.cuh"
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
constexpr int kUnroll = 2;   // rows a lane keeps in flight, two 16-byte pieces each
constexpr int kRun = 8;      // tokens of a warp's run, at most

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

// The last sequence s with seq_start[s] <= t among 0 .. n-1 (-1: none), by all lanes of a warp: 32
// probes a step.
__device__ __forceinline__ int find_seq(const int32_t* start, int n, int t, int lane) {
  return last_start(n, [&](int lo, int step, int len) {
    const bool le = lane * step < len && start[lo + lane * step] <= t;
    return __popc(__ballot_sync(0xffffffffu, le));
  });
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
__global__ void __launch_bounds__(32 * kWarps, 3) kv_append_kernel(const AppendParams p, int wpt, int chunk, uint32_t* err) {
  using P = Piece<T>;
  constexpr int E = P::E;
  constexpr int LPR = HD / E / 2;    // lanes per row: 4 (bf16) or 8 (fp32)
  constexpr int RPW = 32 / LPR;      // rows a warp moves at once
  constexpr int ROWB = HD * sizeof(T);
  __shared__ __align__(16) float2 cs_all[kWarps][kRun][HD / 2];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane % LPR, sub = lane / LPR;
  const int share = warp % wpt;  // which of the token's row sets
  const long long t0 = (static_cast<long long>(blockIdx.x) * (kWarps / wpt) + warp / wpt) * chunk;
  if (t0 >= p.n_tokens) return;
  const int first = static_cast<int>(t0), n = static_cast<int>(min(static_cast<long long>(chunk), p.n_tokens - t0));

  // ---- the run's places, a lane a token: sequence, cache position, page
  int pos = 0;
  long long k_at = -1, v_at = 0;  // byte offsets of the token's slot; -1: the token is not written
  {
    const int t = first + lane;
    int s = -1, left = 0;  // the token's sequence, and its rows from the token on
    if (p.seq_start) {
      s = find_seq(p.seq_start, p.n_seqs + 1, first, lane);  // the first token's; the others' at or behind it
      if (lane < n) {
        s = sequence_of(p.seq_start, p.n_seqs, p.n_tokens, t, s, left);
        if (s < 0) {
          *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
          s = p.n_seqs;
        }
      }
    } else {
      s = t / p.per_seq;
      left = (s + 1) * p.per_seq - t;
    }
    if (lane < n && s < p.n_seqs) {  // (s == n_seqs: padding rows behind the last sequence)
      const long long at = in_bounds(s >= 0 && s < p.n_seqs, err, 97) ? static_cast<long long>(p.lens[s]) - left : -1;
      pos = static_cast<int>(at);
      const int page_i = pos / p.page_size;
      if (at < 0 || page_i >= p.max_pages) {
        *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
      } else {
        const int page = p.table[s * p.table_stride + page_i];
        if (page < 0 || page >= p.n_pages) {
          *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
        } else {
          const long long slot = static_cast<long long>(pos - page_i * p.page_size) * p.Hkv * ROWB;
          k_at = page * p.k_page_stride + slot;
          v_at = page * p.v_page_stride + slot;
        }
      }
    }
    if (p.positions && lane < n) pos = p.positions[t];
  }
  // ---- the run's angles, a lane a frequency
  const bool rotate = p.half > 0;
  if (rotate) {
    const unsigned long long step = lane < p.half ? turns64(p.inv_freq[lane]) : 0ull;
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const int at = __shfl_sync(0xffffffffu, pos, i);
      if (lane < p.half) {
        // pi h goes to sincospi, and the rest turns the result: sin(h + l) = sin h + l cos h to l^2 / 2 < 2^-43
        float h, l, sv, cv;
        angle_parts(at, step, h, l);
        sincospif(h, &sv, &cv);
        cs_all[warp][i][lane] = make_float2(fmaf(-l, sv, cv), fmaf(l, cv, sv));
      }
    }
    __syncwarp();
  }

  // ---- the rows: queries, keys, values
  // Half-split: lanes 0 .. half / E - 1 take the pieces j and j + half / E, which turn with each other; the others
  // two neighbours each of those that do not turn. Interleaved: pieces 2 j and 2 j + 1.
  const int half_p = p.half / E;
  const bool pair = rotate && !p.interleaved && j < half_p;
  const bool turned = rotate && (p.interleaved ? 2 * j * E < 2 * p.half : pair);
  const int o0 = (pair ? j : 2 * j) * 16, o1 = (pair ? j + half_p : 2 * j + 1) * 16;  // bytes into the row
  const int n_q = p.q ? p.H : 0;
  const int rows = n_q + 2 * p.Hkv;
  for (int i = 0; i < n; ++i) {
    const long long kd = __shfl_sync(0xffffffffu, k_at, i), vd = __shfl_sync(0xffffffffu, v_at, i);
    if (kd < 0) continue;
    const long long t = first + i;
    if (!in_bounds(t < p.n_tokens && kd + p.Hkv * ROWB <= p.n_pages * p.k_page_stride && vd + p.Hkv * ROWB <= p.n_pages * p.v_page_stride,
                   err, 98))
      continue;
    const uint8_t *q = p.q + t * p.q_stride, *k = p.k + t * p.k_stride, *v = p.v + t * p.v_stride;
    uint8_t *qd = p.q_out + t * p.q_out_stride, *kdst = p.k_pages + kd, *vdst = p.v_pages + vd;
    float c[E], sn[E];
    if (turned) {
#pragma unroll
      for (int e = 0; e < E; ++e) {  // of angle j E + e in both layouts
        const float2 a = cs_all[warp][i][j * E + e];
        c[e] = a.x;
        sn[e] = a.y;
      }
    }
    for (int r0 = share * RPW; r0 < rows; r0 += wpt * RPW * kUnroll) {
      uint4 x[kUnroll][2];
#pragma unroll
      for (int w = 0; w < kUnroll; ++w) {
        const int r = r0 + w * wpt * RPW + sub;
        const uint8_t* src = r < n_q ? q + r * ROWB : r < n_q + p.Hkv ? k + (r - n_q) * ROWB : v + (r - n_q - p.Hkv) * ROWB;
        if (r < rows) {
          x[w][0] = *reinterpret_cast<const uint4*>(src + o0);
          x[w][1] = *reinterpret_cast<const uint4*>(src + o1);
        }
      }
#pragma unroll
      for (int w = 0; w < kUnroll; ++w) {
        const int r = r0 + w * wpt * RPW + sub;
        if (r >= rows) break;
        uint4 y0 = x[w][0], y1 = x[w][1];
        if (turned && r < n_q + p.Hkv) {
          float a[E], b[E];
          P::unpack(y0, a);
          P::unpack(y1, b);
          if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
              a[e] = a0 * c[e / 2] - a1 * sn[e / 2];
              a[e + 1] = a1 * c[e / 2] + a0 * sn[e / 2];
              b[e] = b0 * c[E / 2 + e / 2] - b1 * sn[E / 2 + e / 2];
              b[e + 1] = b1 * c[E / 2 + e / 2] + b0 * sn[E / 2 + e / 2];
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float a0 = a[e], b0 = b[e];
              a[e] = a0 * c[e] - b0 * sn[e];
              b[e] = b0 * c[e] + a0 * sn[e];
            }
          }
          y0 = P::pack(a);
          y1 = P::pack(b);
        }
        uint8_t* dst = r < n_q ? qd + r * ROWB : r < n_q + p.Hkv ? kdst + (r - n_q) * ROWB : vdst + (r - n_q - p.Hkv) * ROWB;
        *reinterpret_cast<uint4*>(dst + o0) = y0;
        *reinterpret_cast<uint4*>(dst + o1) = y1;
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
  // (in place, a warp rewrites the rows it has read; with two strides it would write rows that others have yet to read)
  if (a->q && a->q == a->q_out && a->q_stride != a->q_out_stride && a->n_tokens > 1)
    return bad(WENC_ERR_INVALID_ARG, "kv_append: in place, q_stride %lld and q_out_stride %lld must be the same", a->q_stride,
               a->q_out_stride);
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
  // queries that neither turn nor move need no pass (in place, the strides are one: checked above)
  if (p.half == 0 && p.q == p.q_out) p.q = nullptr;

  const int rpw = a->dtype == WENC_DTYPE_F32 ? 4 : 8;  // rows a warp moves at once
  const int rows = (p.q ? p.H : 0) + 2 * p.Hkv;
  // Few tokens: several warps share one token's rows, so that the rows' loads go out together.
  // Many: a warp takes a run of tokens and finds its sequence and angle steps once.
  int wpt = 1;
  while (wpt < kWarps && wpt * rpw < rows && static_cast<long long>(a->n_tokens) * wpt < 16ll * sms) wpt *= 2;
  const long long warps = static_cast<long long>(a->n_tokens) * wpt;
  int chunk = static_cast<int>((warps + 24ll * sms - 1) / (24ll * sms));
  if (chunk > kRun) chunk = kRun;
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
