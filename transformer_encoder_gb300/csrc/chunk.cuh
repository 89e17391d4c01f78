// chunk.cuh -- what the kernels of wenc_chunk_attention share (chunk_attn.cu, chunk_tc.cu): the call's parameters, a
// sequence's tokens and keys, the keys that a run of its tokens sees, and a row's plain evaluation.
//
// Token i of a sequence that brings m tokens and has len keys stands at position p = len - m + i and sees the keys
//   0 <= j <= p  with  j > p - window  or  j < sinks.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_index.cuh"
#include "mma.cuh"
#include "ptx.cuh"

namespace wenc_dev {

struct ChunkParams {
  const uint8_t* q;
  uint8_t* out;
  long long q_stride, out_stride;  // bytes between tokens
  const uint8_t *k_pages, *v_pages;
  uint32_t k_page16, v_page16, row16;  // between pages, and between a page's slots, in units of 16 bytes
  const int32_t *table, *lens, *seq_start;
  long long table_stride;
  int n_tokens, n_seqs, per_seq, max_new, H, Hkv, r, n_pages, page_size, page_shift, max_pages;
  int window, sinks;          // window 2^30: every key up to the token's own
  float scale_log2;           // >= 0
  uint32_t q_flip, q_keep;    // a negative scale turns the queries' signs (per 32 bits), a zero one clears them
};

// A sequence of the call: its first row, tokens and keys (tokens 0 where the lengths or offsets are out of range, reported).
struct ChunkSeq {
  int row0, m, len;
};

// The tokens of rows [start, end) of the call; 0, reported, where they are out of range or more than the call allows.
__device__ __forceinline__ int chunk_tokens(const ChunkParams& p, int start, int end, uint32_t* err) {
  if (start >= 0 && end >= start && end <= p.n_tokens && end - start <= p.max_new) return end - start;
  *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
  return 0;
}

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int s, uint32_t* err) {
  ChunkSeq q{s * p.per_seq, p.per_seq, 0};
  if (p.seq_start) {
    q.row0 = p.seq_start[s];
    q.m = chunk_tokens(p, q.row0, p.seq_start[s + 1], err);
  }
  if (q.m > 0) {
    q.len = p.lens[s];
    if (q.len < 0 || q.len > static_cast<long long>(p.max_pages) * p.page_size) {
      *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
      q.m = q.len = 0;
    }
  }
  return q;
}

// A key's place: its 16-byte unit within K's pages and V's, or false where the page is out of range (reported).
__device__ __forceinline__ bool chunk_slot(const ChunkParams& p, int seq, int key, int hk, uint32_t row_units, uint64_t& k16,
                                           uint64_t& v16, uint32_t* err) {
  const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
  if (!in_bounds(seq >= 0 && seq < p.n_seqs && pi >= 0 && pi < p.max_pages && hk < p.Hkv, err, 116)) return false;
  const int page = p.table[seq * p.table_stride + pi];
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages)) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
    return false;
  }
  const uint32_t at = static_cast<uint32_t>(key - pi * p.page_size) * p.row16 + hk * row_units;
  k16 = static_cast<uint64_t>(page) * p.k_page16 + at;
  v16 = static_cast<uint64_t>(page) * p.v_page16 + at;
  return true;
}

// The products with V are formed for all of a tile's rows, with weights of 0 where a row does not see a key, and in parts; but
// 0 x inf and 0 x NaN are NaN, so a value that is no number would reach rows that do not see it, and weighted sums of values
// near the largest float may leave the range. Elements of a row's O that are no numbers, and all of a row whose sum is none or
// 0 (rare: they are found by that), are formed again here, in plain fp32 from the keys alone that the row sees, with weights of
// at most 1. That goes through all keys twice, so nothing whose waits have a limit may wait for it. Eight lanes hold a row:
// token position pos, elements c8 .. c8 + 7 in v and sum l; all lanes of a warp call, in: the lane's row is one of the call's.
// lo, hi, first: keys [lo, hi) and [0, first) hold all that the warp's rows see.
template <typename T>
__device__ __noinline__ void chunk_redo(const ChunkParams& p, int seq, int hk, const uint8_t* q_row, int pos, bool in, int lo, int hi,
                                        int first, int c8, float* v, float* l_io, uint32_t* err) {
  constexpr uint32_t units = 64 * sizeof(T) / 16;
  float q[8] = {};
  if (in) load8(reinterpret_cast<const T*>(q_row) + c8, q);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (p.q_keep == 0u) q[e] = 0.0f;
    else if (p.q_flip != 0u) q[e] = -q[e];
  auto each_key = [&](auto&& f) {
#pragma unroll 1
    for (int key = first > 0 ? 0 : lo; key < hi; ++key) {
      if (key >= first && key < lo) key = lo;
      uint64_t k16, v16;
      if (!chunk_slot(p, seq, key, hk, units, k16, v16, err)) continue;
      const bool sees = in && key <= pos && (key > pos - p.window || key < p.sinks);
      float kf[8], dot = 0.0f;
      load8(reinterpret_cast<const T*>(p.k_pages + (k16 << 4)) + c8, kf);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(q[e], kf[e], dot);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      f(reinterpret_cast<const T*>(p.v_pages + (v16 << 4)) + c8, sees, dot * p.scale_log2);
    }
  };
  float m = -CUDART_INF_F, l = 0.0f, o[8] = {};
  each_key([&](const T*, bool sees, float s) {
    if (sees) m = s != s ? s : fmaxf(m, s);
  });
  const float u = m == -CUDART_INF_F ? 0.0f : m;
  each_key([&](const T* row, bool sees, float s) {
    if (!sees) return;
    const float w = ex2_approx(s - u);
    l += w;
    float vf[8];
    load8(row, vf);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(w, vf[e], o[e]);
  });
  // (the lane's other elements turn to the sum of these weights, so that none leaves the range on its way to the division; a row
  // without weights, which a value that it does not see may have turned to NaN, is all formed here: zeros)
  bool bad[8], any = false;
  const bool again = !(fabsf(*l_io) < CUDART_INF_F) || *l_io == 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) any |= bad[e] = again || !(fabsf(v[e]) < CUDART_INF_F);
  if (!in || !any) return;
  const float f = l / *l_io;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = bad[e] ? o[e] : v[e] * f;
  // (scores of -inf alone leave no weights either, but exp(s - max s) of them is no number; from position 0 on a token sees a key)
  *l_io = l == 0.0f && pos >= 0 ? CUDART_NAN_F : l;
}

// Whether a row needs no second evaluation: its sum and values are all numbers, and it has weights where it sees a key.
__device__ __forceinline__ bool chunk_numbers(const float (&v)[8], float l, int pos) {
  if (l == 0.0f && pos >= 0) return false;
  float zero = l * 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) zero = fmaf(v[e], 0.0f, zero);
  return zero == 0.0f;
}

// Eight elements of an output row, normalised (a row without a visible key: zeros).
template <typename T>
__device__ __forceinline__ void chunk_write8(const ChunkParams& p, int token, int head, int c8, const float (&v)[8], float l,
                                             uint32_t* err) {
  if (!in_bounds(token >= 0 && token < p.n_tokens && head >= 0 && head < p.H, err, 117)) return;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  uint8_t* dst = p.out + static_cast<long long>(token) * p.out_stride + (head * 64 + c8) * static_cast<int>(sizeof(T));
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
  }
}

}  // namespace wenc_dev

namespace wenc_host {

// A unit of chunk_tc.cu that was cut: where it belongs and its pieces (0: no unit was cut here).
struct ChunkCut {
  int seq, hk, x, pieces;
};
// A CTA's run of steps: where it begins and how many it holds (as chunk_tc.cu's Walk has them), and whether rows of units that are
// whole within it have to be formed again (they carry kChunkMark).
struct ChunkRun {
  int redo;
  int hk, seq, x, skip, m, len, row0;
  long long left, at;
};
// In an output row's first elements: two bf16 numbers that no rounding gives (a NaN comes out as 0x7fff).
constexpr uint32_t kChunkMark = 0xffffffffu;
struct ChunkTcArgs {
  int few;             // rows per key head up to which a sequence is chunk_attn.cu's
  int tokens;          // of a row tile: 128 / r
  int per_unit;        // of a unit: two tiles'
  ChunkCut* cuts;      // [CTAs]
  ChunkRun* runs;      // [CTAs]
  float* part_o;       // [CTAs][2][256][64]
  float2* part_ml;     // [CTAs][2][256]: (maximum in log2 units, sum)
};
size_t chunk_tc_workspace(int sms);
// The sequences with more than `few` rows per key head (bf16, scale > 0, at most 128 query heads per key head). Two launches.
cudaError_t launch_chunk_tc(const wenc_dev::ChunkParams& p, int few, void* workspace, uint32_t* err, int sms, cudaStream_t stream);

}  // namespace wenc_host
