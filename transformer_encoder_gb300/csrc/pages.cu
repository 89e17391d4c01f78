// pages.cu -- a step's places in a paged cache, and the pages that it gives back, built on the GPU from lengths.
//
// A server that keeps its requests' lengths in device memory needs, before the kernels of a step (append.cu, chunk_attn.cu)
// run: pages for the new tokens, their entries in the block table, the rows' offsets, positions and slots. With
// b = ceil(len / page) the entries that a sequence holds and need = ceil((len + new) / page) - b those it gets,
//   seq_start = running sum of new,  base = running sum of need,
//   entry b + i of a sequence <- free_pages[count - 1 - (base + i)],
//   row t of sequence s: position len + (t - seq_start[s]), slot = table[position / page] * page + position % page.
// And when sequences end, or a window has moved past a page: the entries of sequence s that go back, in two ranges [a0, b0)
// and [a1, b1) (gives() in decode_index.cuh), are written behind the free pages in order of sequence and entry.
//
// What bounds them: launch and latency for a decode step (a few kilobytes), and the rows' 12 bytes each for prompts. Every
// block sums the lengths itself (4 or 9 bytes a sequence, from L2) instead of waiting for another's sums, so there is one
// launch, no barrier over the grid and nothing kept between calls. kv_extend works by rows: a row knows whether it opens a page
// (position % page == 0) and then fetches that page from the free ones itself, so no row waits for the table. Measured on the
// device: kv_extend 5.2 us for a token of each of 256 sequences, 10.1 us for 2048 with up to 500 tokens each (half a million
// rows); kv_release 5.2 us for 256 sequences, 9.4 us for 4096 streams with a window.
#include <cuda_runtime.h>

#include <cstdio>

#include "decode_index.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "wenc.h"

wenc_status wenc_internal_fail(wenc_status s, const char* msg);
void wenc_internal_clear_error();
wenc_status wenc_internal_device(int* sms, uint32_t** err);

namespace {

using namespace wenc_dev;
using wenc_host::Range;
using wenc_host::share;
using wenc_host::table_bytes;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                     // sequences a thread takes of a chunk
constexpr int kChunk = kThreads * kPer;     // sequences of a chunk
constexpr int kMaxSeqs = 1 << 16;

struct ExtendParams {
  const int32_t *new_tokens, *lens, *free_pages, *free_count;
  int32_t* table;
  long long table_stride;
  int32_t *lens_out, *count_out, *seq_start, *positions;
  long long* slots;
  int n_seqs, n_rows, n_free, page_size, max_pages;
  int page_shift;      // of a power of two, else -1
  int per;             // sequences a thread takes of a chunk, at most kPer
  int rows_per_block;  // a multiple of 4
};

__device__ __forceinline__ void data_error(uint32_t* err, uint32_t site) {
  *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (site << 8);
}

// Sums of two numbers over the block; `part` holds 2 kWarps numbers. Begins with a barrier.
__device__ __forceinline__ void block_sum2(long long& a, long long& b, long long* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    part[threadIdx.x >> 5] = a;
    part[kWarps + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  a = b = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    a += part[w];
    b += part[kWarps + w];
  }
}

// Exclusive running sums of (a, b) over the block's threads, and the sums in (ta, tb). Begins with a barrier; `part` as above.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb, long long* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sa = a, sb = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, sa, d), ub = __shfl_up_sync(0xffffffffu, sb, d);
    if (lane >= d) {
      sa += ua;
      sb += ub;
    }
  }
  __syncthreads();
  if (lane == 31) {
    part[warp] = sa;
    part[kWarps + warp] = sb;
  }
  __syncthreads();
  long long ba = 0, bb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long pa = part[w], pb = part[kWarps + w];
    if (w < warp) {
      ba += pa;
      bb += pb;
    }
    ta += pa;
    tb += pb;
  }
  a = ba + sa - a;
  b = bb + sb - b;
}

// The rows' places; a block takes rows_per_block rows, and every gridDim.x-th chunk's lengths and offsets.
__global__ void __launch_bounds__(kThreads) kv_extend_kernel(const ExtendParams p, uint32_t* err) {
  __shared__ int start[kChunk + 1], len[kChunk], first_free[kChunk];  // a chunk's first rows, lengths before, pages given before
  __shared__ long long part[2 * kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int cap = p.max_pages * p.page_size;
  auto pages = [&](int n) {  // that n tokens take
    return p.page_shift >= 0 ? static_cast<int>((static_cast<uint32_t>(n) + p.page_size - 1u) >> p.page_shift) : pages_of(n, p.page_size);
  };
  const int count = p.free_count[0];
  const int r0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * p.rows_per_block, static_cast<long long>(p.n_rows)));
  const int r1 = static_cast<int>(min(static_cast<long long>(r0) + p.rows_per_block, static_cast<long long>(p.n_rows)));
  // Is there room for all of it? (Else the call gives nothing to anyone.) Known from a first pass over the lengths when they are
  // more than one chunk, else from the chunk's own sums.
  long long all_rows = 0, all_pages = 0;
  bool bad_len = false, bad = false;
  auto fits = [&](int m, int l) { return m >= 0 && l >= 0 && l <= cap && m <= cap - l; };
  auto judge = [&]() {
    bad = bad_len || all_rows > p.n_rows || count < 0 || count > p.n_free || all_pages > count;
    if (blockIdx.x == 0 && tid == 0) {
      if (bad) data_error(err, bad_len ? 81 : all_rows > p.n_rows ? 82 : 79);
      p.count_out[0] = bad ? count : count - static_cast<int>(all_pages);
      p.seq_start[0] = 0;
    }
  };
  const bool one_chunk = p.n_seqs <= kChunk;
  if (!one_chunk) {
#pragma unroll 4
    for (int s = tid; s < p.n_seqs; s += kThreads) {
      const int m = p.new_tokens[s], l = p.lens[s];
      if (fits(m, l)) {
        all_rows += m;
        all_pages += pages(l + m) - pages(l);
      } else {
        bad_len = true;
      }
    }
    bad_len = __syncthreads_or(bad_len);
    block_sum2(all_rows, all_pages, part);
    judge();
  }

  int row_base = 0, page_base = 0;
  for (int c = 0; c == 0 || c * kChunk < p.n_seqs; ++c) {
    const bool mine = c % gridDim.x == blockIdx.x;
    // (chunks whose rows lie behind the block's are of no use to it, unless a later one's lengths are its own)
    const int ahead = static_cast<int>((blockIdx.x + gridDim.x - c % gridDim.x) % gridDim.x);
    if (c > 0 && row_base >= r1 && static_cast<long long>(c + ahead) * kChunk >= p.n_seqs) break;
    const int s0 = c * kChunk + tid * p.per;  // (per: sequences a thread takes, kPer but in a small batch)
    int m[kPer], l[kPer], need[kPer];
    long long a = 0, b = 0, ta, tb;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool in = i < p.per && s0 + i < p.n_seqs;
      m[i] = in ? p.new_tokens[s0 + i] : 0;
      l[i] = in ? p.lens[s0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool ok = !bad && fits(m[i], l[i]);
      if (!bad && !ok) bad_len = true;
      need[i] = ok ? pages(l[i] + m[i]) - pages(l[i]) : 0;
      a += ok ? m[i] : 0;
      b += need[i];
    }
    if (one_chunk) bad_len = __syncthreads_or(bad_len);
    block_scan2(a, b, ta, tb, part);  // (its barrier: the last chunk's rows are done with the tables)
    if (one_chunk) {
      all_rows = ta;
      all_pages = tb;
      judge();
      if (bad) a = b = ta = tb = 0;
    }
    int ra = static_cast<int>(a) + row_base, pb = static_cast<int>(b) + page_base;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= p.per) break;
      start[tid * p.per + i] = ra;
      len[tid * p.per + i] = l[i];
      first_free[tid * p.per + i] = count - 1 - pb;
      if (!bad) {
        ra += m[i];
        pb += need[i];
      }
      if (mine && s0 + i < p.n_seqs) {
        p.lens_out[s0 + i] = bad ? l[i] : l[i] + m[i];
        p.seq_start[s0 + i + 1] = ra;
      }
    }
    if (tid == 0) start[kThreads * p.per] = row_base + static_cast<int>(ta);
    __syncthreads();
    // ---- the block's rows of this chunk, four neighbours a thread
    const int lo = max(r0, row_base), hi = min(r1, row_base + static_cast<int>(ta));
    for (int t0 = (lo & ~3) + 4 * tid; t0 < hi; t0 += 4 * kThreads) {
      int s = 0;  // the last sequence of the chunk that starts at or before the first of the rows
      {
        const int t = max(t0, lo);
        int n = kThreads * p.per;
        while (n > 1) {
          const int half = n >> 1;
          if (start[s + half] <= t) {
            s += half;
            n -= half;
          } else {
            n = half;
          }
        }
      }
      int pos[4];
      long long slot[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + i;
        pos[i] = 0;
        slot[i] = -1;
        if (t < lo || t >= hi) continue;
        while (start[s + 1] <= t) ++s;  // (t < hi: a sequence of the chunk has the row)
        const int at = len[s] + (t - start[s]), entry = p.page_shift >= 0 ? at >> p.page_shift : at / p.page_size;
        const int off = at - entry * p.page_size, fresh = entry - pages(len[s]);
        int32_t* place = p.table + static_cast<long long>(c * kChunk + s) * p.table_stride + entry;
        int page = -1;
        if (in_bounds(c * kChunk + s < p.n_seqs && entry >= 0 && entry < p.max_pages, err, 110)) {
          if (fresh < 0) {
            page = *place;
          } else if (in_bounds(first_free[s] - fresh >= 0 && first_free[s] - fresh < p.n_free, err, 111)) {
            page = p.free_pages[first_free[s] - fresh];
            if (off == 0) *place = page;
          }
        }
        pos[i] = at;
        slot[i] = static_cast<long long>(page) * p.page_size + off;
        if (page < 0) {
          slot[i] = -1;
          data_error(err, 80);
        }
      }
      if (t0 >= lo && t0 + 4 <= hi) {
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        longlong2* d = reinterpret_cast<longlong2*>(p.slots + t0);
        d[0] = make_longlong2(slot[0], slot[1]);
        d[1] = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + i >= lo && t0 + i < hi) {
            p.positions[t0 + i] = pos[i];
            p.slots[t0 + i] = slot[i];
          }
      }
    }
    row_base += static_cast<int>(ta);
    page_base += static_cast<int>(tb);
  }
  // ---- rows behind the last sequence's
  for (int t = max(r0, bad ? 0 : static_cast<int>(all_rows)) + tid; t < r1; t += kThreads) {
    p.positions[t] = 0;
    p.slots[t] = -1;
  }
}

struct ReleaseParams {
  const int32_t *lens, *table, *free_count, *trimmed;
  const uint8_t* finished;
  int32_t *free_pages, *lens_out, *count_out, *trimmed_out;
  long long table_stride;
  int n_seqs, n_free, page_size, max_pages;
  int window, first;    // window 0: none; first: the entries that hold the first tokens that stay
  int seqs_per_block;   // a multiple of 32
};

// One warp a sequence's entries; the block's sequences 32 at a time, a lane each.
__global__ void __launch_bounds__(kThreads) kv_release_kernel(const ReleaseParams p, uint32_t* err) {
  __shared__ long long part[2 * kWarps];
  __shared__ int4 span[32];
  __shared__ int base[33];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int count = p.free_count[0];
  const int mine0 = blockIdx.x * p.seqs_per_block, mine1 = min(p.n_seqs, mine0 + p.seqs_per_block);
  // the ranges of a sequence's entries that go back, and what its mark becomes
  auto spans = [&](int s, int& mark, bool& bad) {
    const int l = p.lens[s], gone = p.trimmed ? p.trimmed[s] : 0;
    mark = gone;
    if (l < 0 || l > static_cast<long long>(p.max_pages) * p.page_size || gone < 0 || gone > p.max_pages) {
      bad = true;
      return make_int4(0, 0, 0, 0);
    }
    return gives(l, p.finished && p.finished[s] != 0, gone, p.window, p.first, p.page_size, mark);
  };
  // ---- all that goes back, and what goes back before this block's
  long long all = 0, before = 0;
  bool bad_len = false;
#pragma unroll 4
  for (int s = tid; s < p.n_seqs; s += kThreads) {
    int mark;
    const int4 x = spans(s, mark, bad_len);
    const int n = x.y - x.x + x.w - x.z;
    all += n;
    if (s < mine0) before += n;
  }
  bad_len = __syncthreads_or(bad_len);
  block_sum2(all, before, part);
  const bool bad_room = count < 0 || all + count > p.n_free, bad = bad_len || bad_room;
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) data_error(err, bad_len ? 81 : 79);
    p.count_out[0] = bad ? count : count + static_cast<int>(all);
  }
  int at = bad ? 0 : count + static_cast<int>(before);
  for (int s0 = mine0; s0 < mine1; s0 += 32) {
    __syncthreads();
    if (tid < 32) {
      const int s = s0 + tid;
      int4 x = make_int4(0, 0, 0, 0);
      if (s < mine1) {
        int mark;
        bool ignored = false;
        x = spans(s, mark, ignored);
        const bool done = p.finished && p.finished[s] != 0;
        p.lens_out[s] = done && !bad ? 0 : p.lens[s];
        if (p.trimmed_out) p.trimmed_out[s] = !bad ? mark : p.trimmed ? p.trimmed[s] : 0;
        if (bad) x = make_int4(0, 0, 0, 0);
      }
      const int n = x.y - x.x + x.w - x.z;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (tid >= d) sum += up;
      }
      span[tid] = x;
      base[tid + 1] = sum;
      if (tid == 0) base[0] = 0;
    }
    __syncthreads();
    for (int i = tid >> 5; i < 32; i += kWarps) {
      const int4 x = span[i];
      const int n0 = x.y - x.x, n = base[i + 1] - base[i];
      const int32_t* row = p.table + static_cast<long long>(s0 + i) * p.table_stride;
#pragma unroll 4
      for (int j = tid & 31; j < n; j += 32) {
        const int entry = j < n0 ? x.x + j : x.z + j - n0, to = at + base[i] + j;
        if (!in_bounds(s0 + i < p.n_seqs && entry >= 0 && entry < p.max_pages && to >= 0 && to < p.n_free, err, 112)) continue;
        const int page = row[entry];
        if (page < 0) data_error(err, 80);
        p.free_pages[to] = page;
      }
    }
    at += base[32];
  }
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}


wenc_status launch_failed(const char* what, cudaError_t e) {
  char buf[200];
  snprintf(buf, sizeof(buf), "%s launch: %s", what, cudaGetErrorString(e));
  return wenc_internal_fail(WENC_ERR_CUDA, buf);
}

}  // namespace

extern "C" wenc_status wenc_kv_extend(const wenc_kv_extend_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!a) return bad(WENC_ERR_INVALID_ARG, "kv_extend: args is NULL");
  if (!a->free_pages || !a->free_count || !a->free_count_out || !a->seq_start ||
      (a->n_seqs > 0 && (!a->new_tokens || !a->lens || !a->block_table || !a->lens_out)))
    return bad(WENC_ERR_INVALID_ARG, "kv_extend: an array is NULL");
  if (a->n_seqs < 0 || a->page_size < 1 || a->max_pages < 1 || a->n_free_pages < 1 || a->n_rows < 0)
    return bad(WENC_ERR_INVALID_ARG, "kv_extend: sizes must be positive (n_seqs and n_rows may be 0)");
  if (a->n_rows > 0 && (!a->positions || !a->slots)) return bad(WENC_ERR_INVALID_ARG, "kv_extend: positions or slots is NULL");
  if (a->n_seqs > kMaxSeqs) return bad(WENC_ERR_UNSUPPORTED, "kv_extend: %lld sequences, more than %lld", a->n_seqs, kMaxSeqs);
  if (a->n_rows > 0x7ffffff0) return bad(WENC_ERR_UNSUPPORTED, "kv_extend: n_rows %lld passes 2^31 - 16", a->n_rows);
  if (static_cast<long long>(a->max_pages) * a->page_size > 0x7fffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "kv_extend: max_pages %lld x page_size %lld passes 2^31 - 1", a->max_pages, a->page_size);
  if (a->n_seqs > 1 && a->block_table_stride < a->max_pages)
    return bad(WENC_ERR_INVALID_ARG, "kv_extend: block_table_stride %lld < max_pages %lld", a->block_table_stride, a->max_pages);
  if ((reinterpret_cast<uintptr_t>(a->positions) | reinterpret_cast<uintptr_t>(a->slots)) & 15u)
    return bad(WENC_ERR_INVALID_ARG, "kv_extend: positions and slots must be 16-byte aligned");
  // (blocks read the inputs while others write)
  const long long seqs = 4ll * a->n_seqs, rows = a->n_rows;
  const Range in[] = {{a->new_tokens, seqs}, {a->lens, seqs}, {a->free_count, 4}, {a->free_pages, 4ll * a->n_free_pages}};
  const Range out[] = {{a->lens_out, seqs}, {a->free_count_out, 4}, {a->seq_start, seqs + 4}, {a->positions, 4 * rows},
                       {a->slots, 8 * rows}, {a->block_table, table_bytes(a->n_seqs, a->block_table_stride, a->max_pages)}};
  if (share(in, out)) return bad(WENC_ERR_INVALID_ARG, "kv_extend: the outputs and the table must lie apart from the inputs");
  if (share(out)) return bad(WENC_ERR_INVALID_ARG, "kv_extend: the outputs and the table must lie apart from one another");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  ExtendParams p;
  p.new_tokens = a->new_tokens;
  p.lens = a->lens;
  p.free_pages = a->free_pages;
  p.free_count = a->free_count;
  p.table = a->block_table;
  p.table_stride = a->block_table_stride;
  p.lens_out = a->lens_out;
  p.count_out = a->free_count_out;
  p.seq_start = a->seq_start;
  p.positions = a->positions;
  p.slots = reinterpret_cast<long long*>(a->slots);
  p.n_seqs = a->n_seqs;
  p.n_rows = a->n_rows;
  p.n_free = a->n_free_pages;
  p.page_size = a->page_size;
  p.max_pages = a->max_pages;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a->page_size == 1 << s) p.page_shift = s;
  p.per = a->n_seqs <= kThreads ? 1 : kPer;
  // four rows a thread and pass; two blocks an SM at most
  long long blocks = (static_cast<long long>(a->n_rows) + 4 * kThreads - 1) / (4 * kThreads);
  if (blocks > 2ll * sms) blocks = 2ll * sms;
  if (blocks < 1) blocks = 1;
  p.rows_per_block = static_cast<int>(((a->n_rows + blocks - 1) / blocks + 3) / 4 * 4);
  const cudaError_t e = wenc_host::launch_pdl(kv_extend_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                                              reinterpret_cast<cudaStream_t>(stream), p, err);
  return e == cudaSuccess ? WENC_OK : launch_failed("kv_extend", e);
}

extern "C" wenc_status wenc_kv_release(const wenc_kv_release_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  if (!a) return bad(WENC_ERR_INVALID_ARG, "kv_release: args is NULL");
  if (!a->free_pages || !a->free_count || !a->free_count_out || (a->n_seqs > 0 && (!a->lens || !a->block_table || !a->lens_out)))
    return bad(WENC_ERR_INVALID_ARG, "kv_release: an array is NULL");
  if (a->n_seqs > 0 && !a->finished && a->window == 0) return bad(WENC_ERR_INVALID_ARG, "kv_release: neither finished nor a window");
  if (a->n_seqs > 0 && ((a->trimmed == nullptr) != (a->trimmed_out == nullptr) || (a->window > 0) != (a->trimmed != nullptr)))
    return bad(WENC_ERR_INVALID_ARG, "kv_release: trimmed and trimmed_out go with a window");
  if (a->n_seqs < 0 || a->page_size < 1 || a->max_pages < 1 || a->n_free_pages < 1)
    return bad(WENC_ERR_INVALID_ARG, "kv_release: sizes must be positive (n_seqs may be 0)");
  if (a->window < 0 || a->sinks < 0) return bad(WENC_ERR_INVALID_ARG, "kv_release: window or sinks is negative");
  if (a->n_seqs > kMaxSeqs) return bad(WENC_ERR_UNSUPPORTED, "kv_release: %lld sequences, more than %lld", a->n_seqs, kMaxSeqs);
  if (static_cast<long long>(a->max_pages) * a->page_size > 0x7fffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "kv_release: max_pages %lld x page_size %lld passes 2^31 - 1", a->max_pages, a->page_size);
  if (a->n_seqs > 1 && a->block_table_stride < a->max_pages)
    return bad(WENC_ERR_INVALID_ARG, "kv_release: block_table_stride %lld < max_pages %lld", a->block_table_stride, a->max_pages);
  const long long seqs = 4ll * a->n_seqs;
  const Range in[] = {{a->lens, seqs}, {a->trimmed, seqs}, {a->free_count, 4}, {a->finished, a->n_seqs},
                      {a->block_table, table_bytes(a->n_seqs, a->block_table_stride, a->max_pages)}};
  const Range out[] = {{a->lens_out, seqs}, {a->trimmed_out, seqs}, {a->free_count_out, 4}, {a->free_pages, 4ll * a->n_free_pages}};
  if (share(in, out)) return bad(WENC_ERR_INVALID_ARG, "kv_release: the outputs and free_pages must lie apart from the inputs");
  if (share(out)) return bad(WENC_ERR_INVALID_ARG, "kv_release: the outputs and free_pages must lie apart from one another");
  int sms = 0;
  uint32_t* err = nullptr;
  const wenc_status dst = wenc_internal_device(&sms, &err);
  if (dst != WENC_OK) return dst;
  ReleaseParams p;
  p.lens = a->lens;
  p.table = a->block_table;
  p.free_count = a->free_count;
  p.trimmed = a->trimmed;
  p.finished = a->finished;
  p.free_pages = a->free_pages;
  p.lens_out = a->lens_out;
  p.count_out = a->free_count_out;
  p.trimmed_out = a->trimmed_out;
  p.table_stride = a->block_table_stride;
  p.n_seqs = a->n_seqs;
  p.n_free = a->n_free_pages;
  p.page_size = a->page_size;
  p.max_pages = a->max_pages;
  p.window = a->window;
  p.first = a->window > 0 ? pages_of(a->sinks, a->page_size) : 0;
  // (a block reads every length before its own: more sequences a block when there are many)
  const int per = (a->n_seqs + 2 * sms - 1) / (2 * sms);
  p.seqs_per_block = (per + 31) / 32 * 32;
  if (p.seqs_per_block < 32) p.seqs_per_block = 32;
  const int blocks = a->n_seqs > 0 ? (a->n_seqs + p.seqs_per_block - 1) / p.seqs_per_block : 1;
  const cudaError_t e = wenc_host::launch_pdl(kv_release_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                                              reinterpret_cast<cudaStream_t>(stream), p, err);
  return e == cudaSuccess ? WENC_OK : launch_failed("kv_release", e);
}
