// prefix_attn.cu -- attention of a decode step whose sequences share long prefixes.
//
// The beams of a window attend to the same cross-attention keys, and requests behind one prompt to
// the same prompt keys; each sequence adds keys of its own, kept in pages (append.cu). For query
// row (token i of sequence s, head h), with g the group of s and key head h / (H / Hkv):
//   out = softmax(scale * q . [K_prefix(g); K_own(s)]) [V_prefix(g); V_own(s)],
// every prefix key visible, own key j visible when j <= lens[s] - q_len + i, zeros where nothing is
// (inferencelayer 0.2.4 src/whisper_gpu.rs, DEC_QATTN; oxinfer 0.0.5 src/whisper/model.rs,
// CrossLayer::attend and attention_masked).
//
// Rows of one key head: (sequence of the group, token, query head of the key head), so the prefix is read
// once for all of a group. What bounds it: bytes of K and V for a few rows (a decode step), the tensor
// pipe for hundreds. Hence two forms:
//
// Up to 64 rows per key head (beams): one launch. A cluster of 1 to 8 CTAs attends one (group, key
// head): its key list is the prefix followed by the own keys of each sequence of the group, cut into
// tiles that belong to one of these segments each, and every CTA takes an equal run of tiles. Own keys
// are scored against all the item's rows (the MMA is 16 rows high whether one or 16 are wanted) and
// masked to their sequence's. The CTAs' results (m, l, O) are joined through distributed shared memory:
// no workspace and no second kernel.
// More rows: a work item is a share of a group's prefix, or of one sequence's own keys; items write
// partial results to the workspace and a second kernel joins them.
//
// Inside a CTA, up to 16 rows: the four warps split the keys of each tile, each warp with its own ring
// of cp.async stages, no barrier between them, joined once at the end. More rows: the warps split the
// rows (16 each) and share the tiles.
// Scores use mma.sync (m16n8k16 bf16, m16n8k8 TF32): 16 rows is its height, where a tcgen05 tile
// would be 64 or 128 rows high and mostly empty.
// bf16: P is split into two bf16 parts before P V, so its rounding (2^-16 after the split) does not
// add to the output's own. fp32: every product is three TF32 products of two-part operands.
#include <cuda_bf16.h>
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
uint32_t* wenc_internal_error_word(std::string* why);
bool wenc_internal_is_sm103(std::string* why);
int wenc_internal_sm_count();

namespace {

using namespace wenc_dev;

constexpr int HD = 64;
constexpr int kThreads = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;  // 0 source bytes: the 16 are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo with both parts TF32 (11 significant bits each, nearest, ties away): the parts
// miss x by at most 2^-24 |x|.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = (__float_as_uint(x - __uint_as_float(hi)) + 0x1000u) & 0xffffe000u;
}

struct PrefixParams {
  const uint8_t* q;
  uint8_t* out;
  long long q_stride, out_stride;  // bytes between tokens
  const uint8_t *kp, *vp;
  long long k_group, k_token, v_group, v_token;  // bytes
  const uint8_t *k_pages, *v_pages;
  long long k_page, v_page, page_row;  // bytes between pages; bytes of one page slot
  const int32_t *group_start, *prefix_lens, *table, *lens;
  long long table_stride;
  int n_seqs, q_len, H, Hkv, r, n_groups, max_group, prefix_max, n_pages, page_size, page_shift, max_pages;
  int np, ns;                    // prefix and own-key splits of the two-launch form (0: no such keys)
  int row_tiles;                 // row tiles per item of this launch (two-launch form)
  int cluster;                   // CTAs per item (one-launch form)
  float scale_log2;              // >= 0
  uint32_t q_flip, q_keep;       // a negative scale turns the queries' signs (per 32 bits), a zero one clears them
  float* part_o;                 // [(token * H + head) * (np + ns) + slot][64]
  float2* part_ml;               // the same without [64]: (maximum in log2 units, sum)
};

// WR warps along the rows, WK along the keys of a tile.
template <typename T, int WR>
struct Cfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int WK = 4 / WR;
  static constexpr int KW = (F32 ? 16 : 32) * (WR == 4 ? 2 : 1);  // keys of a tile one warp scores
  static constexpr int KT = KW * WK;                              // keys per tile
  static constexpr int ROWB = HD * sizeof(T);
  static constexpr int STAGES = WR == 4 ? 4 : 3;
  static constexpr uint32_t HALF = KT * ROWB;  // bytes of K (or V) per stage
  static constexpr uint32_t STAGE = 2 * HALF;
  static constexpr uint32_t SMEM = STAGES * STAGE;
  static_assert(SMEM >= 4u * 16 * HD * 4 + 4 * 16 * 8, "the ring also holds the warps' results");
};

// What one CTA attends: rows [row0, row0 + 16 WR) of the n_rows of one key head, against its run of the
// tiles of a list of segments: segment 0 is the prefix, segment i the own keys of sequence i - 1 of the
// item, which only that sequence's rows see.
struct Item {
  const uint8_t *kp, *vp;   // first prefix key of the key head
  int prefix_len;
  int seq0, n_own;          // first sequence, and how many bring own keys (0: none do)
  int row0, n_rows;
  int token0, hk;           // row x is token token0 + x / r, query head hk r + x % r
  int split, n_splits;
};

constexpr int kMaxOwn = 64;  // own-key segments of an item: at most one per row of a 64-row tile
struct SegTable {
  int tile0[kMaxOwn + 2];    // first tile of each segment, and the end
  int len[kMaxOwn + 1];      // its keys
};

// 16-byte granule `c` of key row `row` within a tile. bf16 rows have 8 granules (all 32 banks), fp32
// rows 16; the XOR spreads the rows an ldmatrix (or the quads of a fragment load) touches at once
// over all banks.
template <bool F32>
__device__ __forceinline__ uint32_t granule(int row, int c) {
  if constexpr (F32)
    return row * 256u + ((c ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2))) << 4);
  else
    return row * 128u + ((c ^ (row & 7)) << 4);
}

// One CTA's share: leaves O (unnormalised) in shared memory as [16 WR][64] floats and (m, l) per row
// behind it at kMlOffset, m in log2 units. All threads return after a barrier.
constexpr uint32_t kMlOffset = 4 * 16 * HD * 4;

template <typename T, int WR>
__device__ __forceinline__ void attend(const PrefixParams& p, const Item& it, uint8_t* smem, SegTable& seg, uint32_t* err) {
  using C = Cfg<T, WR>;
  constexpr bool F32 = C::F32;
  constexpr int WK = C::WK, KW = C::KW, KT = C::KT, ST = C::STAGES;
  constexpr int CH = C::ROWB / 16;  // granules per row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = WR == 4 ? warp : 0, wk = WK == 4 ? warp : 0;
  const int g = lane >> 2, tq = lane & 3;
  const uint32_t s0 = smem_u32(smem);

  // ---- the segments' tiles: a running sum over up to 65 lengths, by warp 0
  if (warp == 0) {
    int base = (it.prefix_len + KT - 1) / KT;
    if (lane == 0) {
      seg.tile0[0] = 0;
      seg.len[0] = it.prefix_len;
      seg.tile0[1] = base;
    }
    for (int i0 = 0; i0 < it.n_own; i0 += 32) {
      const int i = i0 + lane;
      int n = i < it.n_own ? p.lens[it.seq0 + i] : 0;
      if (n < 0 || n > static_cast<long long>(p.max_pages) * p.page_size) {
        *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
        n = 0;
      }
      int sum = (n + KT - 1) / KT;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      if (i < it.n_own) {
        seg.len[1 + i] = n;
        seg.tile0[2 + i] = base + sum;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  const int n_tiles = seg.tile0[1 + it.n_own];
  const int per = (n_tiles + it.n_splits - 1) / it.n_splits;
  const int tile0 = it.split * per;
  const int n_mine = max(0, min(per, n_tiles - tile0));

  // ---- tile loads: a warp of the key-split form loads the keys it scores itself; else the CTA
  constexpr int LOADERS = WK == 4 ? 32 : kThreads;
  constexpr int LROWS = WK == 4 ? KW : KT;
  constexpr int NL = LROWS * CH / LOADERS;
  const int lt = WK == 4 ? lane : threadIdx.x;
  const int lc = lt % CH, lr = (WK == 4 ? wk * KW : 0) + lt / CH;
  int lseg = 0;  // segment of the next tile to load
  auto load = [&](int j, int stage) {
    while (tile0 + j >= seg.tile0[lseg + 1]) ++lseg;
    const uint32_t sk = s0 + stage * C::STAGE, sv = sk + C::HALF;
    const int key0 = (tile0 + j - seg.tile0[lseg]) * KT, n_keys = seg.len[lseg];
    if (lseg == 0) {
      const uint8_t* ks = it.kp + (key0 + lr) * p.k_token + lc * 16;
      const uint8_t* vs = it.vp + (key0 + lr) * p.v_token + lc * 16;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int row = lr + i * (LOADERS / CH);
        const bool ok = key0 + row < n_keys;
        cp_async16(sk + granule<F32>(row, lc), ok ? ks : it.kp, ok);
        cp_async16(sv + granule<F32>(row, lc), ok ? vs : it.vp, ok);
        ks += (LOADERS / CH) * p.k_token;
        vs += (LOADERS / CH) * p.v_token;
      }
    } else {
      const int32_t* table = p.table + (it.seq0 + lseg - 1) * p.table_stride;
      int page[NL], slot[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int key = key0 + lr + i * (LOADERS / CH);
        const int pi = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
        slot[i] = key - pi * p.page_size;
        page[i] = key < n_keys ? table[pi] : -1;
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int row = lr + i * (LOADERS / CH);
        const bool ok = page[i] >= 0 && page[i] < p.n_pages;
        if (!ok && key0 + row < n_keys) *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (80u << 8);
        const long long at = slot[i] * p.page_row + it.hk * C::ROWB + lc * 16;
        cp_async16(sk + granule<F32>(row, lc), ok ? p.k_pages + page[i] * p.k_page + at : p.k_pages, ok);
        cp_async16(sv + granule<F32>(row, lc), ok ? p.v_pages + page[i] * p.v_page + at : p.v_pages, ok);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < ST - 1; ++j) {
    if (j < n_mine) load(j, j);
    cp_async_commit();
  }

  // ---- the warp's 16 query rows as A fragments; rows past the end are zeros
  const int ra = it.row0 + wr * 16 + g, rb = ra + 8;
  auto q_row = [&](int x) {
    const int tok = x / p.r;
    return p.q + static_cast<long long>(it.token0 + tok) * p.q_stride + (it.hk * p.r + x - tok * p.r) * C::ROWB;
  };
  constexpr int KS = F32 ? 8 : 4;  // k steps of one score product
  uint32_t qa[KS][4], ql[F32 ? KS : 1][4];
  {
    const uint8_t *pa = ra < it.n_rows ? q_row(ra) : nullptr, *pb = rb < it.n_rows ? q_row(rb) : nullptr;
    if constexpr (F32) {
      // k index tq (and tq + 4) of step 2j (and 2j + 1) stands for element 4 (tq + 4j) + {0, 1} ({2, 3})
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        uint4 a = pa ? *reinterpret_cast<const uint4*>(pa + (tq + 4 * j) * 16) : z;
        uint4 b = pb ? *reinterpret_cast<const uint4*>(pb + (tq + 4 * j) * 16) : z;
        auto part = [&](uint32_t x, uint32_t& hi, uint32_t& lo) {
          split_tf32(__uint_as_float((x & p.q_keep) ^ p.q_flip), hi, lo);
        };
        part(a.x, qa[2 * j][0], ql[2 * j][0]);
        part(b.x, qa[2 * j][1], ql[2 * j][1]);
        part(a.y, qa[2 * j][2], ql[2 * j][2]);
        part(b.y, qa[2 * j][3], ql[2 * j][3]);
        part(a.z, qa[2 * j + 1][0], ql[2 * j + 1][0]);
        part(b.z, qa[2 * j + 1][1], ql[2 * j + 1][1]);
        part(a.w, qa[2 * j + 1][2], ql[2 * j + 1][2]);
        part(b.w, qa[2 * j + 1][3], ql[2 * j + 1][3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int e = (16 * k + 2 * tq) * 2;
        auto part = [&](const uint8_t* x) { return x ? (*reinterpret_cast<const uint32_t*>(x) & p.q_keep) ^ p.q_flip : 0u; };
        qa[k][0] = part(pa ? pa + e : nullptr);
        qa[k][1] = part(pb ? pb + e : nullptr);
        qa[k][2] = part(pa ? pa + e + 16 : nullptr);
        qa[k][3] = part(pb ? pb + e + 16 : nullptr);
      }
    }
  }
  // sequence of the item and token of this thread's two rows
  const int per_seq = p.q_len * p.r;
  const int sa = ra / per_seq, sb = rb / per_seq;
  const int ta = (ra - sa * per_seq) / p.r, tb = (rb - sb * per_seq) / p.r;
  const int row_first = it.row0 + wr * 16, row_end = min(row_first + 16, it.n_rows);  // warp-uniform

  float o[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
  float ma = -CUDART_INF_F, mb = -CUDART_INF_F, la = 0.0f, lb = 0.0f;
  const float sc = p.scale_log2;

  int cseg = 0;
  for (int j = 0; j < n_mine; ++j) {
    cp_async_wait<ST - 2>();
    if constexpr (WK == 4) __syncwarp();
    else __syncthreads();
    if (j + ST - 1 < n_mine) load(j + ST - 1, (j + ST - 1) % ST);
    cp_async_commit();
    while (tile0 + j >= seg.tile0[cseg + 1]) ++cseg;
    const int kb = wk * KW;  // first key of the tile this warp scores
    const int key0 = (tile0 + j - seg.tile0[cseg]) * KT + kb, n_keys = seg.len[cseg];
    // nothing to score: no rows, no keys, or own keys of a sequence none of the warp's rows belong to
    if (row_first >= row_end || key0 >= n_keys) continue;
    if (cseg > 0 && (row_end <= (cseg - 1) * per_seq || row_first >= cseg * per_seq)) continue;
    const uint32_t sk = s0 + (j % ST) * C::STAGE, sv = sk + C::HALF;

    // ---- scores of 16 rows x KW keys
    float s[KW / 8][4];
#pragma unroll
    for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
      if constexpr (F32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 kv = lds_f4(sk + granule<true>(kb + 8 * n + g, tq + 4 * c));
          uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
          split_tf32(kv.x, h0, l0);
          split_tf32(kv.y, h1, l1);
          split_tf32(kv.z, h2, l2);
          split_tf32(kv.w, h3, l3);
          mma_tf32(s[n], ql[2 * c], h0, h1);
          mma_tf32(s[n], qa[2 * c], l0, l1);
          mma_tf32(s[n], qa[2 * c], h0, h1);
          mma_tf32(s[n], ql[2 * c + 1], h2, h3);
          mma_tf32(s[n], qa[2 * c + 1], l2, l3);
          mma_tf32(s[n], qa[2 * c + 1], h2, h3);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 32 elements of d at a time
          uint32_t b[4];
          ldsm_x4(b, sk + granule<false>(kb + 8 * n + (lane & 7), 4 * c + (lane >> 3)));
          mma_bf16(s[n], qa[2 * c], b[0], b[1]);
          mma_bf16(s[n], qa[2 * c + 1], b[2], b[3]);
        }
      }
    }
    // ---- mask, running maximum and sum (log2 units)
    int lim_a = n_keys, lim_b = n_keys;  // keys of this segment each of this thread's rows sees
    if (cseg > 0) {
      lim_a = sa == cseg - 1 ? n_keys - p.q_len + 1 + ta : 0;
      lim_b = sb == cseg - 1 ? n_keys - p.q_len + 1 + tb : 0;
    }
    if (cseg > 0 || key0 + KW > n_keys) {
#pragma unroll
      for (int n = 0; n < KW / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 8 * n + 2 * tq + (e & 1) >= (e < 2 ? lim_a : lim_b)) s[n][e] = -CUDART_INF_F;
    }
    float xa = -CUDART_INF_F, xb = -CUDART_INF_F;
#pragma unroll
    for (int n = 0; n < KW / 8; ++n) {
      xa = fmax3(xa, s[n][0], s[n][1]);
      xb = fmax3(xb, s[n][2], s[n][3]);
    }
    xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
    xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
    xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
    xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
    xa = fmaxf(xa * sc, ma);
    xb = fmaxf(xb * sc, mb);
    const float ua = xa == -CUDART_INF_F ? 0.0f : xa, ub = xb == -CUDART_INF_F ? 0.0f : xb;
    const float fa = ex2_approx(ma - ua), fb = ex2_approx(mb - ub);
    ma = xa;
    mb = xb;
    la *= fa;
    lb *= fb;
#pragma unroll
    for (int n = 0; n < KW / 8; ++n) {
      s[n][0] = ex2_approx(fmaf(s[n][0], sc, -ua));
      s[n][1] = ex2_approx(fmaf(s[n][1], sc, -ua));
      s[n][2] = ex2_approx(fmaf(s[n][2], sc, -ub));
      s[n][3] = ex2_approx(fmaf(s[n][3], sc, -ub));
      la += s[n][0] + s[n][1];
      lb += s[n][2] + s[n][3];
    }
    // ---- O += P V. fp32: the tile's product is formed on its own and added in one rounding, so that the
    // tensor core's accumulation (which truncates) runs over one tile only
    float t[F32 ? 8 : 1][4];
    if constexpr (F32) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[n][e] = 0.0f;
    } else {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        o[n][0] *= fa;
        o[n][1] *= fa;
        o[n][2] *= fb;
        o[n][3] *= fb;
      }
    }
    if constexpr (F32) {
      // k index t of a step stands for key 2t, t + 4 for key 2t + 1 (where the scores already are);
      // column index g of product n for element 4g + n % 4 + 32 (n / 4)
#pragma unroll
      for (int k = 0; k < KW / 8; ++k) {
        uint32_t ph[4], pl[4];
        split_tf32(s[k][0], ph[0], pl[0]);
        split_tf32(s[k][2], ph[1], pl[1]);
        split_tf32(s[k][1], ph[2], pl[2]);
        split_tf32(s[k][3], ph[3], pl[3]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float4 v0 = lds_f4(sv + granule<true>(kb + 8 * k + 2 * tq, g + 8 * c));
          const float4 v1 = lds_f4(sv + granule<true>(kb + 8 * k + 2 * tq + 1, g + 8 * c));
          const float w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint32_t h0, l0, h1, l1;
            split_tf32(w0[n], h0, l0);
            split_tf32(w1[n], h1, l1);
            mma_tf32(t[4 * c + n], pl, h0, h1);
            mma_tf32(t[4 * c + n], ph, l0, l1);
            mma_tf32(t[4 * c + n], ph, h0, h1);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        o[n][0] = fmaf(o[n][0], fa, t[n][0]);
        o[n][1] = fmaf(o[n][1], fa, t[n][1]);
        o[n][2] = fmaf(o[n][2], fb, t[n][2]);
        o[n][3] = fmaf(o[n][3], fb, t[n][3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KW / 16; ++k) {
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = s[2 * k + (e >> 1)][2 * (e & 1)], y = s[2 * k + (e >> 1)][2 * (e & 1) + 1];
          ph[e] = pack_bf16x2(x, y);
          pl[e] = pack_bf16x2(x - __uint_as_float(ph[e] << 16), y - __uint_as_float(ph[e] & 0xffff0000u));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 elements of d at a time
          uint32_t b[4];
          ldsm_x4_t(b, sv + granule<false>(kb + 16 * k + (lane & 15), 2 * c + (lane >> 4)));
          mma_bf16(o[2 * c], ph, b[0], b[1]);
          mma_bf16(o[2 * c + 1], ph, b[2], b[3]);
          mma_bf16(o[2 * c], pl, b[0], b[1]);
          mma_bf16(o[2 * c + 1], pl, b[2], b[3]);
        }
      }
    }
  }
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);

  // ---- the warps' results through shared memory (over the ring): O [4][16][64], (m, l) [4][16]
  cp_async_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(smem + kMlOffset);
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    float* d0 = so + (warp * 16 + g) * HD;
    float* d1 = d0 + 8 * HD;
    const int c0 = F32 ? 8 * tq + (n & 3) + 32 * (n >> 2) : 8 * n + 2 * tq, c1 = F32 ? c0 + 4 : c0 + 1;
    d0[c0] = o[n][0];
    d0[c1] = o[n][1];
    d1[c0] = o[n][2];
    d1[c1] = o[n][3];
  }
  if (tq == 0) {
    sml[warp * 16 + g] = make_float2(ma, la);
    sml[warp * 16 + g + 8] = make_float2(mb, lb);
  }
  __syncthreads();
  if constexpr (WK == 4) {  // join of the four warps: 8 threads a row, 8 elements each
    const int x = threadIdx.x >> 3, c8 = (threadIdx.x & 7) * 8;
    float m = -CUDART_INF_F, l = 0.0f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WK; ++w) m = fmaxf(m, sml[w * 16 + x].x);
    const float u = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float2 ml = sml[w * 16 + x];
      const float f = ex2_approx(ml.x - u);
      l += f * ml.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += f * so[(w * 16 + x) * HD + c8 + e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) so[x * HD + c8 + e] = v[e];
    if (c8 == 0) sml[x] = make_float2(m, l);
    __syncthreads();
  }
}

// Eight elements of an output row, normalised (a row without a visible key: zeros).
template <typename T>
__device__ __forceinline__ void write_out8(const PrefixParams& p, int token, int head, int c8, const float (&v)[8], float l) {
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint8_t* dst = p.out + static_cast<long long>(token) * p.out_stride + (head * HD + c8) * static_cast<int>(sizeof(T));
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
  }
}

// The sequences of a group (a range that leads outside the batch, or a group larger than max_group,
// is cut and reported).
__device__ __forceinline__ void group_range(const PrefixParams& p, int g, int& begin, int& count, uint32_t* err) {
  if (!p.group_start) {
    begin = g * p.max_group;
    count = p.max_group;
    return;
  }
  begin = p.group_start[g];
  const int end = p.group_start[g + 1];
  count = end - begin;
  if (begin < 0 || count < 0 || end > p.n_seqs || count > p.max_group) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (82u << 8);
    count = 0;
  }
}

__device__ __forceinline__ int prefix_len_of(const PrefixParams& p, int grp, uint32_t* err) {
  int n = p.prefix_lens ? p.prefix_lens[grp] : p.prefix_max;
  if (n < 0 || n > p.prefix_max) {
    *reinterpret_cast<volatile uint32_t*>(err) = kErrData | (81u << 8);
    n = 0;
  }
  return n;
}

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t rank_addr(uint32_t saddr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// One-launch form: cluster blockIdx.x / cluster attends one (group, key head), all of its rows.
template <typename T, int WR>
__global__ void __launch_bounds__(kThreads) prefix_cluster_kernel(const PrefixParams p, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  __shared__ SegTable seg;
  pdl_trigger();
  pdl_wait();
  const int item = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
  Item it;
  const int grp = item / p.Hkv;
  it.hk = item % p.Hkv;
  int begin, count;
  group_range(p, grp, begin, count, err);
  if (count == 0) return;  // the whole cluster
  it.kp = p.kp + grp * p.k_group + it.hk * static_cast<int>(HD * sizeof(T));
  it.vp = p.vp + grp * p.v_group + it.hk * static_cast<int>(HD * sizeof(T));
  it.prefix_len = p.kp ? prefix_len_of(p, grp, err) : 0;
  it.seq0 = begin;
  it.n_own = p.k_pages ? count : 0;
  it.row0 = 0;
  it.n_rows = count * p.q_len * p.r;
  it.token0 = begin * p.q_len;
  it.split = rank;
  it.n_splits = p.cluster;
  attend<T, WR>(p, it, smem_dyn, seg, err);
  if (p.cluster > 1) cluster_arrive_wait();
  // the ranks share the rows out: 8 threads a row, 8 elements each
  const uint32_t so = smem_u32(smem_dyn);
  const int c8 = (threadIdx.x & 7) * 8;
  for (int x = rank + p.cluster * (threadIdx.x >> 3); x < it.n_rows; x += p.cluster * (kThreads / 8)) {
    float m = -CUDART_INF_F, l = 0.0f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float2 ml[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < p.cluster) {
        ml[i] = ld_cluster_f2(rank_addr(so + kMlOffset + x * 8, i));
        m = fmaxf(m, ml[i].x);
      }
    }
    const float u = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < p.cluster) {
        const float f = ex2_approx(ml[i].x - u);
        const uint32_t a = rank_addr(so + (x * HD + c8) * 4, i);
        const float4 o0 = ld_cluster_f4(a), o1 = ld_cluster_f4(a + 16);
        l += f * ml[i].y;
        v[0] += f * o0.x; v[1] += f * o0.y; v[2] += f * o0.z; v[3] += f * o0.w;
        v[4] += f * o1.x; v[5] += f * o1.y; v[6] += f * o1.z; v[7] += f * o1.w;
      }
    }
    const int tok = x / p.r;
    write_out8<T>(p, it.token0 + tok, it.hk * p.r + x - tok * p.r, c8, v, l);
  }
  if (p.cluster > 1) cluster_arrive_wait();  // no CTA leaves while another reads its results
}

// Two-launch form: one CTA per (group, key head, split of the prefix, row tile), or (OWN) per
// (sequence, key head, split of its own keys, row tile); writes its rows' partial results.
template <typename T, int WR, bool OWN>
__global__ void __launch_bounds__(kThreads) prefix_part_kernel(const PrefixParams p, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem_dyn[];
  __shared__ SegTable seg;
  pdl_trigger();
  pdl_wait();
  int b = blockIdx.x;
  Item it;
  it.row0 = (b % p.row_tiles) * 16 * WR;
  b /= p.row_tiles;
  it.n_splits = OWN ? p.ns : p.np;
  it.split = b % it.n_splits;
  b /= it.n_splits;
  it.hk = b % p.Hkv;
  const int which = b / p.Hkv;
  int begin = which, count = 1;
  it.kp = p.kp;
  it.vp = p.vp;
  it.prefix_len = 0;
  it.n_own = 1;
  if (!OWN) {
    group_range(p, which, begin, count, err);
    it.kp = p.kp + which * p.k_group + it.hk * static_cast<int>(HD * sizeof(T));
    it.vp = p.vp + which * p.v_group + it.hk * static_cast<int>(HD * sizeof(T));
    it.prefix_len = prefix_len_of(p, which, err);
    it.n_own = 0;
  }
  it.n_rows = count * p.q_len * p.r;
  if (it.row0 >= it.n_rows) return;
  it.seq0 = begin;
  it.token0 = begin * p.q_len;
  attend<T, WR>(p, it, smem_dyn, seg, err);
  const float* so = reinterpret_cast<const float*>(smem_dyn);
  const float2* sml = reinterpret_cast<const float2*>(smem_dyn + kMlOffset);
  const int n_slots = p.np + p.ns, slot = (OWN ? p.np : 0) + it.split, c8 = (threadIdx.x & 7) * 8;
  for (int y = threadIdx.x >> 3; y < 16 * WR; y += kThreads / 8) {
    const int x = it.row0 + y;
    if (x >= it.n_rows) break;
    const int tok = x / p.r, head = it.hk * p.r + x - tok * p.r;
    const float2 ml = sml[y];
    const size_t at = (static_cast<size_t>(it.token0 + tok) * p.H + head) * n_slots + slot;
    if (ml.y > 0.0f) {
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * HD + c8);
      dst[0] = *reinterpret_cast<const float4*>(so + y * HD + c8);
      dst[1] = *reinterpret_cast<const float4*>(so + y * HD + c8 + 4);
    }
    if (c8 == 0) p.part_ml[at] = ml;
  }
}

// Join of the partial results of one (token, head): sixteen lanes, four elements each.
template <typename T>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PrefixParams p) {
  pdl_trigger();
  pdl_wait();
  const long long pair = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
  const int c4 = threadIdx.x & 15;
  const long long n_pairs = static_cast<long long>(p.n_seqs) * p.q_len * p.H;
  if (pair >= n_pairs) return;
  const int token = static_cast<int>(pair / p.H), head = static_cast<int>(pair % p.H);
  // rows of no group have no partial results: left as they were
  if (p.np && p.group_start) {
    const int seq = token / p.q_len;
    int lo = 0, hi = p.n_groups;  // the last group that starts at or before seq
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.group_start[mid] <= seq) lo = mid;
      else hi = mid;
    }
    const int begin = p.group_start[lo], end = p.group_start[lo + 1];
    if (seq < begin || seq >= end || begin < 0 || end > p.n_seqs || end - begin > p.max_group) return;
  }
  const int n = p.np + p.ns;
  const float2* ml = p.part_ml + pair * n;
  const float* po = p.part_o + pair * n * HD + c4 * 4;
  float m = -CUDART_INF_F;
  for (int i = 0; i < n; ++i) m = fmaxf(m, ml[i].x);
  const float u = m == -CUDART_INF_F ? 0.0f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.0f;
  for (int i = 0; i < n; ++i) {
    const float2 x = ml[i];
    if (!(x.y > 0.0f)) continue;  // an empty share wrote no O
    const float f = ex2_approx(x.x - u);
    const float4 o = *reinterpret_cast<const float4*>(po + static_cast<size_t>(i) * HD);
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
    l += f * x.y;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint8_t* dst = p.out + token * p.out_stride + (head * HD + c4 * 4) * sizeof(T);
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

wenc_status bad(wenc_status s, const char* fmt, long long a = 0, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return wenc_internal_fail(s, buf);
}

// How one call is divided, from its sizes alone.
struct Plan {
  int cluster = 0;              // > 0: the one-launch form, CTAs per item
  int wr = 0;                   // its warps along the rows
  int wr_p = 0, wr_s = 0;       // two-launch form: warps along the rows of prefix and own-key items
  int rows_p = 0, rows_s = 0;   // row tiles
  int np = 0, ns = 0;           // key splits
  long long items_p = 0, items_s = 0;  // CTAs (one-launch form: items_p)
  size_t part_o = 0, bytes = 0;  // offset of the (m, l) pairs; workspace bytes
};

int tile_keys(bool f32, int wr) {
  if (wr == 4) return f32 ? Cfg<float, 4>::KT : Cfg<__nv_bfloat16, 4>::KT;
  return f32 ? Cfg<float, 1>::KT : Cfg<__nv_bfloat16, 1>::KT;
}

Plan make_plan(const wenc_prefix_attention_args* a, int sms) {
  Plan pl;
  const bool f32 = a->dtype == WENC_DTYPE_F32;
  const long long r = a->n_heads / a->n_kv_heads;
  const long long rows_s = a->q_len * r;  // rows of one sequence per key head
  const long long group = a->k_prefix ? a->max_group : 1, n_groups = a->k_prefix ? a->n_groups : a->n_seqs;
  const long long rows = group * rows_s;
  const long long own_cap = a->k_pages ? static_cast<long long>(a->max_pages) * a->page_size : 0;
  const long long prefix = a->k_prefix ? a->prefix_max : 0;
  if (rows <= 64) {
    pl.wr = rows <= 16 ? 1 : 4;
    const int kt = tile_keys(f32, pl.wr);
    const long long tiles = (prefix + kt - 1) / kt + group * ((own_cap + kt - 1) / kt);
    const long long items = n_groups * a->n_kv_heads;
    // enough CTAs for about three rounds of two per SM, none without a tile of its own
    pl.cluster = 1;
    while (pl.cluster < 8 && pl.cluster < tiles && items * pl.cluster < 6ll * sms) pl.cluster *= 2;
    pl.items_p = items * pl.cluster;
    return pl;
  }
  auto splits = [&](long long items, long long keys, int wr) {
    const long long tiles = (keys + tile_keys(f32, wr) - 1) / tile_keys(f32, wr);
    long long n = (6ll * sms + items - 1) / items;
    if (n > tiles) n = tiles;
    if (n > 32) n = 32;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  if (a->k_prefix) {
    pl.wr_p = 4;
    pl.rows_p = static_cast<int>((rows + 63) / 64);
    const long long items = n_groups * a->n_kv_heads * pl.rows_p;
    pl.np = splits(items, prefix, pl.wr_p);
    pl.items_p = items * pl.np;
  }
  if (a->k_pages) {
    pl.wr_s = rows_s <= 16 ? 1 : 4;
    pl.rows_s = static_cast<int>((rows_s + 16 * pl.wr_s - 1) / (16 * pl.wr_s));
    const long long items = static_cast<long long>(a->n_seqs) * a->n_kv_heads * pl.rows_s;
    pl.ns = splits(items, own_cap, pl.wr_s);
    pl.items_s = items * pl.ns;
  }
  const size_t n = static_cast<size_t>(a->n_seqs) * a->q_len * a->n_heads * (pl.np + pl.ns);
  pl.part_o = n * HD * sizeof(float);
  pl.bytes = pl.part_o + n * sizeof(float2);
  return pl;
}

// Sizes alone (what the plan needs). Returns false with the status set.
bool check_sizes(const wenc_prefix_attention_args* a, wenc_status* st) {
  auto no = [&](wenc_status s, const char* fmt, long long x = 0, long long y = 0) {
    *st = bad(s, fmt, x, y);
    return false;
  };
  if (!a) return no(WENC_ERR_INVALID_ARG, "prefix_attention: args is NULL");
  if (a->dtype != WENC_DTYPE_F32 && a->dtype != WENC_DTYPE_BF16)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: dtype %lld unknown", a->dtype);
  if (a->head_dim != HD) return no(WENC_ERR_UNSUPPORTED, "head_dim %lld: only 64 is implemented", a->head_dim);
  if (a->n_seqs < 1 || a->q_len < 1 || a->n_heads < 1 || a->n_kv_heads < 1)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_seqs, q_len and the heads must be >= 1");
  if (a->n_heads % a->n_kv_heads != 0)
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: %lld query heads are no multiple of %lld key heads", a->n_heads,
              a->n_kv_heads);
  if (static_cast<long long>(a->n_seqs) * a->q_len > (1ll << 28) || a->n_heads > 4096)
    return no(WENC_ERR_UNSUPPORTED, "prefix_attention: more than 2^28 tokens or 4096 heads");
  if (!a->k_prefix && !a->k_pages) return no(WENC_ERR_INVALID_ARG, "prefix_attention: neither prefix nor pages");
  if ((a->k_prefix == nullptr) != (a->v_prefix == nullptr) || (a->k_pages == nullptr) != (a->v_pages == nullptr))
    return no(WENC_ERR_INVALID_ARG, "prefix_attention: keys and values come together");
  if (a->k_prefix) {
    if (a->n_groups < 1 || a->max_group < 1 || a->prefix_max < 1)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_groups, max_group and prefix_max must be >= 1");
    if (a->max_group > a->n_seqs)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: max_group %lld > n_seqs %lld", a->max_group, a->n_seqs);
    if (!a->group_start && static_cast<long long>(a->n_groups) * a->max_group != a->n_seqs)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_groups * max_group = %lld, but n_seqs = %lld (pass group_start)",
                static_cast<long long>(a->n_groups) * a->max_group, a->n_seqs);
    if (a->prefix_max > (1 << 30)) return no(WENC_ERR_UNSUPPORTED, "prefix_attention: prefix_max %lld > 2^30", a->prefix_max);
  }
  if (a->k_pages) {
    if (a->n_pages < 1 || a->page_size < 1 || a->max_pages < 1)
      return no(WENC_ERR_INVALID_ARG, "prefix_attention: n_pages, page_size and max_pages must be >= 1");
    if (static_cast<long long>(a->max_pages) * a->page_size > (1ll << 30))
      return no(WENC_ERR_UNSUPPORTED, "prefix_attention: max_pages %lld x page_size %lld passes 2^30", a->max_pages,
                a->page_size);
  }
  return true;
}

// Shared-memory opt-in, once per device and kernel (a repeat by a racing host thread is harmless).
template <typename K>
cudaError_t opt_in(K kern, uint32_t smem, std::atomic<int>& configured_device) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device.load(std::memory_order_acquire) != dev) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured_device.store(dev, std::memory_order_release);
  }
  return cudaSuccess;
}

template <typename T, int WR>
cudaError_t launch_cluster(const PrefixParams& p, long long blocks, uint32_t* err, cudaStream_t stream) {
  auto kern = prefix_cluster_kernel<T, WR>;
  static std::atomic<int> configured{-1};
  const cudaError_t e = opt_in(kern, Cfg<T, WR>::SMEM, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<T, WR>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, err);
}

template <typename T, int WR, bool OWN>
cudaError_t launch_part(PrefixParams p, int row_tiles, long long blocks, uint32_t* err, cudaStream_t stream) {
  auto kern = prefix_part_kernel<T, WR, OWN>;
  static std::atomic<int> configured{-1};
  const cudaError_t e = opt_in(kern, Cfg<T, WR>::SMEM, configured);
  if (e != cudaSuccess) return e;
  p.row_tiles = row_tiles;
  return wenc_host::launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), Cfg<T, WR>::SMEM, stream, p, err);
}

template <typename T>
cudaError_t launch_all(const PrefixParams& p, const Plan& pl, uint32_t* err, cudaStream_t stream) {
  if (pl.cluster > 0)
    return pl.wr == 1 ? launch_cluster<T, 1>(p, pl.items_p, err, stream) : launch_cluster<T, 4>(p, pl.items_p, err, stream);
  cudaError_t e = cudaSuccess;
  if (pl.items_p > 0) e = launch_part<T, 4, false>(p, pl.rows_p, pl.items_p, err, stream);
  if (e == cudaSuccess && pl.items_s > 0)
    e = pl.wr_s == 1 ? launch_part<T, 1, true>(p, pl.rows_s, pl.items_s, err, stream)
                     : launch_part<T, 4, true>(p, pl.rows_s, pl.items_s, err, stream);
  if (e != cudaSuccess) return e;
  const long long threads = static_cast<long long>(p.n_seqs) * p.q_len * p.H * 16;
  return wenc_host::launch_pdl(prefix_join_kernel<T>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0,
                               stream, p);
}

}  // namespace

extern "C" size_t wenc_prefix_attention_workspace(const wenc_prefix_attention_args* a) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st)) return 0;
  return make_plan(a, wenc_internal_sm_count()).bytes;
}

extern "C" wenc_status wenc_prefix_attention(const wenc_prefix_attention_args* a, wenc_stream_t stream) {
  wenc_internal_clear_error();
  wenc_status st;
  if (!check_sizes(a, &st)) return st;
  if (!a->q || !a->out) return bad(WENC_ERR_INVALID_ARG, "prefix_attention: q or out is NULL");
  if (a->k_pages && (!a->block_table || !a->lens))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: pages need block_table and lens");
  const long long es = a->dtype == WENC_DTYPE_F32 ? 4 : 2, per16 = 16 / es;
  const long long q_row = static_cast<long long>(a->n_heads) * HD, kv_row = static_cast<long long>(a->n_kv_heads) * HD;
  if (a->q_stride < q_row || a->out_stride < q_row)
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a token stride of q or out is smaller than its heads");
  if (a->k_prefix && (a->k_token_stride < kv_row || a->v_token_stride < kv_row || a->k_group_stride < 0 || a->v_group_stride < 0))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a prefix stride is smaller than its heads");
  if (a->k_pages && (a->k_page_stride < kv_row * a->page_size || a->v_page_stride < kv_row * a->page_size))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: a page stride is smaller than a page");
  if (a->k_pages && a->n_seqs > 1 && a->block_table_stride < a->max_pages)
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: block_table_stride %lld < max_pages %lld", a->block_table_stride,
               a->max_pages);
  const void* ptrs[] = {a->q, a->out, a->k_prefix, a->v_prefix, a->k_pages, a->v_pages};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return bad(WENC_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  const long long zero = 0;
  const long long strides[] = {a->q_stride, a->out_stride,
                               a->k_prefix ? a->k_group_stride : zero, a->k_prefix ? a->k_token_stride : zero,
                               a->k_prefix ? a->v_group_stride : zero, a->k_prefix ? a->v_token_stride : zero,
                               a->k_pages ? a->k_page_stride : zero, a->k_pages ? a->v_page_stride : zero};
  for (long long x : strides)
    if (x % per16 != 0) return bad(WENC_ERR_INVALID_ARG, "strides must be multiples of 16 bytes");
  std::string why;
  if (!wenc_internal_is_sm103(&why)) return wenc_internal_fail(WENC_ERR_UNSUPPORTED, why.c_str());
  uint32_t* err = wenc_internal_error_word(&why);
  if (!err) return wenc_internal_fail(WENC_ERR_CUDA, why.c_str());
  const Plan pl = make_plan(a, wenc_internal_sm_count());
  if (pl.items_p > 0x7fffffffll || pl.items_s > 0x7fffffffll)
    return bad(WENC_ERR_UNSUPPORTED, "prefix_attention: %lld work items pass 2^31 - 1", pl.items_p > pl.items_s ? pl.items_p : pl.items_s);
  if (pl.bytes > 0 && (!a->workspace || a->workspace_bytes < pl.bytes))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: workspace of %lld bytes needed, %lld given", static_cast<long long>(pl.bytes),
               a->workspace ? static_cast<long long>(a->workspace_bytes) : 0ll);
  if (pl.bytes > 0 && (reinterpret_cast<uintptr_t>(a->workspace) & 255u))
    return bad(WENC_ERR_INVALID_ARG, "prefix_attention: the workspace must be 256-byte aligned");

  PrefixParams p = {};
  p.q = static_cast<const uint8_t*>(a->q);
  p.out = static_cast<uint8_t*>(a->out);
  p.q_stride = a->q_stride * es;
  p.out_stride = a->out_stride * es;
  p.n_seqs = a->n_seqs;
  p.q_len = a->q_len;
  p.H = a->n_heads;
  p.Hkv = a->n_kv_heads;
  p.r = a->n_heads / a->n_kv_heads;
  if (a->k_prefix) {
    p.kp = static_cast<const uint8_t*>(a->k_prefix);
    p.vp = static_cast<const uint8_t*>(a->v_prefix);
    p.k_group = a->k_group_stride * es;
    p.k_token = a->k_token_stride * es;
    p.v_group = a->v_group_stride * es;
    p.v_token = a->v_token_stride * es;
    p.group_start = a->group_start;
    p.prefix_lens = a->prefix_lens;
    p.n_groups = a->n_groups;
    p.max_group = a->max_group;
    p.prefix_max = a->prefix_max;
  }
  if (a->k_pages) {
    p.k_pages = static_cast<const uint8_t*>(a->k_pages);
    p.v_pages = static_cast<const uint8_t*>(a->v_pages);
    p.k_page = a->k_page_stride * es;
    p.v_page = a->v_page_stride * es;
    p.page_row = kv_row * es;
    p.table = a->block_table;
    p.table_stride = a->block_table_stride;
    p.lens = a->lens;
    p.n_pages = a->n_pages;
    p.page_size = a->page_size;
    p.max_pages = a->max_pages;
    p.page_shift = -1;
    for (int s = 0; s < 31; ++s)
      if (a->page_size == 1 << s) p.page_shift = s;
  }
  if (!a->k_prefix) {  // every sequence a group of its own
    p.n_groups = a->n_seqs;
    p.max_group = 1;
  }
  p.np = pl.np;
  p.ns = pl.ns;
  p.cluster = pl.cluster;
  // |scale| and the queries' signs; a scale of 0 is 1 on queries of 0
  const bool bf = a->dtype == WENC_DTYPE_BF16;
  p.q_flip = a->scale < 0.0f ? (bf ? 0x80008000u : 0x80000000u) : 0u;
  p.q_keep = a->scale == 0.0f ? 0u : 0xffffffffu;
  p.scale_log2 = (a->scale == 0.0f ? 1.0f : a->scale < 0.0f ? -a->scale : a->scale) * 1.4426950408889634f;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(a->workspace) + pl.part_o);
  const cudaError_t e = a->dtype == WENC_DTYPE_F32
                            ? launch_all<float>(p, pl, err, reinterpret_cast<cudaStream_t>(stream))
                            : launch_all<__nv_bfloat16>(p, pl, err, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    char buf[200];
    snprintf(buf, sizeof(buf), "prefix_attention launch: %s", cudaGetErrorString(e));
    return wenc_internal_fail(WENC_ERR_CUDA, buf);
  }
  return WENC_OK;
}
