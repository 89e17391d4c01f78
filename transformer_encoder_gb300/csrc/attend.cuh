// attend.cuh -- a warp's steps of 16 keys against a few query rows, shared by the attention of decode steps (prefix_attn.cu)
// and of chunks (chunk_attn.cu): scores, running softmax, weighted values, and the join of a CTA's warps.
//
// The products are transposed: S^T = K Q^T and O^T = V^T P^T, with 16 keys (or 16 elements of V) as the MMA's M and 8 query
// rows as its N, so that few rows cost eight columns instead of sixteen rows, and the fragments of K and V are loaded once for
// any number of rows.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "mma.cuh"
#include "ptx.cuh"

namespace wenc_dev {

// NR groups of 8 query rows per CTA.
template <typename T, int NR>
struct Cfg {
  static constexpr int HD = 64;                // head width
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int NW = F32 ? 4 : 8;       // warps
  static constexpr int THREADS = 32 * NW;
  static constexpr int KW = 16;                // keys per step of a warp
  static constexpr int ROWS = 8 * NR;
  static constexpr int ROWB = HD * sizeof(T);
  static constexpr int STAGES = 2;
  static constexpr int CTAS = NR == 1 ? 3 : 2;  // per SM, for the registers
  static constexpr uint32_t HALF = KW * ROWB;  // bytes of K (or V) per warp and stage
  static constexpr uint32_t RING = NW * STAGES * 2 * HALF;
  static constexpr uint32_t P_BYTES = F32 ? NW * NR * 16 * 8 * 4 : 0;  // fp32: P on its way to B fragments
  // results over the ring: O [NW][ROWS][OS] floats, (m, l) [NW][ROWS]
  static constexpr int OS = HD + 4;
  static constexpr uint32_t ML = NW * ROWS * OS * 4;
  static constexpr uint32_t RESULTS = ML + NW * ROWS * 8;
  static constexpr uint32_t SMEM = (RING + P_BYTES > RESULTS ? RING + P_BYTES : RESULTS);
};

// 16-byte granule `c` of key row `row` within a warp's stage. bf16 rows have 8 granules (all 32 banks),
// fp32 rows 16; the XOR spreads the rows that an ldmatrix (or a quarter of a fragment load) touches at
// once over all banks.
template <bool F32>
__device__ __forceinline__ uint32_t granule(int row, int c) {
  if constexpr (F32)
    return row * 256u + ((c ^ (((row & 1) << 2) | (row & 2))) << 4);
  else
    return row * 128u + ((c ^ (row & 7)) << 4);
}

// The state of a warp's rows: this thread's columns of O^T and S^T are rows 8 r + 2 (lane % 4) + e.
template <int NR>
struct RowState {
  float o[NR][4][4], m[NR][2], l[NR][2];  // m in log2 units; l of this thread's keys alone until reduced
};

// A query row's share of the B fragments of S^T's product (column g of a group of 8 rows); row == NULL: zeros. The sign of every
// element turns with `flip`, and all are cleared where `keep` is 0.
template <typename T, int KS>
__device__ __forceinline__ void load_query(const uint8_t* row, int tq, uint32_t keep, uint32_t flip, uint32_t (&qh)[KS][2],
                                           uint32_t (&ql)[KS][2]) {
  if constexpr (sizeof(T) == 4) {
    // k index tq (and tq + 4) of step 2j (and 2j + 1) stands for element 4 (tq + 4j) + 0, 1 (2, 3)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 a = row ? *reinterpret_cast<const uint4*>(row + (tq + 4 * j) * 16) : make_uint4(0u, 0u, 0u, 0u);
      auto part = [&](uint32_t v, uint32_t& hi, uint32_t& lo) { split_tf32(__uint_as_float((v & keep) ^ flip), hi, lo); };
      part(a.x, qh[2 * j][0], ql[2 * j][0]);
      part(a.y, qh[2 * j][1], ql[2 * j][1]);
      part(a.z, qh[2 * j + 1][0], ql[2 * j + 1][0]);
      part(a.w, qh[2 * j + 1][1], ql[2 * j + 1][1]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        qh[k][h] = row ? (*reinterpret_cast<const uint32_t*>(row + (16 * k + 8 * h + 2 * tq) * 2) & keep) ^ flip : 0u;
  }
}

// No keys yet; u is the reference in use: m, or 0 while that is -inf.
template <int NR>
__device__ __forceinline__ void clear_rows(RowState<NR>& st, float (&u)[NR][2]) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[r][i][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      st.m[r][e] = -CUDART_INF_F;
      u[r][e] = st.l[r][e] = 0.0f;
    }
  }
}

// S^T of a stage's 16 keys (at sk) and the warp's rows. Element e: key g + 8 (e / 2), row column e % 2.
template <typename T, int NR, int KS, int QL>
__device__ __forceinline__ void step_scores(uint32_t sk, const uint32_t (&qh)[NR][KS][2], const uint32_t (&ql)[QL][KS][2],
                                            float (&s)[NR][4]) {
  constexpr bool F32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[r][e] = 0.0f;
  if constexpr (F32) {
    // the products with a small part are summed apart: the tensor core's sums truncate, and these are 2^-11 as large
    float small[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) small[r][e] = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 ka = lds_f4(sk + granule<true>(g, tq + 4 * c)), kb = lds_f4(sk + granule<true>(g + 8, tq + 4 * c));
      uint32_t h[2][4], w[2][4];
      split_tf32(ka.x, h[0][0], w[0][0]);
      split_tf32(kb.x, h[0][1], w[0][1]);
      split_tf32(ka.y, h[0][2], w[0][2]);
      split_tf32(kb.y, h[0][3], w[0][3]);
      split_tf32(ka.z, h[1][0], w[1][0]);
      split_tf32(kb.z, h[1][1], w[1][1]);
      split_tf32(ka.w, h[1][2], w[1][2]);
      split_tf32(kb.w, h[1][3], w[1][3]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          mma_tf32(small[r], h[i], ql[r][2 * c + i][0], ql[r][2 * c + i][1]);
          mma_tf32(small[r], w[i], qh[r][2 * c + i][0], qh[r][2 * c + i][1]);
          mma_tf32(s[r], h[i], qh[r][2 * c + i][0], qh[r][2 * c + i][1]);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][e] += small[r][e];
  } else {
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm_x4(a, sk + granule<false>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
      for (int r = 0; r < NR; ++r) mma_bf16(s[r], a, qh[r][k][0], qh[r][k][1]);
    }
  }
}

// The running softmax and O^T += V^T P^T over a stage's 16 values (at sv), from scores that are -inf where a row does not
// see the key. sp: the warp's shared memory for P (fp32).
template <typename T, int NR>
__device__ __forceinline__ void step_values(float (&s)[NR][4], float sc, uint32_t sv, uint32_t sp, RowState<NR>& st, float (&u)[NR][2]) {
  constexpr bool F32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  auto &o = st.o;
  auto &m = st.m, &l = st.l;
  bool move = false;  // some score exceeds its row's reference by more than 2^8
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) move |= fmaxf(s[r][e], s[r][e + 2]) * sc > m[r][e] + 8.0f;
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[r][e], s[r][e + 2]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        x = fmaxf(x * sc, m[r][e]);
        const float ref = x == -CUDART_INF_F ? 0.0f : x;
        const float f = ex2_approx(m[r][e] - ref);
        m[r][e] = x;
        u[r][e] = ref;
        l[r][e] *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[r][i][e] *= f;
          o[r][i][e + 2] *= f;
        }
      }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[r][e] = ex2_approx(fmaf(s[r][e], sc, -u[r][e & 1]));
      l[r][e & 1] += s[r][e];
    }
  // ---- O^T += V^T P^T
  if constexpr (F32) {
    // P through shared memory: written as [key][row], read as B fragments (key tq, row g). The tile's
    // product is formed on its own and added in one rounding, so that the tensor core's accumulation
    // (which truncates) runs over one tile only.
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sp + r * 512 + (g * 8 + 2 * tq) * 4), "f"(s[r][0]), "f"(s[r][1]) : "memory");
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sp + r * 512 + ((g + 8) * 8 + 2 * tq) * 4), "f"(s[r][2]), "f"(s[r][3]) : "memory");
    }
    __syncwarp();
    uint32_t ph[NR][2][2], pl[NR][2][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(sp + r * 512 + ((8 * k + 4 * h + tq) * 8 + g) * 4) : "memory");
          split_tf32(x, ph[r][k][h], pl[r][k][h]);
        }
    __syncwarp();
    // row g (g + 8) of product i stands for element 4 g + i (32 + 4 g + i)
    float t[NR][4][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[r][i][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 v0 = lds_f4(sv + granule<true>(8 * k + tq, g)), v1 = lds_f4(sv + granule<true>(8 * k + tq, g + 8));
      const float4 v2 = lds_f4(sv + granule<true>(8 * k + tq + 4, g)), v3 = lds_f4(sv + granule<true>(8 * k + tq + 4, g + 8));
      const float w[4][4] = {{v0.x, v1.x, v2.x, v3.x}, {v0.y, v1.y, v2.y, v3.y}, {v0.z, v1.z, v2.z, v3.z}, {v0.w, v1.w, v2.w, v3.w}};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t vh[4], vl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_tf32(w[i][e], vh[e], vl[e]);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          mma_tf32(t[r][i], vh, pl[r][k][0], pl[r][k][1]);
          mma_tf32(t[r][i], vl, ph[r][k][0], ph[r][k][1]);
          mma_tf32(t[r][i], vh, ph[r][k][0], ph[r][k][1]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] += t[r][i][e];
  } else {
    uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = s[r][2 * h], y = s[r][2 * h + 1];
        const uint32_t hi = pack_bf16x2(x, y);
        const uint32_t lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
        ph[r][h] = movm_t(hi);
        pl[r][h] = movm_t(lo);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 16 elements of V at a time
      uint32_t a[4];
      ldsm_x4_t(a, sv + granule<false>((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        mma_bf16(o[r][i], a, ph[r][0], ph[r][1]);
        mma_bf16(o[r][i], a, pl[r][0], pl[r][1]);
      }
    }
  }
}

// A row's sum over the lanes that hold its keys.
template <int NR>
__device__ __forceinline__ void sum_rows(RowState<NR>& st) {
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      st.l[r][e] += __shfl_xor_sync(0xffffffffu, st.l[r][e], 4);
      st.l[r][e] += __shfl_xor_sync(0xffffffffu, st.l[r][e], 8);
      st.l[r][e] += __shfl_xor_sync(0xffffffffu, st.l[r][e], 16);
    }
}

// All warps' results into shared memory, over the rings; begins and ends with a barrier.
template <typename T, int NR>
__device__ __forceinline__ void share_results(uint8_t* smem, const RowState<NR>& st) {
  using C = Cfg<T, NR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem) + warp * C::ROWS * C::OS;
  float2* sml = reinterpret_cast<float2*>(smem + C::ML) + warp * C::ROWS;
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = 8 * r + 2 * tq + e;
      if (g == 0) sml[x] = make_float2(st.m[r][e], st.l[r][e]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        so[x * C::OS + (C::F32 ? 4 * g + i : 16 * i + g)] = st.o[r][i][e];
        so[x * C::OS + (C::F32 ? 32 + 4 * g + i : 16 * i + g + 8)] = st.o[r][i][e + 2];
      }
    }
  __syncthreads();
}

// Join of the warps' results for row x of the tile, elements c8 .. c8 + 7.
template <typename T, int NR>
__device__ __forceinline__ void join_warps(const uint8_t* smem, int x, int c8, float (&v)[8], float& m, float& l) {
  using C = Cfg<T, NR>;
  const float* so = reinterpret_cast<const float*>(smem);
  const float2* sml = reinterpret_cast<const float2*>(smem + C::ML);
  m = -CUDART_INF_F;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) m = fmaxf(m, sml[w * C::ROWS + x].x);
  const float u = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) {
    const float2 ml = sml[w * C::ROWS + x];
    const float f = ex2_approx(ml.x - u);
    l += f * ml.y;
    const float4* o = reinterpret_cast<const float4*>(so + (w * C::ROWS + x) * C::OS + c8);
    const float4 a = o[0], b = o[1];
    v[0] += f * a.x; v[1] += f * a.y; v[2] += f * a.z; v[3] += f * a.w;
    v[4] += f * b.x; v[5] += f * b.y; v[6] += f * b.z; v[7] += f * b.w;
  }
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

}  // namespace wenc_dev
