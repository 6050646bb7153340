// paged.cuh -- kernels of the paged KV cache: head norms with the rotation,
// the cache's write and read-back, and decode attention over it.
#pragma once

#include "common.cuh"
#include "ntx.h"

namespace ntx {

enum : int { kKvF16 = NTX_F16, kKvQ4 = NTX_Q4_0, kKvQ8 = NTX_Q8_0 };

// Bytes of one row's codes, and of one (page, head)'s codes and scales.
template <int T>
__host__ __device__ constexpr int kv_code_bytes(int D) {
  return T == kKvF16 ? 2 * D : T == kKvQ8 ? D : D / 2;
}
template <int T>
__host__ __device__ constexpr int kv_row_bytes(int D) {
  return kv_code_bytes<T>(D) + (T == kKvF16 ? 0 : D / 16);
}

__device__ __forceinline__ void bad_page(int* status) { atomicExch(status, (int)kStatusBadPage); }

// Where (sequence, position) lies: the first byte of the page's part of head 0
// and the row inside the page; false (status 5) if the cache has no such place.
__device__ __forceinline__ bool kv_place(const ntx_paged_kv& c, int seq, int pos, int64_t* page, int* row,
                                         int* status) {
  const int j = pos / c.page_size;
  if (seq < 0 || seq >= c.n_seqs || j >= c.max_pages) {
    bad_page(status);
    return false;
  }
  const int p = __ldg(c.page_table + (int64_t)seq * c.max_pages + j);
  if (p < 0 || p >= c.n_pages) {
    bad_page(status);
    return false;
  }
  *page = p;
  *row = pos - j * c.page_size;
  return true;
}

// x rounded half away from zero, |x| < 2^22.
__device__ __forceinline__ int round_away(float x) {
  const float a = fabsf(x), f = floorf(a);
  const int t = (int)f + (a - f >= 0.5f ? 1 : 0);  // a - f is exact
  return x < 0.f ? -t : t;
}

// ------------------------------------------------------------- cache write
// Eight lanes hold one block of 32, four consecutive elements each.
template <int T>
__global__ void __launch_bounds__(256) kv_append_kernel(const ntx_paged_kv c, const float* __restrict__ k,
                                                        const float* __restrict__ v, int64_t ks, int64_t vs,
                                                        const int* __restrict__ seq_ids,
                                                        const int* __restrict__ positions, int n_tokens, bool vec,
                                                        int* status) {
  const int D = c.head_dim, nb = D >> 5, row_blocks = c.n_kv_heads * nb;
  const int sub = threadIdx.x & 7;
  const float* src = blockIdx.y ? v : k;
  const int64_t stride = blockIdx.y ? vs : ks;
  uint8_t* pool = static_cast<uint8_t*>(blockIdx.y ? c.v_pages : c.k_pages);
  const int64_t head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D);
  for (int n = blockIdx.x; n < n_tokens; n += gridDim.x) {
    const int pos = __ldg(positions + n);
    if (pos < 0) continue;
    int64_t page;
    int row;
    if (!kv_place(c, seq_ids ? __ldg(seq_ids + n) : n, pos, &page, &row, status)) continue;
    const float* in = src + n * stride;
    for (int b0 = 0; b0 < row_blocks; b0 += 32) {  // the 32 blocks of the CTA's 256 threads
      const int b = b0 + (threadIdx.x >> 3);
      const bool on = b < row_blocks;
      float w[4] = {0.f, 0.f, 0.f, 0.f};
      if (on) {
        const float* p = in + b * 32 + sub * 4;
        if (vec) {
          const float4 t = *reinterpret_cast<const float4*>(p);
          w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = p[i];
        }
      }
      const int head = b / nb, blk = b - head * nb;
      uint8_t* part = pool + (page * c.n_kv_heads + head) * head_bytes;
      if constexpr (T == kKvF16) {
        if (on) {
          uint2 h;
          h.x = float_to_half_bits(w[0]) | ((uint32_t)float_to_half_bits(w[1]) << 16);
          h.y = float_to_half_bits(w[2]) | ((uint32_t)float_to_half_bits(w[3]) << 16);
          *reinterpret_cast<uint2*>(part + ((int64_t)row * D + blk * 32 + sub * 4) * 2) = h;
        }
      } else {
        // |w| as ordered bits: the largest, and whether any is not finite
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(w[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool finite = top < 0x7F800000u;
        float d;
        if constexpr (T == kKvQ8) {
          d = __uint_as_float(top) / 127.0f;
        } else {
          // the first element of the largest magnitude decides the sign
          int key = 64;
#pragma unroll
          for (int i = 3; i >= 0; --i)
            if ((__float_as_uint(w[i]) & 0x7FFFFFFFu) == top) key = 2 * (4 * sub + i) + (w[i] < 0.f ? 1 : 0);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) key = min(key, __shfl_xor_sync(0xffffffffu, key, o));
          const float m = (key & 1) ? -__uint_as_float(top) : __uint_as_float(top);
          d = m * -0.125f;
        }
        const bool zero = top == 0 || !finite;
        int q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = zero ? 0 : round_away(w[i] / d);
          q[i] = T == kKvQ8 ? min(127, max(-127, r)) : min(15, max(0, r + 8));
        }
        const uint32_t codes = (q[0] & 255) | ((q[1] & 255) << 8) | ((q[2] & 255) << 16) | ((uint32_t)(q[3] & 255) << 24);
        if constexpr (T == kKvQ8) {
          if (on) *reinterpret_cast<uint32_t*>(part + (int64_t)row * D + blk * 32 + sub * 4) = codes;
        } else {
          const uint32_t hi = __shfl_down_sync(0xffffffffu, codes, 4, 8);  // elements 16 further on
          if (on && sub < 4)
            *reinterpret_cast<uint32_t*>(part + (int64_t)row * (D / 2) + blk * 16 + sub * 4) = codes | (hi << 4);
        }
        if (on && sub == 0)
          *reinterpret_cast<uint16_t*>(part + (int64_t)c.page_size * kv_code_bytes<T>(D) + ((int64_t)row * nb + blk) * 2) =
              finite ? float_to_half_bits(d) : (uint16_t)0x7FFF;
      }
    }
  }
}

// ------------------------------------------------------------- cache read
template <int T>
__device__ __forceinline__ float kv_element(const uint8_t* part, int page_size, int D, int row, int e) {
  if constexpr (T == kKvF16) {
    return half_bits_to_float(*reinterpret_cast<const uint16_t*>(part + ((int64_t)row * D + e) * 2));
  } else {
    const float d = half_bits_to_float(*reinterpret_cast<const uint16_t*>(
        part + (int64_t)page_size * kv_code_bytes<T>(D) + ((int64_t)row * (D >> 5) + (e >> 5)) * 2));
    if constexpr (T == kKvQ8) return d * (float)(int8_t)part[(int64_t)row * D + e];
    const int byte = part[(int64_t)row * (D / 2) + (e >> 5) * 16 + (e & 15)];
    return d * (float)(((e & 16) ? byte >> 4 : byte & 15) - 8);
  }
}

template <int T>
__global__ void __launch_bounds__(256) kv_read_kernel(const ntx_paged_kv c, float* __restrict__ k,
                                                      float* __restrict__ v, int64_t ks, int64_t vs,
                                                      const int* __restrict__ seq_ids,
                                                      const int* __restrict__ positions, int n_tokens, int* status) {
  const int D = c.head_dim;
  float* dst = blockIdx.y ? v : k;
  if (!dst) return;
  const int64_t stride = blockIdx.y ? vs : ks;
  const uint8_t* pool = static_cast<const uint8_t*>(blockIdx.y ? c.v_pages : c.k_pages);
  const int64_t head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D);
  for (int n = blockIdx.x; n < n_tokens; n += gridDim.x) {
    const int pos = __ldg(positions + n);
    if (pos < 0) continue;
    int64_t page;
    int row;
    if (!kv_place(c, seq_ids ? __ldg(seq_ids + n) : n, pos, &page, &row, status)) continue;
    for (int e = threadIdx.x; e < c.n_kv_heads * D; e += blockDim.x) {
      const int head = e / D;
      dst[n * stride + e] =
          kv_element<T>(pool + (page * c.n_kv_heads + head) * head_bytes, c.page_size, D, row, e - head * D);
    }
  }
}

// ------------------------------------------------------------- head norm + rotation
// One warp per (token, head).
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const float* q, const float* k, float* q_out, float* k_out,
                                                           int64_t qs, int64_t ks, const float* __restrict__ wq,
                                                           const float* __restrict__ wk,
                                                           const int* __restrict__ positions, int n_tokens, int Hq,
                                                           int Hkv, int D, int R, int halves, float theta, float eps) {
  __shared__ float rows[8][256];
  const int lane = threadIdx.x & 31, heads = Hq + Hkv;
  float* x = rows[threadIdx.x >> 5];
  const int64_t total = (int64_t)n_tokens * heads;
  for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < total; i += gridDim.x * 8ll) {
    const int n = (int)(i / heads), h = (int)(i - (int64_t)n * heads);
    const int pos = __ldg(positions + n);
    if (pos < 0) continue;
    const bool is_q = h < Hq;
    const int64_t at = is_q ? n * qs + (int64_t)h * D : n * ks + (int64_t)(h - Hq) * D;
    const float* in = (is_q ? q : k) + at;
    float* out = (is_q ? q_out : k_out) + at;
    const float* w = is_q ? wq : wk;
    float ss = 0.f;
    for (int e = lane; e < D; e += 32) {
      const float t = in[e];
      x[e] = t;
      ss = fmaf(t, t, ss);
    }
    const float r = 1.0f / sqrtf(warp_sum(ss) / (float)D + eps);
    __syncwarp();
    for (int e = lane; e < D; e += 32) x[e] = (x[e] * r) * (w ? __ldg(w + e) : 1.f);
    __syncwarp();
    for (int p = lane; p < R / 2; p += 32) {
      const int e0 = halves ? p : 2 * p, e1 = halves ? p + R / 2 : 2 * p + 1;
      double s, c;
      sincos((double)pos * pow((double)theta, -2.0 * p / R), &s, &c);
      const float a = x[e0], b = x[e1];
      out[e0] = a * (float)c - b * (float)s;
      out[e1] = a * (float)s + b * (float)c;
    }
    for (int e = R + lane; e < D; e += 32) out[e] = x[e];
    __syncwarp();
  }
}

// ------------------------------------------------------------- attention
//
//   out[s][h] = sum_p softmax_p(scale q.k_p) v_p       (p < len[s])
//
// A warp works on items (sequence, KV head, tile of up to 8 of its query heads)
// in chunks of CH positions, with m16n8k16 fp16 matrix instructions and one pass
// over the data: running maximum m (base 2), sum l and output o of a softmax.
//
// fp32 accuracy from fp16 products: a tile has at most 8 query heads, so the
// lower 8 of the instruction's 16 rows are free.  Row g holds the upper 11 bits
// of head g's operand, row g + 8 the rounded remainder; both land in the same
// thread's accumulators (c0, c1 and c2, c3) and are added there: 22 bits of q
// and p at no extra instruction.  Keys and values are exact in fp16: F16 as
// they are, the codes of block types as integers.  A key block's scale
// multiplies its partial score in fp32; a value block's scale multiplies p
// before p is split.  q is first scaled by a power of two that puts its largest
// element in [2^13, 2^14), p times the scales likewise for each chunk, so
// neither overflows fp16 and the remainders lose nothing to its subnormals.
// The matrix instruction's fp32 accumulation truncates, so it only sums one
// block (keys) or one chunk (values); longer sums are ordinary fp32 adds.
//
// Work: the chunks of all items in a row, cut into equal parts, one per warp of
// a grid that fills the GPU, whatever the lengths.  A part that holds a whole
// item writes its output; the others leave (m, l, o) for attn_paged_join_kernel.
// Warps share nothing: each streams K and V chunks through its own ring of
// shared-memory slots with 16-byte asynchronous copies, across items, without a
// barrier.  The order of every sum is fixed by lengths and grid.

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Four 8x8 matrices of 16-bit elements, transposed: lane l gives the address of
// row l % 8 of matrix l / 8 and receives elements (2 (l%4), l/4), (2 (l%4) + 1, l/4).
__device__ __forceinline__ void ldsm4_trans(uint32_t a, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// (x, y) as fp16 pairs: the nearest halves, and the halves nearest to what they leave.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// Four bytes u = q + 128 (after the sign flip) as pairs of exact fp16 integers q.
template <int SEL>
__device__ __forceinline__ uint32_t bytes_h2(uint32_t flipped) {
  const uint32_t h = __byte_perm(flipped, 0x64646464u, SEL);  // 1024 + u
  return h2_bits(__hsub2(bits_h2(h), bits_h2(0x64806480u)));  // - 1152
}
// The low / high nibbles of bytes 0 and 2 as fp16 integers q - 8.
__device__ __forceinline__ uint32_t nib_lo(uint32_t x) {
  return h2_bits(__hsub2(bits_h2((x & 0x000F000Fu) | 0x64006400u), bits_h2(0x64086408u)));  // 1024 + q - 1032
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t x) {
  return h2_bits(__hfma2(bits_h2((x & 0x00F000F0u) | 0x64006400u), bits_h2(0x2C002C00u),
                         bits_h2(0xD480D480u)));  // (1024 + 16 q) / 16 - 72
}

// Positions per chunk, ring slots (one K or V chunk each) and warps.  Eight warps
// per SM carry three 8 KiB slots each of F16; block types are smaller and spend
// more instructions per byte, so they take sixteen warps where 128 registers do.
template <int T, int D>
struct PagedCfg {
  static constexpr int CH = (T == kKvF16 && D == 256) ? 16 : 32;
  static constexpr int SLOTS = (T == kKvF16 || (T == kKvQ8 && D >= 128)) ? 3 : 4;
  static constexpr int CTAS = (D == 256 || (T == kKvF16 && D == 128)) ? 2 : 4;
  static constexpr int WARPS = 4;
  static constexpr int CB = kv_code_bytes<T>(D);          // bytes of a row's codes
  static constexpr int SB = T == kKvF16 ? 0 : D / 16;      // bytes of a row's scales
  static constexpr int SLOT = CH * (CB + SB);
  static constexpr int SMEM = WARPS * SLOTS * SLOT;
};
__host__ __device__ constexpr int paged_part_floats(int rows, int D) { return rows * D + 2 * 8; }

// Position of 16-byte column `col` of a slot row, so that eight consecutive rows
// of one column lie in different banks.
template <int C>
__device__ __forceinline__ int swz8(int row, int col) {
  return C >= 8 ? col ^ (row & 7) : C == 4 ? col ^ ((row >> 1) & 3) : col ^ ((row >> 2) & 1);
}
// The same for a K read: each of a phase's rows is read over 64 (F16) or 32 (Q8_0)
// bytes at once.
template <int T, int C>
__device__ __forceinline__ int swz_k(int row, int col) {
  if constexpr (T == kKvF16) return col ^ ((row & 1) << 2);
  if constexpr (T == kKvQ8) return C >= 8 ? col ^ ((row & 3) << 1) : col ^ (((row >> 1) & 1) << 1);
  return swz8<C>(row, col);
}

__device__ __forceinline__ int seq_len(const ntx_paged_kv& c, const int* lens, int s, int* status) {
  const int n = __ldg(lens + s), most = c.max_pages * c.page_size;
  if (n >= 0 && n <= most) return n;
  bad_page(status);
  return n < 0 ? 0 : most;
}

// A place in the row of all chunks: chunk `ci` of `n` of tile `tile` of sequence `s`.
struct PagedCursor {
  int s, tile, ci, n, len;
  __device__ __forceinline__ void next(const ntx_paged_kv& c, const int* lens, int tiles, int ch, int* status) {
    if (++ci < n) return;
    ci = 0;
    if (++tile < tiles) return;
    tile = 0;
    do {
      if (++s >= c.n_seqs) { n = 0; return; }
      len = seq_len(c, lens, s, status);
      n = (len + ch - 1) / ch;
    } while (n == 0);
  }
};

// Chunks of all sequences before `upto` (all of them: upto >= n_seqs), one tile each.
// Lane i counts k consecutive sequences.
__device__ __forceinline__ int64_t lane_chunks(const ntx_paged_kv& c, const int* lens, int k, int ch, int upto,
                                               int* status) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int i = 0; i < k; ++i) {
    const int s = lane * k + i;
    if (s < c.n_seqs && s < upto) sum += (seq_len(c, lens, s, status) + ch - 1) / ch;
  }
  return sum;
}

template <int T, int D>
__global__ void __launch_bounds__(128, PagedCfg<T, D>::CTAS)
    attn_paged_kernel(const ntx_paged_kv c, const float* __restrict__ q, int64_t qs, float* __restrict__ out,
                      int4* __restrict__ splits, float* __restrict__ part, int Hq, const int* __restrict__ lens,
                      float scale, int* status) {
  using F = PagedCfg<T, D>;
  constexpr int CH = F::CH, C = F::CB / 16, NB = D / 32, NJ = CH / 8, NS = CH / 16, NT = D / 8;
  extern __shared__ __align__(128) uint8_t ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t slots = smem_addr(ring) + warp * (F::SLOTS * F::SLOT);
  const int G = Hq / c.n_kv_heads, rtiles = (G + 7) >> 3, tiles = c.n_kv_heads * rtiles;
  const int wid = warp * gridDim.x + blockIdx.x, all_warps = gridDim.x * F::WARPS;

  // empty sequences: zeros
  for (int s = wid; s < c.n_seqs; s += all_warps)
    if (__ldg(lens + s) <= 0)
      for (int64_t i = lane; i < (int64_t)Hq * D / 4; i += 32)
        reinterpret_cast<float4*>(out + (int64_t)s * Hq * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);

  // ---- this warp's part of the chunks, [c0, c1)
  PagedCursor cur;
  int64_t todo;
  bool item_head;  // false: the part begins inside an item
  {
    const int k = (c.n_seqs + 31) >> 5;
    const int64_t mine = lane_chunks(c, lens, k, CH, c.n_seqs, status) * tiles;
    int64_t upto = mine;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int64_t W = __shfl_sync(0xffffffffu, upto, 31);
    const int64_t n_warps = min64(all_warps, W);  // none without a chunk
    if (wid >= n_warps) {
      if (lane == 0) splits[wid] = make_int4(0, 0, 0, 0);
      return;
    }
    const int64_t c0 = wid * W / n_warps;
    todo = (wid + 1) * W / n_warps - c0;
    const int at = __ffs(__ballot_sync(0xffffffffu, upto > c0)) - 1;  // the lane whose sequences hold c0
    int64_t rest = c0 - __shfl_sync(0xffffffffu, upto - mine, at);
    cur.s = at * k;
    for (;;) {
      cur.len = seq_len(c, lens, cur.s, status);
      cur.n = (cur.len + CH - 1) / CH;
      if (rest < (int64_t)cur.n * tiles) break;
      rest -= (int64_t)cur.n * tiles;
      ++cur.s;
    }
    cur.tile = (int)(rest / cur.n);
    cur.ci = (int)(rest - (int64_t)cur.tile * cur.n);
    item_head = cur.ci == 0;
    // The first warp that begins inside an item describes it for the join: its
    // parts lie in slot 1 of the warp before and slot 0 of this and the next ones.
    if (lane == 0) {
      const int64_t first = c0 - cur.ci;
      int parts = 0;
      if (!item_head && (wid - 1) * W / n_warps <= first) parts = (int)(((first + cur.n) * n_warps - 1) / W) - wid + 2;
      splits[wid] = make_int4(parts, wid - 1, cur.s, cur.tile);
    }
  }

  // ---- loading: the ring's next slot takes K, then V, of chunk `ld`
  const int64_t head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D);
  PagedCursor ld = cur;
  int64_t ld_left = todo;
  int ld_slot = 0;
  bool ld_v = false;
  int ld_page[NS], ld_row[NS];
  auto look_up = [&]() {
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      const int pos = ld.ci * CH + 16 * r, j = pos / c.page_size;
      ld_row[r] = pos - j * c.page_size;
      ld_page[r] = pos < ld.len ? __ldg(c.page_table + (int64_t)ld.s * c.max_pages + j) : -1;
    }
  };
  look_up();
  auto load = [&]() {
    if (ld_left > 0) {
      const uint8_t* pool = static_cast<const uint8_t*>(ld_v ? c.v_pages : c.k_pages);
      const uint32_t slot = slots + ld_slot * F::SLOT;
      const int kvh = ld.tile / rtiles;
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        int left = ld.len - (ld.ci * CH + 16 * r);  // rows of this group that the sequence has
        if (left > 0 && (unsigned)ld_page[r] >= (unsigned)c.n_pages) {
          if (lane == 0) bad_page(status);
          left = 0;
        }
        const uint8_t* src = left > 0 ? pool + ((int64_t)ld_page[r] * c.n_kv_heads + kvh) * head_bytes : pool;
        const uint8_t* codes = left > 0 ? src + (int64_t)ld_row[r] * F::CB : src;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {  // 16 rows of C columns, 32 lanes
          const int idx = i * 32 + lane, row = idx / C, col = idx % C;
          const int pc = ld_v ? swz8<C>(row, col) : swz_k<T, C>(row, col);
          const bool on = row < left;
          cp_async16(slot + (16 * r + row) * F::CB + pc * 16, on ? codes + idx * 16 : pool, on ? 16 : 0);
        }
        if constexpr (F::SB > 0) {
          if (lane < F::SB) {  // 16 rows of SB bytes
            const int valid = max(0, min(16, left * F::SB - lane * 16));
            const uint8_t* sc = src + (int64_t)c.page_size * F::CB + (int64_t)ld_row[r] * F::SB + lane * 16;
            cp_async16(slot + CH * F::CB + r * 16 * F::SB + lane * 16, valid ? sc : pool, valid);
          }
        }
      }
      ld_slot = ld_slot + 1 == F::SLOTS ? 0 : ld_slot + 1;
      if (ld_v) {
        if (--ld_left > 0) {
          ld.next(c, lens, tiles, CH, status);
          look_up();  // used when the next K is loaded, half a chunk from now
        }
      }
      ld_v = !ld_v;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < F::SLOTS - 1; ++i) load();

  // scales of rows 8 j + 2 t and the next one, as pairs of blocks
  auto scales = [&](uint32_t slot, int j, uint32_t sc[NB]) {
    const uint32_t a = slot + CH * F::CB + (8 * j + 2 * t) * F::SB;
    if constexpr (NB == 2) {
      const uint2 v = lds64(a);
      sc[0] = v.x; sc[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < NB / 4; ++i) {
        const uint4 v = lds128(a + 16 * i);
        sc[4 * i] = v.x; sc[4 * i + 1] = v.y; sc[4 * i + 2] = v.z; sc[4 * i + 3] = v.w;
      }
    }
  };
  // of those, the scale of row `odd` and block b
  auto scale_of = [](const uint32_t sc[NB], int odd, int b) {
    const uint32_t u = sc[odd * (NB / 2) + b / 2];
    return half_bits_to_float((b & 1) ? u >> 16 : u);
  };

  uint32_t qf[2 * NB][4];
  float o[NT][2], m = 0.f, l = 0.f, to_log2 = 0.f;
  int slot_i = 0;
  bool fresh = true;

  for (;;) {
    // ---- scores
    cp_async_wait<F::SLOTS - 2>();
    __syncwarp();
    load();
    const int kvh = cur.tile / rtiles, rt = cur.tile - kvh * rtiles;
    const int rows = min(8, G - 8 * rt), head0 = kvh * G + 8 * rt;
    if (fresh) {
      float x[NB][8], top = 0.f;
      const float* qp = q + cur.s * qs + (int64_t)(head0 + g) * D;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        if (g < rows) {
          if constexpr (T == kKvQ4) {
            u = ldg4(qp + 32 * b + 4 * t);
            v = ldg4(qp + 32 * b + 16 + 4 * t);
          } else {
            u = ldg4(qp + 32 * b + 8 * t);
            v = ldg4(qp + 32 * b + 8 * t + 4);
          }
        }
        x[b][0] = u.x; x[b][1] = u.y; x[b][2] = u.z; x[b][3] = u.w;
        x[b][4] = v.x; x[b][5] = v.y; x[b][6] = v.z; x[b][7] = v.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[b][i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with top 2^e in [2^13, 2^14), as far as fp32 has it; 1 for infinities
      const int eb = __float_as_int(top) >> 23;
      const int es = eb == 255 ? 127 : min(254, 267 - eb);
      const float up = __int_as_float(es << 23);
      const float down = es == 254 ? __int_as_float(0x00400000) : __int_as_float((254 - es) << 23);
      to_log2 = scale * down * 1.44269504088896340736f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* y = x[b] + 4 * h;
          // the pairing that the K fragments of this type have
          const int i1 = T == kKvQ4 ? 2 : 1, i2 = T == kKvQ4 ? 1 : 2;
          split2(y[0] * up, y[i1] * up, qf[2 * b + h][0], qf[2 * b + h][1]);
          split2(y[i2] * up, y[3] * up, qf[2 * b + h][2], qf[2 * b + h][3]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = 0.f;
      m = -INFINITY;
      l = 0.f;
      fresh = false;
    }

    float s[NJ][2];
    {
      const uint32_t slot = slots + slot_i * F::SLOT;
      if constexpr (T == kKvF16) {
        float acc[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const uint4 k = lds128(slot + (8 * j + g) * F::CB + swz_k<T, C>(g, 4 * b + t) * 16);
            mma16816(acc[j], qf[2 * b], k.x, k.y);
            mma16816(acc[j], qf[2 * b + 1], k.z, k.w);
          }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          s[j][0] = acc[j][0] + acc[j][2];
          s[j][1] = acc[j][1] + acc[j][3];
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint32_t sc[NB];
          scales(slot, j, sc);
          s[j][0] = s[j][1] = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (T == kKvQ8) {
              uint2 k = lds64(slot + (8 * j + g) * F::CB + swz_k<T, C>(g, 2 * b + (t >> 1)) * 16 + (t & 1) * 8);
              k.x ^= 0x80808080u;
              k.y ^= 0x80808080u;
              mma16816(acc, qf[2 * b], bytes_h2<0x4140>(k.x), bytes_h2<0x4342>(k.x));
              mma16816(acc, qf[2 * b + 1], bytes_h2<0x4140>(k.y), bytes_h2<0x4342>(k.y));
            } else {
              const uint32_t k = lds32(slot + (8 * j + g) * F::CB + swz_k<T, C>(g, b) * 16 + 4 * t), k8 = k >> 8;
              mma16816(acc, qf[2 * b], nib_lo(k), nib_lo(k8));
              mma16816(acc, qf[2 * b + 1], nib_hi(k), nib_hi(k8));
            }
            s[j][0] = fmaf(acc[0] + acc[2], scale_of(sc, 0, b), s[j][0]);
            s[j][1] = fmaf(acc[1] + acc[3], scale_of(sc, 1, b), s[j][1]);
          }
        }
      }
      slot_i = slot_i + 1 == F::SLOTS ? 0 : slot_i + 1;
    }

    // ---- softmax of the chunk
    const int left = cur.len - cur.ci * CH;  // positions the chunk has
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[j][i] *= to_log2;
        if (left < CH && 8 * j + 2 * t + i >= left) s[j][i] = -INFINITY;
        top = fmaxf(top, s[j][i]);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.f : m_new;
    const float fade = ex2(m - base);
    m = m_new;
    l *= fade;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[j][i] = ex2(s[j][i] - base);
        l += s[j][i];
      }
    if (__any_sync(0xffffffffu, fade != 1.f)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= fade;
        o[n][1] *= fade;
      }
    }

    // ---- weighted values
    cp_async_wait<F::SLOTS - 2>();
    __syncwarp();
    load();
    {
      const uint32_t slot = slots + slot_i * F::SLOT;
      // ldmatrix rows: lanes 0-7 and 8-15 the two halves of 16 positions, 16-31 the next column
      const int lr = lane & 15, lc = lane >> 4;
      if constexpr (T == kKvF16) {
        uint32_t p[NS][4];
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          split2(s[2 * k][0] * 16384.f, s[2 * k][1] * 16384.f, p[k][0], p[k][1]);
          split2(s[2 * k + 1][0] * 16384.f, s[2 * k + 1][1] * 16384.f, p[k][2], p[k][3]);
        }
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            uint32_t v[4];
            ldsm4_trans(slot + (16 * k + lr) * F::CB + swz8<C>(lr, n + lc) * 16, v);
            mma16816(a0, p[k], v[0], v[1]);
            mma16816(a1, p[k], v[2], v[3]);
          }
          const float f = 1.f / 16384.f;
          o[n][0] = fmaf(a0[0] + a0[2], f, o[n][0]);
          o[n][1] = fmaf(a0[1] + a0[3], f, o[n][1]);
          o[n + 1][0] = fmaf(a1[0] + a1[2], f, o[n + 1][0]);
          o[n + 1][1] = fmaf(a1[1] + a1[3], f, o[n + 1][1]);
        }
      } else {
        uint32_t sc[NJ][NB];
        __half2 big = __float2half2_rn(0.f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          scales(slot, j, sc[j]);
#pragma unroll
          for (int b = 0; b < NB; ++b) big = __hmax2(big, __habs2(bits_h2(sc[j][b])));
        }
        uint32_t u = h2_bits(big);
        int e = max(u & 0xFFFFu, u >> 16);
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        e >>= 10;  // every |scale| < 2^(e - 14), or infinite
        const float up = __int_as_float((127 + 28 - e) << 23), down = __int_as_float((127 - 28 + e) << 23);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          s[j][0] *= up;
          s[j][1] *= up;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float a[4][4];
#pragma unroll
          for (int n = 0; n < 4; ++n) a[n][0] = a[n][1] = a[n][2] = a[n][3] = 0.f;
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            uint32_t p[4];
            split2(s[2 * k][0] * scale_of(sc[2 * k], 0, b), s[2 * k][1] * scale_of(sc[2 * k], 1, b), p[0], p[1]);
            split2(s[2 * k + 1][0] * scale_of(sc[2 * k + 1], 0, b), s[2 * k + 1][1] * scale_of(sc[2 * k + 1], 1, b),
                   p[2], p[3]);
            if constexpr (T == kKvQ8) {
              uint32_t v[4];
              ldsm4_trans(slot + (16 * k + lr) * F::CB + swz8<C>(lr, 2 * b + lc) * 16, v);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] ^= 0x80808080u;
              mma16816(a[0], p, bytes_h2<0x4240>(v[0]), bytes_h2<0x4240>(v[1]));  // even elements of 16
              mma16816(a[1], p, bytes_h2<0x4341>(v[0]), bytes_h2<0x4341>(v[1]));  // odd ones
              mma16816(a[2], p, bytes_h2<0x4240>(v[2]), bytes_h2<0x4240>(v[3]));
              mma16816(a[3], p, bytes_h2<0x4341>(v[2]), bytes_h2<0x4341>(v[3]));
            } else {
              uint32_t v[2];
              asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                           : "=r"(v[0]), "=r"(v[1])
                           : "r"(slot + (16 * k + lr) * F::CB + swz8<C>(lr, b) * 16));
              const uint32_t w0 = v[0] >> 8, w1 = v[1] >> 8;
              mma16816(a[0], p, nib_lo(v[0]), nib_lo(v[1]));
              mma16816(a[1], p, nib_lo(w0), nib_lo(w1));
              mma16816(a[2], p, nib_hi(v[0]), nib_hi(v[1]));
              mma16816(a[3], p, nib_hi(w0), nib_hi(w1));
            }
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            o[4 * b + n][0] = fmaf(a[n][0] + a[n][2], down, o[4 * b + n][0]);
            o[4 * b + n][1] = fmaf(a[n][1] + a[n][3], down, o[4 * b + n][1]);
          }
        }
      }
      slot_i = slot_i + 1 == F::SLOTS ? 0 : slot_i + 1;
    }

    // ---- end of an item, or of this warp's part
    --todo;
    const bool item_end = cur.ci + 1 == cur.n;
    if (item_end || todo == 0) {
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (g < rows) {
        const bool whole = item_end && item_head;
        float* dst;
        float f = 1.f;
        if (whole) {
          dst = out + ((int64_t)cur.s * Hq + head0 + g) * D;
          f = 1.f / l;
        } else {
          // slot 0: the item that the part begins inside of (or holds nothing but); 1: the one it ends inside of
          float* slot = part + (2ll * wid + (item_head ? 1 : 0)) * paged_part_floats(min(8, G), D);
          dst = slot + 16 + g * D;
          if (t == 0) {
            slot[g] = m;
            slot[8 + g] = l;
          }
        }
        if constexpr (T == kKvF16) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(dst + 8 * n + 2 * t) = make_float2(o[n][0] * f, o[n][1] * f);
        } else {
          // tiles n, n + 1 hold elements 4 t, 4 t + 2 and 4 t + 1, 4 t + 3 of 16
#pragma unroll
          for (int n = 0; n < NT; n += 2)
            *reinterpret_cast<float4*>(dst + 8 * n + 4 * t) =
                make_float4(o[n][0] * f, o[n + 1][0] * f, o[n][1] * f, o[n + 1][1] * f);
        }
      }
      if (todo == 0) break;
      item_head = true;
      fresh = true;
    }
    cur.next(c, lens, tiles, CH, status);
  }
  cp_async_wait<0>();
  pdl_launch_dependents();
}

// Joins the parts of the items that several warps hold: with M the largest m,
// out = sum 2^(m - M) o / sum 2^(m - M) l.  Every CTA gathers the split items
// (main kernel's records, in shared memory); then each warp takes (item, head)
// pairs of few parts, and each CTA (item, head, 32 elements) of many.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 32;  // one for each lane
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const int4* splits, int n_splits,
                                                                      const float* part, float* __restrict__ out,
                                                                      int Hq, int n_kv_heads) {
  extern __shared__ int4 s_item[];  // items of few parts from the front, of many from the back
  __shared__ int s_n[kJoinWarps];
  __shared__ float s_w[kJoinThreads], s_red[kJoinWarps], s_l[kJoinWarps];
  __shared__ __align__(16) float s_o[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = Hq / n_kv_heads, rtiles = (G + 7) >> 3, rows = min(8, G);
  const int64_t stride = paged_part_floats(rows, D);
  int n_few, n_many;
  pdl_wait();
  {  // the same order in every CTA: thread i takes the i-th run of records
    const int run = (n_splits + kJoinThreads - 1) / kJoinThreads;
    const int r0 = min(n_splits, (int)threadIdx.x * run), r1 = min(n_splits, r0 + run);
    int count = 0;  // few in the low, many in the high half
    for (int i = r0; i < r1; ++i) {
      const int parts = splits[i].x;
      count += parts == 0 ? 0 : parts > kFewParts ? 0x10000 : 1;
    }
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_n[warp] = upto;
    __syncthreads();
    int at = upto - count, all = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) at += s_n[w];
      all += s_n[w];
    }
    n_few = all & 0xFFFF;
    n_many = all >> 16;
    int few = at & 0xFFFF, many = at >> 16;
    for (int i = r0; i < r1; ++i) {
      const int4 r = splits[i];
      if (r.x) s_item[r.x > kFewParts ? n_splits - 1 - many++ : few++] = r;
    }
    __syncthreads();
  }
  // part i of an item whose first part is warp w's
  auto slot = [&](int w, int i) { return part + (2ll * (w + i) + (i == 0 ? 1 : 0)) * stride; };
  // the query head of row r of an item, -1 behind the last
  auto head_of = [&](const int4& it, int r) {
    const int kvh = it.w / rtiles, h = (it.w - kvh * rtiles) * 8 + r;
    return h < G ? kvh * G + h : -1;
  };

  constexpr int COLS = D / 4 < 32 ? D / 4 : 32, GRP = 32 / COLS, V = D / 4 / COLS;  // float4 columns of a row
  for (int u = blockIdx.x * kJoinWarps + warp; u < n_few * rows; u += gridDim.x * kJoinWarps) {
    const int4 it = s_item[u / rows];
    const int r = u % rows, h = head_of(it, r);
    if (h < 0) continue;
    float w = -INFINITY, l = 0.f;
    if (lane < it.x) {
      const float* p = slot(it.y, lane);
      w = p[r];
      l = p[8 + r];
    }
    float M = warp_max(w);
    if (M == -INFINITY) M = 0.f;
    w = lane < it.x ? ex2(w - M) : 0.f;
    const float f = 1.f / warp_sum(w * l);
    float4 O[V];
#pragma unroll
    for (int v = 0; v < V; ++v) O[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int grp = lane / COLS, col = lane % COLS;
#pragma unroll 4
    for (int i0 = 0; i0 < it.x; i0 += GRP) {
      const int i = i0 + grp;
      const float e = __shfl_sync(0xffffffffu, w, i & 31);
      if (i < it.x) {
        const float4* p = reinterpret_cast<const float4*>(slot(it.y, i) + 16 + r * D) + col;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float4 x = p[v * COLS];
          O[v].x = fmaf(x.x, e, O[v].x);
          O[v].y = fmaf(x.y, e, O[v].y);
          O[v].z = fmaf(x.z, e, O[v].z);
          O[v].w = fmaf(x.w, e, O[v].w);
        }
      }
    }
    if constexpr (GRP == 2) {
      O[0].x += __shfl_xor_sync(0xffffffffu, O[0].x, 16);
      O[0].y += __shfl_xor_sync(0xffffffffu, O[0].y, 16);
      O[0].z += __shfl_xor_sync(0xffffffffu, O[0].z, 16);
      O[0].w += __shfl_xor_sync(0xffffffffu, O[0].w, 16);
    }
    float4* dst = reinterpret_cast<float4*>(out + ((int64_t)it.z * Hq + h) * D) + col;
    if (grp == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) dst[v * COLS] = make_float4(O[v].x * f, O[v].y * f, O[v].z * f, O[v].w * f);
  }

  constexpr int Z = D / 32;
  for (int u = blockIdx.x; u < n_many * rows * Z; u += gridDim.x) {
    const int4 it = s_item[n_splits - 1 - u / (rows * Z)];
    const int r = u / Z % rows, z = u % Z, h = head_of(it, r);
    if (h < 0) continue;
    float M = -INFINITY;
    for (int i = threadIdx.x; i < it.x; i += kJoinThreads) M = fmaxf(M, slot(it.y, i)[r]);
    M = warp_max(M);
    __syncthreads();  // the last item's reads of the shared arrays are done
    if (lane == 0) s_red[warp] = M;
    __syncthreads();
    M = s_red[0];
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i) M = fmaxf(M, s_red[i]);
    if (M == -INFINITY) M = 0.f;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    const int sub = threadIdx.x >> 3, e = (threadIdx.x & 7) * 4;  // 8 threads read the 32 elements of a part
    for (int base = 0; base < it.x; base += kJoinThreads) {
      const int cnt = min(kJoinThreads, it.x - base);
      if (base) __syncthreads();
      if ((int)threadIdx.x < cnt) {
        const float* p = slot(it.y, base + threadIdx.x);
        const float f = ex2(p[r] - M);
        s_w[threadIdx.x] = f;
        L = fmaf(p[8 + r], f, L);
      }
      __syncthreads();
#pragma unroll 4
      for (int i = sub; i < cnt; i += kJoinThreads / 8) {
        const float f = s_w[i];
        const float4 v = *reinterpret_cast<const float4*>(slot(it.y, base + i) + 16 + r * D + 32 * z + e);
        O.x = fmaf(v.x, f, O.x);
        O.y = fmaf(v.y, f, O.y);
        O.z = fmaf(v.z, f, O.z);
        O.w = fmaf(v.w, f, O.w);
      }
    }
    L = warp_sum(L);
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      O.x += __shfl_xor_sync(0xffffffffu, O.x, o);
      O.y += __shfl_xor_sync(0xffffffffu, O.y, o);
      O.z += __shfl_xor_sync(0xffffffffu, O.z, o);
      O.w += __shfl_xor_sync(0xffffffffu, O.w, o);
    }
    if (lane < 8) *reinterpret_cast<float4*>(&s_o[warp][e]) = O;
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (warp == 0) {
      float sum = 0.f, tot = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) {
        sum += s_o[i][lane];
        tot += s_l[i];
      }
      out[((int64_t)it.z * Hq + h) * D + 32 * z + lane] = sum / tot;
    }
  }
}

}  // namespace ntx
