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
// One CTA of four warps per (query head, sequence); a warp takes every fourth
// position with an online softmax, lanes split the head dimension; the warps'
// (m, l, o) are joined with the log-sum-exp rule.
template <int T, int D>
__global__ void __launch_bounds__(128) attn_paged_kernel(const ntx_paged_kv c, const float* __restrict__ q, int64_t qs,
                                                         float* __restrict__ out, int Hq, const int* __restrict__ lens,
                                                         float scale, int* status) {
  constexpr int E = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, s = blockIdx.y, kvh = h / (Hq / c.n_kv_heads);
  int len = __ldg(lens + s);
  if (len < 0 || len > c.max_pages * c.page_size) {
    if (threadIdx.x == 0) bad_page(status);
    len = max(0, min(len, c.max_pages * c.page_size));
  }
  const int64_t head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D);
  float qr[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qr[i] = q[s * qs + (int64_t)h * D + i * 32 + lane];
    o[i] = 0.f;
  }
  for (int p = warp; p < len; p += 4) {
    const int j = p / c.page_size, row = p - j * c.page_size;
    const int page = __ldg(c.page_table + (int64_t)s * c.max_pages + j);
    const bool ok = page >= 0 && page < c.n_pages;
    if (!ok && lane == 0) bad_page(status);
    const int64_t at = ((int64_t)page * c.n_kv_heads + kvh) * head_bytes;
    float x = 0.f;
    if (ok)
#pragma unroll
      for (int i = 0; i < E; ++i)
        x = fmaf(qr[i], kv_element<T>(static_cast<const uint8_t*>(c.k_pages) + at, c.page_size, D, row, i * 32 + lane), x);
    x = warp_sum(x) * scale;
    const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - base), e = expf(x - base);
    m = mn;
    l = fmaf(l, a, e);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float t = ok ? kv_element<T>(static_cast<const uint8_t*>(c.v_pages) + at, c.page_size, D, row, i * 32 + lane) : 0.f;
      o[i] = fmaf(e, t, o[i] * a);
    }
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int i = 0; i < E; ++i) s_o[warp][i * 32 + lane] = o[i];
  __syncthreads();
  float M = s_m[0];
  for (int w = 1; w < 4; ++w) M = fmaxf(M, s_m[w]);
  if (M == -INFINITY) M = 0.f;
  for (int d = threadIdx.x; d < D; d += 128) {
    float L = 0.f, O = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float e = expf(s_m[w] - M);
      L = fmaf(s_l[w], e, L);
      O = fmaf(s_o[w][d], e, O);
    }
    out[((int64_t)s * Hq + h) * D + d] = len ? O / L : 0.f;
  }
}

}  // namespace ntx
