// paged.cuh -- kernels of the paged KV cache: head norms with the rotation,
// the cache's write and read-back, and decode attention over it.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

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

// Bytes of a pool, for the debug build's checks.
template <int T, int D>
__device__ __forceinline__ int64_t kv_pool_bytes(const ntx_paged_kv& c) {
  return (int64_t)c.n_pages * c.n_kv_heads * c.page_size * kv_row_bytes<T>(D);
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

// A warp of the write and of the read handles one row's piece of kPiece elements,
// four consecutive ones to a lane at a time (eight lanes a block of 32), all its
// loads in flight at once; a row's place is looked up once a piece.  On B200, 24001
// tokens of 8 heads of 128 from Q8_0: 43 us, 5.7 TB/s, 0.87 of a copy's bandwidth;
// 16384 tokens to Q4_0 and back: 65 us (with a search of the first largest by ballot
// and separate checks of zeros and infinities in every block: 69), 28 of them the read
// at 5.6 TB/s.  Writes alone, 16384 tokens: F16 31 us (0.99 of a copy's bandwidth),
// Q8_0 36 (0.72), Q4_0 38 (0.61): block types are bound by their instructions, the F16
// write and the reads by memory.  Pieces of 1024 elements are 3 % faster on long prompts
// and 25 % slower on one token.
constexpr int kPieceSteps = 4, kPiece = kPieceSteps * 128;
constexpr int kTokenWarps = 4;  // tokens of a CTA

// Where a lane's four elements of step i of a piece lie: a step is 128 elements, 128 / D
// heads or a half of one.
template <int T, int D>
struct PieceAt {
  uint8_t *codes, *scales;  // step 0's
  int64_t head_bytes;
  __device__ __forceinline__ PieceAt(const ntx_paged_kv& c, void* pool, int64_t page, int row, int e0) {
    head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D);
    const int e = e0 % D, blk = e / 32, sub = e % 32 / 4;
    uint8_t* part = static_cast<uint8_t*>(pool) + (page * c.n_kv_heads + e0 / D) * head_bytes;
    codes = part + (int64_t)row * kv_code_bytes<T>(D) +
            (T == kKvF16 ? 2 * e : T == kKvQ8 ? e : blk * 16 + (sub & 3) * 4);
    scales = part + (int64_t)c.page_size * kv_code_bytes<T>(D) + row * (D / 16ll) + blk * 2;
  }
  __device__ __forceinline__ uint8_t* code(int i) const {
    return codes + i * 128 / D * head_bytes + kv_code_bytes<T>(i * 128 % D);
  }
  __device__ __forceinline__ uint16_t* scale(int i) const {
    return reinterpret_cast<uint16_t*>(scales + i * 128 / D * head_bytes + i * 128 % D / 16);
  }
  // (debug build) whether this lane's codes and scale of step i lie in the pool
  __device__ __forceinline__ bool inside(const ntx_paged_kv& c, const void* pool, int i, int* status) const {
    const uint8_t* base = static_cast<const uint8_t*>(pool);
    const int64_t bytes = kv_pool_bytes<T, D>(c);
    return chk(status, kChkPagedRow, code(i) - base, bytes) &&
           chk(status, kChkPagedRow, code(i) - base + (T == kKvF16 ? 7 : 3), bytes) &&
           (T == kKvF16 || chk(status, kChkPagedRow, reinterpret_cast<const uint8_t*>(scale(i)) - base + 1, bytes));
  }
};

// ------------------------------------------------------------- cache write
// A code is the fp32 quotient w / d rounded half away from zero.  w times rcp(d),
// within 2^-14 of the quotient (which is at most 127, or 8), tells it unless it is
// next to a half; rounding is by adding 1.5 2^23 (and 8 for Q4_0), whose lowest
// byte is then the code.  Next to a half, and where rcp(d) overflows, the quotient
// itself decides.  Blocks of zeros or with an infinity or a NaN show there too: one
// of their products is not a number, and a warp without any has nothing to look at.
template <int T>
__device__ __forceinline__ uint32_t quotient_code(float w, float d) {
  const float x = fabsf(w / d), f = floorf(x);
  int q = (int)f + (x - f >= 0.5f ? 1 : 0);  // x - f is exact
  q = (w < 0.f) != (d < 0.f) ? -q : q;
  return (uint32_t)(T == kKvQ8 ? min(127, max(-127, q)) : min(15, max(0, q + 8))) & 255u;
}
__device__ __forceinline__ float max_nan(float x, float y, float z) {  // NaN if any is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Codes by the reciprocal; false where one of the four is next to a half or is not a number.
template <int T>
__device__ __forceinline__ bool reciprocal_codes(const float w[4], float d, uint32_t* codes) {
  constexpr float kMagic = T == kKvQ8 ? 12582912.f : 12582920.f;
  float r, e[4];
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = fmaf(w[i], r, kMagic);
    e[i] = fabsf(fmaf(w[i], r, kMagic - y));
    m[i] = __float_as_uint(y);
  }
  const uint32_t c = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
  *codes = T == kKvQ4 ? c - (c >> 4 & 0x01010101u) : c;  // 16, the largest's opposite, is 15
  return max_nan(max_nan(e[0], e[1], e[2]), e[3], 0.f) < 0.5f - 0x1p-14f;
}
__device__ __forceinline__ float larger(float x, float y) { return fabsf(y) > fabsf(x) ? y : x; }

template <int T, int D>
__global__ void __launch_bounds__(kTokenWarps * 32) kv_append_kernel(const ntx_paged_kv c, const float* __restrict__ k,
                                                                     const float* __restrict__ v, int64_t ks,
                                                                     int64_t vs, const int* __restrict__ seq_ids,
                                                                     const int* __restrict__ positions, int n_tokens,
                                                                     bool vec, int pieces, int* status) {
  const int width = c.n_kv_heads * D, lane = threadIdx.x & 31, sub = lane & 7;
  const int n = blockIdx.x * kTokenWarps + (threadIdx.x >> 5);
  if (n >= n_tokens) return;
  const int piece = (int)blockIdx.y % pieces, e0 = piece * kPiece + lane * 4;
  const bool is_v = (int)blockIdx.y >= pieces;
  const float* in = is_v ? v + n * vs : k + n * ks;
  const int pos = __ldg(positions + n);
  float w[kPieceSteps][4];
#pragma unroll
  for (int i = 0; i < kPieceSteps; ++i) {
    const int e = e0 + i * 128;
    w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0.f;
    if (e < width) {
      if (vec) {
        const float4 t = *reinterpret_cast<const float4*>(in + e);
        w[i][0] = t.x; w[i][1] = t.y; w[i][2] = t.z; w[i][3] = t.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][j] = in[e + j];
      }
    }
  }
  int64_t page;
  int row;
  if (pos < 0 || !kv_place(c, seq_ids ? __ldg(seq_ids + n) : n, pos, &page, &row, status)) return;
  const PieceAt<T, D> at(c, is_v ? c.v_pages : c.k_pages, page, row, e0);
#pragma unroll
  for (int i = 0; i < kPieceSteps; ++i) {
    const int e = e0 + i * 128;
    if (e - lane * 4 >= width) break;
    const bool on = e < width && at.inside(c, is_v ? c.v_pages : c.k_pages, i, status);
    if constexpr (T == kKvF16) {
      if (on) {
        uint2 h;
        h.x = float_to_half_bits(w[i][0]) | ((uint32_t)float_to_half_bits(w[i][1]) << 16);
        h.y = float_to_half_bits(w[i][2]) | ((uint32_t)float_to_half_bits(w[i][3]) << 16);
        *reinterpret_cast<uint2*>(at.code(i)) = h;
      }
    } else {
      float d;
      if constexpr (T == kKvQ8) {
        float top = fmaxf(fmaxf(fabsf(w[i][0]), fabsf(w[i][1])), fmaxf(fabsf(w[i][2]), fabsf(w[i][3])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        d = top / 127.0f;
      } else {
        // the first element of the largest magnitude: a tie stays with the lower lane, which has the earlier one
        float m = larger(larger(w[i][0], w[i][1]), larger(w[i][2], w[i][3]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = larger(m, __shfl_down_sync(0xffffffffu, m, o, 8));
        d = __shfl_sync(0xffffffffu, m, 0, 8) * -0.125f;
      }
      uint32_t codes;
      const bool sure = reciprocal_codes<T>(w[i], d, &codes);
      uint16_t scale = float_to_half_bits(d);
      if (__any_sync(0xffffffffu, on && !sure)) {  // zeros and what is not finite too: 0 or an infinity times r
        bool bad = false, some = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bad |= !(fabsf(w[i][j]) < INFINITY);
          some |= w[i][j] != 0.f;
        }
        const unsigned block = 255u << (lane & 24);
        bad = __ballot_sync(0xffffffffu, bad) & block;
        some = __ballot_sync(0xffffffffu, some) & block;
        if (bad || !some) {  // codes of zero
          codes = T == kKvQ8 ? 0u : 0x08080808u;
          scale = bad ? 0x7FFF : T == kKvQ8 ? 0 : 0x8000;
        } else if (!sure) {
          codes = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) codes |= quotient_code<T>(w[i][j], d) << (8 * j);
        }
      }
      if constexpr (T == kKvQ8) {
        if (on) *reinterpret_cast<uint32_t*>(at.code(i)) = codes;
      } else {
        const uint32_t hi = __shfl_down_sync(0xffffffffu, codes, 4, 8);  // elements 16 further on
        if (on && sub < 4) *reinterpret_cast<uint32_t*>(at.code(i)) = codes | (hi << 4);
      }
      if (on && sub == 0) *at.scale(i) = scale;
    }
  }
}

// ------------------------------------------------------------- cache read
template <int T, int D>
__global__ void __launch_bounds__(kTokenWarps * 32) kv_read_kernel(const ntx_paged_kv c, float* __restrict__ k,
                                                                   float* __restrict__ v, int64_t ks, int64_t vs,
                                                                   const int* __restrict__ seq_ids,
                                                                   const int* __restrict__ positions, int n_tokens,
                                                                   bool vec, int pieces, int* status) {
  const int width = c.n_kv_heads * D, lane = threadIdx.x & 31, sub = lane & 7;
  const int n = blockIdx.x * kTokenWarps + (threadIdx.x >> 5);
  if (n >= n_tokens) return;
  const int piece = (int)blockIdx.y % pieces, e0 = piece * kPiece + lane * 4;
  const bool is_v = (int)blockIdx.y >= pieces;
  if (!(is_v ? v : k)) return;
  float* out = is_v ? v + n * vs : k + n * ks;
  const int pos = __ldg(positions + n);
  int64_t page;
  int row;
  if (pos < 0 || !kv_place(c, seq_ids ? __ldg(seq_ids + n) : n, pos, &page, &row, status)) return;
  const PieceAt<T, D> at(c, is_v ? c.v_pages : c.k_pages, page, row, e0);
  uint2 code[kPieceSteps];
  uint16_t scale[kPieceSteps];
#pragma unroll
  for (int i = 0; i < kPieceSteps; ++i) {
    const int e = e0 + i * 128;
    if (e >= width || !at.inside(c, is_v ? c.v_pages : c.k_pages, i, status)) break;
    if constexpr (T == kKvF16) {
      code[i] = *reinterpret_cast<const uint2*>(at.code(i));
    } else {
      code[i].x = *reinterpret_cast<const uint32_t*>(at.code(i));
      scale[i] = *at.scale(i);
    }
  }
#pragma unroll
  for (int i = 0; i < kPieceSteps; ++i) {
    const int e = e0 + i * 128;
    if (e >= width || !at.inside(c, is_v ? c.v_pages : c.k_pages, i, status)) break;
    float4 o;
    if constexpr (T == kKvF16) {
      o = make_float4(half_bits_to_float(code[i].x), half_bits_to_float(code[i].x >> 16),
                      half_bits_to_float(code[i].y), half_bits_to_float(code[i].y >> 16));
    } else {
      const float d = half_bits_to_float(scale[i]);
      constexpr float off = 8388608.f + (T == kKvQ8 ? 128.f : 8.f);  // magic_byte gives 2^23 + u
      const uint32_t u = T == kKvQ8 ? code[i].x ^ 0x80808080u : (code[i].x >> (sub & 4)) & 0x0F0F0F0Fu;
      o = make_float4(magic_byte<0>(u) - off, magic_byte<1>(u) - off, magic_byte<2>(u) - off, magic_byte<3>(u) - off);
      o.x *= d; o.y *= d; o.z *= d; o.w *= d;  // exact: 11 by 8 bits
    }
    if (vec) {
      *reinterpret_cast<float4*>(out + e) = o;
    } else {
      out[e] = o.x; out[e + 1] = o.y; out[e + 2] = o.z; out[e + 3] = o.w;
    }
  }
}

// ------------------------------------------------------------- head norm + rotation
// theta^(-2p/R) to fp64's precision: 2^-x with x = 2p log2(theta) / R as a quotient
// and its remainder (log2 theta in two numbers, the first of 40 bits, so that 2p
// times it is exact).
__device__ __forceinline__ double rope_frequency(int p, int R, double log2_hi, double log2_lo) {
  const double a = 2.0 * p * log2_hi, q = a / R;
  const double rest = (fma(-q, (double)R, a) + 2.0 * p * log2_lo) / R;
  return exp2(-q) * (1.0 - 0.69314718055994530942 * rest);
}

// 1 / sqrt(x): the approximation (2^-22.4) and a step of Newton's, within 2^-23.
__device__ __forceinline__ float rope_rsqrt(float x) {
  const float r = rsqrtf(x), y = r * fmaf(-0.5f * x * r, r, 1.5f);
  return x > 0.f && x < INFINITY ? y : r;
}

// Cosine and sine of t half turns: t less the nearest multiple of a quarter turn is
// exact in fp64 and rounds to fp32 within 2^-27 of a half turn, 2e-8; sine and cosine
// of at most an eighth of a turn are fp32's.  The multiple is rounded by adding
// 1.5 2^52, whose low word then counts quarter turns: any t below 2^50, where an fp64
// angle still tells quarters apart (a theta below 1 brings angles past 2^31).
__device__ __forceinline__ float2 rope_turn(double t) {
  const double m = fma(2.0, t, 6755399441055744.0), n = m - 6755399441055744.0;
  float s, c;
  sincospif((float)fma(-0.5, n, t), &s, &c);
  const unsigned k = (unsigned)__double2loint(m);
  const float x = (k & 1) ? s : c, y = (k & 1) ? c : s;
  return make_float2(((k + 1) & 2) ? -x : x, (k & 2) ? -y : y);
}

// A warp takes a token and some of its heads' rows: a lane forms the cosines and sines
// of its P pairs once for them, then norms and rotates the rows, several in flight.
// Bound by memory: 8192 tokens of 72 heads of 128 take 101 us, 6.0 TB/s, 0.92 of a
// copy's bandwidth (angles shared by a CTA through shared memory: 117 us; sines and
// cosines in fp64: 110; a tile's next rows loaded ahead: 138, the registers cost a
// CTA).  VEC: rows are 16-byte aligned and a lane holds P consecutive pairs;
// otherwise pairs lane, lane + 32, ... with 4-byte accesses: over one buffer again and
// again, half of each head rotated in halves takes 121 us, rows off by 4 bytes 126,
// where aligned rows take 110.
constexpr int kRopeWarps = 8;
__host__ __device__ constexpr int rope_ctas(int P) { return P < 4 ? 4 : 3; }  // per SM, 64 and 80 registers
template <int P, bool HALVES, bool VEC>
__global__ void __launch_bounds__(kRopeWarps * 32, rope_ctas(P))
    qk_norm_rope_kernel(const float* q, const float* k, float* q_out, float* k_out, int64_t qs, int64_t ks,
                        const float* __restrict__ wq, const float* __restrict__ wk, const int* __restrict__ positions,
                        int n_tokens, int Hq, int Hkv, int D, int R, double log2_hi, double log2_lo, float eps,
                        int rows, int shares) {
  // A row's elements are D / 2 pairs: the R / 2 that rotate, then neighbours.
  constexpr int U = VEC && P < 4 ? 4 : 2;  // rows in flight
  const int lane = threadIdx.x & 31, heads = Hq + Hkv, half = R / 2;
  auto pair = [&](int i) { return VEC ? lane * P + i : lane + 32 * i; };
  auto first = [&](int p) { return HALVES && p < half ? p : 2 * p; };
  auto second = [&](int p) { return HALVES && p < half ? p + half : 2 * p + 1; };
  double f[P];
  float w[2][P][2];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = pair(i);
    f[i] = p < half ? rope_frequency(p, R, log2_hi, log2_lo) * 0.31830988618379067154 : 0.0;
    const bool on = 2 * p < D;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float* wt = x ? wk : wq;
      w[x][i][0] = on && wt ? __ldg(wt + first(p)) : 1.f;
      w[x][i][1] = on && wt ? __ldg(wt + second(p)) : 1.f;
    }
  }
  const float inv_d = 1.0f / (float)D;
  const int64_t units = (int64_t)n_tokens * shares;
  for (int64_t unit = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); unit < units;
       unit += (int64_t)gridDim.x * kRopeWarps) {
    const int n = (int)(unit / shares), share = (int)(unit - (int64_t)n * shares);
    const int pos = __ldg(positions + n), h1 = min(heads, (share + 1) * rows);
    int h0 = share * rows;
    if (pos < 0) continue;
    const int64_t at_q = n * qs, at_k = n * ks - (int64_t)Hq * D;  // where head 0's row would be
    float x[U][P][2];
    auto load = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u;
        if (h >= h1) break;
        const bool is_q = h < Hq;
        const float* in = (is_q ? q + at_q : k + at_k) + h * D;
        if constexpr (VEC && HALVES) {
          if constexpr (P == 1) {
            x[u][0][0] = in[lane];
            x[u][0][1] = in[lane + 32];
          } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
              const float2 a = *reinterpret_cast<const float2*>(in + lane * P + i);
              const float2 b = *reinterpret_cast<const float2*>(in + 32 * P + lane * P + i);
              x[u][i][0] = a.x; x[u][i + 1][0] = a.y;
              x[u][i][1] = b.x; x[u][i + 1][1] = b.y;
            }
          }
        } else if constexpr (VEC) {
          if constexpr (P == 1) {
            const float2 a = *reinterpret_cast<const float2*>(in + 2 * lane);
            x[u][0][0] = a.x; x[u][0][1] = a.y;
          } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
              const float4 a = *reinterpret_cast<const float4*>(in + 2 * (lane * P + i));
              x[u][i][0] = a.x; x[u][i][1] = a.y;
              x[u][i + 1][0] = a.z; x[u][i + 1][1] = a.w;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int p = pair(i);
            x[u][i][0] = 2 * p < D ? in[first(p)] : 0.f;
            x[u][i][1] = 2 * p < D ? in[second(p)] : 0.f;
          }
        }
      }
    };
    load();
    float2 turn[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      turn[i] = rope_turn(f[i] * pos);
    }
    for (;;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u;
        if (h >= h1) break;  // (the same in the whole warp)
        const bool is_q = h < Hq;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) ss = fmaf(x[u][i][0], x[u][i][0], fmaf(x[u][i][1], x[u][i][1], ss));
        const float norm = rope_rsqrt(fmaf(warp_sum(ss), inv_d, eps));
        float* out = (is_q ? q_out + at_q : k_out + at_k) + h * D;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int p = pair(i);
          const float a = x[u][i][0] * norm * (is_q ? w[0][i][0] : w[1][i][0]);
          const float b = x[u][i][1] * norm * (is_q ? w[0][i][1] : w[1][i][1]);
          const float2 t = turn[i];
          x[u][i][0] = a * t.x - b * t.y;
          x[u][i][1] = a * t.y + b * t.x;
          if (!(VEC && HALVES) && p >= half) {  // only normed: as it is, infinities too
            x[u][i][0] = a;
            x[u][i][1] = b;
          }
        }
        if constexpr (VEC && HALVES) {
          if constexpr (P == 1) {
            out[lane] = x[u][0][0];
            out[lane + 32] = x[u][0][1];
          } else {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
              *reinterpret_cast<float2*>(out + lane * P + i) = make_float2(x[u][i][0], x[u][i + 1][0]);
              *reinterpret_cast<float2*>(out + 32 * P + lane * P + i) = make_float2(x[u][i][1], x[u][i + 1][1]);
            }
          }
        } else if constexpr (VEC) {
          if constexpr (P == 1) {
            *reinterpret_cast<float2*>(out + 2 * lane) = make_float2(x[u][0][0], x[u][0][1]);
          } else {
#pragma unroll
            for (int i = 0; i < P; i += 2)
              *reinterpret_cast<float4*>(out + 2 * (lane * P + i)) =
                  make_float4(x[u][i][0], x[u][i][1], x[u][i + 1][0], x[u][i + 1][1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int p = pair(i);
            if (2 * p < D) {
              out[first(p)] = x[u][i][0];
              out[second(p)] = x[u][i][1];
            }
          }
        }
      }
      h0 += U;
      if (h0 >= h1) break;
      load();
    }
  }
}

// ------------------------------------------------------------- attention
//
//   out[s][h] = sum_p softmax_p(scale q.k_p) v_p       (p < len[s])
//
// A warp works on items (sequence, KV head, tile of up to 4 NC of its query heads)
// in chunks of CH positions, with m16n8k16 fp16 matrix instructions and one pass
// over the data: running maximum m (base 2), sum l and output o of a softmax.
// Keys (16 positions) and values (16 elements) are the instruction's A, q and p
// its B of 8 columns.
//
// fp32 accuracy from fp16 products: columns 2h and 2h + 1 of a tile belong to head
// h, one with the upper 11 bits of its operand, the other with the rounded
// remainder; both products land in one thread's accumulators and are added there:
// 22 bits of q and p.  Keys and values are exact in fp16: F16 as they are, the
// codes of block types as integers.  A key block's scale multiplies its partial
// score in fp32; a value block's scale multiplies p, again as two fp16 numbers
// (the product of the upper parts, what its rounding leaves, and the product of
// the lower part).  q is first scaled by a power of two that puts its largest
// element in [2^13, 2^14); p is kept 2^14 fold (F16) or 2^10 fold, and value
// scales times a power of two that puts the chunk's largest in [2^4, 2^5): nothing
// overflows fp16, and what its subnormals round off is below 2^-35 of the largest
// weight and 2^-29 of the chunk's largest value.
// Codes enter as signed integers: as (code + 128) or (code + 8), fp16 subnormals that
// take no conversion, keys of Q4_0 would take 9 % less time (49.7 us for 131071
// positions instead of 54.4) and of Q8_0 2 %, but a score would be off by a rounding of
// the offset's share, 128 sum(q), whatever its own size: 20 times a plain fp32
// evaluation's error where a block has one large key and queries have a mean.
// The matrix instruction's fp32 accumulation truncates, so it only sums one block of
// codes, one F16 key (head_dim / 16 instructions) or one chunk of values; longer sums
// are ordinary fp32 adds.
//
// Work: the chunks of all items in a row, cut into equal parts, one per warp of
// a grid that fills the GPU, whatever the lengths.  A part that holds a whole
// item writes its output; the others leave (m, l, o) for attn_paged_join_kernel.
// Warps share nothing: each streams K and V chunks through its own ring of
// shared-memory slots with 16-byte asynchronous copies, across items, without a
// barrier.  The order of every sum is fixed by lengths and grid.
//
// Why not the fifth-generation tensor cores: the work is bound by memory (F16) or by
// taking codes apart (block types), not by products (hmma pipe at 0.10 to 0.17), and
// their operands would have to pass through shared memory once more.
//
// Measured on B200, 32 query heads over 8 KV heads of 128, with the join: one fp16
// sequence of 131071 positions 88 us (6.1 TB/s, 0.93 of a copy's bandwidth; without
// the join 84); Q8_0 54 us (0.81), Q4_0 54.5 us (0.42: 940 instructions a chunk of 32
// positions, issue at 0.61); 64 sequences of 1 to 8191 positions in Q8_0 39 us
// (0.71).  Before items' starts counted as work the longest-running SM of that batch
// took 80 k cycles where the others took 64 k.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_fill(uint32_t dst, const void* src, int valid_bytes) {  // then zeros
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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8x8 matrix of 16-bit elements, a row in 4 lanes
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldsm2_trans(uint32_t a, uint32_t r[2]) {  // two: addresses of lanes 0-15
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a));
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  float d0, d1, d2, d3;
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d0), "=f"(d1), "=f"(d2), "=f"(d3)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  c[0] = d0; c[1] = d1; c[2] = d2; c[3] = d3;
}
__device__ __forceinline__ void mma16816_first(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

constexpr int kMaxTile = 16;  // heads of a tile at most: a part is (m, l)[16], o[heads][D]
__host__ __device__ constexpr int paged_part_floats(int rows, int D) { return rows * D + 2 * kMaxTile; }

// Positions per chunk, ring slots (one K or V chunk each) and CTAs per SM.  A chunk is
// 2 to 8 KiB of keys: 64 positions of the narrow rows (131071 positions of 4 KV
// heads of 64 in Q8_0 in 26.4 us, 28.1 with 32; of 8 of 128 in 4 bits 53.7 and 54.6; not
// for a cluster to an item, where 32 positions are 5.6 us at 480 and 64 are 7.2), 16 of
// fp16 rows of 256.  The CTAs are those whose registers need no spills to speak of: 12
// warps of Q8_0 at 168 registers read the ragged batch of 64 sequences in 39 us, 16 at
// 128 in 41, and 131071 positions in 57 where 16 take 65.
template <int T, int D, int NC, bool ONE>
struct PagedCfg {
  static constexpr int ROW = kv_row_bytes<T>(D);
  static constexpr int CH = ROW <= 72 && D * NC <= 128 && !ONE ? 64 : ROW <= 272 ? 32 : 16;
  static constexpr int SLOTS = 3;
  static constexpr int FOURS = (D == 256 || (T == kKvF16 && D == 128)) ? 2 : D * NC <= 64 ? 4 : NC <= 2 ? 3 : 2;
  static constexpr int WARPS = ONE ? 8 : 4, CTAS = ONE ? FOURS / 2 : FOURS;
  static constexpr int HEADS = 4 * NC;                     // query heads of a tile
  static constexpr int CB = kv_code_bytes<T>(D);           // bytes of a row's codes
  static constexpr int SB = T == kKvF16 ? 0 : D / 16;      // bytes of a row's scales
  static constexpr int SLOT = CH * (CB + SB);
  static constexpr int PART = 4 * paged_part_floats(HEADS, D);  // bytes of a part
  static constexpr int RING = WARPS * SLOTS * SLOT, PARTS = (WARPS + 1) * PART;  // the warps' and the CTA's
  static constexpr int SMEM = ONE && PARTS > RING ? PARTS : RING;
};

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

// A place in the row of all chunks: chunk `ci` of `n` of row tile `rt` of KV head
// `kvh` of sequence `s`.
struct PagedCursor {
  int s, kvh, rt, ci, n, len;
  __device__ __forceinline__ void next(const ntx_paged_kv& c, const int* lens, int rtiles, int ch, int* status) {
    if (++ci < n) return;
    ci = 0;
    if (++rt < rtiles) return;
    rt = 0;
    if (++kvh < c.n_kv_heads) return;
    kvh = 0;
    do {
      if (++s >= c.n_seqs) { n = 0; return; }
      len = seq_len(c, lens, s, status);
      n = (len + ch - 1) / ch;
    } while (n == 0);
  }
};

// Work is counted in units: each chunk one, and kItemUnits more for the start of
// each item (q's fragments, an output to write).  W units in consecutive parts for
// at most `warps` warps, sizes differing by one at most.
constexpr int kItemUnits = 1;
struct PagedParts {
  int n;
  int64_t size, longer;  // the first `longer` parts have size + 1 units
  PagedParts() = default;
  __device__ __forceinline__ PagedParts(int64_t W, int warps) : n((int)min64(W, warps)), size(0), longer(0) {
    if (n == 0) return;
    size = W >> 31 ? W / n : (int)W / n;  // (64-bit divisions only where they are needed)
    longer = W - size * n;
  }
  __device__ __forceinline__ int64_t begin(int w) const { return w * size + min64(w, longer); }
  __device__ __forceinline__ int holder(int64_t unit) const {  // the part of a unit
    const int64_t head = longer * (size + 1);
    if (unit < head) return (int)((unit | size) >> 30 ? unit / (size + 1) : (int)unit / (int)(size + 1));
    unit -= head;
    return (int)(longer + ((unit | size) >> 30 ? unit / size : (int)unit / (int)size));
  }
};
// Units of each of a sequence's items.
__device__ __forceinline__ int item_units(int chunks) { return chunks ? chunks + kItemUnits : 0; }

// Units of the items of k consecutive sequences to a lane (`mine`) and of all up to and with them.
__device__ __forceinline__ int64_t lane_units(const ntx_paged_kv& c, const int* lens, int k, int ch, int tiles,
                                              int64_t& mine, int* status) {
  const int lane = threadIdx.x & 31;
  mine = 0;
  for (int i = 0; i < k; ++i)
    if (lane * k + i < c.n_seqs) mine += item_units((seq_len(c, lens, lane * k + i, status) + ch - 1) / ch);
  mine *= tiles;
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  return upto;
}

// ONE: a cluster of 1 to 8 CTAs to an item, whose warps share its chunks out and join
// through shared memory, the CTAs through the cluster's, in one launch.  Taken where all
// clusters of as many CTAs as give each warp one chunk of the longest sequence that the
// table can hold, or of 8, or as many as there is room for, are resident at once, and for
// tables of at most kOneCtaCtx positions for each of the CTAs.  A group of more than four
// query heads is cut into tiles of four where a warp's positions times heads are no more
// for it: with more clusters, of shorter chains of instructions, which is what a warp
// with one chunk takes its time for.  Against parts and their join, 8 KV heads of 128 in
// Q8_0, us on the device:
//   32 query heads, 1 sequence of 145 / 480 / 2049 / 4000 / 6000 / 8000:
//     4.6 / 5.6 / 7.6 / 8.3 / 10.1 / 11.8 against 7.5 / 8.2 / 9.0 / 9.9 / 10.6 / 12.0
//   64 query heads, 1 of 145 / 1000 / 2049 / 4000 / 6000:
//     4.8 / 6.2 / 7.7 / 10.1 / 12.0 against 8.8 / 9.7 / 10.6 / 12.0 / 13.2 (tiles of eight:
//     6.2 / 7.8 / 9.7 / 10.5 / 12.8)
//   3 of 1000 / 2049 / 4000: 6.2 / 8.1 / 11.3 against 9.1 / 10.8 / 13.1
//   8 of 1000: 8.3 against 11.6; 16 of 480: 7.0 against 11.5
//   1 of 15000: 18.1 against 13.9; 64 of 1 to 400: 19.5 against 13.5 (more items than SMs)
//   one long sequence among short ones waits for its own warps: 7, 91 and 4000: 11.3
//   against 9.7, 3, 4000 and 564: 11.1 against 9.5 (F16 9.9 against 9.6, Q4_0 11.1 against
//   11.3), 4000, 2595 and 2: 11.0 against 10.6
constexpr int kOneCtaCtx = 1024;

template <int T, int D, int NC, bool ONE>
__global__ void __launch_bounds__(PagedCfg<T, D, NC, ONE>::WARPS * 32, PagedCfg<T, D, NC, ONE>::CTAS)
    attn_paged_kernel(const ntx_paged_kv c, const float* __restrict__ q, int64_t qs, float* __restrict__ out,
                      int4* __restrict__ split, float* __restrict__ part, int Hq, const int* __restrict__ lens,
                      float scale, int* status) {
  using F = PagedCfg<T, D, NC, ONE>;
  constexpr int CH = F::CH, C = F::CB / 16, NB = D / 32, NS = CH / 16, NT = D / 16;
  extern __shared__ __align__(128) uint8_t ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t slots = smem_addr(ring) + warp * (F::SLOTS * F::SLOT);
  const int G = Hq / c.n_kv_heads, rtiles = (G + F::HEADS - 1) / F::HEADS;
  const int tiles = c.n_kv_heads * rtiles;
  const int wid = blockIdx.x * F::WARPS + warp, all_warps = gridDim.x * F::WARPS;
  if constexpr (!ONE) {
    pdl_launch_dependents();  // the join's CTAs prepare themselves where there is room
    // empty sequences: zeros
    for (int s = wid; s < c.n_seqs; s += all_warps)
      if (__ldg(lens + s) <= 0)
        for (int64_t i = lane; i < (int64_t)Hq * D / 4; i += 32)
          reinterpret_cast<float4*>(out + (int64_t)s * Hq * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  __shared__ PagedParts s_parts[F::WARPS];
  constexpr int kStart = ONE ? 0 : kItemUnits;

  // ---- this warp's part: its first chunk, and `todo` units from there
  PagedCursor cur;
  int64_t todo;
  const int ctas = ONE ? (int)cooperative_groups::this_cluster().num_blocks() : 1;  // of an item
  const int rank = ONE ? (int)cooperative_groups::this_cluster().block_rank() : 0;
  if constexpr (ONE) {
    const int item = blockIdx.x / ctas;
    cur.s = item / tiles;
    const int tile = item - cur.s * tiles;
    cur.kvh = tile / rtiles;
    cur.rt = tile - cur.kvh * rtiles;
    cur.len = seq_len(c, lens, cur.s, status);
    cur.n = (cur.len + CH - 1) / CH;
    const int w = rank * F::WARPS + warp, warps = ctas * F::WARPS;
    cur.ci = w * cur.n / warps;
    todo = (w + 1) * cur.n / warps - cur.ci;
  } else {
    const int k = (c.n_seqs + 31) >> 5;  // sequences to a lane
    int64_t mine;
    const int64_t upto = lane_units(c, lens, k, CH, tiles, mine, status);
    const PagedParts parts(__shfl_sync(0xffffffffu, upto, 31), all_warps);
    // what the parts of this warp's slots belong to, for the join: nothing yet
    if (lane < 2) split[2 * wid + lane] = make_int4(0, 0, 0, 0);
    if (wid >= parts.n) return;
    s_parts[warp] = parts;
    const int64_t u0 = parts.begin(wid);
    todo = parts.begin(wid + 1) - u0;
    const int at = __ffs(__ballot_sync(0xffffffffu, upto > u0)) - 1;  // the lane whose sequences hold u0
    int64_t rest = u0 - __shfl_sync(0xffffffffu, upto - mine, at);
    cur.s = at * k;
    int units;
    for (;;) {
      cur.len = seq_len(c, lens, cur.s, status);
      cur.n = (cur.len + CH - 1) / CH;
      units = item_units(cur.n);
      if (rest < (int64_t)units * tiles) break;
      rest -= (int64_t)units * tiles;
      ++cur.s;
    }
    const int tile = (int)(rest >> 31 ? rest / units : (int)rest / units);
    const int in_item = (int)(rest - (int64_t)tile * units);
    cur.ci = max(0, in_item - kItemUnits);
    cur.kvh = tile / rtiles;
    cur.rt = tile - cur.kvh * rtiles;
    todo -= max(0, kItemUnits - in_item);
    if (todo <= 0) return;
  }
  bool item_head = cur.ci == 0;  // false: the part begins inside an item
  const bool empty = cur.len <= 0;
  const int item_s = cur.s;

  // ---- loading: the ring's next slot takes K or V of chunk `ld`, 16 rows (one page) at a time
  const int64_t head_bytes = (int64_t)c.page_size * kv_row_bytes<T>(D), scales_at = (int64_t)c.page_size * F::CB;
  PagedCursor ld = cur;
  int64_t ld_left = todo;
  uint32_t ld_slot = slots;
  int ld_j, ld_row, ld_page[NS], ld_first[NS];  // next page index and row in it; pages and first rows of chunk `ld`
  auto look_up = [&](bool item) {
    if (item) {
      ld_j = ld.ci * CH / c.page_size;
      ld_row = ld.ci * CH - ld_j * c.page_size;
      const int h0 = F::HEADS * ld.rt;  // its query heads are read a chunk from now
      const float* qp = q + ld.s * qs + (int64_t)(ld.kvh * G + h0) * D;
      for (int i = lane; i < min(F::HEADS, G - h0) * (D / 32); i += 32)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(qp + 32 * i));
    }
    const int* row = c.page_table + (int64_t)ld.s * c.max_pages;
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      ld_first[r] = ld_row;
      ld_page[r] = ld.ci * CH + 16 * r < ld.len &&
                           chk(status, kChkPagedTable, (int64_t)ld.s * c.max_pages + ld_j, (int64_t)c.n_seqs * c.max_pages)
                       ? __ldg(row + ld_j)
                       : -1;
      if ((ld_row += 16) == c.page_size) {
        ld_row = 0;
        ++ld_j;
      }
    }
  };
  look_up(true);
  // This lane's 16-byte pieces of 16 rows of C columns: row i (32/C) + lane/C, column
  // lane % C; i changes only bits 4 to 6 of the swizzled place besides its row's start.
  const uint32_t lane_off = lane * 16;
  const uint32_t lane_k = lane / C * F::CB + swz_k<T, C>(lane / C, lane % C) * 16;
  const uint32_t lane_v = lane / C * F::CB + swz8<C>(lane / C, lane % C) * 16;
  int64_t ld_at[NS];  // byte offset of this lane's first piece in either pool
  int ld_rows[NS];    // rows to copy, the others are zeros
  auto load = [&](auto is_v) {
    constexpr bool V = decltype(is_v)::value;
    if (ld_left > 0) {
      const uint8_t* pool = static_cast<const uint8_t*>(V ? c.v_pages : c.k_pages);
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        if constexpr (!V) {
          int rows = ld.len - (ld.ci * CH + 16 * r), page = ld_page[r];
          if (rows > 0 && (unsigned)page >= (unsigned)c.n_pages) {
            if (lane == 0) bad_page(status);
            rows = 0;
          }
          if constexpr (kCheck) {  // (debug build) the rows' last code and scale, and their slot
            const int64_t part = ((int64_t)page * c.n_kv_heads + ld.kvh) * head_bytes, end = ld_first[r] + min(rows, 16);
            if (rows > 0 && !(chk(status, kChkPagedLoad, part + end * F::CB - 1, kv_pool_bytes<T, D>(c)) &&
                              chk(status, kChkPagedLoad, part + scales_at + end * F::SB - 1, kv_pool_bytes<T, D>(c))))
              rows = 0;
          }
          if (rows <= 0) page = 0;
          ld_rows[r] = rows;
          ld_at[r] = ((int64_t)page * c.n_kv_heads + ld.kvh) * head_bytes + lane_off;
        }
        const uint8_t* codes = pool + ld_at[r] + (int64_t)ld_first[r] * F::CB;
        const uint8_t* sc = pool + ld_at[r] + (scales_at + (int64_t)ld_first[r] * F::SB);
        const uint32_t dst = ld_slot + 16 * r * F::CB + (V ? lane_v : lane_k);
        const uint32_t dst_sc = ld_slot + CH * F::CB + r * 16 * F::SB + lane_off;
        auto place = [&](int i) {
          constexpr int RPI = C >= 32 ? 1 : 32 / C;  // rows per i
          return (dst ^ ((V ? swz8<C>(i * RPI, 0) : swz_k<T, C>(i * RPI, 0)) * 16)) + i * RPI * F::CB;
        };
        // (debug build) a piece's place inside its slot's codes, or scales, and the slot inside the ring
        auto in_slot = [&](uint32_t to, int first, int end) {
          return chk(status, kChkPagedSlot, (int64_t)to - ld_slot - first, end - first - 15) &&
                 chk(status, kChkPagedSlot, (int64_t)ld_slot - smem_addr(ring) + F::SLOT - 1, F::RING);
        };
        constexpr int kCodes = CH * F::CB;
        if (ld_rows[r] >= 16) {
#pragma unroll
          for (int i = 0; i < C / 2; ++i)
            if (in_slot(place(i), 0, kCodes)) cp_async16(place(i), codes + i * 512);
          if (F::SB > 0 && lane < F::SB && in_slot(dst_sc, kCodes, F::SLOT)) cp_async16(dst_sc, sc);
        } else {
#pragma unroll
          for (int i = 0; i < C / 2; ++i) {
            const bool on = i * (32 / C) + lane / C < ld_rows[r];
            if (in_slot(place(i), 0, kCodes)) cp_async16_fill(place(i), on ? codes + i * 512 : pool, on ? 16 : 0);
          }
          if (F::SB > 0 && lane < F::SB && in_slot(dst_sc, kCodes, F::SLOT)) {
            const int valid = max(0, min(16, ld_rows[r] * F::SB - lane * 16));
            cp_async16_fill(dst_sc, valid ? sc : pool, valid);
          }
        }
      }
      ld_slot = ld_slot + F::SLOT == slots + F::SLOTS * F::SLOT ? slots : ld_slot + F::SLOT;
      if constexpr (V) {
        // the pages of the next chunk are used half a chunk from now
        if (--ld_left > 0) {
          const bool item = ld.ci + 1 == ld.n;
          if (item) ld_left -= kStart;
          if (ld_left > 0) {
            ld.next(c, lens, rtiles, CH, status);
            look_up(item);
          }
        }
      }
    }
    cp_async_commit();
  };
  uint32_t slot = slots;
  auto next_slot = [&]() { slot = slot + F::SLOT == slots + F::SLOTS * F::SLOT ? slots : slot + F::SLOT; };
  constexpr std::false_type kK{};
  constexpr std::true_type kV{};
  load(kK);
  load(kV);
  static_assert(F::SLOTS == 3);  // while K (V) of a chunk is used, K (V) of the next is loaded

  // scales of a row, two blocks a word
  auto scales = [&](uint32_t row, uint32_t sc[NB / 2]) {
    const uint32_t a = slot + CH * F::CB + row * F::SB;
    if constexpr (NB == 2) {
      sc[0] = lds32(a);
    } else if constexpr (NB == 4) {
      const uint2 v = lds64(a);
      sc[0] = v.x; sc[1] = v.y;
    } else {
      const uint4 v = lds128(a);
      sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
    }
  };

  // p is kept 2^kPBits fold, in l and o too
  constexpr float kPBits = T == kKvF16 ? 14.f : 10.f;
  // This lane's heads: t of column tile c as a softmax row (with positions g, g + 8 of 16)
  // and in o (with two elements of 16); g / 2 in q's fragments.
  uint32_t qf[NC][NB][4];
  float o[NC][NT][2], m[NC], l[NC], to_log2[NC];
  bool fresh = true;
  int rows = min(F::HEADS, G - F::HEADS * cur.rt), head0 = cur.kvh * G + F::HEADS * cur.rt;
  if constexpr (ONE) {  // a warp without a chunk
#pragma unroll
    for (int ct = 0; ct < NC; ++ct) {
      m[ct] = -INFINITY;
      l[ct] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[ct][n][0] = o[ct][n][1] = 0.f;
    }
  }
  auto in_out = [&](int s, int head) {  // (debug build) a row of the output
    return chk(status, kChkPagedOut, s, c.n_seqs) && chk(status, kChkPagedOut, head, Hq);
  };
  // this lane's elements of o, times f, to a row
  auto store = [&](int ct, float* dst, float f) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (T == kKvF16) {
        dst[16 * n + g] = o[ct][n][0] * f;
        dst[16 * n + 8 + g] = o[ct][n][1] * f;
      } else {
        *reinterpret_cast<float2*>(dst + 16 * n + 2 * g) = make_float2(o[ct][n][0] * f, o[ct][n][1] * f);
      }
    }
  };

  while (todo > 0) {
    if (fresh) {  // ---- an item's q, while its first keys are on the way
      rows = min(F::HEADS, G - F::HEADS * cur.rt);
      head0 = cur.kvh * G + F::HEADS * cur.rt;
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        const int h = 4 * ct + (g >> 1);
        const float* qp = q + cur.s * qs + (int64_t)(head0 + h) * D;
        // The two lanes of a head's columns (one keeps the upper parts, one the remainders) form every other block
        // each, and exchange.
        const int odd = g & 1;
        float x[NB / 2][8], top = 0.f;
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
          const float* p = qp + 32 * (2 * i + odd);
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
          if (h < rows) {
            u = ldg4(p + (T == kKvQ4 ? 4 * t : 8 * t));
            v = ldg4(p + (T == kKvQ4 ? 16 + 4 * t : 8 * t + 4));
          }
          x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
          x[i][4] = v.x; x[i][5] = v.y; x[i][6] = v.z; x[i][7] = v.w;
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[i][j]));
        }
#pragma unroll
        for (int y = 1; y < 8; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
        // 2^e with top 2^e in [2^13, 2^14), as far as fp32 has it; 1 for infinities
        const int eb = __float_as_int(top) >> 23;
        const int es = eb == 255 ? 127 : min(254, 267 - eb);
        const float up = __int_as_float(es << 23);
        const float down = es == 254 ? __int_as_float(0x00400000) : __int_as_float((254 - es) << 23);
        to_log2[ct] = __shfl_sync(0xffffffffu, scale * down * 1.44269504088896340736f, 8 * t);
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // the pairs that a key fragment of this type has: elements 0 1, 2 3, ... or 0 2, 1 3, ... of this lane's
            const int j0 = T == kKvQ4 ? 4 * (j >> 1) + (j & 1) : 2 * j, j1 = T == kKvQ4 ? j0 + 2 : j0 + 1;
            uint32_t hi, lo;
            split2(x[i][j0] * up, x[i][j1] * up, hi, lo);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? hi : lo, 4);
            qf[ct][2 * i][j] = odd ? other : hi;
            qf[ct][2 * i + 1][j] = odd ? lo : other;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) o[ct][n][0] = o[ct][n][1] = 0.f;
        m[ct] = -INFINITY;
        l[ct] = 0.f;
      }
      fresh = false;
    }

    // ---- scores
    cp_async_wait<F::SLOTS - 2>();
    __syncwarp();
    load(kK);

    float s[NC][NS][2];
    if constexpr (T == kKvF16) {
      float acc[NC][NS][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const uint32_t a = slot + (16 * k + g) * F::CB + swz_k<T, C>(g, 4 * b + t) * 16;
          const uint4 u = lds128(a), v = lds128(a + 8 * F::CB);
          const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
          for (int ct = 0; ct < NC; ++ct) {
            if (b == 0) mma16816_first(acc[ct][k], a0, qf[ct][b][0], qf[ct][b][1]);
            else mma16816(acc[ct][k], a0, qf[ct][b][0], qf[ct][b][1]);
            mma16816(acc[ct][k], a1, qf[ct][b][2], qf[ct][b][3]);
          }
        }
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          s[ct][k][0] = acc[ct][k][0] + acc[ct][k][1];
          s[ct][k][1] = acc[ct][k][2] + acc[ct][k][3];
        }
    } else {
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        uint32_t sc[2][NB / 2];
        scales(16 * k + g, sc[0]);
        scales(16 * k + g + 8, sc[1]);
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) s[ct][k][0] = s[ct][k][1] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t a0[4], a1[4];
          if constexpr (T == kKvQ8) {
            const uint32_t a = slot + (16 * k + g) * F::CB + swz_k<T, C>(g, 2 * b + (t >> 1)) * 16 + (t & 1) * 8;
            uint2 u = lds64(a), v = lds64(a + 8 * F::CB);
            u.x ^= 0x80808080u; u.y ^= 0x80808080u; v.x ^= 0x80808080u; v.y ^= 0x80808080u;
            a0[0] = bytes_h2<0x4140>(u.x); a0[1] = bytes_h2<0x4140>(v.x);
            a0[2] = bytes_h2<0x4342>(u.x); a0[3] = bytes_h2<0x4342>(v.x);
            a1[0] = bytes_h2<0x4140>(u.y); a1[1] = bytes_h2<0x4140>(v.y);
            a1[2] = bytes_h2<0x4342>(u.y); a1[3] = bytes_h2<0x4342>(v.y);
          } else {
            const uint32_t a = slot + (16 * k + g) * F::CB + swz_k<T, C>(g, b) * 16 + 4 * t;
            const uint32_t u = lds32(a), v = lds32(a + 8 * F::CB), u8 = u >> 8, v8 = v >> 8;
            a0[0] = nib_lo(u); a0[1] = nib_lo(v); a0[2] = nib_lo(u8); a0[3] = nib_lo(v8);
            a1[0] = nib_hi(u); a1[1] = nib_hi(v); a1[2] = nib_hi(u8); a1[3] = nib_hi(v8);
          }
          float d[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = __half22float2(bits_h2(sc[i][b / 2]));
            d[i] = (b & 1) ? f.y : f.x;
          }
#pragma unroll
          for (int ct = 0; ct < NC; ++ct) {
            float acc[4];
            mma16816_first(acc, a0, qf[ct][b][0], qf[ct][b][1]);
            mma16816(acc, a1, qf[ct][b][2], qf[ct][b][3]);
            s[ct][k][0] = fmaf(acc[0] + acc[1], d[0], s[ct][k][0]);
            s[ct][k][1] = fmaf(acc[2] + acc[3], d[1], s[ct][k][1]);
          }
        }
      }
    }
    next_slot();

    // ---- softmax of the chunk
    const int left = cur.len - cur.ci * CH;  // positions the chunk has
#pragma unroll
    for (int ct = 0; ct < NC; ++ct) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[ct][k][i] *= to_log2[ct];
          top = fmaxf(top, s[ct][k][i]);
        }
      if (left < CH) {  // behind the sequence
        top = -INFINITY;
#pragma unroll
        for (int k = 0; k < NS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (16 * k + 8 * i + g >= left) s[ct][k][i] = -INFINITY;
            top = fmaxf(top, s[ct][k][i]);
          }
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float m_new = fmaxf(m[ct], top), zero = m_new == -INFINITY ? 0.f : m_new, base = zero - kPBits;
      const float fade = ex2(m[ct] - zero);
      m[ct] = m_new;
      l[ct] *= fade;
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[ct][k][i] = ex2(s[ct][k][i] - base);
          l[ct] += s[ct][k][i];
        }
      if (__any_sync(0xffffffffu, fade != 1.f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[ct][n][0] *= fade;
          o[ct][n][1] *= fade;
        }
      }
    }

    // ---- weighted values
    cp_async_wait<F::SLOTS - 2>();
    __syncwarp();
    load(kV);
    if constexpr (T == kKvF16) {
      uint32_t p[NC][NS][2];
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          uint32_t hi, lo;
          split2(s[ct][k][0], s[ct][k][1], hi, lo);
          p[ct][k][0] = transpose8(__byte_perm(hi, lo, 0x5410));
          p[ct][k][1] = transpose8(__byte_perm(hi, lo, 0x7632));
        }
      // ldmatrix rows: positions 0-7 of two columns, then 8-15 of them
      const int lr = (lane & 7) + ((lane >> 4) << 3), lc = (lane >> 3) & 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t v[NS][4];
#pragma unroll
        for (int k = 0; k < NS; ++k) ldsm4_trans(slot + (16 * k + lr) * F::CB + swz8<C>(lr, 2 * n + lc) * 16, v[k]);
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
          float a[4];
          mma16816_first(a, v[0], p[ct][0][0], p[ct][0][1]);
#pragma unroll
          for (int k = 1; k < NS; ++k) mma16816(a, v[k], p[ct][k][0], p[ct][k][1]);
          o[ct][n][0] += a[0] + a[1];
          o[ct][n][1] += a[2] + a[3];
        }
      }
    } else {
      uint32_t sc[NS][2][NB / 2];
      __half2 big = __float2half2_rn(0.f);
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          scales(16 * k + 8 * i + g, sc[k][i]);
#pragma unroll
          for (int b = 0; b < NB / 2; ++b) big = __hmax2(big, __habs2(bits_h2(sc[k][i][b])));
        }
      uint32_t u = h2_bits(big);
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) u = h2_bits(__hmax2(bits_h2(u), bits_h2(__shfl_xor_sync(0xffffffffu, u, x))));
      const int e = (int)max(u & 0xFFFFu, u >> 16) >> 10;
      // The largest scale is in [2^(e - 15), 2^(e - 14)), subnormal or infinite; times 2^up it
      // comes to [2^4, 2^5).  What is beyond 2^15 goes to p.
      const int up = min(15, 19 - e);
      const float down = __int_as_float((127 - 19 + e) << 23);
      const __half2 by = bits_h2((uint32_t)(up + 15) * 0x04000400u);
      __half2 ph[NC][NS], pl[NC][NS];
#pragma unroll
      for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const float f = e < 4 ? __int_as_float((127 + 4 - e) << 23) : 1.f;
          uint32_t hi, lo;
          split2(s[ct][k][0] * f, s[ct][k][1] * f, hi, lo);
          ph[ct][k] = bits_h2(hi);
          pl[ct][k] = bits_h2(lo);
        }
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int b = 0; b < NB / 2; ++b) sc[k][i][b] = h2_bits(__hmul2(bits_h2(sc[k][i][b]), by));
      const int lr = lane & 15, lc = lane >> 4;  // ldmatrix rows: 16 positions, then those of the next column
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float a[NC][2][4];
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          // value fragments: rows g and g + 8 are elements 2 g and 2 g + 1 of 16
          uint32_t v[2][4];
          if constexpr (T == kKvQ8) {
            uint32_t r[4];
            ldsm4_trans(slot + (16 * k + lr) * F::CB + swz8<C>(lr, 2 * b + lc) * 16, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[i] ^= 0x80808080u;
              v[i >> 1][2 * (i & 1)] = bytes_h2<0x4240>(r[i]);
              v[i >> 1][2 * (i & 1) + 1] = bytes_h2<0x4341>(r[i]);
            }
          } else {
            uint32_t r[2];
            ldsm2_trans(slot + (16 * k + lr) * F::CB + swz8<C>(lr, b) * 16, r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t r8 = r[i] >> 8;
              v[0][2 * i] = nib_lo(r[i]);
              v[0][2 * i + 1] = nib_lo(r8);
              v[1][2 * i] = nib_hi(r[i]);
              v[1][2 * i + 1] = nib_hi(r8);
            }
          }
          const __half2 d = bits_h2(__byte_perm(sc[k][0][b / 2], sc[k][1][b / 2], (b & 1) ? 0x7632 : 0x5410));
#pragma unroll
          for (int ct = 0; ct < NC; ++ct) {
            // p d of positions g, g + 8, in two numbers again
            const __half2 hi = __hmul2(ph[ct][k], d);
            const __half2 rest = __hfma2(ph[ct][k], d, __hneg2(hi));  // exact
            const uint32_t x = h2_bits(hi), y = h2_bits(__hfma2(pl[ct][k], d, rest));
            const uint32_t p0 = transpose8(__byte_perm(x, y, 0x5410)), p1 = transpose8(__byte_perm(x, y, 0x7632));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (k == 0) mma16816_first(a[ct][i], v[i], p0, p1);
              else mma16816(a[ct][i], v[i], p0, p1);
            }
          }
        }
#pragma unroll
        for (int ct = 0; ct < NC; ++ct)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[ct][2 * b + i][0] = fmaf(a[ct][i][0] + a[ct][i][1], down, o[ct][2 * b + i][0]);
            o[ct][2 * b + i][1] = fmaf(a[ct][i][2] + a[ct][i][3], down, o[ct][2 * b + i][1]);
          }
      }
    }
    next_slot();

    // ---- end of an item, or of this warp's part
    --todo;
    const bool item_end = cur.ci + 1 == cur.n;
    if constexpr (!ONE) {
      if (item_end) todo -= kItemUnits;
      if (item_end || todo <= 0) {
        const bool whole = item_end && item_head;
        // slot 1: an item that this part begins, for others to end; slot 0: one that another part began
        const int64_t at = 2ll * wid + (item_head ? 1 : 0);
        float* p = part + at * paged_part_floats(min(F::HEADS, G), D);
        // the item's first warp and number of parts, where its output goes
        if (!whole && lane == 0 && chk(status, kChkPagedPart, at, 2ll * all_warps)) {
          const PagedParts parts = s_parts[warp];
          // units up to the chunk after this one, less the item's own
          const int64_t first = parts.begin(wid + 1) - max((int64_t)0, todo + (item_end ? kItemUnits : 0)) - cur.ci - 1;
          const int w0 = parts.holder(first), n_parts = parts.holder(first + cur.n - 1) - w0 + 1;
          split[at] = make_int4(w0, n_parts, cur.s, (head0 << 5) | rows);
        }
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
          const int h = 4 * ct + t;
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[ct] += __shfl_xor_sync(0xffffffffu, l[ct], x);
          if (h >= rows) continue;
          if (whole) {
            if (in_out(cur.s, head0 + h)) store(ct, out + ((int64_t)cur.s * Hq + head0 + h) * D, 1.f / l[ct]);
          } else if (chk(status, kChkPagedPart, at, 2ll * all_warps) && chk(status, kChkPagedPart, h, min(F::HEADS, G))) {
            if (g == 0) *reinterpret_cast<float2*>(p + 2 * h) = make_float2(m[ct], l[ct]);
            store(ct, p + 2 * kMaxTile + h * D, 1.f);
          }
        }
        if (todo <= 0) break;
        item_head = true;
        fresh = true;
      }
    }
    cur.next(c, lens, rtiles, CH, status);
  }
  cp_async_wait<0>();

  if constexpr (ONE) {
    static_assert(F::WARPS == 8);
    auto at = [&](int w) { return reinterpret_cast<float*>(ring + w * F::PART); };
    auto in_part = [&](int w, int h) {  // (debug build) a row of a part
      return chk(status, kChkPagedPart, (w + 1ll) * F::PART - 1, F::SMEM) && chk(status, kChkPagedPart, h, F::HEADS);
    };
    __syncthreads();  // every warp is done with its ring
#pragma unroll
    for (int ct = 0; ct < NC; ++ct) {
      const int h = 4 * ct + t;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[ct] += __shfl_xor_sync(0xffffffffu, l[ct], x);
      if (h >= rows || !in_part(warp, h)) continue;
      if (g == 0) *reinterpret_cast<float2*>(at(warp) + 2 * h) = make_float2(m[ct], l[ct]);
      store(ct, at(warp) + 2 * kMaxTile + h * D, 1.f);
    }
    __syncthreads();
    // parts `at(0)` to `at(n - 1)`, 8 at most, joined: elements 4 i to 4 i + 3 of the item's rows, and the row's (m, l)
    auto join = [&](auto part_at, int n, int i, float2& ml) {
      const int h = i / (D / 4);
      float M = -INFINITY;
      float2 x[8];
      float4 y[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        x[w] = make_float2(-INFINITY, 0.f);
        y[w] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w < n) {
          const float* p = part_at(w);
          x[w] = *reinterpret_cast<const float2*>(p + 2 * h);
          y[w] = reinterpret_cast<const float4*>(p + 2 * kMaxTile)[i];
        }
        M = fmaxf(M, x[w].x);
      }
      const float base = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float f = ex2(x[w].x - base);
        L = fmaf(x[w].y, f, L);
        O.x = fmaf(y[w].x, f, O.x); O.y = fmaf(y[w].y, f, O.y); O.z = fmaf(y[w].z, f, O.z); O.w = fmaf(y[w].w, f, O.w);
      }
      ml = make_float2(M, L);
      return O;
    };
    auto finish = [&](int i, float4 O, float L) {
      if (!in_out(item_s, head0 + i / (D / 4))) return;
      const float f = empty ? 0.f : 1.f / L;  // an empty sequence: zeros
      reinterpret_cast<float4*>(out + ((int64_t)item_s * Hq + head0) * D)[i] =
          make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
    };
    const int pieces = rows * (D / 4);
    float2 ml;
    if (ctas == 1) {
      for (int i = threadIdx.x; i < pieces; i += F::WARPS * 32) {
        const float4 O = join(at, F::WARPS, i, ml);
        finish(i, O, ml.y);
      }
    } else {
      // the CTA's part, then every CTA joins its share of the cluster's
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      float* own = at(F::WARPS);
      for (int i = threadIdx.x; i < pieces; i += F::WARPS * 32) {
        const float4 O = join(at, F::WARPS, i, ml);
        if (!in_part(F::WARPS, i / (D / 4))) continue;
        reinterpret_cast<float4*>(own + 2 * kMaxTile)[i] = O;
        if (i % (D / 4) == 0) *reinterpret_cast<float2*>(own + 2 * (i / (D / 4))) = ml;
      }
      cluster.sync();
      for (int i = rank * F::WARPS * 32 + threadIdx.x; i < pieces; i += ctas * F::WARPS * 32) {
        const float4 O = join([&](int r) { return (const float*)cluster.map_shared_rank(own, r); }, ctas, i, ml);
        finish(i, O, ml.y);
      }
      cluster.sync();  // nobody's shared memory goes before it has been read
    }
  }
}

// Joins the parts of the items that several warps hold: with M the largest m,
// out = sum 2^(m - M) o / sum 2^(m - M) l.  There is a CTA for every warp of the main
// kernel, and an item's output is shared out among the CTAs of its parts.  By their
// number a warp takes a head's whole row, all parts at once; or 32 elements of it,
// four parts for every element; or a CTA 16 elements of it, 32 parts for every one.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 8, kManyParts = 64;
constexpr int kMaxPagedSeqs = 1024;

struct PagedMerge {  // a running join of parts, four elements a thread
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void scale_to(float m) {
    const float f = ex2(M - (m == -INFINITY ? 0.f : m));
    M = m;
    L *= f;
    O.x *= f; O.y *= f; O.z *= f; O.w *= f;
  }
  __device__ __forceinline__ void add(float m, float l, float4 o) {  // M is at least m
    const float f = ex2(m - (M == -INFINITY ? 0.f : M));
    L = fmaf(l, f, L);
    O.x = fmaf(o.x, f, O.x); O.y = fmaf(o.y, f, O.y); O.z = fmaf(o.z, f, O.z); O.w = fmaf(o.w, f, O.w);
  }
  // parts first, first + step, ... below n; at(i) is part i, e the four elements in it, of head `row`
  template <class At>
  __device__ __forceinline__ void parts(At at, int first, int step, int n, int row, int e) {
    constexpr int BATCH = 8;
    for (int i0 = first; i0 < n; i0 += step * BATCH) {
      float2 ml[BATCH];
      float4 o[BATCH];
      float top = M;
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        ml[b] = make_float2(-INFINITY, 0.f);
        o[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int i = i0 + b * step;
        if (i < n) {
          const float* p = at(i);
          ml[b] = *reinterpret_cast<const float2*>(p + 2 * row);
          o[b] = *reinterpret_cast<const float4*>(p + e);
        }
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) top = fmaxf(top, ml[b].x);
      scale_to(top);
#pragma unroll
      for (int b = 0; b < BATCH; ++b) add(ml[b].x, ml[b].y, o[b]);
    }
  }
  __device__ __forceinline__ void with_lane(int x) {  // and what the lane `x` away has
    scale_to(fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x)));
    L += __shfl_xor_sync(0xffffffffu, L, x);
    O.x += __shfl_xor_sync(0xffffffffu, O.x, x);
    O.y += __shfl_xor_sync(0xffffffffu, O.y, x);
    O.z += __shfl_xor_sync(0xffffffffu, O.z, x);
    O.w += __shfl_xor_sync(0xffffffffu, O.w, x);
  }
  __device__ __forceinline__ void store(float* to) const {
    const float f = 1.f / L;
    *reinterpret_cast<float4*>(to) = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
  }
};

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const int4* split, const float* part,
                                                                      float* __restrict__ out, int Hq, int rows_max,
                                                                      int n_seqs, int* status) {
  __shared__ float s_m[kJoinWarps][4], s_l[kJoinWarps][4];
  __shared__ __align__(16) float4 s_o[kJoinWarps][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = blockIdx.x;
  const int64_t stride = paged_part_floats(rows_max, D);
  pdl_wait();
  const int4 both[2] = {split[2 * w], split[2 * w + 1]};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int4 it = both[k];  // first warp, parts, sequence, first head and number of heads
    if (it.y == 0) continue;
    const int heads = it.w & 31;
    if constexpr (kCheck) {  // (debug build) the item's parts, their rows, its output
      if (!(chk(status, kChkPagedJoin, it.x, w + 1ll) && chk(status, kChkPagedJoin, it.x + it.y - 1ll, gridDim.x) &&
            chk(status, kChkPagedJoin, heads - 1, rows_max) && chk(status, kChkPagedOut, it.z, n_seqs) &&
            chk(status, kChkPagedOut, (it.w >> 5) + heads - 1, Hq)))
        continue;
    }
    const float* base = part + 2ll * it.x * stride;  // the first part is in slot 1 of its warp, the others in slot 0
    auto at = [&](int i) { return base + (2ll * i + (i == 0)) * stride; };
    float* to = out + ((int64_t)it.z * Hq + (it.w >> 5)) * D;
    if (it.y > kManyParts) {
      constexpr int Z = D / 16;
      for (int u = w - it.x; u < heads * Z; u += it.y) {
        const int h = u / Z, e = h * D + u % Z * 16 + lane % 4 * 4;
        PagedMerge y;
        y.parts(at, threadIdx.x >> 2, kJoinThreads / 4, it.y, h, 2 * kMaxTile + e);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) y.with_lane(o);
        __syncthreads();  // the last unit's reads are done
        if (lane < 4) {
          s_o[warp][lane] = y.O;
          s_m[warp][lane] = y.M;
          s_l[warp][lane] = y.L;
        }
        __syncthreads();
        if (threadIdx.x < 4) {
          PagedMerge a;
#pragma unroll
          for (int i = 0; i < kJoinWarps; ++i) {
            a.scale_to(fmaxf(a.M, s_m[i][lane]));
            a.add(s_m[i][lane], s_l[i][lane], s_o[i][lane]);
          }
          a.store(to + e);
        }
      }
    } else if (it.y > kFewParts) {
      constexpr int Z = D / 32;
      for (int u = (w - it.x) * kJoinWarps + warp; u < heads * Z; u += it.y * kJoinWarps) {
        const int h = u / Z, e = h * D + u % Z * 32 + lane % 8 * 4;
        PagedMerge y;
        y.parts(at, lane >> 3, 4, it.y, h, 2 * kMaxTile + e);
        y.with_lane(8);
        y.with_lane(16);
        if (lane < 8) y.store(to + e);
      }
    } else {
      constexpr int ROW = D < 128 ? D : 128, Z = D / ROW;
      for (int u = (w - it.x) * kJoinWarps + warp; u < heads * Z; u += it.y * kJoinWarps) {
        const int h = u / Z, e = h * D + u % Z * ROW + lane % (ROW / 4) * 4;
        PagedMerge y;
        y.parts(at, 0, 1, it.y, h, 2 * kMaxTile + e);
        if (lane < ROW / 4) y.store(to + e);
      }
    }
  }
}

}  // namespace ntx
