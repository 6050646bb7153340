// paged.cu -- the C entries of the paged KV cache: argument checks and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "launch.h"
#include "ntx.h"
#include "paged.cuh"
#include "per_device.h"

namespace ntx {
namespace {

constexpr int kMaxGroup = 64;

int failf(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(code, buf);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// n rows of `width` floats, `stride` floats apart.
struct Rows {
  const float* first;
  int64_t stride, width;
};
using wide_int = __int128;  // any stride that the arguments can hold
wide_int floor_div(wide_int a, wide_int b) { return a / b - (a % b < 0); }  // b > 0

// Whether a row of a and a row of b share a byte; what lies between rows does not count.
bool rows_overlap(const Rows& a, const Rows& b, int64_t n) {
  if (n < 1 || a.width < 1 || b.width < 1 || !a.first || !b.first) return false;
  const wide_int x = reinterpret_cast<uintptr_t>(a.first), y = reinterpret_cast<uintptr_t>(b.first), d = y - x;
  const wide_int sa = (wide_int)a.stride * 4, sb = (wide_int)b.stride * 4, wa = a.width * 4, wb = b.width * 4;
  if (x + (n - 1) * sa + wa <= y || y + (n - 1) * sb + wb <= x) return false;  // apart as a whole, as most are
  if (n == 1) return true;
  // row i of a meets row j of b:  d - wa < i sa - j sb < d + wb
  if (sa == sb) {
    const wide_int lo = floor_div(d - wa, sa) + 1, hi = -floor_div(-(d + wb), sa) - 1;  // of i - j
    return (lo > 1 - n ? lo : 1 - n) <= (hi < n - 1 ? hi : n - 1);
  }
  for (int64_t i = 0; i < n; ++i) {
    const wide_int at = i * sa - d;  // at - wb < j sb < at + wa
    const wide_int lo = floor_div(at - wb, sb) + 1, hi = -floor_div(-(at + wa), sb) - 1;
    if ((lo > 0 ? lo : 0) <= (hi < n - 1 ? hi : n - 1)) return true;
  }
  return false;
}

int row_bytes(int type, int D) {
  switch (type) {
    case NTX_F16: return kv_row_bytes<kKvF16>(D);
    case NTX_Q8_0: return kv_row_bytes<kKvQ8>(D);
    case NTX_Q4_0: return kv_row_bytes<kKvQ4>(D);
    default: return 0;
  }
}

int check_sizes(const char* who, int type, int n_kv_heads, int head_dim, int page_size, int n_pages) {
  if (!row_bytes(type, 128)) return failf(NTX_ERR_QTYPE, "%s: cache type %d is none of F16, Q8_0, Q4_0", who, type);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return failf(NTX_ERR_SHAPE, "%s: head_dim %d is none of 64, 128, 256", who, head_dim);
  if (n_kv_heads < 1 || n_kv_heads > 1024) return failf(NTX_ERR_SHAPE, "%s: n_kv_heads %d outside 1..1024", who, n_kv_heads);
  if (page_size < 16 || page_size % 16 || page_size > (1 << 30))
    return failf(NTX_ERR_SHAPE, "%s: page_size %d is not a multiple of 16 up to 2^30", who, page_size);
  if (n_pages < 1) return failf(NTX_ERR_SHAPE, "%s: n_pages %d", who, n_pages);
  return NTX_OK;
}

int check_kv(const char* who, const ntx_paged_kv* kv) {
  if (!kv) return failf(NTX_ERR_INVALID_ARG, "%s: kv is NULL", who);
  const int rc = check_sizes(who, kv->type, kv->n_kv_heads, kv->head_dim, kv->page_size, kv->n_pages);
  if (rc) return rc;
  if (kv->n_seqs < 1 || kv->n_seqs > kMaxPagedSeqs)
    return failf(NTX_ERR_SHAPE, "%s: n_seqs %d outside 1..%d", who, kv->n_seqs, kMaxPagedSeqs);
  if (kv->max_pages < 1 || (int64_t)kv->max_pages * kv->page_size > (1 << 30))
    return failf(NTX_ERR_SHAPE, "%s: max_pages %d x page_size %d outside 1..2^30", who, kv->max_pages, kv->page_size);
  return NTX_OK;
}

int check_kv_pointers(const char* who, const ntx_paged_kv* kv) {
  if (!kv->k_pages || !kv->v_pages || !kv->page_table) return failf(NTX_ERR_INVALID_ARG, "%s: NULL cache pointer", who);
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16) || !aligned(kv->page_table, 4))
    return failf(NTX_ERR_ALIGN, "%s: pools must be 16-byte and page_table 4-byte aligned", who);
  return NTX_OK;
}

// What ntx_kv_append and ntx_kv_read share.
int check_tokens(const char* who, const ntx_paged_kv* kv, const float* k, const float* v, int64_t ks, int64_t vs,
                 const int32_t* seq_ids, const int32_t* positions, int n_tokens) {
  int rc = check_kv(who, kv);
  if (rc) return rc;
  const int64_t width = (int64_t)kv->n_kv_heads * kv->head_dim;
  if (n_tokens < 0) return failf(NTX_ERR_SHAPE, "%s: n_tokens %d", who, n_tokens);
  if (!seq_ids && n_tokens > kv->n_seqs)
    return failf(NTX_ERR_SHAPE, "%s: %d tokens without seq_ids for %d sequences", who, n_tokens, kv->n_seqs);
  if ((k && ks < width) || (v && vs < width))
    return failf(NTX_ERR_SHAPE, "%s: row stride below n_kv_heads * head_dim = %lld", who, (long long)width);
  if (n_tokens == 0) return NTX_OK;
  if (!positions) return failf(NTX_ERR_INVALID_ARG, "%s: positions is NULL", who);
  if (!aligned(k, 4) || !aligned(v, 4) || !aligned(seq_ids, 4) || !aligned(positions, 4))
    return failf(NTX_ERR_ALIGN, "%s: pointers must be 4-byte aligned", who);
  return check_kv_pointers(who, kv);
}

bool rows16(const float* p, int64_t stride) { return aligned(p, 16) && stride % 4 == 0; }

// Pieces of a token's row of keys (or values), and the grid over them: at most 512 pieces, 1024 heads of 256 elements.
int token_pieces(const ntx_paged_kv* kv) { return (kv->n_kv_heads * kv->head_dim + kPiece - 1) / kPiece; }
dim3 token_grid(int n_tokens, int pieces) {
  return dim3((unsigned)(((int64_t)n_tokens + kTokenWarps - 1) / kTokenWarps), (unsigned)pieces);
}

template <class F>
cudaError_t with_type(int type, F f) {
  switch (type) {
    case NTX_F16: return f(std::integral_constant<int, kKvF16>{});
    case NTX_Q8_0: return f(std::integral_constant<int, kKvQ8>{});
    default: return f(std::integral_constant<int, kKvQ4>{});
  }
}

template <class F>
cudaError_t with_dim(int D, F f) {
  switch (D) {
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    default: return f(std::integral_constant<int, 256>{});
  }
}

// Kernel attributes are set on first use on a device.
template <class K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// Column tiles of four query heads that share one pass over the keys and values
// of their KV head: 1 for groups up to 4, 2 up to 8, else 4; 2 at most for
// head_dim 256, where q and o of 16 heads are more than the registers hold.
template <class F>
cudaError_t with_attn(const ntx_paged_kv* kv, int n_q_heads, F f) {
  const int G = n_q_heads / kv->n_kv_heads;
  return with_type(kv->type, [&](auto t) {
    return with_dim(kv->head_dim, [&](auto d) {
      if (G <= 4) return f(t, d, std::integral_constant<int, 1>{});
      if constexpr (decltype(d)::value <= 128)
        if (G > 8) return f(t, d, std::integral_constant<int, 4>{});
      return f(t, d, std::integral_constant<int, 2>{});
    });
  });
}

// Workspace: two records of 16 bytes and two parts for each warp of the attention kernel.
size_t paged_ws(const ntx_paged_kv* kv, int n_q_heads) {
  size_t n = 0;
  with_attn(kv, n_q_heads, [&](auto t, auto d, auto nc) {
    using F = PagedCfg<decltype(t)::value, decltype(d)::value, decltype(nc)::value, false>;
    const size_t warps = (size_t)sm_count() * F::CTAS * F::WARPS;
    const int G = n_q_heads / kv->n_kv_heads;
    n = warps * 2 * (sizeof(int4) + sizeof(float) * paged_part_floats(G < F::HEADS ? G : F::HEADS, kv->head_dim));
    return cudaSuccess;
  });
  return n;
}

template <class O>
void one_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int64_t grid, int ctas, cudaStream_t stream) {
  cfg->gridDim = dim3((unsigned)grid);
  cfg->blockDim = dim3(O::WARPS * 32);
  cfg->dynamicSmemBytes = O::SMEM;
  cfg->stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)ctas;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// How a cluster of CTAs to an item runs: as many CTAs as give each warp one chunk of the
// longest sequence that the table can hold, or the most of which all clusters are resident
// at once (15 of 8 CTAs on a B200 of 148 SMs that hold one each; asked for once on a device,
// so that the order of an output's sums does not depend on what ran on another).
struct OneGrid {
  int64_t items, work;  // work: a warp's positions times heads at most
  int most, ctas;       // 0: more items than CTAs are resident
};
template <int T, int D, int NC>
cudaError_t one_grid(const ntx_paged_kv& kv, int G, OneGrid* grid) {
  using O = PagedCfg<T, D, NC, true>;
  static std::atomic<unsigned long long> done{0};
  static PerDevice<9> fit;  // clusters of that many CTAs that are resident at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (e = allow_smem(attn_paged_kernel<T, D, NC, true>, O::SMEM, done)) != cudaSuccess) return e;
  OneGrid g{(int64_t)kv.n_seqs * kv.n_kv_heads * ((G + O::HEADS - 1) / O::HEADS), 0, 0, 0};
  const int64_t chunks = ((int64_t)kv.max_pages * kv.page_size + O::CH - 1) / O::CH;
  for (int c = 1; c <= 8; ++c) {
    int n;
    e = fit.get(dev, c, &n, [&](int* clusters) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      one_config<O>(&cfg, attr, c, c, nullptr);
      return cudaOccupancyMaxActiveClusters(clusters, attn_paged_kernel<T, D, NC, true>, &cfg);
    });
    if (e != cudaSuccess) return e;
    if (g.items > n) continue;
    g.most = c;
    if (g.ctas * O::WARPS < chunks) g.ctas = c;
  }
  if (g.ctas) g.work = (chunks + g.ctas * O::WARPS - 1) / (g.ctas * O::WARPS) * O::CH * O::HEADS;
  *grid = g;
  return cudaSuccess;
}

template <int T, int D, int NC>
cudaError_t launch_attn_one(const OneGrid& g, const ntx_paged_kv& kv, const float* q, int64_t qs, float* out, int Hq,
                            const int32_t* lens, float scale, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  one_config<PagedCfg<T, D, NC, true>>(&cfg, attr, g.items * g.ctas, g.ctas, stream);
  return cudaLaunchKernelEx(&cfg, attn_paged_kernel<T, D, NC, true>, kv, q, qs, out, (int4*)nullptr, (float*)nullptr, Hq,
                            lens, scale, device_status_ptr());
}

template <int T, int D, int NC>
cudaError_t launch_attn_paged(const ntx_paged_kv& kv, const float* q, int64_t qs, float* out, int Hq,
                              const int32_t* lens, float scale, void* ws, cudaStream_t stream) {
  using F = PagedCfg<T, D, NC, false>;
  static std::atomic<unsigned long long> done{0};
  const int grid = sm_count() * F::CTAS, warps = grid * F::WARPS, G = Hq / kv.n_kv_heads;
  const int64_t ctx = (int64_t)kv.max_pages * kv.page_size;
  cudaError_t e;
  if (ctx <= 8 * kOneCtaCtx) {
    OneGrid one;
    if ((e = one_grid<T, D, NC>(kv, G, &one)) != cudaSuccess) return e;
    if (ctx <= kOneCtaCtx * one.most) {
      if constexpr (NC > 1) {  // four heads to a tile where a warp's work is no more for it
        OneGrid narrow;
        if ((e = one_grid<T, D, 1>(kv, G, &narrow)) != cudaSuccess) return e;
        if (narrow.most && narrow.work <= one.work)
          return launch_attn_one<T, D, 1>(narrow, kv, q, qs, out, Hq, lens, scale, stream);
      }
      return launch_attn_one<T, D, NC>(one, kv, q, qs, out, Hq, lens, scale, stream);
    }
  }
  int4* split = static_cast<int4*>(ws);
  float* part = reinterpret_cast<float*>(split + 2 * (size_t)warps);
  e = allow_smem(attn_paged_kernel<T, D, NC, false>, F::SMEM, done);
  if (e != cudaSuccess) return e;
  attn_paged_kernel<T, D, NC, false><<<grid, F::WARPS * 32, F::SMEM, stream>>>(kv, q, qs, out, split, part, Hq, lens, scale,
                                                                       device_status_ptr());
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(warps);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D>, (const int4*)split, (const float*)part, out, Hq,
                            G < F::HEADS ? G : F::HEADS, kv.n_seqs, device_status_ptr());
}

int finish(const char* who, cudaError_t e) { return e == cudaSuccess ? NTX_OK : record_cuda_error(e, who); }

}  // namespace
}  // namespace ntx

using namespace ntx;

extern "C" {

uint64_t ntx_paged_kv_bytes(int type, int n_kv_heads, int head_dim, int page_size, int n_pages) {
  if (check_sizes("ntx_paged_kv_bytes", type, n_kv_heads, head_dim, page_size, n_pages)) return 0;
  const unsigned __int128 n = (unsigned __int128)row_bytes(type, head_dim) * page_size * n_kv_heads * n_pages;
  if (n >> 62) {
    failf(NTX_ERR_SHAPE, "ntx_paged_kv_bytes: the pool is larger than 2^62 bytes");
    return 0;
  }
  return (uint64_t)n;
}

int ntx_qk_norm_rope(const float* q, const float* k, float* q_out, float* k_out, int64_t q_stride, int64_t k_stride,
                     const float* wq, const float* wk, const int32_t* positions, int n_tokens, int n_q_heads,
                     int n_kv_heads, int head_dim, int rot_dim, int pairing, float theta, float eps, void* stream) {
  const char* who = "ntx_qk_norm_rope";
  if (head_dim < 2 || head_dim > 256 || head_dim % 2) return failf(NTX_ERR_SHAPE, "%s: head_dim %d", who, head_dim);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2) return failf(NTX_ERR_SHAPE, "%s: rot_dim %d", who, rot_dim);
  if (n_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > 65536 || n_kv_heads > 65536)
    return failf(NTX_ERR_SHAPE, "%s: %d tokens, %d and %d heads", who, n_tokens, n_q_heads, n_kv_heads);
  if (pairing != NTX_ROPE_ADJACENT && pairing != NTX_ROPE_HALVES)
    return failf(NTX_ERR_INVALID_ARG, "%s: pairing %d", who, pairing);
  if (!(theta > 0.f) || !std::isfinite(theta) || !(eps >= 0.f) || !std::isfinite(eps))
    return failf(NTX_ERR_INVALID_ARG, "%s: bad theta or eps", who);
  const int64_t nq = (int64_t)n_q_heads * head_dim, nk = (int64_t)n_kv_heads * head_dim;
  if (q_stride < nq || k_stride < nk) return failf(NTX_ERR_SHAPE, "%s: stride below the row", who);
  if (n_tokens == 0 || n_q_heads + n_kv_heads == 0) return NTX_OK;
  if (!positions || (nq && (!q || !q_out)) || (nk && (!k || !k_out)))
    return failf(NTX_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned(q, 4) || !aligned(k, 4) || !aligned(q_out, 4) || !aligned(k_out, 4) || !aligned(wq, 4) ||
      !aligned(wk, 4) || !aligned(positions, 4))
    return failf(NTX_ERR_ALIGN, "%s: pointers must be 4-byte aligned", who);
  const Rows rq{q, q_stride, nq}, rk{k, k_stride, nk}, rqo{q_out, q_stride, nq}, rko{k_out, k_stride, nk};
  if ((q != q_out && rows_overlap(rq, rqo, n_tokens)) || (k != k_out && rows_overlap(rk, rko, n_tokens)) ||
      rows_overlap(rq, rko, n_tokens) || rows_overlap(rk, rqo, n_tokens) || rows_overlap(rqo, rko, n_tokens))
    return failf(NTX_ERR_INVALID_ARG, "%s: an output overlaps an input it does not replace, or the other output", who);
  const int heads = n_q_heads + n_kv_heads;
  // whole rows of 64, 128 or 256 in 16-byte pieces; the halves' pairs are as wide apart as the lanes only when all rotate
  const bool vec = (head_dim == 64 || head_dim == 128 || head_dim == 256) && rows16(q, q_stride) && rows16(k, k_stride) &&
                   rows16(q_out, q_stride) && rows16(k_out, k_stride) &&
                   (pairing == NTX_ROPE_ADJACENT || rot_dim == head_dim);
  // log2(theta) as a number of 40 bits and the rest
  const long double lg = std::log2((long double)theta);
  const double lg_hi = (double)std::nearbyint(lg * 17179869184.0L) / 17179869184.0, lg_lo = (double)(lg - lg_hi);
  // Rows of a token that a warp takes: enough shares for eight rounds of the warps that the SMs hold, one row at
  // least, all at most; from five on, fours (what a warp has in flight) in shares as even as three more allow: 72
  // heads in 6 shares of 12 take 110 us where 4 of 16 and one of 8 take 113.
  const int room = sm_count() * rope_ctas(head_dim <= 128 ? 1 : 4);
  int rows = (int)min64(heads, (int64_t)n_tokens * heads / ((int64_t)room * kRopeWarps * 8) + 1);
  int shares = (heads + rows - 1) / rows;
  if (rows > 4) {
    int best = heads;  // rows that the last share lacks
    for (int n = shares, end = shares + 3; n <= end && best; ++n) {
      const int r = ((heads + n - 1) / n + 3) / 4 * 4;
      if (r * n - heads < best) {
        best = r * n - heads;
        rows = r;
      }
    }
    shares = (heads + rows - 1) / rows;
  }
  const int grid = (int)min64(((int64_t)n_tokens * shares + kRopeWarps - 1) / kRopeWarps, room);
  auto run = [&](auto p, auto halves, auto v) {
    qk_norm_rope_kernel<decltype(p)::value, decltype(halves)::value, decltype(v)::value>
        <<<grid, kRopeWarps * 32, 0, (cudaStream_t)stream>>>(q, k, q_out, k_out, q_stride, k_stride, wq, wk, positions,
                                                            n_tokens, n_q_heads, n_kv_heads, head_dim, rot_dim, lg_hi,
                                                            lg_lo, eps, rows, shares);
    return cudaGetLastError();
  };
  auto by_pairing = [&](auto p, auto v) {
    return pairing == NTX_ROPE_HALVES ? run(p, std::true_type{}, v) : run(p, std::false_type{}, v);
  };
  auto by_vec = [&](auto p) { return vec ? by_pairing(p, std::true_type{}) : by_pairing(p, std::false_type{}); };
  if (head_dim <= 64) return finish(who, by_vec(std::integral_constant<int, 1>{}));
  if (head_dim <= 128) return finish(who, by_vec(std::integral_constant<int, 2>{}));
  return finish(who, by_vec(std::integral_constant<int, 4>{}));
}

int ntx_kv_append(const ntx_paged_kv* kv, const float* k, const float* v, int64_t k_stride, int64_t v_stride,
                  const int32_t* seq_ids, const int32_t* positions, int n_tokens, void* stream) {
  const char* who = "ntx_kv_append";
  const int rc = check_tokens(who, kv, k, v, k_stride, v_stride, seq_ids, positions, n_tokens);
  if (rc || n_tokens == 0) return rc;
  if (!k || !v) return failf(NTX_ERR_INVALID_ARG, "%s: NULL pointer", who);
  const bool vec = rows16(k, k_stride) && rows16(v, v_stride);
  const int pieces = token_pieces(kv);
  return finish(who, with_type(kv->type, [&](auto t) {
    return with_dim(kv->head_dim, [&](auto d) {
      kv_append_kernel<decltype(t)::value, decltype(d)::value>
          <<<token_grid(n_tokens, 2 * pieces), kTokenWarps * 32, 0, (cudaStream_t)stream>>>(
              *kv, k, v, k_stride, v_stride, seq_ids, positions, n_tokens, vec, pieces, device_status_ptr());
      return cudaGetLastError();
    });
  }));
}

int ntx_kv_read(const ntx_paged_kv* kv, float* k, float* v, int64_t k_stride, int64_t v_stride,
                const int32_t* seq_ids, const int32_t* positions, int n_tokens, void* stream) {
  const char* who = "ntx_kv_read";
  const int rc = check_tokens(who, kv, k, v, k_stride, v_stride, seq_ids, positions, n_tokens);
  if (rc || n_tokens == 0 || (!k && !v)) return rc;
  const bool vec = (!k || rows16(k, k_stride)) && (!v || rows16(v, v_stride));
  const int pieces = token_pieces(kv);
  return finish(who, with_type(kv->type, [&](auto t) {
    return with_dim(kv->head_dim, [&](auto d) {
      kv_read_kernel<decltype(t)::value, decltype(d)::value>
          <<<token_grid(n_tokens, 2 * pieces), kTokenWarps * 32, 0, (cudaStream_t)stream>>>(
              *kv, k, v, k_stride, v_stride, seq_ids, positions, n_tokens, vec, pieces, device_status_ptr());
      return cudaGetLastError();
    });
  }));
}

size_t ntx_attn_paged_workspace_bytes(const ntx_paged_kv* kv, int n_q_heads) {
  const char* who = "ntx_attn_paged_workspace_bytes";
  if (check_kv(who, kv) || n_q_heads < 1 || n_q_heads % kv->n_kv_heads || n_q_heads / kv->n_kv_heads > kMaxGroup) return 0;
  return paged_ws(kv, n_q_heads);
}

int ntx_attn_decode_paged(const ntx_paged_kv* kv, const float* q, int64_t q_stride, float* out, int n_q_heads,
                          const int32_t* ctx_lens, float scale, void* workspace, size_t ws_bytes, void* stream) {
  const char* who = "ntx_attn_decode_paged";
  int rc = check_kv(who, kv);
  if (rc) return rc;
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads || n_q_heads / kv->n_kv_heads > kMaxGroup)
    return failf(NTX_ERR_SHAPE, "%s: %d query heads over %d KV heads", who, n_q_heads, kv->n_kv_heads);
  const int64_t width = (int64_t)n_q_heads * kv->head_dim;
  if (q_stride < width) return failf(NTX_ERR_SHAPE, "%s: q_stride below n_q_heads * head_dim", who);
  if (!std::isfinite(scale)) return failf(NTX_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (!q || !out || !ctx_lens || !workspace) return failf(NTX_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if ((rc = check_kv_pointers(who, kv)) != NTX_OK) return rc;
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 4 || !aligned(workspace, 16) || !aligned(ctx_lens, 4))
    return failf(NTX_ERR_ALIGN, "%s: q, its rows, out and workspace must be 16-byte aligned", who);
  if (rows_overlap({q, q_stride, width}, {out, width, width}, kv->n_seqs))
    return failf(NTX_ERR_INVALID_ARG, "%s: out overlaps q", who);
  if (ws_bytes < ntx_attn_paged_workspace_bytes(kv, n_q_heads))
    return failf(NTX_ERR_NOMEM, "%s: workspace too small", who);
  return finish(who, with_attn(kv, n_q_heads, [&](auto t, auto d, auto nc) {
    return launch_attn_paged<decltype(t)::value, decltype(d)::value, decltype(nc)::value>(
        *kv, q, q_stride, out, n_q_heads, ctx_lens, scale, workspace, (cudaStream_t)stream);
  }));
}

}  // extern "C"
