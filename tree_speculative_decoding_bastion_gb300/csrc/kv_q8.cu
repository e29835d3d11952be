// Writing tokens to the 8-bit context cache and reading them back.
//
// Tokens of any number join a request's context at its end: a prompt, a
// chunk of it, a decoded token (append), or the path that verification
// accepted (commit: the rows that acc_nodes names, root first).  Both are the
// same copy with a quantisation on the way (q8.cuh); reading back is the
// inverse, exact in f32 and in bf16 (four significant bits).
//
// What bounds it: bytes.  A row of d elements is read once (d * 2 or 4 bytes)
// and written once (d + 1 bytes); the arithmetic is a maximum over the row
// and one conversion per element.  So a lane owns 16 elements (two or four
// 16-byte loads, one 16-byte store), the d / 16 lanes of a row reduce its
// maximum by shuffles, and several rows per lane are in flight at once.
// Measured (6.7 TB/s is what a copy reaches): 4 prompts of up to 8191 fp32 tokens
// (8 heads of 128, 228 MB) 50 us, 4.6 TB/s; 16 contexts of up to 8192 read back
// to bf16 (536 MB) 85.8 us, 6.3 TB/s; one token 3.9 us, 16 accepted paths 6.5 us
// (dependent loads: counts, page or node, row).
#include <algorithm>

#include "q8.cuh"

namespace bst {

constexpr int Q8_THREADS = 256;
constexpr int Q8_UNROLL = 4;       // rows in flight per lane: reading back, and writing from bf16
constexpr int Q8_ONE_THREADS = 1024;
constexpr int Q8_ONE_UNROLL = 2;
template <class Tag>
constexpr int q8_write_unroll() { return Tag::kVec == 8 ? Q8_UNROLL : Q8_UNROLL / 2; }   // 128 bytes either way

// 16 consecutive elements as floats
template <class Tag>
struct Load16 {
  static constexpr int kVecs = 16 / Tag::kVec;
  uint4 v[kVecs];
  BST_DEV void load(const uint4 *p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ld_stream16(p + i);
  }
  BST_DEV void unpack(float *x) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) unpack16<Tag>(v[i], x + i * Tag::kVec);
  }
};

// Maximum over the `gs` lanes (a power of two) that share a row.
BST_DEV uint32_t group_max(uint32_t m, int gs) {
  for (int o = gs >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(FULL, m, o));
  return m;
}

// One row's lane: codes of 16 elements and the row's scale byte.
template <class Tag>
BST_DEV uint4 quantise16(const Load16<Tag> &in, bool have, int gs, uint32_t *byte) {
  float x[16];
  in.unpack(x);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, finite_abs_bits(x[i]));
  m = group_max(have ? m : 0u, gs);
  *byte = q8_scale_byte(m);
  const float inv = q8_inv_scale(*byte);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = cvt_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | (cvt_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

BST_DEV int64_t cache_capacity(const RowCache &c) {
  return c.block_table ? static_cast<int64_t>(c.max_pages) * c.page_size : c.L_max;
}

struct WriteParams {
  const uint4 *k_new, *v_new;    // [B, T, Hkv, d]
  uint4 *k, *v;                  // codes
  uint8_t *ks, *vs;              // scale bytes
  RowCache cache;
  int T, Hkv, K;                 // K: commit, columns of nodes - 1
  int passes;                    // how often a CTA of the grid goes on to the next rows (kv_q8_write_kernel)
  int lanes, gs;                 // d / 16 lanes hold a row; gs: the power of two at or above
  const int32_t *count;          // append: tokens per request; commit: acc_len (tokens - 1)
  const int32_t *nodes;          // commit: [B, K + 1] rows of k_new; append: NULL (row i)
  const int32_t *ctx_len;
  int32_t *ctx_out;
  uint32_t *dev_err;
};

// What request b brings: its tokens, the place of the first, and whether its
// counts make sense (its pages and path nodes are checked apart).
struct WriteRequest {
  int cnt, ctx;
  uint32_t bad;
};
BST_DEV WriteRequest write_request(const WriteParams &p, int b) {
  WriteRequest r;
  const int raw = p.count[b];
  r.cnt = p.nodes ? raw + 1 : raw;
  r.ctx = p.ctx_len[b];
  r.bad = 0;
  if (p.nodes ? (raw < 0 || raw > p.K) : (raw < 0 || raw > p.T))
    r.bad = BASTION_DEVERR_N;
  else if (r.ctx < 0 || static_cast<int64_t>(r.ctx) + r.cnt > cache_capacity(p.cache))
    r.bad = BASTION_DEVERR_CTX;
  return r;
}
// This thread's part of the check of a request whose counts make sense: error bits.
BST_DEV uint32_t write_checks(const WriteParams &p, int b, const WriteRequest &r, int threads) {
  uint32_t bad = 0;
  if (p.nodes)
    for (int i = threadIdx.x; i < r.cnt; i += threads) {
      const int node = p.nodes[static_cast<int64_t>(b) * (p.K + 1) + i];
      if (node < 0 || node >= p.T) bad |= BASTION_DEVERR_N;
    }
  if (p.cache.block_table && r.cnt > 0) {
    // page ids first .. end - 1, four at a time where they lie in aligned words of four
    const int32_t *row = p.cache.block_table + static_cast<int64_t>(b) * p.cache.max_pages;
    const int first = r.ctx / p.cache.page_size, end = (r.ctx + r.cnt - 1) / p.cache.page_size + 1;
    const int head = min(end, first + static_cast<int>((0 - (reinterpret_cast<uintptr_t>(row + first) >> 2)) & 3));
    const int fours = (end - head) >> 2;
    const int4 *four = reinterpret_cast<const int4 *>(row + head);
    const uint32_t pages = static_cast<uint32_t>(p.cache.num_pages);
    uint32_t top = 0;                         // (a negative id is a large one)
#pragma unroll 4
    for (int i = threadIdx.x; i < fours; i += threads) {
      const int4 v = __ldg(four + i);
      top = max(max(top, max(static_cast<uint32_t>(v.x), static_cast<uint32_t>(v.y))),
                max(static_cast<uint32_t>(v.z), static_cast<uint32_t>(v.w)));
    }
    const int rest = (head - first) + (end - head - 4 * fours);   // at most six, before and behind
    if (static_cast<int>(threadIdx.x) < rest) {
      const int i = first + static_cast<int>(threadIdx.x);
      top = max(top, static_cast<uint32_t>(__ldg(row + (i < head ? i : i + 4 * fours))));
    }
    if (top >= pages) bad |= BASTION_DEVERR_PAGE;
  }
  return bad;
}

// Rows r, r + step, ... (U of them) of a request's 2 cnt Hkv: K's, then V's.
// load() reads them and finds their places, store() quantises and writes them:
// the checks lie in between, so that their latency hides behind the rows'.
template <class Tag, int U>
struct WriteRows {
  Load16<Tag> in[U];
  int64_t dst[U];

  BST_DEV void load(const WriteParams &p, int b, const WriteRequest &q, int r, int step, int lane_in_row) {
    const int half = q.cnt * p.Hkv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int rr = r + u * step;
      dst[u] = -1;
      if (rr < 2 * half && lane_in_row < p.lanes) {
        const int k = rr < half ? rr : rr - half;
        const int i = k / p.Hkv, h = k - i * p.Hkv;
        int node = i;
        if (p.nodes) {
          node = p.nodes[static_cast<int64_t>(b) * (p.K + 1) + i];
          if (node < 0 || node >= p.T) continue;            // the checks refuse the request
        }
        const int64_t row = (static_cast<int64_t>(b) * p.T + node) * p.Hkv + h;
        in[u].load((rr < half ? p.k_new : p.v_new) + (row * p.lanes + lane_in_row) * Load16<Tag>::kVecs);
        dst[u] = cache_row(p.cache, p.Hkv, b, h, q.ctx + i);
      }
    }
  }
  BST_DEV void store(const WriteParams &p, const WriteRequest &q, int r, int step, int lane_in_row) {
    const int half = q.cnt * p.Hkv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool is_v = r + u * step >= half;
      uint32_t byte;
      if (dst[u] < 0) {
#pragma unroll
        for (int i = 0; i < Load16<Tag>::kVecs; ++i) in[u].v[i] = make_uint4(0, 0, 0, 0);
      }
      const uint4 codes = quantise16<Tag>(in[u], dst[u] >= 0, p.gs, &byte);   // every lane takes part in the shuffles
      if (dst[u] >= 0) {
        (is_v ? p.v : p.k)[dst[u] * p.lanes + lane_in_row] = codes;
        if (lane_in_row == 0) (is_v ? p.vs : p.ks)[dst[u]] = static_cast<uint8_t>(byte);
      }
    }
  }
};

// Many tokens: CTA (x, b) takes a stretch of consecutive rows of request b;
// kv_q8_advance_kernel then moves ctx_out.  128 bytes a lane in flight and four
// CTAs an SM: with five and six 51.7 and 57.7 us for 48.7, with half, one and a
// half and twice the rows a lane 50.8, 52.8 and 55.  Every CTA checks all pages of
// its request before it writes, so its stretch grows with the request's pages
// (launch_kv_write_q8): the checks read a part of what the rows read, not its square.
template <class Tag>
__global__ void __launch_bounds__(Q8_THREADS, 4) kv_q8_write_kernel(const WriteParams p) {
  constexpr int U = q8_write_unroll<Tag>();
  const int b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int per_pass = Q8_THREADS / p.gs;
  const int r0 = blockIdx.x * p.passes * per_pass * U;
  const WriteRequest q = write_request(p, b);
  if (q.bad || r0 >= 2 * q.cnt * p.Hkv) return;     // uniform
  const int lane_in_row = threadIdx.x & (p.gs - 1);
  int r = r0 + static_cast<int>(threadIdx.x) / p.gs;
  WriteRows<Tag, U> rows;
  rows.load(p, b, q, r, per_pass, lane_in_row);
  if (__syncthreads_or(write_checks(p, b, q, Q8_THREADS) != 0)) return;
  rows.store(p, q, r, per_pass, lane_in_row);
  const int end = min(r0 + p.passes * per_pass * U, 2 * q.cnt * p.Hkv);
  for (int first = r0 + per_pass * U; first < end; first += per_pass * U) {   // uniform
    r += per_pass * U;
    rows.load(p, b, q, r, per_pass, lane_in_row);
    rows.store(p, q, r, per_pass, lane_in_row);
  }
}

__global__ void __launch_bounds__(Q8_ONE_THREADS) kv_q8_advance_kernel(const WriteParams p) {
  const int b = blockIdx.x;
  pdl_wait();   // the rows are written: nobody reads ctx_len any more, which ctx_out may be
  pdl_trigger();
  const WriteRequest q = write_request(p, b);
  const uint32_t bad = q.bad ? q.bad : write_checks(p, b, q, blockDim.x);
  if (bad) set_err(p.dev_err, bad);
  const bool ok = !__syncthreads_or(bad != 0);
  if (threadIdx.x == 0) p.ctx_out[b] = ok ? q.ctx + q.cnt : q.ctx;
}

// Few tokens: one CTA per request writes its rows and moves ctx_out, one
// launch (the checks' barrier separates every read of ctx_len[b] from the
// write of ctx_out[b], which may be the same word).
template <class Tag>
__global__ void __launch_bounds__(Q8_ONE_THREADS) kv_q8_write_one_kernel(const WriteParams p) {
  const int b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const WriteRequest q = write_request(p, b);
  const int per_pass = Q8_ONE_THREADS / p.gs;
  const int lane_in_row = threadIdx.x & (p.gs - 1);
  const int r = static_cast<int>(threadIdx.x) / p.gs;
  WriteRows<Tag, Q8_ONE_UNROLL> rows;
  uint32_t bad = q.bad;
  if (!bad) {
    rows.load(p, b, q, r, per_pass, lane_in_row);
    bad = write_checks(p, b, q, Q8_ONE_THREADS);
  }
  if (bad && (threadIdx.x == 0 || !q.bad)) set_err(p.dev_err, bad);
  const bool ok = !__syncthreads_or(bad != 0);
  if (ok && q.cnt > 0) rows.store(p, q, r, per_pass, lane_in_row);
  if (threadIdx.x == 0) p.ctx_out[b] = ok ? q.ctx + q.cnt : q.ctx;
}

struct ReadParams {
  const uint4 *k, *v;
  const uint8_t *ks, *vs;
  RowCache cache;
  int T, Hkv, lanes, gs;
  const int32_t *start, *count;
  uint4 *k_out, *v_out;          // [B, T, Hkv, d]
  uint32_t *dev_err;
};

template <class Tag>
BST_DEV uint4 pack_out(const float *f);
template <>
BST_DEV uint4 pack_out<F32Tag>(const float *f) { return pack16<F32Tag>(f); }
template <>
BST_DEV uint4 pack_out<BF16Tag>(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class Tag>
__global__ void __launch_bounds__(Q8_THREADS) kv_q8_read_kernel(const ReadParams p) {
  constexpr int OV = 16 / Tag::kVec;
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  pdl_wait();
  pdl_trigger();
  const int cnt = p.count[b];
  const int s = p.start[b];
  const bool first = blockIdx.x == 0 && !is_v && threadIdx.x == 0;
  if (cnt < 0 || cnt > p.T) {
    if (first) set_err(p.dev_err, BASTION_DEVERR_N);
    return;
  }
  if (s < 0 || static_cast<int64_t>(s) + cnt > cache_capacity(p.cache)) {
    if (first) set_err(p.dev_err, BASTION_DEVERR_CTX);
    return;
  }
  const int per_pass = Q8_THREADS / p.gs;
  const int lane_in_row = threadIdx.x & (p.gs - 1);
  const int r = blockIdx.x * per_pass * Q8_UNROLL + static_cast<int>(threadIdx.x) / p.gs;
  const int rows = cnt * p.Hkv;
  if (lane_in_row >= p.lanes) return;
  const uint4 *codes = is_v ? p.v : p.k;
  const uint8_t *scales = is_v ? p.vs : p.ks;
  uint4 *out = is_v ? p.v_out : p.k_out;
  uint4 in[Q8_UNROLL];
  uint32_t byte[Q8_UNROLL];
#pragma unroll
  for (int u = 0; u < Q8_UNROLL; ++u) {
    const int rr = r + u * per_pass;
    in[u] = make_uint4(0, 0, 0, 0);
    byte[u] = 0;
    if (rr < rows) {
      const int i = rr / p.Hkv, h = rr - i * p.Hkv;
      const int64_t src = cache_row(p.cache, p.Hkv, b, h, s + i);
      if (src >= 0) {
        in[u] = ld_stream16(codes + src * p.lanes + lane_in_row);
        byte[u] = __ldg(scales + src);
      } else {
        set_err(p.dev_err, BASTION_DEVERR_PAGE);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < Q8_UNROLL; ++u) {
    const int rr = r + u * per_pass;
    if (rr < rows) {
      const float sc = q8_scale(byte[u]);
      const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
      float f[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 two = e4m3x2_f32((w[i >> 1] >> ((i & 1) * 16)) & 0xffffu);
        f[2 * i] = two.x * sc;
        f[2 * i + 1] = two.y * sc;
      }
      uint4 *dst = out + ((static_cast<int64_t>(b) * p.T * p.Hkv + rr) * p.lanes + lane_in_row) * OV;
#pragma unroll
      for (int i = 0; i < OV; ++i) __stcs(dst + i, pack_out<Tag>(f + i * Tag::kVec));
    }
  }
}

// ------------------------------------------------------------------ host side
static int group_of(int lanes) {
  int g = 1;
  while (g < lanes) g <<= 1;
  return g;
}

cudaError_t launch_kv_write_q8(const void *k_new, const void *v_new, bool bf16, int B, int T, int Hkv, int d, int K,
                               const int32_t *count, const int32_t *nodes, void *k, void *v, uint8_t *ks, uint8_t *vs,
                               int64_t L_max, const int32_t *block_table, int max_pages, int num_pages, int page_size,
                               const int32_t *ctx_len, int32_t *ctx_out, uint32_t *dev_err, int sms,
                               cudaStream_t stream) {
  WriteParams p{};
  p.k_new = static_cast<const uint4 *>(k_new);
  p.v_new = static_cast<const uint4 *>(v_new);
  p.k = static_cast<uint4 *>(k);
  p.v = static_cast<uint4 *>(v);
  p.ks = ks;
  p.vs = vs;
  p.cache = RowCache{L_max, block_table, max_pages, num_pages, page_size};
  p.T = T;
  p.Hkv = Hkv;
  p.K = K;
  p.lanes = d / 16;
  p.gs = group_of(p.lanes);
  p.count = count;
  p.nodes = nodes;
  p.ctx_len = ctx_len;
  p.ctx_out = ctx_out;
  p.dev_err = dev_err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = fill_launch_attrs(attr);
  cfg.stream = stream;
  const int64_t most = static_cast<int64_t>(nodes ? K + 1 : T) * Hkv;
  // What one CTA takes in one pass goes to one CTA a request, in one launch; more to
  // a grid and a second launch that moves ctx_out (8 heads of 128, bf16, 1 and 16
  // requests: 8 tokens 4.0 us either, with a grid 4.9 and 5.0; 16 tokens, one pass, 4.7,
  // with a grid 5.0 and 5.1; 32 tokens in two passes 7.3 and 7.5, with a grid 4.8 and 5.2).
  if (2 * most <= Q8_ONE_THREADS / p.gs * Q8_ONE_UNROLL) {
    cfg.gridDim = dim3(B, 1, 1);
    cfg.blockDim = dim3(Q8_ONE_THREADS, 1, 1);
    return bf16 ? cudaLaunchKernelEx(&cfg, kv_q8_write_one_kernel<BF16Tag>, p)
                : cudaLaunchKernelEx(&cfg, kv_q8_write_one_kernel<F32Tag>, p);
  }
  const int per_pass = Q8_THREADS / p.gs * (bf16 ? q8_write_unroll<BF16Tag>() : q8_write_unroll<F32Tag>());
  const int64_t all = (2 * most + per_pass - 1) / per_pass;
  // Stretches so long that the page ids a CTA reads are at most 1/16 of the bytes that it
  // moves, as far as the grid still fills the GPU (131072 tokens of 8 heads of 128 in
  // bf16: pages of 8 192 us, of 64 182, of one token 260; one pass a CTA and page ids
  // one by one 294, 197 and 1165; without pages 154).
  const int64_t page_bytes = block_table ? 4 * (static_cast<int64_t>(T) / page_size + 1) : 0;
  const int64_t pass_bytes = static_cast<int64_t>(per_pass) * (d * (bf16 ? 2 : 4) + d + 1);
  const int64_t fill = std::max<int64_t>(1, all * B / (4 * sms));
  p.passes = static_cast<int>(std::min(fill, (16 * page_bytes + pass_bytes - 1) / pass_bytes));
  p.passes = std::max(p.passes, 1);
  cfg.gridDim = dim3(static_cast<unsigned>((all + p.passes - 1) / p.passes), B, 1);
  cfg.blockDim = dim3(Q8_THREADS, 1, 1);
  cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, kv_q8_write_kernel<BF16Tag>, p)
                       : cudaLaunchKernelEx(&cfg, kv_q8_write_kernel<F32Tag>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(B, 1, 1);
  cfg.blockDim = dim3(page_bytes > 4096 ? Q8_ONE_THREADS : Q8_THREADS, 1, 1);   // a thread for every four page ids or so
  return cudaLaunchKernelEx(&cfg, kv_q8_advance_kernel, p);
}

cudaError_t launch_kv_read_q8(const void *k, const void *v, const uint8_t *ks, const uint8_t *vs, int64_t L_max,
                              const int32_t *block_table, int max_pages, int num_pages, int page_size, bool bf16,
                              int B, int T, int Hkv, int d, const int32_t *start, const int32_t *count, void *k_out,
                              void *v_out, uint32_t *dev_err, cudaStream_t stream) {
  ReadParams p{};
  p.k = static_cast<const uint4 *>(k);
  p.v = static_cast<const uint4 *>(v);
  p.ks = ks;
  p.vs = vs;
  p.cache = RowCache{L_max, block_table, max_pages, num_pages, page_size};
  p.T = T;
  p.Hkv = Hkv;
  p.lanes = d / 16;
  p.gs = group_of(p.lanes);
  p.start = start;
  p.count = count;
  p.k_out = static_cast<uint4 *>(k_out);
  p.v_out = static_cast<uint4 *>(v_out);
  p.dev_err = dev_err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = fill_launch_attrs(attr);
  cfg.stream = stream;
  const int per_cta = Q8_THREADS / p.gs * Q8_UNROLL;
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(T) * Hkv + per_cta - 1) / per_cta), B, 2);
  cfg.blockDim = dim3(Q8_THREADS, 1, 1);
  return bf16 ? cudaLaunchKernelEx(&cfg, kv_q8_read_kernel<BF16Tag>, p)
              : cudaLaunchKernelEx(&cfg, kv_q8_read_kernel<F32Tag>, p);
}

}  // namespace bst
