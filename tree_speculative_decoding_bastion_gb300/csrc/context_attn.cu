// Attention of the tree tokens over an 8-bit context cache, or behind a prefix
// that the batch shares, on the tensor cores (bf16 inputs).
//
//   out[b,i,h] = softmax_j(q[b,i,h] . key_j * scale) value_j
//
// over the shared prefix, the request's own context and the tree nodes of the
// row's mask.  How the work is divided, and how partial results join:
// attn_work.cuh.
//
// Orientation.  A tile's scores are computed transposed, S^T = K Q^T with the
// 128 keys as the M rows of the MMA and the query rows as its N columns, and
// so is the output, O^T = V^T P^T with the d columns of V as M.  Both MMAs take
// K and V as they lie in the cache (K-major and MN-major), straight from TMA.
//   * N is chosen per piece (16, 32, 64 or 128 columns): a decoded token's few
//     rows cost an eighth of a full tile, not a full tile.
//   * A thread owns one key: that key's scale, its validity and its place in
//     the page are per-thread scalars, so the 8-bit cache's scales cost one
//     multiplication of a packed pair.
//   * Row maxima would cost reductions across lanes, so none is taken per tile:
//     scores are held against a row's reference (a maximum of earlier
//     tiles), and only where some score exceeds it by more than 2^TH, which a
//     vote of the tile's threads finds, are new references reduced, 2^HEAD above
//     the maximum, and O rescaled.  The result does not depend on the reference.
//
// 8-bit tiles.  K's and V's codes enter the MMA as they are (kind::f8f6f4);
// Q and P are split into 8-bit parts, so that what they lose stays below what the
// bf16 output loses:
//   Q 2^-e = hi + lo, both e4m3, e the row's scale exponent (q8.cuh) or at most
//     3 more: a bf16 has eight significant bits, hi takes the upper four
//     (rounded), the signed remainder fits the four of lo -- the sum is exact for
//     elements of at least 2^-6.8 of the row's amax, and off by at most 2^-10 2^e,
//     2^-14 of the amax, below.
//   The weights that meet the codes are those times their key's V scale, u =
//     2^(score + ev); a row's reference is a maximum of score + ev, so u is held
//     against the row's largest u.  u 2^8 = hi + mid + lo, all e5m2, by way of f16: hi
//     and mid are cut off after three significant bits of what is left, lo is
//     rounded to its three.  Of an f16's eleven bits two at most are then lost: off
//     by at most 2^-9 relative, with the f16's rounding 2^-8.8 (a bf16 2^-8), 2^-11
//     in the mean square and of either sign.  The smallest step of an e5m2 is 2^-16 and the row's
//     largest weight lies at 2^7 at least (up to 2^15): a weight below 2^-15 of the
//     largest is off by up to 2^-24 of it instead.  (With two parts, e5m2 and
//     e4m3, a weight below 2^-12 of the largest had three bits: 20000 equal keys
//     behind a sink came out off by 3%.)
// The tree's own keys and values are bf16 and use kind::f16 with the bf16 Q,
// on the same accumulators.
//
// Roles: warps 0-15 softmax (warp w: keys 32 (w mod 4) .. + 31, the lanes of
// its TMEM quarter; row group w / 4), warp 16 TMA producer of K, warp 19 of V,
// warp 17 MMA issuer, warp 18 the records of attn_work.cuh.
// S^T passes through two TMEM buffers, P through two in shared memory (128 rows with
// an 8-bit cache: one), K and
// V through a ring of slots (of a tile of the cache's type, 128 x d codes or
// bf16; in an 8-bit cache's ring a bf16 tree tile takes two) in the order in which
// the MMAs take them, K0 K1 V0 K2 V1 ..: a freed slot is filled at once, where in
// the order K0 V0 K1 V1 .. the copy of K waited behind that of the V before it,
// whose slot is freed a tile later.  A piece's tiles of one size form a section
// (context tiles and tree tiles of an 8-bit cache are two, else all are one): of m
// tiles, K(0) is its item 0, K(i) item 2 i - 1, V(i) item 2 i + 2, the last V item
// 2 m - 1.
// Measured: a CTA begins its first tile 5 us after launch (the partition 2, Q, the
// first references); then an 8-bit tile of 128 rows takes 4.9 thousand cycles, bound by the
// softmax's instructions (issue slots 50% busy, tensor pipe 29%: 4 trees of 128
// over 32768 keys 531 us), a bf16 one 2.4 thousand (16 trees behind 16381 shared
// keys 235 us), an 8-bit tile of few rows 1.9 thousand, bound by latency (16 tokens
// over 512 to 8192 keys 45.5 us, 3.5 TB/s).
// Every mbarrier wait is bounded in time; after an expiry the CTA issues no
// further copies, walks its loops to the end with at most two polls a wait and
// reports BASTION_DEVERR_TIMEOUT.
#include <type_traits>

#include "context_attn.cuh"
#include "sm100_ptx.cuh"

namespace bst {

constexpr int CT_THREADS = 640;         // five warpgroups: softmax four times, then TMA of K, MMA, records, TMA of V
constexpr int CT_SM = 512;              // softmax threads
constexpr int CT_GROUPS = 4;            // row groups: one warpgroup each
constexpr int CT_K_WARP = 16;            // TMA producers
constexpr int CT_MMA_WARP = 17;
constexpr int CT_V_WARP = 19;
constexpr int CT_R = 128;               // rows per tile
constexpr int CT_SBUF = 2;              // S^T buffers: S(j + 2) is issued after P V(j), which follows P(j)
constexpr int CT_LOOK = 2;              // S^T tiles issued ahead of P V
constexpr int CT_MAX_SLOTS = 16;
constexpr uint64_t CT_WAIT_NS = 200ull * 1000ull * 1000ull;
constexpr float CT_UNSET = -1e30f;      // reference of a row that has seen no key

struct CtxParams {
  AttnWork w;
  CtxGeo own, prefix;
  const uint16_t *q;
  const uint16_t *vt;                   // the tree's values (their size; the tiles come by TMA)
  const uint32_t *mask;                 // 32-bit words of the ancestor masks
  float scale_log2;
  uint16_t *out;
};

struct CtxBars {
  uint64_t q_full;                      // the piece's Q (a warp's arrival each)
  uint64_t full[CT_MAX_SLOTS], empty[CT_MAX_SLOTS];
  uint64_t s_full[CT_SBUF];
  uint64_t p_full[2];                   // P of a tile (16 arrivals: a softmax warp's each, or two of half the warps)
  uint64_t pv_done[2];                  // P V of the buffer's tile finished: buffer free, O updated
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int unset[CT_GROUPS];                 // a row of the group has seen no key yet
  int top_ctx, top_tree;                // 8-bit cache: largest V scale byte of the piece's keys, and the one that the tree's values would have
  AttnShare share;
};

// RM: the most rows of a piece, 128, or 64 in calls whose units have no more
// (launch_ctx_attn): half the room for Q and P, and more for K and V in flight.
template <int D, bool Q8, int RM>
struct CtxLayout {
  static constexpr int SLOT = CA_KEYS * D * (Q8 ? 1 : 2);   // a tile of the cache's keys or of its values
  static constexpr int WIDE = Q8 ? 2 : 1;               // slots of a bf16 tile
  static constexpr int QB = RM * D * 2;                 // Q in bf16
  static constexpr int Q8B = RM == 64 ? 128 * 128 : QB; // ... in two 8-bit parts
  // P in tiles of 128 keys x 128 bytes.  bf16: a tile of 64 rows.  8-bit: 128 rows of a
  // part, or 64 of two side by side.  Without an 8-bit cache two buffers.  With one,
  // three tiles: of 128 rows the three parts of one buffer (the pass that tests a
  // tile's scores comes before any weight is written, and P V of the tile before is
  // done by then); of up to 64 rows, whose streams are independent, two buffers of
  // hi and mid, and a tile of both buffers' lo.
  static constexpr int PT = CA_KEYS * 128;
  static constexpr int P_TILES = Q8 ? 3 : RM / 32;
  static BST_DEV int p_buffer(bool two, int pb) { return Q8 ? (two ? pb * PT : 0) : pb * (RM / 64) * PT; }
  static BST_DEV int p_mid(bool two) { return two ? 64 : PT; }                       // from hi
  static BST_DEV int p_lo(bool two, int pb) { return two ? (2 - pb) * PT + pb * 64 : 2 * PT; }
  static constexpr int Q16_OFF = 0;
  static constexpr int Q8_OFF = QB;
  static constexpr int RING_OFF = Q8 ? QB + Q8B : QB;
  // what 227 KB leave: head_dim 128: 6 slots with an 8-bit cache, 4 without (64 rows: 8 and 5)
  static constexpr int ROOM = (227 * 1024 - RING_OFF - P_TILES * PT - 3 * 1024) / SLOT;
  static constexpr int SLOTS = (ROOM < CT_MAX_SLOTS ? ROOM : CT_MAX_SLOTS) / WIDE * WIDE;
  static constexpr int P_OFF = RING_OFF + SLOTS * SLOT;
  static constexpr int MREF_OFF = P_OFF + P_TILES * PT;  // float[128] references
  static constexpr int QSC_OFF = MREF_OFF + 512;        // float[128] (8-bit cache) row scale of the 8-bit Q times scale log2(e)
  // int[128] maxima as ordered integers, lowest between uses; then the rises of
  // the references, at the end the rows' factors (floats)
  static constexpr int XM_OFF = QSC_OFF + 512;
  static constexpr int TAB_OFF = XM_OFF + 512;          // int[128] row table
  static constexpr int BAR_OFF = TAB_OFF + 512;
  static constexpr int USED = BAR_OFF + 512;
  // at least 120 KB: one CTA owns the SM and its 512 TMEM columns
  static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static_assert(sizeof(CtxBars) <= 512, "barriers");
  static_assert(USED <= 227 * 1024, "exceeds the shared memory of one CTA");
  // (at least three tiles of the larger kind: the producers' waits by parity, see `take`)
  static_assert(SLOTS >= 3 * WIDE && SLOTS % WIDE == 0, "ring");
};

// One lane of a converged warp.
BST_DEV uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// The MMA, and its commit, issued by the lane whose `leader` is set.
BST_DEV void mma_if(uint32_t leader, bool f8, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                    uint32_t accumulate) {
  if (f8)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
BST_DEV void commit_if(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// Instruction descriptor: D fp32, formats of A and B (kind::f16: 1 = bf16;
// kind::f8f6f4: 0 = e4m3, 1 = e5m2), majorness (1 = MN), M = 128, N.
BST_DEV uint32_t ctx_idesc(int afmt, int bfmt, int a_mn, int b_mn, int N) {
  return (1u << 4) | (static_cast<uint32_t>(afmt) << 7) | (static_cast<uint32_t>(bfmt) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
// Shared-memory descriptor, 64-byte swizzle (layout 4); the 128-byte one is sdesc_sw128.
BST_DEV uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | 1ull << 46 | 4ull << 61;
}

// 32 lanes x 8 consecutive columns per thread
BST_DEV void tmem_ld8(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : BST_R8(r, 0) : "r"(taddr));
}
BST_DEV void tmem_wait_ld8(uint32_t *r) { asm volatile("tcgen05.wait::ld.sync.aligned;" : BST_W8(r, 0)::"memory"); }
BST_DEV void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), BST_I8(r, 0)
               : "memory");
}
// 8 NC columns (NC 1, 2 or 4), waited for
template <int NC>
BST_DEV void tmem_ld_rows(uint32_t taddr, uint32_t *s) {
  if constexpr (NC == 4) {
    tmem_ld32(taddr, s);
    tmem_wait_ld32(s);
  } else if constexpr (NC == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : BST_R8(s, 0), BST_R8(s, 8)
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : BST_W8(s, 0), BST_W8(s, 8)::"memory");
  } else {
    tmem_ld8(taddr, s);
    tmem_wait_ld8(s);
  }
}

// Named barriers of the softmax warps: 1 to 4 the row groups, 5 all.
BST_DEV void bar_group(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
BST_DEV bool vote_group(int g, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + g), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
BST_DEV void bar_softmax() { asm volatile("bar.sync 5, 512;" ::: "memory"); }
// One arrival of a warp whose lanes wrote shared memory for the tensor core.
BST_DEV void warp_arrive(uint64_t *bar, uint32_t count) {
  fence_proxy_async();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// order-preserving float <-> int (signed comparison)
BST_DEV int ordered(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
BST_DEV float unordered(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }
constexpr int ORDERED_LOWEST = static_cast<int>(0x807fffffu);   // ordered(-inf)

// maximum over the warp (NaN left out)
BST_DEV float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
BST_DEV float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
BST_DEV uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A pair of weights as f16, whose upper byte is the e5m2 that it is cut off to.
BST_DEV uint32_t weight_pair(float2 v) {
  uint32_t h;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v.y), "f"(v.x));
  return h;
}
// The upper bytes of two pairs (four codes), and what a pair has left without them (exact).
BST_DEV uint32_t upper_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
BST_DEV uint32_t without_upper(uint32_t h) {
  uint32_t rest;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(h & 0xff00ff00u));
  return rest;
}
// A pair rounded to e5m2 codes (16 bits).
BST_DEV uint32_t e5m2_pair(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// A pair of scaled query elements (at most 448) as e4m3 codes hi and lo.
BST_DEV void split_query(float2 v, uint32_t &hi, uint32_t &lo) {
  uint32_t h, back, rest;
  uint16_t a, b;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v.y), "f"(v.x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(rest));
  hi = a;
  lo = b;
}
BST_DEV uint32_t two16(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
// MMA columns of a piece of `rows` rows
BST_DEV int columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// 2^k as a float (0 below the normals, at most 2^127)
BST_DEV float pow2i(int k) { return k < -126 ? 0.f : __int_as_float((min(k, 127) + 127) << 23); }

// What a softmax thread knows of its key in one tile.
struct CtxKey {
  bool valid;
  float ck;     // 2^(exponent of the K scale)
  int ev;       // exponent of the V scale
};

// Position of the softmax warps in the CTA's whole range: S^T / P tiles and
// ring slots before the current piece.
struct CtxCounts {
  int tiles, slots;
};

template <int D, bool Q8, int RM>
struct CtxSoftmax {
  using LY = CtxLayout<D, Q8, RM>;
  // How far a score (with its V scale) may exceed its row's reference (log2)
  // before the reference is raised, and how far above the row's largest score it is
  // then set.  A larger sum of the two means fewer changes.  bf16 weights are exact
  // to their eight bits at any size, so HEAD costs nothing but the last 2^16 of the
  // fp32 range downwards; a weight is at most 2^8, as in the attention over
  // bf16 caches alone, and O stays finite while keys x |V| is below 2^120
  // (16 trees behind 16381 shared keys: 231 us; HEAD 8 238, HEAD 0 305, before the
  // sum took the rounded weights).
  // The 8-bit parts have no such room (SHIFT + TH = 15: the largest weight is then
  // 2^15, an f16).  A larger SHIFT means finer small weights; where the sizes of keys vary
  // as e^(N/2), TH = 4 is exceeded in a quarter of a range's tiles, 7 in an eighth.
  static constexpr float TH = Q8 ? 7.f : 8.f;
  static constexpr float HEAD = Q8 ? 0.f : 16.f;
  static constexpr int SHIFT = 8;
  static constexpr int LOWEST = -100;  // smallest exponent that V scales are held against

  // The largest scale byte of the V rows of the piece's context that this thread
  // looks at (byte 255 is a NaN, not a size).  Eight keys at a time where the scales lie
  // in aligned words of eight: a read of 1/128 of the piece's bytes.  (A key at a time: 16
  // single tokens over 512 to 8192 keys 61 us for 56.  What it costs beside taking the
  // exponent from the first keys, which later ones may exceed by far: there 55, for
  // 64 single tokens behind 8192 keys, with 512 short units, 45 -> 48.)
  static BST_DEV int top_context(const CtxParams &p, const AttnPiece &pc, int tid) {
    const CtxGeo &geo = pc.prefix ? p.prefix : p.own;
    const int first = pc.t0 * CA_KEYS, stop = min(pc.L, min(pc.t1, pc.ctx_tiles) * CA_KEYS);
    const bool paged = geo.rows.block_table != nullptr;
    const bool words = ((reinterpret_cast<uintptr_t>(geo.vs) | (paged ? 0 : geo.rows.L_max)) & 7) == 0;
    const int shift = paged ? 31 - __clz(geo.rows.page_size) : 0;
    const int32_t *pages = paged ? geo.rows.block_table + static_cast<int64_t>(pc.b) * geo.rows.max_pages : nullptr;
    const uint32_t base = static_cast<uint32_t>(paged ? pc.kvh : (static_cast<int64_t>(pc.b) * p.w.Hkv + pc.kvh) * geo.rows.L_max);
    auto scale_at = [&](int key) -> const uint8_t * {          // NULL: a bad page
      uint32_t row = base + static_cast<uint32_t>(key);
      if (paged) {
        const uint32_t page = static_cast<uint32_t>(__ldg(pages + (key >> shift)));
        if (page >= static_cast<uint32_t>(geo.rows.num_pages)) return nullptr;
        row = ((page * static_cast<uint32_t>(p.w.Hkv) + base) << shift) + (key & ((1 << shift) - 1));
      }
      return geo.vs + row;
    };
    if (words) {
      uint32_t top4 = 0;
#pragma unroll 4
      for (int key = first + 8 * tid; key < stop; key += 8 * CT_SM) {
        const uint8_t *at = scale_at(key);
        if (!at) continue;
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(at));
        const int n = stop - key;              // bytes that count
        const uint32_t m0 = n >= 4 ? ~0u : ~(~0u << (8 * n)), m1 = n >= 8 ? ~0u : n <= 4 ? 0u : ~(~0u << (8 * (n - 4)));
        const uint32_t a = w.x & m0 & ~__vcmpeq4(w.x, ~0u), c = w.y & m1 & ~__vcmpeq4(w.y, ~0u);
        top4 = __vmaxu4(top4, __vmaxu4(a, c));
      }
      return static_cast<int>(max(max(top4 & 255u, (top4 >> 8) & 255u), max((top4 >> 16) & 255u, top4 >> 24)));
    }
    int top = 0;
#pragma unroll 4
    for (int key = first + tid; key < stop; key += CT_SM) {
      const uint8_t *at = scale_at(key);
      const int byte = at ? __ldg(at) : 0;
      top = max(top, byte == 255 ? 0 : byte);
    }
    return top;
  }
  // ... and the one that the tree's values would have as one row.
  static BST_DEV int top_tree(const CtxParams &p, const AttnPiece &pc, int tid) {
    if (pc.t1 <= pc.ctx_tiles) return 0;
    constexpr int CPR = D / 8;                 // 16-byte chunks of a row
    uint32_t top = 0;
#pragma unroll 2
    for (int i = tid; i < pc.nb * CPR; i += CT_SM) {
      const int64_t row = (static_cast<int64_t>(pc.b) * p.w.n_max + i / CPR) * p.w.Hkv + pc.kvh;
      float x[8];
      unpack16<BF16Tag>(__ldg(reinterpret_cast<const uint4 *>(p.vt + row * D) + i % CPR), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, finite_abs_bits(x[e]));
    }
    return static_cast<int>(q8_scale_byte(top));
  }

  // The piece's rows of Q into shared memory: bf16 for bf16 tiles, two e4m3
  // parts and the row scale for 8-bit ones.
  // With fewer than 128 rows the two parts are one operand of twice the rows (lo
  // behind hi), and the sum of their scores is taken on the way out of TMEM: half
  // as many MMAs, whose count and not whose size costs there.
  // Returns the rows' common scale (times scale log2(e)) where there is one, else
  // 0: rows whose own scales lie within 2^COMMON take the largest, which saves two
  // multiplications a score (4 trees of 128 over 32768 keys: 527 us for 566, 16 trees of
  // 8 to 64 204 for 214) and costs elements below 2^-6.8 (not 2^-9.8) of a row's amax
  // their last bits: a score is off by at most 2^-14 amax scale sum |k| over those, in a
  // row whose largest element is 30 times the others some 3e-4 in the mean square, a
  // tenth of what the bf16 rounding of q itself was.
  static constexpr int COMMON = 3;
  static BST_DEV float load_q(const CtxParams &p, uint8_t *smem, CtxBars *bars, const AttnPiece &pc, int rows, int tid) {
    const bool need16 = !Q8 || pc.t1 > pc.ctx_tiles, need8 = Q8 && pc.t0 < pc.ctx_tiles;
    constexpr int CPR = D / 8;                 // 16-byte chunks of a row
    constexpr int STEP = CT_SM / CPR;          // rows per pass
    const int *table = reinterpret_cast<const int *>(smem + LY::TAB_OFF);
    const int c = tid % CPR;
    uint4 v[RM / STEP];
#pragma unroll
    for (int i = 0; i < RM / STEP; ++i) {
      const int r = tid / CPR + i * STEP;
      v[i] = make_uint4(0, 0, 0, 0);
      if (i * STEP < rows) {
        const int at = table[r];
        if (at >= 0) v[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(at) * D) + c);
      }
    }
    if constexpr (Q8) {                        // the sizes of V, while the rows are on their way
      const int ctx = __reduce_max_sync(FULL, top_context(p, pc, tid)), tree = __reduce_max_sync(FULL, top_tree(p, pc, tid));
      if ((tid & 31) == 0) atomicMax(&bars->top_ctx, ctx), atomicMax(&bars->top_tree, tree);
    }
    float common = 0.f;
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < RM / STEP; ++i) {
        const int r = tid / CPR + i * STEP;
        if (i * STEP < rows) store_q16(smem, r, c, v[i]);
      }
    } else {
      int *bytes = reinterpret_cast<int *>(smem + LY::XM_OFF);   // the rows' scale bytes (xm is free before the first tile)
#pragma unroll
      for (int i = 0; i < RM / STEP; ++i) {
        const int r = tid / CPR + i * STEP;
        if (i * STEP < rows) {                 // uniform over the softmax warps
          if (need16) store_q16(smem, r, c, v[i]);
          if (need8) {
            const uint32_t m = 0x7fff7fffu;
            uint32_t mx = __float_as_uint(vmax16<BF16Tag>(make_uint4(v[i].x & m, v[i].y & m, v[i].z & m, v[i].w & m)));
            if (__any_sync(FULL, mx >= 0x7f800000u)) {   // infinities, or nothing but NaN: over the finite elements
              float x[8];
              unpack16<BF16Tag>(v[i], x);
              mx = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) mx = max(mx, finite_abs_bits(x[e]));
            }
#pragma unroll
            for (int o = CPR / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(FULL, mx, o));
            if (c == 0) bytes[r] = static_cast<int>(q8_scale_byte(mx));
          }
        }
      }
      bar_softmax();
      if (need8) {
        int hi_byte = 0, lo_byte = 255;        // over the rows that are not zero
        for (int r = tid & 31; r < rows; r += 32) {
          const int y = bytes[r];
          hi_byte = max(hi_byte, y);
          if (y > 0) lo_byte = min(lo_byte, y);
        }
        hi_byte = __reduce_max_sync(FULL, hi_byte);
        lo_byte = __reduce_min_sync(FULL, lo_byte);
        const bool same = hi_byte - lo_byte <= COMMON;
        if (same) common = q8_scale(static_cast<uint32_t>(hi_byte)) * p.scale_log2;
#pragma unroll
        for (int i = 0; i < RM / STEP; ++i) {
          const int r = tid / CPR + i * STEP;
          if (r < rows) {                      // (a pass may reach beyond the rows)
            float x[8];
            unpack16<BF16Tag>(v[i], x);
            const uint32_t byte = static_cast<uint32_t>(same ? hi_byte : bytes[r]);
            const float inv = q8_inv_scale(byte);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)   // (an infinite element has no finite score: inf - inf makes it NaN)
              split_query(make_float2(fmaf(x[2 * e], inv, x[2 * e] - x[2 * e]), fmaf(x[2 * e + 1], inv, x[2 * e + 1] - x[2 * e + 1])),
                          hi[e], lo[e]);
            // 128 rows: two tiles of 128-byte rows (head_dim 64: both parts side by side in one)
            uint8_t *base = smem + LY::Q8_OFF;
            const int ch = c >> 1, sub = (c & 1) * 8;
            const bool beside = D == 64 && rows == CT_R;
            const int rl = r + (beside ? 0 : rows), cl = ch + (beside ? 4 : 0);
            *reinterpret_cast<uint2 *>(base + r * 128 + ((ch ^ (r & 7)) << 4) + sub) = make_uint2(two16(hi[0], hi[1]), two16(hi[2], hi[3]));
            *reinterpret_cast<uint2 *>(base + rl * 128 + ((cl ^ (rl & 7)) << 4) + sub) = make_uint2(two16(lo[0], lo[1]), two16(lo[2], lo[3]));
            if (c == 0) reinterpret_cast<float *>(smem + LY::QSC_OFF)[r] = q8_scale(byte) * p.scale_log2;
          }
        }
      }
      bar_softmax();                           // the scale bytes are read
      if (tid < CT_R) bytes[tid] = ORDERED_LOWEST;
    }
    return common;
  }
  static BST_DEV void store_q16(uint8_t *smem, int r, int c, const uint4 &v) {
    *reinterpret_cast<uint4 *>(smem + LY::Q16_OFF + (c >> 3) * (RM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
  }

  // C of this thread's columns of TMEM.
  template <int C>
  static BST_DEV void load_columns(uint32_t t, float (&x)[C]) {
    uint32_t s[C];
    tmem_ld_rows<C / 8>(t, s);
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = __uint_as_float(s[i]);
  }
  // C of this thread's rows of S^T, raw (an 8-bit tile: not yet times the row's
  // scale of Q); LO > 0: the scores of Q's lo part lie LO columns on.
  template <int C, int LO>
  static BST_DEV void raw_scores(uint32_t tS, float (&x)[C]) {
    load_columns<C>(tS, x);
    if constexpr (LO > 0) {
#pragma unroll
      for (int c = 0; c < C; c += 8) {
        float y[8];
        load_columns<8>(tS + LO + c, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c + i] += y[i];
      }
    }
  }
  // ... against the references, in the log2 domain: S row_scale ck - m.  `own`:
  // the rows' scales are not in cs2 already.
  template <int C, bool F8, bool REF>
  static BST_DEV void against(bool own, const float *qsc, float2 cs2, const float *mref, float (&x)[C]) {
    if (F8 && own) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(qsc + i);
        const float2 a = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(q.x, q.y));
        const float2 b = __fmul2_rn(make_float2(x[i + 2], x[i + 3]), make_float2(q.z, q.w));
        x[i] = a.x, x[i + 1] = a.y, x[i + 2] = b.x, x[i + 3] = b.y;
      }
    }
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[i + 2], x[i + 3]);
      if constexpr (REF) {
        const float4 m = *reinterpret_cast<const float4 *>(mref + i);
        a = __ffma2_rn(a, cs2, make_float2(-m.x, -m.y));
        b = __ffma2_rn(b, cs2, make_float2(-m.z, -m.w));
      } else {
        a = __fmul2_rn(a, cs2);
        b = __fmul2_rn(b, cs2);
      }
      x[i] = a.x, x[i + 1] = a.y, x[i + 2] = b.x, x[i + 3] = b.y;
    }
  }
  // Scores that the rows of a tree tile do not see (bits: lane i holds row i's mask over the warp's keys).
  template <int C>
  static BST_DEV void hide(uint32_t bits, int first, bool valid, float (&x)[C]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint32_t w = __shfl_sync(FULL, bits, first + i);
      if (!valid || !((w >> lane) & 1u)) x[i] = -CUDART_INF_F;
    }
  }

  // C <= 32 values per lane summed over the 32 lanes: lane i < C returns value i's sum.
  template <int C>
  static BST_DEV float across_lanes(float (&v)[C]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
    // lanes beyond the values first fold onto them
#pragma unroll
    for (; o >= C; o >>= 1) {
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] += __shfl_xor_sync(FULL, v[i], o);
    }
#pragma unroll
    for (; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float keep = (lane & o) ? v[i + o] : v[i];
        const float send = (lane & o) ? v[i] : v[i + o];
        v[i] = keep + __shfl_xor_sync(FULL, send, o);
      }
    }
    return v[0];
  }

  // One piece.  With 128 columns of S^T every row group takes a quarter of each
  // tile's rows.  With fewer (TWO) there are two streams, the even and the odd tiles
  // of the CTA: groups 0 and 1 take half the rows each of one, groups 2 and 3
  // of the other, with references, sums and an O of their own, which are joined
  // at the end -- a tile of few rows costs its latencies, so two are in flight.
  // HR rows per group; arrays of per-row state hold stream s at 64 s.
  template <int HR, bool TWO>
  static BST_DEV void piece(const CtxParams &p, uint8_t *smem, CtxBars *bars, const AttnPiece &pc, CtxCounts &cnt,
                            uint32_t tbase, int cta, float common) {
    constexpr int C = HR < 16 ? HR : 16;     // rows handled together: scores are not kept between passes
    constexpr int STEP = TWO ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kq = warp & 3, grp = warp >> 2;
    const int key = kq * 32 + lane;
    const int stream = TWO ? grp >> 1 : 0;
    const int r0 = (TWO ? grp & 1 : grp) * HR;   // first row
    const int v0 = stream * 64 + r0;             // its place in the state
    const uint32_t lane_off = static_cast<uint32_t>(kq * 32) << 16;
    const uint32_t tO = tbase + CT_SBUF * 128 + lane_off + v0;
    volatile int *abort = &bars->abort;
    float *mref = reinterpret_cast<float *>(smem + LY::MREF_OFF) + v0;
    float *rise = reinterpret_cast<float *>(smem + LY::XM_OFF) + v0;
    int *xm = reinterpret_cast<int *>(smem + LY::XM_OFF) + v0;
    const float *qsc = reinterpret_cast<const float *>(smem + LY::QSC_OFF) + r0;
    const int *table = reinterpret_cast<const int *>(smem + LY::TAB_OFF) + r0;
    const CtxGeo &geo = pc.prefix ? p.prefix : p.own;
    const AttnWork &w = p.w;
    const bool paged = geo.rows.block_table != nullptr;
    const uint8_t *const k_scales = geo.ks, *const v_scales = geo.vs;
    const uint32_t num_pages = static_cast<uint32_t>(geo.rows.num_pages);

    float2 l[HR / 2];
#pragma unroll
    for (int i = 0; i < HR / 2; ++i) l[i] = make_float2(0.f, 0.f);
    // The exponent that V scales are held against: the largest of the piece, so that no
    // key's lies above, and at least LOWEST (values below 2^-100 may come out as zero).
    const int E = Q8 ? max(max(bars->top_ctx, bars->top_tree), LOWEST + 127) - 127 : 0;
    const int ev_tree = Q8 ? max(bars->top_tree, LOWEST + 127) - 127 : 0;
    bool unset = true;       // uniform over the group: a row has seen no key
    float low = 0.f;         // bf16 tiles: the lowest of the rows' references
    const bool own = common == 0.f;          // 8-bit tiles: every row of Q has a scale of its own
    const int t_first = pc.t0 + (TWO ? (stream ^ cnt.tiles) & 1 : 0);
    // the thread's key of its next tile: scales loaded a tile ahead, the page two
    const int shift = paged ? 31 - __clz(geo.rows.page_size) : 0;
    const int32_t *pages = paged ? geo.rows.block_table + static_cast<int64_t>(pc.b) * geo.rows.max_pages : nullptr;
    const uint32_t base = paged ? static_cast<uint32_t>(pc.kvh)
                                : static_cast<uint32_t>((static_cast<int64_t>(pc.b) * w.Hkv + pc.kvh) * geo.rows.L_max);
    const int stop = min(pc.L, pc.t1 * CA_KEYS);             // keys from here on are not this piece's
    bool bad_page = false, ok_n = false;
    uint32_t kb_n = 0, vb_n = 0;
    int page_n = 0;
    auto next_page = [&](int pos) {
      if (paged && pos < stop) page_n = __ldg(pages + (pos >> shift));
    };
    auto next_key = [&](int pos) {
      ok_n = pos < stop;
      uint32_t row = base + static_cast<uint32_t>(pos);
      if (paged) {
        const bool bad = static_cast<uint32_t>(page_n) >= num_pages;
        bad_page = bad_page || (ok_n && bad);
        ok_n = ok_n && !bad;
        row = ((static_cast<uint32_t>(page_n) * static_cast<uint32_t>(w.Hkv) + base) << shift) + (pos & ((1 << shift) - 1));
      }
      if (Q8 && ok_n) kb_n = __ldg(k_scales + row), vb_n = __ldg(v_scales + row);
      next_page(pos + STEP * CA_KEYS);
    };
    next_page(t_first * CA_KEYS + key);
    next_key(t_first * CA_KEYS + key);

    auto tile = [&](auto f8_, auto tree_, int t) {
      constexpr bool F8 = decltype(f8_)::value, TREE = decltype(tree_)::value;
      constexpr int LO = F8 && TWO ? 2 * HR : 0;
      const int idx = cnt.tiles + t - pc.t0;                  // of all the CTA's tiles
      // ---- this thread's key
      CtxKey kx;
      uint32_t bits = 0u;
      if constexpr (TREE) {
        kx.valid = (t - pc.ctx_tiles) * CA_KEYS + key < pc.nb;
        kx.ck = 1.f;
        kx.ev = ev_tree;
        // lane i: the mask word of row i over this warp's keys
        const int W32 = ((w.n_max + 63) >> 6) * 2;
        const int word = (t - pc.ctx_tiles) * 4 + kq;
        const int at = lane < HR ? table[lane] : -1;
        if (at >= 0 && word < W32) bits = __ldg(p.mask + static_cast<int64_t>(at / w.Hq) * W32 + word);
      } else {
        kx.valid = ok_n;
        // (a V scale that is the format's NaN, too, makes the key's scores NaN: it
        // turns every row that sees it into NaN)
        kx.ck = F8 ? q8_scale(vb_n == 255u ? 255u : kb_n) : 1.f;
        kx.ev = F8 ? static_cast<int>(vb_n) - 127 : 0;
        next_key((t + STEP) * CA_KEYS + key);
      }
      const bool masked = TREE || paged || (t + 1) * CA_KEYS > pc.L;
      const int sb = idx % CT_SBUF;
      const uint32_t tS = tbase + lane_off + sb * 128 + r0;
      // (S^T of a tile is issued after P V of the tile two before it: that one's P
      // buffer is free and its O complete when this wait is over)
      mbar_wait(&bars->s_full[sb], (idx / CT_SBUF) & 1, abort, CT_WAIT_NS);
      __syncwarp();
      tc_fence_after();
      const float cs = F8 ? (own ? kx.ck : kx.ck * common) : p.scale_log2;
      const float2 cs2 = make_float2(cs, cs);
      // What the key adds to a score that is held against a reference (log2): its V
      // scale, but no less than TH - 64, so that the row sum, which V scales do not
      // enter, stays finite (a score is at most 2^64 above its reference).
      const float lift = Q8 ? fmaxf(static_cast<float>(kx.ev - E), TH - 64.f) : 0.f;
      // ---- do the rows' references hold for this tile?
      bool raised = unset;
      if (!unset) {
        auto largest = [](const float (&x)[C]) {
          float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < C; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
          return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        };
        // bf16: the largest raw score against the lowest reference, which with 2^24 of
        // room settles nearly every tile (8-bit, with 2^7: no gain measured); then
        // row by row.  (In chunks, as all passes: half the scores in registers took
        // 456 and 229 us where all at once took 459 and 232, with the spills.)
        bool over = true, mine = false;
        if (!TREE && !F8) {
          float most = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < HR; c += C) {
            float x[C];
            raw_scores<C, LO>(tS + c, x);
            most = fmaxf(most, largest(x));
          }
          over = vote_group(grp, kx.valid && fmaf(most, cs, -low) > TH);
        }
        if (over) {
          float most = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < HR; c += C) {
            float x[C];
            raw_scores<C, LO>(tS + c, x);
            against<C, F8, true>(own, qsc + c, cs2, mref + c, x);
            if constexpr (TREE) hide<C>(bits, c, kx.valid, x);
            most = fmaxf(most, largest(x));
          }
          mine = kx.valid && most + lift > TH;
          over = vote_group(grp, mine);
        }
        raised = over;
        if (raised && __any_sync(FULL, mine)) {
          // the few scores above the threshold raise their rows' references, by
          // whole powers of two
#pragma unroll
          for (int c = 0; c < HR; c += C) {
            float y[C];
            raw_scores<C, LO>(tS + c, y);
            against<C, F8, true>(own, qsc + c, cs2, mref + c, y);
            if constexpr (TREE) hide<C>(bits, c, kx.valid, y);
            if (kx.valid) {
#pragma unroll
              for (int i = 0; i < C; ++i) {
                const float z = y[i] + lift;
                if (z > TH) atomicMax(&xm[c + i], ordered(z));
              }
            }
          }
        }
      } else {
        // a row without a reference (the piece's first tile): the maxima over
        // this tile's keys, for all rows
        if (t != t_first) bar_group(grp);    // the last such tile's flag and maxima are read and reset
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < HR; c += C) {
          float x[C];
          raw_scores<C, LO>(tS + c, x);
          against<C, F8, false>(own, qsc + c, cs2, mref + c, x);
          if constexpr (TREE) hide<C>(bits, c, kx.valid, x);
#pragma unroll
          for (int i = 0; i < C; ++i) {
            const float r = warp_max(kx.valid ? x[i] + lift : -CUDART_INF_F);
            if (lane == c + i) mx = r;
          }
        }
        if (lane < HR) atomicMax(&xm[lane], ordered(mx));
        if (key == 0) bars->unset[grp] = 0;
      }
      if (raised) {
        const bool started = t != t_first;
        bar_group(grp);
        if (key < HR) {                      // a thread settles a row
          const int o = xm[key];
          const float mo = mref[key];
          float up, mn;
          if (unset) {
            const float top = unordered(o);
            mn = isnan(top) ? 0.f : fmaxf(mo, top + HEAD);   // (a NaN is a seen key; its row stays NaN)
            up = mn - mo;
            if (mn == CT_UNSET && table[key] >= 0) bars->unset[grp] = 1;
          } else {
            up = o == ORDERED_LOWEST ? 0.f : ceilf(unordered(o)) + HEAD;
            mn = mo + up;
          }
          mref[key] = mn;
          if (started)
            rise[key] = up;
          else
            xm[key] = ORDERED_LOWEST;
        }
        bar_group(grp);
        unset = *const_cast<volatile int *>(&bars->unset[grp]) != 0;
        if (!Q8) low = -warp_max(lane < HR && table[lane] >= 0 ? -mref[lane] : -CUDART_INF_F);
        if (started) {
          // what was summed against the old references
          if (!TWO) {
            mbar_wait(&bars->pv_done[(idx - 1) & 1], ((idx - 1) >> 1) & 1, abort, CT_WAIT_NS);
            __syncwarp();
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < HR; c += C) {
            float4 f[C / 4];
            bool any = false;
#pragma unroll
            for (int e = 0; e < C / 4; ++e) {
              f[e] = *reinterpret_cast<const float4 *>(rise + c + 4 * e);
              any = any || f[e].x != 0.f || f[e].y != 0.f || f[e].z != 0.f || f[e].w != 0.f;
            }
            if (!any) continue;              // uniform: the same words for all
            float o[C];
            load_columns<C>(tO + c, o);
            uint32_t n[C];
#pragma unroll
            for (int e = 0; e < C; e += 4) {
              const float2 a = make_float2(ex2f(-f[e / 4].x), ex2f(-f[e / 4].y)), b = make_float2(ex2f(-f[e / 4].z), ex2f(-f[e / 4].w));
              l[(c + e) / 2] = __fmul2_rn(l[(c + e) / 2], a);
              l[(c + e) / 2 + 1] = __fmul2_rn(l[(c + e) / 2 + 1], b);
              n[e] = __float_as_uint(o[e] * a.x);
              n[e + 1] = __float_as_uint(o[e + 1] * a.y);
              n[e + 2] = __float_as_uint(o[e + 2] * b.x);
              n[e + 3] = __float_as_uint(o[e + 3] * b.y);
            }
#pragma unroll
            for (int e = 0; e < C; e += 8) tmem_st8(tO + c + e, n + e);
          }
          tmem_wait_st();
          bar_group(grp);                    // everyone has read the rises
          if (key < HR) xm[key] = ORDERED_LOWEST;
        }
      }
      // ---- P^T: 2^x, the row sums, and the parts for the second MMA
      const int pb = idx & 1;
      uint8_t *P = smem + LY::P_OFF + LY::p_buffer(TWO, pb);
      if (Q8 && !TWO && t != t_first) {        // one buffer: P V of the tile before has read it
        mbar_wait(&bars->pv_done[(idx - 1) & 1], ((idx - 1) >> 1) & 1, abort, CT_WAIT_NS);
        __syncwarp();
      }
      // with its V scale (a tree's value carries its own), in units of 2^(E - SHIFT)
      const float wj = !Q8 ? 1.f : !kx.valid ? 0.f : pow2i((TREE ? 0 : kx.ev) - E + SHIFT);
      const float2 w2 = make_float2(wj, wj);
#pragma unroll
      for (int c = 0; c < HR; c += C) {
        float x[C];
        raw_scores<C, LO>(tS + c, x);
        against<C, F8, true>(own, qsc + c, cs2, mref + c, x);
        if constexpr (TREE) {
          hide<C>(bits, c, kx.valid, x);
        } else if (masked) {
          if (!kx.valid) {
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = -CUDART_INF_F;
          }
        }
        const int rc = (r0 + c) >> 3;        // index of the 8-row chunk
        uint32_t w[C / 2];                   // pairs: bf16, or f16
#pragma unroll
        for (int e = 0; e < C / 2; ++e) {
          float2 v = make_float2(ex2f(x[2 * e]), ex2f(x[2 * e + 1]));
          if constexpr (!F8) {
            // bf16 weights: the sum is that of the rounded ones, so that what a weight loses
            // costs only its share of the differences between the values (error against
            // 64 bits behind a shared prefix 0.0023 -> 0.0018, where the output's rounding is
            // 0.0016; 64 single tokens 57 -> 58 us, 16 trees 232 -> 235)
            w[e] = bf16x2(v.x, v.y);
            v = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
          }
          l[c / 2 + e] = __fadd2_rn(l[c / 2 + e], v);
          if constexpr (Q8) v = __fmul2_rn(v, w2);
          if constexpr (F8)
            w[e] = weight_pair(v);
          else if constexpr (Q8)
            w[e] = bf16x2(v.x, v.y);         // (times a power of two: exact)
        }
        if constexpr (F8) {
          // into the 16-byte chunk of the rows in the key's line
          auto put = [&](int tile, int chunk, auto four) {
            uint8_t *at = P + tile + key * 128 + ((((rc >> 1) + chunk) ^ (key & 7)) << 4);
            if constexpr (C == 16)
              *reinterpret_cast<uint4 *>(at) = make_uint4(four(0), four(2), four(4), four(6));
            else
              *reinterpret_cast<uint2 *>(at + (rc & 1) * 8) = make_uint2(four(0), four(2));
          };
          auto upper = [&](int e) { return upper_bytes(w[e], w[e + 1]); };
          auto cut = [&] {
#pragma unroll
            for (int e = 0; e < C / 2; ++e) w[e] = without_upper(w[e]);
          };
          put(0, 0, upper);
          cut();
          put(TWO ? 0 : LY::PT, TWO ? 4 : 0, upper);
          cut();
          put(TWO ? (2 - pb) * LY::PT : 2 * LY::PT, TWO ? 4 * pb : 0, [&](int e) { return two16(e5m2_pair(w[e]), e5m2_pair(w[e + 1])); });
        } else {
#pragma unroll
          for (int k = 0; k < C / 8; ++k)
            *reinterpret_cast<uint4 *>(P + ((rc + k) >> 3) * LY::PT + key * 128 + ((((rc + k) & 7) ^ (key & 7)) << 4)) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      }
      // ---- values behind the last key must not reach the MMA (0 x NaN).  It takes
      // keys in steps of KSTEP: the rest of the last step is zeroed (rows of a bad
      // page came as zeros)
      constexpr int KSTEP = F8 ? 32 : 16;
      const int keys = (TREE ? pc.nb + (pc.ctx_tiles - t) * CA_KEYS : pc.L - t * CA_KEYS);
      if (r0 == 0 && keys < CA_KEYS && (keys & (KSTEP - 1)) != 0 && kq == (keys >> 5)) {   // uniform over the warp
        const int split = Q8 ? max(min(pc.ctx_tiles, pc.t1), pc.t0) : pc.t1;
        const int s0 = t < split ? pc.t0 : split, s1 = t < split ? split : pc.t1;      // the tile's section of the ring
        const int vslot = cnt.slots + (t < split ? 0 : 2 * (split - pc.t0)) +
                          (t + 1 == s1 ? 2 * (s1 - s0) - 1 : 2 * (t - s0) + 2) * (F8 ? 1 : LY::WIDE);
        const int st = vslot % LY::SLOTS;
        mbar_wait(&bars->full[st], (vslot / LY::SLOTS) & 1, abort, CT_WAIT_NS);
        __syncwarp();
        if (key >= keys && key < ((keys + KSTEP - 1) & ~(KSTEP - 1))) {
          const uint4 z = make_uint4(0, 0, 0, 0);
          uint8_t *vs = smem + LY::RING_OFF + st * LY::SLOT;
          if constexpr (F8) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) reinterpret_cast<uint4 *>(vs + key * D)[c] = z;
          } else {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
              for (int c = 0; c < 8; ++c) reinterpret_cast<uint4 *>(vs + h * (CA_KEYS * 128) + key * 128)[c] = z;
          }
        }
      }
      warp_arrive(&bars->p_full[pb], STEP);
    };
    int t = t_first;
    for (const int end = min(pc.t1, pc.ctx_tiles); t < end; t += STEP)
      tile(std::integral_constant<bool, Q8>{}, std::false_type{}, t);
    for (; t < pc.t1; t += STEP) tile(std::false_type{}, std::true_type{}, t);
    if (bad_page) set_err(w.dev_err, BASTION_DEVERR_PAGE);

    // ---- end of the piece: O^T after the last P V, sums over the keys
    const int last = cnt.tiles + pc.t1 - pc.t0 - 1;
    auto wait_pv = [&](int i) { mbar_wait(&bars->pv_done[i & 1], (i >> 1) & 1, abort, CT_WAIT_NS); };
    if (TWO && pc.t1 - pc.t0 > 1 && ((last ^ stream) & 1)) wait_pv(last - 1);   // (else last's barrier might be two phases behind)
    wait_pv(last);
    __syncwarp();
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem + LY::P_OFF) + v0;   // P's buffers are free: [key quarter][state]
    {
      float v[HR];
#pragma unroll
      for (int i = 0; i < HR; ++i) v[i] = (i & 1) ? l[i / 2].y : l[i / 2].x;
      const float sum = across_lanes<HR>(v);
      if (lane < HR) part[kq * CT_R + lane] = sum;
    }
    if (TWO)
      bar_softmax();
    else
      bar_group(grp);
    const bool whole = pc.t0 == 0 && pc.t1 == pc.T && !w.prefix_len;
    float *slot = w.slots + piece_slot(w, cta, pc.t0 == 0, pc.unit) * slot_floats(CT_R, D);
    if (key < HR && stream == 0) {
      auto state_sum = [&](int i) { return (part[i] + part[CT_R + i]) + (part[2 * CT_R + i] + part[3 * CT_R + i]); };
      const float unit = Q8 ? pow2i(E - SHIFT) : 1.f;
      float sum = state_sum(key), m = mref[key], f0 = unit, f1 = 0.f;
      if (TWO) {
        // the two streams' sums and outputs, against the larger reference
        const float m1 = mref[64 + key], top = fmaxf(m, m1);
        const float a = ex2f(m - top), b = ex2f(m1 - top);
        sum = sum * a + state_sum(64 + key) * b;
        m = top;
        f0 *= a;
        f1 = b * unit;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;        // a row that sees no key is zero
      rise[key] = f0 * inv;
      if (TWO) rise[64 + key] = f1 * inv;
      if (!whole && table[key] >= 0)
        slot[static_cast<int64_t>(CT_R) * D + r0 + key] = sum == 0.f ? -CUDART_INF_F : m + log2f(sum);
    }
    if (TWO)
      bar_softmax();
    else
      bar_group(grp);
    // rows of the output: with two streams the four groups share them again
    constexpr int OR = TWO ? (HR >= 16 ? HR / 2 : 8) : HR;
    constexpr int OC = OR < 16 ? 8 : 16;
    const int o0 = grp * OR;
    if (kq * 32 < D && (!TWO || o0 < 2 * HR)) {
      const bool two = TWO && pc.t1 - pc.t0 > 1;             // else one stream had no tile: its O holds anything
      const int only = TWO ? 64 * (last & 1) : 0;
      const float *factor = reinterpret_cast<const float *>(smem + LY::XM_OFF);
      const int *rows = reinterpret_cast<const int *>(smem + LY::TAB_OFF) + o0;
      const uint32_t tR = tbase + CT_SBUF * 128 + lane_off + o0;
#pragma unroll
      for (int c = 0; c < OR; c += OC) {
        float o[OC];
        load_columns<OC>(tR + (two ? 0 : only) + c, o);
        const float *f0 = factor + (two ? 0 : only) + o0 + c;
#pragma unroll
        for (int i = 0; i < OC; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(f0 + i);
          o[i] *= f.x, o[i + 1] *= f.y, o[i + 2] *= f.z, o[i + 3] *= f.w;
        }
        if (two) {
          float o1[OC];
          load_columns<OC>(tR + 64 + c, o1);
#pragma unroll
          for (int i = 0; i < OC; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(factor + 64 + o0 + c + i);
            o[i] = fmaf(o1[i], f.x, o[i]), o[i + 1] = fmaf(o1[i + 1], f.y, o[i + 1]);
            o[i + 2] = fmaf(o1[i + 2], f.z, o[i + 2]), o[i + 3] = fmaf(o1[i + 3], f.w, o[i + 3]);
          }
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < OC; ++i) {
            const int at = rows[c + i];
            if (at >= 0) p.out[static_cast<int64_t>(at) * D + key] = static_cast<uint16_t>(bf16x2(o[i], 0.f));
          }
        } else {
          float *dst = slot + (o0 + c) * D + key;            // (rows that are not there have their place in the slot too)
#pragma unroll
          for (int i = 0; i < OC; ++i) dst[i * D] = o[i];
        }
      }
    }
    tc_fence_before();
  }
};

template <int D, bool Q8, int RM>
__global__ void __launch_bounds__(CT_THREADS, 1) ctx_attn_kernel(const __grid_constant__ CtxMaps maps, const CtxParams p) {
  using LY = CtxLayout<D, Q8, RM>;
  constexpr int NH = D / 64;                 // 128-byte column blocks of a bf16 row
  extern __shared__ uint8_t smem[];
  // the swizzled tiles need a 1024-byte aligned base, which the layout takes as given
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_err(p.w.dev_err, BASTION_DEVERR_LAYOUT);
    return;
  }
  CtxBars *bars = reinterpret_cast<CtxBars *>(smem + LY::BAR_OFF);
  volatile int *abort = &bars->abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnWork &w = p.w;
  if (tid == 0) {
    mbar_init(&bars->q_full, CT_SM / 32);
    for (int i = 0; i < LY::SLOTS; ++i) mbar_init(&bars->full[i], 1), mbar_init(&bars->empty[i], 1);
    for (int i = 0; i < CT_SBUF; ++i) mbar_init(&bars->s_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->p_full[i], CT_SM / 32), mbar_init(&bars->pv_done[i], 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == CT_K_WARP && lane < 6) {
    const CUtensorMap *m = lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.pk : lane == 3 ? &maps.pv : lane == 4 ? &maps.kt : &maps.vt;
    tma_prefetch_desc(m);
  }
  if (warp == CT_MMA_WARP) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) attn_share(w, blockIdx.x, &bars->share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  const AttnShare &share = bars->share;      // read where needed: the small roles have few registers
  if (share.kind == 0) {                     // uniform over the CTA
    if (warp == CT_MMA_WARP) tmem_dealloc(tbase, 512);
    return;
  }
  AttnIter it;
  attn_begin(w, share, it);
  AttnPiece pc;

  // 640 threads x 96 registers at launch = 512 x 104 + 128 x 64
  if (warp >= CT_SM / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == CT_K_WARP || warp == CT_V_WARP) {
      // ------------------------------------------------ TMA producers (a lane per copy box)
      // One warp for K and one for V: a box takes its lane some 70 cycles, and with
      // both in one warp a page of 16 keys was issued more slowly than its tile
      // was worked off (16 requests of 512 to 8192 keys, one token each, 8-bit pages
      // of 16: 60 us, with two warps 48; one lane issuing all boxes: 90).
      const bool kv = warp == CT_V_WARP;
      int st = 0, turn = 0;                  // the slot of the next tile, and how often the ring has gone round
      uint32_t used = 0, parity = 0;         // slots filled so far, and the parity of their last turn
      bool run = true;
      auto advance = [&](int n) {
        st += n;
        if (st >= LY::SLOTS) st -= LY::SLOTS, ++turn;
      };
      // Room for the next tile: wait for its slots, announce its bytes (on the first).
      // (A wait by parity must not be two phases off: the tile before a slot's last one
      // is long used up when its warp comes here, as that warp's previous tile, at most
      // six slots back, has waited for what lay SLOTS before it.)
      auto take = [&](int n, uint32_t bytes) {
        if (turn > 0) {
          if (!mbar_wait(&bars->empty[st], (turn - 1) & 1, abort, CT_WAIT_NS)) run = false;
          if (n == 2 && !mbar_wait(&bars->empty[st + 1], (turn - 1) & 1, abort, CT_WAIT_NS)) run = false;
          run = __all_sync(FULL, run);
        }
        if (run) {
          if (lane == 0) {
            mbar_expect_tx(&bars->full[st], bytes);
            if (n == 2) mbar_expect_tx(&bars->full[st + 1], 0);
          }
          used |= 1u << st;
          parity = (parity & ~(1u << st)) | static_cast<uint32_t>(turn & 1) << st;
        }
        __syncwarp();
      };
      while (run && attn_next(w, share, it, pc)) {
        const CtxGeo &geo = pc.prefix ? p.prefix : p.own;
        const CUtensorMap *map = pc.prefix ? (kv ? &maps.pv : &maps.pk) : (kv ? &maps.v : &maps.k);
        const CUtensorMap *tree_map = kv ? &maps.vt : &maps.kt;
        const bool paged = geo.rows.block_table != nullptr;
        const int box = paged ? geo.rows.page_size : CT_BOX;   // <= 128, divides 128
        const int shift = 31 - __clz(box);
        const int ctx_end = min(pc.t1, pc.ctx_tiles);
        // lane's box within a tile: 8-bit: box lane; bf16: box lane / NH, column block lane % NH
        const int mybox = Q8 ? lane : lane / NH;
        const int mycol = Q8 ? 0 : (lane % NH) * 64;
        const int at = mybox << shift;                         // first key of the box
        const int32_t *pages = paged ? geo.rows.block_table + static_cast<int64_t>(pc.b) * geo.rows.max_pages : nullptr;
        auto has_box = [&](int t) { return at < CA_KEYS && t * CA_KEYS + at < pc.L; };
        // third coordinate and on: a page, or a row of the contiguous cache
        auto page_of = [&](int t) -> int {
          if (!paged || t >= ctx_end || !has_box(t)) return 0;
          const int page = __ldg(pages + ((t * CA_KEYS + at) >> shift));
          return static_cast<uint32_t>(page) < static_cast<uint32_t>(geo.rows.num_pages) ? page : geo.rows.num_pages;   // outside: zeros
        };
        auto copy = [&](uint8_t *dst, uint64_t *bar, int t, int page) {
          if (paged)
            tma_load_4d(dst, map, bar, mycol, 0, pc.kvh, page);
          else
            tma_load_3d(dst, map, bar, mycol, t * CA_KEYS + at, pc.b * w.Hkv + pc.kvh);
        };
        const int wide = Q8 ? max(ctx_end, pc.t0) : pc.t1;     // first tile of the second section
        int page_n = page_of(pc.t0);
        for (int t = pc.t0; run && t < pc.t1; ++t) {
          const int s0 = t < wide ? pc.t0 : wide, s1 = t < wide ? wide : pc.t1;
          const int unit = t < pc.ctx_tiles ? 1 : LY::WIDE;
          if (kv && t == s0) advance((s1 - s0 == 1 ? 1 : 2) * unit);
          uint8_t *dst = smem + LY::RING_OFF + st * LY::SLOT;
          uint64_t *bar = &bars->full[st];
          if (t < pc.ctx_tiles) {
            const int page = page_n;
            page_n = page_of(t + 1);
            const int left = min(pc.L - t * CA_KEYS, CA_KEYS);
            const uint32_t rows = static_cast<uint32_t>((left + box - 1) >> shift) << shift;   // copied: whole boxes
            take(1, rows * D * (Q8 ? 1 : 2));
            dst += Q8 ? at * D : (lane % NH) * (CA_KEYS * 128) + at * 128;
            if (run && has_box(t)) copy(dst, bar, t, page);
          } else {
            const int k0 = (t - pc.ctx_tiles) * CA_KEYS;
            const int nbox = (min(pc.nb - k0, CA_KEYS) + CT_TREE_BOX - 1) / CT_TREE_BOX;
            take(LY::WIDE, static_cast<uint32_t>(nbox * CT_TREE_BOX * D * 2));
            const int bx = lane / NH, h = lane % NH;
            if (run && bx < nbox)
              tma_load_3d(dst + h * (CA_KEYS * 128) + bx * CT_TREE_BOX * 128, tree_map, bar, h * 64, pc.kvh,
                          pc.b * w.n_max + k0 + bx * CT_TREE_BOX);
          }
          advance((kv ? (t + 2 >= s1 ? 1 : 2) : (t == s0 ? 1 : 2) + (t + 1 == s1 ? 1 : 0)) * unit);
        }
      }
      // the copies in flight land before the CTA goes away (nobody else waits for them after an abort)
      if (*abort)
        for (int i = 0; i < LY::SLOTS; ++i)
          for (int k = 0; ((used >> i) & 1u) && k < 2000 && !mbar_try_wait(&bars->full[i], (parity >> i) & 1u); ++k) __nanosleep(100);
    } else if (warp == CT_MMA_WARP) {
      // ------------------------------------------------ MMA issuer
      // The whole warp walks the loops with values that are the same in every lane
      // (`same` hands them out by a warp reduction, whose result the hardware keeps
      // in its uniform registers, where the MMA's operands have to be); one lane
      // issues.
      const auto same = [](int x) { return __reduce_max_sync(FULL, x); };
      const uint32_t leader = elect_one();
      int tiles_q = 0, tiles_p = 0;          // S^T and P V tiles issued
      int slots_q = 0, slots_p = 0;          // the ring slots (mod SLOTS) of the next K and V
      uint32_t turn_q = 0, turn_p = 0;       // and the parity of their turns round the ring
      int pieces = 0;
      const uint64_t q16 = sdesc_sw128(smem_u32(smem + LY::Q16_OFF), 16, 1024);
      const uint64_t q8 = sdesc_sw128(smem_u32(smem + LY::Q8_OFF), 16, 1024);
      const uint32_t tb = static_cast<uint32_t>(same(static_cast<int>(tbase)));
      auto advance = [](int &slot, uint32_t &turn, int n) {
        slot += n;
        if (slot >= LY::SLOTS) slot -= LY::SLOTS, turn ^= 1u;
      };
      while (attn_next(w, share, it, pc)) {
        const int N = same(columns(pc.rows));
        const bool two = RM < CT_R || N < CT_R;
        const int t0 = same(pc.t0), t1 = same(pc.t1), ctx_tiles = same(pc.ctx_tiles);
        const int ctx_keys = same(pc.L), tree_keys = same(pc.nb);
        const int wide = Q8 ? max(min(ctx_tiles, t1), t0) : t1;   // the sections: tiles [t0, wide), [wide, t1)
        mbar_wait(&bars->q_full, pieces & 1, abort, CT_WAIT_NS);
        ++pieces;
        __syncwarp();
        tc_fence_after();
        auto issue_qk = [&](int t) {
          const bool f8 = Q8 && t < ctx_tiles;
          const int st = slots_q;
          mbar_wait(&bars->full[st], turn_q, abort, CT_WAIT_NS);
          __syncwarp();
          tc_fence_after();
          const uint32_t kaddr = smem_u32(smem + LY::RING_OFF + st * LY::SLOT);
          const uint32_t dS = tb + (tiles_q & 1) * 128;
          if (f8) {
            const uint64_t kd = D == 128 ? sdesc_sw128(kaddr, 16, 1024) : sdesc_sw64(kaddr, 16, 512);
            const uint32_t id = ctx_idesc(0, 0, 0, 0, two ? 2 * N : N);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_if(leader, true, dS, kd + ((kk * 32) >> 4), q8 + ((kk * 32) >> 4), id, kk ? 1u : 0u);
            if (!two) {
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                const uint32_t lo = (D == 128 ? CT_R * 128 : 64) + kk * 32;
                mma_if(leader, true, dS, kd + ((kk * 32) >> 4), q8 + (lo >> 4), id, 1u);
              }
            }
          } else {
            const uint64_t kd = sdesc_sw128(kaddr, 16, 1024);
            const uint32_t id = ctx_idesc(1, 1, 0, 0, N);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t in = (kk & 3) * 32, off = ((kk >> 2) * (CA_KEYS * 128) + in) >> 4;
              mma_if(leader, false, dS, kd + off, q16 + (((kk >> 2) * (RM * 128) + in) >> 4), id, kk ? 1u : 0u);
            }
          }
          commit_if(leader, &bars->s_full[tiles_q & 1]);
          commit_if(leader, &bars->empty[st]);
          if (Q8 && !f8) commit_if(leader, &bars->empty[st + 1]);
          const int s0 = t < wide ? t0 : wide, s1 = t < wide ? wide : t1;
          advance(slots_q, turn_q, ((t == s0 ? 1 : 2) + (t + 1 == s1 ? 1 : 0)) * (f8 ? 1 : LY::WIDE));
          ++tiles_q;
        };
        auto issue_pv = [&](int t) {
          const bool f8 = Q8 && t < ctx_tiles;
          const int s0 = t < wide ? t0 : wide, s1 = t < wide ? wide : t1;
          if (t == s0) advance(slots_p, turn_p, (s1 - s0 == 1 ? 1 : 2) * (f8 ? 1 : LY::WIDE));
          const int st = slots_p;
          const uint32_t turn = turn_p;
          const int pb = tiles_p & 1;
          mbar_wait(&bars->full[st], turn, abort, CT_WAIT_NS);
          mbar_wait(&bars->p_full[pb], (tiles_p >> 1) & 1, abort, CT_WAIT_NS);
          __syncwarp();
          tc_fence_after();
          const uint32_t vaddr = smem_u32(smem + LY::RING_OFF + st * LY::SLOT);
          const uint64_t pd = sdesc_sw128(smem_u32(smem + LY::P_OFF + LY::p_buffer(two, pb)), LY::PT, 1024);
          // (fewer than 128 columns: even and odd tiles have an O each)
          const uint32_t dO = tb + CT_SBUF * 128 + (two ? pb * 64 : 0);
          const uint32_t first = t < t0 + (two ? 2 : 1) ? 0u : 1u;
          // keys that are there: the steps behind them are left out
          const int keys = t < ctx_tiles ? ctx_keys - t * CA_KEYS : tree_keys - (t - ctx_tiles) * CA_KEYS;
          // V^T as the MN-major A operand: 8 keys per swizzle group; head_dim 64 fills
          // half of the 128 rows, the others repeat what lies behind and are not read
          if (f8) {
            const uint64_t vd = D == 128 ? sdesc_sw128(vaddr, 16384, 1024) : sdesc_sw64(vaddr, 8192, 512);
            const uint32_t id = ctx_idesc(0, 1, 1, 1, N);
            const uint32_t mid = LY::p_mid(two), lo = LY::p_lo(two, pb);
            if (keys > CA_KEYS - 32) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((kk * 4096) >> 4), id, kk ? 1u : first);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((mid + kk * 4096) >> 4), id, 1u);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((lo + kk * 4096) >> 4), id, 1u);
            } else {
              for (int kk = 0; kk * 32 < keys; ++kk) {
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((kk * 4096) >> 4), id, kk ? 1u : first);
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((mid + kk * 4096) >> 4), id, 1u);
                mma_if(leader, true, dO, vd + ((kk * 32 * D) >> 4), pd + ((lo + kk * 4096) >> 4), id, 1u);
              }
            }
          } else {
            const uint32_t id = ctx_idesc(1, 1, 1, 1, N);
            const uint64_t vd = sdesc_sw128(vaddr, CA_KEYS * 128, 1024);
            if (keys > CA_KEYS - 16) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_if(leader, false, dO, vd + ((kk * 2048) >> 4), pd + ((kk * 2048) >> 4), id, kk ? 1u : first);
            } else {
              for (int kk = 0; kk * 16 < keys; ++kk)
                mma_if(leader, false, dO, vd + ((kk * 2048) >> 4), pd + ((kk * 2048) >> 4), id, kk ? 1u : first);
            }
          }
          commit_if(leader, &bars->pv_done[pb]);
          commit_if(leader, &bars->empty[st]);
          if (Q8 && !f8) commit_if(leader, &bars->empty[st + 1]);
          advance(slots_p, turn_p, (t + 2 >= s1 ? 1 : 2) * (f8 ? 1 : LY::WIDE));
          ++tiles_p;
        };
        for (int t = t0; t < min(t1, t0 + CT_LOOK); ++t) issue_qk(t);
        for (int t = t0; t < t1; ++t) {
          issue_pv(t);
          if (t + CT_LOOK < t1) issue_qk(t + CT_LOOK);
        }
      }
      // every MMA has finished before TMEM is released
      commit_if(leader, &bars->drain);
      for (int k = 0; k < 2000000 && !mbar_try_wait(&bars->drain, 0); ++k) {
      }
      __syncwarp();
    } else if (warp == CT_MMA_WARP + 1) {
      // ------------------------------------------------ records of the units that begin here
      if (lane == 0)
        while (attn_next(w, share, it, pc))
          if (pc.t0 == 0) attn_record(w, share, pc);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------ softmax warps
    using SM = CtxSoftmax<D, Q8, RM>;
    CtxCounts cnt{0, 0};
    float *mref = reinterpret_cast<float *>(smem + LY::MREF_OFF);
    int *table = reinterpret_cast<int *>(smem + LY::TAB_OFF);
    while (attn_next(w, share, it, pc)) {
      const int N = columns(pc.rows);
      bar_softmax();                         // the previous piece's tables are no longer read
      int *starts = reinterpret_cast<int *>(smem + LY::P_OFF);   // P's buffers are free between pieces
      if (pc.prefix) {
        if (warp == 0) prefix_row_starts(w, lane, starts);
        bar_softmax();
      }
      row_table(w, pc, starts, tid, CT_SM, table);
      if (Q8 && tid == 0) bars->top_ctx = bars->top_tree = 0;
      if (tid < CT_R)
        mref[tid] = CT_UNSET, reinterpret_cast<int *>(smem + LY::XM_OFF)[tid] = ORDERED_LOWEST;
      bar_softmax();
      const float common = SM::load_q(p, smem, bars, pc, N, tid);
      warp_arrive(&bars->q_full, 1);
      if (Q8) bar_softmax();                 // the row scales, and `xm` as the tiles want it
      if (RM == 128 && N == 128) {
        if constexpr (RM == 128) SM::template piece<32, false>(p, smem, bars, pc, cnt, tbase, blockIdx.x, common);
      } else if (N == 64)
        SM::template piece<32, true>(p, smem, bars, pc, cnt, tbase, blockIdx.x, common);
      else if (N == 32)
        SM::template piece<16, true>(p, smem, bars, pc, cnt, tbase, blockIdx.x, common);
      else
        SM::template piece<8, true>(p, smem, bars, pc, cnt, tbase, blockIdx.x, common);
      cnt.tiles += pc.t1 - pc.t0;
      const int ctx = Q8 ? max(0, min(pc.t1, pc.ctx_tiles) - pc.t0) : 0;   // 8-bit tiles
      cnt.slots += 2 * (LY::WIDE * (pc.t1 - pc.t0) - ctx);
    }
  }

  // all roles are done with TMEM
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == CT_MMA_WARP) tmem_dealloc(tbase, 512);
  if (*abort && tid == 0) set_err(w.dev_err, BASTION_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ host side
static_assert(CT_R == CTX_ROWS_BF16, "the plan's row tile");

cudaError_t prepare_ctx_attn() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *fn, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, static_cast<int>(cudaSharedmemCarveoutMaxShared));
  };
  auto both = [&](auto d_, auto q8_) {
    constexpr int D = decltype(d_)::value;
    constexpr bool Q8 = decltype(q8_)::value;
    set(reinterpret_cast<const void *>(ctx_attn_kernel<D, Q8, 64>), CtxLayout<D, Q8, 64>::SMEM);
    set(reinterpret_cast<const void *>(ctx_attn_kernel<D, Q8, 128>), CtxLayout<D, Q8, 128>::SMEM);
  };
  both(std::integral_constant<int, 128>{}, std::false_type{});
  both(std::integral_constant<int, 128>{}, std::true_type{});
  both(std::integral_constant<int, 64>{}, std::false_type{});
  both(std::integral_constant<int, 64>{}, std::true_type{});
  return e;
}

cudaError_t launch_ctx_attn(const AttnWork &w, int d, bool q8, const CtxMaps &maps, const CtxGeo &own,
                            const CtxGeo &prefix, const void *q, const void *vt, const uint64_t *mask, float scale,
                            void *out, cudaStream_t stream) {
  CtxParams p{};
  p.w = w;
  p.own = own;
  p.prefix = prefix;
  p.q = static_cast<const uint16_t *>(q);
  p.vt = static_cast<const uint16_t *>(vt);
  p.mask = reinterpret_cast<const uint32_t *>(mask);
  p.scale_log2 = scale * kLog2e;
  p.out = static_cast<uint16_t *>(out);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = fill_launch_attrs(attr);
  cfg.stream = stream;
  cfg.gridDim = dim3(w.nctas, 1, 1);
  cfg.blockDim = dim3(CT_THREADS, 1, 1);
  // The most rows that a unit of this call can have.  Up to 64, the layout with more
  // K and V in flight (each call on its own, cold L2): 8-bit decoding of 16 requests of
  // 512 to 8192 keys 58.5 -> 55.8 us, trees of 16 nodes of 8 such requests 65.0 -> 63.0,
  // 4 requests behind 8192 shared bf16 keys 30.2 -> 29.2.
  const int64_t rows = static_cast<int64_t>(w.prefix_len ? w.B : 1) * w.n_max * w.g;
  auto go = [&](auto d_, auto q8_, auto rm_) {
    constexpr int D = decltype(d_)::value, RM = decltype(rm_)::value;
    constexpr bool Q8 = decltype(q8_)::value;
    cfg.dynamicSmemBytes = CtxLayout<D, Q8, RM>::SMEM;
    return cudaLaunchKernelEx(&cfg, ctx_attn_kernel<D, Q8, RM>, maps, p);
  };
  auto by_rows = [&](auto d_, auto q8_) {
    return rows <= 64 ? go(d_, q8_, std::integral_constant<int, 64>{}) : go(d_, q8_, std::integral_constant<int, 128>{});
  };
  auto by_type = [&](auto d_) { return q8 ? by_rows(d_, std::true_type{}) : by_rows(d_, std::false_type{}); };
  const cudaError_t e = d == 128 ? by_type(std::integral_constant<int, 128>{}) : by_type(std::integral_constant<int, 64>{});
  if (e != cudaSuccess) return e;
  return launch_ctx_attn_merge(w, d, true, out, stream);
}

}  // namespace bst
