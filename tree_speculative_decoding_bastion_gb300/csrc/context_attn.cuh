// What the C ABI hands to the context attention's kernels.
#pragma once

#include <cuda.h>

#include "attn_work.cuh"
#include "q8.cuh"

namespace bst {

constexpr int CTX_ROWS_BF16 = 128;      // rows per tile of the tensor-core path
constexpr int CTX_ROWS_F32 = 32;        // and of the fp32 path
constexpr int CT_BOX = 64;              // rows of a contiguous cache's copy box
constexpr int CT_TREE_BOX = 32;         // rows of a tree tile's copy box

struct RowSource {            // rows of one cache
  const void *k, *v;          // f32 rows or e4m3 codes
  const uint8_t *ks, *vs;     // scale bytes (8-bit caches)
  RowCache geo;
};

struct CtxGeo {                         // a cache as the tensor-core path sees it (its rows come by TMA)
  const uint8_t *ks, *vs;               // scale bytes (8-bit)
  RowCache rows;
};

struct CtxMaps {
  CUtensorMap k, v, pk, pv, kt, vt;
};

cudaError_t prepare_ctx_attn();
cudaError_t prepare_ctx_attn_f32();
cudaError_t launch_ctx_attn(const AttnWork &w, int d, bool q8, const CtxMaps &maps, const CtxGeo &own,
                            const CtxGeo &prefix, const void *q, const void *vt, const uint64_t *mask, float scale,
                            void *out, cudaStream_t stream);
cudaError_t launch_ctx_attn_f32(const AttnWork &w, int d, bool q8, const RowSource &own, const RowSource &prefix,
                                const float *q, const float *kt, const float *vt, const uint64_t *mask, float scale,
                                float *out, cudaStream_t stream);

}  // namespace bst
