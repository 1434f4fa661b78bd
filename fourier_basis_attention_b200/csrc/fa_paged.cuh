// fa_paged.cuh -- what the kernels over a paged cache share: the batch on the device, the
// key range of a tile of query rows, and the tensor map of a pool.
#pragma once

#include <cuda.h>

#include "fa_host.h"
#include "fa_internal.cuh"

namespace fa {

// Watchdog sites of the paged calls (kernel ids of fa_device_status).
enum : unsigned int {
  WD_PAGED = 8u << 8,        // waits of the paged attention kernels
  WD_PAGED_ENTRY = FA_WATCHDOG_PAGED_ENTRY << 8,  // a device-side entry out of range
  WD_ENTRY_LENGTH = WD_PAGED_ENTRY | 1u,  // q_start / kv_len
  WD_ENTRY_PAGE = WD_PAGED_ENTRY | 2u,    // page_table
};

struct PagedBatch {
  const int* table;
  const int* q_start;
  const int* kv_len;
  int B, Hq, Hkv, G, page, num_pages, max_pages, total_q, max_q, max_kv;
};

// New tokens [q0, q0 + n) of a sequence and its cached tokens kv (the new ones included).
struct SeqSpan {
  int q0, n, kv;
};

__device__ __forceinline__ void flag_entry(unsigned int site) { atomicCAS(&g_watchdog, 0u, site); }

// The span of sequence b; one whose entries break the shape's bounds is empty and flagged.
__device__ __forceinline__ SeqSpan seq_span(const PagedBatch& p, int b) {
  SeqSpan s;
  s.q0 = p.q_start[b];
  const int end = p.q_start[b + 1];
  s.kv = p.kv_len[b];
  s.n = end - s.q0;
  if (s.q0 < 0 || end < s.q0 || end > p.total_q || s.n > p.max_q || s.kv < 0 || s.kv > p.max_kv) {
    flag_entry(WD_ENTRY_LENGTH);
    s.q0 = s.n = s.kv = 0;
  }
  return s;
}

// The page that holds cached token j of sequence b; -1 (flagged) if the entry is out of range.
__device__ __forceinline__ int page_of(const PagedBatch& p, int b, int j) {
  const int pg = p.table[(long long)b * p.max_pages + j / p.page];
  if ((unsigned)pg < (unsigned)p.num_pages) return pg;
  flag_entry(WD_ENTRY_PAGE);
  return -1;
}

// Keys [lo, hi) that the query rows [r0, r1) of a sequence see, rows numbered token * G +
// head (r1 <= n * G). Empty: hi <= lo.
__device__ __forceinline__ void row_keys(const SeqSpan& s, int G, int window, int r0, int r1,
                                         int* lo, int* hi) {
  const int first = s.kv - s.n + r0 / G, last = s.kv - s.n + (r1 - 1) / G;
  *hi = last + 1;
  *lo = window > 0 ? max(0, first - window + 1) : 0;
}

// A wait by all lanes of a warp, with one answer for all: each lane polls the barrier, the abort word
// and the clock by itself, so that where a wait runs out lanes may differ, and a warp that branched on
// that would meet at different votes for good.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          unsigned int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, site));
}

// Overlap with the kernel launched next: it may be set up once every CTA of this one has called
// allow_next_kernel (or has left), and waits for this one to complete where it calls
// wait_earlier_kernel. The first kernel of a call waits for whatever ran before it, and only then
// lets the next be set up: so a later kernel of the call that needs none of the first one's results
// may wait at its end, and its completion covers both.
__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_earlier_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Launches a kernel that may be set up while the one before it on the stream still runs.
template <typename... A, typename... B>
cudaError_t launch_clusters(void (*kernel)(A...), dim3 grid, int cluster, int threads, size_t smem,
                            cudaStream_t stream, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... A, typename... B>
cudaError_t launch_overlapped(void (*kernel)(A...), dim3 grid, int threads, size_t smem,
                              cudaStream_t stream, const B&... args) {
  return launch_clusters(kernel, grid, 1, threads, smem, stream, args...);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Chunks that the keys of `tokens` neighbouring tokens can touch, in a cache or a window.
int chunk_slots(const fa_paged_shape& s, int window, int chunk, int tokens);

// Tensor-core tiles of a batch (fa_paged_tc.cu); tok = 0: not used.
struct TilePlan {
  int tok, box, tiles, chunk, slots;
  int pair;  // 128-row tiles a CTA
  size_t records;  // partial results
};
cudaError_t tile_plan(const fa_paged_shape& s, int window, TilePlan* t);
// Rows of sequences with more than skip_rows query rows a KV head.
cudaError_t launch_tiles(const fa_paged_shape& s, const fa_paged_cache& c, const TilePlan& t,
                         const void* q, int64_t q_stride, float scale, int window, void* out,
                         int64_t out_stride, float* lse, float* part_o, float2* part_ml,
                         int skip_rows, cudaStream_t stream, const char** why);

cudaError_t launch_weight_tiles(const fa_paged_shape& s, const fa_paged_cache& c, const void* q,
                                int64_t q_stride, float scale, int window, const float* lse,
                                float* weights, int64_t weights_ld, int skip_rows,
                                cudaStream_t stream, const char** why);

// 2-D map of a pool: rows of 128 bf16 in (page, head, slot) order, boxes of 64 dims x `rows`
// rows in the 128-byte swizzle.
bool encode_pool(CUtensorMap* map, const void* pool, const fa_paged_shape& s, int rows);

PagedBatch paged_batch(const fa_paged_shape& s, const fa_paged_cache& c);

}  // namespace fa
