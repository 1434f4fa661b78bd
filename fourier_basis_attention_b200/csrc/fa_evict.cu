// fa_evict.cu -- which tokens of a paged cache stay, by the attention weight they gathered,
// and their move into other pages.
//
// Selection, per (sequence, KV head): a weight becomes an unsigned key in the order of the
// numbers (NaN 0, behind every number; sink and recent tokens 2^32 - 1, before them). The
// keep-th largest key is found a byte at a time from the top (four passes, each a histogram
// of the keys that share the bytes found so far); tokens above it stay, and of those equal to
// it the first in order fill the rest. A last pass in token order writes their indices.
// The move reads and writes each kept row once.
#include "fa_paged.cuh"

namespace fa {

constexpr int EV_THREADS = 1024;
constexpr int EM_THREADS = 256;
constexpr int EM_ROWS = 32;  // kept rows a CTA

struct EvictParams {
  PagedBatch src, dst;
  const float* weights;
  long long weights_ld;
  int keep, sink, recent;
  const uint4 *K, *V;
  uint4 *dst_K, *dst_V;
  float* dst_weights;
  long long dst_weights_ld;
  int *index, *dst_len;
};

__device__ __forceinline__ int evict_len(const PagedBatch& p, int b) {
  const int kv = p.kv_len[b];
  if (kv >= 0 && kv <= p.max_kv) return kv;
  flag_entry(WD_ENTRY_LENGTH);
  return 0;
}

__device__ __forceinline__ uint32_t evict_key(float w, int j, int kv, int sink, int recent) {
  if (j < sink || j >= kv - recent) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 and +0 are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const __grid_constant__ EvictParams P) {
  __shared__ int hist[256];
  __shared__ int sums[2][EV_THREADS / 32];
  __shared__ int found[2];  // byte, tokens still wanted among the keys that share the prefix
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kv = evict_len(P.src, b), m = min(kv, P.keep);
  const float* w = P.weights + ((long long)b * P.src.Hkv + g) * P.weights_ld;
  int* index = P.index + ((long long)b * P.src.Hkv + g) * P.keep;
  if (g == 0 && tid == 0) P.dst_len[b] = m;
  for (int i = m + tid; i < P.keep; i += EV_THREADS) index[i] = -1;
  if (kv <= P.keep) {
    for (int i = tid; i < m; i += EV_THREADS) index[i] = i;
    return;
  }
  uint32_t prefix = 0;
  int want = m;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j = tid; j < kv; j += EV_THREADS) {
      const uint32_t key = evict_key(w[j], j, kv, P.sink, P.recent);
      if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {  // the byte at which the count from the top reaches `want`
      int own[8], total = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) total += own[i] = hist[8 * lane + i];
      int higher = total;  // keys in this lane's bins and the ones above
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_down_sync(0xFFFFFFFFu, higher, d);
        if (lane + d < 32) higher += x;
      }
      higher -= total;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        if (higher < want && higher + own[i] >= want) {
          found[0] = 8 * lane + i;
          found[1] = want - higher;
        }
        higher += own[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    want = found[1];
  }
  // tokens in order: above the key, or equal to it and among the first `want` of those
  int kept = 0, equal = 0;  // before this block of tokens
  for (int j0 = 0; j0 < kv; j0 += EV_THREADS) {
    const int j = j0 + tid;
    const uint32_t key = j < kv ? evict_key(w[j], j, kv, P.sink, P.recent) : 0u;
    const bool eq = j < kv && key == prefix, gt = j < kv && key > prefix;
    const unsigned below = (1u << lane) - 1u;
    const unsigned be = __ballot_sync(0xFFFFFFFFu, eq), bg = __ballot_sync(0xFFFFFFFFu, gt);
    if (lane == 0) {
      sums[0][warp] = __popc(bg);
      sums[1][warp] = __popc(be);
    }
    __syncthreads();
    int g_before = 0, e_before = 0, g_all = 0, e_all = 0;
#pragma unroll
    for (int i = 0; i < EV_THREADS / 32; ++i) {
      const int sg = sums[0][i], se = sums[1][i];
      g_before += i < warp ? sg : 0;
      e_before += i < warp ? se : 0;
      g_all += sg;
      e_all += se;
    }
    const int e_rank = equal + e_before + __popc(be & below);
    if (gt || (eq && e_rank < want))
      index[kept + g_before + __popc(bg & below) + min(e_rank, want)] = j;
    kept += g_all;
    equal += e_all;
    __syncthreads();
  }
}

// 16 lanes a row of 256 bytes; K and V of EM_ROWS kept tokens of one (sequence, KV head).
__global__ void __launch_bounds__(EM_THREADS) evict_move_kernel(const __grid_constant__ EvictParams P) {
  const int g = blockIdx.y, b = blockIdx.z;
  const int sub = threadIdx.x & 15;
  const long long bh = (long long)b * P.src.Hkv + g;
#pragma unroll
  for (int r = threadIdx.x >> 4; r < EM_ROWS; r += EM_THREADS / 16) {
    const int i = blockIdx.x * EM_ROWS + r;
    if (i >= P.keep) break;
    const int j = P.index[bh * P.keep + i];
    if (j < 0) break;
    const int ps = page_of(P.src, b, j), pd = page_of(P.dst, b, i);
    if (ps < 0 || pd < 0) continue;
    const long long s = ((long long)(ps * P.src.Hkv + g) * P.src.page + j % P.src.page) * 16 + sub;
    const long long d = ((long long)(pd * P.dst.Hkv + g) * P.dst.page + i % P.dst.page) * 16 + sub;
    const uint4 k = P.K[s], v = P.V[s];
    P.dst_K[d] = k;
    P.dst_V[d] = v;
    if (sub == 0 && P.dst_weights)
      P.dst_weights[bh * P.dst_weights_ld + i] = P.weights[bh * P.weights_ld + j];
  }
}

FA_WATCHDOG_READER(read_watchdog_evict)

// ------------------------------------------------------------------------- host side
cudaError_t evict_workspace(const fa_paged_shape&, int, size_t* bytes) {
  *bytes = 0;
  return cudaSuccess;
}

cudaError_t launch_evict(const fa_paged_shape& s, const fa_paged_cache& c, const float* weights,
                         int64_t weights_ld, int keep, int sink, int recent,
                         const fa_paged_shape& ds, const fa_paged_cache& dc, float* dst_weights,
                         int64_t dst_weights_ld, int32_t* index, int32_t* dst_len, void*,
                         cudaStream_t stream) {
  EvictParams P;
  P.src = paged_batch(s, c);
  P.dst = paged_batch(ds, dc);
  P.weights = weights;
  P.weights_ld = weights_ld;
  P.keep = keep;
  P.sink = sink;
  P.recent = recent;
  P.K = static_cast<const uint4*>(c.K);
  P.V = static_cast<const uint4*>(c.V);
  P.dst_K = static_cast<uint4*>(dc.K);
  P.dst_V = static_cast<uint4*>(dc.V);
  P.dst_weights = dst_weights;
  P.dst_weights_ld = dst_weights_ld;
  P.index = index;
  P.dst_len = dst_len;
  evict_select_kernel<<<dim3((unsigned)s.Hkv, (unsigned)s.B), EV_THREADS, 0, stream>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((keep + EM_ROWS - 1) / EM_ROWS), (unsigned)s.Hkv, (unsigned)s.B);
  evict_move_kernel<<<grid, EM_THREADS, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace fa
