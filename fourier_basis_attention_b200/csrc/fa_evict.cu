// fa_evict.cu -- which tokens of a paged cache stay, by the attention weight they gathered,
// and their move into other pages.
//
// Selection, per (sequence, KV head): a weight becomes an unsigned key in the order of the
// numbers (NaN 0, behind every number; sink and recent tokens 2^32 - 1, before them). The
// keep-th largest key is found from the top in digits of 11, 11 and 10 bits, each by a
// histogram of the keys that share the digits found so far; tokens above it stay, and of those
// equal to it the first in order fill the rest. A cluster of CTAs holds a row's keys in shared
// memory (the weights are read once) and sums its histograms there; every CTA then writes the
// indices of its own tokens behind those of the CTAs before it. 11 bits are sign, exponent and
// two bits of the mantissa: weights fall into tens of bins, so that few lanes of a warp count
// into the same one.
// The move reads and writes each kept row once.
//   Measured (B200): 131072 tokens of 8 KV heads to 16384, 140 MB, in 47 us (selection 25, move
// 24 when each starts cold); 24 sequences of up to 8191 to 2001, 370 MB, in 78 us (16 and 59, the
// move at 95% of the measured copy bandwidth in rows of 256 bytes). The selection is a chain of 3 digits of some 3 us: a count, a
// cluster barrier, a read of 64 KB of histograms, a scan.
#include "fa_paged.cuh"

namespace fa {

constexpr int EV_THREADS = 1024;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048;
constexpr int EV_CLUSTER = 8;       // CTAs a row at most
constexpr int EV_HELD = 16384;      // keys a CTA holds in shared memory; more are read again
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

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One cluster of `size` CTAs a (sequence, KV head); CTA r has the tokens [r per, (r + 1) per).
__global__ void __launch_bounds__(EV_THREADS)
    evict_select_kernel(const __grid_constant__ EvictParams P, int size, int held) {
  allow_next_kernel();
  extern __shared__ __align__(16) uint32_t keys[];
  // counts of a digit, and their sums over the cluster; one histogram a digit, so that no CTA
  // waits for the others to have read it
  __shared__ __align__(16) int hists[3][EV_BINS], sums[EV_BINS];
  __shared__ int above[EV_WARPS], equal[EV_WARPS], mine[2];
  __shared__ int found[2];  // digit; tokens still wanted among the keys that share the prefix
  const int rank = size > 1 ? (int)cluster_ctarank() : 0;
  const int g = blockIdx.x / size, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kv = evict_len(P.src, b), m = min(kv, P.keep);
  const float* w = P.weights + ((long long)b * P.src.Hkv + g) * P.weights_ld;
  int* index = P.index + ((long long)b * P.src.Hkv + g) * P.keep;
  if (g == 0 && rank == 0 && tid == 0) P.dst_len[b] = m;
  const int all = size * EV_THREADS, me = rank * EV_THREADS + tid;
  for (int i = m + me; i < P.keep; i += all) index[i] = -1;
  if (kv <= P.keep) {
    for (int i = me; i < m; i += all) index[i] = i;
    return;
  }
  const int per = ((kv + size - 1) / size + 31) & ~31;
  const int first = min(rank * per, kv), n = min(per, kv - first);
  const int n_held = min(n, held);
  auto far_key = [&](int i) { return evict_key(w[first + i], first + i, kv, P.sink, P.recent); };
  uint32_t prefix = 0;
  int want = m;
  for (int i = tid; i < 3 * EV_BINS; i += EV_THREADS) hists[0][i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t known = digit == 0 ? 0u : digit == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    int* hist = hists[digit];
    if (digit == 0) {
      // the weights come in once: 8 loads a thread on their way at a time
      for (int i0 = tid; i0 < n_held; i0 += 8 * EV_THREADS) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (i0 + u * EV_THREADS < n_held) x[u] = w[first + i0 + u * EV_THREADS];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = i0 + u * EV_THREADS;
          if (i >= n_held) break;
          const uint32_t key = evict_key(x[u], first + i, kv, P.sink, P.recent);
          keys[i] = key;
          atomicAdd(&hist[key >> 21], 1);
        }
      }
    } else {
      for (int i = 4 * tid; i < n_held; i += 4 * EV_THREADS) {
        const uint4 q = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if ((k[u] & known) == prefix && i + u < n_held) atomicAdd(&hist[(k[u] >> shift) & mask], 1);
      }
    }
    for (int i = n_held + tid; i < n; i += EV_THREADS) {
      const uint32_t key = far_key(i);
      if ((key & known) == prefix) atomicAdd(&hist[(key >> shift) & mask], 1);
    }
    if (size > 1) {
      cluster_sync_all();
      if (tid < EV_BINS / 4) {
        const uint32_t at = smem_u32(hist + 4 * tid);
        int4 v[EV_CLUSTER];
#pragma unroll
        for (int r = 0; r < EV_CLUSTER; ++r)
          if (r < size) v[r] = ld_cluster_int4(mapa_shared(at, r));
        int4 t = v[0];
#pragma unroll
        for (int r = 1; r < EV_CLUSTER; ++r)
          if (r < size) {
            t.x += v[r].x;
            t.y += v[r].y;
            t.z += v[r].z;
            t.w += v[r].w;
          }
        *reinterpret_cast<int4*>(sums + 4 * tid) = t;
      }
    }
    __syncthreads();
    const int* total = size > 1 ? sums : hist;
    // the digit at which the count from the top reaches `want`: 2 bins a thread
    static_assert(EV_BINS == 2 * EV_THREADS, "bins a thread");
    const int2 own = *reinterpret_cast<const int2*>(total + 2 * tid);
    const int sum = own.x + own.y;
    int higher = sum;  // counts of this lane's bins and the warp's above
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_down_sync(0xFFFFFFFFu, higher, d);
      if (lane + d < 32) higher += x;
    }
    if (lane == 0) above[warp] = higher;
    __syncthreads();
    higher -= sum;
    higher += __reduce_add_sync(0xFFFFFFFFu, lane > warp ? above[lane] : 0);
    static_assert(EV_WARPS == 32, "a warp sums the warps' counts");
    if (higher < want && higher + own.y >= want) {
      found[0] = 2 * tid + 1;
      found[1] = want - higher;
    }
    higher += own.y;
    if (higher < want && higher + own.x >= want) {
      found[0] = 2 * tid;
      found[1] = want - higher;
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    want = found[1];
  }
  // a warp's tokens [w0, w1): above the key, equal to it
  const int seg = ((n + EV_WARPS - 1) / EV_WARPS + 31) & ~31;
  const int w0 = min(warp * seg, n), w1 = min(w0 + seg, n);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t key = i < n_held ? keys[i] : far_key(i);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  __syncthreads();  // `above` is read no more
  if (lane == 0) {
    above[warp] = gt;
    equal[warp] = eq;
  }
  __syncthreads();
  const int gt_w = above[lane], eq_w = equal[lane];
  int gt_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? gt_w : 0);
  int eq_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? eq_w : 0);
  if (size > 1) {
    if (warp == 0) {
      const int gt_all = __reduce_add_sync(0xFFFFFFFFu, gt_w), eq_all = __reduce_add_sync(0xFFFFFFFFu, eq_w);
      if (lane == 0) {
        mine[0] = gt_all;
        mine[1] = eq_all;
      }
    }
    cluster_sync_all();
    int gt_r = 0, eq_r = 0;
    if (lane < rank) {
      gt_r = ld_cluster_s32(mapa_shared(smem_u32(&mine[0]), lane));
      eq_r = ld_cluster_s32(mapa_shared(smem_u32(&mine[1]), lane));
    }
    gt_before += __reduce_add_sync(0xFFFFFFFFu, gt_r);
    eq_before += __reduce_add_sync(0xFFFFFFFFu, eq_r);
    cluster_sync_all();  // the CTA's shared memory is read no more
  }
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i >= w1 ? 0u : i < n_held ? keys[i] : far_key(i);
    const bool is_gt = i < w1 && key > prefix, is_eq = i < w1 && key == prefix;
    const unsigned bg = __ballot_sync(0xFFFFFFFFu, is_gt), be = __ballot_sync(0xFFFFFFFFu, is_eq);
    const int e_rank = eq_before + __popc(be & below);
    if (is_gt || (is_eq && e_rank < want))
      index[gt_before + __popc(bg & below) + min(e_rank, want)] = first + i;
    gt_before += __popc(bg);
    eq_before += __popc(be);
  }
}

// 16 lanes a row of 256 bytes; K and V of EM_ROWS kept tokens of one (sequence, KV head). A
// thread's rows are all on their way before the first is stored.
__global__ void __launch_bounds__(EM_THREADS, 8) evict_move_kernel(const __grid_constant__ EvictParams P) {
  constexpr int N = EM_ROWS / (EM_THREADS / 16);
  const int g = blockIdx.y, b = blockIdx.z;
  const int sub = threadIdx.x & 15;
  const long long bh = (long long)b * P.src.Hkv + g;
  int j[N];
  wait_earlier_kernel();
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int i = blockIdx.x * EM_ROWS + u * (EM_THREADS / 16) + (threadIdx.x >> 4);
    j[u] = i < P.keep ? P.index[bh * P.keep + i] : -1;
  }
  uint4 k[N], v[N];
  long long d[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    d[u] = -1;
    if (j[u] < 0) continue;
    const int i = blockIdx.x * EM_ROWS + u * (EM_THREADS / 16) + (threadIdx.x >> 4);
    const int ps = page_of(P.src, b, j[u]), pd = page_of(P.dst, b, i);
    if (ps < 0 || pd < 0) continue;
    const long long r = ((long long)(ps * P.src.Hkv + g) * P.src.page + j[u] % P.src.page) * 16 + sub;
    d[u] = ((long long)(pd * P.dst.Hkv + g) * P.dst.page + i % P.dst.page) * 16 + sub;
    k[u] = P.K[r];
    v[u] = P.V[r];
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if (d[u] < 0) continue;
    P.dst_K[d[u]] = k[u];
    P.dst_V[d[u]] = v[u];
    if (sub == 0 && P.dst_weights) {
      const int i = blockIdx.x * EM_ROWS + u * (EM_THREADS / 16) + (threadIdx.x >> 4);
      P.dst_weights[bh * P.dst_weights_ld + i] = P.weights[bh * P.weights_ld + j[u]];
    }
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
  // CTAs a row: as many as leave each at least 2048 tokens and are all resident (one an SM: two
  // would take half the registers, and the spills cost more: 57 against 47 us for one cache of
  // 131072 tokens, 8 KV heads)
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)s.B * s.Hkv;
  int size = 1;
  while (size < EV_CLUSTER && rows * size * 2 <= sms && s.max_kv >= 4096LL * size) size *= 2;
  const int per = ((s.max_kv + size - 1) / size + 31) & ~31;
  int held = per < EV_HELD ? (per > 0 ? per : 32) : EV_HELD;
  const void* fn = reinterpret_cast<const void*>(evict_select_kernel);
  // the limit counts the static arrays too, so it is raised for every size
  if ((e = raise_smem_limit(fn, EV_HELD * 4)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.Hkv * size), (unsigned)s.B, 1);
  cfg.blockDim = dim3(EV_THREADS, 1, 1);
  cfg.dynamicSmemBytes = (size_t)held * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&P, &size, &held};
  if ((e = cudaLaunchKernelExC(&cfg, fn, args)) != cudaSuccess) return e;
  const dim3 grid((unsigned)((keep + EM_ROWS - 1) / EM_ROWS), (unsigned)s.Hkv, (unsigned)s.B);
  return launch_overlapped(evict_move_kernel, grid, EM_THREADS, 0, stream, P);
}

}  // namespace fa
