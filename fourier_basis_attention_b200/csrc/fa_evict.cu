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
//   Measured (B200): 131072 tokens of 8 KV heads to 16384, 140 MB, in 42 us (selection 18, move
// 24 when each starts cold); 24 sequences of up to 8191 to 2001, 370 MB, in 75 us (15 and 59, the
// move at 95% of the measured copy bandwidth in rows of 256 bytes). The selection is a chain of
// steps: the weights' way in 4 us, three digits of 2 to 3 (a count, a barrier, a scan), the
// indices 3. Summing the histograms of a cluster by adding nonzero counts to the CTA that owns a
// bin took 6 us less than reading all 8 histograms in each.
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

__device__ __forceinline__ int2 ld_cluster_int2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster of `size` CTAs a (sequence, KV head); CTA r has the tokens [r per, (r + 1) per).
__global__ void __launch_bounds__(EV_THREADS)
    evict_select_kernel(const __grid_constant__ EvictParams P, int size, int held) {
  wait_earlier_kernel();
  allow_next_kernel();
  extern __shared__ __align__(16) uint32_t keys[];
  // counts of a digit; their sums over the cluster, 1 / size of the bins in each CTA
  __shared__ __align__(16) int hist[EV_BINS], sums[3][EV_BINS];
  __shared__ int above[EV_WARPS], equal[EV_WARPS];
  __shared__ __align__(8) int mine[2];
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
  // keys [i, i + 4) of the CTA; those past n are 0
  auto four = [&](int i, uint32_t (&k)[4]) {
    if (i + 4 <= n_held) {
      const uint4 q = *reinterpret_cast<const uint4*>(keys + i);
      k[0] = q.x; k[1] = q.y; k[2] = q.z; k[3] = q.w;
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) k[u] = i + u >= n ? 0u : i + u < n_held ? keys[i + u] : far_key(i + u);
    }
  };
  for (int i = tid; i < 3 * EV_BINS; i += EV_THREADS) sums[0][i] = 0;
  static_assert(EV_BINS == 2 * EV_THREADS, "a thread owns two bins");
  *reinterpret_cast<int2*>(hist + 2 * tid) = make_int2(0, 0);
  __syncthreads();
  if (size > 1) cluster_arrive();  // the sums are zero
  uint32_t prefix = 0;
  int want = m;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t known = digit == 0 ? 0u : digit == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    if (digit == 0) {
      // the weights come in once: 16 loads a thread on their way at a time
      for (int i0 = tid; i0 < n_held; i0 += 16 * EV_THREADS) {
        float x[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          if (i0 + u * EV_THREADS < n_held) x[u] = w[first + i0 + u * EV_THREADS];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int i = i0 + u * EV_THREADS;
          if (i >= n_held) break;
          const uint32_t key = evict_key(x[u], first + i, kv, P.sink, P.recent);
          keys[i] = key;
          atomicAdd(&hist[key >> 21], 1);
        }
      }
      for (int i = n_held + tid; i < n; i += EV_THREADS) atomicAdd(&hist[far_key(i) >> 21], 1);
    } else {
      for (int i = 4 * tid; i < n; i += 4 * EV_THREADS) {
        uint32_t k[4];
        four(i, k);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if ((k[u] & known) == prefix && i + u < n) atomicAdd(&hist[(k[u] >> shift) & mask], 1);
      }
    }
    __syncthreads();
    // this thread's two bins: their counts go to the CTA that sums them, and the sums come back
    int2 own = *reinterpret_cast<const int2*>(hist + 2 * tid);
    *reinterpret_cast<int2*>(hist + 2 * tid) = make_int2(0, 0);
    if (size > 1) {
      const uint32_t at = mapa_shared(smem_u32(&sums[digit][2 * tid]), (uint32_t)(2 * tid / (EV_BINS / size)));
      if (digit == 0) cluster_wait();
      if (own.x) add_cluster(at, own.x);
      if (own.y) add_cluster(at + 4, own.y);
      cluster_sync_all();
      own = ld_cluster_int2(at);
    }
    // the digit at which the count from the top reaches `want`
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
    static_assert(EV_WARPS == 32, "a warp sums the warps' counts");
    higher += __reduce_add_sync(0xFFFFFFFFu, lane > warp ? above[lane] : 0);
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
  // a warp's tokens [w0, w1), 4 a lane: above the key, equal to it (counts of 128 in 16 bits each)
  const int seg = ((n + EV_WARPS - 1) / EV_WARPS + 127) & ~127;
  const int w0 = min(warp * seg, n), w1 = min(w0 + seg, n);
  int gt = 0, eq = 0;
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    uint32_t k[4];
    four(i, k);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      gt += k[u] > prefix;
      eq += k[u] == prefix && i + u < n;
    }
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) {
    above[warp] = gt;  // every warp is past its last use: found was read after a barrier
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
    int2 before = make_int2(0, 0);
    if (lane < rank) before = ld_cluster_int2(mapa_shared(smem_u32(mine), lane));
    gt_before += __reduce_add_sync(0xFFFFFFFFu, before.x);
    eq_before += __reduce_add_sync(0xFFFFFFFFu, before.y);
    cluster_arrive();  // reads no other CTA's shared memory any more
  }
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane;
    uint32_t k[4] = {0u, 0u, 0u, 0u};
    if (i < w1) four(i, k);
    int own = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) own += (k[u] > prefix ? 1 : 0) + (k[u] == prefix && i + u < w1 ? 1 << 16 : 0);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += x;
    }
    const int step = __shfl_sync(0xFFFFFFFFu, upto, 31);
    int gi = gt_before + ((upto - own) & 0xFFFF), ei = eq_before + ((upto - own) >> 16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool is_gt = k[u] > prefix, is_eq = k[u] == prefix && i + u < w1;
      if (is_gt || (is_eq && ei < want)) index[gi + min(ei, want)] = first + i + u;
      gi += is_gt;
      ei += is_eq;
    }
    gt_before += step & 0xFFFF;
    eq_before += step >> 16;
  }
  if (size > 1) cluster_wait();  // nor does another CTA read this one's
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
  if ((e = launch_clusters(evict_select_kernel, dim3((unsigned)(s.Hkv * size), (unsigned)s.B), size, EV_THREADS,
                           (size_t)held * 4, stream, P, size, held)) != cudaSuccess)
    return e;
  const dim3 grid((unsigned)((keep + EM_ROWS - 1) / EM_ROWS), (unsigned)s.Hkv, (unsigned)s.B);
  return launch_overlapped(evict_move_kernel, grid, EM_THREADS, 0, stream, P);
}

}  // namespace fa
