// fa_paged.cu -- attention of new tokens over a paged cache and the weights that keys gather,
// for tiles of 16 query rows (a row = one token and one query head of a KV head).
//
//   o_i = sum_j exp2(c s_ij - m_i) v_j / l_i,  l_i = sum_j exp2(c s_ij - m_i),  c = scale log2 e,
// in one pass over the keys with a running maximum m and sum l. The keys of a tile are split
// into chunks of equal length, one CTA each; within a chunk each warp streams its own blocks
// of 16 keys (and values) through a ring of TMA boxes and keeps its own m, l and o, so that
// no warp waits for another until the end, when the CTA's warps merge in shared memory and
// the chunks in their cluster or in a second kernel (in a fixed order, so repeated calls give
// identical bits).
//
// P is rounded to bf16 for the product with V: the tensor cores take both operands in one type, and
// a second product with what the rounding left would double their work in the 128-row tiles. The sum
// l is of the unrounded weights, which the log-sum-exp needs. After the output's own rounding to bf16
// (1.65e-3 of it, root mean square) the error against 64 bits grows by 0.1% (one token over 2048
// keys) to 2% (701 tokens, window 1024).
//
// Few rows make this the read of K and V: 512 bytes a key and head against 16 x 512 flops on
// warp-level bf16 MMA (m16n8k16; a 128-row tcgen05 tile would be 7/8 empty here).
#include <math.h>
#include <string.h>

#include "fa_paged.cuh"

namespace fa {

constexpr int PR_ROWS = 16;     // query rows a tile
constexpr int PR_KEYS = 16;     // keys a block
constexpr int PR_WARPS = 4;
constexpr int PR_THREADS = PR_WARPS * 32;
constexpr int PR_BOX = PR_KEYS * 128;       // 64 dims x 16 keys
constexpr int PR_STAGES = 2;
constexpr int PR_STAGE = 4 * PR_BOX;        // K and V, two boxes each
constexpr int PW_STAGES = 3;
constexpr int PW_STAGE = 2 * PR_BOX;        // K only
constexpr int PR_OLD = FA_HEAD_DIM + 4;     // fp32 row of the merge buffer
constexpr int PR_DEEP = 6;                  // stages of a launch that leaves SMs idle
constexpr int PW_DEEP = 12;
constexpr int PR_CLUSTER = 8;               // chunks that a cluster merges
constexpr int PR_RING = PR_WARPS * PR_STAGES * PR_STAGE;
static_assert(PR_WARPS * PR_ROWS * (PR_OLD + 2) * 4 + PR_ROWS * (FA_HEAD_DIM + 2) * 4 <= PR_RING,
              "merge buffers fit");

struct RowsParams {
  PagedBatch p;
  int window, tiles, chunk, slots;  // tiles of rows, keys a chunk, partial results a row
  int max_rows;  // sequences of more rows a KV head are another kernel's (0: none are)
  int cluster;   // the chunks of a tile are one cluster of `slots` CTAs
  float scale_log2;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* out;
  long long out_stride;
  float* lse;
  float* part_o;    // [row][slot][128], row as part_row gives it
  float2* part_ml;  // [row][slot]
  float* weights;
  long long weights_ld;
};

// Partial results are numbered by (token, head), or, where only sequences of at most max_rows
// rows have some, by (sequence, KV head, row): max_q bounds a batch of long sequences too.
__device__ __forceinline__ long long part_row(const PagedBatch& p, int max_rows, int b, int g,
                                              long long token, int head, int row) {
  return max_rows > 0 ? ((long long)b * p.Hkv + g) * max_rows + row : token * p.Hq + head;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void* row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row)));
}
__device__ __forceinline__ float2 ld_cluster_float2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_float4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Byte of element (row, dim) in a block of PR_KEYS rows held as two swizzled 64-dim boxes.
__device__ __forceinline__ int box_byte(int row, int dim) {
  return (dim >> 6) * PR_BOX + row * 128 + ((((dim & 63) >> 3) ^ (row & 7)) << 4);
}

// A fragments of 16 query rows (rows past `rows` are zero): k-step s holds dims 16 s .. + 15.
__device__ __forceinline__ void load_q(const RowsParams& P, const SeqSpan& s, int g, int r0,
                                       int rows, int lane, uint32_t (&qf)[8][4]) {
  const __nv_bfloat16* src[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = r0 + (lane >> 2) + 8 * u;
    src[u] = nullptr;
    if (r < r0 + rows)
      src[u] = P.q + (long long)(s.q0 + r / P.p.G) * P.q_stride +
               (g * P.p.G + r % P.p.G) * FA_HEAD_DIM + 2 * (lane & 3);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const __nv_bfloat16* x = src[v & 1];
      qf[k][v] = x ? *reinterpret_cast<const uint32_t*>(x + 16 * k + 8 * (v >> 1)) : 0u;
    }
}

// scores of 16 rows x 16 keys: two accumulator fragments (keys 0-7, 8-15).
__device__ __forceinline__ void block_scores(const uint32_t (&qf)[8][4], const uint8_t* kblk,
                                             int lane, float (&sc)[2][4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int v = 0; v < 4; ++v) sc[n][v] = 0.0f;
  const int row = (lane & 7) + ((lane >> 4) << 3), dsel = ((lane >> 3) & 1) * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t b[4];
    ldmatrix_x4(b, kblk + box_byte(row, 16 * k + dsel));
    mma_16816(sc[0], qf[k], b[0], b[1]);
    mma_16816(sc[1], qf[k], b[2], b[3]);
  }
}

// A warp's ring of key blocks: blocks k0 + (w + i * PR_WARPS) * 16, i = 0, 1, ... below k_end.
template <int STAGES, int BYTES, bool VALUES>
struct BlockRing {
  uint8_t* buf;
  uint64_t* full;
  const CUtensorMap *tk, *tv;
  const PagedBatch* p;
  int b, g, k0, n;  // first key of the warp, number of its blocks

  // Row of the pools at which block i starts. An entry out of range lies behind the pool: the
  // copy fills the box with zeros.
  __device__ int row_of(int i) const {
    const int j = k0 + i * PR_WARPS * PR_KEYS;
    const int pg = page_of(*p, b, j);
    return pg < 0 ? p->num_pages * p->Hkv * p->page : (pg * p->Hkv + g) * p->page + j % p->page;
  }
  __device__ void issue(int i, int row) const {
    const int s = i % STAGES;
    uint8_t* dst = buf + s * BYTES;
    mbar_arrive_expect_tx(&full[s], BYTES);
    tma_load_2d(dst, tk, &full[s], 0, row);
    tma_load_2d(dst + PR_BOX, tk, &full[s], 64, row);
    if (VALUES) {
      tma_load_2d(dst + 2 * PR_BOX, tv, &full[s], 0, row);
      tma_load_2d(dst + 3 * PR_BOX, tv, &full[s], 64, row);
    }
  }
  // Lets copies in flight land before the CTA's shared memory goes away (abort path).
  __device__ void drain(int from) const {
    for (int i = from; i < min(n, from + STAGES); ++i) {
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u))
        if (globaltimer_ns() - t0 > 200000000ull) break;
    }
  }
};

// STAGES: blocks of a warp on their way, PR_STAGES with 3 CTAs an SM, or PR_DEEP with one.
template <int STAGES>
__global__ void __launch_bounds__(PR_THREADS, STAGES == PR_STAGES ? 3 : 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const __grid_constant__ RowsParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full[PR_WARPS][STAGES];
  __shared__ int abort_word;
  wait_earlier_kernel();
  allow_next_kernel();
  const PagedBatch& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = blockIdx.x % P.slots, tile = blockIdx.x / P.slots;
  const int g = blockIdx.y, b = blockIdx.z;
  const SeqSpan s = seq_span(p, b);
  const int r0 = tile * PR_ROWS, rows = min(PR_ROWS, s.n * p.G - r0);
  if (rows <= 0 || (P.max_rows > 0 && s.n * p.G > P.max_rows)) return;
  int lo, hi;
  row_keys(s, p.G, P.window, r0, r0 + rows, &lo, &hi);
  const bool single = P.slots == 1;
  // chunk `slot` of the keys: chunks lie at multiples of P.chunk, the first holds lo
  const int c0 = (lo / P.chunk + slot) * P.chunk;
  const int k_lo = max(lo & ~(PR_KEYS - 1), c0), k_hi = min(hi, c0 + P.chunk);
  if (k_lo >= k_hi && !(single || P.cluster || (slot == 0 && hi <= lo))) return;  // the merge skips it

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < PR_WARPS * STAGES; ++i) mbar_init(&full[0][0] + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort_flag = &abort_word;

  BlockRing<STAGES, PR_STAGE, true> ring;
  ring.buf = smem + warp * STAGES * PR_STAGE;
  ring.full = full[warp];
  ring.tk = &tk;
  ring.tv = &tv;
  ring.p = &p;
  ring.b = b;
  ring.g = g;
  ring.k0 = k_lo + warp * PR_KEYS;
  const int left = k_hi - ring.k0;
  ring.n = left > 0 ? (left + PR_WARPS * PR_KEYS - 1) / (PR_WARPS * PR_KEYS) : 0;
  if (lane < min(STAGES, ring.n)) ring.issue(lane, ring.row_of(lane));  // a block a lane

  uint32_t qf[8][4];
  load_q(P, s, g, r0, rows, lane, qf);
  int pos[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = r0 + (lane >> 2) + 8 * u;
    pos[u] = r < r0 + rows ? s.kv - s.n + r / p.G : -1;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int v = 0; v < 4; ++v) o[n][v] = 0.0f;

  for (int i = 0; i < ring.n; ++i) {
    const int st = i % STAGES;
    int next = 0;  // looked up while this block is on its way
    if (lane == 0 && i + STAGES < ring.n) next = ring.row_of(i + STAGES);
    if (!warp_wait(&ring.full[st], (uint32_t)(i / STAGES) & 1u, abort_flag, WD_PAGED | 1u)) {
      if (lane == 0) ring.drain(i);
      break;
    }
    const uint8_t* kblk = ring.buf + st * PR_STAGE;
    const uint8_t* vblk = kblk + 2 * PR_BOX;
    const int j0 = ring.k0 + i * PR_WARPS * PR_KEYS;
    float sc[2][4];
    block_scores(qf, kblk, lane, sc);
    // edge blocks hold keys that some row does not see
    const bool edge = j0 + PR_KEYS > s.kv - s.n + r0 / p.G + 1 ||
                      (P.window > 0 && j0 <= s.kv - s.n + (r0 + rows - 1) / p.G - P.window);
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x = sc[n][v] * P.scale_log2;
        if (edge) {
          const int j = j0 + 8 * n + 2 * (lane & 3) + (v & 1), q = pos[v >> 1];
          if (j > q || (P.window > 0 && j <= q - P.window)) x = -INFINITY;
        }
        sc[n][v] = x;
        mx[v >> 1] = fmaxf(mx[v >> 1], x);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xFFFFFFFFu, mx[u], 1));
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xFFFFFFFFu, mx[u], 2));
      const float base = mx[u] == -INFINITY ? 0.0f : mx[u];
      const float f = exp2_approx(m[u] - base);
      m[u] = mx[u];
      l[u] *= f;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][2 * u] *= f;
        o[n][2 * u + 1] *= f;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int v = 2 * u; v < 2 * u + 2; ++v) {
          sc[n][v] = exp2_approx(sc[n][v] - base);
          l[u] += sc[n][v];
        }
    }
    const uint32_t pf[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                            pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
    // values of keys outside [lo, hi) may be anything, NaN too: they count as zero
    uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
    const bool ragged = j0 < lo || j0 + PR_KEYS > hi;
    if (ragged) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = j0 + 8 * h + 2 * (lane & 3);
        keep[h] = (j >= lo && j < hi ? 0x0000FFFFu : 0u) |
                  (j + 1 >= lo && j + 1 < hi ? 0xFFFF0000u : 0u);
      }
    }
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vd = (lane >> 4) * 8;
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
      uint32_t v[4];
      ldmatrix_x4_trans(v, vblk + box_byte(vrow, 8 * n + vd));
      if (ragged) {
        v[0] &= keep[0];
        v[1] &= keep[1];
        v[2] &= keep[0];
        v[3] &= keep[1];
      }
      mma_16816(o[n], pf, v[0], v[1]);
      mma_16816(o[n + 1], pf, v[2], v[3]);
    }
    __syncwarp();
    if (lane == 0 && i + STAGES < ring.n) ring.issue(i + STAGES, next);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xFFFFFFFFu, l[u], 1);
    l[u] += __shfl_xor_sync(0xFFFFFFFFu, l[u], 2);
  }

  // merge the warps: o, m, l of each in shared memory (the rings are idle)
  __syncthreads();
  float* mo = reinterpret_cast<float*>(smem);
  float2* ml = reinterpret_cast<float2*>(mo + PR_WARPS * PR_ROWS * PR_OLD);
  float* sum_o = reinterpret_cast<float*>(ml + PR_WARPS * PR_ROWS);  // the CTA's, for its cluster
  float2* sum_ml = reinterpret_cast<float2*>(sum_o + PR_ROWS * FA_HEAD_DIM);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (lane >> 2) + 8 * u;
    float* dst = mo + (warp * PR_ROWS + r) * PR_OLD + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 16; ++n)
      *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * u], o[n][2 * u + 1]);
    if ((lane & 3) == 0) ml[warp * PR_ROWS + r] = make_float2(m[u], l[u]);
  }
  __syncthreads();
  for (int w = threadIdx.x; w < rows * (FA_HEAD_DIM / 4); w += PR_THREADS) {
    const int r = w / (FA_HEAD_DIM / 4), d = 4 * (w % (FA_HEAD_DIM / 4));
    float mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < PR_WARPS; ++i) mm = fmaxf(mm, ml[i * PR_ROWS + r].x);
    const float base = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < PR_WARPS; ++i) {
      const float2 e = ml[i * PR_ROWS + r];
      const float f = exp2_approx(e.x - base);
      ll = fmaf(e.y, f, ll);
      const float4 x = *reinterpret_cast<const float4*>(mo + (i * PR_ROWS + r) * PR_OLD + d);
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z);
      acc.w = fmaf(x.w, f, acc.w);
    }
    const long long t = s.q0 + (r0 + r) / p.G;
    const int h = g * p.G + (r0 + r) % p.G;
    if (P.cluster) {
      *reinterpret_cast<float4*>(sum_o + r * FA_HEAD_DIM + d) = acc;
      if (d == 0) sum_ml[r] = make_float2(mm, ll);
    } else if (single) {
      const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
      *reinterpret_cast<uint2*>(P.out + t * P.out_stride + h * FA_HEAD_DIM + d) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (d == 0 && P.lse) P.lse[t * p.Hq + h] = 0.693147180559945309f * (mm + log2f(ll));
    } else {
      const long long rec = part_row(p, P.max_rows, b, g, t, h, r0 + r) * P.slots + slot;
      *reinterpret_cast<float4*>(P.part_o + rec * FA_HEAD_DIM + d) = acc;
      if (d == 0) P.part_ml[rec] = make_float2(mm, ll);
    }
  }
  if (!P.cluster) return;
  // the cluster's CTAs (rank = slot) take every slots-th row each and read all CTAs' sums of it
  cluster_sync_all();
  for (int r = slot + P.slots * warp; r < rows; r += P.slots * PR_WARPS) {
    const uint32_t ao = smem_u32(sum_o + r * FA_HEAD_DIM + 4 * lane), am = smem_u32(sum_ml + r);
    float2 e[PR_CLUSTER];
    float4 x[PR_CLUSTER];
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < PR_CLUSTER; ++k) {
      e[k] = make_float2(-INFINITY, 0.0f);
      x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k < P.slots) {
        e[k] = ld_cluster_float2(mapa_shared(am, k));
        x[k] = ld_cluster_float4(mapa_shared(ao, k));
      }
      mm = fmaxf(mm, e[k].x);
    }
    const float base = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < PR_CLUSTER; ++k) {
      const float f = exp2_approx(e[k].x - base);
      ll = fmaf(e[k].y, f, ll);
      acc.x = fmaf(x[k].x, f, acc.x);
      acc.y = fmaf(x[k].y, f, acc.y);
      acc.z = fmaf(x[k].z, f, acc.z);
      acc.w = fmaf(x[k].w, f, acc.w);
    }
    const long long t = s.q0 + (r0 + r) / p.G;
    const int h = g * p.G + (r0 + r) % p.G;
    const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
    *reinterpret_cast<uint2*>(P.out + t * P.out_stride + h * FA_HEAD_DIM + 4 * lane) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (lane == 0 && P.lse) P.lse[t * p.Hq + h] = 0.693147180559945309f * (mm + log2f(ll));
  }
  cluster_sync_all();  // the CTA's shared memory is read no more
}

struct JoinParams {
  PagedBatch p;
  int window, chunk, slots;
  int tile_rows;           // rows whose keys were split together
  int max_rows, min_rows;  // as RowsParams::max_rows; rows of a sequence must exceed min_rows
  int rows;                // rows a sequence and KV head may have, where max_rows is set
  const float* part_o;
  const float2* part_ml;
  __nv_bfloat16* out;
  long long out_stride;
  float* lse;
};

// Joins the chunks of each row. SPLIT warps a row, every SPLIT-th chunk each, then the warps in
// order: 8 where rows are few and chunks may be many (one token over 30000 keys in 118 chunks: 48
// us with one warp a row, 35 with 8), 1 where there are thousands of rows (a chunk of 100 tokens:
// 30 us with 8, 23 with 1; 64 decode tokens: 338 and 325).
template <int SPLIT>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ JoinParams P) {
  __shared__ float4 part[SPLIT][32];
  __shared__ float2 part_ml[SPLIT];
  const PagedBatch& p = P.p;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % SPLIT;
  const long long at = (long long)blockIdx.x * (8 / SPLIT) + (threadIdx.x >> 5) / SPLIT;
  int b = 0, r = 0, g = 0;  // sequence, row of it in its KV head
  SeqSpan s;
  bool live = false;
  if (P.max_rows > 0) {
    r = (int)(at % P.rows);
    g = (int)(at / P.rows % p.Hkv);
    b = (int)(at / P.rows / p.Hkv);
    if (b < p.B) {
      s = seq_span(p, b);
      live = r < s.n * p.G && s.n * p.G <= P.max_rows;
    }
  } else {
    const int t = (int)(at / p.Hq), h = (int)(at % p.Hq);
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int i = b0 + lane + 1;
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, i <= p.B && p.q_start[i] <= t));
      b += n;
      if (n < 32) break;
    }
    if (t < p.total_q && b < p.B) {
      s = seq_span(p, b);
      live = t >= s.q0 && t - s.q0 < s.n && s.n * p.G > P.min_rows;
      g = h / p.G;
      r = (t - s.q0) * p.G + h % p.G;
    }
  }
  wait_earlier_kernel();
  if (!live) return;
  const int tile = r / P.tile_rows;  // rows whose keys were split together
  int lo, hi;
  row_keys(s, p.G, P.window, tile * P.tile_rows, min((tile + 1) * P.tile_rows, s.n * p.G), &lo, &hi);
  const int slots = hi > lo ? (hi - 1) / P.chunk - lo / P.chunk + 1 : 1;
  const long long t = s.q0 + r / p.G;
  const int h = g * p.G + r % p.G;
  const long long row = part_row(p, P.max_rows, b, g, t, h, r);
  const float2* ml = P.part_ml + row * P.slots;
  const float4* po = reinterpret_cast<const float4*>(P.part_o + row * P.slots * FA_HEAD_DIM) + lane;
  float mm = -INFINITY, ll = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float2& e, const float4& x) {
    const float top = fmaxf(mm, e.x), base = top == -INFINITY ? 0.0f : top;
    const float f = exp2_approx(mm - base), fe = exp2_approx(e.x - base);
    mm = top;
    ll = ll * f + e.y * fe;
    acc.x = acc.x * f + x.x * fe;
    acc.y = acc.y * f + x.y * fe;
    acc.z = acc.z * f + x.z * fe;
    acc.w = acc.w * f + x.w * fe;
  };
#pragma unroll 4
  for (int k = warp; k < slots; k += SPLIT) add(ml[k], po[k * (FA_HEAD_DIM / 4)]);
  if (SPLIT > 1) {  // the CTA has one row: all its warps are here
    part[warp][lane] = acc;
    if (lane == 0) part_ml[warp] = make_float2(mm, ll);
    __syncthreads();
    if (warp > 0) return;
    for (int k = 1; k < SPLIT; ++k) add(part_ml[k], part[k][lane]);
  }
  const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
  *reinterpret_cast<uint2*>(P.out + t * P.out_stride + h * FA_HEAD_DIM + 4 * lane) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0 && P.lse) P.lse[t * p.Hq + h] = 0.693147180559945309f * (mm + log2f(ll));
}

// Weights: a warp owns its blocks of 16 keys and runs over every tile of query rows that sees
// them, so a key's sum is taken by one warp in one order.
template <int STAGES>
__global__ void __launch_bounds__(PR_THREADS, STAGES == PW_STAGES ? 4 : 1)
    paged_weights_rows_kernel(const __grid_constant__ CUtensorMap tk,
                              const __grid_constant__ RowsParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full[PR_WARPS][STAGES];
  __shared__ int abort_word;
  wait_earlier_kernel();
  allow_next_kernel();
  const PagedBatch& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const SeqSpan s = seq_span(p, b);
  const int n_rows = s.n * p.G;
  if (n_rows <= 0 || (P.max_rows > 0 && n_rows > P.max_rows)) return;
  int lo, hi;
  row_keys(s, p.G, P.window, 0, n_rows, &lo, &hi);
  const int c0 = (lo / P.chunk + blockIdx.x) * P.chunk;
  const int k_lo = max(lo & ~(PR_KEYS - 1), c0), k_hi = min(hi, c0 + P.chunk);
  if (k_lo >= k_hi) return;
  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < PR_WARPS * STAGES; ++i) mbar_init(&full[0][0] + i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  BlockRing<STAGES, PW_STAGE, false> ring;
  ring.buf = smem + warp * STAGES * PW_STAGE;
  ring.full = full[warp];
  ring.tk = &tk;
  ring.tv = nullptr;
  ring.p = &p;
  ring.b = b;
  ring.g = g;
  ring.k0 = k_lo + warp * PR_KEYS;
  const int left = k_hi - ring.k0;
  ring.n = left > 0 ? (left + PR_WARPS * PR_KEYS - 1) / (PR_WARPS * PR_KEYS) : 0;
  if (lane < min(STAGES, ring.n)) ring.issue(lane, ring.row_of(lane));  // a block a lane

  uint32_t qf[8][4];
  float ls[2];
  int pos[2];
  int have = -1;
  // after the sums are spread over the lanes, a lane holds this key of a block
  const int key = 8 * (lane >> 4) + 2 * (lane & 3) + ((lane >> 3) & 1);
  float* w = P.weights + ((long long)b * p.Hkv + g) * P.weights_ld;
  auto old_weight = [&](int i) {
    const int j = ring.k0 + i * PR_WARPS * PR_KEYS + key;
    return i < ring.n && !(lane & 4) && j >= lo && j < hi ? w[j] : 0.0f;
  };
  float old = old_weight(0);
  for (int i = 0; i < ring.n; ++i) {
    const int st = i % STAGES;
    // the next loads that the block's end needs, a block ahead
    const float old_next = old_weight(i + 1);
    int next = 0;
    if (lane == 0 && i + STAGES < ring.n) next = ring.row_of(i + STAGES);
    if (!warp_wait(&ring.full[st], (uint32_t)(i / STAGES) & 1u, &abort_word, WD_PAGED | 2u)) {
      if (lane == 0) ring.drain(i);
      break;
    }
    const uint8_t* kblk = ring.buf + st * PW_STAGE;
    const int j0 = ring.k0 + i * PR_WARPS * PR_KEYS;
    // tokens that see a key of the block: positions [j0, j0 + 15 + window)
    const int i0 = max(0, j0 - (s.kv - s.n));
    const int i1 = P.window > 0 ? min(s.n, j0 + PR_KEYS - 1 + P.window - (s.kv - s.n)) : s.n;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // keys 2 (lane & 3) + {0, 1} + {0, 8}
    for (int tile = i0 * p.G / PR_ROWS; tile * PR_ROWS < i1 * p.G; ++tile) {
      if (tile != have) {
        have = tile;
        const int r0 = tile * PR_ROWS;
        load_q(P, s, g, r0, min(PR_ROWS, n_rows - r0), lane, qf);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = r0 + (lane >> 2) + 8 * u;
          pos[u] = -1;
          ls[u] = 0.0f;
          if (r < n_rows) {
            pos[u] = s.kv - s.n + r / p.G;
            ls[u] = 1.44269504088896341f *
                    P.lse[(long long)(s.q0 + r / p.G) * p.Hq + g * p.G + r % p.G];
          }
        }
      }
      float sc[2][4];
      block_scores(qf, kblk, lane, sc);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int j = j0 + 8 * n + 2 * (lane & 3) + (v & 1), q = pos[v >> 1];
          const bool seen = j <= q && !(P.window > 0 && j <= q - P.window);
          if (seen) sum[2 * n + (v & 1)] += exp2_approx(fmaf(sc[n][v], P.scale_log2, -ls[v >> 1]));
        }
    }
    __syncwarp();
    if (lane == 0 && i + STAGES < ring.n) ring.issue(i + STAGES, next);
    // sum over the 8 lanes of a key, halving what a lane holds at each exchange
    const bool n1 = lane & 16, odd = lane & 8;
    float a = n1 ? sum[2] : sum[0], c = n1 ? sum[3] : sum[1];
    a += __shfl_xor_sync(0xFFFFFFFFu, n1 ? sum[0] : sum[2], 16);
    c += __shfl_xor_sync(0xFFFFFFFFu, n1 ? sum[1] : sum[3], 16);
    float total = odd ? c : a;
    total += __shfl_xor_sync(0xFFFFFFFFu, odd ? a : c, 8);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, 4);
    const int j = j0 + key;
    if (!(lane & 4) && j >= lo && j < hi) w[j] = old + total;
    old = old_next;
  }
}

FA_WATCHDOG_READER(read_watchdog_paged)

// ------------------------------------------------------------------------- host side
PagedBatch paged_batch(const fa_paged_shape& s, const fa_paged_cache& c) {
  PagedBatch p;
  p.table = c.page_table;
  p.q_start = c.q_start;
  p.kv_len = c.kv_len;
  p.B = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.G = s.Hq / s.Hkv;
  p.page = s.page_size;
  p.num_pages = s.num_pages;
  p.max_pages = s.max_pages;
  p.total_q = s.total_q;
  p.max_q = s.max_q;
  p.max_kv = s.max_kv;
  return p;
}

bool encode_pool(CUtensorMap* map, const void* pool, const fa_paged_shape& s, int rows) {
  const auto encode = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(tensor_map_encoder());
  if (!encode) return false;
  cuuint64_t dims[2] = {FA_HEAD_DIM, (cuuint64_t)s.num_pages * s.Hkv * s.page_size};
  cuuint64_t strides[1] = {FA_HEAD_DIM * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)rows};
  cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys by which a call is split: those that `tokens` neighbouring tokens see in a window of up to
// 1280, else the cache's (on the device, one token over 8 KV heads of 8000 keys, window 600: 8.7 us
// split by the cache's, 6.6 by the window's; 24 such sequences, window 1024: 25 and 20; 64, window
// 128: 15 and 12; with a window of 4000 one took 10 and 13). All of these were caches of 8000 keys: over
// 131072, where 48 chunks of the cache leave 24 CTAs to a window of 4096, one token takes 47 us. Key
// weights, which nothing merges, are split by the cache's (64 sequences, window 600: 17 and 21).
static int rows_span(const fa_paged_shape& s, int window, int tokens) {
  const long long n = (long long)window + tokens;
  return window > 0 && n <= 1280 && n < s.max_kv ? (int)n : s.max_kv;
}

// Keys a chunk, in multiples of 64: `ctas` CTAs for the longest batch the shape allows, but at
// least 256 keys (below that the merge costs more than the chunk's own read). Real batches are
// shorter and ragged, so the targets are many CTAs an SM: 64 sequences of up to 16384 tokens
// decode in 452, 366, 345, 356 us for 2, 8, 32, 64 a SM (3 are resident); key weights of 32
// sequences of up to 8192 take 68, 63, 63, 68 us for 8, 16, 32, 64 (4 are resident). A batch that
// one wave of the `resident` CTAs can read in chunks of at most 768 keys (and few enough of them where
// they are merged) is cut to fill that wave:
// a second, partly filled one costs as much as the first (2 sequences of 8000 keys, 8 KV heads: 19
// us in chunks of 256, 15 in chunks of 320; 8 of 3000 25 and 20).
//   `merged`: partial results that a second kernel reads, so at most 48 chunks a tile (one token over
// 30000 keys, 8 KV heads: 35 us in 118 chunks, 27 in 48). Key weights merge nothing (one token over
// 131072 keys, 1 KV head: 49 us in 48 chunks, 18 in 512; 8 KV heads and a window of 4096: 42 and 16).
static int rows_chunk(const fa_paged_shape& s, int keys, int tiles, int ctas, int resident, bool merged) {
  const long long units = (long long)s.B * s.Hkv * tiles;
  const int most = merged ? 48 : keys;  // chunks a tile
  if (resident >= 2 * units) {
    const long long n = resident / units, c = ((keys + n - 1) / n + 63) / 64 * 64;
    if (c >= 256 && c <= 768 && c * most >= keys) return (int)c;
  }
  const long long want = (ctas + units - 1) / units;
  const long long n = want < most ? want : most;
  const long long c = n > 0 ? ((keys + n - 1) / n + 63) / 64 * 64 : 0;
  return (int)(c < 256 ? 256 : c);
}

int chunk_slots(const fa_paged_shape& s, int window, int chunk, int tokens) {
  long long n = ((long long)s.max_kv + chunk - 1) / chunk;
  if (window > 0) {
    const long long span = (long long)window + tokens;
    const long long m = (span + chunk - 1) / chunk + 1;
    n = m < n ? m : n;
  }
  return (int)(n < 1 ? 1 : n);
}

// How a call runs: tensor-core tiles for sequences of more than 16 rows a KV head, 16-row tiles
// for the others (for all of them where the heads of one token do not fit a tile).
struct AttendPlan {
  TilePlan t;
  RowsParams r;
  size_t rows_records;
};

static cudaError_t attend_plan(const fa_paged_shape& s, int window, AttendPlan* a, size_t* bytes) {
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  if ((e = tile_plan(s, window, &a->t)) != cudaSuccess) return e;
  const int G = s.Hq / s.Hkv;
  const long long rows = (long long)(s.max_q < s.total_q ? s.max_q : s.total_q) * G;
  RowsParams* P = &a->r;
  memset(P, 0, sizeof(*P));
  P->max_rows = a->t.tok > 0 || rows <= PR_ROWS ? PR_ROWS : 0;
  P->tiles = P->max_rows > 0 ? 1 : (int)((rows + PR_ROWS - 1) / PR_ROWS);
  const int tokens = (PR_ROWS + G - 1) / G, keys = rows_span(s, window, tokens);
  P->chunk = rows_chunk(s, keys, P->tiles, 32 * sms, 3 * sms, true);
  P->slots = chunk_slots(s, window, P->chunk, tokens);
  P->window = window;
  // Caches of at most 4096 tokens (or short windows) go in 8 chunks of at least 64 tokens that one
  // cluster merges: the second kernel takes longer than such a chunk (one token over 2048 keys: 12
  // us with it, 10 without). A window starts inside a chunk, so 7 chunks' length is cut. Where that makes more CTAs than are resident, single CTAs pack better than clusters
  // (8 x 8 tiles over 3000 keys: 21 us against 25). Up to 256 tokens one CTA is quicker alone.
  if (P->max_rows > 0 && keys <= 256) {
    P->chunk = s.max_kv > 0 ? (s.max_kv + 63) / 64 * 64 : 64;
    P->slots = 1;
  } else if (P->max_rows > 0 && keys <= PR_CLUSTER * 512 && P->slots > 1 &&
      (long long)s.B * s.Hkv * PR_CLUSTER <= 3LL * sms) {
    const int parts = keys < s.max_kv ? PR_CLUSTER - 1 : PR_CLUSTER;
    const int c = ((keys + parts - 1) / parts + 63) / 64 * 64;
    const int n = chunk_slots(s, window, c, tokens);
    if (n <= PR_CLUSTER) {
      P->chunk = c;
      P->slots = n;
      P->cluster = n > 1;
    }
  }
  a->rows_records = 0;
  if (P->slots > 1 && !P->cluster)
    a->rows_records = (P->max_rows > 0 ? (size_t)s.B * s.Hkv * PR_ROWS : (size_t)s.total_q * s.Hq) * P->slots;
  *bytes = (a->rows_records + a->t.records) * (FA_HEAD_DIM * sizeof(float) + sizeof(float2));
  return cudaSuccess;
}

cudaError_t paged_attend_workspace(const fa_paged_shape& s, int window, size_t* bytes) {
  AttendPlan a;
  return attend_plan(s, window, &a, bytes);
}

cudaError_t launch_paged_attend(const fa_paged_shape& s, const fa_paged_cache& c, const void* q,
                                int64_t q_stride, float scale, int window, void* out,
                                int64_t out_stride, float* lse, void* workspace,
                                cudaStream_t stream, const char** why) {
  AttendPlan a;
  size_t bytes = 0;
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess || (e = attend_plan(s, window, &a, &bytes)) != cudaSuccess) return e;
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml = reinterpret_cast<float2*>(part_o + (a.rows_records + a.t.records) * FA_HEAD_DIM);
  RowsParams& P = a.r;
  P.p = paged_batch(s, c);
  P.scale_log2 = scale * 1.44269504088896341f;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.q_stride = q_stride;
  P.out = static_cast<__nv_bfloat16*>(out);
  P.out_stride = out_stride;
  P.lse = lse;
  P.part_o = part_o;
  P.part_ml = part_ml;
  CUtensorMap tk, tv;
  if (!encode_pool(&tk, c.K, s, PR_KEYS) || !encode_pool(&tv, c.V, s, PR_KEYS)) {
    *why = "cuTensorMapEncodeTiled rejected the pools";
    return cudaErrorInvalidValue;
  }
  // A launch that leaves SMs idle has the shared memory for all of a warp's blocks at once (on the
  // device, one token over 256 keys: 8.0 us with 2 stages, 6.8 with 6; over 2048 keys 9.1 and 7.8).
  const bool deep = (long long)P.slots * P.tiles * s.Hkv * s.B <= sms;
  auto* kernel = deep ? paged_rows_kernel<PR_DEEP> : paged_rows_kernel<PR_STAGES>;
  const int smem = PR_WARPS * (deep ? PR_DEEP : PR_STAGES) * PR_STAGE + 1024;
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(kernel), smem)) != cudaSuccess) return e;
  const dim3 grid((unsigned)(P.slots * P.tiles), (unsigned)s.Hkv, (unsigned)s.B);
  if ((e = launch_clusters(kernel, grid, P.cluster ? P.slots : 1, PR_THREADS, smem, stream, tk, tv, P)) != cudaSuccess)
    return e;
  float* tile_o = part_o + a.rows_records * FA_HEAD_DIM;
  float2* tile_ml = part_ml + a.rows_records;
  if (a.t.tok > 0 &&
      (e = launch_tiles(s, c, a.t, q, q_stride, scale, window, out, out_stride, lse, tile_o, tile_ml,
                        PR_ROWS, stream, why)) != cudaSuccess)
    return e;
  JoinParams J;
  memset(&J, 0, sizeof(J));
  J.p = P.p;
  J.window = window;
  J.out = P.out;
  J.out_stride = out_stride;
  J.lse = lse;
  auto join = [&](int chunk, int slots, int tile_rows, int max_rows, int min_rows, const float* o,
                  const float2* ml) {
    J.chunk = chunk;
    J.slots = slots;
    J.tile_rows = tile_rows;
    J.max_rows = max_rows;
    J.min_rows = min_rows;
    J.part_o = o;
    J.part_ml = ml;
    const long long most = (long long)(s.max_q < s.total_q ? s.max_q : s.total_q) * P.p.G;
    J.rows = most < max_rows ? (int)most : max_rows;
    const long long rows = max_rows > 0 ? (long long)s.B * s.Hkv * J.rows : (long long)s.total_q * s.Hq;
    if (rows == 0) return cudaSuccess;  // max_q = 0: rows behind the last sequence only
    if (rows <= 4 * sms)
      return launch_overlapped(paged_join_kernel<8>, dim3((unsigned)rows), 256, 0, stream, J);
    return launch_overlapped(paged_join_kernel<1>, dim3((unsigned)((rows + 7) / 8)), 256, 0, stream, J);
  };
  if (P.slots > 1 && !P.cluster &&
      (e = join(P.chunk, P.slots, PR_ROWS, P.max_rows, 0, part_o, part_ml)) != cudaSuccess)
    return e;
  if (a.t.slots > 1) e = join(a.t.chunk, a.t.slots, a.t.pair * a.t.tok * P.p.G, 0, PR_ROWS, tile_o, tile_ml);
  return e;
}

cudaError_t launch_paged_weights(const fa_paged_shape& s, const fa_paged_cache& c, const void* q,
                                 int64_t q_stride, float scale, int window, const float* lse,
                                 float* weights, int64_t weights_ld, cudaStream_t stream,
                                 const char** why) {
  RowsParams P;
  memset(&P, 0, sizeof(P));
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  P.p = paged_batch(s, c);
  P.window = window;
  P.scale_log2 = scale * 1.44269504088896341f;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.q_stride = q_stride;
  P.lse = const_cast<float*>(lse);
  P.weights = weights;
  P.weights_ld = weights_ld;
  // tensor-core tiles as in attend_plan
  const long long max_q = s.max_q < s.total_q ? s.max_q : s.total_q;
  const bool tiles = P.p.G <= 128 && max_q * P.p.G > PR_ROWS;
  P.max_rows = tiles ? PR_ROWS : 0;
  P.chunk = rows_chunk(s, s.max_kv, 1, 16 * sms, 4 * sms, false);
  P.slots = chunk_slots(s, window, P.chunk, tiles ? PR_ROWS : (int)max_q);
  CUtensorMap tk;
  if (!encode_pool(&tk, c.K, s, PR_KEYS)) {
    *why = "cuTensorMapEncodeTiled rejected the pool";
    return cudaErrorInvalidValue;
  }
  const bool deep = (long long)P.slots * s.Hkv * s.B <= sms;  // as in launch_paged_attend
  auto* kernel = deep ? paged_weights_rows_kernel<PW_DEEP> : paged_weights_rows_kernel<PW_STAGES>;
  const int smem = PR_WARPS * (deep ? PW_DEEP : PW_STAGES) * PW_STAGE + 1024;
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(kernel), smem)) != cudaSuccess) return e;
  const dim3 grid((unsigned)P.slots, (unsigned)s.Hkv, (unsigned)s.B);
  if ((e = launch_overlapped(kernel, grid, PR_THREADS, smem, stream, tk, P)) != cudaSuccess || !tiles) return e;
  return launch_weight_tiles(s, c, q, q_stride, scale, window, lse, weights, weights_ld, PR_ROWS,
                             stream, why);
}

}  // namespace fa
