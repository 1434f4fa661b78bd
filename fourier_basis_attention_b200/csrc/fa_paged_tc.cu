// fa_paged_tc.cu -- attention of new tokens over a paged cache on tcgen05, for sequences with
// more query rows than one 16-row tile (a row = one token and one query head of a KV head).
//
// An SM works on two tiles of 128 rows and streams the keys and values of their KV head in
// blocks of 128 through a ring of TMA boxes. Per block and tile: S = Q K^T into tensor memory, one
// thread a row turns S into weights P = exp2(c s - m) (running reference m, running sum l),
// writes P back over S in bf16 (the tensor core takes both operands in one type; what that costs is
// said at the 16-row tiles), and O += P V reads P from tensor memory. While one tile's
// threads work on their weights the tensor core works on the other tile. The two are one CTA's,
// which share each block, or two CTAs', of which one starts or ends while the other computes.
//   The reference m follows the running maximum only when it falls behind by 2^8: the weights
// stay below 256, which costs bf16 and fp32 nothing, and scaling O (a pass over it in tensor
// memory) runs a few times a row instead of once a block.
//
// Bound: 4 * 128 flops a (row, key) on the tensor core, and one exp2 (16 a clock and SM): for
// a 128 x 128 tile 1024 clocks each.
//
// The last kernel here sums the weights that keys gather on the same tiles.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "fa_paged.cuh"

namespace fa {

constexpr int PT_KEYS = 128;                  // keys a block
constexpr int PT_TILE = 128;                  // rows a tile
constexpr int PT_HALF = 128 * 128;            // 64 dims x 128 rows
constexpr int PT_BLOCK = 2 * PT_HALF;         // bytes of a block of K, V or Q rows

// An attention CTA of NT tiles: 4 warps a tile turn scores into weights; besides them a producer,
// an MMA warp and two idle ones. A CTA of one tile takes half of the SM's shared and tensor memory
// and registers.
template <int NT>
struct Tiles {
  static constexpr int SOFT = 4 * NT, THREADS = (SOFT + 4) * 32;
  static constexpr int STAGES = NT == 2 ? 5 : 2;  // of the ring of key and value blocks
  // What the warps share besides the blocks (no static arrays: the blocks start at the aligned
  // beginning of shared memory).
  struct Shared {
    uint64_t full[STAGES], empty[STAGES], q_full, s_full[NT], p_full[2 * NT], o_full[NT], drained;
    uint32_t tmem;
    int abort, issued;  // copies into the ring
  };
  static constexpr int SMEM = (NT + STAGES) * PT_BLOCK + (int)sizeof(Shared);
  // Registers after setmaxnreg, a thread: the two sums must not pass what the launch gives the
  // block, or the raise waits for good (launches check it).
  static constexpr int MORE = 208, LESS = NT == 2 ? 88 : 48;
  static constexpr int REGS = SOFT * 32 * MORE + 4 * 32 * LESS;
};
static_assert(Tiles<2>::SMEM <= 232448, "one CTA fits the SM");
static_assert(2 * (Tiles<1>::SMEM + 1024) <= 233472, "two CTAs fit the SM");
constexpr float PT_SLACK = 8.0f;              // log2 by which the maximum may pass m

struct TileParams {
  PagedBatch p;
  int window, chunk, slots, tiles;  // keys a chunk, partial results a row, CTA tiles
  int tok, box;                     // tokens of a 128-row tile, key rows of a TMA box
  int skip_rows;                    // sequences of at most so many rows are another kernel's
  float scale_log2;
  __nv_bfloat16* out;
  long long out_stride;
  float* lse;
  float* part_o;    // [row][slot][128], row = token * Hq + head
  float2* part_ml;  // [row][slot]
};

// Waits for this thread's loads from tensor memory; the values depend on the wait, so that no
// use of them moves before it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&a)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]),
                 "+r"(a[23]), "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]),
                 "+r"(a[30]), "+r"(a[31]));
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&a)[32], uint32_t (&b)[32]) {
  tmem_ld_wait_for(a);
  tmem_ld_wait_for(b);
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The thread of a warp that issues the matrix instructions. They take their operands from
// uniform registers: with a lane number as the condition every operand is moved there one by
// one (100 clocks an instruction, measured, against the 64 that it runs).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Shared-memory descriptors in the 128-byte swizzle with 8-row groups 1024 bytes apart: the
// high word is the same for all, the low one holds the address and the leading byte offset.
constexpr uint32_t PT_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return (addr >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool add,
                                       uint32_t hi = PT_DESC_HI) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(PT_DESC_HI), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// 2^y of a pair on the FMA units: y = n + f with n whole and f in [-1/2, 1/2] (adding and
// subtracting 1.5 * 2^23 rounds; 127 more leaves 2^n's exponent in the low bits), a polynomial for
// 2^f, times 2^n. The polynomial has degree 5 and the constant term 1, so that 2^n is exact; the
// others are the minimax ones for the relative error, found by linear programming on a grid and,
// rounded to fp32, among their neighbours: 9.6e-8 off as written, 1.6e-7 with the roundings of its
// five steps. Arguments below -125 count as -125, minus infinity too; NaN stays NaN.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t exp2_pair(uint64_t y) {
  float y0, y1;
  unpack2(y, &y0, &y1);
  y = pack2(max_or_nan(y0, -125.0f), max_or_nan(y1, -125.0f));
  const uint64_t magic = pack2(12583039.0f, 12583039.0f);
  const uint64_t t = add2(y, magic);
  const uint64_t f = add2(y, fma2(t, pack2(-1.0f, -1.0f), magic));
  uint64_t p = fma2(f, pack2(1.326469006e-03f, 1.326469006e-03f), pack2(9.671482258e-03f, 9.671482258e-03f));
  p = fma2(f, p, pack2(5.550719425e-02f, 5.550719425e-02f));
  p = fma2(f, p, pack2(2.402224392e-01f, 2.402224392e-01f));
  p = fma2(f, p, pack2(6.931470037e-01f, 6.931470037e-01f));
  p = fma2(f, p, pack2(1.000000000e+00f, 1.000000000e+00f));
  float t0, t1;
  unpack2(t, &t0, &t1);
  return mul2(p, pack2(__int_as_float(__float_as_int(t0) << 23), __int_as_float(__float_as_int(t1) << 23)));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Issues the boxes of 128 keys [j0, j0 + 128) of a pool: lanes 0 .. 2 * (128 / box) - 1 hold
// one box each; `row` is the lane's row in the pool (key_row).
__device__ __forceinline__ void load_keys(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int box,
                                          int row, int lane) {
  const int n = PT_KEYS / box;
  if (lane < 2 * n) {
    const int half = lane >= n, i = lane - half * n;
    tma_load_2d(dst + half * PT_HALF + i * box * 128, map, bar, 64 * half, row);
  }
}

// Zeroes rows [0, lo) and [hi, 128) of a block: two rows a turn, 16 lanes each.
__device__ __forceinline__ void hide_values(uint8_t* block, int lo, int hi, int lane) {
  uint8_t* at = block + ((lane >> 3) & 1) * PT_HALF + (lane >> 4) * 128 + (lane & 7) * 16;
  const int up = max(hi, 0) + (lane >> 4);
#pragma unroll 4
  for (int r = lane >> 4; r < lo; r += 2)
    *reinterpret_cast<uint4*>(at + (r & ~1) * 128) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
  for (int r = up; r < PT_KEYS; r += 2)
    *reinterpret_cast<uint4*>(at + (r - (lane >> 4)) * 128) = make_uint4(0u, 0u, 0u, 0u);
}

// Row of the pools at which this lane's box of block j0 starts. Boxes without a key of
// [lo, hi) and entries out of range start behind the pool: the copy fills them with zeros.
__device__ __forceinline__ int key_row(const PagedBatch& p, int b, int g, int j0, int box, int lo,
                                       int hi, int lane) {
  const int n = PT_KEYS / box;
  const int none = p.num_pages * p.Hkv * p.page;
  if (lane >= 2 * n) return none;
  const int j = j0 + (lane % n) * box;
  if (j >= hi || j + box <= lo) return none;
  const int pg = page_of(p, b, j);
  return pg < 0 ? none : (pg * p.Hkv + g) * p.page + j % p.page;
}

// Blocks [a, e), counted from key k_lo, of the CTA's nb that tokens [first, first + n) see.
__device__ __forceinline__ void tile_blocks(int first, int n, int window, int k_lo, int nb, int* a, int* e) {
  const int lo = window > 0 ? max(0, first - window + 1) : 0, hi = n > 0 ? max(0, first + n) : 0;
  *a = max(0, lo / PT_KEYS - k_lo / PT_KEYS);
  *e = max(*a, min(nb, (hi + PT_KEYS - 1) / PT_KEYS - k_lo / PT_KEYS));
}

// The sequence of tile x: tiles of T tokens, those of sequence b from q_start[b] / T + b on
// (ceil(n / T) <= floor((q + n) / T) - floor(q / T) + 1, so the ranges do not overlap).
__device__ __forceinline__ int tile_sequence(const PagedBatch& p, int x, int T, int lane) {
  int b = -1;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int i = b0 + lane;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, i < p.B && p.q_start[i] / T + i <= x));
    b += n;
    if (n < 32) break;
  }
  return b;
}

// Waits (at most 0.2 s) for the last copy into each stage, so that none lands after the CTA. Called
// where any warp gave up a wait, once all have stopped: the producer may have issued its last copy
// before that.
template <int STAGES>
__device__ __forceinline__ void drain_ring(uint64_t* full, int issued) {
  for (int s = 0; s < STAGES; ++s) {
    if (issued <= s) break;
    const int last = (issued - 1 - s) / STAGES;  // uses of stage s before the last one
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(&full[s], (uint32_t)last & 1u))
      if (globaltimer_ns() - t0 > 200000000ull) break;
  }
}

template <int NT>
__device__ __forceinline__ void attend_tiles(const CUtensorMap& tq, const CUtensorMap& tk,
                                             const CUtensorMap& tv, const TileParams& P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int SOFT = Tiles<NT>::SOFT, STAGES = Tiles<NT>::STAGES;
  uint8_t* ring = smem + NT * PT_BLOCK;
  typename Tiles<NT>::Shared& sh = *reinterpret_cast<typename Tiles<NT>::Shared*>(ring + STAGES * PT_BLOCK);
  uint64_t *full = sh.full, *empty = sh.empty, *s_full = sh.s_full, *p_full = sh.p_full;
  if (smem_u32(smem) & 1023u) {  // the swizzle counts from 1024-byte boundaries
    flag_entry(WD_PAGED | 19u);
    return;
  }
  const PagedBatch& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x % p.Hkv, rest = blockIdx.x / p.Hkv;
  const int slot = rest % P.slots;
  const int x = P.tiles - 1 - rest / P.slots;  // late tokens (the most keys) first
  const int T = NT * P.tok;
  const int b = tile_sequence(p, x, T, lane);
  if (b < 0) return;
  const SeqSpan s = seq_span(p, b);
  const int t0 = (x - (s.q0 / T + b)) * T;  // first token of the tile in its sequence
  if (t0 < 0 || t0 >= s.n || s.n * p.G <= P.skip_rows) return;
  const int n_tok = min(T, s.n - t0), p0 = s.kv - s.n + t0;  // tokens, position of the first
  const int two = NT == 2 && n_tok > P.tok;
  const int hi = p0 + n_tok, lo = P.window > 0 ? max(0, p0 - P.window + 1) : 0;
  const bool single = P.slots == 1;
  const int c0 = (lo / P.chunk + slot) * P.chunk;
  const int k_lo = max(lo & ~(PT_KEYS - 1), c0), k_hi = min(hi, c0 + P.chunk);
  const int nb = k_hi > k_lo ? (k_hi - k_lo + PT_KEYS - 1) / PT_KEYS : 0;
  if (nb == 0 && !(single || (slot == 0 && hi <= lo))) return;  // the merge skips it
  int a0, a1, e0, e1;  // blocks that tiles 0 and 1 see
  tile_blocks(p0, min(P.tok, n_tok), P.window, k_lo, nb, &a0, &e0);
  tile_blocks(p0 + P.tok, n_tok - P.tok, P.window, k_lo, nb, &a1, &e1);

  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&sh.o_full[i], 1);
    }
    for (int i = 0; i < 2 * NT; ++i) mbar_init(&p_full[i], 4);
    fence_barrier_init();
  }
  if (warp == SOFT + 1) {
    tmem_alloc(&sh.tmem, 256 * NT);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // S / P of tile t at column 128 t, O at 128 (NT + t)
  volatile int* abort_flag = &sh.abort;
  // NT = 2: 168 registers a thread at launch, 8 warps take 208, 4 keep 88; NT = 1: 128, 4 take 208,
  // 4 keep 48 (the sums are the same)
  if (warp >= SOFT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Tiles<NT>::LESS));
    if (warp == SOFT) {
      // ------------------------------------------------------------------ producer
      int issued = 0;
      if (nb > 0) {
        const int q_bytes = P.tok * p.G * 128;  // of one 64-dim half of a tile
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(q_bytes * (two ? 4 : 2)));
          for (int i = 0; i < (two ? 4 : 2); ++i)
            tma_load_3d(smem + (i >> 1) * PT_BLOCK + (i & 1) * PT_HALF, &tq, &sh.q_full, 64 * (i & 1),
                        g * p.G, s.q0 + t0 + (i >> 1) * P.tok);
        }
        bool ok = true;
        int next = key_row(p, b, g, k_lo, P.box, lo, hi, lane);
        for (int i = 0; i < nb && ok; ++i) {
          const int row = next;  // looked up a block ahead: the page table answers in 0.5 us
          if (i + 1 < nb) next = key_row(p, b, g, k_lo + (i + 1) * PT_KEYS, P.box, lo, hi, lane);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int st = issued % STAGES;
            if (issued >= STAGES)
              ok = warp_wait(&empty[st], (uint32_t)(issued / STAGES - 1) & 1u, abort_flag, WD_PAGED | 3u);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[st], PT_BLOCK);
            __syncwarp();
            load_keys(ring + st * PT_BLOCK, v ? &tv : &tk, &full[st], P.box, row, lane);
            ++issued;
          }
        }
      }
      if (lane == 0) sh.issued = issued;
    } else if (warp == SOFT + 1) {
      // ------------------------------------------------------------------ MMA: one warp for both
      // tiles, so that their products run one after the other and not interleaved
      constexpr uint32_t id_s = idesc_bf16_f32(PT_TILE, PT_KEYS, false);
      constexpr uint32_t id_o = idesc_bf16_f32(PT_TILE, FA_HEAD_DIM, true);
      const uint32_t q_lo = desc_lo(smem_u32(smem), 16), kb_lo = desc_lo(smem_u32(ring), 16);
      const uint32_t v_lo = desc_lo(smem_u32(ring), PT_HALF);
      auto scores = [&](int t, int st) {
        const uint32_t qa = q_lo + t * (PT_BLOCK >> 4), kb = kb_lo + st * (PT_BLOCK >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * PT_HALF + (k & 3) * 32) >> 4;
          mma_ss(tmem + 128 * t, qa + off, kb + off, id_s, k > 0);
        }
        mma_commit(&s_full[t]);
      };
      auto loaded = [&](int c) {  // use c of the ring
        return warp_wait(&full[c % STAGES], (uint32_t)(c / STAGES) & 1u, abort_flag, WD_PAGED | 5u);
      };
      bool ok = nb > 0 && warp_wait(&sh.q_full, 0, abort_flag, WD_PAGED | 4u) && loaded(0);
      if (ok && elect_one()) {
        if (a0 == 0 && e0 > 0) scores(0, 0);
        if (NT == 2 && a1 == 0 && e1 > 0) scores(1, 0);
        mma_commit(&empty[0]);
      }
      for (int i = 0; i < nb; ++i) {
        const int sv = (2 * i + 1) % STAGES, sk = (2 * i + 2) % STAGES;
        const bool more = i + 1 < nb;
        // a wait that finds its phase complete still takes some 100 clocks: these come while the
        // tensor core has work
        ok = ok && loaded(2 * i + 1) && (NT == 1 || !more || loaded(2 * i + 2));
        const int j0 = k_lo + i * PT_KEYS;
        if (ok && (j0 < lo || j0 + PT_KEYS > hi)) {
          // values of keys outside [lo, hi) may be anything, NaN too: they count as zero
          hide_values(ring + sv * PT_BLOCK, lo - j0, hi - j0, lane);
          fence_proxy_async_smem();
        }
        for (int t = 0; t < NT && ok; ++t) {
          const int a = t ? a1 : a0, e = t ? e1 : e0;
          if (a <= i && i < e) {
            // the weights of keys 0-63 and 64-127 of the block: the first product runs while the
            // others are still computed
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = warp_wait(&p_full[2 * t + h], (uint32_t)(i - a) & 1u, abort_flag, WD_PAGED | 6u);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)
                  mma_ts(tmem + 128 * (NT + t), tmem + 128 * t + 8 * k, v_lo + (sv * PT_BLOCK + 2048 * k) / 16,
                         id_o, i > a || k > 0);
                if (h == 1 && NT == 2) {
                  if (more && i + 1 < e) scores(t, sk);
                  if (i + 1 == e) mma_commit(&sh.o_full[t]);
                }
              }
            }
          } else if (NT == 2 && more && i + 1 == a && a < e) {
            if (elect_one()) scores(t, sk);
          }
        }
        if (NT == 1) {
          // two stages: the next values may load once this product is done, the keys before them
          // are waited for last
          if (ok && elect_one()) {
            mma_commit(&empty[sv]);
            if (i + 1 == e0) mma_commit(&sh.o_full[0]);
          }
          ok = ok && (!more || loaded(2 * i + 2));
        }
        if (!ok) break;
        if (elect_one()) {
          if (NT == 2) mma_commit(&empty[sv]);
          if (NT == 1 && more && i + 1 >= a0 && i + 1 < e0) scores(0, sk);
          if (more) mma_commit(&empty[sk]);
        }
      }
      if (nb > 0 && !ok && elect_one()) {
        // tensor memory is released only after every MMA of this CTA has completed
        mma_commit(&sh.drained);
        const unsigned long long w0 = globaltimer_ns();
        while (!mbar_try_wait(&sh.drained, 0))
          if (globaltimer_ns() - w0 > 200000000ull) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Tiles<NT>::MORE));
    if ((warp >> 2) <= two) {
      // ------------------------------------------------------------------ softmax, one row a thread
      const int t = warp >> 2, row = threadIdx.x & 127;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + 128 * t + lanes, to = ts + 128 * NT;
      const int tok = t * P.tok + row / p.G;
      const bool valid = row < P.tok * p.G && tok < n_tok;
      const int pos = valid ? p0 + tok : -1;
      // positions of the warp's rows, blocks of the tile
      const int pw_first = p0 + t * P.tok + (row & ~31) / p.G;
      const int pw_last = p0 + min(t * P.tok + min((row | 31) / p.G, P.tok - 1), n_tok - 1);
      const int a = t ? a1 : a0, e_ = t ? e1 : e0;
      const float c = P.scale_log2;
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int i = a; i < e_; ++i) {
        ok = warp_wait(&s_full[t], (uint32_t)(i - a) & 1u, abort_flag, WD_PAGED | 7u);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[4][32];
        const int j0 = k_lo + i * PT_KEYS;
        tmem_ld_32x32b_x32(ts, sr[0]);
        tmem_ld_32x32b_x32(ts + 32, sr[1]);
        tmem_ld_wait_for(sr[0], sr[1]);
        tmem_ld_32x32b_x32(ts + 64, sr[2]);
        tmem_ld_32x32b_x32(ts + 96, sr[3]);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (v == 2) tmem_ld_wait_for(sr[2], sr[3]);
          // chunks of 32 keys that some row of the warp does not see
          const int j = j0 + 32 * v;
          if (j + 31 > pw_first || (P.window > 0 && j <= pw_last - P.window)) {
            const int up = pos - j, down = P.window > 0 ? up - P.window : -1;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e > up || e <= down) sr[v][e] = 0xFF800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(sr[v][e]), __uint_as_float(sr[v][e + 1]));
        }
        const float top = c * max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        if (i == a) {
          m = top;
        } else {
          const bool behind = valid && top > m + PT_SLACK;
          if (__any_sync(0xFFFFFFFFu, behind)) {
            const float m_new = behind ? top : m;
            const float f = behind ? exp2_approx(m - m_new) : 1.0f;
            m = m_new;
            l *= f;
#pragma unroll 1
            for (int v = 0; v < 4; ++v) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + 32 * v, o);
              tmem_ld_wait_for(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f * __uint_as_float(o[e]));
              tmem_st_32x32b_x32(to + 32 * v, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        const uint64_t c2 = pack2(c, c), b2 = pack2(-base, -base);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t* q = &sr[2 * h + (e >> 4)][2 * (e & 15)];
            const uint64_t y = fma2(pack2(__uint_as_float(q[0]), __uint_as_float(q[1])), c2, b2);
            float y0, y1;
            unpack2(y, &y0, &y1);
            y0 = exp2_approx(y0);
            y1 = exp2_approx(y1);
            sum[e & 1] = add2(sum[e & 1], pack2(y0, y1));
            w[e] = pack_bf16(y0, y1);
          }
          tmem_st_32x32b_x32(ts + 32 * h, w);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
        }
        float l0, l1;
        unpack2(add2(sum[0], sum[1]), &l0, &l1);
        l += l0 + l1;
      }
      if (e_ > a && ok) {
        ok = warp_wait(&sh.o_full[t], 0, abort_flag, WD_PAGED | 8u);
        tc_fence_after();
      }
      if (ok) {
        const long long token = s.q0 + t0 + tok;
        const int h = g * p.G + row % p.G;
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        const long long rec = (token * p.Hq + h) * P.slots + slot;
#pragma unroll 1
        for (int v = 0; v < 4; ++v) {
          uint32_t o[32];
          if (e_ > a) {
            tmem_ld_32x32b_x32(to + 32 * v, o);
            tmem_ld_wait_for(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!valid) continue;
          const int d = 32 * v;
          if (single) {
            uint4* dst = reinterpret_cast<uint4*>(P.out + token * P.out_stride + h * FA_HEAD_DIM + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w[u] = pack_bf16(inv * __uint_as_float(o[8 * e + 2 * u]),
                                 inv * __uint_as_float(o[8 * e + 2 * u + 1]));
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(P.part_o + rec * FA_HEAD_DIM + d);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (valid) {
          if (!single) P.part_ml[rec] = make_float2(m, l);
          else if (P.lse) P.lse[token * p.Hq + h] = 0.693147180559945309f * (m + log2f(l));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == SOFT && lane == 0 && *abort_flag) {
    drain_ring<STAGES>(full, sh.issued);
    drain_ring<1>(&sh.q_full, 1);
  }
  if (warp == SOFT + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256 * NT);
  }
}

template <int NT>
__global__ void __launch_bounds__(Tiles<NT>::THREADS, 3 - NT)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ TileParams P) {
  allow_next_kernel();
  attend_tiles<NT>(tq, tk, tv, P);
  wait_earlier_kernel();  // the rows of short sequences: this kernel needs none of them
}

// Weights that keys gather: w_j += sum_rows exp2(c s_rj - log2 e lse_r). An item is 256 keys (two
// tiles) of a KV head, against which the query rows that see them stream in blocks of 128, as
// S^T = K Q^T: a thread owns a key (a lane of tensor memory) and sums along half its columns, so
// that nothing is reduced across threads but the two halves and a key's sum is taken in one order.
// Scores are double-buffered: the tensor core writes one buffer while the other is summed.
//   -lse / scale joins the product as 16 more dims: the keys hold 1, 1, 1, 0, ..., a row its
// value in three bf16 parts (exact to 2^-24 of it, as an fp32 product would be). Read from shared
// memory by every thread for every column it took as many cycles as the exponentials.
//   Bound: 2 * 144 flops a (row, key) against one exp2: 576 and 1024 clocks for a 128 x 128 tile.
constexpr int PV_SOFT = 16;                   // warps that sum; 4 more as above
constexpr int PV_THREADS = (PV_SOFT + 4) * 32;
constexpr int PV_REGS = PV_SOFT * 32 * 104 + 4 * 32 * 64;
constexpr int PV_STAGES = 4;
constexpr int PV_KEYS = 2 * PT_TILE;
// 16 more dims of 128 rows, unswizzled: 8 rows x 8 dims contiguous, 16 such, then the other dims
constexpr int PV_EXTRA = PT_TILE * 32;
constexpr uint32_t PV_EXTRA_HI = (128u >> 4) | (1u << 14);
constexpr int PV_SMEM = (2 + PV_STAGES) * PT_BLOCK + (1 + PV_STAGES) * PV_EXTRA + 1024;

struct WeightParams {
  PagedBatch p;
  int window, tok, box, skip_rows;
  int key_bits;  // log2 of the keys of an item: 8, or 7 (one tile) where that leaves SMs idle
  float scale_log2, inv_scale;
  const float* lse;
  float* weights;
  long long weights_ld;
};

// The items of a batch in order of sequence, keys and KV head: the first keys, which most rows
// see, first. Only sequences of more than skip_rows rows have any, and CTA i of n takes items
// i, 2n - 1 - i, 2n + i, ..., so that each gets early and late ones. With a CTA for every item that
// the shape allows, 64 single tokens and a chunk of 512 over 4096 keys each took 168 us, 46 of them
// in empty CTAs (now 122), and 32 heads of 6000 tokens 222 (now 181: the next item's keys load
// while the last block is summed). Every warp finds the items by itself, 32 sequences at a time.
struct WeightItems {
  int round = 0, b0 = 0, base = 0;    // first sequence of the group, items before it
  int b, g, q0, n, p0, j0, lo, hi;    // sequence, head, new tokens and their position, keys
  int two, blk0, nb;                  // second tile used, blocks of P.tok tokens that see the keys

  __device__ bool next(const WeightParams& P, int lane) {
    const PagedBatch& p = P.p;
    const int ctas = (int)gridDim.x;
    const int index = round * ctas + (round & 1 ? ctas - 1 - (int)blockIdx.x : (int)blockIdx.x);
    ++round;
    for (; b0 < p.B; b0 += 32) {
      SeqSpan s = {0, 0, 0};
      int first = 0, count = 0;
      if (b0 + lane < p.B) s = seq_span(p, b0 + lane);
      if (s.n * p.G > P.skip_rows && s.kv > 0) {
        if (P.window > 0) first = max(0, s.kv - s.n - P.window + 1);
        count = (((s.kv - 1) >> P.key_bits) - (first >> P.key_bits) + 1) * p.Hkv;
      }
      int end = count;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int below = __shfl_up_sync(0xFFFFFFFFu, end, d);
        if (lane >= d) end += below;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, base + end > index);
      if (past == 0u) {
        base += __shfl_sync(0xFFFFFFFFu, end, 31);
        continue;
      }
      const int l = __ffs(past) - 1;
      const int k = index - base - __shfl_sync(0xFFFFFFFFu, end - count, l);
      b = b0 + l;
      q0 = __shfl_sync(0xFFFFFFFFu, s.q0, l);
      n = __shfl_sync(0xFFFFFFFFu, s.n, l);
      hi = __shfl_sync(0xFFFFFFFFu, s.kv, l);
      lo = __shfl_sync(0xFFFFFFFFu, first, l);
      p0 = hi - n;
      g = k % p.Hkv;
      j0 = ((lo >> P.key_bits) + k / p.Hkv) << P.key_bits;
      two = P.key_bits > 7 && j0 + PT_TILE < hi;
      const int i0 = max(0, j0 - p0);
      const int i1 = P.window > 0 ? min(n, min(j0 + (1 << P.key_bits), hi) - 1 + P.window - p0) : n;
      blk0 = i0 / P.tok;
      nb = (i1 + P.tok - 1) / P.tok - blk0;
      return true;
    }
    return false;
  }
};

// Joins the PV_SOFT warps that sum; true if `flag` was set in any.
__device__ __forceinline__ bool sums_meet(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 512, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)flag)
      : "memory");
  return any != 0;
}

__global__ void __launch_bounds__(PV_THREADS, 1)
    paged_weights_tile_kernel(const __grid_constant__ CUtensorMap tq,
                              const __grid_constant__ CUtensorMap tk,
                              const __grid_constant__ WeightParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * PT_BLOCK;
  uint8_t* ones = ring + PV_STAGES * PT_BLOCK;  // the keys' extra dims
  uint8_t* extra = ones + PV_EXTRA;             // [stage] the rows'
  __shared__ uint64_t full[PV_STAGES], empty[PV_STAGES], k_full, k_empty, s_full[4], s_empty[4], drained;
  __shared__ float half_sum[2][PV_KEYS];
  __shared__ uint32_t tmem_ptr;
  __shared__ int abort_word, issued[2];  // copies of query blocks, of items' keys
  const PagedBatch& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  allow_next_kernel();

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < PV_STAGES; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&k_full, 1);
    mbar_init(&k_empty, 1);
    mbar_init(&drained, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 8);
    }
    fence_barrier_init();
  }
  if (warp == PV_SOFT + 1) {
    tmem_alloc(&tmem_ptr, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  // rows of the blocks that no box fills (128 is not a multiple of G) are zero
  for (int w = threadIdx.x; w < PV_STAGES * 2 * (PT_TILE - P.tok * p.G) * 8; w += PV_THREADS) {
    const int pad = PT_TILE - P.tok * p.G, r = PT_TILE - 1 - w / 8 % pad, h = w / 8 / pad;
    *reinterpret_cast<uint4*>(ring + h * PT_HALF + r * 128 + (w & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  for (int w = threadIdx.x; w < (1 + PV_STAGES) * PV_EXTRA / 16; w += PV_THREADS)
    reinterpret_cast<uint4*>(ones)[w] =
        w < PT_TILE ? make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_ptr;  // scores of tile t, buffer u at columns 128 (2 t + u)
  volatile int* abort_flag = &abort_word;

  if (warp >= PV_SOFT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    WeightItems w;
    int it = 0, c = 0;  // items, blocks so far
    bool ok = true;
    if (warp == PV_SOFT) {
      // ---------------------------------------------------------------- producer
      int k_issued = 0;
      for (; ok && w.next(P, lane); ++it) {
        int row[2];
        for (int t = 0; t < 2; ++t) row[t] = key_row(p, w.b, w.g, w.j0 + t * PT_TILE, P.box, w.lo, w.hi, lane);
        if (it > 0) ok = warp_wait(&k_empty, (uint32_t)(it - 1) & 1u, abort_flag, WD_PAGED | 14u);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&k_full, PT_BLOCK * (1 + w.two));
        __syncwarp();
        load_keys(smem, &tk, &k_full, P.box, row[0], lane);
        if (w.two) load_keys(smem + PT_BLOCK, &tk, &k_full, P.box, row[1], lane);
        ++k_issued;
        for (int i = 0; i < w.nb; ++i, ++c) {
          const int st = c % PV_STAGES;
          if (c >= PV_STAGES)
            ok = warp_wait(&empty[st], (uint32_t)(c / PV_STAGES - 1) & 1u, abort_flag, WD_PAGED | 9u);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[st], (uint32_t)(P.tok * p.G * 256));
            for (int h = 0; h < 2; ++h)
              tma_load_3d(ring + st * PT_BLOCK + h * PT_HALF, &tq, &full[st], 64 * h, w.g * p.G,
                          w.q0 + (w.blk0 + i) * P.tok);
          }
        }
      }
      if (lane == 0) {
        issued[0] = c;
        issued[1] = k_issued;
      }
    } else if (warp == PV_SOFT + 1) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t id = idesc_bf16_f32(PT_TILE, PT_TILE, false);
      const uint32_t a_lo = desc_lo(smem_u32(smem), 16), b_lo = desc_lo(smem_u32(ring), 16);
      const uint32_t one_lo = desc_lo(smem_u32(ones), PV_EXTRA / 2), x_lo = desc_lo(smem_u32(extra), PV_EXTRA / 2);
      int used[2] = {0, 0};  // score buffers of each tile so far
      for (; ok && w.next(P, lane); ++it) {
        ok = warp_wait(&k_full, (uint32_t)it & 1u, abort_flag, WD_PAGED | 10u);
        for (int i = 0; i < w.nb; ++i, ++c) {
          const int st = c % PV_STAGES;
          ok = ok && warp_wait(&full[st], (uint32_t)(c / PV_STAGES) & 1u, abort_flag, WD_PAGED | 11u);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t > w.two) break;
            const int u = used[t] & 1;
            if (used[t] >= 2)
              ok = ok && warp_wait(&s_empty[2 * t + u], (uint32_t)(used[t] / 2 - 1) & 1u, abort_flag, WD_PAGED | 12u);
            if (!ok) break;
            ++used[t];
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t off = ((k >> 2) * PT_HALF + (k & 3) * 32) >> 4;
                mma_ss(tmem + 128 * (2 * t + u), a_lo + t * (PT_BLOCK >> 4) + off,
                       b_lo + st * (PT_BLOCK >> 4) + off, id, k > 0);
              }
              mma_ss(tmem + 128 * (2 * t + u), one_lo, x_lo + st * (PV_EXTRA >> 4), id, true, PV_EXTRA_HI);
              mma_commit(&s_full[2 * t + u]);
              if (t == w.two) {
                mma_commit(&empty[st]);
                if (i + 1 == w.nb) mma_commit(&k_empty);
              }
            }
          }
          __syncwarp();
          if (!ok) break;
        }
      }
      if (!ok && elect_one()) {
        mma_commit(&drained);
        const unsigned long long w0 = globaltimer_ns();
        while (!mbar_try_wait(&drained, 0))
          if (globaltimer_ns() - w0 > 200000000ull) break;
      }
    } else if (warp == PV_SOFT + 2) {
      // ---------------------------------------------------------------- log-sum-exp of the rows,
      // loaded a block ahead
      for (; ok && w.next(P, lane); ++it) {
        auto load = [&](int i, float (&e)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = lane + 32 * x, tok = (w.blk0 + i) * P.tok + row / p.G;
            e[x] = -INFINITY;
            if (i < w.nb && row < P.tok * p.G && tok < w.n)
              e[x] = P.lse[(long long)(w.q0 + tok) * p.Hq + w.g * p.G + row % p.G];
          }
        };
        float next[4];
        load(0, next);
        for (int i = 0; i < w.nb; ++i, ++c) {
          const int st = c % PV_STAGES;
          uint4 e[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            // columns without a row, and rows that see no key, add nothing
            const float v = next[x] == -INFINITY ? -3e38f : -next[x] * P.inv_scale;
            const __nv_bfloat16 a = __float2bfloat16_rn(v);
            const float r = v - __bfloat162float(a);
            const __nv_bfloat16 b = __float2bfloat16_rn(r);
            e[x] = make_uint4(__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16,
                              __bfloat16_as_ushort(__float2bfloat16_rn(r - __bfloat162float(b))), 0u, 0u);
          }
          load(i + 1, next);
          if (c >= PV_STAGES)
            ok = warp_wait(&empty[st], (uint32_t)(c / PV_STAGES - 1) & 1u, abort_flag, WD_PAGED | 13u);
          if (!ok) break;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            reinterpret_cast<uint4*>(extra + st * PV_EXTRA)[lane + 32 * x] = e[x];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------------------------ sums: two threads a key,
    // each with 64 columns of a block
    const int t = warp >> 3, half = (warp >> 2) & 1, row = 32 * (warp & 3) + lane;
    const uint32_t ts = tmem + 256 * t + 64 * half + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t c2 = pack2(P.scale_log2, P.scale_log2);
    WeightItems w;
    int used = 0;  // score buffers so far
    for (int it = 0; w.next(P, lane); ++it) {
      const int jt = w.j0 + t * PT_TILE, j = jt + row;
      bool ok = true;
      uint64_t sum[2] = {0ull, 0ull};
      for (int i = 0; t <= w.two && i < w.nb; ++i, ++used) {
        const int u = used & 1;
        ok = warp_wait(&s_full[2 * t + u], (uint32_t)(used / 2) & 1u, abort_flag, WD_PAGED | 15u);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld_32x32b_x32(ts + 128 * u, sr[0]);
        tmem_ld_32x32b_x32(ts + 128 * u + 32, sr[1]);
        tmem_ld_wait_for(sr[0], sr[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[2 * t + u]);
        // columns [first, last) see the key: tokens from position j on, below j + window
        const int tok0 = (w.blk0 + i) * P.tok, pb = w.p0 + tok0, left = w.n - tok0;
        const bool edge = jt + PT_TILE - 1 > pb || left < P.tok ||
                          (P.window > 0 && pb + P.tok > jt + P.window);
        auto add = [&](auto plain) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t* q = &sr[e >> 4][2 * (e & 15)];
            const uint64_t y = mul2(pack2(__uint_as_float(q[0]), __uint_as_float(q[1])), c2);
            if (decltype(plain)::value && e % 4 == 3) {
              sum[e & 1] = add2(sum[e & 1], exp2_pair(y));
            } else {
              float a0, a1;
              unpack2(y, &a0, &a1);
              sum[e & 1] = add2(sum[e & 1], pack2(exp2_approx(a0), exp2_approx(a1)));
            }
          }
        };
        if (edge) {
          const int first = min(max(j - pb, 0), P.tok) * p.G - 64 * half;
          int end = min(left, P.tok);
          if (P.window > 0) end = min(end, max(0, j + P.window - pb));
          const int last = end * p.G - 64 * half;
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * v + e < first || 32 * v + e >= last) sr[v][e] = 0xFF800000u;
          add(std::false_type());
        } else {
          add(std::true_type());
        }
      }
      float a0, a1;
      unpack2(add2(sum[0], sum[1]), &a0, &a1);
      float* other = &half_sum[it & 1][t * PT_TILE + row];  // the item after next writes it again
      if (half) *other = a0 + a1;
      if (sums_meet(!ok)) break;
      if (!half && t <= w.two && j >= w.lo && j < w.hi)
        P.weights[((long long)w.b * p.Hkv + w.g) * P.weights_ld + j] += a0 + a1 + *other;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == PV_SOFT && lane == 0 && *abort_flag) {
    drain_ring<PV_STAGES>(full, issued[0]);
    drain_ring<1>(&k_full, issued[1]);
  }
  if (warp == PV_SOFT + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_earlier_kernel();  // the keys of short sequences: this kernel needs none of them
}

FA_WATCHDOG_READER(read_watchdog_paged_tc)

// ------------------------------------------------------------------------- host side
bool encode_queries(CUtensorMap* map, const void* q, const fa_paged_shape& s, int64_t stride, int tok) {
  const auto encode = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(tensor_map_encoder());
  if (!encode) return false;
  const int G = s.Hq / s.Hkv;
  cuuint64_t dims[3] = {FA_HEAD_DIM, (cuuint64_t)s.Hq, (cuuint64_t)s.total_q};
  cuuint64_t strides[2] = {FA_HEAD_DIM * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tok};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static cudaError_t prepare_kernel(const void* fn, int smem, int threads, int regs, const char** why) {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, fn);
  if (e != cudaSuccess) return e;
  if (at.numRegs * threads < regs) {
    *why = "the kernel was built with fewer registers than its warps share out";
    return cudaErrorInvalidConfiguration;
  }
  return raise_smem_limit(fn, smem);
}

// Key rows of a TMA box: the largest power of two, at most a block, that divides a page (so
// that no box crosses its end); a whole block where a sequence has one page.
int key_box(const fa_paged_shape& s) {
  if (s.max_kv <= s.page_size) return PT_KEYS;
  int box = 16;
  while (box < PT_KEYS && s.page_size % (2 * box) == 0) box *= 2;
  return box;
}

// Tiles are used where some sequence may have more rows than one 16-row tile and the heads of
// a token fit a 128-row tile. CTAs of one tile, two an SM, where a tile sees at most 10 blocks, of
// which its start and end would take 4, or no sequence fills more than one; else CTAs of two, which
// read each block once. Back to back, one tile a CTA and two: 6 chunks with a window of 1024 96 and 97
// us, 1000 tokens over themselves 24 and 25, 32 prompts of 128 40 and 48, 64 x 30 over 4000 keys 169 and
// 251; 4 x 300 over 2000 keys 71 and 71, 1000 over 2000 41 and 40, 4096 over 16384 1053 and 924.
//   Keys (of the window, where there is one) are split when the tiles of the batch leave SMs idle:
// into chunks of equal length, multiples of a block and at least 2, that fill one wave. More waves
// do not pay: the parts are written and read again (600 tokens over 4000 keys, 80 pairs of tiles:
// 66 us whole, 76 in 3 chunks; 4096 over 16384: 829 and 913 in 2).
cudaError_t tile_plan(const fa_paged_shape& s, int window, TilePlan* t) {
  memset(t, 0, sizeof(*t));
  const int G = s.Hq / s.Hkv;
  const long long max_q = s.max_q < s.total_q ? s.max_q : s.total_q;
  if (G > PT_TILE || max_q * G <= 16) return cudaSuccess;
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  t->tok = PT_TILE / G;
  t->box = key_box(s);
  long long keys = s.max_kv;  // that a tile may see
  if (window > 0 && (long long)window + t->tok < keys) keys = (long long)window + t->tok;
  t->pair = keys <= 1280 || max_q <= t->tok ? 1 : 2;
  const int T = t->pair * t->tok;
  t->tiles = s.total_q / T + s.B;
  const long long units = (long long)((s.total_q + T - 1) / T) * s.Hkv, ctas = (3 - t->pair) * sms;
  const long long want = units < ctas ? ctas / units : 1;
  long long c = want > 1 ? (keys + want - 1) / want : s.max_kv;
  c = (c + PT_KEYS - 1) / PT_KEYS * PT_KEYS;
  t->chunk = (int)(c < 2 * PT_KEYS ? 2 * PT_KEYS : c);
  t->slots = chunk_slots(s, window, t->chunk, T);
  t->records = t->slots == 1 ? 0 : (size_t)s.total_q * s.Hq * t->slots;
  return cudaSuccess;
}

cudaError_t launch_tiles(const fa_paged_shape& s, const fa_paged_cache& c, const TilePlan& t,
                         const void* q, int64_t q_stride, float scale, int window, void* out,
                         int64_t out_stride, float* lse, float* part_o, float2* part_ml,
                         int skip_rows, cudaStream_t stream, const char** why) {
  TileParams P;
  memset(&P, 0, sizeof(P));
  P.p = paged_batch(s, c);
  P.window = window;
  P.chunk = t.chunk;
  P.slots = t.slots;
  P.tiles = t.tiles;
  P.tok = t.tok;
  P.box = t.box;
  P.skip_rows = skip_rows;
  P.scale_log2 = scale * 1.44269504088896341f;
  P.out = static_cast<__nv_bfloat16*>(out);
  P.out_stride = out_stride;
  P.lse = lse;
  P.part_o = part_o;
  P.part_ml = part_ml;
  CUtensorMap tq, tk, tv;
  if (!encode_pool(&tk, c.K, s, t.box) || !encode_pool(&tv, c.V, s, t.box)) {
    *why = "cuTensorMapEncodeTiled rejected the pools";
    return cudaErrorInvalidValue;
  }
  if (!encode_queries(&tq, q, s, q_stride, t.tok)) {
    *why = "cuTensorMapEncodeTiled rejected q";
    return cudaErrorInvalidValue;
  }
  auto launch = [&](auto kernel, auto tiles) {
    using Config = decltype(tiles);
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), Config::SMEM, Config::THREADS,
                                         Config::REGS, why);
    if (e != cudaSuccess) return e;
    const long long ctas = (long long)t.tiles * t.slots * s.Hkv;
    return launch_overlapped(kernel, dim3((unsigned)ctas), Config::THREADS, Config::SMEM, stream, tq, tk, tv, P);
  };
  return t.pair == 2 ? launch(paged_tile_kernel<2>, Tiles<2>()) : launch(paged_tile_kernel<1>, Tiles<1>());
}

cudaError_t launch_weight_tiles(const fa_paged_shape& s, const fa_paged_cache& c, const void* q,
                                int64_t q_stride, float scale, int window, const float* lse,
                                float* weights, int64_t weights_ld, int skip_rows,
                                cudaStream_t stream, const char** why) {
  WeightParams P;
  memset(&P, 0, sizeof(P));
  P.p = paged_batch(s, c);
  P.window = window;
  P.tok = PT_TILE / P.p.G;
  P.box = key_box(s);
  P.skip_rows = skip_rows;
  P.scale_log2 = scale * 1.44269504088896341f;
  P.inv_scale = 1.0f / scale;
  P.lse = lse;
  P.weights = weights;
  P.weights_ld = weights_ld;
  CUtensorMap tq, tk;
  if (!encode_pool(&tk, c.K, s, P.box) || !encode_queries(&tq, q, s, q_stride, P.tok)) {
    *why = "cuTensorMapEncodeTiled rejected the pool or q";
    return cudaErrorInvalidValue;
  }
  const void* fn = reinterpret_cast<const void*>(paged_weights_tile_kernel);
  cudaError_t e = prepare_kernel(fn, PV_SMEM, PV_THREADS, PV_REGS, why);
  if (e != cudaSuccess) return e;
  int sms = 148;
  if ((e = device_sm_count(&sms)) != cudaSuccess) return e;
  const int max_q = s.max_q < s.total_q ? s.max_q : s.total_q;
  const long long heads = (long long)s.Hkv * s.B;
  // One tile an item where two leave half of the SMs idle: more CTAs read more queries from L2, but
  // each works on half the keys (2000 tokens over 2000 keys, 8 KV heads: 88 us in 64 items, 71 in 128).
  P.key_bits = 2 * heads * chunk_slots(s, window, PV_KEYS, max_q) <= sms ? 7 : 8;
  const long long items = heads * chunk_slots(s, window, 1 << P.key_bits, max_q);
  return launch_overlapped(paged_weights_tile_kernel, dim3((unsigned)(items < sms ? items : sms)), PV_THREADS,
                           PV_SMEM, stream, tq, tk, P);
}

}  // namespace fa
