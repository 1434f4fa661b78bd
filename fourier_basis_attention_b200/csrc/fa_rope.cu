// fa_rope.cu -- rotary positions, alone and fused with the write of new tokens into pages.
//
// Pair (a, b) at position p: (a, b) -> m (a cos t - b sin t, b cos t + a sin t), t = p f.
// f / (2 pi) is held as a 64-bit fraction of a turn, whose product with an int32 position is exact
// modulo one turn in integers; sincospif takes its top 32 bits. The angle is off by what the stored
// fraction is, times the position: |p| (2^-52 f / (2 pi) + 2^-64) turns (fp64 frequency, cut), and by
// 2^-32 turns and an fp32 step (an fp32 product p * f is off by 0.03 radians at a million positions).
//
// Memory-bound: each row is read and written once. A CTA takes RT tokens: its threads first
// put the tokens' 64 (cos, sin) pairs into shared memory (one sincospif a pair and token, shared by
// all heads), then walk over (token, head, item), an item being the two 16-byte vectors
// that hold 8 (bf16) or 4 (fp32) pairs. A rot_dim whose halves are not whole vectors goes by rows
// through shared memory instead.
//   Measured (B200): 2 x 16001 x 8 fp32 rows, head-major, 44 us, 262 MB, 90% of the measured copy
// bandwidth (before its set-up overlapped the kernel before it 47, and then one token a CTA 72,
// eight 46, two or four items of a thread on their way 49 and 74: fewer warps fit). The page write
// of 5 prompts of up to 4001 tokens, 373 MB, takes 71 us with two items on their way (before two
// other steps 75, and then with one 81, with four 104, the same with the first loads ahead of the
// look-ups; its q, k and v rows lie apart, so that a warp's accesses are 128-byte pieces).
#include <math.h>
#include <string.h>

#include "fa_paged.cuh"

namespace fa {

constexpr int RP_THREADS = 256;
constexpr int RP_PAIRS = FA_HEAD_DIM / 2;
constexpr int RP_BATCH = 2;  // items of a thread on their way at once in the page write

struct RopeParams {
  int rot, interleaved, transpose;
  float magnitude;
  unsigned long long turns[RP_PAIRS];
};

// magnitude * (cos, sin) of pair i at position pos.
__device__ __forceinline__ float2 rope_cs(const RopeParams& r, int i, int pos) {
  // by a load and not as a constant: those of a warp's 32 pairs would be read one by one (2 x 8001 x
  // 8 bf16 rows: 17.2 us, 14.1 this way)
  unsigned long long turns;
  asm("ld.b64 %0, [%1];" : "=l"(turns) : "l"(r.turns + i));
  const unsigned long long phase = (unsigned long long)(long long)pos * turns;
  // nearest quarter turn, and the rest in [-1/4, 1/4] half turns: fp32 holds that to 2^-26
  const uint32_t turn = (uint32_t)(phase >> 32), quarter = (turn + 0x20000000u) >> 30;
  float s, c;
  sincospif((float)(int)(turn - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);  // * 2^-31
  if (quarter & 1u) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2u) {
    c = -c;
    s = -s;
  }
  return make_float2(r.magnitude * c, r.magnitude * (r.transpose ? -s : s));
}

template <typename T>
struct RopeVec;
template <>
struct RopeVec<float> {
  static constexpr int N = 4;
  using Raw = float4;
  __device__ static Raw raw(const float* p) { return *reinterpret_cast<const float4*>(p); }
  __device__ static void put_raw(float* p, const Raw& x) { *reinterpret_cast<float4*>(p) = x; }
  __device__ static void split(const Raw& x, float* v) {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
  __device__ static Raw join(const float* v) { return make_float4(v[0], v[1], v[2], v[3]); }
  __device__ static float get(float x) { return x; }
  __device__ static float put(float x) { return x; }
};
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int N = 8;
  using Raw = uint4;
  __device__ static Raw raw(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
  __device__ static void put_raw(__nv_bfloat16* p, const Raw& x) { *reinterpret_cast<uint4*>(p) = x; }
  __device__ static void split(const Raw& x, float* v) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static Raw join(const float* v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
  }
  __device__ static float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  __device__ static __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// Item `it` of a row: rotated pairs first, then the dims that pass, N pairs (two vectors) or two
// vectors of passing dims. Loads and stores are apart so that a thread has several items on their
// way.
template <typename T>
struct RopeItem {
  using V = RopeVec<T>;
  static constexpr int N = V::N;
  static constexpr int ITEMS = RP_PAIRS / N;  // a row
  T* y;         // row written; null: no item
  const float2* cs;  // the token's pairs
  int i, da, db;     // first pair (or half the first passing dim), the two dims
  bool turn;
  typename V::Raw a, b;

  __device__ void load(const T* x, int it, int rot, int interleaved) {
    i = it * N;
    turn = 2 * i < rot;
    da = 2 * i;
    db = 2 * i + N;
    if (turn && !interleaved) {
      da = i;
      db = rot / 2 + i;
    }
    a = V::raw(x + da);
    b = V::raw(x + db);
  }
  __device__ void store(int interleaved) const {
    if (!turn) {
      V::put_raw(y + da, a);
      V::put_raw(y + db, b);
      return;
    }
    float p[N], q[N];
    V::split(a, p);
    V::split(b, q);
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 u = cs[i + e / 2], w = cs[i + (N + e) / 2];
        const float p0 = p[e], q0 = q[e];
        p[e] = p0 * u.x - p[e + 1] * u.y;
        p[e + 1] = p[e + 1] * u.x + p0 * u.y;
        q[e] = q0 * w.x - q[e + 1] * w.y;
        q[e + 1] = q[e + 1] * w.x + q0 * w.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 u = cs[i + e];
        const float p0 = p[e];
        p[e] = p0 * u.x - q[e] * u.y;
        q[e] = q[e] * u.x + p0 * u.y;
      }
    }
    V::put_raw(y + da, V::join(p));
    V::put_raw(y + db, V::join(q));
  }
};

// A row whose pairs do not fall into whole vectors: 16 (bf16) or 32 (fp32) lanes take it through
// shared memory, read and written in vectors there and back, rotated in place a pair a lane. (2 x 8001
// x 8 rows, rot_dim 24, 62 and 100, bf16: 21, 22 and 25 us with a pair an item straight from memory,
// 12, 15 and 23 this way; fp32, 62 and 100: 37 and 39, 29 and 31.)
template <typename T>
struct RopeRow {
  using V = RopeVec<T>;
  static constexpr int LANES = FA_HEAD_DIM / V::N;
  static constexpr int STRIDE = FA_HEAD_DIM + 16;  // the two rows of a warp on different banks
  static constexpr int BUF = RP_THREADS / LANES * STRIDE;

  // `buf`: the CTA's; called by all LANES lanes of a row
  __device__ static void turn(const T* x, T* y, const float2* cs, int rot, int interleaved, T* buf) {
    const int l = threadIdx.x % LANES;
    const unsigned lanes = LANES == 32 ? 0xFFFFFFFFu : 0xFFFFu << (threadIdx.x & 16);
    T* row = buf + threadIdx.x / LANES * STRIDE;
    V::put_raw(row + l * V::N, V::raw(x + l * V::N));
    __syncwarp(lanes);
    for (int i = l; i < rot / 2; i += LANES) {
      const int da = interleaved ? 2 * i : i, db = interleaved ? 2 * i + 1 : rot / 2 + i;
      const float2 u = cs[i];
      const float p = V::get(row[da]), q = V::get(row[db]);
      row[da] = V::put(p * u.x - q * u.y);
      row[db] = V::put(q * u.x + p * u.y);
    }
    __syncwarp(lanes);
    V::put_raw(y + l * V::N, V::raw(row + l * V::N));
    __syncwarp(lanes);  // the lanes' next row lies there too
  }
};

template <typename T, bool VECTOR, int RT>
__global__ void __launch_bounds__(RP_THREADS)
    rope_kernel(const __grid_constant__ RopeParams r, const T* x, T* y,
                const int* __restrict__ positions, long long n_tokens, int T_len, int H,
                long long xb, long long xt, long long xh, long long yb, long long yt,
                long long yh) {
  using Item = RopeItem<T>;
  __shared__ float2 cs[RT][RP_PAIRS];
  __shared__ long long off[2][RT];
  wait_earlier_kernel();
  allow_next_kernel();
  const long long n0 = (long long)blockIdx.x * RT;
  const int nt = (int)min((long long)RT, n_tokens - n0);
  if (threadIdx.x < nt) {
    const long long n = n0 + threadIdx.x, b = n / T_len, tt = n - b * T_len;
    off[0][threadIdx.x] = b * xb + tt * xt;
    off[1][threadIdx.x] = b * yb + tt * yt;
  }
  for (int i = threadIdx.x; i < nt * (r.rot / 2); i += RP_THREADS) {
    const int t = i / (r.rot / 2), pair = i - t * (r.rot / 2);
    cs[t][pair] = rope_cs(r, pair, positions[n0 + t]);
  }
  __syncthreads();
  constexpr int ITEMS = VECTOR ? Item::ITEMS : RopeRow<T>::LANES;
  for (int w = threadIdx.x; w < RT * H * ITEMS; w += RP_THREADS) {
    const int row = w / ITEMS, t = row % RT, h = row / RT;
    if (t >= nt) continue;
    if constexpr (VECTOR) {
      Item item;
      item.y = y + off[1][t] + h * yh;
      item.cs = cs[t];
      item.load(x + off[0][t] + h * xh, w % ITEMS, r.rot, r.interleaved);
      item.store(r.interleaved);
    } else {
      __shared__ __align__(16) T buf[RopeRow<T>::BUF];
      RopeRow<T>::turn(x + off[0][t] + h * xh, y + off[1][t] + h * yh, cs[t], r.rot, r.interleaved, buf);
    }
  }
}

struct AppendRows {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *K, *V;
  long long q_stride, q_out_stride, k_stride, v_stride;
  const int* positions;
  int heads;  // q heads to rotate (0 without q) + Hkv keys + Hkv values
  int rotate;
};

// A CTA takes RT tokens. First one warp each finds its sequence (the count of starts <= t), its
// slot and its position; then the angles of all; then the rows.
template <bool VECTOR, int RT>
__global__ void __launch_bounds__(RP_THREADS)
    paged_append_kernel(const __grid_constant__ RopeParams r, const __grid_constant__ PagedBatch p,
                        const __grid_constant__ AppendRows a) {
  using Item = RopeItem<__nv_bfloat16>;
  using Row = RopeRow<__nv_bfloat16>;
  __shared__ float2 cs[RT][RP_PAIRS];
  __shared__ long long slot_of[RT];  // row of the pools, head 0; -1: not cached, -2: no token
  __shared__ int pos_of[RT];
  wait_earlier_kernel();
  allow_next_kernel();
  const int t0 = blockIdx.x * RT, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < RT) {
    const int t = t0 + warp;
    long long slot = -2;
    int j = 0, b = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int i = b0 + lane + 1;
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, i <= p.B && p.q_start[i] <= t));
      b += n;
      if (n < 32) break;
    }
    if (t < p.total_q && b < p.B) {  // not behind the last sequence
      const SeqSpan s = seq_span(p, b);
      const int i = t - s.q0;
      if (i >= 0 && i < s.n) {
        j = s.kv - s.n + i;  // cache index
        slot = -1;
        const int pg = j >= 0 ? page_of(p, b, j) : -1;
        if (pg >= 0) slot = (long long)pg * p.Hkv * p.page + j % p.page;
      }
    }
    if (lane == 0) {
      slot_of[warp] = slot;
      pos_of[warp] = a.positions && slot != -2 ? a.positions[t] : j;
    }
  }
  __syncthreads();
  const int rot = a.rotate ? r.rot : 0;
  for (int i = threadIdx.x; i < RT * (rot / 2); i += RP_THREADS) {
    const int t = i / (rot / 2), pair = i - t * (rot / 2);
    cs[t][pair] = rope_cs(r, pair, pos_of[t]);
  }
  __syncthreads();
  const int nq = a.heads - 2 * p.Hkv;
  // where row `row` of the CTA comes from and goes to; false: nowhere
  auto find = [&](int row, const __nv_bfloat16** x, __nv_bfloat16** y, int* t, int* turned) {
    *t = row / a.heads;
    const int h = row - *t * a.heads;
    if (*t >= RT || slot_of[*t] == -2 || (h >= nq && slot_of[*t] < 0)) return false;
    const long long token = t0 + *t;
    *turned = h < nq + p.Hkv ? rot : 0;
    if (h < nq) {
      *x = a.q + token * a.q_stride + h * FA_HEAD_DIM;
      *y = a.q_out + token * a.q_out_stride + h * FA_HEAD_DIM;
    } else {
      const int g = h - nq, gk = g < p.Hkv ? g : g - p.Hkv;
      *x = g < p.Hkv ? a.k + token * a.k_stride + gk * FA_HEAD_DIM
                     : a.v + token * a.v_stride + gk * FA_HEAD_DIM;
      *y = (g < p.Hkv ? a.K : a.V) + (slot_of[*t] + (long long)gk * p.page) * FA_HEAD_DIM;
    }
    return true;
  };
  if constexpr (VECTOR) {
    for (int w0 = threadIdx.x; w0 < RT * a.heads * Item::ITEMS; w0 += RP_BATCH * RP_THREADS) {
      Item item[RP_BATCH];
#pragma unroll
      for (int u = 0; u < RP_BATCH; ++u) {
        const int w = w0 + u * RP_THREADS;
        const __nv_bfloat16* x;
        int t, turned;
        item[u].y = nullptr;
        if (!find(w / Item::ITEMS, &x, &item[u].y, &t, &turned)) continue;
        item[u].cs = cs[t];
        item[u].load(x, w % Item::ITEMS, turned, r.interleaved);
      }
#pragma unroll
      for (int u = 0; u < RP_BATCH; ++u)
        if (item[u].y) item[u].store(r.interleaved);
    }
  } else {
    __shared__ __align__(16) __nv_bfloat16 buf[Row::BUF];
    for (int w = threadIdx.x; w < RT * a.heads * Row::LANES; w += RP_THREADS) {
      const __nv_bfloat16* x;
      __nv_bfloat16* y;
      int t, turned;
      if (find(w / Row::LANES, &x, &y, &t, &turned)) Row::turn(x, y, cs[t], turned, r.interleaved, buf);
    }
  }
}

FA_WATCHDOG_READER(read_watchdog_rope)

// ------------------------------------------------------------------------- host side
int rope_init(const fa_rope_config* c, fa_rope_plan* rope) {
  const double pi = 3.14159265358979323846;
  const int n = c->rot_dim / 2;
  double base = c->base;
  if (c->scaling == FA_ROPE_NTK && c->rot_dim > 2)
    base *= pow(c->factor, (double)c->rot_dim / (c->rot_dim - 2));
  double a = 0.0, z = 0.0;  // FA_ROPE_YARN: the pairs between which the blend falls
  if (c->scaling == FA_ROPE_YARN) {
    const double per = c->rot_dim / (2.0 * log(base));
    a = fmax(0.0, floor(per * log(c->original_len / (c->high * 2.0 * pi))));
    z = fmin(c->rot_dim - 1.0, ceil(per * log(c->original_len / (c->low * 2.0 * pi))));
    z = fmax(z, a + 0.001);
  }
  memset(rope, 0, sizeof(*rope));
  rope->rot_dim = c->rot_dim;
  rope->interleaved = c->interleaved;
  const double own = c->scaling == FA_ROPE_YARN ? 0.1 * log(c->factor) + 1.0 : 1.0;
  rope->magnitude = (float)(c->magnitude > 0.0 ? c->magnitude : own);
  for (int i = 0; i < n; ++i) {
    double f = pow(base, -2.0 * i / c->rot_dim);
    if (c->scaling == FA_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == FA_ROPE_BANDS || c->scaling == FA_ROPE_YARN) {
      double w = c->scaling == FA_ROPE_BANDS
                     ? (c->original_len * f / (2.0 * pi) - c->low) / (c->high - c->low)
                     : 1.0 - (i - a) / (z - a);
      w = fmin(1.0, fmax(0.0, w));
      f = f / c->factor * (1.0 - w) + f * w;
    }
    const long double turn = (long double)f / 6.283185307179586476925286766559L;
    rope->turns[i] = (uint64_t)(turn * 18446744073709551616.0L);
  }
  return FA_OK;
}

static RopeParams rope_params(const fa_rope_plan* rope, int transpose) {
  RopeParams r;
  memset(&r, 0, sizeof(r));
  if (!rope) return r;
  r.rot = rope->rot_dim;
  r.interleaved = rope->interleaved;
  r.transpose = transpose;
  r.magnitude = rope->magnitude;
  for (int i = 0; i < RP_PAIRS; ++i) r.turns[i] = rope->turns[i];
  return r;
}

// Pairs in whole vectors of n elements: the halves (or the interleaved run) hold a multiple
// of n pairs.
static bool rope_vectors(const RopeParams& r, int n) { return (r.rot / 2) % n == 0; }

template <typename T>
static cudaError_t rope_typed(const RopeParams& r, int B, int T_len, int H, const int* positions,
                              const void* x, const int64_t* xs, void* y, const int64_t* ys,
                              cudaStream_t stream) {
  const long long n = (long long)B * T_len;
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const bool vec = rope_vectors(r, RopeVec<T>::N);
  // 4 tokens a CTA share the set-up once they still fill every SM several times (bf16, back to back,
  // one a CTA and four: 8 heads, 592 tokens 2.6 and 2.4 us, 2367 5.7 and 4.5, 18944 28 and 17; 32 heads,
  // 592 4.0 and 4.3, 2367 9.5 and 11.3, 4736 16.2 and 16.4, 18944 66 and 60; fp32 within 7% from 4736
  // tokens on where heads are 32)
  const bool four = n >= 16LL * sms;
  auto go = [&](auto kernel, int rt) {
    return launch_overlapped(kernel, dim3((unsigned)((n + rt - 1) / rt)), RP_THREADS, 0, stream, r,
                             static_cast<const T*>(x), static_cast<T*>(y), positions, n, T_len, H,
                             (long long)xs[0], (long long)xs[1], (long long)xs[2], (long long)ys[0],
                             (long long)ys[1], (long long)ys[2]);
  };
  if (vec) return four ? go(rope_kernel<T, true, 4>, 4) : go(rope_kernel<T, true, 1>, 1);
  return four ? go(rope_kernel<T, false, 4>, 4) : go(rope_kernel<T, false, 1>, 1);
}

cudaError_t launch_rope(const fa_rope_plan* rope, int B, int T_len, int H, const int* positions,
                        const void* x, const int64_t* xs, void* y, const int64_t* ys, int dtype,
                        int transpose, cudaStream_t stream) {
  const RopeParams r = rope_params(rope, transpose);
  return dtype == FA_F32
             ? rope_typed<float>(r, B, T_len, H, positions, x, xs, y, ys, stream)
             : rope_typed<__nv_bfloat16>(r, B, T_len, H, positions, x, xs, y, ys, stream);
}

cudaError_t launch_paged_append(const fa_paged_shape& s, const fa_paged_cache& c,
                                const fa_rope_plan* rope, const int32_t* positions, const void* q,
                                int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride,
                                cudaStream_t stream) {
  const RopeParams r = rope_params(rope, 0);
  AppendRows a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.K = static_cast<__nv_bfloat16*>(c.K);
  a.V = static_cast<__nv_bfloat16*>(c.V);
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.heads = (q ? s.Hq : 0) + 2 * s.Hkv;
  a.rotate = rope ? 1 : 0;
  const PagedBatch p = paged_batch(s, c);
  int sms = 148;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  // 4 tokens a CTA share the look-ups once they still fill every SM several times (32 + 8 + 8 heads, one
  // a CTA and four: 148 tokens 3.8 and 6.3 us, 592 5.4 and 6.3, 1184 8.7 and 8.0, 2367 15 and 12, 4736 31
  // and 24, 18944 110 and 86)
  auto go = [&](auto kernel, int rt) {
    return launch_overlapped(kernel, dim3((unsigned)((s.total_q + rt - 1) / rt)), RP_THREADS, 0, stream, r, p, a);
  };
  const bool four = s.total_q >= 16 * sms;
  if (rope_vectors(r, RopeVec<__nv_bfloat16>::N))
    return four ? go(paged_append_kernel<true, 4>, 4) : go(paged_append_kernel<true, 1>, 1);
  return four ? go(paged_append_kernel<false, 4>, 4) : go(paged_append_kernel<false, 1>, 1);
}

}  // namespace fa
