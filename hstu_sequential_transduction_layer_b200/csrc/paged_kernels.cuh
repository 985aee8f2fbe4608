// Paged key-value cache of one layer: filling it from U|V|Q|K, attention of one new token a sequence
// over it, and eviction by accumulated attention weight.  None of them has a contraction worth a
// tensor core (one query row a head: one multiply-add per cached element read), so all are bound by
// HBM and, when small, by latency.
//
// Layout: K and V [num_pages, H, page_size, hd], so that one head's part of a page is one contiguous
// block; positions (int32) and timestamps (int64) [num_pages, page_size]; accumulated weights (fp32)
// [num_pages, H, page_size].  A sequence's slot i lives in page table[b][i / page_size] at offset
// i % page_size.
#pragma once

#include "common.cuh"

namespace hstu {
namespace paged {

// The cache as the kernels see it.
struct Cache {
  void* k;
  void* v;
  int32_t* positions;    // nullable: slot i holds position i
  int64_t* timestamps;   // nullable
  float* weights;        // nullable
  int64_t num_pages;
  int ps_shift;          // log2(page_size)
  int H;
};

// What one attention call adds to it.
struct Attn {
  Cache c;
  const void* uvqk;          // [B, 4*H*hd]
  const int32_t* table;      // [B, max_pages]
  int64_t max_pages;
  const int64_t* lens;       // [B], < 0: inactive
  const int64_t* next_pos;   // [B], nullable: lens
  const int64_t* now;        // [B], nullable without a time table
  const float* pos;          // [H, P] or null
  const float* tim;          // [H, Tb] or null
  const float* alibi;        // [H] or null
  int P, Tb;
  float scale;
  int append;
  int64_t B;
  int64_t max_len;           // longest cached length the caller announced
  float* av;                 // [B, H*hd]
};

// Page of a sequence's slot, or -1 (reported) when the table's entry is no page.
__device__ __forceinline__ int64_t page_of(const int32_t* __restrict__ row, int64_t entry,
                                           int64_t num_pages) {
  const int64_t p = row[entry];
  if (p < 0 || p >= num_pages) {
    report(HSTU_ERR_DEVICE_BAD_OFFSETS);
    return -1;
  }
  return p;
}

// Cached length of sequence b, clamped to what its page-table row (and the announced longest
// length) can hold with `extra` more tokens; -1 for an inactive sequence.
__device__ __forceinline__ int64_t cached_len(int64_t len, int64_t most) {
  if (len < 0) return -1;
  if (len > most) {
    report(HSTU_ERR_DEVICE_BAD_OFFSETS);
    return most < 0 ? 0 : most;
  }
  return len;
}

__device__ __forceinline__ int time_bucket(int64_t dt, int Tb) {
  const uint64_t v = 1ull + (uint64_t)(dt < 0 ? 0 : dt);   // floor(log2) = highest set bit
  const int b = 63 - __clzll((long long)v);
  return b < Tb ? b : Tb - 1;
}

// 16 bytes of T as fp32.
template <typename T> struct vec16;
template <> struct vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
};
template <> struct vec16<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const uint4& u, float* f) {
    f[0] = bf16_lo(u.x);
    f[1] = bf16_hi(u.x);
    f[2] = bf16_lo(u.y);
    f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z);
    f[5] = bf16_hi(u.z);
    f[6] = bf16_lo(u.w);
    f[7] = bf16_hi(u.w);
  }
};

// Attention of one new token a sequence, one CTA per (sequence, head).  With n cached tokens,
//   x_j = q.k_j + bias(p - p_j, t - t_j),  a_j = scale * SiLU(x_j),  AV = sum_j a_j v_j + a_self v_self
// (no softmax: parts of the sum join by addition).  The new token is the n+1st row, read from U|V|Q|K
// instead of a page, at distance 0.  A warp takes tiles of TILE rows, 16 bytes a lane and row piece;
// the dot products' partial sums are exchanged so that each lane ends up with one row's score.
constexpr int ATTN_THREADS = 256;
template <typename T, int HD>
__global__ void __launch_bounds__(ATTN_THREADS) attention_kernel(const Attn a) {
  constexpr int E = vec16<T>::N;      // elements a lane holds of a row
  constexpr int LPR = HD / E;         // lanes a row
  constexpr int RPI = 32 / LPR;       // rows a warp-wide load
  constexpr int TILE = 8 * RPI;
  static_assert(LPR >= 8 && LPR <= 32, "a row spans 8 to 32 lanes");
  __shared__ float red[ATTN_THREADS / 32][HD];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sub = lane % LPR, grp = lane / LPR;
  const int64_t b = blockIdx.x / a.c.H;
  const int h = (int)(blockIdx.x % a.c.H);
  const int H = a.c.H, ps = 1 << a.c.ps_shift;
  const int64_t room = a.max_pages << a.c.ps_shift;
  const int64_t most = a.max_len < room - (a.append ? 1 : 0) ? a.max_len : room - (a.append ? 1 : 0);
  const int64_t n = cached_len(a.lens[b], most);
  float* out = a.av + (b * H + h) * HD;
  if (n < 0) {
    for (int i = threadIdx.x; i < HD; i += ATTN_THREADS) out[i] = 0.0f;
    return;
  }
  const bool store = a.append && a.lens[b] == n && n < room;
  const T* row = static_cast<const T*>(a.uvqk) + b * 4 * H * HD + (int64_t)h * HD + sub * E;
  const T *v_new = row + (int64_t)H * HD, *q_new = row + 2LL * H * HD, *k_new = row + 3LL * H * HD;
  float q[E], acc[E];
  vec16<T>::widen(*reinterpret_cast<const uint4*>(q_new), q);
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.0f;
  const int64_t p_new = a.next_pos ? a.next_pos[b] : n, t_new = a.now ? a.now[b] : 0;
  const int32_t* pages = a.table + b * a.max_pages;
  for (int64_t t0 = (int64_t)warp * TILE; t0 <= n; t0 += (ATTN_THREADS / 32) * TILE) {
    uint4 kv[8];
    float part[8];
    int64_t at[8];   // element offset of the lane's piece of each row; -1: no such row
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int64_t j = t0 + i * RPI + grp;
      at[i] = -1;
      kv[i] = make_uint4(0, 0, 0, 0);
      if (j < n) {
        const int64_t pg = page_of(pages, j >> a.c.ps_shift, a.c.num_pages);
        if (pg >= 0) {
          at[i] = (((pg * H + h) << a.c.ps_shift) + (j & (ps - 1))) * HD + sub * E;
          kv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.k) + at[i]);
        }
      } else if (j == n) {
        kv[i] = *reinterpret_cast<const uint4*>(k_new);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float f[E];
      vec16<T>::widen(kv[i], f);
      part[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; e++) part[i] = fmaf(q[e], f[e], part[i]);
    }
    // 8 rows a lane over 8 lanes: each exchange halves the rows a lane sums, so that lane `sub`
    // ends up with row i = sub % 8; wider rows add the remaining lanes' sums
#pragma unroll
    for (int w = 4; w >= 1; w >>= 1) {
#pragma unroll
      for (int i = 0; i < w; i++) {
        const bool up = sub & w;
        const float mine = up ? part[i + w] : part[i], other = up ? part[i] : part[i + w];
        part[i] = mine + __shfl_xor_sync(0xffffffffu, other, w);
      }
    }
#pragma unroll
    for (int w = 8; w < LPR; w <<= 1) part[0] += __shfl_xor_sync(0xffffffffu, part[0], w);
    // the lane's own row
    const int64_t j = t0 + (sub % 8) * RPI + grp;
    float wgt = 0.0f;
    if (j <= n) {
      int64_t slot = -1;
      if (j < n || store) {
        const int64_t pg = page_of(pages, j >> a.c.ps_shift, a.c.num_pages);
        if (pg >= 0) slot = (pg << a.c.ps_shift) + (j & (ps - 1));
      }
      float x = part[0];
      if (j == n || slot >= 0) {
        int64_t dist = 0, dt = 0;
        if (j < n) {
          dist = p_new - (a.c.positions ? (int64_t)a.c.positions[slot] : j);
          if (dist < 0) dist = 0;
          if (a.tim) dt = t_new - a.c.timestamps[slot];
        }
        if (a.pos) x += a.pos[(int64_t)h * a.P + (dist < a.P ? dist : a.P - 1)];
        if (a.tim) x += a.tim[(int64_t)h * a.Tb + time_bucket(dt, a.Tb)];
        if (a.alibi) x -= a.alibi[h] * (float)dist;
        wgt = a.scale * silu_accurate(x);
      }
      if (slot >= 0 && sub < 8) {
        if (a.c.weights) {
          const int64_t pg = slot >> a.c.ps_shift;
          float* wp = a.c.weights + ((pg * H + h) << a.c.ps_shift) + (slot & (ps - 1));
          *wp = j < n ? *wp + fabsf(wgt) : fabsf(wgt);
        }
        if (j == n && h == 0) {
          if (a.c.positions) a.c.positions[slot] = (int32_t)p_new;
          if (a.c.timestamps && a.now) a.c.timestamps[slot] = t_new;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float w = __shfl_sync(0xffffffffu, wgt, grp * LPR + i);
      const int64_t jr = t0 + i * RPI + grp;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (at[i] >= 0) u = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.v) + at[i]);
      if (jr == n) {
        u = *reinterpret_cast<const uint4*>(v_new);
        if (store) {
          const int64_t pg = page_of(pages, n >> a.c.ps_shift, a.c.num_pages);
          if (pg >= 0) {
            const int64_t to = (((pg * H + h) << a.c.ps_shift) + (n & (ps - 1))) * HD + sub * E;
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.k) + to) = kv[i];
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.v) + to) = u;
          }
        }
      }
      float f[E];
      vec16<T>::widen(u, f);
      if (at[i] >= 0 || jr == n) {
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = fmaf(w, f[e], acc[e]);
      }
    }
  }
#pragma unroll
  for (int w = LPR; w < 32; w <<= 1)
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], w);
  if (grp == 0)
#pragma unroll
    for (int e = 0; e < E; e++) red[warp][sub * E + e] = acc[e];
  __syncthreads();
  for (int i = threadIdx.x; i < HD; i += ATTN_THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < ATTN_THREADS / 32; w++) s += red[w][i];
    out[i] = s;
  }
}

// Rows of a jagged U|V|Q|K batch into the cache: token t of sequence b goes to slot lens[b] + (t -
// off[b]).  One warp per (token, head).
template <typename T>
__global__ void __launch_bounds__(256) append_kernel(const Cache c, int HD, int64_t Tn, int64_t B,
                                                     const T* __restrict__ uvqk,
                                                     const int64_t* __restrict__ off,
                                                     const int64_t* __restrict__ ts,
                                                     const int32_t* __restrict__ table,
                                                     int64_t max_pages,
                                                     const int64_t* __restrict__ lens,
                                                     const int64_t* __restrict__ next_pos) {
  constexpr int E = vec16<T>::N;
  const int lane = threadIdx.x % 32;
  const int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (item >= Tn * c.H) return;
  const int64_t t = item / c.H;
  const int h = (int)(item % c.H);
  // the last sequence that starts at or before t and has not ended by then
  int64_t lo = 0, hi = B;   // off[lo] <= t < off[hi]
  if (t < off[0] || t >= off[B]) return;   // reported by the offsets check
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  const int64_t i = t - off[lo], n = lens[lo], slot = n + i, room = max_pages << c.ps_shift;
  if (n < 0 || i < 0 || n >= room || slot >= room) {
    if (lane == 0) report(HSTU_ERR_DEVICE_BAD_OFFSETS);
    return;
  }
  const int64_t pg = page_of(table + lo * max_pages, slot >> c.ps_shift, c.num_pages);
  if (pg < 0) return;
  const int ps = 1 << c.ps_shift, o = (int)(slot & (ps - 1));
  const int64_t to = (((pg * c.H + h) << c.ps_shift) + o) * HD;
  const T* src = uvqk + t * 4 * c.H * HD + (int64_t)h * HD;
  for (int e = lane * E; e < HD; e += 32 * E) {
    *reinterpret_cast<uint4*>(static_cast<T*>(c.k) + to + e) =
        *reinterpret_cast<const uint4*>(src + 3LL * c.H * HD + e);
    *reinterpret_cast<uint4*>(static_cast<T*>(c.v) + to + e) =
        *reinterpret_cast<const uint4*>(src + (int64_t)c.H * HD + e);
  }
  if (lane == 0) {
    if (c.weights) c.weights[((pg * c.H + h) << c.ps_shift) + o] = 0.0f;
    if (h == 0) {
      if (c.positions) c.positions[(pg << c.ps_shift) + o] = (int32_t)((next_pos ? next_pos[lo] : n) + i);
      if (c.timestamps && ts) c.timestamps[(pg << c.ps_shift) + o] = ts[t];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Eviction
// ------------------------------------------------------------------------------------------------

// One eviction call: sequences longer than `budget` keep their `recent` newest tokens and, of the
// others, those with the largest accumulated weight (summed over the heads).
struct Evict {
  Cache c;
  const int32_t* table;
  int64_t max_pages, B;
  const int64_t* lens;
  const int64_t* next_pos;   // nullable: lens
  int64_t budget, recent;
  int64_t* new_lens;
  // workspace
  uint32_t* keys;            // [B, room]
  int64_t *to, *from;        // [B, moves]: flat slots (page * page_size + offset)
  int64_t* count;            // [B]
  int64_t room, moves;
};

constexpr uint32_t KEY_RECENT = 0xffffffffu;

// Keys that order tokens by what is kept first: recent ones, then by weight (sums rounded once to
// fp32; NaN last), as unsigned integers.
__device__ __forceinline__ uint32_t weight_key(float s) {
  if (s != s) return 0u;
  s += 0.0f;                                   // -0 and +0 are equal weights
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One thread per slot of every sequence that has to lose tokens.
__global__ void __launch_bounds__(256) evict_keys_kernel(const Evict a) {
  const int64_t b = blockIdx.y;
  const int64_t n = cached_len(a.lens[b], a.room);
  if (n <= a.budget) return;
  const int ps = 1 << a.c.ps_shift;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256) {
    const int64_t pg = page_of(a.table + b * a.max_pages, j >> a.c.ps_shift, a.c.num_pages);
    uint32_t key = 0;
    if (pg >= 0) {
      const int64_t o = j & (ps - 1);
      double s = 0.0;
      for (int h = 0; h < a.c.H; h++) s += (double)a.c.weights[((pg * a.c.H + h) << a.c.ps_shift) + o];
      key = weight_key((float)s);
      const int64_t next = a.next_pos ? a.next_pos[b] : n;
      if ((int64_t)a.c.positions[(pg << a.c.ps_shift) + o] >= next - a.recent) key = KEY_RECENT;
    }
    a.keys[b * a.room + j] = key;
  }
}

constexpr int SEL_THREADS = 1024;

// Exclusive prefix sums of two counts per thread, packed in one int64 (each below 2^31).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const int64_t before = (warp > 0 ? scratch[warp - 1] : 0) + x - v;
  __syncthreads();
  return before;
}

// One CTA per sequence: the budget-th largest key by radix select, 8 bits a pass, then the gaps
// below slot `budget` and the kept slots above it, both in ascending order.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const Evict a) {
  __shared__ unsigned int hist[256];
  __shared__ int64_t scratch[32];
  __shared__ uint32_t s_digit;
  __shared__ int64_t s_k;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x;
  const int64_t len = a.lens[b], n = cached_len(len, a.room);
  if (n <= a.budget) {
    if (tid == 0) {
      a.new_lens[b] = len < 0 ? len : n;
      a.count[b] = 0;
    }
    return;
  }
  const uint32_t* keys = a.keys + b * a.room;
  uint32_t prefix = 0, mask = 0;
  int64_t k = a.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int d = tid; d < 256; d += SEL_THREADS) hist[d] = 0;
    __syncthreads();
    for (int64_t j = tid; j < n; j += SEL_THREADS) {
      const uint32_t key = keys[j];
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int64_t cum = 0;
      int d = 255;
      while (d > 0 && cum + hist[d] < k) cum += hist[d--];
      s_digit = d;
      s_k = k - cum;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    k = s_k;
    __syncthreads();
  }
  // kept: key > prefix, and the first k slots whose key equals it
  const int64_t per = (n + SEL_THREADS - 1) / SEL_THREADS;
  const int64_t j0 = tid * per < n ? tid * per : n, j1 = j0 + per < n ? j0 + per : n;
  int64_t eq = 0;
  for (int64_t j = j0; j < j1; j++) eq += keys[j] == prefix ? 1 : 0;
  const int64_t eq0 = block_scan(eq, scratch);
  int64_t both = 0, seen = eq0;
  for (int64_t j = j0; j < j1; j++) {
    const bool same = keys[j] == prefix, keep = keys[j] > prefix || (same && seen < k);
    seen += same ? 1 : 0;
    if (j < a.budget && !keep) both += 1;
    if (j >= a.budget && keep) both += 1LL << 32;
  }
  const int64_t before = block_scan(both, scratch);
  int64_t gaps = before & 0xffffffffLL, movers = before >> 32;
  seen = eq0;
  const int ps = 1 << a.c.ps_shift;
  for (int64_t j = j0; j < j1; j++) {
    const bool same = keys[j] == prefix, keep = keys[j] > prefix || (same && seen < k);
    seen += same ? 1 : 0;
    if ((j < a.budget) == keep) continue;
    const int64_t pg = page_of(a.table + b * a.max_pages, j >> a.c.ps_shift, a.c.num_pages);
    const int64_t flat = pg < 0 ? -1 : (pg << a.c.ps_shift) + (j & (ps - 1));
    if (keep) a.from[b * a.moves + movers++] = flat; else a.to[b * a.moves + gaps++] = flat;
  }
  if (tid == SEL_THREADS - 1) {
    a.count[b] = gaps;   // as many gaps below the budget as kept slots above it
    a.new_lens[b] = a.budget;
  }
}

// Moves the kept rows into the gaps.  Sources lie at or above slot `budget`, destinations below it,
// so rows move in any order.  One warp per (move, head).
template <typename T>
__global__ void __launch_bounds__(256) evict_move_kernel(const Evict a, int HD) {
  constexpr int E = vec16<T>::N;
  const int64_t b = blockIdx.y, count = a.count[b];
  const int lane = threadIdx.x % 32, ps = 1 << a.c.ps_shift, H = a.c.H;
  for (int64_t it = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; it < count * H;
       it += (int64_t)gridDim.x * 8) {
    const int64_t m = it / H;
    const int h = (int)(it % H);
    const int64_t to = a.to[b * a.moves + m], from = a.from[b * a.moves + m];
    if (to < 0 || from < 0) continue;
    const int64_t rt = ((((to >> a.c.ps_shift) * H + h) << a.c.ps_shift) + (to & (ps - 1)));
    const int64_t rf = ((((from >> a.c.ps_shift) * H + h) << a.c.ps_shift) + (from & (ps - 1)));
    for (int e = lane * E; e < HD; e += 32 * E) {
      T *k = static_cast<T*>(a.c.k), *v = static_cast<T*>(a.c.v);
      *reinterpret_cast<uint4*>(k + rt * HD + e) = *reinterpret_cast<const uint4*>(k + rf * HD + e);
      *reinterpret_cast<uint4*>(v + rt * HD + e) = *reinterpret_cast<const uint4*>(v + rf * HD + e);
    }
    if (lane == 0) {
      a.c.weights[rt] = a.c.weights[rf];
      if (h == 0) {
        a.c.positions[to] = a.c.positions[from];
        if (a.c.timestamps) a.c.timestamps[to] = a.c.timestamps[from];
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Launchers (arguments already checked)
// ------------------------------------------------------------------------------------------------

inline hstu_status_t launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

inline bool head_dim_supported(int dtype, int hd) {
  return dtype == HSTU_BF16 ? hd == 64 || hd == 128 : hd == 32 || hd == 64 || hd == 128;
}

inline hstu_status_t launch_attention(const Attn& a, int dtype, int hd, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.B * a.c.H);
  if (dtype == HSTU_BF16) {
    if (hd == 64) attention_kernel<bf16, 64><<<grid, ATTN_THREADS, 0, st>>>(a);
    else attention_kernel<bf16, 128><<<grid, ATTN_THREADS, 0, st>>>(a);
  } else {
    if (hd == 32) attention_kernel<float, 32><<<grid, ATTN_THREADS, 0, st>>>(a);
    else if (hd == 64) attention_kernel<float, 64><<<grid, ATTN_THREADS, 0, st>>>(a);
    else attention_kernel<float, 128><<<grid, ATTN_THREADS, 0, st>>>(a);
  }
  return launched();
}

inline hstu_status_t launch_append(const Cache& c, int dtype, int hd, int64_t T, int64_t B,
                                   const void* uvqk, const int64_t* off, const int64_t* ts,
                                   const int32_t* table, int64_t max_pages, const int64_t* lens,
                                   const int64_t* next_pos, cudaStream_t st) {
  const unsigned grid = (unsigned)((T * c.H + 7) / 8);
  if (dtype == HSTU_BF16)
    append_kernel<bf16><<<grid, 256, 0, st>>>(c, hd, T, B, (const bf16*)uvqk, off, ts, table,
                                              max_pages, lens, next_pos);
  else
    append_kernel<float><<<grid, 256, 0, st>>>(c, hd, T, B, (const float*)uvqk, off, ts, table,
                                               max_pages, lens, next_pos);
  return launched();
}

inline hstu_status_t launch_evict(const Evict& a, int dtype, int hd, cudaStream_t st) {
  hstu_status_t rc;
  const unsigned gx = (unsigned)(a.room < 256 * 64 ? (a.room + 255) / 256 : 64);
  evict_keys_kernel<<<dim3(gx, (unsigned)a.B), 256, 0, st>>>(a);
  if ((rc = launched()) != HSTU_OK) return rc;
  evict_select_kernel<<<(unsigned)a.B, SEL_THREADS, 0, st>>>(a);
  if ((rc = launched()) != HSTU_OK) return rc;
  const dim3 grid(64, (unsigned)a.B);
  if (dtype == HSTU_BF16) evict_move_kernel<bf16><<<grid, 256, 0, st>>>(a, hd);
  else evict_move_kernel<float><<<grid, 256, 0, st>>>(a, hd);
  return launched();
}

}  // namespace paged
}  // namespace hstu
