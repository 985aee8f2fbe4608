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

// Attention of one new token a sequence.  With n cached tokens,
//   x_j = q.k_j + bias(p - p_j, t - t_j),  a_j = scale * SiLU(x_j),  AV = sum_j a_j v_j + a_self v_self.
// There is no softmax, so parts of the sum join by plain addition.  The new token is the n+1st row,
// read from U|V|Q|K instead of a page, at distance 0.
//
// The unit of work is a tile of TILE rows of one (sequence, head): 4 KB of K and 4 KB of V.  All
// tiles of the batch, in the order (sequence, head, tile), are dealt to the warps of a persistent
// grid in equal contiguous ranges, so that one long history and many ragged ones load the SMs
// alike; every CTA finds its ranges from the lengths itself (one block scan).  A warp that holds
// all tiles of a (sequence, head) writes its row of AV; parts are joined first among the CTA's
// warps in shared memory, then, where a (sequence, head) spans CTAs, by a second kernel, always in
// the same order.
constexpr int ATTN_THREADS = 512;
constexpr int ATTN_WARPS = ATTN_THREADS / 32;

// What a CTA leaves for the joining kernel.
struct Part {
  int32_t pair;     // sequence * H + head of the part that goes on in the next CTA, or -1
  int32_t before;   // 0: no part that began in an earlier CTA; 1: one that goes on; 2: one that ends here
};

// One tile: sequence, head, tile index, the sequence's cached length and tiles a head, and the
// pages of the tile's 16-row pieces (-1: none).
template <int NP>
struct Tile {
  int b, h, i, n, tiles;
  int pg[NP];
};

template <typename T, int HD>
__global__ void __launch_bounds__(ATTN_THREADS, 1) attention_kernel(const Attn a, float* parts, Part* recs) {
  constexpr int E = vec16<T>::N;      // elements a lane holds of a row
  constexpr int LPR = HD / E;         // lanes a row
  constexpr int RPI = 32 / LPR;       // rows a warp-wide load
  constexpr int TILE = 8 * RPI;
  constexpr int NP = TILE > 16 ? TILE / 16 : 1;
  static_assert(LPR >= 8 && LPR <= 32, "a row spans 8 to 32 lanes");
  __shared__ int64_t pre[ATTN_THREADS];
  __shared__ int64_t scratch[ATTN_WARPS];
  __shared__ __align__(16) float sp[ATTN_WARPS][2][HD];
  __shared__ int s_before[ATTN_WARPS], s_pair[ATTN_WARPS];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sub = lane % LPR, grp = lane / LPR;
  const int H = a.c.H, shift = a.c.ps_shift, ps = 1 << shift, B = (int)a.B;
  const int64_t room = (a.max_pages << shift) - (a.append ? 1 : 0);
  const int64_t most = a.max_len < room ? a.max_len : room;
  auto tiles_of = [&](int n) { return n < 0 ? 0 : n / TILE + 1; };   // of n cached rows and the new one

  // tiles a head before each group of C sequences
  const int C = (B + ATTN_THREADS - 1) / ATTN_THREADS;
  int64_t sum = 0;
  for (int b = threadIdx.x * C; b < B && b < (threadIdx.x + 1) * C; b++)
    sum += tiles_of((int)cached_len(a.lens[b], most));
  {
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0 && lane < ATTN_WARPS) {
      int64_t w = scratch[lane];
#pragma unroll
      for (int o = 1; o < ATTN_WARPS; o <<= 1) {
        const int64_t y = __shfl_up_sync((1u << ATTN_WARPS) - 1u, w, o);
        if (lane >= o) w += y;
      }
      scratch[lane] = w;
    }
    __syncthreads();
    pre[threadIdx.x] = x + (warp ? scratch[warp - 1] : 0);
    __syncthreads();
  }
  const int64_t units = pre[ATTN_THREADS - 1] * H;
  const int64_t gw = (int64_t)blockIdx.x * ATTN_WARPS + warp, W = (int64_t)gridDim.x * ATTN_WARPS;
  const int64_t u0 = units * gw / W, u1 = units * (gw + 1) / W;

  if (lane == 0) {
    s_before[warp] = 0;
    s_pair[warp] = -1;
  }
  if (threadIdx.x == 0) recs[blockIdx.x] = {-1, 0};
  if (u0 < u1) {
    using Tl = Tile<NP>;
    auto length = [&](int b) { return (int)cached_len(a.lens[b], most); };
    auto pages = [&](Tl& t) {
      const int32_t* row = a.table + (int64_t)t.b * a.max_pages;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        const int j = t.i * TILE + 16 * p;
        t.pg[p] = j < t.n ? (int)page_of(row, j >> shift, a.c.num_pages) : -1;
      }
    };
    // the first unit: its group by bisection, its sequence by scans over 32 lengths at a time
    Tl cur;
    {
      const int64_t v = u0 / H;
      int lo = 0, hi = ATTN_THREADS - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] > v) hi = mid; else lo = mid + 1;
      }
      int64_t base = lo ? pre[lo - 1] : 0;
      int b0 = lo * C;
      cur.b = B - 1;
      while (b0 < B) {   // ends with a hit: v is below the batch's tiles
        const int b = b0 + lane;
        const int t = b < B ? tiles_of(length(b)) : 0;
        int64_t x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + x > v);
        if (hit) {
          const int f = __ffs(hit) - 1;
          cur.b = b0 + f;
          base += __shfl_sync(0xffffffffu, x - t, f);
          break;
        }
        base += __shfl_sync(0xffffffffu, x, 31);
        b0 += 32;
      }
      cur.n = length(cur.b);
      cur.tiles = cur.n < 0 ? 1 : tiles_of(cur.n);
      const int64_t r = u0 - base * H;
      cur.h = (int)(r / cur.tiles);
      cur.i = (int)(r % cur.tiles);
    }
    pages(cur);
    auto advance = [&](Tl& t) {
      if (++t.i == t.tiles) {
        t.i = 0;
        if (++t.h == H) {
          t.h = 0;
          t.n = -1;
          while (t.n < 0 && t.b + 1 < B) t.n = length(++t.b);
          t.tiles = tiles_of(t.n);
        }
      }
      pages(t);
    };
    auto u_row = [&](const Tl& t, int block) {   // the new token's U, V, Q or K of the head
      return static_cast<const T*>(a.uvqk) + ((int64_t)t.b * 4 + block) * H * HD + (int64_t)t.h * HD + sub * E;
    };
    // rows of K (block 3) or V (block 1) of a tile
    auto load = [&](const Tl& t, const void* pool, int block, uint4 (&r)[8]) {
      const T* base[NP];
      bool full = (t.i + 1) * TILE <= t.n;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        const int o = (t.i * TILE + 16 * p) & (ps - 1);
        base[p] = static_cast<const T*>(pool) + ((((int64_t)t.pg[p] * H + t.h) << shift) + o - 16 * p + grp) * HD + sub * E;
        full = full && t.pg[p] >= 0;
      }
      if (full) {
#pragma unroll
        for (int i = 0; i < 8; i++)
          r[i] = *reinterpret_cast<const uint4*>(base[i * RPI / 16] + i * RPI * HD);
      } else {
        const T* own = u_row(t, block);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int j = t.i * TILE + i * RPI + grp;
          r[i] = make_uint4(0, 0, 0, 0);
          if (j < t.n) {
            if (t.pg[i * RPI / 16] >= 0)
              r[i] = *reinterpret_cast<const uint4*>(base[i * RPI / 16] + i * RPI * HD);
          } else if (j == t.n) {
            r[i] = *reinterpret_cast<const uint4*>(own);
          }
        }
      }
    };
    // the lane's own row of a tile after the exchange of partial sums
    const int mine = (sub % 8) * RPI + grp;
    struct Meta {
      int32_t p;
      int64_t t;
      float w;
    };
    auto own_page = [&](const Tl& t) { return NP > 1 && mine >= 16 ? t.pg[NP - 1] : t.pg[0]; };
    auto load_meta = [&](const Tl& t, Meta& m) {
      const int j = t.i * TILE + mine, pg = own_page(t);
      m.p = j;
      m.t = 0;
      m.w = 0.0f;
      if (j < t.n && pg >= 0) {
        const int64_t s = ((int64_t)pg << shift) + (j & (ps - 1));
        if (a.c.positions && (a.pos || a.alibi)) m.p = a.c.positions[s];
        if (a.tim) m.t = a.c.timestamps[s];
        if (a.c.weights) m.w = a.c.weights[(((int64_t)pg * H + t.h) << shift) + (j & (ps - 1))];
      }
    };
    uint4 k[8], v[8], q = *reinterpret_cast<const uint4*>(u_row(cur, 2));
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.0f;
    Meta meta;
    load(cur, a.c.k, 3, k);
    load_meta(cur, meta);
    Tl nxt = cur;
    if (u0 + 1 < u1) advance(nxt);
    bool whole = cur.i == 0;   // acc holds the (sequence, head) from its first tile on
    for (int64_t u = u0; u < u1; u++) {
      load(cur, a.c.v, 1, v);
      float part[8], f[E], qf[E];
      vec16<T>::widen(q, qf);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        vec16<T>::widen(k[i], f);
        part[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) part[i] = fmaf(qf[e], f[e], part[i]);
      }
      const Meta m = meta;
      const bool more = u + 1 < u1;
      if (more) {
        load(nxt, a.c.k, 3, k);
        load_meta(nxt, meta);
        if (nxt.i == 0) q = *reinterpret_cast<const uint4*>(u_row(nxt, 2));
      }
      // 8 rows a lane over 8 lanes: each exchange halves the rows a lane sums, so that lane `sub`
      // ends up with row sub % 8 of its group; wider rows add the remaining lanes' sums
#pragma unroll
      for (int w = 4; w >= 1; w >>= 1) {
#pragma unroll
        for (int i = 0; i < w; i++) {
          const bool up = sub & w;
          const float own = up ? part[i + w] : part[i], other = up ? part[i] : part[i + w];
          part[i] = own + __shfl_xor_sync(0xffffffffu, other, w);
        }
      }
#pragma unroll
      for (int w = 8; w < LPR; w <<= 1) part[0] += __shfl_xor_sync(0xffffffffu, part[0], w);
      const int j = cur.i * TILE + mine, pg = own_page(cur);
      const int64_t p_new = a.next_pos ? a.next_pos[cur.b] : cur.n;
      float wgt = 0.0f;
      if (j == cur.n || (j < cur.n && pg >= 0)) {
        int64_t dist = 0, dt = 0;
        if (j < cur.n) {
          dist = p_new - m.p;
          if (dist < 0) dist = 0;
          if (a.tim) dt = a.now[cur.b] - m.t;
        }
        float x = part[0];
        if (a.pos) x += a.pos[(int64_t)cur.h * a.P + (dist < a.P ? dist : a.P - 1)];
        if (a.tim) x += a.tim[(int64_t)cur.h * a.Tb + time_bucket(dt, a.Tb)];
        if (a.alibi) x -= a.alibi[cur.h] * (float)dist;
        wgt = a.scale * silu_accurate(x);
        if (a.c.weights && j < cur.n && sub < 8)
          a.c.weights[(((int64_t)pg * H + cur.h) << shift) + (j & (ps - 1))] = m.w + fabsf(wgt);
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float w = __shfl_sync(0xffffffffu, wgt, grp * LPR + i);
        vec16<T>::widen(v[i], f);
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = fmaf(w, f[e], acc[e]);
      }
      const bool last = cur.i == cur.tiles - 1;
      if (last && a.append && a.lens[cur.b] == cur.n && cur.n <= room) {
        // the new row joins the cache: the lane that owns it writes its weight (and, for head 0,
        // position and time), lanes of one row piece each copy K and V
        const int64_t to = page_of(a.table + (int64_t)cur.b * a.max_pages, cur.n >> shift, a.c.num_pages);
        const int64_t o = cur.n & (ps - 1);
        if (to >= 0) {
          const int64_t r = ((to * H + cur.h) << shift) + o;
          if (grp == 0) {
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.k) + r * HD + sub * E) =
                *reinterpret_cast<const uint4*>(u_row(cur, 3));
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.v) + r * HD + sub * E) =
                *reinterpret_cast<const uint4*>(u_row(cur, 1));
          }
          if (j == cur.n && sub < 8) {
            if (a.c.weights) a.c.weights[r] = fabsf(wgt);
            if (cur.h == 0) {
              if (a.c.positions) a.c.positions[(to << shift) + o] = (int32_t)p_new;
              if (a.c.timestamps && a.now) a.c.timestamps[(to << shift) + o] = a.now[cur.b];
            }
          }
        }
      }
      if (last || !more) {
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1)
#pragma unroll
          for (int e = 0; e < E; e++) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], w);
        const int pair = cur.b * H + cur.h;
        float* to = last && whole ? a.av + (int64_t)pair * HD : sp[warp][whole];
        if (grp == 0) {
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4*>(to + sub * E + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        }
        if (lane == 0) {
          if (!whole) s_before[warp] = last ? 2 : 1;
          else if (!last) s_pair[warp] = pair;
        }
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = 0.0f;
        whole = true;
      }
      if (more) {
        cur = nxt;
        if (u + 2 < u1) advance(nxt);
      }
    }
  }
  // rows of inactive sequences
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (a.lens[b] < 0)
      for (int i = threadIdx.x; i < H * HD; i += ATTN_THREADS) a.av[(int64_t)b * H * HD + i] = 0.0f;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a warp's open end is followed by the later warps' parts, up to the one that ends it
  for (int start = warp == 0 ? -1 : warp; start <= warp; start++) {
    // start -1: the part that began in an earlier CTA
    if (start >= 0 && s_pair[start] < 0) continue;
    bool any = start >= 0, ends = false;
    float s[(HD + 31) / 32];
#pragma unroll
    for (int e = 0; e < HD / 32; e++) s[e] = start >= 0 ? sp[start][1][lane + 32 * e] : 0.0f;
    for (int w = start + 1; w < ATTN_WARPS && !ends; w++) {
      // a part from before this warp belongs to the chain; a warp that begins anew has none
      if (s_before[w]) {
        any = true;
#pragma unroll
        for (int e = 0; e < HD / 32; e++) s[e] += sp[w][0][lane + 32 * e];
        ends = s_before[w] == 2;
      }
      if (start < 0 && s_pair[w] >= 0) break;
    }
    if (start < 0) {
      if (lane == 0) recs[blockIdx.x].before = any ? (ends ? 2 : 1) : 0;
      if (any)
#pragma unroll
        for (int e = 0; e < HD / 32; e++) parts[(int64_t)blockIdx.x * 2 * HD + lane + 32 * e] = s[e];
    } else if (ends) {
#pragma unroll
      for (int e = 0; e < HD / 32; e++) a.av[(int64_t)s_pair[start] * HD + lane + 32 * e] = s[e];
    } else {
      if (lane == 0) recs[blockIdx.x].pair = s_pair[start];
#pragma unroll
      for (int e = 0; e < HD / 32; e++) parts[((int64_t)blockIdx.x * 2 + 1) * HD + lane + 32 * e] = s[e];
    }
  }
}

// Joins the parts of the (sequence, head)s that span CTAs, one CTA for each CTA of the attention: its
// open part and the parts of the following CTAs up to the one that ends it, summed in a fixed order.
template <int HD>
__global__ void __launch_bounds__(256) attention_join_kernel(float* av, const float* parts,
                                                             const Part* recs, int ctas) {
  constexpr int L = HD / 4, G = 256 / L;   // lanes a row, rows at a time
  __shared__ int s_end;
  __shared__ float4 red[G][L];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, pair = recs[c].pair;
  if (pair < 0) return;
  if (threadIdx.x == 0) s_end = ctas - 1;
  __syncthreads();
  for (int k = c + 1 + threadIdx.x; k < ctas; k += 256)
    if (recs[k].before == 2) atomicMin(&s_end, k);
  __syncthreads();
  const int l = threadIdx.x % L, g = threadIdx.x / L, end = s_end;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = c + g; k <= end; k += G) {
    if (k > c && recs[k].before == 0) continue;   // a CTA without work
    const float4 x = reinterpret_cast<const float4*>(parts + ((int64_t)k * 2 + (k == c)) * HD)[l];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  red[g][l] = s;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int w = 1; w < G; w++) {
      s.x += red[w][l].x;
      s.y += red[w][l].y;
      s.z += red[w][l].z;
      s.w += red[w][l].w;
    }
    reinterpret_cast<float4*>(av + (int64_t)pair * HD)[l] = s;
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

// CTAs of the attention: one a SM, at most this many (the workspace holds a part record for each).
constexpr int ATTN_MAX_CTAS = 256;
inline size_t attention_workspace_bytes(int hd) {
  return (size_t)ATTN_MAX_CTAS * (2 * hd * sizeof(float) + sizeof(Part));
}

template <typename T, int HD>
hstu_status_t launch_attention_t(const Attn& a, void* ws, int sms, cudaStream_t st) {
  constexpr int TILE = 8 * 32 * vec16<T>::N / HD;
  // no more CTAs than give each warp one tile of the longest announced length
  const int64_t tiles = a.B * a.c.H * (a.max_len / TILE + 1);
  int64_t grid = (tiles + ATTN_WARPS - 1) / ATTN_WARPS;
  if (grid > sms) grid = sms;
  if (grid > ATTN_MAX_CTAS) grid = ATTN_MAX_CTAS;
  float* parts = static_cast<float*>(ws);
  Part* recs = reinterpret_cast<Part*>(parts + (size_t)ATTN_MAX_CTAS * 2 * HD);
  attention_kernel<T, HD><<<(unsigned)grid, ATTN_THREADS, 0, st>>>(a, parts, recs);
  hstu_status_t rc = launched();
  // one CTA joins its warps' parts itself, and a single tile a (sequence, head) has no parts
  if (rc != HSTU_OK || grid == 1 || a.max_len < TILE) return rc;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // its launch overlaps the attention
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attention_join_kernel<HD>, a.av, (const float*)parts,
                         (const Part*)recs, (int)grid) != cudaSuccess)
    return HSTU_ERR_CUDA;
  return launched();
}

inline hstu_status_t launch_attention(const Attn& a, int dtype, int hd, void* ws, int sms,
                                      cudaStream_t st) {
  if (dtype == HSTU_BF16)
    return hd == 64 ? launch_attention_t<bf16, 64>(a, ws, sms, st)
                    : launch_attention_t<bf16, 128>(a, ws, sms, st);
  return hd == 32   ? launch_attention_t<float, 32>(a, ws, sms, st)
         : hd == 64 ? launch_attention_t<float, 64>(a, ws, sms, st)
                    : launch_attention_t<float, 128>(a, ws, sms, st);
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
