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
#include "sm100.cuh"

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

// 16 bytes of T as pairs of fp32.
template <typename T> struct vec16;
template <> struct vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const uint4& u, uint64_t (&f)[2]) {
    f[0] = sm100::f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = sm100::f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <> struct vec16<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const uint4& u, uint64_t (&f)[4]) {
    f[0] = sm100::f2_pack(bf16_lo(u.x), bf16_hi(u.x));
    f[1] = sm100::f2_pack(bf16_lo(u.y), bf16_hi(u.y));
    f[2] = sm100::f2_pack(bf16_lo(u.z), bf16_hi(u.z));
    f[3] = sm100::f2_pack(bf16_lo(u.w), bf16_hi(u.w));
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
// alike; every CTA finds its ranges from the lengths itself (one block scan).  Each warp brings its
// tiles into its own ring in shared memory by bulk copies.  A warp that holds all tiles of a
// (sequence, head) writes its row of AV; parts are joined first among the CTA's warps in shared
// memory, then, where a (sequence, head) spans CTAs, by a second kernel, always in the same order.
constexpr int ATTN_WARPS = 12;
constexpr int ATTN_STAGES = 2;
constexpr int ATTN_THREADS = ATTN_WARPS * 32;
constexpr int ATTN_HALF = 4096;                 // bytes of a tile's K, and of its V
template <int HD> struct AttnSmem {
  static constexpr int RING = ATTN_WARPS * ATTN_STAGES * 2 * ATTN_HALF;
  static constexpr int PARTS = ATTN_WARPS * 2 * HD * 4;
  static constexpr int TOTAL = RING + PARTS + 128;   // + alignment
};

// CTAs of the attention: one a SM, at most this many (the workspace holds a part record for each).
constexpr int ATTN_MAX_CTAS = 256;

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

// Copies `bytes` (a multiple of 16, both addresses 16-byte aligned) and counts them on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}

// a / b for 0 <= a, 0 < b; the 64-bit division takes several times as long as the 32-bit one.
__device__ __forceinline__ int64_t div_by(int64_t a, int b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

template <typename T, int HD>
__global__ void __launch_bounds__(ATTN_THREADS, 1) attention_kernel(const Attn a, float* parts, Part* recs) {
  using sm100::f2_add;
  using sm100::f2_fma;
  using sm100::f2_pack;
  using sm100::f2_unpack;
  constexpr int E = vec16<T>::N;      // elements a lane holds of a row
  constexpr int LPR = HD / E;         // lanes a row
  constexpr int RPI = 32 / LPR;       // rows a warp-wide load
  constexpr int TILE = 8 * RPI;
  constexpr int NP = TILE > 16 ? TILE / 16 : 1;
  constexpr int PIECE = TILE / NP;    // rows a piece
  constexpr int ROW = HD * (int)sizeof(T);
  static_assert(LPR >= 8 && LPR <= 32, "a row spans 8 to 32 lanes");
  static_assert(TILE * ROW == ATTN_HALF, "a tile is 4 KB of K");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((128 - (sm100::smem_u32(smem_raw) & 127)) & 127);
  float(*sp)[2][HD] = reinterpret_cast<float(*)[2][HD]>(smem + AttnSmem<HD>::RING);
  __shared__ int64_t pre[ATTN_THREADS];
  __shared__ int s_len[ATTN_THREADS];
  __shared__ int64_t scratch[ATTN_WARPS];
  __shared__ int s_before[ATTN_WARPS], s_pair[ATTN_WARPS];
  __shared__ __align__(8) uint64_t bars[ATTN_WARPS][ATTN_STAGES];
  __shared__ int s_abort;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sub = lane % LPR, grp = lane / LPR;
  const int H = a.c.H, shift = a.c.ps_shift, ps = 1 << shift, B = (int)a.B;
  const int64_t room = (a.max_pages << shift) - (a.append ? 1 : 0);
  const int64_t most = a.max_len < room ? a.max_len : room;
  auto tiles_of = [&](int n) { return n < 0 ? 0 : n / TILE + 1; };   // of n cached rows and the new one

  if (lane == 0) {
    s_before[warp] = 0;
    s_pair[warp] = -1;
#pragma unroll
    for (int k = 0; k < ATTN_STAGES; k++) sm100::mbar_init(&bars[warp][k], 1);
    sm100::fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    s_abort = 0;
    recs[blockIdx.x] = {-1, 0};
  }
  // tiles a head up to each group of C sequences; with C = 1 the lengths stay in shared memory
  const int C = (B + ATTN_THREADS - 1) / ATTN_THREADS;
  int64_t sum = 0;
  int n_one = -1;
  for (int b = threadIdx.x * C; b < B && b < (threadIdx.x + 1) * C; b++) {
    n_one = (int)cached_len(a.lens[b], most);
    sum += tiles_of(n_one);
  }
  s_len[threadIdx.x] = n_one;
  {
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < ATTN_WARPS; w++) before += w < warp ? scratch[w] : 0;
    pre[threadIdx.x] = x + before;
    __syncthreads();
  }
  auto length = [&](int b) { return C == 1 ? s_len[b] : (int)cached_len(a.lens[b], most); };
  // every warp's share: `share` tiles, one more for the first `over` warps
  const int64_t units = pre[ATTN_THREADS - 1] * H;
  const int gw = blockIdx.x * ATTN_WARPS + warp, W = gridDim.x * ATTN_WARPS;
  const int64_t share = div_by(units, W);
  const int over = (int)(units - share * W);
  const int64_t u0 = gw * share + (gw < over ? gw : over), u1 = u0 + share + (gw < over ? 1 : 0);

  if (u0 < u1) {
    using Tl = Tile<NP>;
    auto pages = [&](Tl& t) {
      const int32_t* row = a.table + (int64_t)t.b * a.max_pages;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        const int j = t.i * TILE + PIECE * p;
        t.pg[p] = j < t.n ? (int)page_of(row, j >> shift, a.c.num_pages) : -1;
      }
    };
    // the first unit: its group by comparing every ATTN_WARPS-th sum, then the sums between, and
    // with more than one sequence a group by scans over 32 lengths at a time
    Tl cur;
    {
      const int64_t v = div_by(u0, H);
      const unsigned c1 = __ballot_sync(0xffffffffu, pre[lane * ATTN_WARPS + ATTN_WARPS - 1] > v);
      const int g = c1 ? __ffs(c1) - 1 : 31;
      const unsigned c2 = __ballot_sync(0xffffffffu, lane < ATTN_WARPS && pre[g * ATTN_WARPS + lane % ATTN_WARPS] > v);
      const int lo = g * ATTN_WARPS + (c2 ? __ffs(c2) - 1 : ATTN_WARPS - 1);
      int64_t base = lo ? pre[lo - 1] : 0;
      cur.b = lo < B ? lo : B - 1;
      if (C > 1) {
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
      }
      cur.n = length(cur.b);
      cur.tiles = cur.n < 0 ? 1 : tiles_of(cur.n);
      const int64_t r = u0 - base * H;
      cur.h = (int)div_by(r, cur.tiles);
      cur.i = (int)(r - (int64_t)cur.h * cur.tiles);
    }
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
    };
    auto u_row = [&](const Tl& t, int block) {   // the new token's U, V, Q or K of the head
      return static_cast<const T*>(a.uvqk) + (((int64_t)t.b * 4 + block) * H + t.h) * HD;
    };
    unsigned char* ring = smem + warp * (ATTN_STAGES * 2 * ATTN_HALF);
    // the tile's K and V rows, piece by piece, and the new token's into the row after the last
    auto issue = [&](const Tl& t, int stage) {
      if (lane == 0) {
        uint64_t* bar = &bars[warp][stage];
        unsigned char* dst = ring + stage * 2 * ATTN_HALF;
        int rows[NP], total = 0;
#pragma unroll
        for (int p = 0; p < NP; p++) {
          const int left = t.n - (t.i * TILE + PIECE * p);
          rows[p] = t.pg[p] < 0 || left <= 0 ? 0 : (left < PIECE ? left : PIECE);
          total += rows[p];
        }
        const bool own = t.i == t.tiles - 1;
        sm100::mbar_arrive_expect_tx(bar, (uint32_t)(total + own) * 2 * ROW);
#pragma unroll
        for (int p = 0; p < NP; p++) {
          if (rows[p] == 0) continue;
          const int64_t at = ((((int64_t)t.pg[p] * H + t.h) << shift) + ((t.i * TILE + PIECE * p) & (ps - 1))) * HD;
          bulk_load(dst + p * PIECE * ROW, static_cast<const T*>(a.c.k) + at, rows[p] * ROW, bar);
          bulk_load(dst + ATTN_HALF + p * PIECE * ROW, static_cast<const T*>(a.c.v) + at, rows[p] * ROW, bar);
        }
        if (own) {
          const int o = (t.n - t.i * TILE) * ROW;
          bulk_load(dst + o, u_row(t, 3), ROW, bar);
          bulk_load(dst + ATTN_HALF + o, u_row(t, 1), ROW, bar);
        }
      }
    };
    // What the lane needs for the row of a tile that is its own after the exchange of partial sums
    // comes in two steps: position, time and weight two tiles ahead (they need the page), the
    // biases they select one tile ahead.
    const int mine = (sub % 8) * RPI + grp;
    struct Raw {
      int p;
      float w;
      int64_t t;
    };
    struct Own {
      float bias, w;
    };
    auto own_page = [&](const Tl& t) { return NP > 1 && mine >= 16 ? t.pg[NP - 1] : t.pg[0]; };
    int p_new = 0;         // position and time of the new token of the tile last looked up
    int64_t t_new = 0;
    auto load_raw = [&](const Tl& t, bool fresh) {
      if (fresh) {
        const int64_t p = a.next_pos ? a.next_pos[t.b] : t.n;
        if (p < 0 || p > 0x7fffffff) report(HSTU_ERR_DEVICE_BAD_OFFSETS);
        p_new = p < 0 ? 0 : (p > 0x7fffffff ? 0x7fffffff : (int)p);
        t_new = a.now ? a.now[t.b] : 0;
      }
      const int j = t.i * TILE + mine, pg = own_page(t);
      Raw m{j, 0.0f, 0};
      if (j < t.n && pg >= 0) {
        const int64_t s = ((int64_t)pg << shift) + (j & (ps - 1));
        if (a.c.positions && (a.pos || a.alibi)) m.p = a.c.positions[s];
        if (a.tim) m.t = a.c.timestamps[s];
        if (a.c.weights) m.w = a.c.weights[(((int64_t)pg * H + t.h) << shift) + (j & (ps - 1))];
      } else {
        m.p = p_new;
        m.t = t_new;
      }
      return m;
    };
    auto look_up = [&](const Tl& t, const Raw& m) {
      Own r{0.0f, m.w};
      const int far = p_new - m.p, dist = far < 0 ? 0 : far;
      if (a.pos) r.bias = a.pos[(int64_t)t.h * a.P + (dist < a.P ? dist : a.P - 1)];
      if (a.tim) r.bias += a.tim[(int64_t)t.h * a.Tb + time_bucket(t_new - m.t, a.Tb)];
      if (a.alibi) r.bias = -a.alibi[t.h] * (float)dist;
      return r;
    };
    auto load_query = [&](const Tl& t) {
      return *reinterpret_cast<const uint4*>(u_row(t, 2) + sub * E);
    };
    // nxt: the tile after cur, in flight; far: the one after that, its pages being looked up
    Tl nxt = cur, far;
    if (u0 + 1 < u1) advance(nxt);
    far = nxt;
    if (u0 + 2 < u1) advance(far);
    pages(cur);
    pages(nxt);
    pages(far);
    uint4 query = load_query(cur);
    __syncwarp();
    issue(cur, 0);
    if (u0 + 1 < u1) issue(nxt, 1);
    Raw raw = load_raw(cur, true);
    Own own = look_up(cur, raw);
    if (u0 + 1 < u1) raw = load_raw(nxt, nxt.i == 0);
    uint64_t acc[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; e++) acc[e] = 0;
    bool whole = cur.i == 0;   // acc holds the (sequence, head) from its first tile on
    int stage = 0, parity = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1; u++) {
      const bool more = u + 1 < u1;
      const uint4 y = query;
      if (more && nxt.i == 0) query = load_query(nxt);
      const bool full = (cur.i + 1) * TILE <= cur.n && cur.pg[0] >= 0 && cur.pg[NP - 1] >= 0;
      const uint4* ks = reinterpret_cast<const uint4*>(ring + stage * 2 * ATTN_HALF) + lane;
      const uint4* vs = ks + ATTN_HALF / 16;
      ok = sm100::mbar_wait(&bars[warp][stage], parity, &s_abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint64_t f[E / 2], qf[E / 2];
      float part[8];
      vec16<T>::widen(y, qf);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        vec16<T>::widen(ks[i * 32], f);
        uint64_t d = sm100::f2_mul(qf[0], f[0]);
#pragma unroll
        for (int e = 1; e < E / 2; e++) d = f2_fma(qf[e], f[e], d);
        float lo, hi;
        f2_unpack(d, lo, hi);
        part[i] = lo + hi;
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
      float wgt = 0.0f;
      if (j == cur.n || (j < cur.n && pg >= 0)) {
        const float x = part[0] + own.bias;
        wgt = a.scale * silu_accurate(x);
        if (a.c.weights && j < cur.n && sub < 8)
          a.c.weights[(((int64_t)pg * H + cur.h) << shift) + (j & (ps - 1))] = own.w + fabsf(wgt);
      }
      if (more) own = look_up(nxt, raw);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float w = __shfl_sync(0xffffffffu, wgt, grp * LPR + i);
        uint4 r = vs[i * 32];
        if (!full) {
          // rows past the new token's, or of no page, hold what was there before
          const int jr = cur.i * TILE + i * RPI + grp;
          if (jr > cur.n || (jr < cur.n && cur.pg[i * RPI / 16] < 0)) r = make_uint4(0, 0, 0, 0);
        }
        vec16<T>::widen(r, f);
        const uint64_t ww = f2_pack(w, w);
#pragma unroll
        for (int e = 0; e < E / 2; e++) acc[e] = f2_fma(ww, f[e], acc[e]);
      }
      const bool last = cur.i == cur.tiles - 1;
      if (last && a.append && a.lens[cur.b] == cur.n && cur.n <= room) {
        // the new row joins the cache: one row piece's lanes copy K and V, the lane that owns the
        // row writes its weight and, for head 0, position and time
        const int64_t to = page_of(a.table + (int64_t)cur.b * a.max_pages, cur.n >> shift, a.c.num_pages);
        const int64_t o = cur.n & (ps - 1);
        if (to >= 0) {
          const int64_t r = ((to * H + cur.h) << shift) + o;
          if (grp == 0) {
            const int at = (cur.n - cur.i * TILE) * LPR + sub - lane;
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.k) + r * HD + sub * E) = ks[at];
            *reinterpret_cast<uint4*>(static_cast<T*>(a.c.v) + r * HD + sub * E) = vs[at];
          }
          if (j == cur.n && sub < 8) {
            if (a.c.weights) a.c.weights[r] = fabsf(wgt);
            if (cur.h == 0) {
              if (a.c.positions)
                a.c.positions[(to << shift) + o] = (int32_t)(a.next_pos ? a.next_pos[cur.b] : cur.n);
              if (a.c.timestamps && a.now) a.c.timestamps[(to << shift) + o] = a.now[cur.b];
            }
          }
        }
      }
      __syncwarp();   // every lane has read the stage
      if (u + 2 < u1) {
        issue(far, stage);
        raw = load_raw(far, far.i == 0);
      }
      if (last || !more) {
        float s[E];
#pragma unroll
        for (int e = 0; e < E / 2; e++) f2_unpack(acc[e], s[2 * e], s[2 * e + 1]);
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1)
#pragma unroll
          for (int e = 0; e < E; e++) s[e] += __shfl_xor_sync(0xffffffffu, s[e], w);
        const int pair = cur.b * H + cur.h;
        float* to = last && whole ? a.av + (int64_t)pair * HD : sp[warp][whole];
        if (grp == 0) {
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4*>(to + sub * E + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
        }
        if (lane == 0) {
          if (!whole) s_before[warp] = last ? 2 : 1;
          else if (!last) s_pair[warp] = pair;
        }
#pragma unroll
        for (int e = 0; e < E / 2; e++) acc[e] = 0;
        whole = true;
      }
      cur = nxt;
      nxt = far;
      if (u + 3 < u1) {
        advance(far);
        pages(far);
      }
      stage ^= 1;
      parity ^= stage == 0;
    }
    if (!__all_sync(0xffffffffu, ok)) {
      // gave up: what is still being copied lands before the CTA goes
      sm100::mbar_drain(&bars[warp][stage], parity);
      sm100::mbar_drain(&bars[warp][stage ^ 1], parity ^ (stage == 1));
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // rows of inactive sequences
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (length(b) < 0)
      for (int i = threadIdx.x; i < H * HD; i += ATTN_THREADS) a.av[(int64_t)b * H * HD + i] = 0.0f;
  __syncthreads();
  // A warp's open end is followed by the later warps' parts, up to the one that ends it.  Parts that
  // began in an earlier CTA come before the first open end.
  const int flag = lane < ATTN_WARPS ? s_before[lane] : 0;
  const unsigned parted = __ballot_sync(0xffffffffu, flag != 0), ends = __ballot_sync(0xffffffffu, flag == 2);
  auto add_parts = [&](unsigned set, bool open, float* to) {
    float s[HD / 32];
#pragma unroll
    for (int e = 0; e < HD / 32; e++) s[e] = open ? sp[warp][1][lane + 32 * e] : 0.0f;
    for (; set; set &= set - 1) {
      const int w = __ffs(set) - 1;
#pragma unroll
      for (int e = 0; e < HD / 32; e++) s[e] += sp[w][0][lane + 32 * e];
    }
#pragma unroll
    for (int e = 0; e < HD / 32; e++) to[lane + 32 * e] = s[e];
  };
  auto up_to_end = [&](unsigned set) {   // the set's warps up to its first end
    const unsigned e = set & ends;
    return e ? set & ((e & (0u - e)) * 2u - 1u) : set;
  };
  const int pair = s_pair[warp];
  if (pair >= 0) {
    const unsigned set = up_to_end(parted & ~((2u << warp) - 1u));
    const bool done = set & ends;
    add_parts(set, true, done ? a.av + (int64_t)pair * HD : parts + ((int64_t)blockIdx.x * 2 + 1) * HD);
    if (!done && lane == 0) recs[blockIdx.x].pair = pair;
  }
  if (warp == 0) {
    const unsigned opens = __ballot_sync(0xffffffffu, lane < ATTN_WARPS && s_pair[lane] >= 0);
    const unsigned first = opens & (0u - opens);   // its own part from before may end there too
    const unsigned set = up_to_end(opens ? parted & (first * 2u - 1u) : parted);
    if (set) {
      add_parts(set, false, parts + (int64_t)blockIdx.x * 2 * HD);
      if (lane == 0) recs[blockIdx.x].before = set & ends ? 2 : 1;
    }
  }
}

// Joins the parts of the (sequence, head)s that span CTAs, one CTA for each CTA of the attention: its
// open part and the parts of the following CTAs up to the one that ends it, summed in a fixed order.
template <int HD>
__global__ void __launch_bounds__(ATTN_MAX_CTAS) attention_join_kernel(float* av, const float* parts,
                                                             const Part* recs, int ctas) {
  constexpr int L = HD / 4, G = ATTN_MAX_CTAS / L;   // lanes a row, rows at a time
  __shared__ int s_end, s_flag[ATTN_MAX_CTAS];
  __shared__ float4 red[G][L];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, pair = recs[c].pair;
  if (threadIdx.x == 0) s_end = ctas - 1;
  const int flag = threadIdx.x < ctas ? recs[threadIdx.x].before : 0;
  s_flag[threadIdx.x] = flag;
  if (pair < 0) return;
  __syncthreads();
  if ((int)threadIdx.x > c && flag == 2) atomicMin(&s_end, (int)threadIdx.x);
  __syncthreads();
  const int l = threadIdx.x % L, g = threadIdx.x / L, end = s_end;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = c + g; k <= end; k += G) {
    if (k > c && s_flag[k] == 0) continue;   // a CTA without work
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
  auto kern = attention_kernel<T, HD>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, AttnSmem<HD>::TOTAL) !=
      cudaSuccess)
    return HSTU_ERR_CUDA;
  kern<<<(unsigned)grid, ATTN_THREADS, AttnSmem<HD>::TOTAL, st>>>(a, parts, recs);
  hstu_status_t rc = launched();
  // one CTA joins its warps' parts itself, and a single tile a (sequence, head) has no parts
  if (rc != HSTU_OK || grid == 1 || a.max_len < TILE) return rc;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // its launch overlaps the attention
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(ATTN_MAX_CTAS);
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
