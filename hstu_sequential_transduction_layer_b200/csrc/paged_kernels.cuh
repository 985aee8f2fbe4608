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

#include <cooperative_groups.h>

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
__device__ __forceinline__ int64_t page_of(const int32_t* row, int64_t entry, int64_t num_pages) {
  const int64_t p = row[entry];
  if (p < 0 || p >= num_pages) {
    report(HSTU_ERR_DEVICE_BAD_OFFSETS);
    return -1;
  }
  return p;
}

// A sequence's cached length, clamped (and reported) to `most`; -1 for an inactive sequence.
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

// a / b for 0 <= a, 0 < b; the 64-bit division takes several times as long as the 32-bit one.
__device__ __forceinline__ int64_t div_by(int64_t a, int b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Programmatic dependent launch: a kernel may be launched while the one before it in the stream
// finishes, and touches global memory only after `after_previous`; `let_next` allows the same to
// the next one.  Every kernel of this file is launched so: without it a launch costs a microsecond
// or two between kernels that take a few (an eviction of 48 histories 34.4 us a call, with it 30.9).
// What an earlier kernel may have written is therefore read by plain loads only: the compiler may
// move loads that it takes for invariant (__ldg, const __restrict__) above the wait.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
// tiles of the batch, in the order (sequence, head, tile), are dealt to the consumer warps of a
// persistent grid in equal contiguous ranges, so that one long history and many ragged ones load
// the SMs alike; every CTA finds its ranges from the lengths itself (one block scan).  One producer
// warp, a lane for each consumer warp, walks the ranges, looks the pages up and fills the warp's
// ring in shared memory with K and V by bulk copies (as few as the pages allow: a copy occupies the
// SM's copy engine for some 75 cycles, however small).  The consumer loads what else its tile needs
// one tile ahead.  A warp that holds all tiles of a (sequence, head) writes its row of AV; parts
// are joined first among the CTA's warps in shared memory, then, where a (sequence, head) spans
// CTAs, by a second kernel, always in the same order.
constexpr int ATTN_WARPS = 11;                  // consumers
constexpr int ATTN_STAGES = 2;
constexpr int ATTN_INFOS = 4;                   // tiles told of: two in flight and two ahead
static_assert(ATTN_STAGES == 2 && ATTN_INFOS == ATTN_STAGES + 2, "the start tells of and fills two stages");
constexpr int ATTN_THREADS = (ATTN_WARPS + 1) * 32;
constexpr int ATTN_NAP = 30;                    // ns between the producer's looks for work
constexpr int ATTN_HALF = 4096;                 // bytes of a tile's K, and of its V
// CTAs of the attention: one a SM, at most this many (the workspace holds a part record for each).
constexpr int ATTN_MAX_CTAS = 256;

// What a consumer is told of a tile: written by the producer beside the rows.
struct __align__(16) TileInfo {
  int32_t pair, b, h;      // sequence * H + head, and both
  int32_t first;           // the tile's first slot
  int32_t left;            // cached rows from the tile's first on; below TILE: its last tile
  int32_t flags;           // bit 0: the first tile; bit 1 + p: 16-row piece p has no page
  int32_t p_new;           // the new token's position and time
  int64_t t_new;
  int64_t row[2];          // rows of the pieces in K, V and weights: (page * H + h) * page_size + offset
  int64_t slot[2];         // and in positions and times: page * page_size + offset
  int64_t to;              // where the new token's row goes, or -1
  int64_t to_slot;         // its slot (page * page_size + offset) for position and time, or -1
};

template <typename T, int HD>
struct AttnCfg {
  static constexpr int E = vec16<T>::N;      // elements a lane holds of a row
  static constexpr int LPR = HD / E;         // lanes a row
  static constexpr int RPI = 32 / LPR;       // rows a warp-wide load
  static constexpr int TILE = 8 * RPI;
  static constexpr int NP = TILE > 16 ? TILE / 16 : 1;
  static constexpr int PIECE = TILE / NP;    // rows a piece: pieces do not cross pages
  static constexpr int ROW = HD * (int)sizeof(T);
  static constexpr int STAGE = 2 * ATTN_HALF;   // K and V
  static constexpr int RING = ATTN_WARPS * ATTN_STAGES * STAGE;
  static constexpr int PARTS = RING, ROWS = PARTS + ATTN_WARPS * 2 * HD * 4;
  static constexpr int SMEM = ROWS + ATTN_WARPS * 2 * 32 * 16 + 128;   // + alignment
  static_assert(LPR >= 8 && LPR <= 32, "a row spans 8 to 32 lanes");
  static_assert(TILE * ROW == ATTN_HALF && NP <= 2, "a tile is 4 KB of K");
};

// What a CTA leaves for the joining kernel.
struct Part {
  int32_t pair;     // sequence * H + head of the part that goes on in the next CTA, or -1
  int32_t before;   // 0: no part that began in an earlier CTA; 1: one that goes on; 2: one that ends here
};

// Copies `bytes` (a multiple of 16, both addresses 16-byte aligned) and counts them on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}

// Copies 4 or 8 bytes for the calling thread, in its current group.
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "n"(N)
               : "memory");
}

__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of the calling thread's groups are in flight.
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(sm100::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

template <typename T, int HD>
__global__ void __launch_bounds__(ATTN_THREADS, 1) attention_kernel(const Attn a, float* parts, Part* recs) {
  using sm100::f2_fma;
  using sm100::f2_pack;
  using sm100::f2_unpack;
  using Cfg = AttnCfg<T, HD>;
  constexpr int E = Cfg::E, LPR = Cfg::LPR, RPI = Cfg::RPI, TILE = Cfg::TILE, NP = Cfg::NP,
                PIECE = Cfg::PIECE, ROW = Cfg::ROW, STAGE = Cfg::STAGE;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((128 - (sm100::smem_u32(smem_raw) & 127)) & 127);
  float(*sp)[2][HD] = reinterpret_cast<float(*)[2][HD]>(smem + Cfg::PARTS);
  __shared__ int pre[ATTN_THREADS], s_len[ATTN_THREADS];
  __shared__ int scratch[ATTN_THREADS / 32];
  __shared__ int s_before[ATTN_WARPS], s_pair[ATTN_WARPS];
  __shared__ TileInfo s_info[ATTN_WARPS][ATTN_INFOS];
  __shared__ int s_issued[ATTN_WARPS];   // tiles whose TileInfo is written
  __shared__ __align__(8) uint64_t full_bar[ATTN_WARPS][ATTN_STAGES], free_bar[ATTN_WARPS][ATTN_STAGES];
  __shared__ int s_abort;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int H = a.c.H, shift = a.c.ps_shift, ps = 1 << shift, B = (int)a.B;
  const int64_t room = (a.max_pages << shift) - (a.append ? 1 : 0);
  const int64_t most = a.max_len < room ? a.max_len : room;
  // a sequence's cached length, doubled, plus 1 where it was clamped (its token is not stored)
  auto coded_len = [&](int b) {
    const int64_t len = a.lens[b], n = cached_len(len, most);
    return n < 0 ? -1 : (int)(2 * n + (n != len));
  };
  auto tiles_of = [&](int n) { return n < 0 ? 0 : n / TILE + 1; };   // of n cached rows and the new one

  if (warp < ATTN_WARPS && lane == 0) {
    s_before[warp] = 0;
    s_issued[warp] = 0;
    s_pair[warp] = -1;
#pragma unroll
    for (int k = 0; k < ATTN_STAGES; k++) {
      sm100::mbar_init(&full_bar[warp][k], 1);
      sm100::mbar_init(&free_bar[warp][k], 1);
    }
    sm100::fence_mbar_init();
  }
  if (threadIdx.x == 0) s_abort = 0;
  after_previous();
  if (threadIdx.x == 0) recs[blockIdx.x] = {-1, 0};
  // tiles a head up to each group of C sequences; with C = 1 the lengths stay in shared memory
  const int C = (B + ATTN_THREADS - 1) / ATTN_THREADS;
  {
    int x = 0, code = -1;
    for (int b = threadIdx.x * C; b < B && b < (int)(threadIdx.x + 1) * C; b++) {
      code = coded_len(b);
      x += tiles_of(code >> 1);
    }
    s_len[threadIdx.x] = code;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < ATTN_THREADS / 32; w++) x += w < warp ? scratch[w] : 0;
    pre[threadIdx.x] = x;
    __syncthreads();
  }
  // every consumer's share: `share` tiles, one more for the first `over` of them
  const uint32_t units = (uint32_t)pre[ATTN_THREADS - 1] * H, W = gridDim.x * ATTN_WARPS;
  const uint32_t share = units / W, over = units - share * W;

  // copies the cached rows of tile k into consumer c's ring; its barrier completes once it is also
  // arrived on
  auto fill = [&](int c, int k) {
    const int stage = k % ATTN_STAGES;
    const TileInfo& t = s_info[c][k % ATTN_INFOS];
    uint64_t* bar = &full_bar[c][stage];
    unsigned char* dst = smem + (c * ATTN_STAGES + stage) * STAGE;
    int rows[NP], sum = 0;
#pragma unroll
    for (int p = 0; p < NP; p++) {
      const int left = t.left - PIECE * p;
      rows[p] = left <= 0 || (t.flags & (2 << p)) ? 0 : (left < PIECE ? left : PIECE);
      sum += rows[p];
    }
    sm100::mbar_expect_tx(bar, (uint32_t)sum * 2 * ROW);
    if (NP > 1 && ps >= TILE) {   // one page
      rows[0] = sum;
      rows[NP - 1] = 0;
    }
#pragma unroll
    for (int p = 0; p < NP; p++) {
      if (rows[p] == 0) continue;
      const int64_t at = t.row[p] * HD;
      bulk_load(dst + p * PIECE * ROW, static_cast<const T*>(a.c.k) + at, rows[p] * ROW, bar);
      bulk_load(dst + ATTN_HALF + p * PIECE * ROW, static_cast<const T*>(a.c.v) + at, rows[p] * ROW, bar);
    }
  };

  int done = 0;   // tiles taken
  if (warp == ATTN_WARPS) {
    const uint32_t gw = blockIdx.x * ATTN_WARPS + lane;
    const uint32_t u0 = gw * share + (gw < over ? gw : over);
    const int count = lane < ATTN_WARPS ? (int)(share + (gw < over ? 1 : 0)) : 0;
    int b = 0, h = 0, i = 0, n = 0, code = 0, tiles = 1;
    int32_t pg[NP];
    auto length = [&](int s) { return C == 1 ? s_len[s] : coded_len(s); };
    // the pages of the tile's pieces, that of the new token's row among them
    auto pages = [&]() {
      const int32_t* row = a.table + (int64_t)b * a.max_pages;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        const int j = i * TILE + PIECE * p;
        pg[p] = j < n + a.append ? row[j >> shift] : -1;
      }
    };
    if (count > 0) {
      // the range's first tile: the first group whose running sum exceeds v, and the sequence in it
      const int v = (int)(u0 / (uint32_t)H);
      int lo = 0, hi = B < ATTN_THREADS ? B - 1 : ATTN_THREADS - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] > v) hi = mid; else lo = mid + 1;
      }
      int base = lo ? pre[lo - 1] : 0;
      b = lo * C;
      code = length(b);
      while (base + tiles_of(code >> 1) <= v && b + 1 < B) {
        base += tiles_of(code >> 1);
        code = length(++b);
      }
      n = code >> 1;
      tiles = n < 0 ? 1 : tiles_of(n);
      const uint32_t r = u0 - (uint32_t)base * H;
      h = (int)(r / (uint32_t)tiles);
      i = (int)(r - (uint32_t)h * tiles);
      pages();
    }
    int p_new = 0, owner = -1, told = 0;
    int64_t t_new = 0;
    // tells the consumer of the walk's tile
    auto tell = [&]() {
      if (owner != b) {
        owner = b;
        const int64_t p = a.next_pos ? a.next_pos[b] : n;
        if (p < 0 || p > 0x7fffffff) report(HSTU_ERR_DEVICE_BAD_OFFSETS);
        p_new = p < 0 ? 0 : (p > 0x7fffffff ? 0x7fffffff : (int)p);
        t_new = a.now ? a.now[b] : 0;
      }
      TileInfo info;
      info.pair = b * H + h;
      info.b = b;
      info.h = h;
      info.first = i * TILE;
      info.left = n - i * TILE;
      info.flags = i == 0;
      info.p_new = p_new;
      info.t_new = t_new;
      info.to = info.to_slot = -1;
#pragma unroll
      for (int p = 0; p < NP; p++) {
        const int left = info.left - PIECE * p, at = (i * TILE + PIECE * p) & (ps - 1);
        if ((uint32_t)pg[p] >= (uint32_t)a.c.num_pages) {
          if (left + a.append > 0) report(HSTU_ERR_DEVICE_BAD_OFFSETS);
          info.flags |= 2 << p;
        }
        info.slot[p] = ((int64_t)pg[p] << shift) + at;
        info.row[p] = (((int64_t)pg[p] * H + h) << shift) + at;
        if (a.append && left >= 0 && left < PIECE && !(code & 1) && !(info.flags & (2 << p))) {
          info.to = info.row[p] + left;
          if (h == 0) info.to_slot = info.slot[p] + left;
        }
      }
      s_info[lane][told % ATTN_INFOS] = info;
      __threadfence_block();
      *reinterpret_cast<volatile int*>(&s_issued[lane]) = ++told;
      if (told < count) {
        if (++i == tiles) {
          i = 0;
          if (++h == H) {
            h = 0;
            code = -1;
            while (code < 0 && b + 1 < B) code = length(++b);
            n = code >> 1;
            tiles = tiles_of(n);
          }
        }
        pages();
      }
    };
    // The consumers fill their first ATTN_STAGES tiles themselves (a warp's copies are issued one lane
    // after another).  From then on a consumer that has seen tile k's barrier complete has been told
    // of tiles k + 1 and k + 2: the arrival comes after.
    for (int k = 0; k < ATTN_STAGES + 2; k++)
      if (told < count) tell();
    done = count < ATTN_STAGES ? count : ATTN_STAGES;
    uint64_t idle = 0;   // since when no lane had anything to refill
    while (__any_sync(0xffffffffu, done < count)) {
      const int stage = done % ATTN_STAGES;
      const bool go = done < count && mbar_test(&free_bar[lane][stage], (done / ATTN_STAGES + 1) & 1);
      if (go) {
        fill(lane, done);
        if (told < count) tell();
        sm100::mbar_arrive(&full_bar[lane][stage]);
        done++;
      }
      if (__any_sync(0xffffffffu, go)) {
        idle = 0;
        continue;
      }
      // bounded, as every wait of this kernel; asleep, so as to leave the issue slots to the consumers
      const uint64_t now = sm100::globaltimer();
      if (idle == 0) idle = now;
      if (lane == 0 && now - idle > 2 * sm100::kWaitLimitNs) {
        s_abort = 1;
        report(HSTU_ERR_DEVICE_TIMEOUT);
      }
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_abort))) break;
      __nanosleep(ATTN_NAP);
    }
    let_next();
  } else {
    const int gw = blockIdx.x * ATTN_WARPS + warp;
    const int count = (int)(share + ((uint32_t)gw < over ? 1 : 0));
    const int sub = lane % LPR, grp = lane / LPR;
    const int mine = (sub % 8) * RPI + grp;   // the lane's own row after the exchange of partial sums
    // What a tile needs besides K and V: the lane's own row's position, time and weight are loaded
    // two tiles ahead, the biases that they select one tile ahead, the lane's piece of Q with the
    // tile before a (sequence, head)'s first, those of the new token's K and V with its last.
    struct __align__(16) Ahead {
      int64_t t;
      int p;
      float w;
    };
    Ahead(*rows)[32] = reinterpret_cast<Ahead(*)[32]>(smem + Cfg::ROWS) + warp * 2;
    uint4 q, k_own, v_own;
    q = k_own = v_own = make_uint4(0, 0, 0, 0);
    auto new_row = [&](const TileInfo& t, int block) {   // the lane's piece of the new token's U, V, Q or K
      return *reinterpret_cast<const uint4*>(static_cast<const T*>(a.uvqk) +
                                             (((int64_t)t.b * 4 + block) * H + t.h) * HD + sub * E);
    };
    auto told_of = [&](int k) -> const TileInfo& { return s_info[warp][k % ATTN_INFOS]; };
    auto on_page = [&](const TileInfo& t) {   // the lane's own row is cached
      return mine < t.left && !(t.flags & (NP > 1 && mine >= PIECE ? 4 : 2));
    };
    auto place = [&](const int64_t* at) { return (NP > 1 && mine >= PIECE ? at[1] - PIECE : at[0]) + mine; };
    auto look_ahead = [&](int k) {   // each lane waits for and reads its own copies only
      const TileInfo& t = told_of(k);
      if (on_page(t)) {
        Ahead* r = &rows[k % 2][lane];
        const int64_t slot = place(t.slot);
        if (a.tim) copy_async<8>(&r->t, a.c.timestamps + slot);
        if (a.c.positions && (a.pos || a.alibi)) copy_async<4>(&r->p, a.c.positions + slot);
        if (a.c.weights) copy_async<4>(&r->w, a.c.weights + place(t.row));
      }
    };
    // loads tile k's biases (used one tile later) and its row's weight
    float bias_p = 0.0f, bias_t = 0.0f, weight = 0.0f;
    auto look_up = [&](int k) {
      const TileInfo& t = told_of(k);
      const bool cached = on_page(t);   // the new token's own row is at distance 0
      const Ahead& r = rows[k % 2][lane];
      if (a.pos || a.alibi) {
        const int far = t.p_new - (a.c.positions ? r.p : t.first + mine), dist = cached && far > 0 ? far : 0;
        if (a.pos) bias_p = a.pos[(int64_t)t.h * a.P + (dist < a.P ? dist : a.P - 1)];
        else bias_p = -a.alibi[t.h] * (float)dist;
      }
      if (a.tim) bias_t = a.tim[(int64_t)t.h * a.Tb + time_bucket(cached ? t.t_new - r.t : 0, a.Tb)];
      if (a.c.weights) weight = r.w;
    };
    auto await = [&](int k) {   // bounded, as every wait of this kernel
      const uint64_t t0 = sm100::globaltimer();
      while (!__all_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_issued[warp]) > k)) {
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_abort))) return false;
        if (__any_sync(0xffffffffu, sm100::globaltimer() - t0 > sm100::kWaitLimitNs)) {
          if (lane == 0) {
            s_abort = 1;
            report(HSTU_ERR_DEVICE_TIMEOUT);
          }
          return false;
        }
      }
      __threadfence_block();
      return true;
    };
    uint64_t acc[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; e++) acc[e] = 0;
    bool whole = true, ok = true;   // whole: acc holds the (sequence, head) from its first tile on
    if (count > 0 && (ok = await(0))) {
      if (lane == 0) {
        fill(warp, 0);
        sm100::mbar_arrive(&full_bar[warp][0]);
      }
      whole = told_of(0).flags & 1;
      q = new_row(told_of(0), 2);
      look_ahead(0);
      copy_async_commit();
      if (count > 1 && (ok = await(1))) {
        if (lane == 0) {
          fill(warp, 1);
          sm100::mbar_arrive(&full_bar[warp][1]);
        }
        look_ahead(1);
      }
      copy_async_commit();
      copy_async_wait<1>();
      look_up(0);
    }
    for (; ok && done < count; done++) {
      const int stage = done % ATTN_STAGES;
      const TileInfo &info = told_of(done), &next = told_of(done + 1);
      unsigned char* src = smem + (warp * ATTN_STAGES + stage) * STAGE;
      const int left = info.left, flags = info.flags, pair = info.pair;
      const bool more = done + 1 < count, last = left < TILE;
      uint4 q_next = q;
      if (more && (next.flags & 1)) q_next = new_row(next, 2);
      if (last) {
        k_own = new_row(info, 3);
        v_own = new_row(info, 1);
      }
      ok = sm100::mbar_wait(&full_bar[warp][stage], (done / ATTN_STAGES) & 1, &s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (done + 2 < count) {
        if (done < ATTN_STAGES && !(ok = await(done + 2))) break;
        look_ahead(done + 2);
      }
      copy_async_commit();
      const uint4* ks = reinterpret_cast<const uint4*>(src) + lane;
      const uint4* vs = ks + ATTN_HALF / 16;
      if (last) {
        // the new token's rows go behind the last cached ones
        if (grp == 0) {
          *reinterpret_cast<uint4*>(src + left * ROW + sub * 16) = k_own;
          *reinterpret_cast<uint4*>(src + ATTN_HALF + left * ROW + sub * 16) = v_own;
        }
        __syncwarp();
      }
      const bool cached = on_page(info);
      uint64_t f[E / 2], qf[E / 2];
      float part[8];
      vec16<T>::widen(q, qf);
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
      float wgt = 0.0f;
      // only here: added where they are loaded, the two would be waited for a tile early
      asm volatile("" : "+f"(bias_p), "+f"(bias_t));
      if (cached || mine == left) {
        wgt = a.scale * silu_accurate(part[0] + (bias_p + bias_t));
        if (a.c.weights && cached && sub < 8) a.c.weights[place(info.row)] = weight + fabsf(wgt);
      }
      copy_async_wait<1>();   // tile done + 1's rows
      if (more) look_up(done + 1);
      const bool full = left >= TILE && !(flags & ~1);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float w = __shfl_sync(0xffffffffu, wgt, grp * LPR + i);
        uint4 r = vs[i * 32];
        if (!full) {
          // rows past the new token's, or of no page, hold what was there before
          const int row = i * RPI + grp;
          if (row > left || (row < left && (flags & (2 << (i * RPI / 16))))) r = make_uint4(0, 0, 0, 0);
        }
        vec16<T>::widen(r, f);
        const uint64_t ww = f2_pack(w, w);
#pragma unroll
        for (int e = 0; e < E / 2; e++) acc[e] = f2_fma(ww, f[e], acc[e]);
      }
      if (last && info.to >= 0) {
        // the new row joins the cache: one group's lanes copy K and V, the lane that owns the row
        // writes its weight and, for head 0, position and time
        if (grp == 0) {
          *reinterpret_cast<uint4*>(static_cast<T*>(a.c.k) + info.to * HD + sub * E) = k_own;
          *reinterpret_cast<uint4*>(static_cast<T*>(a.c.v) + info.to * HD + sub * E) = v_own;
        }
        if (mine == left && sub < 8) {
          if (a.c.weights) a.c.weights[info.to] = fabsf(wgt);
          if (info.to_slot >= 0) {
            if (a.c.positions) a.c.positions[info.to_slot] = info.p_new;
            if (a.c.timestamps && a.now) a.c.timestamps[info.to_slot] = info.t_new;
          }
        }
      }
      if (last)   // rows written here come before the copies that will refill the stage
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();   // every lane has read the stage
      if (lane == 0) sm100::mbar_arrive(&free_bar[warp][stage]);
      if (last || done + 1 == count) {
        float s[E];
#pragma unroll
        for (int e = 0; e < E / 2; e++) f2_unpack(acc[e], s[2 * e], s[2 * e + 1]);
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1)
#pragma unroll
          for (int e = 0; e < E; e++) s[e] += __shfl_xor_sync(0xffffffffu, s[e], w);
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
      q = q_next;
    }
  }
  // rows of inactive sequences
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if ((C == 1 ? s_len[b] : coded_len(b)) < 0)
      for (int i = threadIdx.x; i < H * HD; i += ATTN_THREADS) a.av[(int64_t)b * H * HD + i] = 0.0f;
  __syncthreads();
  if (s_abort) {
    // gave up: what is still being copied lands before the CTA goes
    if (warp < ATTN_WARPS && lane == 0)
      for (int k = done; k < done + ATTN_STAGES; k++)
        sm100::mbar_drain(&full_bar[warp][k % ATTN_STAGES], (k / ATTN_STAGES) & 1);
    return;
  }
  if (warp == ATTN_WARPS) return;
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
  after_previous();
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
// off[b]).  A CTA takes `tokens` tokens: a thread a token finds its sequence by bisection and its
// row's place, then all threads copy, 16 bytes at a time; K and V rows are read in order, 1 to 8 KB a
// token, and written as the heads' separate rows of 128 bytes or more.  HBM-bound.
constexpr int APPEND_TOKENS = 32, APPEND_PIECES = 1024;
template <int LPR>
__global__ void __launch_bounds__(256) append_kernel(const Cache c, int tokens, int64_t Tn, int64_t B,
                                                     const uint4* uvqk, const int64_t* off,
                                                     const int64_t* ts, const int32_t* table,
                                                     int64_t max_pages, const int64_t* lens,
                                                     const int64_t* next_pos) {
  __shared__ int64_t s_row[APPEND_TOKENS];   // the token's row of head 0, or -1
  after_previous();
  // the offsets' own check, over all CTAs
  for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s <= B; s += (int64_t)gridDim.x * 256) {
    const int64_t v = off[s];
    if ((s == 0 && v != 0) || (s == B && v != Tn) || v < 0 || v > Tn || (s > 0 && off[s - 1] > v))
      report(HSTU_ERR_DEVICE_BAD_OFFSETS);
  }
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int shift = c.ps_shift, ps = 1 << shift, H = c.H;
  if (threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t row = -1;
    if (t < Tn && t >= off[0] && t < off[B]) {
      int64_t lo = 0, hi = B;   // off[lo] <= t < off[hi]
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (off[mid] <= t) lo = mid; else hi = mid;
      }
      const int64_t i = t - off[lo], n = lens[lo], slot = n + i, room = max_pages << shift;
      if (n < 0 || n >= room || slot >= room) {
        report(HSTU_ERR_DEVICE_BAD_OFFSETS);
      } else {
        const int64_t pg = page_of(table + lo * max_pages, slot >> shift, c.num_pages);
        if (pg >= 0) {
          const int64_t o = slot & (ps - 1), at = (pg << shift) + o;
          row = ((pg * H) << shift) + o;
          const int64_t p = (next_pos ? next_pos[lo] : n) + i;
          if (p < 0 || p > 0x7fffffff) report(HSTU_ERR_DEVICE_BAD_OFFSETS);
          if (c.positions) c.positions[at] = (int32_t)(p < 0 ? 0 : p > 0x7fffffff ? 0x7fffffff : p);
          if (c.timestamps && ts) c.timestamps[at] = ts[t];
        }
      }
    }
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  // piece x of a token: 16 bytes of K and of V; head x / LPR
  const int width = H * LPR, total = tokens * width;
  constexpr int U = 4;
  for (int x0 = threadIdx.x; x0 < total; x0 += 256 * U) {
    uint4 k[U], v[U];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int x = x0 + u * 256, t = x / width, e = x - t * width;
      to[u] = -1;
      if (x < total && s_row[t] >= 0) {
        const int h = e / LPR;
        to[u] = s_row[t] + ((int64_t)h << shift);
        const uint4* src = uvqk + (t0 + t) * 4 * width + e;
        v[u] = src[width];
        k[u] = src[3 * width];
        if (e % LPR == 0 && c.weights) c.weights[to[u]] = 0.0f;
        to[u] = to[u] * LPR + e % LPR;
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (to[u] < 0) continue;
      __stcs(static_cast<uint4*>(c.k) + to[u], k[u]);
      __stcs(static_cast<uint4*>(c.v) + to[u], v[u]);
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
  uint32_t *to, *from;       // [B, moves]: slots of the pool (page * page_size + offset)
  int64_t* count;            // [B]
  int64_t room, moves;
};

// Keys above every weight's: of recent tokens, and of slots below the budget whose table entry is no
// page.  Nothing can move into those, so they stay among the kept ones (there are at most `budget` of
// them); such slots from the budget on have the lowest key and, as all below the budget come before
// them, are never kept.
constexpr uint32_t KEY_RECENT = 0xfffffffeu, KEY_NO_PAGE = 0xffffffffu;

// The two halves of a cluster barrier; the first publishes nothing.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// Orders tokens by what is kept first, as unsigned integers: by weight (sums rounded once to fp32;
// NaN last).
__device__ __forceinline__ uint32_t weight_key(float s) {
  if (s != s) return 0u;
  s += 0.0f;                                   // -0 and +0 are equal weights
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Selection, one cluster of CTAs per sequence, each on a contiguous part of its slots, each warp on a
// contiguous part of that.  Every thread scores its slots; the first SEL_ROUNDS keys stay in shared
// memory, any further ones go through the workspace.  The budget-th largest key is found by histograms of the
// top 11, the next 11 and the last 10 bits: every CTA counts its own keys, sums all CTAs' bins
// through distributed shared memory and finds the bin for itself; once few keys share the bits found
// so far, every CTA gathers those and finishes alone, with one cluster barrier a step.  Then every
// CTA lists the gaps below slot `budget` and the kept slots from there on among its own, in ascending
// order.  Eleven bits (two of the mantissa) spread accumulated weights over enough bins that the
// shared-memory atomics seldom meet; warps whose keys all fall into one bin add them at once.
//
// Bound by latency and by fetching instructions that run a few times: 8 sequences of 8192 slots and 8
// heads take about 10 us (scores 3.8, search 4.5 in two passes, lists 2).  Hence several CTAs a
// sequence (with one, 8 us longer), 512 threads (256: 5 us longer for 32 771 slots), and loops over
// keys in shared memory (unrolled over registers: 16 000 slots 21.9 us an eviction, so 20.1).
// Exchanging whole histograms through distributed shared memory took 2 us longer.
constexpr int SEL_THREADS = 512, SEL_WARPS = SEL_THREADS / 32, SEL_KEYS = 8, SEL_CLUSTER = 16;
constexpr int SEL_BINS = 2048, SEL_LIST = 1024, SEL_ROUNDS = 16;
constexpr int SEL_SMEM = 2 * SEL_ROUNDS * SEL_THREADS * 4;   // keys and pages of a thread's slots

__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const Evict a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ __align__(16) int s_hist[3][SEL_BINS];
  __shared__ uint32_t s_list[SEL_LIST], s_gathered[SEL_LIST];
  __shared__ int s_listed, s_groups[3][SEL_CLUSTER][SEL_BINS / 32];
  __shared__ int s_warp[SEL_WARPS], s_gaps[SEL_WARPS], s_movers[SEL_WARPS];
  __shared__ int s_count[3][SEL_CLUSTER];      // equal keys, gaps and movers of the cluster's CTAs
  __shared__ int s_found[3];                   // the bin that holds the key searched, how many of its
                                               // keys are kept, and how many there are
  extern __shared__ uint32_t s_own[];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  uint32_t *const s_key = s_own + tid, *const s_page = s_key + SEL_ROUNDS * SEL_THREADS;
  if (tid == 0) s_listed = 0;
  for (int i = tid; i < 3 * SEL_BINS / 4; i += SEL_THREADS)
    reinterpret_cast<int4*>(s_hist)[i] = make_int4(0, 0, 0, 0);
  after_previous();
  let_next();
  const int64_t b = blockIdx.x / S, len = a.lens[b], n64 = cached_len(len, a.room);
  if (n64 <= a.budget) {
    if (rank == 0 && tid == 0) {
      a.new_lens[b] = len < 0 ? len : n64;
      a.count[b] = 0;
    }
    return;
  }
  // the CTAs store to each other from the search's first step on: by then all of them have to have
  // started, which the scoring leaves time for
  if (S > 1) cluster_arrive();
  auto sync = [&]() {
    if (S > 1) cluster.sync(); else __syncthreads();
  };
  const int n = (int)n64, budget = (int)a.budget;   // slots are numbered in 31 bits
  const int shift = a.c.ps_shift, ps = 1 << shift, H = a.c.H;
  const int32_t* pages = a.table + b * a.max_pages;
  // the warp's slots: `rounds` times 32
  const int rounds = (n + S * SEL_THREADS - 1) / (S * SEL_THREADS);
  const int start = (rank * SEL_WARPS + warp) * rounds * 32 + lane;   // < n + 32 * S * SEL_THREADS
  const int64_t oldest = (a.next_pos ? a.next_pos[b] : n64) - a.recent;
  uint32_t* spill = a.keys + b * a.room;

  // scores: the loads of SEL_KEYS slots and four heads are in flight at once
  // (unconditional, from some slot where there is none: a load under a condition is waited for at once)
#pragma unroll 1
  for (int r0 = 0; r0 < rounds; r0 += SEL_KEYS) {
    uint32_t at[SEL_KEYS];      // rows of weights: below 2^32
    int pos[SEL_KEYS];
    double sum[SEL_KEYS];
    unsigned live = 0;
#pragma unroll
    for (int i = 0; i < SEL_KEYS; i++) {
      const int j = start + (r0 + i) * 32;
      at[i] = (uint32_t)pages[(j < n ? j : n - 1) >> shift];
      sum[i] = 0.0;
    }
#pragma unroll
    for (int i = 0; i < SEL_KEYS; i++) {
      const int j = start + (r0 + i) * 32;
      if (r0 + i < rounds && j < n) {
        if (at[i] < (uint32_t)a.c.num_pages) live |= 1u << i;
        else report(HSTU_ERR_DEVICE_BAD_OFFSETS);
      }
      if (r0 + i < SEL_ROUNDS) s_page[(r0 + i) * SEL_THREADS] = live >> i & 1 ? at[i] : ~0u;
      if (!(live >> i & 1)) at[i] = 0;   // any page: the value is dropped
      const int o = j & (ps - 1);
      pos[i] = a.c.positions[((int64_t)at[i] << shift) + o];
      at[i] = ((at[i] * (uint32_t)H) << shift) + o;
    }
#pragma unroll 1
    for (int h = 0; h < H; h += 4) {
      float w[4][SEL_KEYS];
#pragma unroll
      for (int u = 0; u < 4; u++)
#pragma unroll
        for (int i = 0; i < SEL_KEYS; i++)
          w[u][i] = a.c.weights[at[i] + ((uint32_t)(h + u < H ? h + u : H - 1) << shift)];
#pragma unroll
      for (int u = 0; u < 4; u++)
#pragma unroll
        for (int i = 0; i < SEL_KEYS; i++) sum[i] += h + u < H ? (double)w[u][i] : 0.0;
    }
#pragma unroll
    for (int i = 0; i < SEL_KEYS; i++) {
      const int j = start + (r0 + i) * 32;
      uint32_t k = (int64_t)pos[i] >= oldest ? KEY_RECENT : weight_key((float)sum[i]);
      if (!(live >> i & 1)) k = j < budget ? KEY_NO_PAGE : 0u;
      if (r0 + i < SEL_ROUNDS) s_key[(r0 + i) * SEL_THREADS] = k;
      else if (r0 + i < rounds && j < n) spill[j] = k;
    }
  }
  // f(slot, key, its page or some page, whether there is such a slot) for the warp's slots in order;
  // all lanes take part.  Not unrolled: what runs a few times is bound by fetching its instructions.
  auto each = [&](auto f) {
#pragma unroll 1
    for (int r = 0; r < rounds; r++) {
      const int j = start + r * 32;
      uint32_t k, pg;
      if (r < SEL_ROUNDS) {
        k = s_key[r * SEL_THREADS];
        pg = s_page[r * SEL_THREADS];
      } else {
        const int at = j < n ? j : n - 1;
        k = spill[at];
        pg = (uint32_t)pages[at >> shift];
      }
      f(j, k, pg, j < n);
    }
  };
  __syncthreads();   // bins are zero
  if (S > 1) cluster_wait();

  uint32_t prefix = 0, mask = 0;
  int want = budget;          // of the keys that share the prefix, how many are kept
  int in_bin = n;             // and how many there are
  // counts a warp's keys into bins; all lanes take part
  auto count = [&](int* hist, uint32_t k, bool counts, int sh, uint32_t low) {
    const unsigned m = __ballot_sync(0xffffffffu, counts);
    if (m == 0) return;
    const int bin = (int)(k >> sh & low), lead = __ffs(m) - 1;
    const int its = __shfl_sync(0xffffffffu, bin, lead);
    if (__ballot_sync(0xffffffffu, counts && bin == its) == m) {
      if (lane == lead) atomicAdd(&hist[bin], __popc(m));
    } else if (counts) {
      atomicAdd(&hist[bin], 1);
    }
  };
  // The highest bin at which the count from the top reaches `want`, of the cluster's bins or of the
  // CTA's own.  CTAs exchange the sums of groups of 32 bins; the bins of the one group that matters
  // are then read from all of them.
  auto find = [&](int pass, bool all) {
    int* hist = s_hist[pass];
    const int ctas = all ? S : 1;
    for (int c = warp; c < SEL_BINS / 32; c += SEL_WARPS) {
      const int sum = __reduce_add_sync(0xffffffffu, hist[c * 32 + lane]);
      if (lane < ctas) *(all ? cluster.map_shared_rank(&s_groups[pass][rank][c], lane) : &s_groups[pass][0][c]) = sum;
    }
    if (all) sync(); else __syncthreads();
    if (warp == 0) {
      static_assert(SEL_BINS / 32 == 64, "a lane has two groups");
      int lo = 0, hi = 0;     // of groups 2 * lane and 2 * lane + 1
      for (int r = 0; r < ctas; r++) {
        lo += s_groups[pass][r][2 * lane];
        hi += s_groups[pass][r][2 * lane + 1];
      }
      auto from_top = [&](int x) {   // sum over this lane and those above
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_down_sync(0xffffffffu, x, o);
          if (lane + o < 32) x += y;
        }
        return x;
      };
      auto holder = [&](int top) {   // the highest lane at which it reaches `want`
        const unsigned m = __ballot_sync(0xffffffffu, top >= want);
        return m ? 31 - __clz(m) : 0;
      };
      const int top = from_top(lo + hi), l = holder(top);
      int above = __shfl_sync(0xffffffffu, top - lo - hi, l);
      const int upper = __shfl_sync(0xffffffffu, hi, l);
      const bool in_upper = above + upper >= want;
      if (!in_upper) above += upper;
      const int g = 2 * l + in_upper;
      int bin = 0;
      for (int r = 0; r < ctas; r++) bin += (all ? cluster.map_shared_rank(hist, r) : hist)[g * 32 + lane];
      const int fine = above + from_top(bin), f = holder(fine);
      if (lane == f) {
        s_found[0] = g * 32 + f;
        s_found[1] = want - (fine - bin);
        s_found[2] = bin;
      }
    }
    __syncthreads();
  };
  auto take = [&](int sh, uint32_t low) {
    prefix |= (uint32_t)s_found[0] << sh;
    mask |= low << sh;
    want = s_found[1];
    in_bin = s_found[2];
  };
  int sh = 21, pass = 0;
  bool listed = false;
#pragma unroll 1
  for (; pass < 3 && in_bin != want; pass++) {
    const uint32_t low = pass < 2 ? 2047u : 1023u;
    int* hist = s_hist[pass];
    if (pass > 0 && in_bin <= SEL_LIST) {
      listed = true;
      break;
    }
    each([&](int, uint32_t k, uint32_t, bool in) { count(hist, k, in && (k & mask) == prefix, sh, low); });
    __syncthreads();
    find(pass, true);
    take(sh, low);
    sh = pass == 0 ? 10 : 0;
    __syncthreads();   // s_found is read before it is written again
  }
  if (listed) {
    each([&](int, uint32_t k, uint32_t, bool in) {
      const bool counts = in && (k & mask) == prefix;
      const unsigned m = __ballot_sync(0xffffffffu, counts);
      if (m == 0) return;
      int at = 0;
      if (lane == __ffs(m) - 1) at = atomicAdd(&s_listed, __popc(m));
      at = __shfl_sync(0xffffffffu, at, __ffs(m) - 1) + __popc(m & ((1u << lane) - 1u));
      if (counts) s_list[at] = k;
    });
    sync();
    // all CTAs' lists, in_bin keys in all
    for (int r = 0, base = 0; r < S; r++) {
      const int some = *cluster.map_shared_rank(&s_listed, r);
      const uint32_t* list = cluster.map_shared_rank(s_list, r);
      for (int i = tid; i < some; i += SEL_THREADS) s_gathered[base + i] = list[i];
      base += some;
    }
    __syncthreads();
    const int listed_keys = in_bin;
#pragma unroll 1
    for (; pass < 3 && in_bin != want; pass++) {
      const uint32_t low = pass < 2 ? 2047u : 1023u;
      for (int j0 = warp * 32; j0 < listed_keys; j0 += SEL_THREADS) {
        const int j = j0 + lane;
        const uint32_t k = j < listed_keys ? s_gathered[j] : 0u;
        count(s_hist[pass], k, j < listed_keys && (k & mask) == prefix, sh, low);
      }
      __syncthreads();
      find(pass, false);
      take(sh, low);
      sh = pass == 0 ? 10 : 0;
      __syncthreads();
    }
  }
  const bool ties = in_bin != want;   // else all of them are kept: every key >= prefix

  // the CTAs' counts of one quantity, told to the cluster; the sum over the CTAs before this one
  auto before_cta = [&](int which) {
    int sum = 0;
    for (int r = 0; r < rank; r++) sum += s_count[which][r];
    return sum;
  };
  auto tell = [&](int which, int mine) {
    if (tid < S) *cluster.map_shared_rank(&s_count[which][rank], tid) = mine;
  };
  int equal = 0;              // with ties: equal keys in slots before the warp's
  if (ties) {
    int cnt = 0;
    each([&](int, uint32_t k, uint32_t, bool in) { cnt += __popc(__ballot_sync(0xffffffffu, in && k == prefix)); });
    if (lane == 0) s_warp[warp] = cnt;
    __syncthreads();
    const int w = lane < SEL_WARPS ? s_warp[lane] : 0;
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    tell(0, __reduce_add_sync(0xffffffffu, w));
    sync();
    equal += before_cta(0);
  }
  // f(slot, its page, lanes whose slot is a gap, lanes whose slot moves) for the warp's slots in order
  auto each_flagged = [&](auto f) {
    int seen = equal;
    each([&](int j, uint32_t k, uint32_t pg, bool in) {
      bool keep = in && k >= prefix;
      if (ties) {
        const unsigned same = __ballot_sync(0xffffffffu, in && k == prefix);
        keep = in && (k > prefix || (k == prefix && seen + __popc(same & ((1u << lane) - 1u)) < want));
        seen += __popc(same);
      }
      f(j, k, pg, __ballot_sync(0xffffffffu, in && j < budget && !keep),
        __ballot_sync(0xffffffffu, in && j >= budget && keep));
    });
  };
  int gaps = 0, movers = 0;
  each_flagged([&](int, uint32_t, uint32_t, unsigned g, unsigned m) {
    gaps += __popc(g);
    movers += __popc(m);
  });
  if (lane == 0) {
    s_gaps[warp] = gaps;
    s_movers[warp] = movers;
  }
  __syncthreads();
  const int wg = lane < SEL_WARPS ? s_gaps[lane] : 0, wm = lane < SEL_WARPS ? s_movers[lane] : 0;
  int gap_at = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0);
  int mover_at = __reduce_add_sync(0xffffffffu, lane < warp ? wm : 0);
  tell(1, __reduce_add_sync(0xffffffffu, wg));
  tell(2, __reduce_add_sync(0xffffffffu, wm));
  sync();
  gap_at += before_cta(1);
  mover_at += before_cta(2);
  if (rank == 0 && tid == 0) {
    int all = 0;
    for (int r = 0; r < S; r++) all += s_count[1][r];
    a.count[b] = all;         // as many gaps below the budget as kept slots from there on
    a.new_lens[b] = budget;
  }
  each_flagged([&](int j, uint32_t, uint32_t pg, unsigned g, unsigned m) {
    const unsigned bit = 1u << lane;
    if ((g | m) & bit) {      // a slot that has a page: see KEY_NO_PAGE
      const uint32_t flat = (pg << shift) + (j & (ps - 1));
      if (g & bit) a.to[b * a.moves + gap_at + __popc(g & (bit - 1u))] = flat;
      else a.from[b * a.moves + mover_at + __popc(m & (bit - 1u))] = flat;
    }
    gap_at += __popc(g);
    mover_at += __popc(m);
  });
  // (nobody has touched another CTA's shared memory since the last sync: each may leave)
}

// Moves the kept rows into the gaps.  Sources lie at or above slot `budget`, destinations below it,
// so rows move in any order.  LPR lanes of 16 bytes a (token, head), K and V; rows are taken in the
// order (32 moves, head, move), so that neighbours share a page's part of a head.  HBM-bound, on
// pieces of 128 bytes or more in no order: 34 MB read and written in about 14 us.  One piece a thread
// at a time and all 2048 threads of a SM measured best (two or four pieces, fewer threads: 0.1 to 2 us
// longer; more CTAs than fit at once: 1 us, all of it their launch).
template <int LPR>
__global__ void __launch_bounds__(256, 8) evict_move_kernel(const Evict a, int ctas) {
  constexpr int R = 256 / LPR;
  after_previous();
  const int64_t b = blockIdx.x / ctas;
  const int part = (int)(blockIdx.x % ctas), H = a.c.H, shift = a.c.ps_shift, ps = 1 << shift;
  const int sub = threadIdx.x % LPR;
  const int64_t count = a.count[b], items = (count + 31) / 32 * 32 * H;
  const uint32_t *tos = a.to + b * a.moves, *froms = a.from + b * a.moves;
  uint4 *k = static_cast<uint4*>(a.c.k) + sub, *v = static_cast<uint4*>(a.c.v) + sub;
  for (int64_t x = (int64_t)part * R + threadIdx.x / LPR; x < items; x += (int64_t)ctas * R) {
    const int64_t g = x / 32, c = div_by(g, H), m = c * 32 + x % 32;
    if (m >= count) continue;
    const uint32_t h = (uint32_t)(g - c * H), to = tos[m], from = froms[m];
    const uint32_t rt = ((to >> shift) * H + h << shift) + (to & (ps - 1));
    const uint32_t rf = ((from >> shift) * H + h << shift) + (from & (ps - 1));
    const uint4 kr = __ldcs(k + (int64_t)rf * LPR), vr = __ldcs(v + (int64_t)rf * LPR);
    if (sub == 0) {
      a.c.weights[rt] = a.c.weights[rf];
      if (h == 0) {
        a.c.positions[to] = a.c.positions[from];
        if (a.c.timestamps) a.c.timestamps[to] = a.c.timestamps[from];
      }
    }
    __stcs(k + (int64_t)rt * LPR, kr);
    __stcs(v + (int64_t)rt * LPR, vr);
  }
}

// ------------------------------------------------------------------------------------------------
// Launchers (arguments already checked)
// ------------------------------------------------------------------------------------------------

// Launches a kernel of this file (see after_previous), `cluster` CTAs a cluster.
template <typename... P, typename... A>
hstu_status_t launch(void (*kern)(P...), int64_t grid, int threads, int smem, int cluster, cudaStream_t st,
                     A... args) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  if (!succeeded(cudaLaunchKernelEx(&cfg, kern, P(args)...))) return HSTU_ERR_CUDA;
  count_launch();
  return HSTU_OK;
}

inline bool head_dim_supported(int dtype, int hd) {
  return dtype == HSTU_BF16 ? hd == 64 || hd == 128 : hd == 32 || hd == 64 || hd == 128;
}

inline size_t attention_workspace_bytes(int hd) {
  return (size_t)ATTN_MAX_CTAS * (2 * hd * sizeof(float) + sizeof(Part));
}

template <typename T, int HD>
hstu_status_t launch_attention_t(const Attn& a, void* ws, int sms, cudaStream_t st) {
  constexpr int TILE = AttnCfg<T, HD>::TILE, SMEM = AttnCfg<T, HD>::SMEM;
  // no more CTAs than give each warp one tile of the longest announced length; tiles are counted
  // in 32 bits
  const int64_t tiles = a.B * a.c.H * (a.max_len / TILE + 1);
  if (a.max_len >= (1LL << 30) || tiles >= (1LL << 31)) return HSTU_ERR_UNSUPPORTED;
  int64_t grid = (tiles + ATTN_WARPS - 1) / ATTN_WARPS;
  if (grid > sms) grid = sms;
  if (grid > ATTN_MAX_CTAS) grid = ATTN_MAX_CTAS;
  float* parts = static_cast<float*>(ws);
  Part* recs = reinterpret_cast<Part*>(parts + (size_t)ATTN_MAX_CTAS * 2 * HD);
  auto kern = attention_kernel<T, HD>;
  if (!succeeded(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)))
    return HSTU_ERR_CUDA;
  const hstu_status_t rc = launch(kern, grid, ATTN_THREADS, SMEM, 0, st, a, parts, recs);
  // one CTA joins its warps' parts itself, and a single tile a (sequence, head) has no parts
  if (rc != HSTU_OK || grid == 1 || a.max_len < TILE) return rc;
  return launch(attention_join_kernel<HD>, grid, ATTN_MAX_CTAS, 0, 0, st, a.av, parts, recs, (int)grid);
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

inline hstu_status_t launch_append(const Cache& c, int row_bytes, int64_t T, int64_t B,
                                   const void* uvqk, const int64_t* off, const int64_t* ts,
                                   const int32_t* table, int64_t max_pages, const int64_t* lens,
                                   const int64_t* next_pos, cudaStream_t st) {
  // about APPEND_PIECES pieces of K a CTA: wide rows in small groups, so that the SMs get even shares
  int tokens = APPEND_PIECES / (c.H * (row_bytes / 16));
  tokens = tokens < 1 ? 1 : tokens > APPEND_TOKENS ? APPEND_TOKENS : tokens;
  if ((T + tokens - 1) / tokens >= (1LL << 31)) return HSTU_ERR_UNSUPPORTED;
  auto kern = row_bytes == 128 ? append_kernel<8> : row_bytes == 256 ? append_kernel<16> : append_kernel<32>;
  return launch(kern, (T + tokens - 1) / tokens, 256, 0, 0, st, c, tokens, T, B,
                static_cast<const uint4*>(uvqk), off, ts, table, max_pages, lens, next_pos);
}

// Allows the selection clusters of SEL_CLUSTER CTAs, which are more than every device has to offer;
// says whether the current device has room for one (a GPU partition may not).  That is asked once a
// device, and before anything is launched; the permission belongs to the context and is given anew.
inline bool wide_clusters_fit() {
  static std::atomic<int> known[64];   // 0: not asked yet, 1: no, 2: yes
  int dev = 0, clusters = 0;
  if (!succeeded(cudaGetDevice(&dev)) ||
      !succeeded(cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)))
    return false;
  std::atomic<int>* slot = dev < 64 ? &known[dev] : nullptr;
  if (slot && slot->load()) return slot->load() == 2;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = SEL_CLUSTER;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(SEL_CLUSTER);
  cfg.blockDim = dim3(SEL_THREADS);
  cfg.dynamicSmemBytes = SEL_SMEM;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool fit = succeeded(cudaOccupancyMaxActiveClusters(&clusters, evict_select_kernel, &cfg)) && clusters > 0;
  if (slot) slot->store(fit ? 2 : 1);
  return fit;
}

inline hstu_status_t launch_evict(const Evict& a, int row_bytes, int sms, cudaStream_t st) {
  // As many CTAs as hold the keys of a row's slots, and more while there are SMs for them, up to 8
  // (8192 slots 15.2 us an eviction, with four 16.2; 16 384 17.0, 20.0).  Rows of more slots than eight
  // CTAs score in one go get 16 for a few sequences: below that their wider barriers cost more (24 576
  // slots 19.2 us, with eight 18.9; 28 672 19.7, 19.9; 32 768 20.1, 20.8; 40 960 21.0, 25.8; 100 000 28.3,
  // 46.8, one history as six).  Seven such clusters fit the GPU at once, an eighth waits (32 768 slots 38).
  int S = 1;
  while (S < 8 && ((int64_t)S * SEL_THREADS * SEL_ROUNDS < a.room || 2 * S * a.B <= sms)) S *= 2;
  if (!succeeded(cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SEL_SMEM)))
    return HSTU_ERR_CUDA;
  if (8LL * SEL_THREADS * SEL_KEYS < a.room && 3 * SEL_CLUSTER * a.B <= 2 * sms && wide_clusters_fit())
    S = SEL_CLUSTER;
  const hstu_status_t rc = launch(evict_select_kernel, a.B * S, SEL_THREADS, SEL_SMEM, S, st, a);
  if (rc != HSTU_OK) return rc;
  // what fits the SMs at once, over all sequences; at least one each
  const int64_t ctas = (8LL * sms + a.B - 1) / a.B;
  auto kern = row_bytes == 128 ? evict_move_kernel<8> : row_bytes == 256 ? evict_move_kernel<16> : evict_move_kernel<32>;
  return launch(kern, a.B * ctas, 256, 0, 0, st, a, (int)ctas);
}

}  // namespace paged
}  // namespace hstu
