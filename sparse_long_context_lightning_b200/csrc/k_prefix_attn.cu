// Dense absorbed-MQA attention of a batch behind one shared prefix, each query with its own tokens in pages.
//
//   o = sum_k e^{scale q.k - m} v_k / l,  l = sum_k e^{scale q.k - m},  lse = m + ln l,  v = the first 512 dims of k,
// over the Lp rows of the prefix (the same for every query) and own_len[b] rows behind them (block table).
//
// The batch's B * H query rows are cut into tiles of 128, whatever H is, and every tile walks the prefix in blocks of
// 128 keys, then the blocks of its own queries' pages, with one running maximum and sum per row.  2 (576 + 512) flops a
// (row, key) against 1152 bytes a key: from about 190 rows on the matrix units bound it, below that the prefix's bytes.
//
// A CTA pair (cluster of two, tcgen05 cta_group::2, M = 128) takes a tile: each CTA has 64 rows of Q, their logits,
// probabilities and output, so the softmax never leaves the CTA, and feeds half of every B operand: 64 of a block's 128
// keys for S = Q K^T (N = 128) and 256 of the 512 value dims for O += P V (two N = 256 instructions a 16 keys).  A
// 128 x 512 fp32 output would fill a CTA's tensor memory; the pair's 64 rows a CTA take half of it and leave room for
// four buffers of S, so the logits run ahead of the softmax.  The same bytes cannot serve as keys and as values here
// (one descriptor gives both CTAs' halves of B, and the halves are cut along different axes), so a block is loaded
// twice, 1088 bytes a key and CTA, the second time from L2.  Keys arrive in stages of 64 keys x 192 dims (three a
// block) and values in stages of 32 keys, each by one instruction of a three-dimensional map: a warp that issues a load
// waits about 200 clocks before its next, so nine small loads a block held the block at 3750 clocks.  With 64-key
// blocks (N = 64, A read again for each, 22.6 clocks a key and SM against 17.0) the decode batch below took 529 us against
// 470, both before pairs walked in step.  Prefetching blocks into the L2 ahead of the loads gained 2.5 us for one query
// behind 131072 rows and cost the other cases 0.2 to 0.4 us: left out.
// 16 queries of 128 heads behind 131072 rows: 400 us (1460 TFLOP/s, matrix units busy 84% of the time), 470 to 485 us when
// run for seconds, where the power limit holds the clock (1205 to 1245 TFLOP/s; cuBLAS sustains 1385 there).  64 queries
// behind 32749 rows: 403 us, 470 to 487 sustained.  One query of 128 heads behind 131072 rows: 46 to 49 us in a graph, 54
// through a call, of which 28 in the loop (5.4 TB/s from HBM) and 21 in start, partials and join.  4 queries of 16 heads
// behind 1024 rows: 13 us, all latency.
//
// Work is cut evenly: the blocks of all tiles, in order, are one line that 74 pairs divide; a tile that spans pairs
// leaves partial sums (fp32) that a second kernel joins, and one that lies in a pair is written at once (74 queries of 128
// heads with 1000 own tokens each: 30.5 us against 50.3 through partials).  Where a tile holds several queries (H not a multiple of 128),
// each query's own blocks are an accumulation of their own, so that a row never multiplies another sequence's values.
#include <algorithm>

#include "lsa_common.cuh"
#include "sm100_pair.cuh"

namespace lsa {
namespace {

using namespace sm100;

__device__ int g_prefix_timeout;  // set when a bounded wait gave up
__device__ int g_prefix_check;    // set when own_len was outside [0, the table's columns * page] or a page id was bad

constexpr int PA_THREADS = 384;
constexpr int PA_KQ_WARP = 0, PA_QK_WARP = 1, PA_PV_WARP = 2, PA_V_WARP = 3, PA_SM_WARP = 4, PA_SM_WARPS = 8;
constexpr int PA_PAIRS = 74;  // one pair on every two of the 148 SMs
constexpr int PA_T = 128;     // keys of a block
constexpr int PA_ROWS = 128;  // query rows of a tile
constexpr int PA_NK = 3, PA_NV = 4;  // stages
constexpr int PA_NS = 4, PA_NP = 1;  // buffers of S and of P
constexpr int PA_Q_KB = 64 * 128;        // 64 rows x 64 dims
constexpr int PA_Q_BYTES = 9 * PA_Q_KB;  // 72 KB
constexpr int PA_P_KB = 64 * 128;        // 64 rows x 64 keys
constexpr int PA_P_BYTES = 2 * PA_P_KB;
constexpr int PA_KT = PA_T / 2;          // keys of a block that this CTA feeds to S
constexpr int PA_KS = 3;                 // 64-dim parts of a stage of keys
constexpr int PA_K_KB = PA_KT * 128;     // 64 keys x 64 dims
constexpr int PA_K_BYTES = PA_KS * PA_K_KB;
constexpr int PA_VT = 32;                // keys of a stage of values
constexpr int PA_V_KB = PA_VT * 128;     // 32 keys x 64 dims
constexpr int PA_V_BYTES = 4 * PA_V_KB;
constexpr int PA_SMEM = PA_Q_BYTES + PA_NP * PA_P_BYTES + PA_NK * PA_K_BYTES + PA_NV * PA_V_BYTES + 2 * 1024 + 512;
static_assert(PA_SMEM <= 232448, "shared memory");
constexpr uint32_t PT_O = 0, PT_S = 256;  // TMEM columns: O [0, 256), S buffers of 64 from 256
constexpr uint32_t IDESC_QK = idesc_mma(128, PA_T, 1u, 0u);
constexpr uint32_t IDESC_PV2 = idesc_mma(128, 256, 1u, 1u);
constexpr int PA_END = 1;  // what an own item's end counts for when the work is cut, in blocks
constexpr float PA_RESCALE = 8.f;
constexpr int PA_NO_ROW = 0x7FFFFF00;  // behind every map's last row: the box reads as zeros

struct PaArgs {
  const int32_t* own_len;  // [B], or NULL: no own tokens
  const int32_t* table;    // [B, table_ld] page ids
  int64_t table_ld;
  int page_shift;  // log2 of the page size
  int kbox, vbox;  // rows of a page box: min(page, 64 or 32) of keys, min(page, 32) of values
  int n_pages;
  int cap;  // most own tokens: the table's columns * page (clamped to int)
  int H;
  int64_t BH;
  int nT;     // tiles
  int multi;  // tiles may hold rows of several queries
  int64_t Lp;
  int nP;  // prefix blocks
  float scale_log2;
  int2* seg;      // [items] first and last pair of an item; last = -2: written to out already
  float2* ws_ml;  // [partial rows] running max (log2 units), sum
  float* ws_o;    // [partial rows][512]
  uint16_t* out;
  float* lse;
};

// A span: the blocks that one pair walks of a tile's prefix or of one query's pages.  What depends on own_len is read
// once a span (a load a block cost the softmax 780 clocks of 2100).
// Items: a tile where all rows belong to one query; else a tile's prefix part, and each of its queries' own part.
// Of the items that a pair has blocks of, only the first can have begun in an earlier pair.  So a pair has 128 rows for the
// partial of such an item, and the pair in which an item begins writes to rows of the item's own: row r of the queries has
// one for the prefix part (or the whole tile) and one for its query's own part.
// The line counts units: a block is one, and the end of a query's own item (its last products awaited, its rows stored)
// counts for PA_END more: 45.3 -> 42.2 us for 33 queries of 32 heads with up to 2000 own tokens (2 units: 41.1 there, but
// 15.2 -> 15.9 where the items are one block each).
struct Cursor {
  int t, b;  // tile; query whose own blocks are walked, or -1: the prefix
  int pos, cnt;  // units
  int len;       // keys of the prefix or of the query's pages
  int blocks;    // of the prefix or of the query's pages: the units that are blocks
  int real;      // blocks of the span
  int turn, wrap;  // of the span: where the walk begins
  int qlo, qhi;

  static __device__ __forceinline__ int len_of(const PaArgs& a, int b) {
    if (a.own_len == nullptr) return 0;
    return min(max(__ldg(a.own_len + b), 0), a.cap);
  }
  static __device__ __forceinline__ int blocks_of(const PaArgs& a, int b) { return (len_of(a, b) + PA_T - 1) / PA_T; }
  static __device__ __forceinline__ int units(const PaArgs& a, int blocks) {  // of an own part
    return blocks + (a.multi && blocks > 0 ? PA_END : 0);
  }
  __device__ __forceinline__ void tile(const PaArgs& a, int tt) {
    t = tt;
    b = -1;
    cnt = blocks = a.nP;
    len = static_cast<int>(a.Lp);
    const uint32_t r0 = static_cast<uint32_t>(tt) * PA_ROWS, h = static_cast<uint32_t>(a.H);  // rows fit 31 bits
    qlo = static_cast<int>(r0 / h);
    qhi = static_cast<int>((min(r0 + PA_ROWS, static_cast<uint32_t>(a.BH)) - 1) / h);
  }
  __device__ __forceinline__ void settle(const PaArgs& a) {  // to the unit that `pos` counts up to; one must be left
    while (pos >= cnt) {
      pos -= cnt;
      b = b < 0 ? qlo : b + 1;
      if (b <= qhi) {
        len = len_of(a, b);
        blocks = (len + PA_T - 1) / PA_T;
        cnt = units(a, blocks);
      } else if (t + 1 < a.nT) {
        tile(a, t + 1);
      } else {  // not reached unless own_len changed since the blocks were counted: rows outside the maps, zeros
        b = -1;
        cnt = blocks = 0x7FFFFFFF;
      }
    }
  }
  __device__ __forceinline__ void start(const PaArgs& a, int tt, int off) {
    tile(a, tt);
    pos = off;
    settle(a);
  }
  // The units of the span that begins after u of the pair's n, and its blocks (`real`).  A prefix span is walked from the
  // block that is u modulo n, and round: pairs at the same u then read the same few places of the prefix whichever tile
  // they work on, so that a prefix larger than the L2 comes from HBM about once (n differs by one between pairs at most):
  // 16 queries of 128 heads behind 131072 rows (151 MB) 458 -> 398 us.
  __device__ __forceinline__ int span(int u, int n) {
    const int w = min(n - u, cnt - pos);
    real = min(w, max(blocks - pos, 0));
    turn = 0;
    wrap = 0x7FFFFFFF;
    if (b < 0) {
      int r = (u - pos) % n;
      if (r < 0) r += n;
      if (r < real) {
        turn = r;
        wrap = pos + real;
      }
    }
    return w;
  }
  __device__ __forceinline__ int block() const {
    const int x = pos + turn;
    return x >= wrap ? x - real : x;
  }
  __device__ __forceinline__ int id(const PaArgs& a) const {
    return !a.multi ? t : (b < 0 ? qlo + 2 * t : b + 2 * t + 1);
  }
  // blocks of the item before `pos`, and behind it
  __device__ __forceinline__ int item_pos(const PaArgs& a) const { return a.multi || b < 0 ? pos : a.nP + pos; }
  __device__ __forceinline__ int item_left(const PaArgs& a) const {
    return max(blocks - pos, 0) + (a.multi || b >= 0 ? 0 : blocks_of(a, qlo));
  }
};

// the partial of query row r from the pair in which its item begins; the pairs' own rows lie ahead (BH < 2^31 - 2^16)
__device__ __forceinline__ uint32_t part_row(const PaArgs& a, bool own, uint32_t r) {
  return PA_PAIRS * PA_ROWS + (own ? static_cast<uint32_t>(a.BH) : 0u) + r;
}

__device__ __forceinline__ int tile_units(const PaArgs& a, int t) {
  Cursor c;
  c.tile(a, t);
  int n = a.nP;
  if (a.own_len) {
    #pragma unroll 4
    for (int b = c.qlo; b <= c.qhi; ++b) n += Cursor::units(a, Cursor::blocks_of(a, b));
  }
  return n;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PA_THREADS, 1)
    k_prefix_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pk,
                  const __grid_constant__ CUtensorMap tm_pv, const PaArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* q_s = smem_raw;
  unsigned char* p_s = q_s + PA_Q_BYTES;
  unsigned char* k_s = p_s + PA_NP * PA_P_BYTES;
  unsigned char* v_s = k_s + PA_NK * PA_K_BYTES;
  float* mx = reinterpret_cast<float*>(v_s + PA_NV * PA_V_BYTES);  // [2][256]: row maxima of a block, row sums
  uint64_t* q_full = reinterpret_cast<uint64_t*>(mx + 2 * 256);
  uint64_t* q_empty = q_full + 3;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + PA_NK;
  uint64_t* v_full = k_empty + PA_NK;
  uint64_t* v_empty = v_full + PA_NV;
  uint64_t* s_full = v_empty + PA_NV;
  uint64_t* s_empty = s_full + PA_NS;
  uint64_t* p_full = s_empty + PA_NS;
  uint64_t* pv_done = p_full + PA_NP;
  uint64_t* vt_full = pv_done + PA_NP;  // this CTA's values of a stage whose last page is partly filled
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(vt_full + 1);
  int* start_s = reinterpret_cast<int*>(tmem_holder + 1);  // this pair's first tile, unit of it, number of units
  int* abort_flag = start_s + 3;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1);

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&q_full[i], 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < PA_NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < PA_NV; ++i) {
      mbar_init(&v_full[i], 2);  // one arrival a CTA
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < PA_NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 2 * PA_SM_WARPS);  // the softmax warps of both CTAs
    }
    for (int i = 0; i < PA_NP; ++i) {
      mbar_init(&p_full[i], 2 * PA_SM_WARPS);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(vt_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_pk);
    tma_prefetch_desc(&tm_pv);
  }
  if (warp == PA_PV_WARP) tmem_alloc_pair(tmem_holder, 512);
  tc_fence_before();
  cluster_sync_all();  // the barriers and the tensor memory of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // every global access of this kernel comes after the previous kernel of the stream has completed
  pdl_wait();
  pdl_launch_dependents();

  // ---- this pair's part of the line: its first tile, unit of it, and number of units.  Up to 32 tiles, every warp finds
  // it alone (a lane a tile); beyond, thread i sums the tiles [i * per, (i + 1) * per) and the warps meet.
  int tile0 = 0, unit0 = 0, n = 0;
  {
    const int per = a.nT <= 32 ? 1 : (a.nT + PA_THREADS - 1) / PA_THREADS;
    const int me = a.nT <= 32 ? lane : tid;
    const int lo = min(me * per, a.nT), hi = min(lo + per, a.nT);
    int64_t mine = 0;
    for (int t = lo; t < hi; ++t) mine += tile_units(a, t);
    int64_t inc = mine;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    int64_t before = inc - mine, total = __shfl_sync(0xffffffffu, inc, 31);
    if (a.nT > 32) {
      int64_t* sums = reinterpret_cast<int64_t*>(mx);
      if (lane == 31) sums[warp] = inc;
      __syncthreads();
      total = 0;
      for (int w = 0; w < PA_THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
      }
    }
    const int np = static_cast<int>(min(static_cast<int64_t>(PA_PAIRS), total));
    if (pair < np) {
      int64_t s0, s1;
      if (total < (1 << 24)) {  // a 64-bit division takes as long as a load
        s0 = static_cast<uint32_t>(total) * pair / np;
        s1 = static_cast<uint32_t>(total) * (pair + 1) / np;
      } else {
        s0 = total * pair / np;
        s1 = total * (pair + 1) / np;
      }
      n = static_cast<int>(s1 - s0);
      const bool here = s0 >= before && s0 < before + mine;
      if (a.nT <= 32) {
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        tile0 = src;
        unit0 = static_cast<int>(s0 - __shfl_sync(0xffffffffu, before, src));
      } else if (here) {
        int64_t off = s0 - before;
        int t = lo;
        for (int k = tile_units(a, t); off >= k && t + 1 < hi; k = tile_units(a, t)) {
          off -= k;
          ++t;
        }
        start_s[0] = t;
        start_s[1] = static_cast<int>(off);
      }
    }
    // Through shared memory in either case: with the three in the registers that they were found in, the loops of the
    // matrix instructions came out slower (64 queries behind 32749 rows 406 -> 446 us).
    if (tid == 0) {
      if (a.nT <= 32) {
        start_s[0] = tile0;
        start_s[1] = unit0;
      }
      start_s[2] = n;
    }
    __syncthreads();
    tile0 = start_s[0];
    unit0 = start_s[1];
    n = start_s[2];
  }
  Cursor c;
  if (n > 0) c.start(a, tile0, unit0);
  bool ok = true;

  if (warp == PA_KQ_WARP) {
    // ------------------------------------------------------------------ Q and keys: stages of 64 keys x 192 dims
    int loaded = -1, nq = 0;
    uint32_t s = 0, phase = 1;
    // the page of this lane's box among this CTA's keys of own block p, or -1; asked for a block ahead
    auto page_of = [&](int p) {
      const int key = PA_T * p + PA_KT * static_cast<int>(rank) + lane * a.kbox;
      return lane * a.kbox < PA_KT && key < c.len ? a.table[static_cast<int64_t>(c.b) * a.table_ld + (key >> a.page_shift)] : -1;
    };
    for (int u = 0; u < n && ok;) {
      const int w = c.span(u, n), end = c.pos + c.real;
      int pg_next = c.b >= 0 && c.real > 0 ? page_of(c.pos) : -1;
      for (; c.pos < end && ok; ++c.pos) {
        const int key0 = PA_T * c.block() + PA_KT * static_cast<int>(rank);
        // a box past the end reads as zeros: a row outside the map
        int y = PA_NO_ROW;
        if (c.b >= 0) {
          const int pg = pg_next;
          if (c.pos + 1 < end) pg_next = page_of(c.pos + 1);
          if (pg >= 0 && pg < a.n_pages) y = (pg << a.page_shift) + ((key0 + lane * a.kbox) & ((1 << a.page_shift) - 1));
        }
        const bool one = elect_one();
        const bool fresh = c.t != loaded;
        if (fresh) {
          ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (nq & 1) ^ 1));
          if (!ok) break;
          loaded = c.t;
          ++nq;
        }
        for (int j = 0; j < 9; j += PA_KS) {
          ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[s], phase));
          if (!ok) break;
          const uint32_t bar = mapa(smem_u32(&k_full[s]), 0);
          unsigned char* dst = k_s + s * PA_K_BYTES;
          if (fresh && one) {  // the tile's queries arrive in the same parts as its first keys
            if (rank == 0) mbar_expect_tx(&q_full[j / PA_KS], 2 * PA_KS * PA_Q_KB);
            tma_load_3d_pair(q_s + j * PA_Q_KB, &tm_q, mapa(smem_u32(&q_full[j / PA_KS]), 0), 0,
                             c.t * PA_ROWS + 64 * static_cast<int>(rank), j);
          }
          if (one && rank == 0) mbar_expect_tx(&k_full[s], 2 * PA_K_BYTES);
          if (c.b < 0) {
            if (one) tma_load_3d_pair(dst, &tm_k, bar, 0, key0, j);
          } else {
            if (a.kbox == PA_KT) {
              const int y0 = __shfl_sync(0xffffffffu, y, 0);
              if (one) tma_load_3d_pair(dst, &tm_pk, bar, 0, y0, j);
            } else {
              for (int r = 0; r * a.kbox < PA_KT; ++r) {
                const int yr = __shfl_sync(0xffffffffu, y, r);
                if (one)
                  for (int e = 0; e < PA_KS; ++e)
                    tma_load_3d_pair(dst + e * PA_K_KB + r * a.kbox * 128, &tm_pk, bar, 0, yr, j + e);
              }
            }
          }
          __syncwarp();
          if (++s == PA_NK) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      c.pos += w - c.real;
      u += w;
      if (u < n && ok) c.settle(a);
    }
  } else if (warp == PA_V_WARP) {
    // ------------------------------------------------------------------ values: this CTA's 256 dims, stages of 32 keys
    int ntail = 0, tail_s = -1, tail_valid = 0;
    uint32_t s = 0, phase = 1;
    auto page_of = [&](int p) {
      const int key = PA_T * p + lane * a.vbox;
      return lane * a.vbox < PA_T && key < c.len ? a.table[static_cast<int64_t>(c.b) * a.table_ld + (key >> a.page_shift)] : 0;
    };
    // Rows of a partly filled box behind the sequence's end hold anything (NaN too) and would meet p = 0 in the product:
    // such a stage lands on this CTA's own barrier, and before this warp next waits for a free stage it zeroes the rows
    // and hands the stage over.
    auto hand_over = [&]() {
      ok = __all_sync(0xffffffffu, mbar_wait(vt_full, ntail & 1));
      if (!ok) return;
      ++ntail;
      unsigned char* dst = v_s + tail_s * PA_V_BYTES;
      const int rows = (tail_valid + a.vbox - 1) / a.vbox * a.vbox - tail_valid;
      for (int x = lane; x < 4 * rows * 8; x += 32) {
        const int j = x / (rows * 8), e = x - j * rows * 8;
        *reinterpret_cast<uint4*>(dst + j * PA_V_KB + tail_valid * 128 + e * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (elect_one()) mbar_arrive_pair(mapa(smem_u32(&v_full[tail_s]), 0));
      __syncwarp();
      tail_s = -1;
    };
    for (int u = 0; u < n && ok;) {
      const int w = c.span(u, n), end = c.pos + c.real;
      int pg_next = c.b >= 0 && c.real > 0 ? page_of(c.pos) : 0;
      for (; c.pos < end && ok; ++c.pos) {
        const int key0 = PA_T * c.block();
        int y = PA_NO_ROW;
        if (c.b >= 0) {
          const int pg = pg_next, key = key0 + lane * a.vbox;
          if (c.pos + 1 < end) pg_next = page_of(c.pos + 1);
          if (lane * a.vbox < PA_T && key < c.len) {
            if (pg >= 0 && pg < a.n_pages) y = (pg << a.page_shift) + (key & ((1 << a.page_shift) - 1));
            else atomicExch(&g_prefix_check, 1);
          }
        }
        const bool one = elect_one();
        for (int k = 0; k < PA_T && key0 + k < c.len; k += PA_VT) {
          const int valid = min(PA_VT, c.len - key0 - k);
          const bool tail = c.b >= 0 && (valid & (a.vbox - 1)) != 0;
          if (tail_s >= 0 && (tail || !__all_sync(0xffffffffu, mbar_test_wait(&v_empty[s], phase)))) hand_over();
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&v_empty[s], phase));
          if (!ok) break;
          unsigned char* dst = v_s + s * PA_V_BYTES;
          if (one) {
            if (tail) mbar_expect_tx(vt_full, PA_V_BYTES);
            else if (rank == 0) mbar_expect_tx(&v_full[s], 2 * PA_V_BYTES);
            else mbar_arrive_pair(mapa(smem_u32(&v_full[s]), 0));
          }
          __syncwarp();
          const uint32_t bar = tail ? mapa(smem_u32(vt_full), rank) : mapa(smem_u32(&v_full[s]), 0);
          if (c.b < 0) {
            if (one) tma_load_3d_pair(dst, &tm_v, bar, 0, key0 + k, 4 * static_cast<int>(rank));
          } else if (a.vbox == PA_VT) {
            const int y0 = __shfl_sync(0xffffffffu, y, k / PA_VT);
            if (one) tma_load_3d_pair(dst, &tm_pv, bar, 0, y0, 4 * static_cast<int>(rank));
          } else {
            for (int r = 0; r * a.vbox < PA_VT; ++r) {
              const int yr = __shfl_sync(0xffffffffu, y, k / a.vbox + r);
              if (one)
                for (int j = 0; j < 4; ++j)
                  tma_load_3d_pair(dst + j * PA_V_KB + r * a.vbox * 128, &tm_pv, bar, 0, yr, 4 * static_cast<int>(rank) + j);
            }
          }
          __syncwarp();
          if (tail) {
            tail_s = static_cast<int>(s);
            tail_valid = valid;
          }
          if (++s == PA_NV) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      c.pos += w - c.real;
      u += w;
      if (u < n && ok) c.settle(a);
    }
    if (tail_s >= 0 && ok) hand_over();
  } else if (warp == PA_QK_WARP) {
    // ------------------------------------------------------------------ S = Q K^T (issued by the even CTA)
    if (rank == 0 && n > 0 && elect_one()) {
      const uint64_t qdesc = desc_sw128(smem_u32(q_s)), kdesc = desc_sw128(smem_u32(k_s));
      int nq = 0;
      bool fresh = true;
      uint32_t s = 0, phase = 0;
      int i = 0;
      for (int u = 0; u < n && ok;) {
        const int w = c.span(u, n);
        for (const int end = i + c.real; i < end && ok; ++i, ++c.pos) {
          const int sb = i % PA_NS;
          ok = ok && mbar_wait_cluster(&s_empty[sb], ((i / PA_NS) & 1) ^ 1);
          #pragma unroll
          for (int kb = 0; kb < 9; kb += PA_KS) {
            if (fresh) ok = ok && mbar_wait_cluster(&q_full[kb / PA_KS], nq & 1);
            ok = ok && mbar_wait_cluster(&k_full[s], phase);
            if (!ok) break;
            tc_fence_after();
            #pragma unroll
            for (int kk = 0; kk < 4 * PA_KS; ++kk)
              mma_f16_pair(tmem + PT_S + sb * PA_KT, qdesc + (((kb + kk / 4) * PA_Q_KB + kk % 4 * 32) >> 4),
                           kdesc + ((s * PA_K_BYTES + kk / 4 * PA_K_KB + kk % 4 * 32) >> 4), IDESC_QK, (kb | kk) != 0);
            mma_commit_pair(&k_empty[s]);
            if (++s == PA_NK) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) mma_commit_pair(&s_full[sb]);
          if (fresh) ++nq;
          fresh = false;
        }
        c.pos += w - c.real;
        u += w;
        if (u >= n || !ok) break;
        const int t = c.t;
        c.settle(a);
        if (c.t != t && !fresh) {  // (a tile of which this pair had no block brought no queries)
          fresh = true;
          mma_commit_pair(q_empty);
        }
      }
      // no arrival of the other CTA may outlast this one
      for (int j = max(i - PA_NS, 0); j < i && ok; ++j) ok = mbar_wait_cluster(&s_empty[j % PA_NS], (j / PA_NS) & 1);
    }
  } else if (warp == PA_PV_WARP) {
    // ------------------------------------------------------------------ O += P V (issued by the even CTA)
    if (rank == 0 && n > 0 && elect_one()) {
      const uint64_t pdesc = desc_sw128(smem_u32(p_s)), vdesc = desc_sw128_mn(smem_u32(v_s), PA_V_KB, 1024);
      int item = -1;
      uint32_t s = 0, phase = 0;
      for (int u = 0, i = 0; u < n && ok;) {
        uint32_t acc = c.id(a) == item;
        item = c.id(a);
        const int w = c.span(u, n);
        for (const int end = i + c.real; i < end && ok; ++i, ++c.pos) {
          const int pb = i % PA_NP;
          ok = mbar_wait_cluster(&p_full[pb], (i / PA_NP) & 1);
          #pragma unroll
          for (int k = 0; k < PA_T / PA_VT; ++k) {
            if (PA_T * c.block() + PA_VT * k >= c.len) break;
            ok = ok && mbar_wait_cluster(&v_full[s], phase);
            if (!ok) break;
            tc_fence_after();
            #pragma unroll
            for (int kk = 0; kk < PA_VT / 16; ++kk) {
              const uint64_t pd = pdesc + ((pb * PA_P_BYTES + (k >> 1) * PA_P_KB + ((k & 1) * 2 + kk) * 32) >> 4);
              #pragma unroll
              for (int h = 0; h < 2; ++h)
                mma_f16_pair(tmem + PT_O + h * 128, pd, vdesc + ((s * PA_V_BYTES + 2 * h * PA_V_KB + kk * 2048) >> 4),
                             IDESC_PV2, acc);
              acc = 1;
            }
            mma_commit_pair(&v_empty[s]);
            if (++s == PA_NV) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) mma_commit_pair(&pv_done[pb]);
        }
        c.pos += w - c.real;
        u += w;
        if (u < n && ok) c.settle(a);
      }
    }
  } else if (n > 0) {
    // ------------------------------------------------------------------ softmax and partial sums
    // Thread (L, ch): row L % 64 of this CTA, keys [64 kh + 32 ch, + 32) of a block and value dims [256 kh + 128 ch, + 128),
    // kh = L / 64.  A wait that gave up is not waited for again, but the loop goes on: the eight warps meet at a named
    // barrier in every block.
    const int ch = (warp - PA_SM_WARP) >> 2;
    const int L = ((warp - PA_SM_WARP) & 3) * 32 + lane;
    const int row = L & 63, kh = L >> 6;
    const int trow = 64 * static_cast<int>(rank) + row;  // row of the tile
    const uint32_t tlane = tmem + (static_cast<uint32_t>(((warp - PA_SM_WARP) & 3) * 32) << 16);
    const uint32_t t_s = tlane + PT_S + 32 * ch, t_o = tlane + PT_O + 128 * ch;
    const uint32_t c_s_empty = mapa(smem_u32(s_empty), 0), c_p_full = mapa(smem_u32(p_full), 0);
    // the row's other three quarters
    auto row_max = [&](const float* m, float v) {
      return fmaxf(fmaxf(v, m[128 * (ch ^ 1) + L]), fmaxf(m[L ^ 64], m[128 + (L ^ 64)]));
    };
    float m_used = -INFINITY, l = 0.f;
    bool first = true;
    int seg_pos = c.item_pos(a);
    for (int u = 0, i = 0; u < n;) {
      // whether this thread's row is one of the span's
      const int64_t gr = static_cast<int64_t>(c.t) * PA_ROWS + trow;
      const bool live = gr < a.BH && (!a.multi || c.b < 0 || (gr >= static_cast<int64_t>(c.b) * a.H &&
                                                              gr < static_cast<int64_t>(c.b + 1) * a.H));
      const int len = live ? c.len - 64 * kh - 32 * ch : 0;
      const int w = c.span(u, n);
      for (const int end = i + c.real; i < end; ++i, ++c.pos) {
        const int sb = i % PA_NS, pb = i % PA_NP;
        const int nvalid = len - PA_T * c.block();
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[sb], (i / PA_NS) & 1));
        tc_fence_after();
        uint32_t sr[32];
        tmem_ld32(t_s + sb * PA_KT, sr);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(c_s_empty + 8 * sb);
        float z[32];
        #pragma unroll
        for (int k = 0; k < 32; ++k) z[k] = k < nvalid ? __uint_as_float(sr[k]) * a.scale_log2 : -INFINITY;
        float m4[4] = {z[0], z[1], z[2], z[3]};
        #pragma unroll
        for (int k = 4; k < 32; ++k) m4[k & 3] = fmaxf(m4[k & 3], z[k]);
        float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // the row's other keys are other warps'
        mx[256 * (i & 1) + 128 * ch + L] = mt;
        named_bar_sync(1, 32 * PA_SM_WARPS);
        mt = row_max(mx + 256 * (i & 1), mt);
        float alpha = 1.f;
        if (mt > m_used + PA_RESCALE || (first && mt > m_used)) {
          alpha = ex2_approx(m_used - mt);  // 0 from -inf
          m_used = mt;
        }
        const float m_ref = m_used == -INFINITY ? 0.f : m_used;
        uint32_t pk[16];
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
        #pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float p0 = ex2_approx(z[k] - m_ref), p1 = ex2_approx(z[k + 1] - m_ref);
          // the row's sum takes the 32-bit probabilities; P V takes them rounded to bf16 (the matrix unit's type)
          s4[(k >> 1) & 3] += p0 + p1;
          const __nv_bfloat162 p2 = __floats2bfloat162_rn(p0, p1);
          pk[k / 2] = *reinterpret_cast<const uint32_t*>(&p2);
        }
        l = l * alpha + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
        if (i >= PA_NP && ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[pb], ((i / PA_NP) - 1) & 1));
        // O changes its reference only when a maximum grew by more than 2^8 (no product is running then)
        if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[(i - 1) % PA_NP], ((i - 1) / PA_NP) & 1));
          tc_fence_after();
          #pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * k, o);
            tmem_ld_wait();
            #pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(t_o + 32 * k, o);
          }
          tmem_st_wait();
        }
        unsigned char* prow = p_s + pb * PA_P_BYTES + kh * PA_P_KB + row * 128;
        #pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(prow + (((4 * ch + e) ^ (row & 7)) << 4)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(c_p_full + 8 * pb);
        first = false;
      }
      const int id = c.id(a), left = c.item_left(a);
      const bool own = a.multi && c.b >= 0;
      c.pos += w - c.real;
      u += w;
      if (u < n) {
        c.settle(a);
        if (c.id(a) == id) continue;
      }
      if (first) {  // the end of another pair's item: no block of it was here
        if (u < n) seg_pos = c.item_pos(a);
        continue;
      }
      // ---- the item's (or this pair's) last block: the partial sums of its rows
      const int pb = (i - 1) % PA_NP;
      float* ls = mx + 256 * (i & 1);  // the maxima of the block before the last: read by all
      ls[128 * ch + L] = l;
      named_bar_sync(1, 32 * PA_SM_WARPS);
      // one order of addition for all four threads of a row
      const float lt = (ls[row] + ls[128 + row]) + (ls[64 + row] + ls[192 + row]);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[pb], ((i - 1) / PA_NP) & 1));
      tc_fence_after();
      // Through the warp's part of the P buffers (every product is done), 64 bytes of 32 rows at a time: a store
      // instruction writes whole 64-byte pieces of eight rows in place of 32 rows' 16 bytes.
      unsigned char* stage = p_s + (warp - PA_SM_WARP) * 2048;
      const uint32_t live_rows = __ballot_sync(0xffffffffu, live);
      auto put = [&](int e, uint4 v) { *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = v; };
      auto get = [&](int r) { return *reinterpret_cast<const uint4*>(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)); };
      const bool whole = !a.multi && seg_pos == 0 && left == 0;
      if (whole) {
        // the rows' only part: the result itself
        const float inv = lt != 0.f ? 1.f / lt : 0.f;
        #pragma unroll 1
        for (int k = 0; k < 4 && live_rows != 0; ++k) {
          uint32_t o[32];
          tmem_ld32(t_o + 32 * k, o);
          tmem_ld_wait();
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 p2 = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * j]) * inv,
                                                              __uint_as_float(o[8 * e + 2 * j + 1]) * inv);
              u[j] = *reinterpret_cast<const uint32_t*>(&p2);
            }
            put(e, make_uint4(u[0], u[1], u[2], u[3]));
          }
          __syncwarp();
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * e + (lane >> 2);
            const uint4 v = get(r);
            if ((live_rows >> r) & 1)
              *reinterpret_cast<uint4*>(a.out + (gr - lane + r) * 512 + 256 * kh + 128 * ch + 32 * k + 8 * (lane & 3)) = v;
          }
          __syncwarp();
        }
        if (live && kh == 0 && ch == 0 && a.lse) a.lse[gr] = lt != 0.f ? (m_used + log2f(lt)) * 0.6931471805599453f : -INFINITY;
      } else {
        const int64_t prow_i = seg_pos > 0 ? static_cast<uint32_t>(pair * PA_ROWS + trow) : part_row(a, own, static_cast<uint32_t>(gr));
        #pragma unroll 1
        for (int k = 0; k < 8 && live_rows != 0; ++k) {
          uint32_t o[16];
          tmem_ld16(t_o + 16 * k, o);
          tmem_ld_wait();
          #pragma unroll
          for (int e = 0; e < 4; ++e) put(e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
          __syncwarp();
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * e + (lane >> 2);
            const uint4 v = get(r);
            if ((live_rows >> r) & 1)
              *reinterpret_cast<uint4*>(a.ws_o + (prow_i - lane + r) * 512 + 256 * kh + 128 * ch + 16 * k + 4 * (lane & 3)) = v;
          }
          __syncwarp();
        }
        if (live && kh == 0 && ch == 0) a.ws_ml[prow_i] = make_float2(m_used, lt);
      }
      tc_fence_before();
      named_bar_sync(1, 32 * PA_SM_WARPS);  // the next block's probabilities go to the same buffers
      if (rank == 0 && ch == 0 && L == 0) {
        if (seg_pos == 0) a.seg[id].x = pair;
        if (left == 0) a.seg[id].y = whole ? -2 : pair;
      }
      m_used = -INFINITY;
      l = 0.f;
      first = true;
      if (u < n) seg_pos = c.item_pos(a);
    }
  }
  if (!ok) {
    atomicExch(&g_prefix_timeout, 1);
    *abort_flag = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // copies and products that are still in flight end within microseconds
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  cluster_sync_relaxed();  // the other CTA's products and arrivals end here too
  if (warp == PA_PV_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The partials of a row (b, h), from the pairs that shared the row's items, joined by their maxima and sums.
struct RowParts {
  int n0, n;           // partials of the prefix part (or tile), and of it and the own part
  uint32_t f0, f1;     // where the first partial of either lies,
  uint32_t c0, c1;     // and the others: partial i at c + i * 128
  bool done;           // written by the attention itself
  __device__ __forceinline__ void find(const PaArgs& a, uint32_t r) {
    const uint32_t h = static_cast<uint32_t>(a.H);
    const int b = static_cast<int>(r / h), t = static_cast<int>(r / PA_ROWS);
    const int qlo = static_cast<int>(static_cast<uint32_t>(t) * PA_ROWS / h);
    // (written for items that have blocks, so the loads need not wait for the length)
    const int i0 = a.multi ? qlo + 2 * t : t, i1 = a.multi ? b + 2 * t + 1 : t;
    const int2 g0 = a.seg[i0], g1 = a.seg[i1];
    const int own = a.own_len ? __ldg(a.own_len + b) : 0;
    if (own < 0 || own > a.cap) atomicExch(&g_prefix_check, 1);
    const int ob = Cursor::blocks_of(a, b);
    const bool any = (a.multi ? a.nP : a.nP + ob) > 0;
    done = any && g0.y == -2;
    n0 = any ? max(g0.y - g0.x + 1, 0) : 0;
    n = min(n0 + (a.multi && ob > 0 ? max(g1.y - g1.x + 1, 0) : 0), 2 * PA_PAIRS);
    f0 = part_row(a, false, r);
    f1 = part_row(a, true, r);
    c0 = static_cast<uint32_t>(g0.x * PA_ROWS) + r % PA_ROWS;
    c1 = static_cast<uint32_t>((g1.x - n0) * PA_ROWS) + r % PA_ROWS;
  }
  __device__ __forceinline__ int64_t row(int i) const {
    uint32_t v = (i < n0 ? c0 : c1) + static_cast<uint32_t>(i * PA_ROWS);
    v = i == 0 ? f0 : v;
    return i == n0 ? f1 : v;
  }
};
__device__ __forceinline__ uint2 pack4(const float4& v, float inv) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
// (every partial that is joined was written, and one of weight 0 counts too: 0 times an infinity is the formula's NaN)
__device__ __forceinline__ void add_part(float4& acc, float w, const float4& v) {
  acc.x += w * v.x;
  acc.y += w * v.y;
  acc.z += w * v.z;
  acc.w += w * v.w;
}

// Many rows: a warp each, 16 columns a lane, a partial's maximum and sum a lane.
__global__ void __launch_bounds__(128) k_prefix_combine_rows(const PaArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r64 = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r64 >= a.BH) return;
  const uint32_t r = static_cast<uint32_t>(r64);
  RowParts p;
  p.find(a, r);
  if (p.done) return;
  float m = -INFINITY, l = 0.f;
  float4 acc[4];
  #pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b0 = 0; b0 < p.n; b0 += 32) {
    const int i = b0 + lane;
    const float2 ml = i < p.n ? a.ws_ml[p.row(i)] : make_float2(0.f, 0.f);
    const float mn = fmaxf(m, warp_max(ml.y != 0.f ? ml.x : -INFINITY));
    const float old = m == -INFINITY ? 0.f : exp2f(m - mn), w = ml.y != 0.f ? exp2f(ml.x - mn) : 0.f;
    m = mn;
    l = l * old + warp_sum(w * ml.y);
    #pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(acc[k].x * old, acc[k].y * old, acc[k].z * old, acc[k].w * old);
    const int cnt = min(32, p.n - b0);
    #pragma unroll 2
    for (int j = 0; j < cnt; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float4* src = reinterpret_cast<const float4*>(a.ws_o + p.row(b0 + j) * 512);
      #pragma unroll
      for (int k = 0; k < 4; ++k) add_part(acc[k], wj, src[32 * k + lane]);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  #pragma unroll
  for (int k = 0; k < 4; ++k) reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(r) * 512)[32 * k + lane] = pack4(acc[k], inv);
  if (a.lse && lane == 0) a.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// A warp 128 columns of a row, four columns a lane, a partial's maximum and sum a lane; the first U partials' values are on
// their way with them.  No shared memory: its blocks can wait on an SM that the attention fills.
__global__ void __launch_bounds__(128) k_prefix_combine_warps(const PaArgs a) {
  constexpr int U = 8;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r64 = blockIdx.x;
  const int c0 = static_cast<int>(threadIdx.x >> 5) * 128;
  const uint32_t r = static_cast<uint32_t>(r64);
  RowParts p;
  p.find(a, r);
  if (p.done) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b0 = 0; b0 < p.n; b0 += 32) {
    const float2 ml = b0 + lane < p.n ? a.ws_ml[p.row(b0 + lane)] : make_float2(0.f, 0.f);
    const int cnt = min(32, p.n - b0);
    float4 v[U];
    auto load = [&](int j0) {
      #pragma unroll
      for (int k = 0; k < U; ++k)
        v[k] = j0 + k < cnt ? reinterpret_cast<const float4*>(a.ws_o + p.row(b0 + j0 + k) * 512 + c0)[lane]
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    const float mn = fmaxf(m, warp_max(ml.y != 0.f ? ml.x : -INFINITY));
    const float old = m == -INFINITY ? 0.f : exp2f(m - mn), w = ml.y != 0.f ? exp2f(ml.x - mn) : 0.f;
    m = mn;
    l = l * old + warp_sum(w * ml.y);
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
    for (int j0 = 0; j0 < cnt; j0 += U) {
      #pragma unroll
      for (int k = 0; k < U; ++k) add_part(acc, __shfl_sync(0xffffffffu, w, (j0 + k) & 31), v[k]);
      if (j0 + U < cnt) load(j0 + U);
    }
  }
  reinterpret_cast<uint2*>(a.out + r64 * 512 + c0)[lane] = pack4(acc, l != 0.f ? 1.f / l : 0.f);
  if (a.lse && threadIdx.x == 0) a.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Few rows, so many partials each (up to 74): four blocks a row, 128 columns a block; 16 warps take the partials in turn,
// every load of a row on its way before the weights are formed.  The whole call against one block a row (below), in a
// graph: 128 rows of 74 partials 16.9 against 18.1 us, of 56 16.2 against 17.1, of 48 16.0 against 16.6, of 40 16.0 against
// 15.2, of 8 14.0 against 12.8; 64 rows of 74 16.0 against 18.5, of 48 15.5 against 16.0.
__global__ void __launch_bounds__(512, 3) k_prefix_combine_few(const PaArgs a) {
  constexpr int W = 16, U = 5;
  __shared__ float wt[2 * PA_PAIRS];
  __shared__ float red[2 * W];
  __shared__ float4 acc_s[W][32];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t r = blockIdx.x >> 2;
  const int c0 = static_cast<int>(blockIdx.x & 3) * 128;
  RowParts p;
  p.find(a, r);
  if (p.done) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float2 ml = tid < p.n ? a.ws_ml[p.row(tid)] : make_float2(0.f, 0.f);
  auto part = [&](int i) {
    return i < p.n ? *reinterpret_cast<const float4*>(a.ws_o + p.row(i) * 512 + c0 + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 v[U];
  #pragma unroll
  for (int k = 0; k < U; ++k) v[k] = part(warp + W * k);
  float m = warp_max(ml.y != 0.f ? ml.x : -INFINITY);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  #pragma unroll
  for (int w = 0; w < W; ++w) m = fmaxf(m, red[w]);
  const float w_mine = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
  if (tid < p.n) wt[tid] = w_mine;
  float l = warp_sum(w_mine * ml.y);
  if (lane == 0) red[W + warp] = l;
  __syncthreads();
  l = 0.f;
  #pragma unroll
  for (int w = 0; w < W; ++w) l += red[W + w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll
  for (int k = 0; k < U; ++k)
    if (warp + W * k < p.n) add_part(acc, wt[warp + W * k], v[k]);
  for (int i = warp + W * U; i < p.n; i += W) add_part(acc, wt[i], part(i));
  acc_s[warp][lane] = acc;
  __syncthreads();
  if (tid < 64) {  // two columns each
    const float* col = reinterpret_cast<const float*>(acc_s) + 2 * tid;
    float x = 0.f, y = 0.f;
    #pragma unroll
    for (int w = 0; w < W; ++w) {
      x += col[128 * w];
      y += col[128 * w + 1];
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<int64_t>(r) * 512 + c0)[tid] = __floats2bfloat162_rn(x * inv, y * inv);
  }
  if (a.lse && c0 == 0 && tid == 0) a.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Few rows: a block each.  G groups of 128 threads take the partials in turn (four columns a thread), the weights are
// formed once a block: a row behind a long prefix has up to 74 partials and few other rows to hide its loads behind.
__global__ void __launch_bounds__(512) k_prefix_combine(const PaArgs a) {
  constexpr int G = 4, U = 6;
  static_assert(128 * G >= 2 * PA_PAIRS, "a partial's maximum and sum a thread");
  __shared__ float wt[2 * PA_PAIRS];
  __shared__ float4 acc_s[(G - 1) * 128];
  __shared__ float red[2 * 4 * G];
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t r = blockIdx.x;
  RowParts p;
  p.find(a, r);
  if (p.done) return;
  const int parts = p.n;
  auto slot_row = [&](int i) { return p.row(i); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = tid & 127;
  // the parts' maxima and sums, and the first of the values on their way at the same time
  const float2 ml = tid < parts ? a.ws_ml[slot_row(tid)] : make_float2(0.f, 0.f);
  float4 v[U];
  #pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = (tid >> 7) + G * k;
    v[k] = i < parts ? reinterpret_cast<const float4*>(a.ws_o + slot_row(i) * 512)[col] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m = warp_max(ml.y != 0.f ? ml.x : -INFINITY);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  #pragma unroll
  for (int w = 0; w < 4 * G; ++w) m = fmaxf(m, red[w]);
  const float w_mine = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
  if (tid < parts) wt[tid] = w_mine;
  float l = w_mine * ml.y;
  l = warp_sum(l);
  if (lane == 0) red[4 * G + warp] = l;
  __syncthreads();
  l = 0.f;
  #pragma unroll
  for (int w = 0; w < 4 * G; ++w) l += red[4 * G + w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0k = tid >> 7; i0k < parts; i0k += G * U) {
    float4 nx[U];
    #pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0k + G * (U + k);
      nx[k] = i < parts ? reinterpret_cast<const float4*>(a.ws_o + slot_row(i) * 512)[col] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    #pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0k + G * k;
      add_part(acc, i < parts ? wt[i] : 0.f, v[k]);
      v[k] = nx[k];
    }
  }
  if (tid >= 128) acc_s[tid - 128] = acc;
  __syncthreads();
  if (tid >= 128) return;
  #pragma unroll
  for (int g = 0; g < G - 1; ++g) add_part(acc, 1.f, acc_s[g * 128 + tid]);
  reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(r) * 512)[tid] = pack4(acc, l != 0.f ? 1.f / l : 0.f);
  if (a.lse && tid == 0) a.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encoder();

// Latent rows as [9 parts of 64 dims][rows][64 dims]: a box of `parts` x box_rows x 64 lands as that many operands of
// 128-byte rows one behind another (128-byte swizzle), by one instruction.
static int make_map_parts(CUtensorMap* m, const void* ptr, int64_t rows, int box_rows, int parts) {
  EncodeTiledFn fn = encoder();
  if (!fn) {
    set_last_error("cuTensorMapEncodeTiled unavailable");
    return LSA_ERR_CUDA;
  }
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), 9};
  cuuint64_t strides[2] = {1152, 128};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(parts)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_last_error("cuTensorMapEncodeTiled failed");
    return LSA_ERR_CUDA;
  }
  return LSA_OK;
}

// Scratch: seg int2 [items] | (max, sum) [partial rows] | O [partial rows][512] fp32.
struct PrefixLayout {
  int64_t nT, items, rows;
  bool multi;
  size_t o_ml, o_o, total;
};
static PrefixLayout prefix_ws_layout(int64_t B, int H) {
  PrefixLayout p;
  p.nT = cdiv(B * H, PA_ROWS);
  p.multi = H % PA_ROWS != 0 && B > 1;
  p.items = p.multi ? B + 2 * p.nT : p.nT;
  p.rows = PA_PAIRS * PA_ROWS + (p.multi ? 2 : 1) * B * H;
  p.o_ml = align_up(static_cast<size_t>(p.items) * 8, 256);
  p.o_o = p.o_ml + align_up(static_cast<size_t>(p.rows) * 8, 256);
  p.total = p.o_o + static_cast<size_t>(p.rows) * 512 * 4;
  return p;
}

size_t prefix_attn_ws_bytes(int64_t B, int H) { return B > 0 ? prefix_ws_layout(B, H).total : 0; }

int launch_prefix_attn(const void* q, int64_t B, int H, const void* prefix, int64_t Lp, const void* pages,
                       int64_t n_pages, int page, const int32_t* table, int64_t table_ld, const int32_t* own_len,
                       float scale, void* out, float* lse, void* ws, cudaStream_t s) {
  const PrefixLayout p = prefix_ws_layout(B, H);
  unsigned char* base = static_cast<unsigned char*>(ws);
  PaArgs a;
  a.own_len = own_len;
  a.table = table;
  a.table_ld = table_ld;
  a.page_shift = 0;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.kbox = page < PA_KT ? page : PA_KT;
  a.vbox = page < PA_VT ? page : PA_VT;
  a.n_pages = static_cast<int>(n_pages);
  a.cap = static_cast<int>(table_ld * page < 0x7FFFFF00 ? table_ld * page : 0x7FFFFF00);
  a.H = H;
  a.BH = B * H;
  a.nT = static_cast<int>(p.nT);
  a.multi = p.multi && own_len != nullptr;
  a.Lp = Lp;
  a.nP = static_cast<int>(cdiv(Lp, PA_T));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.seg = reinterpret_cast<int2*>(base);
  a.ws_ml = reinterpret_cast<float2*>(base + p.o_ml);
  a.ws_o = reinterpret_cast<float*>(base + p.o_o);
  // an absent part's maps cover the queries: nothing is loaded through them
  CUtensorMap tq, tk, tv, tpk, tpv;
  const int64_t own_rows = n_pages * page;
  int st = make_map_parts(&tq, q, a.BH, 64, PA_KS);
  if (st == LSA_OK) st = make_map_parts(&tk, Lp > 0 ? prefix : q, Lp > 0 ? Lp : a.BH, PA_KT, PA_KS);
  if (st == LSA_OK) st = make_map_parts(&tv, Lp > 0 ? prefix : q, Lp > 0 ? Lp : a.BH, PA_VT, 4);
  if (st == LSA_OK)
    st = make_map_parts(&tpk, own_rows > 0 ? pages : q, own_rows > 0 ? own_rows : a.BH, a.kbox, a.kbox == PA_KT ? PA_KS : 1);
  if (st == LSA_OK)
    st = make_map_parts(&tpv, own_rows > 0 ? pages : q, own_rows > 0 ? own_rows : a.BH, a.vbox, a.vbox == PA_VT ? 4 : 1);
  if (st != LSA_OK) return st;
  LSA_CUDA_TRY(func_smem_once(reinterpret_cast<const void*>(k_prefix_attn), PA_SMEM));
  LSA_CUDA_TRY(launch_pdl(k_prefix_attn, dim3(2 * PA_PAIRS), dim3(PA_THREADS), PA_SMEM, s, 0u, tq, tk, tv, tpk, tpv, a));
  // About how many partials a row has chooses the join.  Few: a warp for 128 columns, against a block a row: 4 tiles of 18
  // partials 33.5 against 34.6 us, 8 of 9 43.7 against 50.2, one of 8 12.6 against 12.8; one of 12 13.8 against 12.9, of 32
  // 18.2 against 14.6, two of 10 14.0 against 13.3, three of 25 19.7 against 18.4 (of 16 15.4 against 16.0: the rule takes
  // no account of three).  Many tiles, most rows written already: a warp a row (74 tiles 48.8 us against 54.8).  The lengths
  // of own tokens are not known here: where those take most of the pairs, the prefix has fewer partials than this counts.
  const int64_t blocks = a.nP + (own_len && !a.multi ? cdiv(a.cap, PA_T) : 0);  // of a tile, at most
  const int64_t parts = std::min<int64_t>(blocks, PA_PAIRS / std::min(a.nT, PA_PAIRS)) + (a.multi ? 1 : 0);
  const dim3 rows(static_cast<unsigned>(a.BH));
  if (a.nT > PA_PAIRS / 2)
    return cuda_status(launch_pdl(k_prefix_combine_rows, dim3(static_cast<unsigned>(cdiv(a.BH, 4))), dim3(128), 0, s, 0u, a));
  if (a.nT >= 4 || parts <= 8) return cuda_status(launch_pdl(k_prefix_combine_warps, rows, dim3(128), 0, s, 0u, a));
  if (a.nT == 1 && parts >= 48)
    return cuda_status(launch_pdl(k_prefix_combine_few, dim3(static_cast<unsigned>(4 * a.BH)), dim3(512), 0, s, 0u, a));
  return cuda_status(launch_pdl(k_prefix_combine, rows, dim3(512), 0, s, 0u, a));
}

// The kernel's flags, read and cleared: give-up and device check; -1: CUDA error.
int take_prefix_flags(int* check) {
  int v = 0, c = 0;
  if (cudaMemcpyFromSymbol(&v, g_prefix_timeout, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyFromSymbol(&c, g_prefix_check, sizeof(int)) != cudaSuccess) return -1;
  const int zero = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_prefix_timeout, &zero, sizeof(int)) != cudaSuccess) return -1;
  if (c != 0 && cudaMemcpyToSymbol(g_prefix_check, &zero, sizeof(int)) != cudaSuccess) return -1;
  *check = c;
  return v;
}

}  // namespace lsa
