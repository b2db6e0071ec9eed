// Few tokens: y[t][n] = sum_k x[t][k] w[e N + n][k].
//
// The kernel is bound by the weights' bytes, so everything else is arranged to
// keep their copies in flight.  Weight codes are the A operand (128 rows a
// tile, one or two blocks a stage, copied by TMA as they lie in memory); the tokens
// are the B operand (16 or 32 of them); `tcgen05.mma kind::mxf8f6f4.block_scale`
// multiplies and applies both scale bytes.  x comes a chunk of four blocks at a
// time, into slots apart from the stages, so that it does not wait for weights:
// for very few tokens four warps read it in its own type and quantise it (as
// cql_fp8_quantize does) straight into the slots, and no kernel runs before;
// else it is block-scaled already and copied by TMA.  The same warps put the
// scale words of both operands into tensor memory.
//
// Scale operands: the MMA reads a scale byte a row for each K = 32 step from
// tensor memory, row r at lane r % 32 (in each lane quarter) and column
// r / 32, the byte chosen in the instruction descriptor.  The 32-bit cell is a
// word of the scale plane (four consecutive blocks), so a word a row serves a
// chunk, and the four K = 32 steps of a block use the same byte.
//
// Where the tiles are too few to fill the GPU, the CTAs of a cluster (`split`
// of them) share a tile, each a range of the blocks; each CTA then sums the
// slice of token columns that it owns over the cluster's partial results, which
// they push into its shared memory, in rank order: the result does not depend on
// timing.
//
// Roles (320 threads, two CTAs an SM; four consecutive warps reach all four
// lane quarters of tensor memory):
//   warp 0     TMA producer of the weights
//   warp 1     tensor-memory allocator, single-thread MMA issuer
//   warps 2..5 x and scales
//   warps 6..9 epilogue (lane = row of W: a warp stores 32 consecutive outputs
//              of a token)
// Every mbarrier wait is bounded; on expiry the kernel records CQL_ERR_TIMEOUT
// (detail 40 weights, 41 MMA, 42 x and scales, 43 epilogue), waits for its own
// copies and MMAs, and winds down.  A role that copies ends when all that it has
// copied is multiplied: no copy and no commit is under way when a CTA ends.
//
// Measured (bf16, calls in a chain, weights not in L2): 11008 x 4096, one token
// 10.4 us for 45.5 MB, 67 % of the copy bandwidth, reading exactly the weights'
// bytes from DRAM; 4096 x 11008, 16 tokens 13.0 us, the quantise kernel included;
// 32 experts of 2048 x 1024, 24 tokens 13.9 us.  With more bytes the share grows
// (32 experts of 4096 x 4096, 10 tokens each, 545 MB: 83.5 us, 6.5 TB/s): what is
// left of a small call is its start (launch, barriers and tensor memory, the first
// copies' latency) and its end (the last sums and stores), some 3 us.  The second
// CTA on an SM and the copies that start before the kernel in front is done hide
// a part of both.
#include <cuda.h>

#include "fp8_query.h"
#include "fp8_tile.cuh"

namespace cql {
namespace {

constexpr int DC_THREADS = 320;
constexpr int DC_MAX_STAGES = 6;
constexpr int DC_XSLOTS = 2;                      // chunks of x (and scales) in flight
constexpr uint32_t DC_SF_COLS = 8;                // a slot: 4 columns of weight scales, 1 of token scales

struct DcParams {
  F8Tokens tok;
  const uint32_t* wscale;                         // [quads][wrows]
  int64_t wrows;
  const uint32_t* xscale;                         // [quads][tokens], or
  const void* x;                                  // [tokens][ldx]
  int64_t ldx;
  int cols, vec;
  int n, units, row_tiles, stages, split;
  int early;                                      // weights and offsets may be read before the kernel before is done
  int debug;                                      // x is withheld, the waits are short
  uint32_t tmem_cols;
  void* y;
  int ydt, yvec;                                  // yvec: rows of y are 16-byte aligned
  int64_t ldy;
  uint32_t* status;
  F8Bounds in;
};

struct DcCtl {
  uint64_t full[DC_MAX_STAGES], empty[DC_MAX_STAGES];
  uint64_t xfull[DC_XSLOTS], xempty[DC_XSLOTS], xbytes[2];
  uint64_t dfull[2], dempty[2], drain, red;
  uint8_t byte[2][32][4];                         // scale bytes of a chunk's tokens
  uint32_t tmem_base;
};

// Columns of partial results that a CTA may receive.
CQL_HD int dc_red_columns(int nt, int split) { return split * ((nt + split - 1) / split); }

CQL_DEV void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}

// If `on`: all earlier MMAs done -> an arrival on the barrier.
CQL_DEV void commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(on)
      : "memory");
}

// A row of W's outputs for the tile's first cnt tokens, from element `at` of y on.
template <int N>
CQL_DEV void store_tokens(const DcParams& p, int64_t at, const float (&acc)[N], int cnt) {
  if (p.ydt == CQL_DT_F32) {
    float* y = reinterpret_cast<float*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) y[i * p.ldy] = acc[i];         // 16-bit types below: the call's one rounding
  } else if (p.ydt == CQL_DT_F16) {
    __half* y = reinterpret_cast<__half*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) y[i * p.ldy] = __float2half_rn(acc[i]);
  } else {
    __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) y[i * p.ldy] = __float2bfloat16_rn(acc[i]);
  }
}

// DT: x's type, or -1: block-scaled.  NT: tokens a tile.  U: blocks of a stage.  Two
// take fewer barriers; with 32 tokens the x slots and the partial results leave
// room for one or two such stages, and four of one block keep more on its way:
// 4096 x 11008, 24 tokens 15.9 us with two blocks, 13.8 with one; 4096 x 4096, 16
// tokens (NT 16) 8.3 and 8.4.
template <int DT, int NT, int U>
__global__ void __launch_bounds__(DC_THREADS, 2)
    k_fp8_decode(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, DcParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr uint32_t X_BLOCK = NT * 128u, X_SLOT = 4u * X_BLOCK, STAGE = U * kF8ABytes;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xs = ring + (uint32_t)p.stages * STAGE;
  float* red = reinterpret_cast<float*>(xs + DC_XSLOTS * X_SLOT);     // split > 1: [split][columns of a CTA][128]
  DcCtl& S = *reinterpret_cast<DcCtl*>(red + (p.split > 1 ? dc_red_columns(NT, p.split) * kF8Rows : 0));
  const F8Map map(&S + 1, p.tok.experts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool early = p.early != 0;
  const int rank = p.split > 1 ? (int)cluster_rank() : 0;
  const int u0 = (int)((int64_t)p.units * rank / p.split), u1 = (int)((int64_t)p.units * (rank + 1) / p.split);
  const int first = p.split > 1 ? (int)blockIdx.x / p.split : (int)blockIdx.x;
  bool failed = false;                            // the epilogue's waits ran out
  // units of the first tile whose copies start before anything else is set up
  const int tt = (p.tok.tokens + NT - 1) / NT;    // token tiles of a row tile, where there is one expert
  const int ahead = early && p.tok.offsets == nullptr && first < p.row_tiles * tt ? min(p.stages, u1 - u0) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    for (int i = 0; i < ahead; ++i) {
      mbar_expect_tx(&S.full[i], STAGE);
      tma_load_3d(ring + (uint32_t)i * STAGE, &tmW, &S.full[i], 0, first / tt * kF8Rows, U * (u0 + i));
    }
    for (int s = 0; s < DC_XSLOTS; ++s) {
      mbar_init(&S.xfull[s], DT < 0 ? 5 : 4);
      mbar_init(&S.xempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.xbytes[s], 4);
      mbar_init(&S.dfull[s], 1);
      mbar_init(&S.dempty[s], 4);
    }
    mbar_init(&S.drain, 1);
    mbar_init(&S.red, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                 "r"(p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!early) pdl_wait();
  if (warp == 0) f8_scan(p.tok, map, p.status);
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_arrive();              // this CTA's barriers are there
  tc_fence_after();
  // The next kernel may start from here on, not before: it could take the
  // tensor memory that this CTA still has to allocate, and then wait for it.
  if (!early) pdl_launch_dependents();
  const uint32_t tmem = S.tmem_base;
  const int tiles = map.start[p.tok.experts] * p.row_tiles;
  const uint32_t sf0 = tmem + 2u * NT;            // scale slots behind the accumulators
  const int step = p.split > 1 ? tiles : (int)gridDim.x;              // split: a cluster has one tile

  if (warp == 0) {
    if (elect_one()) {
      // ---------------- TMA producer ----------------
      Ring at{0, 0};
      uint64_t lim = f8_limit(p.debug);
      int done = ahead;
      for (int i = 0; i < ahead; ++i) at.next(p.stages);
      for (int id = first; id < tiles && lim != 0; id += step) {
        const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
        const int row = t.expert * p.n + t.rt * kF8Rows;
        for (int u = u0 + done; u < u1; ++u) {
          f8_wait(&S.empty[at.s], at.phase ^ 1, lim);
          const uint32_t on = lim != 0;
          expect_if(on ? STAGE : 0u, &S.full[at.s]);
          tma_load_3d_if(on, ring + (uint32_t)at.s * STAGE, &tmW, &S.full[at.s], 0, row, U * u);
          at.next_if(on, p.stages);
        }
        done = 0;
      }
      for (int i = 0; i < p.stages; ++i) f8_wait(&S.empty[i], at.last(i), lim);
      if (lim == 0) {
        set_error(p.status, CQL_ERR_TIMEOUT, 40);
        uint64_t more = f8_limit(p.debug);       // copies in flight
        for (int i = 0; i < p.stages; ++i) f8_wait(&S.full[i], at.last(i), more);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------- MMA issuer ----------------
      const uint32_t idesc = f8_idesc(kF8Rows, NT);
      const uint64_t desc_a = smem_desc_sw128(smem_u32(ring)), desc_x = smem_desc_sw128(smem_u32(xs));
      uint32_t gc = 0;
      Ring at{0, 0}, xat{0, 0};
      uint64_t lim = f8_limit(p.debug);
      for (int id = first; id < tiles && lim != 0; id += step) {
        int chain = u0;                           // where the next accumulator chain starts
        uint32_t acc = 0;                         // the accumulator holds a sum already
        uint32_t ready = 0;                       // the next unit's copy is known to have landed
        auto unit = [&](int u) {
          f8_wait_if(ready ^ 1, &S.full[at.s], at.phase, lim);
          tc_fence_after();
          const uint32_t stage = (uint32_t)at.s;
          at.next(p.stages);
          ready = f8_peek(&S.full[at.s], at.phase);
          const uint32_t d = tmem + (gc & 1) * NT, sfa = sf0 + (uint32_t)xat.s * DC_SF_COLS;
          const uint64_t da = desc_a + (uint64_t)(stage * (STAGE >> 4));
          const uint64_t db = desc_x + (uint64_t)((uint32_t)(4 * xat.s + (U * u & 3)) * (X_BLOCK >> 4));
#pragma unroll
          for (int kk = 0; kk < 4 * U; ++kk)
            mma_f8(d, da + (kk >> 2) * (kF8ABytes >> 4) + 2 * (kk & 3), db + (kk >> 2) * (X_BLOCK >> 4) + 2 * (kk & 3),
                   idesc | f8_byte(U * u + (kk >> 2)), sfa, sfa + 4, kk == 0 ? acc : 1u);
          commit_if(lim != 0, &S.empty[stage]);
          acc = 1;
        };
        for (int u = u0; u < u1;) {               // a chunk at a time
          const int end = min(u1, (u | (4 / U - 1)) + 1);
          f8_wait_if(u == chain, &S.dempty[gc & 1], ((gc >> 1) & 1) ^ 1, lim);
          f8_wait(&S.xfull[xat.s], xat.phase, lim);
          if (lim == 0) break;
          for (; u < end; ++u) unit(u);
          commit_if(lim != 0, &S.xempty[xat.s]);
          xat.next(DC_XSLOTS);
          const uint32_t over = u == f8_chain_end<U>(chain, u1);
          commit_if(over & (lim != 0), &S.dfull[gc & 1]);
          gc += over;
          acc ^= over;
          chain = over ? u : chain;
        }
      }
      if (lim == 0) {
        set_error(p.status, CQL_ERR_TIMEOUT, 41);
        uint64_t more = f8_limit(p.debug);
        commit_if(1u, &S.drain);                  // MMAs in flight
        f8_wait(&S.drain, 0, more);
      }
    }
  } else if (warp < 6) {
    // ---------------- x and scales ----------------
    constexpr int XDT = DT < 0 ? CQL_DT_F32 : DT;
    using Raw = Raw16<XDT>;
    const int q = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    uint32_t sc = 0;
    Ring at{0, 0};
    uint64_t lim = f8_limit(p.debug);
    bool waited = !early, ok = true;
    for (int id = first; id < tiles && ok; id += step) {
      const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
      const int n0 = t.rt * kF8Rows + lane, cnt = t.t1 - t.t0, c0 = U * u0 >> 2, c1 = (U * u1 - 1) >> 2;
      const uint32_t* ws = p.wscale + (int64_t)t.expert * p.n + n0;
      auto weight_scales = [&](int c, uint32_t(&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)               // rows past the expert's last: any finite scale.  From L2: see k_fp8_quantize
          v[j] = c <= c1 && n0 + 32 * j < p.n && CQL_IN(p.status, ws - p.wscale + (int64_t)c * p.wrows + 32 * j, p.in.wscale, 411)
                     ? ld_cg_u32(ws + (int64_t)c * p.wrows + 32 * j)
                     : 0x7F7F7F7Fu;
      };
      uint32_t next[4];                           // the next chunk's, on their way
      weight_scales(c0, next);
      if (!waited) {
        pdl_wait();
        pdl_launch_dependents();
        waited = true;
      }
      // 16 columns of token k in chunk c (zeros behind the range and the row)
      auto fetch_x = [&](int c, int k, Raw& r) {
        const int kb = 4 * c + (lane >> 3), col = kb * kGroup + (lane & 7) * 16;
        r = Raw{};
        if (kb >= U * u0 && kb < U * u1 && k < cnt &&
            (col >= p.cols || CQL_IN(p.status, (int64_t)(t.t0 + k) * p.ldx + min(col + 15, p.cols - 1), p.in.x, 413)))
          load16<XDT>(r, p.x, (int64_t)(t.t0 + k) * p.ldx + col, col, p.cols, p.vec);
      };
      Raw ahead_x{};
      if (DT >= 0) fetch_x(c0, (q + (c0)) & 3, ahead_x);
      uint32_t xnext = 0x7F7F7F7Fu;
      auto token_scale = [&](int c) {
        const int64_t i = (int64_t)c * p.tok.tokens + t.t0 + lane;
        if (lane < cnt && CQL_IN(p.status, i, p.in.xscale, 412)) xnext = ld_cg_u32(p.xscale + i);
      };
      if (DT < 0) token_scale(c0);
      for (int c = c0; c <= c1; ++c, ++sc, at.next(DC_XSLOTS)) {
        const uint32_t v[4] = {next[0], next[1], next[2], next[3]};
        uint32_t xword = xnext;
        weight_scales(c + 1, next);
        uint8_t* slot = xs + (uint32_t)at.s * X_SLOT;
        if constexpr (DT < 0) {
          if (c < c1) token_scale(c + 1);
          f8_wait(&S.xempty[at.s], at.phase ^ 1, lim);
          ok = __all_sync(0xffffffffu, lim != 0);
          if (!ok) break;
          if (q == 0 && p.debug == 0 && elect_one()) {
            mbar_expect_tx(&S.xfull[at.s], X_SLOT);
            tma_load_3d(slot, &tmX, &S.xfull[at.s], 0, t.t0, 4 * c);
          }
          __syncwarp();
        } else {
          // lane / 8: the block of the chunk, lane % 8: 16 of its columns; the
          // four warps take the tokens in turn, starting with another one each
          // chunk (one token: the chunks go round the warps).  A warp's first
          // token of the next chunk is on its way while this one is quantised.
          const int kb = 4 * c + (lane >> 3);
          const bool mine = kb >= U * u0 && kb < U * u1;
          uint8_t* bt = slot + (uint32_t)(lane >> 3) * X_BLOCK;
          Raw raw = ahead_x;
          fetch_x(c + 1, (q + c + 1) & 3, ahead_x);
          f8_wait(&S.xempty[at.s], at.phase ^ 1, lim);
          ok = __all_sync(0xffffffffu, lim != 0);
          if (!ok) break;
          for (int k = (q + c) & 3; k < cnt; k += 4) {
            uint32_t byte;
            const uint4 w = quantize16<XDT>(raw, byte);
            if (k + 4 < cnt) fetch_x(c, k + 4, raw);
            if (mine) {
              *reinterpret_cast<uint4*>(bt + k * 128 + (((lane & 7) ^ (k & 7)) << 4)) = w;
              if ((lane & 7) == 0) S.byte[sc & 1][k][lane >> 3] = (uint8_t)byte;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.xbytes[sc & 1]);
        }
        // weight scales go up while the other warps finish; then every warp's
        // scale bytes are there
        __syncwarp();
        tc_fence_after();
        const uint32_t sf = sf0 + lanes + (uint32_t)at.s * DC_SF_COLS;
        tmem_st4(sf, v);
        if constexpr (DT >= 0) {
          f8_wait(&S.xbytes[sc & 1], (sc >> 1) & 1, lim);
          ok = __all_sync(0xffffffffu, lim != 0);
          if (!ok) break;
          if (lane < cnt) xword = *reinterpret_cast<const uint32_t*>(S.byte[sc & 1][lane]);
          __syncwarp();
        }
        tmem_st1(sf + 4, xword);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && (DT < 0 || p.debug == 0)) mbar_arrive(&S.xfull[at.s]);
      }
    }
    for (int s = 0; s < DC_XSLOTS; ++s) f8_wait(&S.xempty[s], at.last(s), lim);
    if (!__all_sync(0xffffffffu, lim != 0)) {
      if (lane == 0) set_error(p.status, CQL_ERR_TIMEOUT, 42);
      uint64_t more = f8_limit(p.debug);         // copies of x in flight
      for (int s = 0; DT < 0 && s < DC_XSLOTS; ++s) f8_wait(&S.xfull[s], at.last(s), more);
    }
  } else {
    // ---------------- epilogue ----------------
    const int q = warp & 3, row = 32 * q + lane;
    uint32_t gc = 0;
    uint64_t lim = f8_limit(p.debug);
    bool ok = true, pushed = false;
    if (early) pdl_wait();                        // y may be in use by the kernel before
    for (int id = first; id < tiles && ok; id += step) {
      const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
      const int n = t.rt * kF8Rows + row;
      float acc[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
      for (int u = u0; u < u1; u = f8_chain_end<U>(u, u1), ++gc) {
        const uint32_t buf = gc & 1;
        f8_wait(&S.dfull[buf], (gc >> 1) & 1, lim);
        ok = __all_sync(0xffffffffu, lim != 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + buf * NT;
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float v[16];
          tmem_ld_wait<16>(base + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.dempty[buf]);
      }
      if (!ok) break;
      const int cnt = t.t1 - t.t0;
      const int64_t y0 = (int64_t)t.t0 * p.ldy + n;
      if (p.split == 1) {
        if (n < p.n && CQL_IN(p.status, y0 + (int64_t)(cnt - 1) * p.ldy, p.in.y, 414)) store_tokens<NT>(p, y0, acc, cnt);
      } else {
        // Each CTA owns a slice of the token columns: the others' partial results
        // of it arrive at [source][column][128 rows] and count on its barrier.
        const int own = (cnt + p.split - 1) / p.split;
        const int mine = min(own, cnt - rank * own);
        if (threadIdx.x == 6 * 32 && mine > 0) mbar_expect_tx(&S.red, (uint32_t)(p.split * mine * kF8Rows) * 4u);
        cluster_wait();                           // the cluster's barriers are there
        const uint32_t to = smem_u32(red) + (uint32_t)(rank * own * kF8Rows + row) * 4u, bar = smem_u32(&S.red);
        int dst = 0, j0 = 0;                      // column i: column j0 of CTA dst
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (i >= cnt) break;
          if (CQL_IN(p.status, dst, p.split, 416) &&
              CQL_IN(p.status, rank * own + j0, dc_red_columns(NT, p.split), 417))
            push_cluster(to + (uint32_t)(j0 * kF8Rows) * 4u, bar, (uint32_t)dst, acc[i]);
          const bool next = ++j0 == own;
          j0 = next ? 0 : j0;
          dst += next ? 1 : 0;
        }
        cluster_arrive();
        pushed = true;
        if (mine > 0) f8_wait(&S.red, 0, lim);
        const int n4 = t.rt * kF8Rows + 4 * lane;
        for (int c = warp - 6; c < mine; c += 4) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < 8; ++r) {           // in rank order
            if (r >= p.split) break;
            const float4 v = *reinterpret_cast<const float4*>(red + (r * own + c) * kF8Rows + 4 * lane);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
          const int64_t at = (int64_t)(t.t0 + rank * own + c) * p.ldy + n4;
          if (n4 < p.n && CQL_IN(p.status, at + min(4, p.n - n4) - 1, p.in.y, 415))
            store4(p.y, p.ydt, at, sum, p.n - n4, p.yvec);
        }
        ok = __all_sync(0xffffffffu, lim != 0);
      }
    }
    if (!ok && lane == 0) set_error(p.status, CQL_ERR_TIMEOUT, 43);
    failed = !ok;
    if (p.split > 1 && !pushed) {                 // nothing to push
      cluster_wait();
      cluster_arrive();
    }
  }
  __syncwarp();
  if (p.split > 1) {
    if (warp < 6) {                               // the epilogue's cluster barriers
      cluster_wait();
      cluster_arrive();
    }
    cluster_wait();                               // no CTA of the cluster pushes to this one any more
    if (failed) f8_pause();                       // what they have pushed, and this one did not wait for
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
}

constexpr int DC_SMEM = 113 * 1024;               // two CTAs an SM

// Never launched: a kernel of the same size to ask about.  Asked about a kernel
// that allocates tensor memory the runtime counts one CTA an SM.
__global__ void __launch_bounds__(DC_THREADS, 2) k_fp8_decode_size() {}

// How many clusters of 2 .. 8 CTAs run at once on the current device: a cluster
// lies within one part of the GPU, so fewer than its CTAs / split.
struct ClustersAtOnce {
  int n[9];
};
cudaError_t clusters_at_once(ClustersAtOnce& c) {
  static KeptAnswer kept[64][9];                  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (int split = 2; split <= 8; ++split) {
    e = (cudaError_t)kept[dev & 63][split].get(c.n[split], [split](int& n) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)split);
      cfg.blockDim = dim3(DC_THREADS);
      cfg.dynamicSmemBytes = DC_SMEM;
      cudaLaunchAttribute at{};
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = (unsigned)split;
      at.val.clusterDim.y = 1;
      at.val.clusterDim.z = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      n = 0;
      const cudaError_t r = cudaFuncSetAttribute(k_fp8_decode_size, cudaFuncAttributeMaxDynamicSharedMemorySize, DC_SMEM);
      return (int)(r != cudaSuccess ? r : cudaOccupancyMaxActiveClusters(&n, k_fp8_decode_size, &cfg));
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int DT, int NT, int U>
cudaError_t launch(const Fp8Product& f, DcParams& p, cudaStream_t st) {
  const int sms = device_sm_count();
  p.tok.nt = NT;
  // token tiles: at most one partly filled tile an expert
  int64_t tt = (int64_t)p.tok.tokens / NT + f.experts;
  if (tt > p.tok.tokens) tt = p.tok.tokens;
  if (f.offsets == nullptr) tt = (p.tok.tokens + NT - 1) / NT;
  const int64_t tiles = tt * p.row_tiles;
  p.units = (f.w.blocks + U - 1) / U;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = ensure_smem_attr(attr_done, (const void*)k_fp8_decode<DT, NT, U>, DC_SMEM);
  if (e != cudaSuccess) return e;
  // Split as far as all clusters run at once, with one to spare, and each CTA keeps
  // four blocks.  A second round of clusters costs more than the split gives: 9472 x
  // 4096, one token, 74 clusters of 4 of which 71 run at once 14.2 us, of 3 9.5.
  p.split = 1;
  ClustersAtOnce at_once;
  e = clusters_at_once(at_once);
  if (e != cudaSuccess) return e;
  for (int s = 2; s <= 8 && tiles * s <= 2 * sms && U * p.units >= 4 * s; ++s)
    if (tiles < at_once.n[s]) p.split = s;
  p.tmem_cols = 2 * NT + DC_XSLOTS * DC_SF_COLS <= 64 ? 64 : 128;
  constexpr uint32_t STAGE = U * kF8ABytes;
  const uint32_t xbytes = DC_XSLOTS * 4u * NT * 128u;
  const uint32_t red = p.split > 1 ? (uint32_t)dc_red_columns(NT, p.split) * kF8Rows * 4u : 0u;
  const uint32_t ctl = (uint32_t)sizeof(DcCtl) + F8Map::bytes(f.experts);
  const uint32_t room = (uint32_t)DC_SMEM - 1024u - xbytes - red - ctl;
  p.stages = (int)(room / STAGE);
  if (p.stages > DC_MAX_STAGES) p.stages = DC_MAX_STAGES;
  if (p.stages < 1) return cudaErrorInvalidConfiguration;
  const int smem = (int)(1024u + (uint32_t)p.stages * STAGE + xbytes + red + ctl);
  CUtensorMap mw, mx;
  if (!make_map_codes(&mw, f.w_base, (uint64_t)f.w.rows, (uint64_t)f.w.blocks, kF8Rows, U)) return cudaErrorInvalidValue;
  mx = mw;
  if (DT < 0 && !make_map_codes(&mx, f.x_base, (uint64_t)f.x.rows, (uint64_t)f.x.blocks, NT, 4))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  const int64_t ctas = p.split > 1 ? tiles * p.split : (tiles < 2 * sms ? tiles : 2 * sms);
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(DC_THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_decode<DT, NT, U>, mw, mx, p);
}

}  // namespace

// Against the pair kernel (bf16 x, us a call in a chain of calls).  Up to 32 tokens
// an expert there is one token tile: 4096 x 11008, 24 tokens 13.8 and 18.8; 28672 x
// 8192, 32 tokens 39.0 and 44.2; 11008 x 4096, 32 tokens 14.0 and 13.1; 32 experts of
// 2048 x 1024 with 32 each 17.8 and 20.7.  Up to 64 the weights are read twice, the
// second time from L2, which small ones still gain from: 2048 x 4096, 64 tokens 9.5
// and 10.5; 1024 x 4096 7.9 and 10.0; 64 experts of 1024 x 1024 with 64 each 21.5 and
// 24.6; but 4096 x 4096 11.4 and 10.8, 28672 x 8192 51 and 45.
// The experts' loads are not known here, their mean is.  This kernel and the pair
// kernel with loads as 1 / rank, and with every token at one expert:
//   64 of 1024 x 1024, mean 16  19.0 and 21.2, 11.4 and 11.9; mean 64 24.4 and 27.1, 18.4 and 20.2
//   32 of 2048 x 2048, mean 16  29.5 and 31.7, 14.8 and 13.6; mean 64 39.0 and 38.2, 25.9 and 23.0
//   8 of 4096 x 4096,  mean 16  31.6 and 29.7, 15.1 and 12.5; mean 32 30.9 and 32.8, 16.4 and 17.5
bool fp8_decodes(int tokens, int experts, int64_t weights) {
  const int per = (tokens + experts - 1) / experts;
  return per <= 32 || (per <= 64 && weights <= 8 << 20);
}
// Quantising on the way saves a kernel but its time grows with the tokens:
// 11008 x 4096, 4 tokens 11.6, 8 tokens 12.4 against 11.7 after a quantise
// kernel, 16 tokens 16.2 against 12.3.  Here too the mean stands for the loads: 32
// experts of 2048 x 2048, mean 2, even 24.5 against 25.7, as 1 / rank 28.4 against
// 23.5, every token at one 11.8 against 8.8; 8 of 4096 x 4096, every token at one
// 20.5 against 12.4.
bool fp8_decode_quantizes(int tokens, int experts) { return (tokens + experts - 1) / experts <= 4; }

cudaError_t ready_fp8_decode() {
  ClustersAtOnce at_once;
  return clusters_at_once(at_once);
}

cudaError_t launch_fp8_decode(const Fp8Product& f, cudaStream_t st) {
  DcParams p{};
  p.tok.offsets = f.offsets;
  p.tok.experts = f.experts;
  p.tok.tokens = (int)f.x.rows;
  p.wscale = reinterpret_cast<const uint32_t*>(f.w_base + f.w.scales_off);
  p.wrows = f.w.rows;
  p.xscale = f.x_base ? reinterpret_cast<const uint32_t*>(f.x_base + f.x.scales_off) : nullptr;
  p.x = f.raw;
  p.ldx = f.ldx;
  p.cols = f.w.cols;
  const int es = f.xdt == CQL_DT_F32 ? 4 : 2;
  p.vec = (reinterpret_cast<uintptr_t>(f.raw) & 15) == 0 && (f.ldx * es) % 16 == 0;
  p.n = f.n;
  p.row_tiles = (f.n + kF8Rows - 1) / kF8Rows;
  p.early = f.early;
  p.debug = f.debug;
  p.y = f.y;
  p.ydt = f.ydt;
  p.yvec = (reinterpret_cast<uintptr_t>(f.y) & 15) == 0 && (f.ldy * (f.ydt == CQL_DT_F32 ? 4 : 2)) % 16 == 0;
  p.ldy = f.ldy;
  p.status = f.status;
  p.in = {f.w.scales_len / 4, f.x.scales_len / 4, fp8_extent(f.x.rows, f.ldx, f.w.cols), fp8_extent(f.x.rows, f.ldy, f.n)};
  if (f.x_base != nullptr) {
    const bool wide = (p.tok.tokens + f.experts - 1) / f.experts > 16;
    return wide ? launch<-1, 32, 1>(f, p, st) : launch<-1, 16, 2>(f, p, st);
  }
  if (f.xdt == CQL_DT_F32) return launch<CQL_DT_F32, 16, 2>(f, p, st);
  if (f.xdt == CQL_DT_F16) return launch<CQL_DT_F16, 16, 2>(f, p, st);
  return launch<CQL_DT_BF16, 16, 2>(f, p, st);
}

}  // namespace cql
