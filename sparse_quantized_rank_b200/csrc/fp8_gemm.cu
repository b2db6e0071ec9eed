// Many tokens: y[t][n] = sum_k x[t][k] w[e N + n][k], both operands
// block-scaled already.
//
// A pair of CTAs (cta_group::2) computes a tile of 256 weight rows x nt tokens:
// each CTA copies its 128 rows of the weights and half of the tokens, and one
// `tcgen05.mma kind::mxf8f6f4.block_scale` over both CTAs' shared memory
// multiplies and applies both scale bytes.  Against one CTA's tile of 128 rows
// the tokens' codes cross from L2 once instead of twice.  Each CTA's tensor
// memory holds its 128 rows of the tile, in one of two accumulators, and the
// scale words: its own 128 rows', and all nt tokens'.
//
// Scale operands: the MMA reads a scale byte a row for each K = 32 step from
// tensor memory, row r at lane r % 32 (in each lane quarter) and column
// r / 32, the byte chosen in the instruction descriptor.  The 32-bit cell is a
// word of the scale plane (four consecutive blocks), so a word a row serves a
// chunk of 512 columns.
//
// nt (32 .. 224, a multiple of 32) follows the number of tokens (launch_fp8_gemm).
//
// Roles (512 threads, one CTA an SM, persistent over the tiles):
//   warps 0, 2  copies of the weights, of the tokens (each CTA its own halves;
//               the bytes count on the first CTA's barrier)
//   warp 1      tensor-memory allocator; in the first CTA the MMA issuer
//   warps 4..7  scale words: global -> registers -> tensor memory
//   warps 8..15 epilogue: partial sums of the segments in registers, one
//               rounding, a turn through shared memory, 16-byte stores
// Every mbarrier wait is bounded; on expiry the kernel records CQL_ERR_TIMEOUT
// (detail 44 copies, 45 MMA, 46 scale words, 47 epilogue), waits for its own copies
// and MMAs, and winds down.  A role that copies ends when all that it has copied is
// multiplied: no copy and no commit is under way when a CTA ends.
//
// What bounds it.  A block of a 256 x 224 tile is 448 cycles of MMA and 30 KB a
// CTA, 67 bytes a cycle, about what an SM takes from L2 (copies alone: 19 TB/s
// over all SMs).  74 tiles of 18944 x 4096 at a time, a block takes 260 ns with
// zeros as data and 340 ns with random ones: the 1000 W cap lowers the clock, so
// large products are bound by power (18944 x 4096, 1792 tokens: 96 us, 2900
// TFLOP/s).  11008 x 4096, 2048 block-scaled tokens: 71 to 77 us, 2500 TFLOP/s (one
// after another 89, at the power cap).  The busiest pair has six tiles, 86,016
// cycles of MMA in the 110,000 to 114,000 that the call takes at 1.55 GHz; start and
// end are some 9,000 of the rest.  For the other 15,000 to 19,000, 10 to 12 us, no
// cause has been measured.  Few tokens an expert are bound by the weights' bytes: 32 experts of
// 4096 x 4096, 64 tokens each 92 us, 6.1 TB/s.
#include <cuda.h>

#include "fp8_query.h"
#include "fp8_tile.cuh"

namespace cql {
namespace {

constexpr int GM_THREADS = 512;
constexpr int GM_MAX_STAGES = 8;
constexpr int GM_NT = 224;                        // most tokens a tile
constexpr int GM_ACC = GM_NT / 2;                 // accumulator columns of an epilogue thread
constexpr int GM_SF_SLOTS = 4;
constexpr uint32_t GM_SF_COLS = 12;               // a slot: 4 columns of weight scales, up to 8 of token scales
constexpr int GM_REGS_SUM = 128 * 40 + 128 * 104 + 256 * 176, GM_REGS_DEC = 104;   // setmaxnreg of the roles below
static_assert(2 * GM_NT + GM_SF_SLOTS * GM_SF_COLS <= 512, "tensor-memory columns");

struct GmParams {
  F8Tokens tok;
  const uint32_t* wscale;                         // [quads][wrows]
  const uint32_t* xscale;                         // [quads][tokens]
  int64_t wrows;
  int n, units, row_tiles, stages;
  int early;                                      // weights and offsets may be read before the kernel before is done
  int debug;                                      // x is withheld, the waits are short
  void* y;
  int ydt, yvec;                                  // yvec: rows of y are 16-byte aligned
  int64_t ldy;
  uint32_t* status;
  F8Bounds in;
};

struct GmCtl {
  uint64_t full[GM_MAX_STAGES], empty[GM_MAX_STAGES];
  uint64_t sfull[GM_SF_SLOTS], sempty[GM_SF_SLOTS];
  uint64_t dfull[2], dempty[2], drain;
  uint32_t tmem_base;
};

CQL_DEV void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// If `on`: all earlier MMAs done -> an arrival on the barrier in the CTAs of `mask`.
CQL_DEV void commit_pair_if(uint32_t on, uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(mask), "r"(on)
      : "memory");
}
// If `on`: a copy into this CTA's shared memory whose bytes count on the barrier of
// the pair's first CTA (the same address with the CTA bit cleared).
CQL_DEV void tma_load_pair_if(uint32_t on, void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "@p cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar) & 0xFEFFFFFFu), "r"(x), "r"(y), "r"(z), "r"(on)
      : "memory");
}
// An arrival on the barrier of the cluster's CTA `rank`.  It orders tensor-memory
// accesses (which the tcgen05 fences around it do), no shared or global memory:
// with release semantics at cluster scope it costs some 700 cycles.
CQL_DEV void arrive_cluster(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}" ::"r"(smem_u32(bar)),
      "r"(rank)
      : "memory");
}

// A warp's 32 rows of W (lane = row) of sixteen tokens (fp32: eight) through its
// 1 KB of shared memory, so that a thread stores 16 consecutive bytes of a token.
// This code is unrolled over the accumulators, so it is kept short: what does not
// store whole vectors is a loop of its own, four stores in flight (with that and
// 32-column reads 7 experts of 10722 x 124, 759 tokens, went from 38 to 31 us).
// Sixteen tokens of all eight warps take some 640 cycles where every SM stores at
// once: the SMs' way to L2.  The rounding to y's type is the call's only one.
struct Out {
  int64_t ldy;
  int n_left;                                     // outputs from the warp's first row on
  bool vec;                                       // rows of y are 16-byte aligned and all 32 outputs exist
};
// y: the first token's first output.  left: tokens that exist.
CQL_DEV void store_tokens16(uint32_t* buf, const float* acc, uint16_t* y, int left, int dt, const Out& o) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[i * 32 + lane] = pack16(acc[2 * i], acc[2 * i + 1], dt);
  __syncwarp();
  if (o.vec) {
    const int t = 2 * (lane >> 2);
    const uint4 a = *reinterpret_cast<const uint4*>(buf + lane * 8), b = *reinterpret_cast<const uint4*>(buf + lane * 8 + 4);
    uint16_t* to = y + t * o.ldy + 8 * (lane & 3);
    if (t < left)
      *reinterpret_cast<uint4*>(to) = make_uint4(prmt(a.x, a.y, 0x5410u), prmt(a.z, a.w, 0x5410u), prmt(b.x, b.y, 0x5410u),
                                                 prmt(b.z, b.w, 0x5410u));
    if (t + 1 < left)
      *reinterpret_cast<uint4*>(to + o.ldy) = make_uint4(prmt(a.x, a.y, 0x7632u), prmt(a.z, a.w, 0x7632u),
                                                         prmt(b.x, b.y, 0x7632u), prmt(b.z, b.w, 0x7632u));
  } else if (lane < o.n_left) {
#pragma unroll 4
    for (int t = 0; t < min(16, left); ++t) y[t * o.ldy + lane] = (uint16_t)(buf[(t >> 1) * 32 + lane] >> (16 * (t & 1)));
  }
  __syncwarp();
}
CQL_DEV void store_tokens32(uint32_t* buf, const float* acc, uint32_t* y, int left, const Out& o) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[i * 32 + lane] = __float_as_uint(acc[i]);
  __syncwarp();
  if (o.vec) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = (lane >> 3) + 4 * r;
      if (t < left)
        *reinterpret_cast<uint4*>(y + t * o.ldy + 4 * (lane & 7)) = *reinterpret_cast<const uint4*>(buf + (lane + 32 * r) * 4);
    }
  } else if (lane < o.n_left) {
#pragma unroll 4
    for (int t = 0; t < min(8, left); ++t) y[t * o.ldy + lane] = buf[t * 32 + lane];
  }
  __syncwarp();
}

// Token columns that a tile multiplies: its tokens, up to a multiple of 32.  The
// copies are nt / 2 rows each all the same; rows behind the columns are not read.
// With uneven experts many tiles are partly filled, and long runs are bound by
// power: 32 experts of 2048 x 2048, 4096 uneven tokens, one call after another
// 51.3 us with nt columns for every tile, 50.0 like this.
CQL_DEV int gm_columns(const F8Tile& t) { return (t.t1 - t.t0 + 31) & ~31; }

// U: blocks of a unit.
template <int U>
__global__ void __launch_bounds__(GM_THREADS, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, GmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nt = p.tok.nt;
  // a stage: this CTA's share of a unit, [U][128 rows] of the weights, [U][nt / 2] of the tokens
  const uint32_t x_block = (uint32_t)nt * 64u, stage_bytes = U * (kF8ABytes + x_block);
  uint32_t* bounce = reinterpret_cast<uint32_t*>(ring + (uint32_t)p.stages * stage_bytes);     // 1 KB a warp
  GmCtl& S = *reinterpret_cast<GmCtl*>(bounce + 8 * 256);
  const F8Map map(&S + 1, p.tok.experts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), head = rank & ~1u;            // head: the pair's first CTA
  const uint16_t pair = (uint16_t)(3u << head);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 2);                   // the first CTA's two copying warps
      mbar_init(&S.empty[s], 1);
    }
    for (int s = 0; s < GM_SF_SLOTS; ++s) {
      mbar_init(&S.sfull[s], 8);                  // four warps of either CTA
      mbar_init(&S.sempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.dfull[s], 1);
      mbar_init(&S.dempty[s], 16);                // eight warps of either CTA
    }
    mbar_init(&S.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&S.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const bool early = p.early != 0;
  if (!early) pdl_wait();
  if (warp == 0) f8_scan(p.tok, map, p.status);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                               // the cluster's barriers and tensor memory are there
  cluster_wait();
  tc_fence_after();
  // The next kernel may start from here on, not before: it could take the
  // tensor memory that a CTA still has to allocate, and then wait for it.
  if (!early) pdl_launch_dependents();
  const uint32_t tmem = S.tmem_base;
  bool arrived = false;                           // at the closing cluster barrier
  const int tiles = map.start[p.tok.experts] * p.row_tiles;
  const uint32_t sf0 = tmem + 2u * nt;            // scale slots behind the accumulators
  const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  // Register split: GM_REGS_SUM of the 512 * 128 at launch (ready_gemm).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if ((warp & 1) == 0 && warp < 4 && elect_one()) {
      // ---------------- copies: warp 0 weights, warp 2 tokens ----------------
      const bool x = warp == 2;
      if (early && x) pdl_wait();
      const CUtensorMap* tm = x ? &tmX : &tmW;
      const uint32_t off = x ? U * kF8ABytes : 0u;
      // the pair's bytes, on its first CTA's barrier
      const uint32_t expect = rank == head ? 2 * U * (x ? x_block : kF8ABytes) : 0u;
      const int half = (int)(rank & 1);
      const uint32_t copies = !x || p.debug == 0;
      Ring at{0, 0};
      uint64_t lim = f8_limit(p.debug);
      for (int id = first; id < tiles && lim != 0; id += step) {
        const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
        const int row = x ? t.t0 + half * (gm_columns(t) >> 1) : t.expert * p.n + (2 * t.rt + half) * kF8Rows;
        for (int u = 0; u < p.units; ++u) {
          f8_wait(&S.empty[at.s], at.phase ^ 1, lim);
          const uint32_t on = copies & (lim != 0);
          expect_if(on ? expect : 0u, &S.full[at.s]);
          tma_load_pair_if(on, ring + (uint32_t)at.s * stage_bytes + off, tm, &S.full[at.s], 0, row, U * u);
          at.next_if(on, p.stages);
        }
      }
      for (int i = 0; i < p.stages; ++i) f8_wait(&S.empty[i], at.last(i), lim);
      if (lim == 0) {
        set_error(p.status, CQL_ERR_TIMEOUT, 44);
        // Copies in flight.  Both CTAs' show on the first one's barriers alone.
        uint64_t more = f8_limit(p.debug);
        if (rank == head) {
          for (int i = 0; i < p.stages; ++i) f8_wait(&S.full[i], at.last(i), more);
        } else {
          f8_pause();
        }
      }
    } else if (warp == 1 && rank == head && elect_one()) {
      // ---------------- MMA issuer ----------------
      // a tile's descriptor is made while the MMAs of the tile before run
      auto make_idesc = [&](int id) {
        return id < tiles ? f8_idesc(2 * kF8Rows, gm_columns(f8_tile(p.tok, map, p.row_tiles, id))) : 0u;
      };
      uint32_t idesc = make_idesc(first);
      const uint64_t desc0 = smem_desc_sw128(smem_u32(ring));
      uint32_t gc = 0;
      Ring at{0, 0}, sat{0, 0};
      uint64_t lim = f8_limit(p.debug);
      for (int id = first; id < tiles && lim != 0; id += step) {
        int chain = 0;                            // where the next accumulator chain starts
        uint32_t acc = 0;                         // the accumulator holds a sum already
        uint32_t ready = 0;                       // the next unit's copies are known to have landed
        auto unit = [&](int u) {
          f8_wait_if(ready ^ 1, &S.full[at.s], at.phase, lim);
          tc_fence_after();
          const uint32_t stage = (uint32_t)at.s;
          at.next(p.stages);
          ready = f8_peek(&S.full[at.s], at.phase);
          const uint32_t d = tmem + (gc & 1) * nt, sfa = sf0 + (uint32_t)sat.s * GM_SF_COLS;
          const uint64_t da = desc0 + (uint64_t)(stage * (stage_bytes >> 4));
          const uint64_t db = da + (U * kF8ABytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4 * U; ++kk)
            mma_f8_pair(d, da + (kk >> 2) * (kF8ABytes >> 4) + 2 * (kk & 3),
                        db + (uint64_t)((kk >> 2) * (x_block >> 4)) + 2 * (kk & 3), idesc | f8_byte(U * u + (kk >> 2)),
                        sfa, sfa + 4, kk == 0 ? acc : 1u);
          commit_pair_if(lim != 0, &S.empty[stage], pair);
          acc = 1;
        };
        // A chunk at a time (4 / U units): with the waits and commits of a
        // chunk out of the way a unit's own take less time than its MMAs.
        for (int u = 0; u < p.units;) {
          const int end = min(p.units, u + 4 / U);
          f8_wait_if(u == chain, &S.dempty[gc & 1], ((gc >> 1) & 1) ^ 1, lim);
          f8_wait(&S.sfull[sat.s], sat.phase, lim);
          if (lim == 0) break;
          if (end - u == 4 / U) {
#pragma unroll
            for (int i = 0; i < 4 / U; ++i) unit(u + i);
            u = end;
          } else {
            for (; u < end; ++u) unit(u);
          }
          commit_pair_if(lim != 0, &S.sempty[sat.s], pair);
          sat.next(GM_SF_SLOTS);
          const uint32_t over = u == f8_chain_end<U>(chain, p.units);
          commit_pair_if(over & (lim != 0), &S.dfull[gc & 1], pair);
          gc += over;
          acc ^= over;
          chain = over ? u : chain;
        }
        idesc = make_idesc(id + step);
      }
      // Both CTAs' epilogues have read the last accumulators: their arrivals are
      // the last ones that come to this CTA.
      for (uint32_t i = gc < 2 ? 0 : gc - 2; i < gc && lim != 0; ++i) f8_wait(&S.dempty[i & 1], (i >> 1) & 1, lim);
      if (lim == 0) {
        set_error(p.status, CQL_ERR_TIMEOUT, 45);
        uint64_t more = f8_limit(p.debug);
        commit_pair_if(1u, &S.drain, (uint16_t)(1u << head));         // MMAs in flight
        f8_wait(&S.drain, 0, more);
      }
    }
  } else if (warp < 8) {
    // ---------------- scale words ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    Ring at{0, 0};
    uint64_t lim = f8_limit(p.debug);
    bool ok = true;
    if (early) {
      pdl_wait();
      pdl_launch_dependents();
    }
    const int c1 = U * (p.units - 1) >> 2;        // chunks 0 .. c1
    for (int id = first; id < tiles && ok; id += step) {
      const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
      const int n0 = (2 * t.rt + (int)(rank & 1)) * kF8Rows + lane;
      const uint32_t* ws = p.wscale + (int64_t)t.expert * p.n + n0;
      const uint32_t* xs = p.xscale + t.t0 + lane;
      for (int c = 0; c <= c1 && ok; c += 4) {
        uint32_t w[4][12];                        // four chunks' words, on their way together
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j)             // rows past the expert's last: any finite scale.  From L2: see k_fp8_quantize
            w[i][j] = c + i <= c1 && n0 + 32 * j < p.n &&
                              CQL_IN(p.status, ws - p.wscale + (int64_t)(c + i) * p.wrows + 32 * j, p.in.wscale, 421)
                          ? ld_cg_u32(ws + (int64_t)(c + i) * p.wrows + 32 * j)
                          : 0x7F7F7F7Fu;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[i][4 + j] = c + i <= c1 && 32 * j < nt && t.t0 + 32 * j + lane < t.t1 &&
                                  CQL_IN(p.status, xs - p.xscale + (int64_t)(c + i) * p.tok.tokens + 32 * j, p.in.xscale, 422)
                              ? ld_cg_u32(xs + (int64_t)(c + i) * p.tok.tokens + 32 * j)
                              : 0x7F7F7F7Fu;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c + i > c1) break;
          f8_wait(&S.sempty[at.s], at.phase ^ 1, lim);
          ok = __all_sync(0xffffffffu, lim != 0);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sf = sf0 + lanes + (uint32_t)at.s * GM_SF_COLS;
          tmem_st4(sf, w[i]);
          tmem_st4(sf + 4, w[i] + 4);
          if (nt > 128) tmem_st4(sf + 8, w[i] + 8);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(&S.sfull[at.s], head);
          at.next(GM_SF_SLOTS);
        }
      }
    }
    for (int i = 0; i < GM_SF_SLOTS; ++i) f8_wait(&S.sempty[i], at.last(i), lim);
    if (!__all_sync(0xffffffffu, lim != 0) && lane == 0) set_error(p.status, CQL_ERR_TIMEOUT, 46);
  } else {
    // ---------------- epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int q = warp & 3, h = (warp - 8) >> 2;
    uint32_t* buf32 = bounce + (warp - 8) * 256;
    uint32_t gc = 0;
    uint64_t lim = f8_limit(p.debug);
    bool ok = true;
    if (early) pdl_wait();                        // y may be in use by the kernel before
    for (int id = first; id < tiles && ok; id += step) {
      const F8Tile t = f8_tile(p.tok, map, p.row_tiles, id);
      const int n0 = t.rt * 2 * kF8Rows + (int)(rank & 1) * kF8Rows;
      const int part = gm_columns(t) >> 1, c0 = h * part;             // this warp's token columns [c0, c0 + part)
      float acc[GM_ACC];
#pragma unroll
      for (int i = 0; i < GM_ACC; ++i) acc[i] = 0.0f;
      for (int u = 0; u < p.units; u = f8_chain_end<U>(u, p.units), ++gc) {
        const uint32_t buf = gc & 1;
        f8_wait(&S.dfull[buf], (gc >> 1) & 1, lim);
        ok = __all_sync(0xffffffffu, lim != 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + buf * nt + c0;
#pragma unroll
        for (int c = 0; c < GM_ACC; c += 32) {
          if (c + 32 <= part) {
            float v[32];
            tmem_ld32(base + c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < GM_ACC) acc[c + i] += v[i];
          } else if (c < part) {
            float v[16];
            tmem_ld_wait<16>(base + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(&S.dempty[buf], head);
      }
      if (!ok) break;
      if (id + step >= tiles) {
        // The accumulators are read, and the first CTA waits for the arrivals that
        // say so: the pair may end while this is stored.  A release behind the
        // stores waits for all of them, some 1300 cycles (4096 x 4096, 640 tokens:
        // 13.8 us with it, 13.1 like this).
        tc_fence_before();
        cluster_arrive();
      }
      const int nw = n0 + 32 * q, left = t.t1 - t.t0 - c0;
      const Out o{p.ldy, p.n - nw, p.yvec && nw + 32 <= p.n};
      const int64_t y0 = (int64_t)(t.t0 + c0) * p.ldy + nw;
      // the warp's last output
      if (left <= 0 || o.n_left <= 0 ||
          !CQL_IN(p.status, y0 + (int64_t)(min(left, part) - 1) * p.ldy + min(32, o.n_left) - 1, p.in.y, 423))
        continue;
      if (p.ydt == CQL_DT_F32) {
        uint32_t* y = reinterpret_cast<uint32_t*>(p.y) + y0;
#pragma unroll
        for (int c = 0; c < GM_ACC; c += 8)
          if (c < part && c < left) store_tokens32(buf32, acc + c, y + c * p.ldy, left - c, o);
      } else {
        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + y0;
#pragma unroll
        for (int c = 0; c < GM_ACC; c += 16)
          if (c < part && c < left) store_tokens16(buf32, acc + c, y + c * p.ldy, left - c, p.ydt, o);
      }
    }
    if (!ok && lane == 0) set_error(p.status, CQL_ERR_TIMEOUT, 47);
    arrived = ok && first < tiles;
  }
  __syncwarp();
  if (!arrived) {
    tc_fence_before();
    cluster_arrive_release();
  }
  cluster_wait();                                 // nothing of the cluster reads or signals this CTA any more
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

// The kernel may be launched on the current device, and its registers at launch hold
// the split that its roles make of them.
template <int U>
static cudaError_t ready_gemm() {
  static std::atomic<uint64_t> attr_done{0};
  static KeptAnswer kept;
  cudaError_t e = ensure_smem_attr(attr_done, (const void*)k_fp8_gemm<U>, 227 * 1024);
  if (e != cudaSuccess) return e;
  int regs = 0;
  e = (cudaError_t)kept.get(regs, [](int& n) {
    cudaFuncAttributes a;
    const cudaError_t r = cudaFuncGetAttributes(&a, (const void*)k_fp8_gemm<U>);
    n = r == cudaSuccess ? a.numRegs : 0;
    return (int)r;
  });
  if (e != cudaSuccess) return e;
  return register_split_fits(regs, GM_THREADS, GM_REGS_SUM, GM_REGS_DEC) ? cudaSuccess : cudaErrorInvalidConfiguration;
}

cudaError_t ready_fp8_gemm() {
  const cudaError_t e = ready_gemm<1>();
  return e != cudaSuccess ? e : ready_gemm<2>();
}

template <int U>
static cudaError_t launch_gemm(const Fp8Product& f, GmParams& p, int64_t tiles, cudaStream_t st) {
  const cudaError_t e = ready_gemm<U>();
  if (e != cudaSuccess) return e;
  const int pairs = device_sm_count() / 2, nt = p.tok.nt;
  p.units = (f.w.blocks + U - 1) / U;
  const uint32_t stage = U * (kF8ABytes + (uint32_t)nt * 64u);
  const uint32_t behind = 8u * 1024u + (uint32_t)sizeof(GmCtl) + F8Map::bytes(f.experts);
  p.stages = (int)((227u * 1024u - 1024u - behind) / stage);
  if (p.stages > GM_MAX_STAGES) p.stages = GM_MAX_STAGES;
  if (p.stages < 2) return cudaErrorInvalidConfiguration;
  const int smem = (int)(1024u + (uint32_t)p.stages * stage + behind);
  CUtensorMap mw, mx;
  if (!make_map_codes(&mw, f.w_base, (uint64_t)f.w.rows, (uint64_t)f.w.blocks, kF8Rows, U) ||
      !make_map_codes(&mx, f.x_base, (uint64_t)f.x.rows, (uint64_t)f.x.blocks, (uint32_t)(nt / 2), U))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(GM_THREADS);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp8_gemm<U>, mw, mx, p);
}

cudaError_t launch_fp8_gemm(const Fp8Product& f, cudaStream_t st) {
  GmParams p{};
  p.tok.offsets = f.offsets;
  p.tok.experts = f.experts;
  p.tok.tokens = (int)f.x.rows;
  p.wscale = reinterpret_cast<const uint32_t*>(f.w_base + f.w.scales_off);
  p.xscale = reinterpret_cast<const uint32_t*>(f.x_base + f.x.scales_off);
  p.wrows = f.w.rows;
  p.n = f.n;
  p.row_tiles = (f.n + 2 * kF8Rows - 1) / (2 * kF8Rows);
  p.early = f.early;
  p.debug = f.debug;
  p.y = f.y;
  p.ydt = f.ydt;
  p.yvec = (reinterpret_cast<uintptr_t>(f.y) & 15) == 0 && (f.ldy * (f.ydt == CQL_DT_F32 ? 4 : 2)) % 16 == 0;
  p.ldy = f.ldy;
  p.status = f.status;
  p.in = {f.w.scales_len / 4, f.x.scales_len / 4, 0, fp8_extent(f.x.rows, f.ldy, f.n)};
  // Token tiles.  A block of a tile takes about 90 + 0.69 nt ns (measured on one
  // pair: 142 ns at nt 64, 173 at 128, 244 at 224), so the cost of a choice is
  // the number of rounds over the pairs times 130 + nt.  The host does not know the
  // experts' loads: the rule takes them for even and every tile for full.  The copies
  // are nt tokens wide for every tile; the MMAs of a part-filled one are narrower
  // (gm_columns), so with uneven loads the true cost is below the rule's and a wider
  // nt may be the better one (32 experts of 2048 x 2048, 4096 tokens, loads as 1 /
  // rank: nt 128, 384 tiles, 5.2 rounds; 160 would be 360 tiles, 4.9; not timed).
  const int pairs = device_sm_count() / 2;
  const int per = (p.tok.tokens + f.experts - 1) / f.experts;         // tokens of an expert, evenly loaded
  int64_t best = 0, tiles = 0;
  for (int nt = 32; nt <= GM_NT; nt += 32) {
    const int64_t n = (int64_t)f.experts * ((per + nt - 1) / nt) * p.row_tiles;
    const int64_t cost = (n + pairs - 1) / pairs * (130 + nt);
    if (best != 0 && cost >= best) continue;
    best = cost;
    p.tok.nt = nt;
  }
  // at most one partly filled token tile an expert
  tiles = (int64_t)p.tok.tokens / p.tok.nt + f.experts;
  if (tiles > p.tok.tokens) tiles = p.tok.tokens;
  if (f.offsets == nullptr) tiles = (p.tok.tokens + p.tok.nt - 1) / p.tok.nt;
  tiles *= p.row_tiles;
  return p.tok.nt > 64 ? launch_gemm<1>(f, p, tiles, st) : launch_gemm<2>(f, p, tiles, st);
}

}  // namespace cql
