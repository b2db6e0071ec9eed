// What the two block-scaled FP8 product kernels share: bounded waits, cluster
// primitives, the ring position, and the tiles of ragged experts.
#pragma once
#include "fp8.cuh"
#include "tc.cuh"

namespace cql {

constexpr int kF8Rows = 128;                      // weight rows of a CTA's tile (tensor-memory lanes)
constexpr uint32_t kF8ABytes = kF8Rows * 128;     // their codes of one block
// K goes in units of one or two blocks: a copy of each operand and a barrier a
// unit.  The block behind an odd last one reads as zero codes.
// Blocks of one accumulator chain (2048 columns, up to three blocks more where
// a range starts inside a chunk).  The tensor core truncates
// when it adds to its accumulator, an error that grows with the chain: 4096
// columns in one chain were 1.8e-6 off, 11008 6.4e-6 (relative, 2-norm).
// Chains of at most 2048 are summed in fp32 registers.
constexpr int kF8Seg = 16;

// Waits for a barrier's phase if `on`; bounded by `lim` clock cycles.  Once a
// wait has run out, lim is 0 and every further one tries just once: the role
// signals nothing and issues no copy any more, so that those which wait for it
// run out as well, and stops at the next turn where it looks at lim.
// The loop is written in PTX, without a result to branch on: a wait that finds
// its phase complete costs the issuing thread about 50 cycles like this, 190
// where C++ branches on the outcome (measured on single-thread loops; the MMA
// and copy loops below are flat for the same reason).  The first try carries no
// suspend-time hint, which costs a completed phase 50 cycles more; a warp that
// has to wait is suspended and leaves the issue slots to the others.  The lanes of
// a warp may leave it one after the other: __syncwarp before a tcgen05 or cluster
// operation of the warp.
CQL_DEV void f8_wait_if(uint32_t on, uint64_t* bar, uint32_t parity, uint64_t& lim) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u64 t, e;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "@p bra D;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%2], %3;\n\t"
      "@p bra D;\n\t"
      "mov.u64 e, %%clock64;\n\t"
      "add.u64 e, e, %0;\n\t"
      "L:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%2], %3, %4;\n\t"
      "@p bra D;\n\t"
      "mov.u64 t, %%clock64;\n\t"
      "setp.lt.u64 q, t, e;\n\t"
      "@q bra L;\n\t"
      "D:\n\t"
      "selp.u64 %0, %0, 0, p;\n\t}"
      : "+l"(lim)
      : "r"(on), "r"(smem_u32(bar)), "r"(parity), "r"(kTcSuspendNs)
      : "memory");
}
CQL_DEV void f8_wait(uint64_t* bar, uint32_t parity, uint64_t& lim) { f8_wait_if(1u, bar, parity, lim); }
// Whether the phase is complete already: asked before the MMAs of one unit are
// issued, for the next unit's copies, so that the answer costs no time.
CQL_DEV uint32_t f8_peek(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done;
}
// debug: a test withholds x to let the waits run out.
CQL_DEV uint64_t f8_limit(int debug) { return (uint64_t)(debug ? kTcDebugWaitCycles : kTcWaitCycles); }
// Some 2 ms, for copies from the cluster's other CTAs that no barrier of this one
// counts any more (after a wait that ran out): their last chance to land.
constexpr long long kF8Pause = 4000000ll;
CQL_DEV void f8_pause() {
  const long long t0 = clock64();
  while (clock64() - t0 < kF8Pause) {
  }
}
// If bytes > 0: an arrival that expects them.
CQL_DEV void expect_if(uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}

// If `on`: tma_load_3d.
CQL_DEV void tma_load_3d_if(uint32_t on, void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %6, 0;\n\t"
      "@p cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(on)
      : "memory");
}

// One lane of a converged warp.
CQL_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The two halves of a cluster barrier, reached by whole warps.  The forms that let
// lanes come one by one stood here, behind code where lanes part, when now and then
// a push went to a CTA that had not started; that a barrier completed early for it
// is inferred by reading, not shown.
// cluster_arrive orders no memory accesses (barriers are initialised before it
// under fence.mbarrier_init).
CQL_DEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
CQL_DEV void cluster_arrive_release() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
CQL_DEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
CQL_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A float into the shared memory of the cluster's CTA `rank`, counted on its
// barrier there (addresses as this CTA has them).
CQL_DEV void push_cluster(uint32_t addr, uint32_t bar, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 ra, rb;\n\t"
      "mapa.shared::cluster.u32 ra, %0, %2;\n\t"
      "mapa.shared::cluster.u32 rb, %1, %2;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [ra], %3, [rb];\n\t}" ::"r"(addr),
      "r"(bar), "r"(rank), "f"(v)
      : "memory");
}

// Four consecutive outputs of a token, v[0 .. left) of them, at element `at` of
// y; vec: `at` is a multiple of 16 bytes' elements.
CQL_DEV void store4(void* y, int dt, int64_t at, float4 v, int left, bool vec) {
  if (vec && left >= 4) {
    if (dt == CQL_DT_F32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + at) = v;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(y) + at) =
          make_uint2(pack16(v.x, v.y, dt), pack16(v.z, v.w, dt));
  } else {
    if (left > 0) store_out(y, dt, (uint64_t)at, v.x);
    if (left > 1) store_out(y, dt, (uint64_t)at + 1, v.y);
    if (left > 2) store_out(y, dt, (uint64_t)at + 2, v.z);
    if (left > 3) store_out(y, dt, (uint64_t)at + 3, v.w);
  }
}

CQL_DEV void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
CQL_DEV void tmem_st4(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// Instruction descriptor: e4m3 x e4m3, both K-major, fp32 accumulator, UE8M0
// scales, M = m, N = n.  The scale byte of block kb is ORed in by f8_byte.
CQL_HD uint32_t f8_idesc(int m, int n) { return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27); }
CQL_HD uint32_t f8_byte(int kb) { return ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29); }

// Where the accumulator chain that starts at unit u (U blocks a unit) of a range
// up to u1 ends: the first chunk border at or behind kF8Seg blocks.
template <int U>
CQL_HD int f8_chain_end(int u, int u1) {
  const int end = (u + (kF8Seg + 3) / U) & ~(4 / U - 1);
  return end < u1 ? end : u1;
}

// Position in a ring: the slot and the parity of its round (kept by counting:
// a division by a runtime number of slots costs a role more than the rest of
// its turn).
struct Ring {
  int s;
  uint32_t phase;
  CQL_DEV void next(int slots) { next_if(1u, slots); }
  CQL_DEV void next_if(uint32_t on, int slots) {
    s += (int)on;
    const bool wrap = s == slots;
    s = wrap ? 0 : s;
    phase ^= wrap ? 1u : 0u;
  }
  // parity of slot i's last round
  CQL_DEV uint32_t last(int i) const { return phase ^ (i < s ? 0u : 1u); }
};

// Sizes that the checked build holds indices against: words of the two scale
// planes, elements of x and y.
struct F8Bounds {
  uint64_t wscale, xscale, x, y;
};

// The tokens of the experts, cut into tiles of nt tokens.
struct F8Tokens {
  const int32_t* offsets;                         // [experts + 1], or null: one expert, every token
  int experts, tokens, nt;
};
struct F8Tile {
  int expert, rt, t0, t1;                         // row tile rt of the expert, tokens [t0, t1)
};

// Tokens [offsets[e], offsets[e+1]) of an expert; a pair that does not lie in
// order within [0, tokens] is an empty expert (and an error: false).  Read past L1:
// the kernels before are done, but a launch that starts early says so only by its wait.
CQL_DEV bool f8_segment(const F8Tokens& p, int e, int& t0, int& t1) {
  if (p.offsets == nullptr) {
    t0 = 0;
    t1 = p.tokens;
    return true;
  }
  t0 = __ldcg(p.offsets + e);
  t1 = __ldcg(p.offsets + e + 1);
  if (t0 >= 0 && t0 <= t1 && t1 <= p.tokens) return true;
  t0 = t1 = 0;
  return false;
}

// What a CTA keeps of the experts in shared memory: seg[e] = tokens [x, y) of an
// expert, start[e] = token tiles of the experts before it (start[experts]: all).
struct F8Map {
  int2* seg;
  int* start;
  CQL_HD static uint32_t bytes(int experts) { return 12u * (uint32_t)experts + 4u; }
  CQL_DEV F8Map(void* at, int experts) : seg(reinterpret_cast<int2*>(at)), start(reinterpret_cast<int*>(seg + experts)) {}
};

// Fills the map.  One warp.
CQL_DEV void f8_scan(const F8Tokens& p, const F8Map& m, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  bool bad = false;
  for (int e0 = 0; e0 < p.experts; e0 += 32) {
    const int e = e0 + lane;
    int t0 = 0, t1 = 0;
    if (e < p.experts) {
      bad |= !f8_segment(p, e, t0, t1);
      m.seg[e] = make_int2(t0, t1);
    }
    int v = (t1 - t0 + p.nt - 1) / p.nt;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (e < p.experts) m.start[e + 1] = base + v;
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) m.start[0] = 0;
  if (__any_sync(0xffffffffu, bad) && blockIdx.x == 0 && lane == 0) set_error(status, CQL_ERR_RANGE, 401);
}

// Tile `id`: experts in order, then row tiles, then token tiles (the token
// tiles of one weight tile are neighbours: the weights come from L2 after the
// first).
CQL_DEV F8Tile f8_tile(const F8Tokens& p, const F8Map& m, int row_tiles, int id) {
  int lo = 0, hi = p.experts - 1;
  while (lo < hi) {                               // last e with start[e] * row_tiles <= id
    const int mid = (lo + hi + 1) >> 1;
    if (m.start[mid] * row_tiles <= id) lo = mid;
    else hi = mid - 1;
  }
  const int tt = m.start[lo + 1] - m.start[lo];
  const int local = id - m.start[lo] * row_tiles;
  const int2 seg = m.seg[lo];
  F8Tile t;
  t.expert = lo;
  t.rt = tt == 1 ? local : local / tt;
  t.t0 = seg.x + (local - t.rt * tt) * p.nt;
  t.t1 = min(seg.y, t.t0 + p.nt);
  return t;
}

}  // namespace cql
