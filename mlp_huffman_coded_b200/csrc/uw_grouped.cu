// Reconstructive GEMM over groups of rows (one compressed matrix per group)
// with a fused epilogue: the products of a mixture of experts
//   y[s] = act(x[rows[s]] W_e^T + b_e) + r[s],       e = the group of slot s,
//   h[s] = SiLU(x[rows[s]] G_e^T) * (x[rows[s]] U_e^T)
// and, with one group, the product of one matrix with bias, activation and
// residual in its epilogue.
//
// Method: Cloudflare, "Unweight: how we compressed an LLM 22% without
// sacrificing quality", section "How the reconstructive matmul works"
// (compressed tiles staged on chip, rebuilt there, fed to the tensor cores).
// The page speaks of one matrix; the groups and the epilogue are not on it.
//
// What bounds it: with few rows per group, the bytes of the active groups'
// packs (1.502 per weight plus 2 per verbatim weight); with many, the MMA
// rate and the rebuild of each 128 x 64 weight tile (193 ALU instructions per
// warp at one per two cycles: 386 cycles, against 2 N cycles for the four MMAs
// of N columns).
//
// Layout of the work:
//  * W is the MMA's A operand (128 weight rows = 128 TMEM lanes), the rows of
//    the group are the N side (16..256 columns): decode-time groups of a few
//    rows cost one N = 16 MMA, and nothing is padded to 128 rows.
//  * The work is tiles (group, 128 weight rows, columns) of K / 64 k-blocks.
//    Group sizes are read on the device; every CTA computes the same table of
//    tiles and takes whole tiles in waves and then an equal run of the k-blocks
//    that are left (stream-K), so ragged groups, few large tiles and many
//    small ones balance alike.  A group without rows has no tiles: its weights
//    are never read.
//  * Every ring slot carries ONE tile record (12304 bytes and its verbatim
//    rows): it goes back to the producer as soon as that tile is rebuilt, so
//    nearly all of the weight ring is in flight to HBM at any time.
//  * With SwiGLU, the gate and the up tile of a k-block follow each other
//    through the same rings and share the activation tile; both sums stay in
//    tensor memory and meet in the epilogue, so g and u are never rounded or
//    stored.
//  * The rows of x arrive in TMA boxes of 64 and 16 rows, or, where a group's
//    rows are scattered, by TMA gather (4 row numbers per copy) while groups
//    are small; the gather takes about 75 cycles per 4 rows, so beyond
//    kGatherCap rows per tile a small kernel first copies the rows next to
//    each other.
//  * A tile shared by several CTAs: each writes its FP32 sums to a slot of
//    its own (a CTA has at most two such tiles, its first and its last) and
//    takes a ticket; the last adds all of them in CTA order and runs the
//    epilogue.  Nobody waits for another CTA; the sum does not depend on
//    timing.
//  * Barrier waits are bounded: a timeout records UW_ERR_TIMEOUT, drains
//    copies and MMAs in flight, frees tensor memory and returns.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

// Warp roles: 0 = weight producer, 1 = activation producer, 2..3 = MMA
// issuers (warp 2 owns tensor memory), 4..19 = four rebuild groups of 4 warps
// (group g rebuilds tiles i with i % 4 == g), 20..23 = epilogue.
constexpr int kGroups = 4;
constexpr int kMaxIssuers = 2;
constexpr int kWarpW = 0, kWarpX = 1, kWarpMma = 2, kWarpRebuild = 4, kWarpEpi = kWarpRebuild + 4 * kGroups;
constexpr int kThreads = 32 * (kWarpEpi + 4);
constexpr int kMaxSlots = 16;
constexpr int kWBatch = 4;  // tiles that the weight producer issues at a time
// Columns (times matrices) of a CTA's last tile above which all warps empty its
// accumulators: 1000 rows of 4096 x 4096 34.1 us against 38.5, 664 rows of 7292
// x 576 with GELU 32.3 / 37.6; one row of 4096 x 4096 takes 1 us more by it.
constexpr int kTogether = 48;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBody = 12304, kBodyIdx = 8192, kBodyMask = 12288;  // pack record of a tile (uw.h)
constexpr uint32_t kMinTail = 8;  // verbatim rows staged per tile, at least
constexpr size_t kSmemLimit = 227 * 1024;
constexpr size_t kSmemFloor = 120 * 1024;  // one CTA (and one owner of tensor memory) per SM

// One group's share of the schedule.
struct SchedEntry {
  int tile0;      // first tile
  int start;      // first slot
  int count;      // slots
  int n_nt;       // column tiles in bits 16.., columns per tile (multiple of 16) in bits 0..15
};

struct GParams {
  int E, N, KB, x_rows, n_rows;
  int n_mt, n_mt_all;   // row tiles of the schedule (pairs with PAIR), and of the matrix
  int grid, cap;        // columns per tile, at most
  int n_iss, n_acc;
  int sx, sa, sw;       // ring slots: activations, A tiles (tensor memory), weight records
  uint32_t x_slot_bytes, w_base, w_slot_bytes, sched_off, turn_off, bar_off, a_col0;
  int vec;              // rows of y and the residual start on 16 bytes
  int vcap;             // verbatim rows staged per record
  int join;             // what joining a shared tile costs, in k-blocks
  int min_run;          // shortest run of a shared tile, in k-blocks
  int early;            // offsets are not the previous kernel's output
  int gather;           // x rows by number (TMA gather), else in boxes
  const int32_t* offsets;
  const int32_t* rows;
  const ExpertDesc* table[2];
  ExpertDesc one;       // the only group's record when table[0] is NULL
  const uint16_t* bias;
  const uint16_t* residual;
  int act, out_fp32;
  void* y;
  float* partials;
  long long partial_stride;  // floats of one partial slot
  uint32_t* counters;
  uint32_t* status;
};

// A tile shared by CTAs c_first..c_last whose last part this CTA delivered;
// first_slot: the partial slot of c_first (the others use their slot 0).
struct Todo {
  int e, mt, slot0, nvalid, c_first, c_last, first_slot, pad;
};

// The tiles (group, row tile, column tile), column tiles of a row tile next to
// each other, are dealt out in waves of one tile per CTA: CTAs that work at
// the same time share weight tiles (the column tiles of a row tile) and
// activation tiles through L2.  What does not fill waves evenly (up to two
// tiles per CTA) is cut into equal runs of k-blocks (stream-K).  Contiguous
// shares for all tiles instead read the weights of three column tiles three
// times from HBM: a CTA came to its next column tile when L2 had moved on.
struct Share {
  int grid, waves;        // CTAs that take part, whole tiles per CTA
  int sk_each, sk_long;   // k-blocks of the tiles after the waves: lengths of the runs
  int u0, u1;             // this CTA's run of them
};

// A CTA's work as segments: runs of k-blocks of one tile.  Every role walks
// the same sequence.
struct Seg {
  int wave, u;        // waves done, next k-block of the run
  int e, mt, nt;
  int kb0, kb1;
  int ntile, slot0, nvalid;
  int tile_u;         // first k-block of the whole tile in the run's count
};

struct GBars {
  uint64_t wfull[kMaxSlots], wempty[kMaxSlots];
  uint64_t xfull[kMaxSlots], xempty[kMaxSlots];
  uint64_t afull[kMaxSlots], aempty[kMaxSlots];
  uint64_t acc_full[2], acc_empty[2], drain[kMaxIssuers];
  uint32_t tail_first[kMaxSlots];  // per weight slot: first verbatim row of its tile
  uint32_t tmem_base, abort, n_todo;
  // the last segment, when all warps finish it: accumulator buffer, first tile
  uint32_t together, last_acc, last_tile;
  Share share;
  Seg first, last;     // segments
  ExpertDesc desc[2];  // the first segment's matrices
  Todo todo[2];
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Takes a ticket: releases this thread's writes and those of the threads it
// has met at a CTA barrier, and acquires what earlier tickets released.
__device__ __forceinline__ uint32_t ticket(uint32_t* p) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// One lane of the warp, the same every time (a converged warp elects alike).
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// A warp's wait.  The polling loop stays out of line: with it inlined at every
// wait the loops outgrow the instruction caches (decode products +5%).
__device__ __noinline__ bool warp_wait_long(uint64_t* bar, uint32_t parity, GBars* b, uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, &b->abort, status));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, GBars* b, uint32_t* status) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_long(bar, parity, b, status);
}

// the 4 epilogue warps (named barrier 1)
__device__ __forceinline__ bool group_and(bool v) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return out != 0;
}
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Four rows of a 2-D tensor map (box one row high) at column c, packed one
// below the other.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int c, int r0, int r1, int r2, int r3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------- schedule ------------------------------------

// a / b for 0 <= a, 0 < b, from the approximate quotient: the set-up is a
// chain of divisions, and the exact one takes 40 instructions.
__device__ __forceinline__ int quick_div(int a, int b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  // (modulo 2^32: q b may pass 2^31 where a is near it)
  int r = static_cast<int>(static_cast<uint32_t>(a) - static_cast<uint32_t>(q) * static_cast<uint32_t>(b));
  while (r < 0) {
    --q;
    r += b;
  }
  while (r >= b) {
    ++q;
    r -= b;
  }
  return q;
}

// Runs of the k-blocks: the first sk_long CTAs have one more than the others.
__device__ __forceinline__ int units_before(int c, const Share& h) { return c * h.sk_each + min(c, h.sk_long); }
// CTA whose run holds k-block u
__device__ __forceinline__ int unit_owner(int u, const Share& h) {
  const int in_long = h.sk_long * (h.sk_each + 1);
  return u < in_long ? quick_div(u, h.sk_each + 1) : h.sk_long + quick_div(u - in_long, h.sk_each);
}

// wide: some group has more than one column tile
__device__ __forceinline__ Share share_of(int cta, int tiles, bool wide, const GParams& p) {
  Share h;
  // few tiles are not cut into runs shorter than min_run (joining many parts
  // costs more than it saves); the CTAs beyond have nothing, and every CTA
  // that the shares count has at least one k-block
  h.grid = min(p.grid, max(tiles, quick_div(tiles * p.KB, p.min_run)));
  h.waves = h.sk_each = h.sk_long = h.u0 = h.u1 = 0;
  if (cta >= h.grid) return h;
  const int full = quick_div(tiles, h.grid), rest = tiles - full * h.grid;
  // The run of the last, partial wave is long enough to be worth joining
  // alone only when it is some k-blocks long; then a wave more leaves fewer
  // column tiles apart in time from those they share weights with.  (8 x 512
  // rows of 4096 x 14336: 568 us with runs of 1.6 tiles, 487 with runs of 0.6
  // after the waves; without column tiles to share with, 1 row of 8 experts,
  // 59.5 against 62.1.)
  const bool wave_more = wide && rest * p.KB >= 2 * p.join * h.grid;
  h.waves = rest && full && !wave_more ? full - 1 : full;
  const int units = (tiles - h.waves * h.grid) * p.KB;
  // The last tiles are shared out only where that saves more k-blocks than
  // joining the parts costs
  if (units <= h.grid * p.KB && p.KB <= quick_div(units, h.grid) + p.join) {
    h.waves += cta < tiles - h.waves * h.grid ? 1 : 0;
  } else if (h.waves < full && 2 * p.KB <= quick_div(units, h.grid) + p.join) {
    h.waves = full + (cta < rest ? 1 : 0);
  } else if (units) {
    h.sk_each = quick_div(units, h.grid);
    h.sk_long = units - h.sk_each * h.grid;
    h.u0 = units_before(cta, h);
    h.u1 = units_before(cta + 1, h);
  }
  return h;
}

__device__ __forceinline__ void seg_fill(Seg& s, const SchedEntry* sched, const GParams& p, int tile) {
  // the last entry with tile0 <= tile, from the current one on (entries
  // without tiles share their successor's tile0)
  if (tile >= sched[s.e + 1].tile0) {
    int lo = s.e + 1, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sched[mid].tile0 <= tile) lo = mid;
      else hi = mid;
    }
    s.e = lo;
  }
  const SchedEntry en = sched[s.e];
  const int n_nt = en.n_nt >> 16;
  s.mt = tile - en.tile0;
  s.nt = 0;
  if (n_nt > 1) {
    const int local = s.mt;
    s.mt = quick_div(local, n_nt);
    s.nt = local - s.mt * n_nt;
  }
  s.ntile = en.n_nt & 0xFFFF;
  s.slot0 = en.start + s.nt * s.ntile;
  s.nvalid = min(s.ntile, en.count - s.nt * s.ntile);
}
__device__ __forceinline__ void seg_here(Seg& s, const SchedEntry* sched, const GParams& p, const Share& h, int cta) {
  if (s.wave < h.waves) {
    s.kb0 = 0;
    s.kb1 = p.KB;
    seg_fill(s, sched, p, s.wave * h.grid + cta);
  } else {
    const int tile = quick_div(s.u, p.KB);
    s.kb0 = s.u - tile * p.KB;
    s.kb1 = min(p.KB, s.kb0 + (h.u1 - s.u));
    s.tile_u = s.u - s.kb0;
    seg_fill(s, sched, p, h.waves * h.grid + tile);
  }
}
// first segment of a share that is not empty
__device__ __forceinline__ void seg_init(Seg& s, const SchedEntry* sched, const GParams& p, const Share& h, int cta) {
  s.wave = 0;
  s.u = h.u0;
  s.e = 0;
  s.tile_u = 0;
  seg_here(s, sched, p, h, cta);
}
// whether the segment is the share's last
__device__ __forceinline__ bool seg_last(const Seg& s, const Share& h) {
  return s.wave < h.waves ? s.wave + 1 == h.waves && h.u0 >= h.u1 : s.u + (s.kb1 - s.kb0) >= h.u1;
}
// false when the share is done
__device__ __forceinline__ bool seg_next(Seg& s, const SchedEntry* sched, const GParams& p, const Share& h, int cta) {
  if (s.wave < h.waves) ++s.wave;
  else s.u += s.kb1 - s.kb0;
  if (s.wave >= h.waves && s.u >= h.u1) return false;
  seg_here(s, sched, p, h, cta);
  return true;
}

struct Ring {
  int slot;
  uint32_t use;
};
__device__ __forceinline__ void ring_next(Ring& r, int slots, int step = 1) {  // step <= slots
  r.slot += step;
  if (r.slot >= slots) {
    r.slot -= slots;
    ++r.use;
  }
}

// Row tile of matrix m of the k-block: with PAIR the two "matrices" are two
// row tiles of one (the last one twice where their number is odd).
template <bool PAIR>
__device__ __forceinline__ int row_tile(const GParams& p, int mt, int m) {
  return PAIR ? min(2 * mt + m, p.n_mt_all - 1) : mt;
}

// ------------------------------- rebuild -------------------------------------
// One thread owns one weight row of the tile: 64 BF16 values as 32 words.
// Plain 16-byte shared-memory reads (the record's chunk order keeps them free
// of bank conflicts); exponents come from two byte permutes per four indices.
__device__ __forceinline__ void rebuild_row(const PaletteTables& pal, bool uniform, uint32_t body, int r,
                                            uint32_t (&o)[32]) {
  uint32_t iw[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 v = lds128(body + kBodyIdx + r * 32 + ((j ^ ((r >> 2) & 1)) << 4));
    iw[4 * j] = v.x;
    iw[4 * j + 1] = v.y;
    iw[4 * j + 2] = v.z;
    iw[4 * j + 3] = v.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 s = lds128(body + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    const uint32_t sw[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t nib = iw[2 * j + h];
      uint32_t e0, e1;
      if (uniform) {
        e0 = lookup4_uniform(pal, nib);
        e1 = lookup4_uniform(pal, nib >> 16);
      } else {
        e0 = lookup4_mixed(pal, nib);
        e1 = lookup4_mixed(pal, nib >> 16);
      }
      rebuild4(sw[2 * h], e0, o[8 * j + 4 * h + 0], o[8 * j + 4 * h + 1]);
      rebuild4(sw[2 * h + 1], e1, o[8 * j + 4 * h + 2], o[8 * j + 4 * h + 3]);
    }
  }
}

__device__ __forceinline__ PaletteTables load_palette(const ExpertDesc* d) {
  const uint4 a = *reinterpret_cast<const uint4*>(&d->lo0);
  const uint4 b = *reinterpret_cast<const uint4*>(&d->b7lo0);
  PaletteTables t;
  t.lo0 = a.x;
  t.lo1 = a.y;
  t.hi0 = a.z;
  t.hi1 = a.w;
  t.b7lo0 = b.x;
  t.b7lo1 = b.y;
  t.b7hi0 = b.z;
  t.b7hi1 = b.w;
  t.keep = d->keep;
  return t;
}

// ------------------------------- epilogue ------------------------------------
// FP32 throughout; the only rounding is the store's.  The GELU forms are
// written so that they lose nothing where 1 + erf or 1 + tanh would cancel.
// Divisions are the fast ones: 2 units in the last place for divisors below
// 2^126, 0 beyond.  What FP32 outputs can rely on is stated at uw_activation.

// v / (1 + exp(-t)) for v and t of one sign, from e = exp(-|t|): exp(-t) leaves
// the range where the result is still a normal number (SiLU(-90) = -7.4e-38).
// The divisor is at most 2.
__device__ __forceinline__ float times_sigmoid(float v, float t, float e) {
  return __fdividef(t > 0.0f ? v : v * e, 1.0f + e);
}

// SiLU(v) for a product that is rounded to BF16 next: the fast exponential
// (relative error at most 2^-23 (2 + 1.2 |v|), far below BF16's 2^-8).
__device__ __forceinline__ float silu_fast(float v) { return times_sigmoid(v, v, __expf(-fabsf(v))); }

// Phi(-a) = erfc(a / sqrt 2) / 2 for a >= 0, as exp(-a^2 / 2) t P(t) with
// z = a / sqrt 2, t = 1 / (1 + z / 2).  P: a minimax fit of erfcx(z) / t on z
// in [0, 10], relative error 4.3e-8.  Evaluated in FP32 it is within 44 2^-24,
// the fast exponential within 2^-23 (2 + 0.6 a^2) and the rounding of its
// argument within 2^-24 a^2 / 2, all relative: a Phi(-a) is within 1e-7
// everywhere.  erfcf took twice as long: 664 rows of 7292 x 576 with GELU
// 41.9 us by it, 33.9 by this.
__device__ __forceinline__ float normal_tail(float a) {
  const float t = __fdividef(1.0f, 1.0f + 0.35355339f * a);
  float q = -0.05906814024f;
  q = fmaf(q, t, 0.28457132234f);
  q = fmaf(q, t, -0.48719307450f);
  q = fmaf(q, t, 0.27806013281f);
  q = fmaf(q, t, -0.02662133204f);
  q = fmaf(q, t, 0.20268523569f);
  q = fmaf(q, t, 0.24310412906f);
  q = fmaf(q, t, 0.28237526394f);
  q = fmaf(q, t, 0.28208642012f);
  return 0.5f * __expf(-0.5f * a * a) * t * q;
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case UW_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];  // NaN stays
      break;
    case UW_ACT_GELU:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float tail = normal_tail(fabsf(v[j]));
        v[j] *= v[j] > 0.0f ? 1.0f - tail : tail;
      }
      break;
    case UW_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float t = 1.5957691216057308f * (v[j] + 0.044715f * v[j] * v[j] * v[j]);  // 2 sqrt(2 / pi) (...)
        v[j] = times_sigmoid(v[j], t, expf(-fabsf(t)));
      }
      break;
    case UW_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = times_sigmoid(v[j], v[j], expf(-fabsf(v[j])));
      break;
    default: break;
  }
}

template <int NMAT, bool PAIR>
__device__ __forceinline__ void load_bias(const GParams& p, int e, int mt, int r, float (&bias)[NMAT]) {
#pragma unroll
  for (int m = 0; m < NMAT; ++m) {
    // (unclamped: the second half of an odd last pair is past p.N)
    const int n = (PAIR ? 2 * mt + m : mt) * 128 + r;
    bias[m] = p.bias && n < p.N
                  ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.bias)[static_cast<int64_t>(e) * p.N + n])
                  : 0.0f;
  }
}

// Where rows of y start on 16 bytes (p.vec) a warp turns its 32 rows x 8 slots
// around in shared memory and lane l stores 8 consecutive values of slot
// l / 4, rows 8 (l % 4) ..: the index of the first one, or -1.
__device__ __forceinline__ int64_t turned_index(const GParams& p, int cc, int n, int slot0, int nvalid) {
  const int lane = threadIdx.x & 31;
  const int n0 = n - lane + (lane & 3) * 8;
  return (lane >> 2) < nvalid - cc * 8 && n0 < p.N ? static_cast<int64_t>(slot0 + cc * 8 + (lane >> 2)) * p.N + n0 : -1;
}
// The residual of those 8 values, asked for ahead of the sums it is added to.
__device__ __forceinline__ uint4 turned_residual(const GParams& p, int64_t i) {
  return i >= 0 ? *reinterpret_cast<const uint4*>(p.residual + i) : make_uint4(0, 0, 0, 0);
}

// Values of matrix row n for slots slot0 + 8 cc ..: residual, store.  `turn`:
// 1 KB of the warp's own.
__device__ __forceinline__ void store8(const GParams& p, float (&v)[8], int cc, int n, int slot0, int nvalid,
                                       const uint4& residual, float* turn) {
  const int lane = threadIdx.x & 31;
  if (p.vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn[j * 32 + lane] = v[j];
    __syncwarp();
    const float4 q0 = *reinterpret_cast<const float4*>(turn + lane * 8);
    const float4 q1 = *reinterpret_cast<const float4*>(turn + lane * 8 + 4);
    __syncwarp();
    const int64_t i = turned_index(p, cc, n, slot0, nvalid);
    if (i < 0) return;
    float f[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
    if (p.residual) {
      const uint32_t w4[4] = {residual.x, residual.y, residual.z, residual.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] += __uint_as_float(w4[j] << 16);
        f[2 * j + 1] += __uint_as_float(w4[j] & 0xFFFF0000u);
      }
    }
    if (p.out_fp32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.y) + i);
      dst[0] = make_float4(f[0], f[1], f[2], f[3]);
      dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }
  // a lane's own row: 32 consecutive values of a slot per warp
  const int cols = n < p.N ? nvalid - cc * 8 : 0;
  const int64_t i = static_cast<int64_t>(slot0 + cc * 8) * p.N + n;
  if (p.residual) {
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.residual) + i;
    __nv_bfloat16 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = j < cols ? src[static_cast<int64_t>(j) * p.N] : __nv_bfloat16();
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += __bfloat162float(r[j]);
  }
  if (p.out_fp32) {
    float* dst = static_cast<float*>(p.y) + i;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cols) dst[static_cast<int64_t>(j) * p.N] = v[j];
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.y) + i;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cols) dst[static_cast<int64_t>(j) * p.N] = __float2bfloat16_rn(v[j]);
  }
}

// The residuals of eight columns of a tile.
template <int NMAT, bool PAIR>
__device__ __forceinline__ void load_residual(const GParams& p, int cc, int mt, int slot0, int nvalid, int r,
                                              uint4 (&res)[NMAT]) {
#pragma unroll
  for (int m = 0; m < NMAT; ++m) {
    res[m] = make_uint4(0, 0, 0, 0);
    if ((NMAT == 1 || PAIR) && p.vec && p.residual)
      res[m] = turned_residual(p, turned_index(p, cc, (PAIR ? 2 * mt + m : mt) * 128 + r, slot0, nvalid));
  }
}

// Eight columns of a tile: the sums of its matrices (row r of the tile) to y.
template <int NMAT, bool PAIR>
__device__ __forceinline__ void emit(const GParams& p, float (&a)[NMAT][8], int cc, int mt, int slot0, int nvalid,
                                     int r, const float (&bias)[NMAT], const uint4 (&res)[NMAT], float* turn) {
  if constexpr (NMAT == 2 && !PAIR) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[0][j] = silu_fast(a[0][j]) * a[1][j];
    store8(p, a[0], cc, mt * 128 + r, slot0, nvalid, res[0], turn);
  } else {
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      if (p.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[m][j] += bias[m];
      }
      activate(a[m], p.act);
      store8(p, a[m], cc, (PAIR ? 2 * mt + m : mt) * 128 + r, slot0, nvalid, res[m], turn);
    }
  }
}

// Warp-wide load of 8 consecutive 32-bit columns of the thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}

// Whether the segment is part of a tile that other CTAs work on too.
__device__ __forceinline__ bool is_part(const Seg& s, const GParams& p) { return s.kb1 - s.kb0 != p.KB; }

// A segment's sums out of tensor memory: to y, or, when it is a part of a
// tile, to the CTA's partial slot.  Warps 4 k .. 4 k + 3 take every n_groups-th
// 8 columns from `group` on; row r of the tile is the thread's.
template <int NMAT, bool PAIR>
__device__ __forceinline__ void drain(const GParams& p, const Share& share, const Seg& s, int cta, uint32_t taddr,
                                      int first_tile, int r, int group, int n_groups, float* turn) {
  const int n_kb = s.kb1 - s.kb0;
  const int n_chunks = (s.nvalid + 7) >> 3;
  auto sums = [&](int cc, float (&a)[NMAT][8]) {
    // With one matrix and two issuers: the issuers' sums in the order of their
    // first k-block (a segment of one k-block has only one)
    uint32_t v[2][8];
    const uint32_t at = taddr + static_cast<uint32_t>(cc * 8);
    if constexpr (NMAT == 2) {
      tmem_ld8(at, v[0]);
      tmem_ld8(at + p.cap, v[1]);
    } else {
      const uint32_t i0 = static_cast<uint32_t>(first_tile % p.n_iss);
      tmem_ld8(at + i0 * p.cap, v[0]);
      if (p.n_iss == 2 && n_kb > 1) tmem_ld8(at + (i0 ^ 1u) * p.cap, v[1]);
    }
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[0][j] = __uint_as_float(v[0][j]);
      if constexpr (NMAT == 2) a[NMAT - 1][j] = __uint_as_float(v[1][j]);
      else if (p.n_iss == 2 && n_kb > 1) a[0][j] += __uint_as_float(v[1][j]);
    }
  };
  if (n_kb == p.KB) {
    float bias[NMAT];
    load_bias<NMAT, PAIR>(p, s.e, s.mt, r, bias);
#pragma unroll 1
    for (int cc = group; cc < n_chunks; cc += n_groups) {
      float a[NMAT][8];
      uint4 res[NMAT];
      load_residual<NMAT, PAIR>(p, cc, s.mt, s.slot0, s.nvalid, r, res);
      sums(cc, a);
      emit<NMAT, PAIR>(p, a, cc, s.mt, s.slot0, s.nvalid, r, bias, res, turn);
    }
    return;
  }
  // the CTA's slot 0 holds the tile that opens its run, slot 1 a later one;
  // [matrix][chunk of 8 columns][half][weight row][4 columns]
  float4* mine = reinterpret_cast<float4*>(
      p.partials + (2 * static_cast<int64_t>(cta) + (share.u0 >= s.tile_u ? 0 : 1)) * p.partial_stride);
#pragma unroll 1
  for (int cc = group; cc < n_chunks; cc += n_groups) {
    float a[NMAT][8];
    sums(cc, a);
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      float4* dst = mine + (m * n_chunks + cc) * 256 + r;
      __stcg(dst, make_float4(a[m][0], a[m][1], a[m][2], a[m][3]));
      __stcg(dst + 128, make_float4(a[m][4], a[m][5], a[m][6], a[m][7]));
    }
  }
}

// One thread, after every store of the part has met it at a barrier: takes the
// tile's ticket, and notes the tile when this was the last part.
__device__ __forceinline__ void deliver(const GParams& p, const Share& share, const Seg& s, GBars* bars) {
  const int c_first = unit_owner(s.tile_u, share);
  const int c_last = unit_owner(s.tile_u + p.KB - 1, share);
  // a CTA opens at most one tile that others finish: its counter
  if (ticket(p.counters + c_first) != static_cast<uint32_t>(c_last - c_first)) return;
  p.counters[c_first] = 0;  // all have arrived: ready for the next launch
  Todo& t = bars->todo[bars->n_todo++];
  t.e = s.e;
  t.mt = s.mt;
  t.slot0 = s.slot0;
  t.nvalid = s.nvalid;
  t.c_first = c_first;
  t.c_last = c_last;
  t.first_slot = units_before(c_first, share) >= s.tile_u ? 0 : 1;
}

// ------------------------------- the kernel ----------------------------------
template <int NMAT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x64,
                   const __grid_constant__ GParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t smem_s = smem_u32(smem);
  GBars* bars = reinterpret_cast<GBars*>(smem + p.bar_off);
  SchedEntry* sched = reinterpret_cast<SchedEntry*>(smem + p.sched_off);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  // ---- set-up: barriers, tensor memory and the table of tiles
  const int cta = static_cast<int>(blockIdx.x);
  auto desc = [&](int m, int e) -> const ExpertDesc* { return p.table[m] ? p.table[m] + e : &p.one; };
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  } else if (warp == kWarpX && lane == 0) {
    prefetch_tensormap(&tm_x);
    if (!p.gather) prefetch_tensormap(&tm_x64);
  } else if (warp == kWarpW) {
    if (lane < p.sw) {
      mbar_init(&bars->wfull[lane], 1);
      mbar_init(&bars->wempty[lane], 4);
    }
    if (lane < p.sx) {
      mbar_init(&bars->xfull[lane], 1);
      mbar_init(&bars->xempty[lane], NMAT);
    }
    if (lane < p.sa) {
      mbar_init(&bars->afull[lane], 4);
      mbar_init(&bars->aempty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&bars->acc_full[lane], p.n_iss);
      mbar_init(&bars->acc_empty[lane], 4);
    }
    if (lane < kMaxIssuers) mbar_init(&bars->drain[lane], 1);
    if (lane == 0) {
      bars->abort = 0;
      bars->n_todo = 0;
      bars->together = 0;
    }
    mbar_fence_init();
    __syncwarp();
    if (!p.early) griddep_wait();
    int base = 0;
    bool bad = false, wide = false;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int a = 0, b = 0;
      if (e < p.E) {
        // through L2: with `early` no wait stands between the kernel that
        // wrote them and these reads, so L1 may hold the previous routing's
        a = p.offsets ? __ldcg(p.offsets + e) : 0;
        b = p.offsets ? __ldcg(p.offsets + e + 1) : p.n_rows;
      }
      // offsets that leave [0, n_rows] or fall: nothing is computed
      bad |= a < 0 || b < a || b > p.n_rows;
      const int cnt = bad ? 0 : b - a;
      const int n_nt = cnt <= p.cap ? min(cnt, 1) : quick_div(cnt + p.cap - 1, p.cap);
      const int each = n_nt > 1 ? quick_div(cnt + n_nt - 1, n_nt) : cnt;
      const int ntile = max(16, (each + 15) & ~15);
      const int tiles = n_nt * p.n_mt;
      wide |= n_nt > 1;
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      if (e < p.E) {
        SchedEntry en;
        en.tile0 = base + incl - tiles;
        en.start = a;
        en.count = cnt;
        en.n_nt = (n_nt << 16) | ntile;
        sched[e] = en;
      }
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
      if (lane == 0) record_status(p.status, UW_ERR_INVALID_ARG);
      base = 0;
    }
    if (lane == 0) sched[p.E].tile0 = base;
    __syncwarp();
    // this CTA's share and its first segment, found once for every role
    const Share h = share_of(cta, base, __any_sync(0xFFFFFFFFu, wide), p);
    Seg s;
    if (h.waves > 0 || h.u0 < h.u1) {
      seg_init(s, sched, p, h, cta);
      // its matrices' records for every role, and the tile records of the
      // first batch
      constexpr int kDescs = NMAT == 2 && !PAIR ? 2 : 1;
      constexpr int kWords = sizeof(ExpertDesc) / 16;
      if (lane < kDescs * kWords)
        reinterpret_cast<uint4*>(bars->desc)[lane] =
            reinterpret_cast<const uint4*>(desc(lane / kWords, s.e))[lane % kWords];
      __syncwarp();
      if (lane < min(kWBatch, (s.kb1 - s.kb0) * NMAT)) {
        const int m = NMAT == 2 ? lane & 1 : 0;
        const uint8_t* src = bars->desc[PAIR ? 0 : m].pack +
                             (static_cast<uint64_t>(row_tile<PAIR>(p, s.mt, m)) * p.KB + s.kb0 + lane / NMAT) * kBody;
        mbar_expect_tx(&bars->wfull[lane], kBody);
        bulk_load(smem + p.w_base + static_cast<uint32_t>(lane) * p.w_slot_bytes, src, kBody, &bars->wfull[lane]);
      }
    }
    if (lane == 0) {
      bars->share = h;
      bars->first = s;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const Share& share = bars->share;
  const bool work = share.waves > 0 || share.u0 < share.u1;
  const int first_e = bars->first.e;
  auto matrix = [&](int m, int e) -> const ExpertDesc* { return e == first_e ? &bars->desc[m] : desc(m, e); };

  if (warp == kWarpW) {
    // --------------------------- weight producer ----------------------------
    // One lane per tile, kWBatch tiles at a time: each waits for its slot,
    // then issues its record and its verbatim rows (one contiguous run).  One
    // thread alone took about 650 cycles per tile, more than HBM needs for
    // one (530).  The lanes hold the verbatim offsets of the next 31 k-blocks.
    constexpr int kSpan = 28;  // k-blocks per set of offsets: whole batches, and one offset more
    if (work) {
      const uint64_t once = l2_evict_first();
      Seg s = bars->first;
      Ring rw{0, 0};
      int issued = 0;
      bool ok = true;
      const int m = NMAT == 2 ? lane & 1 : 0;  // this lane's matrix
      do {
        // lane l: offset of tile kb + l
        const ExpertDesc* d0 = matrix(0, s.e);
        const ExpertDesc* d1 = NMAT == 2 && !PAIR ? matrix(1, s.e) : d0;
        const int64_t t0 = static_cast<int64_t>(row_tile<PAIR>(p, s.mt, 0)) * p.KB;
        const int64_t t1 = static_cast<int64_t>(row_tile<PAIR>(p, s.mt, 1)) * p.KB;
        const uint32_t* off0 = d0->pack_off + t0 + lane;
        const uint32_t* off1 = d1->pack_off + t1 + lane;
        const int last = s.kb1 - lane;
        uint32_t v0 = s.kb0 <= last ? __ldg(off0 + s.kb0) : 0u;
        uint32_t v1 = NMAT == 2 && s.kb0 <= last ? __ldg(off1 + s.kb0) : 0u;
        const ExpertDesc* d = m ? d1 : d0;
        const uint8_t* pack = d->pack + static_cast<uint64_t>(m ? t1 : t0) * kBody;
        const uint8_t* tails = d->tails;
        const uint32_t n_verb = d->n_verbatim;
        // weights that a later column tile reads again stay in L2
        const bool reread = (sched[s.e].n_nt >> 16) > 1;
        for (int kb = s.kb0; kb < s.kb1 && ok; kb += kSpan) {
          const uint32_t w0 = kb + kSpan <= last ? __ldg(off0 + kb + kSpan) : 0u;
          const uint32_t w1 = NMAT == 2 && kb + kSpan <= last ? __ldg(off1 + kb + kSpan) : 0u;
          const int n = min(kSpan, s.kb1 - kb) * NMAT;
          for (int i0 = 0; i0 < n; i0 += kWBatch) {
            const int j = (i0 + lane) / NMAT;  // k-block of this lane's tile
            const int count = min(kWBatch, n - i0);
            Ring mine = rw;
            ring_next(mine, p.sw, lane & (kWBatch - 1));
            bool good = true;
            if (lane < count && mine.use > 0)
              good = mbar_wait(&bars->wempty[mine.slot], (mine.use - 1) & 1, &bars->abort, p.status);
            ok = __all_sync(0xFFFFFFFFu, good);
            if (!ok) break;
            if (lane < count && issued > 0) {  // (the first batch's are on their way)
              // the record first: it does not wait for the offsets to arrive
              uint8_t* slot = smem + p.w_base + static_cast<uint32_t>(mine.slot) * p.w_slot_bytes;
              uint64_t* bar = &bars->wfull[mine.slot];
              const uint8_t* src = pack + static_cast<uint64_t>(kb + j) * kBody;
              mbar_expect_tx(bar, kBody);
              if (reread) bulk_load(slot, src, kBody, bar);
              else bulk_load_hint(slot, src, kBody, bar, once);
            }
            uint32_t a = __shfl_sync(0xFFFFFFFFu, v0, j & 31), b = __shfl_sync(0xFFFFFFFFu, v0, (j + 1) & 31);
            if constexpr (NMAT == 2) {
              const uint32_t a1 = __shfl_sync(0xFFFFFFFFu, v1, j & 31), b1 = __shfl_sync(0xFFFFFFFFu, v1, (j + 1) & 31);
              if (m) {
                a = a1;
                b = b1;
              }
            }
            if (lane < count) {
              uint32_t rows = 0;
              if (b < a || b - a > 128u || b > n_verb) record_status(p.status, UW_ERR_CORRUPT);
              else rows = min(b - a, static_cast<uint32_t>(p.vcap));
              bars->tail_first[mine.slot] = a;
              mbar_arrive_expect_tx(&bars->wfull[mine.slot], rows * 128u);
              if (rows)
                bulk_load(smem + p.w_base + static_cast<uint32_t>(mine.slot) * p.w_slot_bytes + kBody,
                          tails + static_cast<uint64_t>(a) * 128u, rows * 128u, &bars->wfull[mine.slot]);
            }
            __syncwarp();
            issued += count;
            ring_next(rw, p.sw, count);
          }
          v0 = w0;
          v1 = w1;
        }
      } while (ok && seg_next(s, sched, p, share, cta));
      // every issued copy lands before the CTA exits (already so unless a
      // wait gave up)
      if (lane == 0)
        for (int q = max(0, issued - p.sw); q < issued; ++q)
          mbar_wait(&bars->wfull[q % p.sw], static_cast<uint32_t>(q / p.sw) & 1, nullptr, p.status);
    }
    __syncwarp();
  } else if (warp == kWarpX) {
    // ------------------------- activation producer --------------------------
    if (work) {
      griddep_wait();
      Seg s = bars->first;
      Ring rx{0, 0};
      int issued = 0;
      bool ok = true;
      do {
        // lane l gathers rows 4 l .. 4 l + 3 of the tile, past the tile's
        // last row the last one again (never stored)
        int r[4] = {};
        // rows in boxes of 64, the rest in boxes of 16: lane l issues one
        const int big = s.ntile >> 6;
        const int lanes = p.gather ? s.ntile >> 2 : big + ((s.ntile & 63) >> 4);
        const int row = lane < big ? 64 * lane : 64 * big + 16 * (lane - big);
        if (p.gather) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            r[q] = __ldcg(p.rows + s.slot0 + min(4 * lane + q, s.nvalid - 1));
            if (r[q] < 0 || r[q] >= p.x_rows) {
              record_status(p.status, UW_ERR_INVALID_ARG);
              r[q] = 0;
            }
          }
        }
        for (int kb = s.kb0; kb < s.kb1; ++kb) {
          if (rx.use > 0) ok = warp_wait(&bars->xempty[rx.slot], (rx.use - 1) & 1, bars, p.status);
          if (!ok) break;
          uint64_t* bar = &bars->xfull[rx.slot];
          if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(s.ntile) * 128u);
          __syncwarp();
          uint8_t* dst = smem + static_cast<uint32_t>(rx.slot) * p.x_slot_bytes;
          if (lane < lanes) {
            if (p.gather) tma_gather4(dst + lane * 512, &tm_x, kb * 64, r[0], r[1], r[2], r[3], bar);
            else if (lane < big) tma_load_2d(dst + row * 128, &tm_x64, kb * 64, s.slot0 + row, bar);
            else tma_load_2d(dst + row * 128, &tm_x, kb * 64, s.slot0 + row, bar);
          }
          ++issued;
          ring_next(rx, p.sx);
        }
      } while (ok && seg_next(s, sched, p, share, cta));
      if (lane == 0)
        for (int q = max(0, issued - p.sx); q < issued; ++q)
          mbar_wait(&bars->xfull[q % p.sx], static_cast<uint32_t>(q / p.sx) & 1, nullptr, p.status);
    }
    __syncwarp();
  } else if (warp < kWarpRebuild) {
    // ----------------------------- MMA issuers ------------------------------
    // Tile i of the CTA's sequence belongs to issuer i % n_iss, which sums
    // into an accumulator of its own (one thread issues an MMA only every
    // ~120 cycles, several overlap).  Ring sizes are multiples of what keeps
    // a slot with one issuer, so each sees every phase of its slots.
    const int iss = warp - kWarpMma;
    // The whole warp runs the loop and one elected lane issues: with uniform
    // control flow the operands stay in uniform registers.
    if (iss < p.n_iss && work) {
      Seg s = bars->first;
      // with two matrices issuer m has matrix m's tile of every k-block; with
      // one, the issuers take turns
      const int per = p.n_iss / NMAT, kstep = NMAT * per;
      const int m = NMAT == 2 ? iss : 0;
      Ring rx{0, 0}, ra{m, 0};
      int skip = NMAT == 2 ? 0 : iss;  // k-blocks before this issuer's next
      if (NMAT == 1) {
        rx.slot = skip;
        ra.slot = skip;
      }
      uint32_t ab = 0, seg = 0;
      bool ok = true;
      const uint64_t x_desc0 = smem_desc_sw128(smem_s);
      const uint32_t x_step = p.x_slot_bytes >> 4;
      do {
        if (seg >= static_cast<uint32_t>(p.n_acc)) {
          ok = warp_wait(&bars->acc_empty[ab], (seg / p.n_acc - 1) & 1, bars, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t idesc = idesc_bf16_f32(s.ntile);
        const uint32_t d = tmem + (ab * p.n_iss + iss) * static_cast<uint32_t>(p.cap);
        uint32_t acc = 0;
        const int n_kb = s.kb1 - s.kb0;
        int kb = skip;
        for (; kb < n_kb; kb += per) {
          ok = warp_wait(&bars->xfull[rx.slot], rx.use & 1, bars, p.status) &&
               warp_wait(&bars->afull[ra.slot], ra.use & 1, bars, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem + p.a_col0 + static_cast<uint32_t>(ra.slot) * 32;
          const uint64_t b = x_desc0 + static_cast<uint64_t>(static_cast<uint32_t>(rx.slot) * x_step);
          if (elect_one()) {
            mma_ts(d, a, b, idesc, acc);
            mma_ts(d, a + 8, b + 2, idesc, 1u);
            mma_ts(d, a + 16, b + 4, idesc, 1u);
            mma_ts(d, a + 24, b + 6, idesc, 1u);
            tc_commit(&bars->aempty[ra.slot]);
            tc_commit(&bars->xempty[rx.slot]);
          }
          __syncwarp();
          acc = 1;
          ring_next(rx, p.sx, per);
          ring_next(ra, p.sa, kstep);
        }
        if (!ok) break;
        skip = kb - n_kb;
        if (elect_one()) tc_commit(&bars->acc_full[ab]);
        __syncwarp();
        ++seg;
        if (++ab == static_cast<uint32_t>(p.n_acc)) ab = 0;
      } while (seg_next(s, sched, p, share, cta));
      // every MMA issued so far finishes before tensor memory is freed
      if (elect_one()) tc_commit(&bars->drain[iss]);
      __syncwarp();
      mbar_wait(&bars->drain[iss], 0, nullptr, p.status);
    }
    __syncwarp();
  } else if (warp < kWarpEpi) {
    // ------------------------------- rebuild --------------------------------
    // a warp reaches the TMEM lanes 32 (warp % 4) .., so those are its rows
    const int w = warp & 3;
    const int r = w * 32 + lane;
    const int grp = (warp - kWarpRebuild) >> 2;
    if (work) {
      Seg s = bars->first;
      // the groups take turns; with two matrices a group's tiles are all of
      // one (kGroups is even)
      constexpr int kStep = kGroups / NMAT;  // k-blocks from one tile of a group to the next
      Ring rw{grp, 0}, ra{grp, 0};
      int skip = grp / NMAT;
      bool ok = true;
      PaletteTables pal{};
      bool uniform = true;
      int cur_e = -1;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16) + p.a_col0;
      do {
        if (cur_e != s.e) {
          const ExpertDesc* d = matrix(NMAT == 2 && !PAIR ? grp & 1 : 0, s.e);
          pal = load_palette(d);
          uniform = d->mixed == 0;
          cur_e = s.e;
        }
        const int n_kb = s.kb1 - s.kb0;
        int kb = skip;
#pragma unroll 1
        for (; kb < n_kb; kb += kStep) {
          ok = warp_wait(&bars->wfull[rw.slot], rw.use & 1, bars, p.status);
          if (!ok) break;
          const uint32_t body = smem_s + p.w_base + static_cast<uint32_t>(rw.slot) * p.w_slot_bytes;
          // verbatim rows: one mask bit per row, no per-element test
          const uint32_t mw = lds32(body + kBodyMask + 4 * w);
          uint32_t o[32];
          if (uniform) rebuild_row(pal, true, body, r, o);
          else rebuild_row(pal, false, body, r, o);
          if ((mw >> lane) & 1) {
            const uint4 mk = lds128(body + kBodyMask);
            const int idx = (w > 0 ? __popc(mk.x) : 0) + (w > 1 ? __popc(mk.y) : 0) + (w > 2 ? __popc(mk.z) : 0) +
                            __popc(mw & ((1u << lane) - 1));
            if (idx < p.vcap) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 v = lds128(body + kBody + idx * 128 + 16 * c);
                o[4 * c] = v.x;
                o[4 * c + 1] = v.y;
                o[4 * c + 2] = v.z;
                o[4 * c + 3] = v.w;
              }
            } else {
              // more verbatim rows than staged ones: from HBM
              const ExpertDesc* d = matrix(NMAT == 2 && !PAIR ? grp & 1 : 0, s.e);
              const uint64_t g = static_cast<uint64_t>(bars->tail_first[rw.slot]) + idx;
              if (g < d->n_verbatim) {
                const uint4* src = reinterpret_cast<const uint4*>(d->tails + g * 128u);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const uint4 v = __ldg(src + c);
                  o[4 * c] = v.x;
                  o[4 * c + 1] = v.y;
                  o[4 * c + 2] = v.z;
                  o[4 * c + 3] = v.w;
                }
              } else {
                record_status(p.status, UW_ERR_CORRUPT);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->wempty[rw.slot]);
          // the A slot is free once the MMAs of its previous use are done
          if (ra.use > 0) {
            ok = warp_wait(&bars->aempty[ra.slot], (ra.use - 1) & 1, bars, p.status);
            if (!ok) break;
          }
          tc_fence_after();
          tmem_st32(lanes + static_cast<uint32_t>(ra.slot) * 32, o);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->afull[ra.slot]);
          ring_next(rw, p.sw, kGroups);
          ring_next(ra, p.sa, kGroups);
        }
        skip = kb - n_kb;
      } while (ok && seg_next(s, sched, p, share, cta));
    }
  } else {
    // ------------------------------- epilogue -------------------------------
    // outputs and the workspace may be in use by the previous kernel on the
    // stream until it has completed
    griddep_wait();
    if (warp == kWarpEpi && lane == 0) griddep_launch_dependents();
    if (work) {
      const int w = warp & 3;  // TMEM lanes 32 w ..
      const int r = w * 32 + lane;
      Seg s = bars->first;
      uint32_t seg = 0;
      int first_tile = 0;  // the segment's first tile in the CTA's sequence
      float* turn = reinterpret_cast<float*>(smem + p.turn_off) + w * 256;
      do {
        const uint32_t ab = seg % p.n_acc;
        if (seg_last(s, share) && !is_part(s, p) && (s.nvalid * NMAT > kTogether)) {
          // left to all warps
          if (warp == kWarpEpi && lane == 0) {
            bars->last = s;
            bars->last_acc = ab;
            bars->last_tile = first_tile;
            bars->together = 1;
          }
          break;
        }
        bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars->acc_full[ab], (seg / p.n_acc) & 1, &bars->abort, p.status));
        if (!group_and(ok)) break;
        tc_fence_after();
        drain<NMAT, PAIR>(p, share, s, cta,
                          tmem + (static_cast<uint32_t>(w * 32) << 16) + ab * p.n_iss * static_cast<uint32_t>(p.cap),
                          first_tile, r, 0, 1, turn);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->acc_empty[ab]);
        if (is_part(s, p)) {
          group_sync();
          if (warp == kWarpEpi && lane == 0) deliver(p, share, s, bars);
        }
        ++seg;
        first_tile += (s.kb1 - s.kb0) * NMAT;
      } while (seg_next(s, sched, p, share, cta));
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every role is done and every MMA has completed.  The rings are idle: their
  // memory is where the warps turn values around from here on.
  float* turn = reinterpret_cast<float*>(smem) + warp * 256;
  const int r = (warp & 3) * 32 + lane;
  if (bars->together) {
    // ---- the last tile, whole and wide: all warps empty its accumulators (6
    // groups of 4 warps, 8 columns each) instead of the epilogue's 4 with the
    // others idle
    tc_fence_after();
    if (!*static_cast<volatile uint32_t*>(&bars->abort))
      drain<NMAT, PAIR>(p, share, bars->last, cta,
                        tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                            bars->last_acc * p.n_iss * static_cast<uint32_t>(p.cap),
                        static_cast<int>(bars->last_tile), r, warp >> 2, kThreads / 128, turn);
    tc_fence_before();
    __syncthreads();
  }
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // ---- tiles shared by several CTAs that this one completes (at most its
  // first and its last): the contributors' parts, added in CTA order.
  for (int i = 0; i < static_cast<int>(bars->n_todo); ++i) {
    const Todo t = bars->todo[i];
    const int n_chunks = (t.nvalid + 7) >> 3;
    float bias[NMAT];
    load_bias<NMAT, PAIR>(p, t.e, t.mt, r, bias);
#pragma unroll 1
    for (int cc = warp >> 2; cc < n_chunks; cc += kThreads / 128) {
      float a[NMAT][8];
      uint4 res[NMAT];
      load_residual<NMAT, PAIR>(p, cc, t.mt, t.slot0, t.nvalid, r, res);
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        // contributors in CTA order, the loads of two in flight
        const int64_t at = static_cast<int64_t>(m * n_chunks + cc) * 256 + r;
        auto part = [&](int c) -> const float4* {
          const int64_t slot = 2 * static_cast<int64_t>(c) + (c == t.c_first ? t.first_slot : 0);
          return reinterpret_cast<const float4*>(p.partials + slot * p.partial_stride) + at;
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) a[m][j] = 0.0f;
        auto add = [&](const float4& lo, const float4& hi) {
          a[m][0] += lo.x;
          a[m][1] += lo.y;
          a[m][2] += lo.z;
          a[m][3] += lo.w;
          a[m][4] += hi.x;
          a[m][5] += hi.y;
          a[m][6] += hi.z;
          a[m][7] += hi.w;
        };
#pragma unroll 1
        for (int c = t.c_first; c <= t.c_last; c += 2) {
          const float4* p0 = part(c);
          const float4* p1 = part(min(c + 1, t.c_last));
          const float4 a0 = __ldcg(p0), a1 = __ldcg(p0 + 128), b0 = __ldcg(p1), b1 = __ldcg(p1 + 128);
          add(a0, a1);
          if (c < t.c_last) add(b0, b1);
        }
      }
      emit<NMAT, PAIR>(p, a, cc, t.mt, t.slot0, t.nvalid, r, bias, res, turn);
    }
  }
}

// ------------------------- rows next to each other ---------------------------
// out[s] = x[rows[s]] for the slots of all groups: 16-byte pieces.
struct PermuteParams {
  const uint4* x;
  const int32_t* rows;
  const int32_t* offsets;
  uint4* out;
  int E, x_rows, n_rows, pieces;  // pieces of 16 bytes per row
  uint32_t* status;
};
__global__ void __launch_bounds__(256) permute_kernel(const PermuteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int first = max(0, p.offsets[0]), last = min(p.n_rows, p.offsets[p.E]);
  for (int s = first + static_cast<int>(blockIdx.x); s < last; s += static_cast<int>(gridDim.x)) {
    int r = p.rows[s];
    if (r < 0 || r >= p.x_rows) {
      if (threadIdx.x == 0) record_status(p.status, UW_ERR_INVALID_ARG);
      r = 0;
    }
    const uint4* src = p.x + static_cast<int64_t>(r) * p.pieces;
    uint4* dst = p.out + static_cast<int64_t>(s) * p.pieces;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.pieces; i += 256) dst[i] = __ldcg(src + i);
  }
}

// ------------------------------- host side -----------------------------------

// Rows per tile up to which scattered rows are gathered by TMA.  Measured with
// SwiGLU products: 16 rows 62.4 us gathered, 63.6 laid next to each other
// first; 32 rows 235.6 / 217.4.
constexpr int kGatherCap = 16;
// Two row tiles share the activation tile above this many columns per tile
// and from this many units per CTA on (grouped_plan).
constexpr int kPairCap = 64, kPairUnits = 128;

struct GLayout {
  int cap = 16, n_iss = 1, n_acc = 1, sx = 2, sa = 2, sw = 2, vcap = 0;
  uint32_t x_slot_bytes = 0, w_base = 0, w_slot_bytes = 0, sched_off = 0, turn_off = 0, bar_off = 0, a_col0 = 0;
  size_t smem = 0;
};

// The widest tile: what tensor memory and shared memory hold, and no more than
// the rows there are.
int most_columns(int n_rows, int nmat) { return std::min(nmat == 2 ? 192 : 256, (n_rows + 15) / 16 * 16); }

// Whether the schedule's indices hold every split of n_rows into E groups at
// this width: column tiles of a group in 15 bits, k-blocks of all tiles in 31.
bool schedule_fits(int n_rows, int E, int cap, int n_mt, int KB) {
  const int64_t tiles = std::min<int64_t>(n_rows, n_rows / cap + E);
  return n_rows / cap + 1 <= 0x7FFF && tiles * n_mt * KB <= 0x7FFFFFFF;
}

// Columns per tile, at most: the width for which an estimate of the launch is
// smallest, in units of one k-block of a tile (about 500 cycles).  Wide tiles
// rebuild each weight tile less often, narrow ones give more tiles to spread
// over the CTAs and less to carry through the epilogue.  A k-block costs the
// larger of the rebuild (0.7; its 386 cycles of the ALU pipe would be 0.77) and the
// MMAs (2 cycles per column), the weights
// once from HBM 1.06 (per column tile when tiles are shared out and the
// weights outgrow L2: their column tiles then come at different times); a
// tile's epilogue 0.7 per 8 columns and 2, behind the next tile's k-blocks
// where there are two accumulators, a quarter of that for the last one of a
// CTA; sharing a tile out the writing (half of that), a ticket and the adding up
// of the parts, which 6 groups of warps do 8 columns each at a time.  A wider
// tile has to win by 3%: it takes shared memory from the weight ring.
// Measured against the widest tile: 512 rows of 1024 x 1024 8.0 us at 64 columns, 15.2 at 256; 128 rows of
// 1024 x 4096 11.8 at 32, 23.3 at 128; 450 rows of 5896 x 1088 15.6 at 160,
// 17.9 at 240; but 1000 rows of 4096 x 4096 38.5 at 256, 51.5 at 176.
// Groups of several experts vary in size: an average group of `avg` rows is
// taken to need one column tile of 2 avg columns, else avg / width + 3/4, and
// no width below 32 is taken (8 experts of 14336 x 4096, SwiGLU: 8 rows on
// average 231 us at 16, 217 at 32; 64 rows 377 at 96, 267 at 128, 289 at 192).
int pick_cap(int n_rows, int E, int nmat, int n_mt, int KB, int sms) {
  static const int kWidths[] = {16, 32, 48, 64, 96, 128, 160, 192, 224, 256};
  const int most = most_columns(n_rows, nmat);
  const double groups = std::min(n_rows, E), avg = n_rows / groups;
  const double weights = nmat * groups * n_mt * KB;  // tiles of them
  int best = most;
  double least = 0;
  for (const int width : kWidths) {
    int cap = std::min(width, most);
    double cols = cap >= 2 * avg ? 1.0 : avg / cap + 0.75;
    if (E == 1) {
      const int n_nt = (n_rows + cap - 1) / cap;
      cap = ((n_rows + n_nt - 1) / n_nt + 15) / 16 * 16;
      cols = n_nt;
    } else if (cap < std::min(32, most)) {
      continue;
    }
    // (millions of rows need wide tiles; grouped_plan refuses what none holds)
    if (width < most && !schedule_fits(n_rows, E, cap, n_mt, KB)) continue;
    const double tiles = groups * n_mt * cols, chunks = std::max(1.0, avg / cols / 8), waves = std::ceil(tiles / sms);
    const double main = KB * nmat * std::max(0.7, std::min<double>(cap, avg / cols + 15) * 0.004);
    const double epi = 0.7 * chunks * nmat + 2;
    const bool two = 2 * nmat * cap <= 256;
    const double each = two ? std::max(main, epi) : main + epi;
    const double hbm = 1.06 * weights / sms;
    const double last = std::min<double>(cap, avg / cols) * nmat > kTogether ? epi / 4 : epi;
    const double whole = std::max(hbm, (waves - 1) * each + main + last);
    const double again = weights * 12304 > 64e6 ? cols : 1.0;
    const double shared = std::max(hbm * again, tiles / sms * each) + 0.5 * epi + 4 +
                          nmat * std::ceil(chunks / 6) * (1 + 0.35 * std::max(2.0, sms / tiles));
    const double cost = std::min(whole, shared);
    if (least == 0 || cost < 0.97 * least) {
      least = cost;
      best = cap;
    }
    if (width >= most) break;
  }
  return best;
}

bool make_glayout(int cap, int E, int nmat, GLayout* out) {
  GLayout l;
  l.cap = cap;
  // tensor memory: accumulators (n_acc buffers x n_iss issuers x cap
  // columns), then 32 columns per A tile
  l.n_acc = 2 * nmat * l.cap <= 256 ? 2 : 1;
  l.n_iss = nmat;
  while (2 * l.n_iss <= kMaxIssuers && l.n_acc * 2 * l.n_iss * l.cap <= 256) l.n_iss *= 2;
  l.a_col0 = (static_cast<uint32_t>(l.n_acc * l.n_iss * l.cap) + 31u) & ~31u;
  const int per = l.n_iss / nmat;            // issuers per matrix: an x slot stays with one of them
  const int step_a = std::max(l.n_iss, kGroups);
  l.sa = std::min(kMaxSlots, static_cast<int>((kTmemCols - l.a_col0) / 32));
  l.sa -= l.sa % step_a;
  l.x_slot_bytes = static_cast<uint32_t>(l.cap) * 128;
  const uint32_t sched_bytes = (static_cast<uint32_t>(E + 1) * sizeof(SchedEntry) + 127u) & ~127u;
  const uint32_t turn_bytes = 4 * 32 * 8 * 4;  // the epilogue warps' values
  const uint32_t fixed = sched_bytes + turn_bytes + ((sizeof(GBars) + 127u) & ~127u) + 128u + 1024u;
  if (l.sa < step_a || fixed >= kSmemLimit / 2) return false;
  const uint32_t room = static_cast<uint32_t>(kSmemLimit) - fixed;
  // measured: 8 slots at 16 columns (4: +2%), 4 at 192 (3: +2%, 5: +20%, the
  // weight ring falls to 4 slots), 3 at 256 (4: +7%)
  l.sx = l.cap <= 32 ? 8 : (l.cap <= 64 ? 6 : (l.cap <= 192 ? 4 : 3));
  l.sx -= l.sx % per;
  const uint32_t w_room = room - static_cast<uint32_t>(l.sx) * l.x_slot_bytes;
  l.sw = std::min(kMaxSlots, static_cast<int>(w_room / (kBody + kMinTail * 128u)));
  l.sw -= l.sw % kGroups;
  if (l.sw < kWBatch || l.sx < 1) return false;
  l.vcap = static_cast<int>(std::min(128u, (w_room / static_cast<uint32_t>(l.sw) - kBody) / 128u));
  l.w_slot_bytes = kBody + static_cast<uint32_t>(l.vcap) * 128u;  // a multiple of 16
  l.w_base = static_cast<uint32_t>(l.sx) * l.x_slot_bytes;
  l.sched_off = (l.w_base + static_cast<uint32_t>(l.sw) * l.w_slot_bytes + 127u) & ~127u;
  l.turn_off = l.sched_off + sched_bytes;
  l.bar_off = l.turn_off + turn_bytes;
  l.smem = std::max<size_t>(l.bar_off + ((sizeof(GBars) + 127u) & ~127u) + 1024u, kSmemFloor);
  if (l.smem > kSmemLimit) return false;
  *out = l;
  return true;
}

struct GPlan {
  GLayout lay;
  int n_mt = 0, KB = 0, grid = 0;
  bool pair = false;
  size_t partial_stride = 0;  // floats
  size_t permuted = 0;        // offset of the rows laid next to each other, 0: none
  size_t bytes = 0;           // workspace
};

uw_status grouped_plan(int64_t N, int64_t K, int E, int n_rows, bool swiglu, bool scattered, int sms, GPlan* out) {
  if (E < 1 || E > kMaxExperts || n_rows < 0) return UW_ERR_INVALID_ARG;
  if (n_rows > 0x7FFF * 256) return UW_ERR_UNSUPPORTED_SHAPE;  // (below; and the sums here stay in range)
  if (N < 1 || K < 64 || K % 64 != 0 || K > 32768 || N > (int64_t(1) << 31) - 128) return UW_ERR_UNSUPPORTED_SHAPE;
  GPlan g;
  g.n_mt = static_cast<int>((N + 127) / 128);
  g.KB = static_cast<int>(K / 64);
  // Large groups: two row tiles share each activation tile, which halves what
  // the activations cost in L2 and shared-memory traffic, where there are
  // enough units that the coarser tiles do not cost more by being split.
  // Measured, pairs against single tiles: 8 x 512 rows of 4096 x 14336 644 /
  // 778 us, 8 x 64 rows 140 / 180; but 512 rows of one 14336 x 4096 matrix
  // (73 pair units per CTA) 87 / 76.
  const int n = std::max(n_rows, 1);
  int cap = swiglu ? 0 : pick_cap(n, E, 1, g.n_mt, g.KB, sms);
  const int cap2 = pick_cap(n, E, 2, swiglu ? g.n_mt : (g.n_mt + 1) / 2, g.KB, sms);
  const int64_t pair_units =
      static_cast<int64_t>((g.n_mt + 1) / 2) * std::max<int64_t>(E > 1 ? std::min(n_rows, E) : 1, n_rows / cap2) * g.KB;
  g.pair = !swiglu && g.n_mt > 1 && cap > kPairCap && pair_units >= static_cast<int64_t>(kPairUnits) * sms &&
           schedule_fits(n_rows, E, cap2, (g.n_mt + 1) / 2, g.KB);
  const int nmat = swiglu || g.pair ? 2 : 1;
  if (nmat == 2) cap = cap2;
  if (g.pair) g.n_mt = (g.n_mt + 1) / 2;
  if (!make_glayout(cap, E, nmat, &g.lay)) return UW_ERR_UNSUPPORTED_SHAPE;
  // the most units any split of n_rows into E groups can give
  const int64_t tiles = std::min<int64_t>(n_rows, n_rows / g.lay.cap + E);
  const int64_t units = tiles * g.n_mt * g.KB;
  if (!schedule_fits(n_rows, E, g.lay.cap, g.n_mt, g.KB)) return UW_ERR_UNSUPPORTED_SHAPE;
  g.grid = static_cast<int>(std::min<int64_t>(std::max<int64_t>(units, 1), sms));
  g.partial_stride = static_cast<size_t>(nmat) * 128 * g.lay.cap;
  // The workspace does not depend on the width that was picked, so that it
  // never falls with n_rows: one for the largest batch serves every smaller one.
  const int64_t most_units = std::min<int64_t>(n_rows, n_rows / 16 + E) * ((N + 127) / 128) * g.KB;
  const int most1 = most_columns(n, 1), most2 = most_columns(n, 2);
  const size_t columns = swiglu || most1 > kPairCap ? 2 * most2 : most1;
  g.bytes = kWsHeader + kCounterBytes +
            align_up(2 * static_cast<size_t>(std::min<int64_t>(most_units, sms)) * 128 * columns * 4, 256);
  if (scattered && most1 > kGatherCap) {
    if (g.lay.cap > kGatherCap) g.permuted = g.bytes;
    g.bytes += align_up(static_cast<size_t>(n_rows) * K * 2, 256);
  }
  *out = g;
  return UW_OK;
}

template <int NMAT, bool PAIR>
uw_status launch_grouped_kernel(const CUtensorMap& tx, const CUtensorMap& tx64, const GParams& gp, size_t smem,
                                cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev & 63], [&] {
    attr_err[dev & 63] = cudaFuncSetAttribute(grouped_kernel<NMAT, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(kSmemLimit));
  });
  if (attr_err[dev & 63] != cudaSuccess) return UW_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gp.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, grouped_kernel<NMAT, PAIR>, tx, tx64, gp);
  note_launch();
  if (err != cudaSuccess) return cuda_status(err);
  return cuda_status(cudaGetLastError());
}

uw_status launch_permute(const PermuteParams& q, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, permute_kernel, q);
  note_launch();
  if (err != cudaSuccess) return cuda_status(err);
  return cuda_status(cudaGetLastError());
}

int sms_or_default() {
  DeviceInfo dev;
  return device_info(&dev) == UW_OK ? dev.sm_count : 148;
}

}  // namespace

// The device record of one compressed matrix (direct-palette form).
uw_status expert_desc(const uw_matrix* m, ExpertDesc* out) {
  uw_status st = check_matrix(m);
  if (st != UW_OK) return st;
  if (!m->pack || !m->pack_off || !aligned16(m->pack) || !aligned16(m->pack_off)) return UW_ERR_INVALID_ARG;
  const int64_t n_tiles = (m->L.rows + 127) / 128 * (m->L.cols / 64);
  if (m->L.n_verbatim > 0xFFFFFFFFll) return UW_ERR_UNSUPPORTED_SHAPE;
  bool mixed = false;
  const PaletteTables t = palette_tables(m->cb.palette, m->cb.code_len, &mixed);
  ExpertDesc d;
  std::memset(&d, 0, sizeof(d));
  d.pack = m->pack;
  d.tails = m->pack + static_cast<uint64_t>(n_tiles) * kBody;
  d.pack_off = m->pack_off;
  d.n_verbatim = static_cast<uint32_t>(m->L.n_verbatim);
  d.mixed = mixed ? 1 : 0;
  d.lo0 = t.lo0;
  d.lo1 = t.lo1;
  d.hi0 = t.hi0;
  d.hi1 = t.hi1;
  d.b7lo0 = t.b7lo0;
  d.b7lo1 = t.b7lo1;
  d.b7hi0 = t.b7hi0;
  d.b7hi1 = t.b7hi1;
  d.keep = t.keep;
  *out = d;
  return UW_OK;
}

size_t grouped_ws_bytes(int64_t N, int64_t K, int E, int n_rows, bool swiglu, bool scattered) {
  GPlan g;
  return grouped_plan(N, K, E, n_rows, swiglu, scattered, sms_or_default(), &g) == UW_OK ? g.bytes : 0;
}

uw_status launch_grouped(const GroupedArgs& a, cudaStream_t s) {
  DeviceInfo dev;
  uw_status st = device_info(&dev);
  if (st != UW_OK) return st;
  GPlan g;
  if ((st = grouped_plan(a.N, a.K, a.E, a.n_rows, a.swiglu, a.rows != nullptr, dev.sm_count, &g)) != UW_OK) return st;
  if (!a.x || !a.y || !a.ws || !aligned16(a.x) || !aligned16(a.y) || !aligned16(a.ws) || a.x_rows < 1)
    return UW_ERR_INVALID_ARG;
  if (!aligned_to(a.offsets, 4) || !aligned_to(a.rows, 4) || !aligned_to(a.bias, 2) || !aligned_to(a.residual, 2))
    return UW_ERR_INVALID_ARG;
  if (a.activation < UW_ACT_NONE || a.activation > UW_ACT_SILU || a.out_type < UW_OUT_BF16 ||
      a.out_type > UW_OUT_FP32)
    return UW_ERR_INVALID_ARG;
  if (a.ws_bytes < g.bytes) return UW_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const void* x = a.x;
  int x_rows = a.x_rows;
  const bool gather = a.rows && !g.permuted;
  if (g.permuted) {
    PermuteParams q;
    q.x = reinterpret_cast<const uint4*>(a.x);
    q.rows = a.rows;
    q.offsets = a.offsets;
    q.out = reinterpret_cast<uint4*>(ws + g.permuted);
    q.E = a.E;
    q.x_rows = a.x_rows;
    q.n_rows = a.n_rows;
    q.pieces = static_cast<int>(a.K / 8);
    q.status = reinterpret_cast<uint32_t*>(ws);
    if ((st = launch_permute(q, std::min(a.n_rows, 8 * dev.sm_count), s)) != UW_OK) return st;
    x = q.out;
    x_rows = a.n_rows;
  }
  CUtensorMap tx;
  if ((st = make_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, static_cast<uint64_t>(a.K),
                               static_cast<uint64_t>(x_rows), static_cast<uint64_t>(a.K) * 2, 64, gather ? 1 : 16,
                               CU_TENSOR_MAP_SWIZZLE_128B)) != UW_OK)
    return st;
  CUtensorMap tx64 = tx;
  if (!gather && g.lay.cap >= 64 &&
      (st = make_tensor_map_2d(&tx64, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, static_cast<uint64_t>(a.K),
                               static_cast<uint64_t>(x_rows), static_cast<uint64_t>(a.K) * 2, 64, 64,
                               CU_TENSOR_MAP_SWIZZLE_128B)) != UW_OK)
    return st;
  GParams p;
  std::memset(&p, 0, sizeof(p));
  p.E = a.E;
  p.N = static_cast<int>(a.N);
  p.KB = g.KB;
  p.n_mt = g.n_mt;
  p.n_mt_all = static_cast<int>((a.N + 127) / 128);
  p.x_rows = x_rows;
  p.n_rows = a.n_rows;
  p.gather = gather ? 1 : 0;
  p.grid = g.grid;
  p.cap = g.lay.cap;
  p.n_iss = g.lay.n_iss;
  p.n_acc = g.lay.n_acc;
  p.sx = g.lay.sx;
  p.sa = g.lay.sa;
  p.sw = g.lay.sw;
  p.x_slot_bytes = g.lay.x_slot_bytes;
  p.w_base = g.lay.w_base;
  p.w_slot_bytes = g.lay.w_slot_bytes;
  p.sched_off = g.lay.sched_off;
  p.turn_off = g.lay.turn_off;
  p.vec = a.N % 8 == 0 && aligned16(a.residual);
  p.bar_off = g.lay.bar_off;
  p.a_col0 = g.lay.a_col0;
  p.vcap = g.lay.vcap;
  // Measured by switching it off (0) and to 1000: 256 rows of 14336 x 4096
  // 44.9 us split, 37.1 whole (64 k-blocks against 48); 64 experts of
  // 2048 x 1024 37.4 / 35.7; but one row of 4096 x 14336 20.5 / 57.6
  p.join = 6 + g.lay.cap / 8;
  // Runs of r of a tile's KB k-blocks take 0.7 r, adding up its KB / r parts
  // 0.35 each for every 48 columns: least in all at the root of half KB
  p.min_run = std::max(1, static_cast<int>(std::sqrt(0.5 * g.KB * ((g.lay.cap + 47) / 48))));
  // (the permuting kernel lets this one in after waiting for its own
  // predecessor, which may have written the offsets)
  p.early = a.offsets == nullptr || a.offsets_ready || g.permuted;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.table[0] = static_cast<const ExpertDesc*>(a.table[0]);
  p.table[1] = static_cast<const ExpertDesc*>(a.table[1]);
  if (a.one) p.one = *a.one;
  p.bias = a.bias;
  p.residual = a.residual;
  p.act = a.activation;
  p.out_fp32 = a.out_type == UW_OUT_FP32;
  p.y = a.y;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.counters = reinterpret_cast<uint32_t*>(ws + kWsHeader);
  p.partials = reinterpret_cast<float*>(ws + kWsHeader + kCounterBytes);
  p.partial_stride = static_cast<long long>(g.partial_stride);
  if (a.swiglu) return launch_grouped_kernel<2, false>(tx, tx64, p, g.lay.smem, s);
  return g.pair ? launch_grouped_kernel<2, true>(tx, tx64, p, g.lay.smem, s)
                : launch_grouped_kernel<1, false>(tx, tx64, p, g.lay.smem, s);
}

}  // namespace uw

using namespace uw;

extern "C" size_t uw_experts_table_bytes(int32_t n_experts) {
  return n_experts < 1 || n_experts > kMaxExperts ? 0 : static_cast<size_t>(n_experts) * sizeof(ExpertDesc);
}

extern "C" uw_status uw_experts_init(const uw_matrix* const* mats, int32_t n_experts, void* table, size_t table_bytes,
                                     uw_experts* out, void* stream) {
  if (!mats || !table || !out || n_experts < 1 || n_experts > kMaxExperts || !aligned16(table)) return UW_ERR_INVALID_ARG;
  if (table_bytes < uw_experts_table_bytes(n_experts)) return UW_ERR_WORKSPACE_TOO_SMALL;
  ExpertDesc host[64];  // records go out in batches: no allocation that could throw
  for (int32_t e = 0; e < n_experts; ++e) {
    if (!mats[e]) return UW_ERR_INVALID_ARG;
    if (mats[e]->L.rows != mats[0]->L.rows || mats[e]->L.cols != mats[0]->L.cols) return UW_ERR_UNSUPPORTED_SHAPE;
    const uw_status st = expert_desc(mats[e], &host[0]);
    if (st != UW_OK) return st;
  }
  DeviceInfo dev;
  uw_status st = device_info(&dev);
  if (st != UW_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t e0 = 0; e0 < n_experts; e0 += 64) {
    const int32_t n = std::min(64, n_experts - e0);
    for (int32_t i = 0; i < n; ++i)
      if ((st = expert_desc(mats[e0 + i], &host[i])) != UW_OK) return st;
    if (cudaMemcpyAsync(static_cast<ExpertDesc*>(table) + e0, host, static_cast<size_t>(n) * sizeof(ExpertDesc),
                        cudaMemcpyHostToDevice, s) != cudaSuccess)
      return UW_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return UW_ERR_CUDA;  // the host records change next
  }
  std::memset(out, 0, sizeof(*out));
  out->n_experts = n_experts;
  out->rows = mats[0]->L.rows;
  out->cols = mats[0]->L.cols;
  out->table = table;
  return UW_OK;
}

namespace {
bool experts_ok(const uw_experts* w) { return w && w->table && aligned16(w->table); }
}  // namespace

extern "C" size_t uw_grouped_workspace_bytes(const uw_experts* w, int32_t n_rows, int32_t swiglu) {
  return w ? grouped_ws_bytes(w->rows, w->cols, w->n_experts, n_rows, swiglu != 0, true) : 0;
}

extern "C" uw_status uw_gemm_grouped(const uw_experts* w, const uint16_t* x, int32_t x_rows, const int32_t* rows,
                                     const int32_t* offsets, int32_t n_rows, const uw_epilogue* epi, void* y,
                                     void* ws, size_t ws_bytes, void* stream) {
  if (!experts_ok(w) || !offsets || n_rows < 0 || x_rows < 0) return UW_ERR_INVALID_ARG;
  if (!rows && x_rows < n_rows) return UW_ERR_INVALID_ARG;  // row s of x is slot s
  if (n_rows == 0) return UW_OK;
  GroupedArgs a;
  a.N = w->rows;
  a.K = w->cols;
  a.E = w->n_experts;
  a.table[0] = w->table;
  a.x = x;
  a.x_rows = x_rows;
  a.rows = rows;
  a.offsets = offsets;
  a.n_rows = n_rows;
  if (epi) {
    a.bias = epi->bias;
    a.residual = epi->residual;
    a.activation = epi->activation;
    a.out_type = epi->out_type;
  }
  a.y = y;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  return launch_grouped(a, static_cast<cudaStream_t>(stream));
}

extern "C" uw_status uw_gemm_grouped_swiglu(const uw_experts* gate, const uw_experts* up, const uint16_t* x,
                                            int32_t x_rows, const int32_t* rows, const int32_t* offsets,
                                            int32_t n_rows, uint16_t* h, void* ws, size_t ws_bytes, void* stream) {
  if (!experts_ok(gate) || !experts_ok(up) || !offsets || n_rows < 0 || x_rows < 0) return UW_ERR_INVALID_ARG;
  if (gate->n_experts != up->n_experts || gate->rows != up->rows || gate->cols != up->cols) return UW_ERR_INVALID_ARG;
  if (!rows && x_rows < n_rows) return UW_ERR_INVALID_ARG;
  if (n_rows == 0) return UW_OK;
  GroupedArgs a;
  a.N = gate->rows;
  a.K = gate->cols;
  a.E = gate->n_experts;
  a.swiglu = true;
  a.table[0] = gate->table;
  a.table[1] = up->table;
  a.x = x;
  a.x_rows = x_rows;
  a.rows = rows;
  a.offsets = offsets;
  a.n_rows = n_rows;
  a.y = h;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  return launch_grouped(a, static_cast<cudaStream_t>(stream));
}

extern "C" size_t uw_gemm_epilogue_workspace_bytes(const uw_layout* L, int32_t batch) {
  return L ? grouped_ws_bytes(L->rows, L->cols, 1, batch, false, false) : 0;
}

extern "C" uw_status uw_gemm_epilogue(const uw_matrix* m, const uint16_t* x, int32_t batch, const uw_epilogue* epi,
                                      void* y, void* ws, size_t ws_bytes, void* stream) {
  if (!m || batch < 0) return UW_ERR_INVALID_ARG;
  ExpertDesc d;
  const uw_status st = expert_desc(m, &d);
  if (st != UW_OK) return st;
  if (batch == 0) return UW_OK;
  GroupedArgs a;
  a.N = m->L.rows;
  a.K = m->L.cols;
  a.E = 1;
  a.one = &d;
  a.x = x;
  a.x_rows = batch;
  a.n_rows = batch;
  if (epi) {
    a.bias = epi->bias;
    a.residual = epi->residual;
    a.activation = epi->activation;
    a.out_type = epi->out_type;
  }
  a.y = y;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  return launch_grouped(a, static_cast<cudaStream_t>(stream));
}
