// kv_prefill.cuh -- causal attention of the new tokens of every sequence over
// its cache rows, on the fifth-generation tensor cores.
//
// Rows and jobs.  The G query heads of a kv head read the same keys, so a row
// of the matrix product is a (token, head) pair: a tile is floor(128 / G) whole
// tokens, row = token * G + head, in the 128 rows of a tensor-core product, and a
// job is two such tiles of one sequence and kv head, which share every key and
// value tile.  A key tile is 128 cache rows (a unit of a job's work).
//
// One block per SM runs a piece of the line of all jobs:
//   warps 0, 2  load key tiles (0), query and value tiles (2) (tiled TMA, keys and
//               values one box per page piece, 128-byte swizzle); warp 0 also
//               walks the block's piece of the line and posts one record per job
//               in a ring, so that the others do no arithmetic on jobs
//   warps 1, 3  issue the products, S_t = Q_t K^T and O_t += P_t V for tile t, both
//               with the accumulator in tensor memory; P is the A operand straight
//               from tensor memory, V the transposed (MN-major) B operand
//   warps 4-7   softmax of tile 0, one row per thread: S from tensor memory to
//               registers, running maximum and sum in fp32, P (bf16) back to
//               tensor memory; O's rescale, where a maximum rises by more than
//               2^8 (rare after the first tiles), and the results
//   warps 8-11  the same for tile 1
// The tensor cores work on one tile while the other's softmax runs.  64-dim heads
// leave tensor memory for P beside S, so that the next S, of the next job if need
// be, is made while the softmax still works on this one; a warp per tile issues
// their products, and neither tile waits for the other.  128-dim heads fill tensor
// memory (2 x 128 columns S, 2 x 128 O): P takes S's place, its product starts when
// half of it is there, and one warp issues both tiles' products in turn (a warp
// each: 228 to 260 us where this took 223).
//
// Bound: with 128-dim heads the tensor cores (4 D operations a pair; 8192 tokens of
// 16 heads, 275 GFLOP, take 183 us: 1.50 PFLOP/s, 0.78 of a measured GEMM's rate),
// with 64-dim heads the chain of steps of the softmax warps (8192 tokens of 32 heads:
// 257 us, 1.07 PFLOP/s).  A unit of two tiles has 32768 pairs: their exponentials take
// an SM 1040 cycles, their scaling, sums, maxima and rounding as many on other pipes;
// the softmax warps alone took 1625, with the products beside them about 2100, and no
// pipe is full (eight prompts of 512-2048 tokens: exponentials 0.34 of the active
// cycles, products 0.33, issue slots 0.43).  Short prompts are bound by the start (3 us
// of look-ups), the jobs' starts and ends (2.5 units a job: 20 of the 72 units of those
// eight prompts' blocks) and the joins (4 of their 84 us).  Where the compiler puts the
// softmax loop moves the times of 64-dim heads by up to 4 % (257 to 268 us).
//
// The line's measure is keys: a job costs its visible rows and PF_JOB_COST for
// its start and end, and is cut wherever an equal share of the whole ends (or
// at the job's border where that is near).  Parts of one job end as partial
// states that a dependent kernel joins.  Everything is found on the device
// from lens and cu.
//
// The weights P are rounded to bf16 (2^-8 of each weight at most, as the output's
// own rounding); their sum is taken before the rounding.  Cache rows
// from len on are never part of a product: the tile that holds the end of a
// sequence takes its values through cp.async with zeros behind the end.  Rows
// that a query does not see have weight zero, which times an infinite or NaN
// value of a later token would still be NaN: rows whose result is not finite
// although their weights are, are redone by attn_row.
//
// Every wait is bounded in time: where the block gets no further for two seconds
// (mk_kv_set_wait_timeout), all warps leave through the common end: the loaders wait
// for their copies and the product warps for their products in flight, then the tensor
// memory is freed and the status word set.
#pragma once
#include <cuda.h>

#include "attn_tc.cuh"
#include "kv_attn.cuh"
#include "mk_tc.cuh"

namespace mk {

constexpr int PF_THREADS = 384;
constexpr int PF_REGS = 168;      // per thread at launch (setmaxnreg deals them out anew)
constexpr int PF_ROWS = 256;      // rows of a job
constexpr int PF_UNIT = 128;      // cache rows of a unit
constexpr int PF_JOB_COST = 320;  // a job's start and end, in keys (measured: 2.3 to 2.6 units)
// A part of a job is not worth less: a cut costs another start and end, 2.5 units, and
// the join, 3 to 5 us with units of 1.1.  One prompt, us with 7, 6 and 5 units:
//   32/8 heads of 64, tokens   768 18.2 18.2 17.1   960 19.1 19.1 19.9   1024 18.2 20.6 20.9
//   16/4 heads of 128, tokens  768 21.5 21.6 20.1   960 23.9 24.0 26.2   1024 21.1 23.4 23.9
//                             1100 26.6 28.3 27.2  1280 26.9 27.3 26.1   1500 28.7 27.1 26.8
constexpr int PF_MIN_SHARE = 7 * PF_UNIT;
// A cut so many keys from a job's border moves there: a partial state and its join
// cost about as much.
constexpr int PF_SNAP = 4 * PF_UNIT;
constexpr int PF_AFTER = 1 << 30;
constexpr unsigned long long PF_DRAIN_NS = 2000000000ull;  // for what is in flight at the end

template <int D>
struct PfShape {
  static constexpr bool SEP = D == 64;  // P beside S in tensor memory
  static constexpr int TILE = 128 * D * 2;
  static constexpr int STAGES = D == 64 ? 4 : 2;  // of keys, and as many of values
  static constexpr int SMEM = 1024 + 2 * TILE + 2 * STAGES * TILE;
  static constexpr uint32_t S_COL = 0, O_COL = 256, P_COL = SEP ? 256 + 2 * D : 0;
  static constexpr size_t STATE = (size_t)PF_ROWS * (D + 2);  // floats: o [D/4][256][4], m, l [256]
};

// Scratch: two partial states per block, then what each block's piece begins with.
struct PfPart {
  int b, h, j;       // its first job
  int inside, more;  // it begins inside that job; it holds anything
  int row, rows[2];  // of the job: first token's row of q, rows of its tiles
};

struct PfArgs {
  AttnArgs a;
  int per;       // tokens of a tile
  int negate;    // the scale is negative: scale2 is its magnitude, Q K^T is negated
  float scale2;  // |scale| log2 e
  int box;       // rows of a TMA box
  unsigned long long wait_ns;  // how long a block may get no further
};

// ---- the line of jobs ------------------------------------------------------
struct PfSeq {
  int b, len, first, n;  // sequence, its rows, its new tokens' first row and number
  int jobs;              // of one kv head
};

struct PfJob {
  PfSeq s;
  int h, j;
};

struct PfCut {
  PfJob job;
  int unit;       // 0: before the job; PF_AFTER: behind it; else a cut inside it
  long long off;  // of the cut from the job's start
};

MK_DEV PfSeq pf_seq(const PfArgs& p, int b) {
  PfSeq s{};
  s.b = b;
  if (b < p.a.bt.batch) {
    s.len = kv_len(p.a.kv, p.a.bt, b);
    kv_new_tokens(p.a.bt, b, s.first, s.n);
    s.jobs = (s.n + 2 * p.per - 1) / (2 * p.per);
  }
  return s;
}

// Keys before job j of one kv head.
MK_DEV long long pf_before(const PfArgs& p, const PfSeq& s, int j) {
  const long long base = max(0, s.len - s.n) + PF_JOB_COST;
  return base * j + (long long)p.per * j * (j + 1);
}

// Cache rows that the job's token range [.., last] sees, and its units.
MK_DEV int pf_seen(const PfSeq& s, int token) { return max(0, s.len - s.n + token + 1); }
MK_DEV int pf_units(const PfArgs& p, const PfJob& w) {
  return (pf_seen(w.s, min(w.s.n, 2 * p.per * (w.j + 1)) - 1) + PF_UNIT - 1) / PF_UNIT;
}

// How the line is cut: part i begins at quot * i + rest * i / parts.
struct PfLine {
  long long total, quot;
  int parts, rest;
  MK_DEV long long begin(int i) const { return quot * i + (unsigned)rest * (unsigned)i / (unsigned)parts; }
};

// The whole line (one warp; s0: this lane's sequence among the first 32).
MK_DEV PfLine pf_line(const PfArgs& p, int blocks, int lane, const PfSeq& s0) {
  long long n = 0;
  int jobs = 0;
  for (int b = lane; b < p.a.bt.batch; b += 32) {
    const PfSeq s = b < 32 ? s0 : pf_seq(p, b);
    n += pf_before(p, s, s.jobs);
    jobs += s.jobs;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    n += __shfl_xor_sync(0xFFFFFFFFu, n, w);
    jobs += __shfl_xor_sync(0xFFFFFFFFu, jobs, w);
  }
  PfLine l;
  l.total = n * p.a.kv.Hkv;
  // As many parts as jobs while a block each is there, more where they are an eighth more:
  // fewer move every cut for the sake of a few blocks (1100 tokens of 32/8 heads of 64,
  // 144 jobs: 21.1 us, 22.3 as 149 parts; 2048 of 16/4 heads of 128, 128 jobs: 36.2, 34.0
  // as 152 parts).
  const long long all = (long long)jobs * p.a.kv.Hkv, cut = min((long long)blocks, l.total / PF_MIN_SHARE);
  l.parts = (int)(8 * cut < 9 * all ? min((long long)blocks, all) : cut);
  if (l.parts > 0) {
    l.quot = l.total / l.parts;
    l.rest = (int)(l.total - l.quot * l.parts);
  }
  return l;
}

// Unit of a job at which a cut `off` keys from its start falls.
MK_DEV int pf_unit_at(const PfArgs& p, const PfJob& w, long long off) {
  const int units = pf_units(p, w);
  const long long size = pf_before(p, w.s, w.j + 1) - pf_before(p, w.s, w.j);
  if (off <= PF_SNAP) return off == 0 || off < size - off ? 0 : PF_AFTER;
  if (size - off <= PF_SNAP) return PF_AFTER;
  const long long u = (off + PF_UNIT / 2) / PF_UNIT;
  return u >= units ? PF_AFTER : (int)u;
}

// Where cut c (keys from the start) falls; from the total on, the end of the
// line (one warp, c the same or not on its lanes as `c0` for the even and `c1`
// for the odd ones: two cuts for the price of one).
MK_DEV PfCut pf_find(const PfArgs& p, long long c0, long long c1, int lane, const PfSeq& s0) {
  long long before = 0;
  PfCut r{};
  r.job.s.b = p.a.bt.batch;
  const long long c = lane & 1 ? c1 : c0;
  long long rem = -1;
  for (int b0 = 0; b0 < p.a.bt.batch; b0 += 32) {
    const PfSeq s = b0 == 0 ? s0 : pf_seq(p, b0 + lane);
    const long long own = pf_before(p, s, s.jobs) * p.a.kv.Hkv;
    long long incl = own;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, w);
      if (lane >= w) incl += y;
    }
    const unsigned hit0 = __ballot_sync(0xFFFFFFFFu, own > 0 && before + incl > c0);
    const unsigned hit1 = __ballot_sync(0xFFFFFFFFu, own > 0 && before + incl > c1);
    const unsigned hit = lane & 1 ? hit1 : hit0;
    const int src = hit ? __ffs(hit) - 1 : 0;
    PfSeq t;
    t.b = b0 + src;
    t.len = __shfl_sync(0xFFFFFFFFu, s.len, src);
    t.first = __shfl_sync(0xFFFFFFFFu, s.first, src);
    t.n = __shfl_sync(0xFFFFFFFFu, s.n, src);
    t.jobs = __shfl_sync(0xFFFFFFFFu, s.jobs, src);
    const long long start = before + __shfl_sync(0xFFFFFFFFu, incl - own, src);
    if (hit && rem < 0) {
      r.job.s = t;
      rem = c - start;
    }
    if (hit0 && hit1) break;
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  if (rem >= 0) {
    // kv head, then the last job that starts at or before rem: estimates in
    // floating point, put right in whole numbers
    const PfSeq& q = r.job.s;
    const long long one = pf_before(p, q, q.jobs);
    int h = min((int)((float)rem / (float)one), p.a.kv.Hkv - 1);
    while (h > 0 && one * h > rem) h--;
    while (one * (h + 1) <= rem) h++;
    rem -= one * h;
    r.job.h = h;
    const float base = (float)(max(0, q.len - q.n) + PF_JOB_COST) + p.per;
    int j = (int)((sqrtf(base * base + 4.f * p.per * (float)rem) - base) / (2 * p.per));
    j = min(max(j, 0), q.jobs - 1);
    while (j > 0 && pf_before(p, q, j) > rem) j--;
    while (j + 1 < q.jobs && pf_before(p, q, j + 1) <= rem) j++;
    r.job.j = j;
    r.off = rem - pf_before(p, q, j);
    r.unit = pf_unit_at(p, r.job, r.off);
  }
  return r;
}

// The cut that lane `src` found.
MK_DEV PfCut pf_shfl(const PfCut& c, int src) {
  PfCut r;
  r.job.s.b = __shfl_sync(0xFFFFFFFFu, c.job.s.b, src);
  r.job.s.len = __shfl_sync(0xFFFFFFFFu, c.job.s.len, src);
  r.job.s.first = __shfl_sync(0xFFFFFFFFu, c.job.s.first, src);
  r.job.s.n = __shfl_sync(0xFFFFFFFFu, c.job.s.n, src);
  r.job.s.jobs = __shfl_sync(0xFFFFFFFFu, c.job.s.jobs, src);
  r.job.h = __shfl_sync(0xFFFFFFFFu, c.job.h, src);
  r.job.j = __shfl_sync(0xFFFFFFFFu, c.job.j, src);
  r.unit = __shfl_sync(0xFFFFFFFFu, c.unit, src);
  r.off = __shfl_sync(0xFFFFFFFFu, c.off, src);
  return r;
}

MK_DEV void pf_next(const PfArgs& p, PfJob& w) {
  if (++w.j < w.s.jobs) return;
  w.j = 0;
  if (++w.h < p.a.kv.Hkv) return;
  w.h = 0;
  do {
    w.s = pf_seq(p, w.s.b + 1);
  } while (w.s.b < p.a.bt.batch && w.s.jobs == 0);
}

MK_DEV bool pf_same(const PfJob& x, const PfJob& y) {
  return x.s.b == y.s.b && x.h == y.h && x.j == y.j;
}

// What the roles need to know about a job, and how they pass it on.
struct PfRec {
  int b, h, len;        // sequence, kv head, cache rows (b < 0: no more jobs)
  int row, pos;         // first token of the job: its row of q, its position
  int ka, e[2];         // units [ka, e[t]) for tile t
  int rows[2];          // rows of tile t (none: <= 0)
  int whole, slot;      // all units of the job; slot of its partial state
};

// A block's way along its piece of the line.
struct PfWalk {
  PfJob job;
  PfCut end;
  int ka, kb;       // units of the present job
  bool whole;       // all of them
  bool first;       // the piece's first job
  bool inside;      // the piece begins inside a job
  bool more;

  MK_DEV void begin(const PfArgs& p, int part, int lane) {
    const PfSeq s0 = pf_seq(p, lane);
    const PfLine line = pf_line(p, gridDim.x, lane, s0);
    more = inside = false;
    job.s.b = -1;
    if (part >= line.parts) return;
    const PfCut both = pf_find(p, line.begin(part), line.begin(part + 1), lane, s0);
    const PfCut c = pf_shfl(both, 0);
    end = pf_shfl(both, 1);
    job = c.job;
    ka = c.unit;
    inside = ka > 0 && ka < PF_AFTER;
    if (pf_same(c.job, end.job) && c.unit == end.unit) return;
    if (ka == PF_AFTER) {
      pf_next(p, job);
      ka = 0;
    }
    first = true;
    more = true;
    settle(p);
  }
  MK_DEV void settle(const PfArgs& p) {
    if (job.s.b >= p.a.bt.batch || (pf_same(job, end.job) && end.unit == 0)) {
      more = false;
      return;
    }
    const int units = pf_units(p, job);
    kb = pf_same(job, end.job) ? min(end.unit, units) : units;
    whole = ka == 0 && kb == units;
  }
  MK_DEV void next(const PfArgs& p) {
    first = false;
    if (pf_same(job, end.job)) {
      more = false;
      return;
    }
    pf_next(p, job);
    ka = 0;
    settle(p);
  }
  // The present job, or the end.
  MK_DEV void record(const PfArgs& p, PfRec& r) const {
    r.b = -1;
    if (!more) return;
    r.b = job.s.b;
    r.h = job.h;
    r.len = job.s.len;
    const int token = 2 * job.j * p.per;
    r.row = job.s.first + token;
    r.pos = job.s.len - job.s.n + token;
    r.ka = ka;
#pragma unroll
    for (int t = 0; t < 2; t++) {
      r.rows[t] = tokens_of(p, t) * p.a.G;
      r.e[t] = end_of(p, t);
    }
    r.whole = whole;
    r.slot = first ? 0 : 1;
  }
  // What the join needs to know of the piece (at its beginning).
  MK_DEV void part(const PfArgs& p, PfPart& r) const {
    r.b = job.s.b;
    r.h = job.h;
    r.j = job.j;
    r.inside = inside;
    r.more = more;
    r.row = job.s.first + 2 * job.j * p.per;
    r.rows[0] = tokens_of(p, 0) * p.a.G;
    r.rows[1] = tokens_of(p, 1) * p.a.G;
  }
  // Tokens of tile t, and the end of the units that it takes part in.
  MK_DEV int tokens_of(const PfArgs& p, int t) const {
    return min(p.per, job.s.n - (2 * job.j + t) * p.per);
  }
  MK_DEV int end_of(const PfArgs& p, int t) const {
    const int n = tokens_of(p, t);
    if (n <= 0) return ka;
    const int last = (2 * job.j + t) * p.per + n - 1;
    return max(ka, min(kb, (pf_seen(job.s, last) + PF_UNIT - 1) / PF_UNIT));
  }
};

// ---- small pieces ----------------------------------------------------------
constexpr int PF_RECS = 4;

struct PfShared {
  alignas(8) unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4];
  unsigned long long rec_full[PF_RECS], rec_empty[PF_RECS];
  unsigned long long q_full[2], q_empty[2], s_full[2], s_free[2], p_half[2], p_full[2], pv_done[2], o_empty[2];
  unsigned long long drain;
  PfRec rec[PF_RECS];
  uint32_t tmem;
  volatile int abort;
  // When waiting ends (globaltimer): put off by the key loader as it gets on, which
  // hangs on all other roles, and by a warp that is about to redo a row.
  // (wait_ns from the parameters at each use instead: 8192 tokens of 64-dim heads 261 ->
  // 268 us, by the place of the code alone.)
  unsigned long long limit, wait_ns;
};

MK_DEV void pf_put_off(PfShared& sh, unsigned long long ns) { atomicMax(&sh.limit, gtimer() + ns); }

// Wait for phase `n` (counted from 0) of a barrier; false if the block gave up.
// (Few instructions: some 30 places wait, and what they fetch counts.)
MK_DEV bool pf_wait(PfShared& sh, const unsigned long long* bar, uint32_t n) {
  const uint32_t b = smem_u32(bar);
  for (uint32_t it = 0; !mbar_try(b, n & 1); it++) {
    if ((it & 63) != 63) continue;
    if (sh.abort) return false;
    if (gtimer() > *(volatile unsigned long long*)&sh.limit) sh.abort = 1;
  }
  return true;
}

// The next record (one warp): false if the block gave up or there are no more jobs.
MK_DEV bool pf_take(PfShared& sh, uint32_t& n, PfRec& r, bool lead) {
  const int i = n % PF_RECS;
  if (!__all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.rec_full[i], n / PF_RECS))) return false;
  r = sh.rec[i];
  __syncwarp();
  if (lead) mbar_arrive(smem_u32(&sh.rec_empty[i]));
  n++;
  return r.b >= 0;
}

// Tiled 3-D TMA load of one box, as tma_load_2d.
MK_DEV void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// Low and high words of shared-memory matrix descriptors in the 128-byte
// swizzle (the fields are those of sw128_desc): 8-row atoms 1024 bytes apart.
// For a transposed (MN-major) operand a row holds 64 elements along N, an atom 8
// rows along K, and the next 64 elements of N follow at +16384 (the leading offset).
constexpr uint32_t DESC_HI = 0x40004040u;
MK_DEV uint32_t desc_lo(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
MK_DEV uint32_t desc_lo_mn(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((16384u >> 4) << 16); }

// D[tmem] (+)= A * B^T, both operands from shared memory.
MK_DEV void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(DESC_HI)
      : "memory");
}

// The same with the A operand from tensor memory.
MK_DEV void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(DESC_HI)
      : "memory");
}

// True on one lane of the (whole) warp.
MK_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

#define PF_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define PF_R16(x, i) PF_R4(x, i), PF_R4(x, i + 4), PF_R4(x, i + 8), PF_R4(x, i + 12)
#define PF_U4(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3])
#define PF_U16(x, i) PF_U4(x, i), PF_U4(x, i + 4), PF_U4(x, i + 8), PF_U4(x, i + 12)
#define PF_I4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define PF_I16(x, i) PF_I4(x, i), PF_I4(x, i + 4), PF_I4(x, i + 8), PF_I4(x, i + 12)

// 64 consecutive columns of this thread's tensor-memory lane; they are there
// after tmem_ld64_wait, which all uses depend on.
MK_DEV void tmem_ld64(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
      "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, "
      "%36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, "
      "%53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : PF_R16(x, 0), PF_R16(x, 16), PF_R16(x, 32), PF_R16(x, 48)
      : "r"(addr)
      : "memory");
}
MK_DEV void tmem_ld64_wait(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : PF_U16(x, 0), PF_U16(x, 16), PF_U16(x, 32), PF_U16(x, 48)::"memory");
}

MK_DEV void tmem_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : PF_R16(x, 0), PF_R16(x, 16)
      : "r"(addr)
      : "memory");
}
template <int N>
MK_DEV void tmem_ldn(uint32_t addr, uint32_t* x) {
  if (N == 64) {
    tmem_ld64(addr, x);
    tmem_ld64_wait(x);
  } else {
    tmem_ld32(addr, x);
  }
}
MK_DEV void tmem_st32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::PF_I16(x, 0),
      PF_I16(x, 16), "r"(addr)
      : "memory");
}
MK_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

MK_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest of 64 floats (NaN counts as none).
MK_DEV float max64(const uint32_t* x) {
  float m[4];
#pragma unroll
  for (int c = 0; c < 4; c++) {
    m[c] = fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 4]));
#pragma unroll
    for (int i = 8; i < 64; i += 8)
      m[c] = max3(m[c], __uint_as_float(x[i + c]), __uint_as_float(x[i + c + 4]));
  }
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// 2^x to about 2 units in the last place; results below 2^-126 are zero.
MK_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MK_DEV void cp_async16_zfill(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(PF_THREADS, 1)
kv_prefill_kernel(const __grid_constant__ PfArgs p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Sh = PfShape<D>;
  constexpr int C = D / 64;  // 64-column halves of a tile
  constexpr bool SEP = Sh::SEP;
  constexpr uint32_t NS = Sh::STAGES;
  extern __shared__ unsigned char raw[];
  __shared__ PfShared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t q_smem = base, k_ring = base + 2 * Sh::TILE, v_ring = k_ring + NS * Sh::TILE;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; i++) {
      mbar_init(smem_u32(&sh.k_full[i]), 1);
      mbar_init(smem_u32(&sh.k_empty[i]), SEP ? 2 : 1);
      mbar_init(smem_u32(&sh.v_full[i]), 1);
      mbar_init(smem_u32(&sh.v_empty[i]), SEP ? 2 : 1);
    }
    for (int i = 0; i < PF_RECS; i++) {
      mbar_init(smem_u32(&sh.rec_full[i]), 1);
      mbar_init(smem_u32(&sh.rec_empty[i]), SEP ? 11 : 10);  // the warps that read it
    }
    for (int t = 0; t < 2; t++) {
      mbar_init(smem_u32(&sh.q_full[t]), 1);
      mbar_init(smem_u32(&sh.q_empty[t]), 1);
      mbar_init(smem_u32(&sh.s_full[t]), 1);
      mbar_init(smem_u32(&sh.s_free[t]), 4);
      mbar_init(smem_u32(&sh.p_half[t]), 4);
      mbar_init(smem_u32(&sh.p_full[t]), 4);
      mbar_init(smem_u32(&sh.pv_done[t]), 1);
      mbar_init(smem_u32(&sh.o_empty[t]), 4);
    }
    mbar_init(smem_u32(&sh.drain), 2);
    sh.abort = 0;
    sh.wait_ns = p.wait_ns;
    sh.limit = gtimer() + p.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const AttnArgs& a = p.a;
  PfPart* parts = (PfPart*)(a.ws + (size_t)gridDim.x * 2 * Sh::STATE);

  // The block's registers, PF_REGS x 384, are dealt out anew: 128 x 104 + 256 x 200.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || warp == 2) {
      // ------------------------------------- keys (warp 0), values (warp 2) ----
      const bool is_v = warp == 2;
      const uint32_t ring = is_v ? v_ring : k_ring;
      unsigned long long* full = is_v ? sh.v_full : sh.k_full;
      const unsigned long long* empty = is_v ? sh.v_empty : sh.k_empty;
      const void* map = is_v ? &vmap : &kmap;
      const uint64_t policy = policy_evict_normal();
      const int shift = a.kv.shift, in_block = a.kv.table ? a.kv.block - 1 : 0x7FFFFFFF;
      const uint32_t my_box = (uint32_t)lane * p.box;
      uint32_t n = 0, taken = 0;  // stages filled, records taken (or posted)
      bool ok = true;
      PfRec w;
      uint32_t q_used = 0, q_phase = 0;  // by tile: loaded before; phase of q_empty
      PfWalk walk;
      if (!is_v) {
        walk.begin(p, blockIdx.x, lane);
        if (lane == 0) walk.part(p, parts[blockIdx.x]);
      }
      // Warp 0: the present job's record, for itself and the other warps; the one
      // after the last job says so.
      auto post = [&]() {
        const int i = taken % PF_RECS;
        if (taken >= PF_RECS && !__all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.rec_empty[i], taken / PF_RECS - 1)))
          return false;
        walk.record(p, w);
        if (lane == 0) {
          sh.rec[i] = w;
          mbar_arrive(smem_u32(&sh.rec_full[i]));
        }
        __syncwarp();
        taken++;
        return w.b >= 0;
      };
      while (ok && (is_v ? pf_take(sh, taken, w, lane == 0) : post())) {
        const int kb = max(w.e[0], w.e[1]);
        if (kb == w.ka) {
          if (!is_v) walk.next(p);
          continue;
        }
        if (is_v) {  // the queries: one box of whole tokens and their heads per tile
          const int tile_rows = p.per * a.G;
#pragma unroll
          for (int t = 0; t < 2; t++) {
            if (w.e[t] == w.ka) continue;
            if (q_used >> t & 1) {
              ok = ok && __all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.q_empty[t], q_phase >> t & 1));
              q_phase ^= (uint32_t)ok << t;  // (no load follows a wait that failed)
            }
            q_used |= (uint32_t)ok << t;
            if (ok && lane == 0) {
              const uint32_t bar = smem_u32(&sh.q_full[t]), dst = q_smem + t * Sh::TILE;
              mbar_expect_tx(bar, (uint32_t)tile_rows * D * 2);
#pragma unroll
              for (int c = 0; c < C; c++)
                tma_load_3d(dst + c * 16384, &qmap, 64 * c, w.h * a.G, w.row + t * p.per, bar,
                            policy);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        // Block of this lane's box of a unit, looked up one unit ahead; a lane
        // whose box begins behind the sequence's end has none to load.
        const int* table = a.kv.table + (size_t)w.b * a.kv.table_stride;
        auto lookup = [&](int unit) {
          const int r = min(unit * PF_UNIT + (int)my_box, w.len - 1);
          return a.kv.table ? __ldg(table + (r >> shift)) : w.b;
        };
        int ahead = lookup(w.ka);
        for (int j = w.ka; j < kb; j++) {
          const int blk = ahead;
          if (j + 1 < kb) ahead = lookup(j + 1);
          const uint32_t st = n % NS, dst = ring + st * Sh::TILE, bar = smem_u32(&full[st]);
          if (n >= NS) ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &empty[st], n / NS - 1));
          if (!ok) break;
          n++;
          const int row = j * PF_UNIT, left = w.len - row;
          if (is_v && left < PF_UNIT) {
            // the end of the sequence: zeros behind it
            const int k = lane % (D / 8);  // 16-byte chunk of a row
#pragma unroll 4
            for (int r = lane / (D / 8); r < PF_UNIT; r += 32 / (D / 8)) {
              const int b = __shfl_sync(0xFFFFFFFFu, blk, r / p.box);
              const bool in = r < left && (unsigned)b < (unsigned)a.kv.n_blocks;
              const long long src = ((long long)b * a.kv.Hkv + w.h) * a.kv.block + ((row + r) & in_block);
              cp_async16_zfill(dst + (k >> 3) * 16384 + r * 128 + (((k ^ r) & 7) << 4),
                               in ? a.kv.v + src * D + k * 8 : a.kv.v, in);
            }
            if (__any_sync(0xFFFFFFFFu, (int)my_box < left && (unsigned)blk >= (unsigned)a.kv.n_blocks))
              kv_fail(MK_ERR_INVALID_ARG);
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          } else {
            // boxes that hold rows of the sequence (behind its end the keys' scores
            // are masked, whatever the stage still holds)
            const int used = min(PF_UNIT, (left + p.box - 1) / p.box * p.box);  // rows
            if (lane == 0) mbar_expect_tx(bar, (uint32_t)used * D * 2);
            __syncwarp();
            if ((int)my_box < used) {
              const int r = (row + (int)my_box) & in_block;
              long long y = ((long long)blk * a.kv.Hkv + w.h) * a.kv.block + r;
              if ((unsigned)blk >= (unsigned)a.kv.n_blocks) {
                kv_fail(MK_ERR_INVALID_ARG);
                y = (long long)a.kv.n_blocks * a.kv.Hkv * a.kv.block;  // outside: zeros
              }
#pragma unroll
              for (int c = 0; c < C; c++)
                tma_load_2d(dst + c * 16384 + my_box * 128, map, 64 * c, (int)y, bar, policy);
            }
            __syncwarp();
          }
          if (!is_v && j == w.ka) walk.next(p);  // while the copy runs
          if (!is_v && (n & 63) == 0 && lane == 0) pf_put_off(sh, sh.wait_ns);
        }
      }
      // The copies in flight, with a limit: nobody else may be waiting for them, since the
      // block can give up after this warp has issued its last.
      const unsigned long long t0 = gtimer();
      for (uint32_t i = n > NS ? n - NS : 0; i < n; i++)
        while (!mbar_try(smem_u32(&full[i % NS]), (i / NS) & 1) && gtimer() - t0 < PF_DRAIN_NS) {
        }
      for (int t = 0; t < 2; t++)  // (the queries' last load has q_empty's phase)
        while ((q_used >> t & 1) && !mbar_try(smem_u32(&sh.q_full[t]), q_phase >> t & 1) &&
               gtimer() - t0 < PF_DRAIN_NS) {
        }
    } else {
      // --------------------------------------------------------- products ----
      // (the whole warp takes every step, so that addresses stay in uniform
      // registers; one elected lane issues)
      const bool lead = elect_one();
      const uint32_t id_qk = idesc_bf16(128, 128) | (p.negate ? 1u << 13 : 0u);
      const uint32_t id_pv = idesc_bf16(128, D) | (1u << 16);
      const uint32_t q_desc = desc_lo(q_smem), k_desc = desc_lo(k_ring), v_desc = desc_lo_mn(v_ring);
      uint32_t ks = 0, kp = 0, vs = 0, vp = 0;  // stages and their phases
      // by tile, bit t: phases of s_free, p_half / p_full, q_full, o_empty; whether
      // an S, an O has been made
      uint32_t ph_s = 0, ph_p = 0, ph_q = 0, ph_o = 0, any_s = 0, any_o = 0;
      uint32_t taken = 0;  // records
      bool ok = true;
      PfRec w;
      auto wait = [&](const unsigned long long* bar, uint32_t phase) {
        ok = ok && __all_sync(0xFFFFFFFFu, pf_wait(sh, bar, phase));
      };
      auto wait_tile = [&](const unsigned long long* bars, uint32_t& phases, int t) {
        wait(&bars[t], (phases >> t) & 1);
        phases ^= 1u << t;
      };
      // S_t = Q_t K^T of the present key stage
      auto qk = [&](int t, bool last) {
        if (SEP) {
          if (any_s >> t & 1) wait_tile(sh.s_free, ph_s, t);
          any_s |= 1u << t;
        }
        if (!ok) return;
        tc_fence_after();
        const uint32_t ad = q_desc + t * (Sh::TILE >> 4), bd = k_desc + ks * (Sh::TILE >> 4);
        if (lead) {
#pragma unroll
          for (int s = 0; s < D / 16; s++)
            mma_ss(tmem + Sh::S_COL + 128 * t, ad + (s >> 2) * 1024 + (s & 3) * 2,
                   bd + (s >> 2) * 1024 + (s & 3) * 2, id_qk, s > 0);
          tc_commit(smem_u32(&sh.s_full[t]));
          if (last) tc_commit(smem_u32(&sh.q_empty[t]));
        }
        __syncwarp();
      };
      // O_t += P_t V of the present value stage (in halves as P comes, where S waits
      // for the place that P has)
      auto pv = [&](int t, bool first, bool last) {
        if (first) {
          if (any_o >> t & 1) wait_tile(sh.o_empty, ph_o, t);
          any_o |= 1u << t;
        }
        const uint32_t bd = v_desc + vs * (Sh::TILE >> 4);
        const uint32_t o_col = tmem + Sh::O_COL + D * t;
        const uint32_t p_col = tmem + (SEP ? Sh::P_COL + 64 * t : Sh::S_COL + 128 * t);
#pragma unroll
        for (int half = SEP ? 1 : 0; half < 2; half++) {
          wait(half == 0 ? &sh.p_half[t] : &sh.p_full[t], (ph_p >> t) & 1);
          if (!ok) return;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int s = SEP ? 0 : 4 * half; s < 4 * half + 4; s++)
              mma_ts(o_col, p_col + 8 * s, bd + s * 128, id_pv, !first || s > 0);
          }
          __syncwarp();
        }
        ph_p ^= 1u << t;
        if (lead && (SEP || last)) tc_commit(smem_u32(&sh.pv_done[t]));
        __syncwarp();
      };
      auto k_wait = [&]() { wait(&sh.k_full[ks], kp); };
      auto k_next = [&]() {
        if (ok && lead) tc_commit(smem_u32(&sh.k_empty[ks]));
        if (++ks == NS) { ks = 0; kp ^= 1; }
      };
      auto v_next = [&]() {
        if (ok && lead) tc_commit(smem_u32(&sh.v_empty[vs]));
        if (++vs == NS) { vs = 0; vp ^= 1; }
      };
      if (SEP) {
        // 64-dim heads, a warp per tile: the exponentials bound them, and neither
        // tile's softmax may wait for the other's
        // (the S of a unit, of the next job if need be, comes before the P of the one
        // before it)
        const int t = warp >> 1;
        auto s_of = [&](int j, int ka, int e) {
          if (j == ka && j < e) wait_tile(sh.q_full, ph_q, t);
          k_wait();
          if (j < e) qk(t, j + 1 == e);
          k_next();
        };
        // The next job and its first S.  One job only, though it may have no units:
        // the record behind it may have to wait for the products not yet issued.
        auto take = [&]() {
          const bool got = pf_take(sh, taken, w, lane == 0);
          if (got && w.ka < max(w.e[0], w.e[1])) s_of(w.ka, w.ka, t == 0 ? w.e[0] : w.e[1]);
          return got;
        };
        bool more = take();
        while (more && ok) {
          const int ka = w.ka, e = t == 0 ? w.e[0] : w.e[1], kb = max(w.e[0], w.e[1]);
          for (int j = ka; j < kb && ok; j++) {
            if (j + 1 < kb)
              s_of(j + 1, ka, e);
            else
              more = take();
            wait(&sh.v_full[vs], vp);
            if (j < e) pv(t, j == ka, j + 1 == e);
            v_next();
          }
          if (ka == kb) more = take();
        }
      } else if (warp == 1) {
        // 128-dim heads, one warp: the products bound them, and the tiles take turns
        while (ok && pf_take(sh, taken, w, lane == 0)) {
          const int ka = w.ka, e0 = w.e[0], e1 = w.e[1], kb = max(e0, e1);
          if (ka == kb) continue;
          k_wait();
          if (ka < e0) {
            wait_tile(sh.q_full, ph_q, 0);
            qk(0, ka + 1 == e0);
          }
          if (ka < e1) {
            wait_tile(sh.q_full, ph_q, 1);
            qk(1, ka + 1 == e1);
          }
          k_next();
          for (int j = ka; j < kb && ok; j++) {
            wait(&sh.v_full[vs], vp);
            if (j < e0) pv(0, j == ka, j + 1 == e0);
            if (j + 1 < kb) k_wait();
            if (j + 1 < e0) qk(0, j + 2 == e0);
            if (j < e1) pv(1, j == ka, j + 1 == e1);
            v_next();
            if (j + 1 < e1) qk(1, j + 2 == e1);
            if (j + 1 < kb) k_next();
          }
        }
      }
      // the products in flight still read shared and write tensor memory
      if (lead) tc_commit(smem_u32(&sh.drain));
      const unsigned long long t0 = gtimer();
      while (!mbar_try(smem_u32(&sh.drain), 0))
        if (gtimer() - t0 > PF_DRAIN_NS) {
          sh.abort = 1;
          break;
        }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ------------------------------------------------------------- softmax ----
    const int t = (warp - 4) >> 2;
    const int r = 32 * (warp & 3) + lane;  // row of the tile
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + lane_base + Sh::S_COL + 128 * t;
    const uint32_t o_addr = tmem + lane_base + Sh::O_COL + D * t;
    const uint32_t p_addr = SEP ? tmem + lane_base + Sh::P_COL + 64 * t : s_addr;
    const int row = 128 * t + r, row_token = t * p.per + r / a.G, row_head = r % a.G;
    uint32_t taken = 0, sp = 0, vp = 0;  // records; phases of s_full and pv_done
    bool ok = true;
    PfRec w;
    while (ok && pf_take(sh, taken, w, lane == 0)) {
      const int rows = t == 0 ? w.rows[0] : w.rows[1];
      const int ka = w.ka, kb = t == 0 ? w.e[0] : w.e[1];
      if (rows <= 0) continue;
      // the last cache row this row sees (rows that do not exist: every one)
      const int last = r < rows ? w.pos + row_token : 0x3FFFFFFF;
      float m = -INFINITY, l = 0.f;
      for (int j = ka; j < kb; j++) {
        ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.s_full[t], sp));
        if (!ok) break;
        sp ^= 1;
        tc_fence_after();
        const int limit = last - j * PF_UNIT;  // columns 0 .. limit count
        // A job's last units are masked in tensor memory, in a small loop: selects on
        // the registers of S cost every unit a tenth of its time, and a copy of the
        // unit for them costs every job its instruction fetches.
        if (__any_sync(0xFFFFFFFFu, limit < PF_UNIT - 1)) {
#pragma unroll 1
          for (int c = 0; c < PF_UNIT; c += 32) {
            if (!__any_sync(0xFFFFFFFFu, limit < c + 31)) continue;
            uint32_t y[32];
            tmem_ld32(s_addr + c, y);
#pragma unroll
            for (int i = 0; i < 32; i++)
              if (c + i > limit) y[i] = 0xFF800000u;  // -inf
            tmem_st32(s_addr + c, y);
          }
          tmem_st_wait();
        }
        uint32_t x[128];
        tmem_ld64(s_addr, x);
        // (the maximum of the first half while the second half comes)
        tmem_ld64_wait(x);
        tmem_ld64(s_addr + 64, x + 64);
        const float mx_a = max64(x);
        tmem_ld64_wait(x + 64);
        if (SEP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.s_free[t]));
        }
        const float mx = fmaxf(mx_a, max64(x + 64)) * p.scale2;
        const bool higher = mx > m + 8.f, raise = __any_sync(0xFFFFFFFFu, higher);
        // O and P are this thread's to write once the product before is done (where
        // P takes S's place, this S is the sign of it)
        if (SEP && j > ka) {
          ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.pv_done[t], vp));
          if (!ok) break;
          vp ^= 1;
          tc_fence_after();
        }
        if (raise) {
          // (each row by its own scores alone, so that no row's bits depend on another)
          const float f = higher ? join_weight(m, mx) : 1.f;
          if (higher) m = mx;
          l *= f;
          if (j > ka) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t y[32];
              tmem_ld32(o_addr + c, y);
#pragma unroll
              for (int i = 0; i < 32; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tmem_st32(o_addr + c, y);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 sc = make_float2(p.scale2, p.scale2), ng = make_float2(neg, neg);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; half++) {
          uint32_t y[32];
#pragma unroll
          for (int i = 0; i < 32; i++) {
            const int k = 64 * half + 2 * i;
            float2 e = ffma2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sc, ng);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[i & 1] = fadd2(sum[i & 1], e);
            y[i] = bf2(e.x, e.y);
          }
          tmem_st32(p_addr + 32 * half, y);
          if (SEP && half == 0) continue;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(half == 0 ? &sh.p_half[t] : &sh.p_full[t]));
        }
        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      }
      if (!ok) break;
      // -- the job's end: out = o / l, or a partial state
      if (kb > ka) {
        ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.pv_done[t], vp));
        if (!ok) break;
        vp ^= 1;
        tc_fence_after();
      }
      const bool mine = r < rows;
      const int hq = w.h * a.G + row_head;
      const long long tok = w.row + row_token;
      float* st = a.ws + ((size_t)blockIdx.x * 2 + w.slot) * Sh::STATE;
      uint16_t* out = (uint16_t*)a.o.p + tok * a.o.ts + hq * a.o.hs;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      constexpr int N = D == 64 ? 64 : 32;  // columns at a time (shorter code, 2 % of the whole)
      float bad = 0.f;
      if (kb > ka) {
#pragma unroll 1
        for (int c = 0; c < D; c += N) {
          uint32_t y[N];
          tmem_ldn<N>(o_addr + c, y);
          // (a sum is finite where all are, but for sums beyond the range: then the row is
          // redone for nothing)
          float2 b[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < N; i += 2)
            b[i >> 1 & 1] = fadd2(b[i >> 1 & 1], make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])));
          bad += ((b[0].x + b[1].x) + (b[0].y + b[1].y)) * 0.f;
          if (mine && w.whole) {
            const float2 f = make_float2(inv, inv), zero = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N; i += 8) {
              uint32_t z[4];
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const float2 v = ffma2(make_float2(__uint_as_float(y[i + 2 * e]),
                                                   __uint_as_float(y[i + 2 * e + 1])), f, zero);
                z[e] = bf2(v.x, v.y);
              }
              *(uint4*)(out + c + i) = make_uint4(z[0], z[1], z[2], z[3]);
            }
          } else if (mine) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
              *(uint4*)(st + ((size_t)(c + i) / 4 * PF_ROWS + row) * 4) =
                  make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.o_empty[t]));
      } else if (mine && w.whole) {
#pragma unroll 1
        for (int c = 0; c < D; c += 8) *(uint4*)(out + c) = make_uint4(0, 0, 0, 0);
      }
      if (mine) {
        if (w.whole) {
          if (a.lse) a.lse[tok * a.Hq + hq] = state_lse(m, l);
        } else {
          st[PF_ROWS * D + row] = m;
          st[PF_ROWS * D + PF_ROWS + row] = l;
        }
      }
      __syncwarp();
      unsigned redo = __ballot_sync(0xFFFFFFFFu, mine && !(bad == 0.f) && isfinite(l));
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        const int rr = __shfl_sync(0xFFFFFFFFu, row, src);
        const int end = __shfl_sync(0xFFFFFFFFu, last, src) + 1;
        const int hh = w.h * a.G + __shfl_sync(0xFFFFFFFFu, row_head, src);
        const long long row_tok = w.row + __shfl_sync(0xFFFFFFFFu, row_token, src);
        // (some 65 ns a cache row)
        if (lane == 0) pf_put_off(sh, sh.wait_ns + 1000ull * (unsigned)w.len);
        float m1, l1, o1[D / 32];
        attn_row<D>(a.kv, w.b, w.h, (const uint16_t*)a.q.p + row_tok * a.q.ts + hh * a.q.hs,
                    a.scale, ka * PF_UNIT, min(end, kb * PF_UNIT), m1, l1, o1);
        // a partial state keeps the row's m and l, which are sound
        const float f1 = w.whole ? (l1 == 0.f ? 0.f : 1.f / l1)
                                 : join_weight(m1 * LOG2E, __shfl_sync(0xFFFFFFFFu, m, src));
#pragma unroll
        for (int e = 0; e < D / 32; e++) {
          const int dim = lane * (D / 32) + e;
          if (w.whole)
            ((uint16_t*)a.o.p)[row_tok * a.o.ts + hh * a.o.hs + dim] = to_bf16(o1[e] * f1);
          else
            st[((size_t)(dim / 4) * PF_ROWS + rr) * 4 + dim % 4] = o1[e] * f1;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && sh.abort) kv_fail(MK_ERR_TIMEOUT);
}

// Block (x, y): if part x + 1 is the first to begin inside its job, joins rows
// [32 y, 32 y + 32) of that job's parts: the last job of part x, then the first
// jobs of the parts from x + 1 on that begin inside the same job.  A warp has 32
// rows, one per lane, and an eighth of the head's dimensions.
template <int D>
__global__ void __launch_bounds__(256, 4) kv_prefill_join_kernel(const __grid_constant__ PfArgs p, int blocks) {
  using Sh = PfShape<D>;
  constexpr int N = D / 32;  // float4 pieces per warp
  constexpr int F = 8 / N;   // states in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnArgs& a = p.a;
  const PfPart* parts = (const PfPart*)(a.ws + (size_t)blocks * 2 * Sh::STATE);
  const int i = blockIdx.x + 1;
  pdl_wait();
  const PfPart job = parts[i], prev = parts[i - 1];
  auto same = [&](const PfPart& x) { return x.b == job.b && x.h == job.h && x.j == job.j; };
  if (!job.inside || (prev.inside && same(prev))) return;
  const int row = 32 * blockIdx.y + lane, tile = row >> 7, r = row & 127;
  const bool live = r < job.rows[tile];
  if (r - lane >= job.rows[tile]) return;  // (the whole block)
  // The parts behind part i - 1, 32 at a time: how many begin inside the job, and
  // which of them hold anything.
  float m = -INFINITY, l = 0.f;
  float4 o[N];
#pragma unroll
  for (int c = 0; c < N; c++) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  // Joins the states of parts k0 + (bits of mask), the loads of F at a time in flight
  // (four blocks to an SM; with 128-dim heads twice the loads and half the blocks took
  // 4 us more); slot: of the first part's state.
  auto join = [&](int k0, unsigned mask, int slot) {
    while (mask) {
      float mi[F], li[F];
      float4 y[F][N];
#pragma unroll
      for (int n = 0; n < F; n++) {
        const bool in = mask != 0 && live;
        const int k = k0 + (mask ? __ffs(mask) - 1 : 0);
        mask &= mask - 1;
        const float* st = a.ws + ((size_t)k * 2 + slot) * Sh::STATE;
        mi[n] = in ? st[PF_ROWS * D + row] : -INFINITY;
        li[n] = in ? st[PF_ROWS * D + PF_ROWS + row] : 0.f;
#pragma unroll
        for (int c = 0; c < N; c++)
          y[n][c] = in ? *(const float4*)(st + ((size_t)(warp * N + c) * PF_ROWS + row) * 4)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int n = 0; n < F; n++) {
        if (li[n] == 0.f) continue;  // no weight; o was not written
        const float top = fmaxf(m, mi[n]), f = join_weight(m, top), g = join_weight(mi[n], top);
        m = top;
        l = l * f + li[n] * g;
#pragma unroll
        for (int c = 0; c < N; c++) {
          o[c].x = o[c].x * f + y[n][c].x * g;
          o[c].y = o[c].y * f + y[n][c].y * g;
          o[c].z = o[c].z * f + y[n][c].z * g;
          o[c].w = o[c].w * f + y[n][c].w * g;
        }
      }
    }
  };
  // (the job may be the first one of part i - 1, too)
  join(i - 1, 1u, prev.more && same(prev) ? 0 : 1);
  for (int k0 = i; k0 < blocks; k0 += 32) {
    PfPart x{};
    x.b = -1;
    if (k0 + lane < blocks) x = parts[k0 + lane];
    const unsigned ours = __ballot_sync(0xFFFFFFFFu, x.b >= 0 && x.inside && same(x));
    const unsigned more = __ballot_sync(0xFFFFFFFFu, x.more);
    const unsigned run = ours == 0xFFFFFFFFu ? ours : (1u << __ffs(~ours) - 1) - 1;  // up to the first that is not
    join(k0, run & more, 0);
    if (run != 0xFFFFFFFFu) break;
  }
  if (!live) return;
  const int hq = job.h * a.G + r % a.G;
  const long long tok = job.row + tile * p.per + r / a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* out = (uint16_t*)a.o.p + tok * a.o.ts + hq * a.o.hs + warp * N * 4;
#pragma unroll
  for (int c = 0; c < N; c++)
    *(uint2*)(out + 4 * c) = l == 0.f ? make_uint2(0, 0)
                                      : make_uint2(bf2(o[c].x * inv, o[c].y * inv),
                                                   bf2(o[c].z * inv, o[c].w * inv));
  if (a.lse && warp == 0) a.lse[tok * a.Hq + hq] = state_lse(m, l);
}

}  // namespace mk
