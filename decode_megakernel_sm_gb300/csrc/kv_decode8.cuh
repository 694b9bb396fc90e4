// kv_decode8.cuh -- decode attention over an 8-bit cache: the line of units of kv_decode.cuh
// with the rows through shared memory.
//
// Bound: the cache's bytes, 132 for a row's key and value of 64 dims, but only just: 16 rows are
// 2.1 KB, 90 cycles of an SM at the measured bandwidth, in which its four schedulers issue 360
// instructions at most, and making bf16 fragments of the codes takes 130.  So what the bf16
// kernel does for every load (an address, a predicate, registers that wait) is done for 32 rows
// at once here: a warp has a ring of stages of its own, four lanes start a bulk copy each of 32
// rows' codes and group bytes (where these are not whole 16 bytes, lanes copy them piece by
// piece), and all arrives on one barrier.  Loads into registers, as in the bf16 kernel, took 253 us
// for 32 sequences of 16384-32768 rows, 8 kv heads of 64; this takes 205, 4.2 TB/s, and 181 with 4
// heads of 128, 4.5 TB/s.  What bounds it now is the chain of dependent instructions: four warps to a
// scheduler issue in 0.6 of its cycles.  (Three blocks of more registers and deeper rings 229 where
// four took 219; five 206 where four took 202.)  (Weights as bf16 alone, without the
// remainder: 196 and 174, but twice the error where few of them count.)
//
// A warp waits for its own copies alone, for as long as the limit says (mk_kv_set_wait_timeout);
// then it goes on without them and without any more, the status word is set, and at the end it
// waits (with a limit again) for those in flight.  Most copies are there a step before: of a
// cache that L2 holds few calls wait 1 ns, of a larger one nearly all do somewhere.
#pragma once
#include "kv_decode.cuh"

namespace mk {

constexpr unsigned long long DEC8_DRAIN_NS = 2000000000ull;
// A try that waits may do so for 4 us (measured: 3.85 to 4.01, whatever hint of the time it is
// given), so shorter limits are kept by tries that do not wait.
constexpr unsigned long long DEC8_TRY_NS = 8192;

template <int D, int NT>
struct Dec8Shape {
  static constexpr int BLOCKS = D == 64 ? (NT == 1 ? 4 : 3) : 2;  // per SM
  static constexpr int STAGES = 2;  // per warp
  static constexpr int GROUPS = D / KV_GROUP, PER = 16 / GROUPS;  // rows of 16 group bytes
  static constexpr int PIECES = 32 / PER + 1;                     // of those, where they begin inside one
  static constexpr int KEYS = 0, VALUES = 32 * D, KEY_BYTES = 64 * D, VALUE_BYTES = KEY_BYTES + 16 * PIECES;
  static constexpr int STAGE = VALUE_BYTES + 16 * PIECES;
  static constexpr int SMEM = DEC_WARPS * STAGES * STAGE;
};

// Sixteen bytes of global memory to shared, of which the first `size` count (the others become 0).
MK_DEV void cp_async16_zfill_n(uint32_t dst, const void* src, int size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
// As mbar_try, without waiting.
MK_DEV bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for a phase's end; whether it came in time.  (A call: inside the step's code it took
// 207.3 us where this takes 205.3, 32 sequences of 16384-32768 rows, 8 kv heads of 64.)
__device__ __noinline__ bool dec8_wait(uint32_t bar, uint32_t phase, unsigned long long ns) {
  const unsigned long long t0 = gtimer();
  bool there;
  do {
    there = ns < DEC8_TRY_NS ? mbar_test(bar, phase) : mbar_try(bar, phase);
  } while (!there && gtimer() - t0 <= ns);
  return there;
}
// Arrives on the barrier once this thread's copies are there.
MK_DEV void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, Dec8Shape<D, NT>::BLOCKS)
kv_decode8_kernel(const __grid_constant__ AttnArgs a, unsigned long long wait_ns) {
  using Sh = DecShape<D, NT>;
  using Sh8 = Dec8Shape<D, NT>;
  constexpr int HB = Sh::HB, UNIT = DEC_UNIT<true>, STAGES = Sh8::STAGES;
  extern __shared__ __align__(128) unsigned char rings[];
  __shared__ DecShared<D, HB> sh;
  __shared__ alignas(8) unsigned long long full[DEC_WARPS][STAGES];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks_of_heads = (a.G + HB - 1) / HB, items = a.kv.Hkv * blocks_of_heads;
  const long long total = dec_total<UNIT>(a.kv, a.bt, lane) * items;
  const int parts = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= parts) return;
  const long long u0 = part_begin(total, parts, blockIdx.x), u1 = part_begin(total, parts, blockIdx.x + 1);
  const float scale2 = a.scale * LOG2E;
  if (threadIdx.x == 0) sh.redo = 0;
  unsigned char* ring = rings + warp * STAGES * Sh8::STAGE;
  if (lane == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(smem_u32(&full[warp][i]), 1 + 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  auto next = [&](DecPlace& p) {
    if (++p.unit < p.units) return;
    p.unit = 0;
    if (++p.item < items) return;
    p.item = 0;
    if (++p.b < a.bt.batch) {
      p.len = kv_len(a.kv, a.bt, p.b);
      p.units = dec_units<UNIT>(p.len);
    }
  };
  // The blocks of this warp's rows of a unit, first half and second (unchecked).
  const bool one = !a.kv.table || a.kv.block >= 32;  // of one block
  auto look = [&](const DecPlace& p, int (&blk)[2]) {
    const int j = p.unit * UNIT + 32 * warp;
    const int* table = a.kv.table + (size_t)p.b * a.kv.table_stride;
    blk[0] = blk[1] = p.b;
    if (a.kv.table && j < p.len) blk[0] = blk[1] = __ldg(table + (j >> a.kv.shift));
    if (!one && j + 16 < p.len) blk[1] = __ldg(table + (j + 16 >> a.kv.shift));
  };
  // What this lane copies of a whole unit: bytes of a row, from and to where.
  const int my_row = lane & 2 ? Sh8::GROUPS : D;
  const uint8_t* my_src = lane & 2 ? (lane & 1 ? a.kv.vs : a.kv.ks) : (const uint8_t*)(lane & 1 ? a.kv.v : a.kv.k);
  const uint32_t my_at = lane & 2 ? (lane & 1 ? Sh8::VALUE_BYTES : Sh8::KEY_BYTES) : lane & 1 ? Sh8::VALUES : Sh8::KEYS;
  // Starts the copies of a unit into stage s; whether there is anything in each half, as bits.
  const uint64_t policy = policy_evict_normal();
  bool gave_up = false;
  uint32_t pending = 0;  // stages with copies in flight
  auto fill = [&](const DecPlace& p, const int (&blk)[2], int s) -> uint32_t {
    const int j = p.unit * UNIT + 32 * warp, n = min(32, p.len - j);
    if (n <= 0 || gave_up) return 0;
    const bool bad0 = (unsigned)blk[0] >= (unsigned)a.kv.n_blocks, bad1 = (unsigned)blk[1] >= (unsigned)a.kv.n_blocks;
    const int n0 = bad0 ? 0 : min(n, 16), n1 = bad1 ? 0 : max(n - 16, 0);
    if (bad0 || (bad1 && n > 16)) kv_fail(MK_ERR_INVALID_ARG);
    if (n0 + n1 == 0) return 0;
    const int h = blocks_of_heads == 1 ? p.item : p.item / blocks_of_heads;  // (few need the division)
    const uint32_t bar = smem_u32(&full[warp][s]), dst = smem_u32(ring + s * Sh8::STAGE);
    const int mask = a.kv.table ? a.kv.block - 1 : 0x7FFFFFFF;
    const long long row0 = ((long long)blk[0] * a.kv.Hkv + h) * a.kv.block + (j & mask);
    const long long row1 = one ? row0 + 16 : ((long long)blk[1] * a.kv.Hkv + h) * a.kv.block + (j + 16 & mask);
    const int before = a.kv.table ? 0 : (int)(row0 & (Sh8::PER - 1));
    if (n == 32 && one && before == 0) {  // (most units) keys, values and their group bytes, a copy each
      if (lane == 0) mbar_expect_tx(bar, 64 * (D + Sh8::GROUPS));
      __syncwarp();
      if (lane < 4) bulk_g2s(dst + my_at, my_src + row0 * my_row, 32 * my_row, bar, policy);
      mbar_arrive(bar);
      pending |= 1u << s;
      return 3;
    }
    if (lane == 0) mbar_expect_tx(bar, 2 * D * (n0 + n1));
    __syncwarp();
    if (lane < 4) {  // keys and values, of both halves at once where they are neighbours
      const bool value = lane & 1, second = lane & 2;
      const int rows = second ? (one ? 0 : n1) : one ? n0 + n1 : n0;
      if (rows > 0)
        bulk_g2s(dst + (value ? Sh8::VALUES : Sh8::KEYS) + (second ? 16 * D : 0),
                 (const uint8_t*)(value ? a.kv.v : a.kv.k) + (second ? row1 : row0) * D, rows * D, bar, policy);
    }
    // group bytes, 16 at a time from such a boundary on (rows that do not exist: zeros)
    const int i = lane & 15, first = Sh8::PER * i - before;
    if (i < Sh8::PIECES) {
      const uint8_t* bytes = lane < 16 ? a.kv.ks : a.kv.vs;
      const long long row = first >= 16 ? row1 + first - 16 : row0 + first;
      const int size = (first >= 16 ? n1 : n0) > 0 ? min(max(n - first, 0), Sh8::PER) * Sh8::GROUPS : 0;
      cp_async16_zfill_n(dst + (lane < 16 ? Sh8::KEY_BYTES : Sh8::VALUE_BYTES) + 16 * i,
                         size > 0 ? bytes + row * Sh8::GROUPS : bytes, size);
    }
    cp_async_arrive(bar);
    pending |= 1u << s;
    return (n0 > 0 ? 1u : 0u) | (n1 > 0 ? 2u : 0u);
  };
  uint32_t phases = 0;  // by stage: of its barrier
  // Whether the stage's copies are there in time.
  auto wait = [&](int s, unsigned long long ns) {
    const uint32_t bar = smem_u32(&full[warp][s]), phase = phases >> s & 1;
    if (!__all_sync(0xFFFFFFFFu, mbar_test(bar, phase))) {
      const bool there = dec8_wait(bar, phase, ns);
      if (!__all_sync(0xFFFFFFFFu, there)) return false;
    }
    phases ^= 1u << s;
    pending &= ~(1u << s);
    return true;
  };

  // `ahead` is where the next fill is; its blocks are looked up a unit before.
  DecPlace p = dec_find<UNIT>(a.kv, a.bt, items, u0, lane), ahead = p;
  DecWarp<D, NT> w;
  int blk[2];
  look(ahead, blk);
  int filled = 0, todo = (int)(u1 - u0), fill_to = 0;  // units; the stage that is filled next
  uint32_t halves = 0;                                 // by stage: two bits
  auto fill_next = [&]() {
    halves = halves & ~(3u << 2 * fill_to) | fill(ahead, blk, fill_to) << 2 * fill_to;
    if (++fill_to == STAGES) fill_to = 0;
    if (++filled < todo) {
      next(ahead);
      look(ahead, blk);
    }
  };
  for (int i = 0; i < STAGES - 1 && i < todo; i++) fill_next();
  bool fresh = true, first = true;  // item: of the block
  int from = 0, s = 0;              // first unit of the item in this block; stage
  for (int i = 0; i < todo; i++) {
    if (fresh) {
      const int h = p.item / blocks_of_heads, hb = p.item % blocks_of_heads, head0 = h * a.G + hb * HB;
      w.init((const uint16_t*)a.q.p + p.b * a.q.ts + head0 * a.q.hs, a.q.hs, min(HB, a.G - hb * HB), lane);
      fresh = false;
      from = p.unit;
    }
    if (filled < todo) fill_next();
    const uint32_t both = halves >> 2 * s & 3;
    if (both && !gave_up && !wait(s, wait_ns)) gave_up = true;
    if (both && !gave_up) {
      const int j = p.unit * UNIT + 32 * warp, n = p.len - j;
      const unsigned head = (unsigned)p.b * a.kv.Hkv + (blocks_of_heads == 1 ? p.item : p.item / blocks_of_heads);
      const int before = a.kv.table ? 0 : (int)(head * a.kv.block & (Sh8::PER - 1));
      const unsigned char* stage = ring + s * Sh8::STAGE;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        if (!(both >> half & 1)) continue;
        DecRows8<D> rows;
        rows.read(stage + Sh8::KEYS + 16 * D * half, stage + Sh8::VALUES + 16 * D * half,
                  stage + Sh8::KEY_BYTES + Sh8::GROUPS * (16 * half + before),
                  stage + Sh8::VALUE_BYTES + Sh8::GROUPS * (16 * half + before), before, lane);
        w.step(rows, n - 16 * half, scale2, lane);
      }
    }
    if (p.unit == p.units - 1 || i == todo - 1) {  // the item's end, or this block's
      const int h = p.item / blocks_of_heads, hb = p.item % blocks_of_heads;
      dec_end_item<D, NT, true>(a, sh, w, p.b, h, h * a.G + hb * HB, min(HB, a.G - hb * HB),
                                from == 0 && p.unit == p.units - 1,
                                a.ws + ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * Sh::STATE, from * UNIT,
                                min(p.len, (p.unit + 1) * UNIT));
      fresh = true;
      first = false;
    }
    next(p);
    if (++s == STAGES) s = 0;
    __syncwarp();  // the stage may be filled again
  }
  if (gave_up) {
    if (lane == 0) kv_fail(MK_ERR_TIMEOUT);
    for (int i = 0; i < STAGES; i++)
      if (pending >> i & 1) wait(i, DEC8_DRAIN_NS);
  }
}

}  // namespace mk
