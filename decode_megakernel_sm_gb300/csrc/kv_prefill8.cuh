// kv_prefill8.cuh -- what the prefill attention has besides for an 8-bit cache
// (included by kv_prefill.cuh): the codes' way into the bf16 tiles.
//
// Warps 0 and 2 load codes into rings of their own (tiled TMA, the swizzle as wide as a row of
// codes), and four more warps make the tiles from them: 12 and 13 the keys', 14 and 15 the
// values', each half of a stage's rows.  A value is a bf16 number exactly, so from the tile on
// nothing is different, and no scale enters the softmax.  A lane takes 16 codes of a row, the
// eight lanes of a quarter warp eight rows, so that reads and writes hit eight bank groups, and
// reads some such before it works on them (one after the other took twice as long).  The group
// bytes come with the codes, by cp.async that arrives on the stage's barrier: a load of them would
// stall the loader, and in the warps that make tiles the fence that shows these to the tensor cores
// waits for loads in flight.  Rows from the sequence's end on become zeros.
//
// A fresh prompt's rows are read by every job behind them, and making their tiles anew for each
// costs the softmax warps time that they are short of (instructions fetched beside theirs).  So
// where there are many new tokens a kernel widens their rows first, into scratch as long as
// the new tokens, and units of such rows alone come from there, by TMA, as of a bf16 cache.
//
// Bound: as the bf16 cache's prefill where rows are widened (8192 tokens of 16/4 heads of 128 192 us,
// 0.75 of a measured GEMM's rate; a unit takes the bf16 kernel's time, the widening 5 us).  Few
// tokens over long caches wait for the tiles: 45 us for 4 x 5-16 tokens over 8000-20000 rows, where
// the bytes are 10 and the bf16 cache's kernel takes 33; a tile's two warps work 1300 cycles on a
// unit of 64-dim heads, and what is fetched for them slows the softmax beside.  So with a chunk
// over a long cache, whose old rows every job makes anew: 512 tokens over 16384 rows 84 us where
// the bf16 cache takes 73 (16/4 heads of 128: 72 and 59), 2048 tokens 283 and 236 (218 and 163).
#pragma once

namespace mk {

constexpr int PF8_THREADS = 512;
constexpr int PF8_REGS = 128;  // per thread at launch, dealt out anew: 128 x 88 + 256 x 184 + 128 x 56
constexpr int PF8_REGS_ISSUE = 88, PF8_REGS_SOFTMAX = 184, PF8_REGS_CONVERT = 56;
static_assert(128 * PF8_REGS_ISSUE + 256 * PF8_REGS_SOFTMAX + 128 * PF8_REGS_CONVERT <= PF8_THREADS * PF8_REGS,
              "the block would wait for registers that it does not hold");
// New tokens of a sequence times query heads per kv head, on average, from which on their rows are
// widened first.  In us, not widened and widened, heads of 64 (32/8) and of 128 (16/4): one prompt
// of 512 tokens 15.8 16.6, 18.6 18.3; of 1024 21.0 21.1, 25.6 23.6; of 2048 39.9 38.7, 41.3 38.2; eight of 512
// 36.0 35.1, 32.6 31.6; of 1024 82.8 74.2, 67.2 60.8; 512 tokens over 16384 rows 84.3 87.2, 72.3 75.1.
constexpr int PF8_WIDEN = 4096;
constexpr int PF8_PIECES = 17;  // of 16 group bytes: the rows of a stage, one more where they begin inside one

template <int D>
struct Pf8Shape {
  static constexpr int ROWS = D == 64 ? 128 : 64;    // of a stage of codes
  static constexpr int STAGE = ROWS * D;             // bytes
  static constexpr int STAGES = D == 64 ? 3 : 2;     // of keys, and as many of values
  static constexpr int PIECE = 16 / (D / KV_GROUP);  // rows of 16 group bytes
  static constexpr int SMEM = PfShape<D>::SMEM + 2 * STAGES * STAGE;
};

template <int D>
struct Pf8Shared {
  static constexpr int STAGES = Pf8Shape<D>::STAGES;
  alignas(8) unsigned long long full[2][STAGES], empty[2][STAGES];  // keys, values
  uint4 bytes[2][STAGES][PF8_PIECES];  // the rows' group bytes
  int fresh[PF_RECS];  // of a record's job: the first unit of new tokens' rows alone
};
static_assert(Pf8Shape<128>::SMEM + sizeof(Pf8Shared<128>) + sizeof(PfShared) <= 232448, "shared memory of a block");
static_assert(Pf8Shape<64>::SMEM + sizeof(Pf8Shared<64>) + sizeof(PfShared) <= 232448, "shared memory of a block");

template <bool INC, int N>
MK_DEV void pf8_registers() {
  if (INC)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

MK_DEV uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
MK_DEV uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
MK_DEV void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// How many rows before a stage's first one lie with it in 16 group bytes (a page begins at a
// multiple of 16 rows, a sequence in one piece anywhere; stages are multiples of 16 from there).
template <int D>
MK_DEV int pf8_before(const KvView& kv, const PfRec& w) {
  return kv.table ? 0 : (int)((unsigned)(w.b * kv.Hkv + w.h) * (unsigned)kv.block & (Pf8Shape<D>::PIECE - 1));
}

// Whether a unit is loaded whole: rows of new tokens alone, which are there as bf16.
MK_DEV bool pf8_whole(const PfArgs& p, const PfRec& w, int fresh, int unit) {
  return p.widened && unit >= fresh && (unit + 1) * PF_UNIT <= w.len;
}

// As pf_take.
template <int D>
MK_DEV bool pf8_take(PfShared& sh, const Pf8Shared<D>& sh8, uint32_t& n, PfRec& r, int& fresh, bool lead) {
  const int i = n % PF_RECS;
  if (!__all_sync(0xFFFFFFFFu, pf_wait(sh, &sh.rec_full[i], n / PF_RECS))) return false;
  fresh = ((const volatile int*)sh8.fresh)[i];
  __syncwarp();
  return pf_take(sh, n, r, lead);
}

// One warp makes its half (`odd`: the second) of every stage of the block's key (v: value) tiles.
template <int D>
MK_DEV void pf8_convert(const PfArgs& p, PfShared& sh, Pf8Shared<D>& sh8, int v, int odd, int lane, uint32_t codes,
                        uint32_t ring, unsigned long long* full, const unsigned long long* empty) {
  using Sh8 = Pf8Shape<D>;
  constexpr uint32_t NS = PfShape<D>::STAGES, TILE = PfShape<D>::TILE;
  // Pieces of 8 rows and 64 dims, N read before the first is worked on.  64-dim heads are bound by
  // the softmax warps, which lose by every instruction that is fetched beside theirs: a short loop
  // (eight prompts 118 us; unrolled 126).  128-dim heads wait for the tiles: unrolled (226; 247).
  constexpr int N = D == 64 ? 2 : 4, PIECES = Sh8::ROWS / 16 * (D / 64), UNROLL = D == 64 ? 1 : PIECES / N;
  const int r8 = lane & 7, c4 = lane >> 3;
  uint32_t taken = 0, n = 0, k = 0;  // records, tiles, stages of codes
  bool ok = true;
  PfRec w;
  int fresh;
  while (ok && pf8_take(sh, sh8, taken, w, fresh, lane == 0)) {
    const int kb = max(w.e[0], w.e[1]), before = pf8_before<D>(p.a.kv, w);
    for (int j = w.ka; j < kb && ok; j++) {
      const int left = w.len - j * PF_UNIT;
      const uint32_t st = n % NS;
      if (pf8_whole(p, w, fresh, j)) {
        n++;
        continue;
      }
      // (of widened rows the codes come when their tile is free)
      if (!p.widened && n >= NS) ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &empty[st], n / NS - 1));
      if (!ok) break;
      n++;
#pragma unroll 1
      for (int c = 0; c < PF_UNIT; c += Sh8::ROWS) {
        const bool some = c < left;  // (else zeros)
        const uint32_t cs = k % Sh8::STAGES;
        if (some) {
          ok = __all_sync(0xFFFFFFFFu, pf_wait(sh, &sh8.full[v][cs], k / Sh8::STAGES));
          if (!ok) break;
          k++;
        }
        const int half = odd * (Sh8::ROWS / 2);
        const uint32_t src = codes + cs * Sh8::STAGE, dst = ring + st * TILE + (c + half + r8) * 128;
        const uint32_t bytes = smem_u32(sh8.bytes[v][cs]) + (D / KV_GROUP) * before;
#pragma unroll UNROLL
        for (int i0 = 0; i0 < PIECES; i0 += N) {
          // piece i: 16 codes, chunk c16 of row r of the stage
          uint4 q[N];
          uint32_t e[N];
#pragma unroll
          for (int i = 0; i < N; i++) {
            const int r = half + 8 * ((i0 + i) / (D / 64)) + r8, c16 = 4 * ((i0 + i) % (D / 64)) + c4;
            q[i] = make_uint4(0, 0, 0, 0);
            e[i] = 0;
            if (some) {
              q[i] = lds128(src + r * D + ((D == 64 ? c16 ^ (r8 >> 1) : c16 ^ r8) << 4));
              e[i] = lds8(bytes + (D / KV_GROUP) * r + (c16 >> 1));
            }
          }
#pragma unroll
          for (int i = 0; i < N; i++) {
            const uint32_t scale = kv8_scale2(e[i]), k8 = 2 * c4;
            const uint32_t to = dst + 8 * ((i0 + i) / (D / 64)) * 128 + (i0 + i) % (D / 64) * 16384;
            sts128(to + ((k8 ^ r8) << 4), kv8_widen(q[i].x, q[i].y, scale));
            sts128(to + (((k8 + 1) ^ r8) << 4), kv8_widen(q[i].z, q[i].w, scale));
          }
        }
        if (some) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh8.empty[v][cs]));
        }
      }
      if (!ok) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full[st]));
    }
  }
}

}  // namespace mk
