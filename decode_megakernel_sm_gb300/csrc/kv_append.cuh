// kv_append.cuh -- rotate the new tokens' queries and keys, write keys and
// values into the cache.
//
// Mathematics: with p the token's position and f_t = theta^(-2t/D) the pair
// (x_t, x_{t+D/2}) turns by the angle p f_t.  The angle is formed in whole
// turns as a 64-bit fraction: F_t = round(2^64 f_t / 2 pi) is made on the host
// and p * F_t mod 2^64 is the fraction of a turn, exact but for the rounding
// of F_t (p * 2^-54 turns, the double's last place), so far positions lose
// nothing and no table of positions is needed.  sincospif then evaluates the
// half-turns.
//
// Bound: bytes.  A token reads and writes (Hq + 2 Hkv) D elements once, in pieces of
// 16 elements: 8 of the lower and the matching 8 of the upper half of a head.  A
// block takes NT tokens: each warp finds one token's sequence and cache row, all
// threads make the tokens' cos/sin pairs, and then each thread keeps one token and
// one piece of the head, with its eight pairs in registers, and goes through every
// HL-th head, KV_APPEND_HEADS at a time with their loads in flight together.  (A
// thread per piece, which divides its index and reads its pairs for every head,
// took 28.7 us where this takes 24.6: 11198 tokens of 48 heads of 64, 69 MB read and
// 69 MB written, 21.7 us for a copy.)
#pragma once
#include "kv_common.cuh"

namespace mk {

constexpr int KV_APPEND_THREADS = 128;
constexpr int KV_APPEND_TOKENS = 4;  // per block, where there are enough tokens for all SMs
constexpr int KV_APPEND_HEADS = 3;

struct AppendArgs {
  KvView kv;
  KvBatch bt;
  Rows q, k, v, qo;
  int Hq;
  int rotate;
  unsigned long long freq[64];
};

// Eight consecutive elements as they are, and as floats.
template <bool F32>
struct Eight {
  uint4 w[F32 ? 2 : 1];
  MK_DEV void load(const void* base, long long off) {
    const uint4* p = F32 ? (const uint4*)((const float*)base + off) : (const uint4*)((const uint16_t*)base + off);
    w[0] = p[0];
    if (F32) w[F32 ? 1 : 0] = p[1];
  }
  MK_DEV void get(float (&f)[8]) const {
    if (F32) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const uint4& v = w[F32 ? i : 0];
        f[4 * i] = __uint_as_float(v.x);
        f[4 * i + 1] = __uint_as_float(v.y);
        f[4 * i + 2] = __uint_as_float(v.z);
        f[4 * i + 3] = __uint_as_float(v.w);
      }
    } else {
      unpack8(w[0], f);
    }
  }
};

MK_DEV void store8(uint16_t* p, const float (&f)[8]) {
  *(uint4*)p = make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
}

template <int D, bool F32, int NT>
__global__ void __launch_bounds__(KV_APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int HALF = D / 2, PIECES = D / 16, U = KV_APPEND_HEADS;
  constexpr int HL = KV_APPEND_THREADS / NT / PIECES;  // threads of a token's piece
  static_assert(NT <= KV_APPEND_THREADS / 32, "a warp looks up a token");
  __shared__ float2 cs[NT][HALF];  // (cos, sin)
  __shared__ int pos[NT];          // -1: nothing to do
  __shared__ long long row0[NT];   // pool row of kv head 0, or -1 (no page)
  const int t0 = blockIdx.x * NT, nt = min(NT, a.bt.n_tokens - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < nt) {
    const int t = t0 + warp;
    const int b = kv_seq_of_token(a.bt, t, lane);
    if (lane == 0) {
      int p = -1;
      long long r = -1;
      if (b < a.bt.batch) {
        int first, n;
        kv_new_tokens(a.bt, b, first, n);
        // (a row before the first sequence, or offsets that fall: no token of b)
        if (first <= t && t < first + n) p = kv_len(a.kv, a.bt, b) - (first + n - t);
        if (p >= 0) r = kv_row_of(a.kv, b, 0, p);
      }
      pos[warp] = p;
      row0[warp] = r;
    }
  }
  __syncthreads();
  if (a.rotate) {
    for (int i = threadIdx.x; i < nt * HALF; i += KV_APPEND_THREADS) {
      const int w = i / HALF, t = i % HALF;
      const long long turn = (long long)((unsigned long long)(unsigned)max(pos[w], 0) * a.freq[t]);
      float s, c;
      sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
      cs[w][t] = make_float2(c, s);
    }
    __syncthreads();
  }
  const int w = threadIdx.x / (HL * PIECES), t = threadIdx.x % PIECES * 8;
  if (w >= nt || pos[w] < 0) return;
  const long long token = t0 + w, row = row0[w];
  float2 z[8];
#pragma unroll
  for (int e = 0; e < 8; e++) z[e] = a.rotate ? cs[w][t + e] : make_float2(1.f, 0.f);
  const int heads = a.Hq + 2 * a.kv.Hkv;  // of q, then of k, then of v
  const int turning = a.rotate ? a.Hq + a.kv.Hkv : 0;
  for (int h0 = threadIdx.x / PIECES % HL; h0 < heads; h0 += HL * U) {
    Eight<F32> lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      int h = h0 + u * HL;
      if (h >= heads) break;
      const Rows* src = &a.q;
      if (h >= a.Hq) {
        h -= a.Hq;
        src = &a.k;
        if (h >= a.kv.Hkv) {
          h -= a.kv.Hkv;
          src = &a.v;
        }
      }
      const long long off = token * src->ts + h * src->hs + t;
      lo[u].load(src->p, off);
      hi[u].load(src->p, off + HALF);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      int h = h0 + u * HL;
      if (h >= heads) break;
      float f[8], g[8];
      lo[u].get(f);
      hi[u].get(g);
      uint16_t* dst = (uint16_t*)a.qo.p + token * a.qo.ts + h * a.qo.hs;
      const bool turn = h < turning;
      if (h >= a.Hq) {
        if (row < 0) continue;  // no page
        h -= a.Hq;
        const bool key = h < a.kv.Hkv;
        if (!key) h -= a.kv.Hkv;
        dst = (uint16_t*)(key ? a.kv.k : a.kv.v) + (row + (long long)h * a.kv.block) * D;
      }
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float c = f[e], d = g[e];
          f[e] = c * z[e].x - d * z[e].y;
          g[e] = d * z[e].x + c * z[e].y;
        }
      }
      store8(dst + t, f);
      store8(dst + HALF + t, g);
    }
  }
}

}  // namespace mk
