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
// Bound: bytes.  A token reads and writes (Hq + 2 Hkv) D elements once.  A
// block takes KV_APPEND_TOKENS tokens: its first warps find each token's
// sequence and cache row, all threads make the cos/sin pairs of the tokens
// once (they serve every head), then each thread moves 16-element pieces: 8
// elements of the lower and the matching 8 of the upper half.
#pragma once
#include "kv_common.cuh"

namespace mk {

constexpr int KV_APPEND_THREADS = 256;
constexpr int KV_APPEND_TOKENS = 4;

struct AppendArgs {
  KvView kv;
  KvBatch bt;
  Rows q, k, v, qo;
  int Hq;
  int rotate;
  unsigned long long freq[64];
};

// Eight consecutive elements as floats.
template <bool F32>
MK_DEV void load8(const void* base, long long off, float (&f)[8]) {
  if (F32) {
    const float4* p = (const float4*)((const float*)base + off);
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(*(const uint4*)((const uint16_t*)base + off), f);
  }
}

MK_DEV void store8(uint16_t* p, const float (&f)[8]) {
  *(uint4*)p = make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
}

template <int D, bool F32>
__global__ void __launch_bounds__(KV_APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int HALF = D / 2, PIECES = D / 16, NT = KV_APPEND_TOKENS;
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
        const int after = a.bt.cu ? __ldg(a.bt.cu + b + 1) - t : 1;
        p = kv_len(a.kv, a.bt, b) - after;
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
  const int heads = a.Hq + 2 * a.kv.Hkv, per = heads * PIECES;
  for (int i = threadIdx.x; i < nt * per; i += KV_APPEND_THREADS) {
    const int w = i / per, j = i - w * per;
    if (pos[w] < 0) continue;
    const int head = j / PIECES, t = (j % PIECES) * 8;
    const bool is_q = head < a.Hq;
    const int h = is_q ? head : (head - a.Hq < a.kv.Hkv ? head - a.Hq : head - a.Hq - a.kv.Hkv);
    const bool is_v = head >= a.Hq + a.kv.Hkv;
    if (!is_q && row0[w] < 0) continue;
    const Rows& src = is_q ? a.q : is_v ? a.v : a.k;
    const long long off = (t0 + w) * src.ts + h * src.hs + t;
    float lo[8], hi[8];
    load8<F32>(src.p, off, lo);
    load8<F32>(src.p, off + HALF, hi);
    if (a.rotate && !is_v) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float2 z = cs[w][t + e];
        const float x = lo[e], y = hi[e];
        lo[e] = x * z.x - y * z.y;
        hi[e] = y * z.x + x * z.y;
      }
    }
    uint16_t* dst;
    if (is_q)
      dst = (uint16_t*)a.qo.p + (t0 + w) * a.qo.ts + h * a.qo.hs;
    else
      dst = (uint16_t*)(is_v ? a.kv.v : a.kv.k) + (row0[w] + (long long)h * a.kv.block) * D;
    store8(dst + t, lo);
    store8(dst + HALF + t, hi);
  }
}

}  // namespace mk
