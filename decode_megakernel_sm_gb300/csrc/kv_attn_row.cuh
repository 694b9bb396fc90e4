// kv_attn_row.cuh -- attention of one query row over a range of cache rows by
// one warp, on the CUDA cores in fp32: every row of the cache outside the
// range stays unread, so nothing that a masked row holds can reach the result.
#pragma once
#include "kv_common.cuh"

namespace mk {

// Rows [j0, j1) of (sequence b, kv head h); q: this row's D elements.  Ends
// with the running maximum m (of scale * q.k, natural units; -inf for an
// empty range), the sum l relative to it and, on lane i, the unnormalised
// output's dims [i * D / 32, (i + 1) * D / 32).  All lanes call together.
template <int D>
MK_DEV void attn_row(const KvView& kv, int b, int h, const uint16_t* q, float scale, int j0, int j1,
                     float& m, float& l, float (&o)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; e++) o[e] = 0.f;
  for (int j = j0; j < j1; j += 32) {
    const int mine = j + lane;
    long long row = -1;
    if (mine < j1) row = kv_row_of(kv, b, h, mine);
    float s = -INFINITY;
    if (row >= 0) {
      const uint4* kr = (const uint4*)(kv.k + row * D);
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; c++) {
        float x[8], y[8];
        unpack8(__ldg(kr + c), x);
        unpack8(__ldg((const uint4*)q + c), y);
#pragma unroll
        for (int e = 0; e < 8; e++) acc = fmaf(x[e], y[e], acc);
      }
      s = acc * scale;
    }
    float mx = s;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
    const float mn = fmaxf(m, mx);
    const float old = m == mn ? 1.f : expf(m - mn);
    const float p = s == -INFINITY ? 0.f : expf(s - mn);  // (also where mn is -inf)
    m = mn;
    l = l * old + warp_sum(p);
#pragma unroll
    for (int e = 0; e < E; e++) o[e] *= old;
    for (int i = 0; i < min(32, j1 - j); i++) {
      const float pi = __shfl_sync(0xFFFFFFFFu, p, i);
      const long long ri = __shfl_sync(0xFFFFFFFFu, row, i);
      if (ri < 0) continue;
#pragma unroll
      for (int e = 0; e < E; e++) o[e] = fmaf(pi, bf1(kv.v[ri * D + lane * E + e]), o[e]);
    }
  }
}

}  // namespace mk
