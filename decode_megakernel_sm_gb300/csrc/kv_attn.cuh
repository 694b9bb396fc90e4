// kv_attn.cuh -- what the two attention operators share: their arguments, the
// partial states of a split row, and how partial states are joined.
//
// A partial state of a query row over some of its cache rows is (o, m, l):
// with x_j = scale * log2(e) * q.k_j, m at least about the largest x_j, l =
// sum 2^(x_j - m), o = sum 2^(x_j - m) v_j, all fp32.  States over disjoint
// ranges join by m = max m_i, l = sum l_i 2^(m_i - m), o likewise; the result
// is o / l and lse = (m + log2 l) ln 2.  An empty range has l = 0, m = -inf.
#pragma once
#include "kv_attn_row.cuh"

namespace mk {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct AttnArgs {
  KvView kv;
  KvBatch bt;
  Rows q, o;
  float* lse;
  float scale;
  int Hq, G;  // query heads; query heads per kv head
  float* ws;  // partial states
};

// 2^(m - top) for states that join under `top`; a state without weight
// (m = -inf) counts nothing, also where top is -inf itself.
MK_DEV float join_weight(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

MK_DEV float state_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * LN2; }

// Split of `total` units of work over `parts` blocks: block i's first unit.
MK_DEV long long part_begin(long long total, int parts, int i) { return total * i / parts; }

}  // namespace mk
