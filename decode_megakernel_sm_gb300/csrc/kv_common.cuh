// kv_common.cuh -- what the KV-cache operators (append, decode attention,
// prefill attention) share on the device: the cache view, the batch
// description, and the status word their checks write.
#pragma once
#include "mk_device.cuh"

namespace mk {

// Programmatic dependent launch: a call's later kernels (those that join partial states,
// and the prefill behind the one that widens an 8-bit cache's rows for it) start while
// the one before still runs, and wait for all of its work before they read any.
// A call's first kernel starts plainly: on an idle stream, where a caller's every launch
// finds it, the early start costs 3 to 10 us more than it saves.
MK_DEV void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
MK_DEV void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What the operators found since mk_kv_status() last looked, as bits, and what it took.
constexpr int KV_FOUND_CONTENTS = 1, KV_FOUND_TIMEOUT = 2;
__device__ int kv_status_word = 0, kv_status_taken = 0;

MK_DEV void kv_fail(int code) {
  atomicOr(&kv_status_word, code == MK_ERR_TIMEOUT ? KV_FOUND_TIMEOUT : KV_FOUND_CONTENTS);
}

// Takes and clears in one step: kernels on other streams may add to the word meanwhile.
__global__ void kv_status_take() { kv_status_taken = atomicExch(&kv_status_word, 0); }

// Two floats rounded to bf16, the first in the low half.
MK_DEV uint32_t bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct KvView {
  const uint16_t* k;
  const uint16_t* v;
  const int* table;  // nullptr: sequence b is block b
  int table_stride;
  int n_blocks, Hkv, block;
  int shift;  // log2(block) with a table
  long long cap;  // rows a sequence can have: table_stride * block, or block
  const uint8_t* ks;  // 8-bit cache: the group bytes of the rows (k and v are codes)
  const uint8_t* vs;
};

struct KvBatch {
  const int* lens;
  const int* cu;  // nullptr: one new token per sequence
  int batch, n_tokens;
};

struct Rows {
  void* p;
  long long ts, hs;  // strides in elements
};

// Cache rows of sequence b, the new tokens' included; a length that the view
// cannot hold is cut to it and reported.
MK_DEV int kv_len(const KvView& kv, const KvBatch& bt, int b) {
  int n = __ldg(bt.lens + b);
  if (n < 0 || n > kv.cap) {
    kv_fail(MK_ERR_INVALID_ARG);
    n = n < 0 ? 0 : (int)kv.cap;
  }
  return n;
}

// Pool block of row p < kv.cap of sequence b, or -1 (reported) if the table
// names none.
MK_DEV int kv_block_of(const KvView& kv, int b, int p) {
  if (!kv.table) return b;
  const int blk = __ldg(kv.table + (size_t)b * kv.table_stride + (p >> kv.shift));
  if ((unsigned)blk >= (unsigned)kv.n_blocks) {
    kv_fail(MK_ERR_INVALID_ARG);
    return -1;
  }
  return blk;
}

// Pool row (in units of D elements) of row p of (sequence b, kv head h), or -1.
MK_DEV long long kv_row_of(const KvView& kv, int b, int h, int p) {
  const int blk = kv_block_of(kv, b, p);
  if (blk < 0) return -1;
  const int r = kv.table ? (p & (kv.block - 1)) : p;
  return ((long long)blk * kv.Hkv + h) * kv.block + r;
}

// First row of sequence b's new tokens in q / k / v / out, and their number;
// offsets that fall or leave the rows are cut to them and reported.
MK_DEV void kv_new_tokens(const KvBatch& bt, int b, int& first, int& n) {
  if (!bt.cu) {
    first = b;
    n = 1;
    return;
  }
  const int from = __ldg(bt.cu + b), to = __ldg(bt.cu + b + 1);
  if (from < 0 || to < from || to > bt.n_tokens) kv_fail(MK_ERR_INVALID_ARG);
  first = min(max(from, 0), bt.n_tokens);
  n = max(min(to, bt.n_tokens) - first, 0);
}

// Sequence that new token t belongs to (batch: none, a padding row), found by
// one warp: the number of sequences that end at or before t.  All lanes call.
// Reports offsets that fall or leave the rows, whichever sequence has them.
MK_DEV int kv_seq_of_token(const KvBatch& bt, int t, int lane) {
  if (!bt.cu) return t;
  int b = 0;
  bool bad = false;
  for (int i0 = 0; i0 < bt.batch; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < bt.batch;
    const int from = in ? __ldg(bt.cu + i) : 0, to = in ? __ldg(bt.cu + i + 1) : 0;
    bad |= from < 0 || to < from || to > bt.n_tokens;
    b += __popc(__ballot_sync(0xFFFFFFFFu, in && to <= t));
  }
  if (bad) kv_fail(MK_ERR_INVALID_ARG);
  return b;
}

}  // namespace mk
