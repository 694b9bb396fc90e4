// kv_ops.cu -- the KV-cache operators' entry points: checks of the arguments,
// choice of the kernel, launch.  No state, no allocation.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <limits>
#include <mutex>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "kv_append.cuh"
#include "kv_decode.cuh"
#include "kv_prefill.cuh"

namespace mk {

// A failed runtime call: its error is this call's status, and none of a later call.
static int cuda_failed() {
  cudaGetLastError();
  return MK_ERR_CUDA;
}
static int status_of(cudaError_t e) { return e == cudaSuccess ? MK_OK : cuda_failed(); }

// Streaming multiprocessors of the current device, 0 on an error.
static int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Launch a kernel; `early`: so that it may start while the one before it in the
// stream still runs, which it waits for itself (griddepcontrol.wait).
template <typename... P>
static cudaError_t launch(bool early, void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                          cudaStream_t s, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Four tokens to a block keep more loads in flight for one look-up (24.6 us against 33.9
// with one, 11198 tokens of 48 heads of 64); one token to a block starts sooner (3.1 us
// against 3.9 for a single token), so few tokens take that.
template <int D, bool F32>
static cudaError_t append_launch(const AppendArgs& a, int n_sm, cudaStream_t s) {
  constexpr int NT = KV_APPEND_TOKENS;
  const int n = a.bt.n_tokens;
  if (n <= NT * n_sm) return launch(false, kv_append_kernel<D, F32, 1>, dim3(n), KV_APPEND_THREADS, 0, s, a);
  return launch(false, kv_append_kernel<D, F32, NT>, dim3((n + NT - 1) / NT), KV_APPEND_THREADS, 0, s, a);
}

// Query heads of one item of the decode kernel: 8 fill half of a tensor-core
// tile and are enough for most group sizes; more share the cache's bytes.
static int decode_tiles(int G) { return G <= 8 ? 1 : 2; }

template <int D, int NT>
static size_t decode_ws(int n_sm) {
  using Sh = DecShape<D, NT>;
  return (size_t)n_sm * Sh::BLOCKS * 2 * Sh::STATE * sizeof(float);
}

template <int D, int NT, int W>
static cudaError_t join_launch(const AttnArgs& a, int grid, long long rows, cudaStream_t s) {
  constexpr int PER = JOIN_WARPS / W;
  return launch(true, kv_decode_join_kernel<D, NT, W>, dim3((unsigned)((rows + PER - 1) / PER)),
                32 * JOIN_WARPS, 0, s, a, grid);
}

// Blocks of the cluster that takes an item, or 0 where the line does: as many of 1, 2,
// 4, 8 as the SMs hold for all items (16 do not fit everywhere: 16 items of 128-dim
// heads took 10 us where 8 take 5), as long as the longest sequence that the cache can
// hold is 4 units for each.  A cluster is one launch and no search, but balances
// nothing.  Line and clusters, in us, 8 kv heads of 64: one sequence of 1024 rows 6.3
// and 4.8, of 2048 6.9 and 6.2, of 4096 8.1 and 8.5; 16 of 1024 12.9 and 9.7, one of
// 1024 among 15 of 64 6.8 and 7.0.  With 8 units 16 of 2048 would gain (19.1 and 15.1),
// one of 2048 among 15 of 64 would lose as much (7.6 and 11.3).  A caller that waits
// for each call saves 3 us more for the second launch.
static int cluster_size(long long items, int grid, long long cap) {
  int size = 1;
  if (items > grid) return 0;
  while (size < 8 && items * size * 2 <= grid) size *= 2;
  return cap <= 4ll * DEC_UNIT * size ? size : 0;
}

template <int D, int NT>
static cudaError_t cluster_launch(const AttnArgs& a, int items, int size, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(items * size);
  cfg.blockDim = dim3(DEC_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = size;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_decode_cluster_kernel<D, NT>, a);
}

template <int D, int NT>
static int decode_launch(const AttnArgs& a, int n_sm, cudaStream_t s) {
  using Sh = DecShape<D, NT>;
  const int grid = n_sm * Sh::BLOCKS;
  const long long rows = (long long)a.bt.batch * a.Hq;
  const long long items = (long long)a.bt.batch * a.kv.Hkv * ((a.G + Sh::HB - 1) / Sh::HB);
  if (const int size = cluster_size(items, grid, a.kv.cap))
    return status_of(cluster_launch<D, NT>(a, (int)items, size, s));
  if (rows > 0x7FFFFFFFll || items > 0x7FFFFFFFll / (a.kv.cap / DEC_UNIT + 1)) return MK_ERR_UNSUPPORTED;
  if (launch(false, kv_decode_kernel<D, NT>, dim3(grid), DEC_THREADS, 0, s, a) != cudaSuccess)
    return cuda_failed();
  // Warps per row of the join: where items are few, each is split into many states
  // (about grid / items): 8 items of 32768 rows 18.9 us with eight warps, 20.0 with
  // four; 256 items of 512-2048 rows 24.0 with eight, 21.3 with four.
  return status_of(items <= grid / 16 ? join_launch<D, NT, 8>(a, grid, rows, s)
                                      : join_launch<D, NT, 4>(a, grid, rows, s));
}

// The CUDA driver's tensor-map encoder, or nullptr.
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    PFN_cuTensorMapEncodeTiled_v12000 f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", (void**)&f, 12000,
                                         cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return f;
  }();
  return enc;
}

// Whether the kernel was compiled to the registers its warps deal out among
// themselves (fewer would leave them waiting), and may use its shared memory.
// Found once per device.
template <int D>
static bool prefill_ready() {
  static std::atomic<uint64_t> known{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (known.load(std::memory_order_relaxed) & bit) return true;
  cudaFuncAttributes at{};
  if (cudaFuncGetAttributes(&at, kv_prefill_kernel<D>) != cudaSuccess || at.numRegs != PF_REGS ||
      cudaFuncSetAttribute(kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           PfShape<D>::SMEM) != cudaSuccess)
    return false;
  known.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// How long a prefill block may get no further, in ns (mk_kv_set_wait_timeout).
constexpr uint64_t WAIT_NS = 2000000000ull;
static std::atomic<uint64_t> wait_ns{WAIT_NS};

template <int D>
static int prefill_launch(const AttnArgs& a, int n_sm, cudaStream_t s) {
  const auto enc = tensor_map_encoder();
  if (!enc || !prefill_ready<D>()) return cuda_failed();
  const long long rows = (long long)a.kv.n_blocks * a.kv.Hkv * a.kv.block;
  if (rows >= 0x7FFFFFFFll) return MK_ERR_UNSUPPORTED;
  PfArgs p{};
  p.a = a;
  p.per = PF_ROWS / 2 / a.G;
  p.negate = a.scale < 0.f;
  // (a scale of zero: the smallest number, which keeps masked scores at -inf and takes
  // finite ones to below 2^-20)
  p.scale2 = std::fmax(std::fabs(a.scale) * LOG2E, std::numeric_limits<float>::denorm_min());
  p.wait_ns = wait_ns.load(std::memory_order_relaxed);
  p.box = a.kv.table && a.kv.block < PF_UNIT ? a.kv.block : PF_UNIT;
  CUtensorMap maps[3];
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)p.box}, es[2] = {1, 1};
  for (int i = 0; i < 2; i++)
    if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)(i == 0 ? a.kv.k : a.kv.v), dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MK_ERR_CUDA;
  // queries: [token][head][D], boxes of a tile's tokens and one kv head's heads
  const cuuint64_t qdims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.bt.n_tokens};
  const cuuint64_t qstrides[2] = {(cuuint64_t)(a.q.hs * 2), (cuuint64_t)(a.q.ts * 2)};
  const cuuint32_t qbox[3] = {64, (cuuint32_t)a.G, (cuuint32_t)p.per}, qes[3] = {1, 1, 1};
  if (enc(&maps[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q.p, qdims, qstrides, qbox, qes,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MK_ERR_CUDA;
  if (launch(false, kv_prefill_kernel<D>, dim3(n_sm), PF_THREADS, PfShape<D>::SMEM, s, p, maps[0],
             maps[1], maps[2]) != cudaSuccess ||
      (n_sm > 1 && launch(true, kv_prefill_join_kernel<D>, dim3(n_sm - 1, PF_ROWS / 32), 256, 0, s, p,
                          n_sm) != cudaSuccess))
    return cuda_failed();
  return MK_OK;
}

// ------------------------------------------------------- argument checks ----
static bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Rows of D elements of `size` bytes, each on a 16-byte boundary.
static bool rows_ok(const mk_rows* r, size_t size) {
  return r && r->p && aligned(r->p, 16) && (r->token_stride * (long)size) % 16 == 0 &&
         (r->head_stride * (long)size) % 16 == 0;
}

// Rows that are written: no two of the [n][heads] overlap (the strides nest).
static bool out_ok(const mk_rows* r, int n, int heads, int D) {
  if (!rows_ok(r, 2)) return false;
  const long long ts = std::llabs(r->token_stride), hs = std::llabs(r->head_stride);
  if (n == 1 || heads == 1) return (n == 1 || ts >= D) && (heads == 1 || hs >= D);
  return ts > hs ? hs >= D && ts >= hs * (heads - 1) + D : ts >= D && hs >= ts * (n - 1) + D;
}

// Where rows lie in memory, in bytes: n[0] x n[1] pieces of `size`, step[i] apart
// (tokens, heads; steps that are not negative, none where there is one piece).
using wide = __int128;
struct Place {
  wide at, size, n[2], step[2];
  wide end() const { return at + (n[0] - 1) * step[0] + (n[1] - 1) * step[1] + size; }
};

static Place place(const void* p, wide bytes) { return {(wide)(uintptr_t)p, bytes, {1, 1}, {0, 0}}; }

static Place place(const mk_rows* r, int n, int heads, int D, size_t size) {
  Place x{(wide)(uintptr_t)r->p, (wide)D * size, {n, heads}, {r->token_stride, r->head_stride}};
  for (int i = 0; i < 2; i++) {
    x.step[i] *= size;
    if (x.step[i] < 0) {
      x.at += (x.n[i] - 1) * x.step[i];
      x.step[i] = -x.step[i];
    }
    if (x.n[i] == 1 || x.step[i] == 0) {
      x.n[i] = 1;
      x.step[i] = 0;
    }
  }
  return x;
}

// Whether [a, a + na) and [b, b + nb) are disjoint, all their shifts by the period too.
static bool apart(wide a, wide na, wide b, wide nb, wide period) {
  wide d = (b - a) % period;
  if (d < 0) d += period;
  return d >= na && d + nb <= period;
}

// Whether two places share no byte: one lies before the other, or both repeat with one
// period (slices of one wider row) and their parts of it are apart, as wholes or, by
// tokens, head by head.  False where that does not show it.
static bool disjoint(const Place& x, const Place& y) {
  if (x.end() <= y.at || y.end() <= x.at) return true;
  for (int i = 0; i < 2; i++) {
    const wide period = x.n[i] == 1 ? y.step[i] : x.step[i];
    if (period == 0 || (x.n[i] > 1 && y.n[i] > 1 && x.step[i] != y.step[i])) continue;
    const int o = 1 - i;
    if (apart(x.at, (x.n[o] - 1) * x.step[o] + x.size, y.at, (y.n[o] - 1) * y.step[o] + y.size, period))
      return true;
    if (i == 1 || x.n[1] * y.n[1] > 1 << 14) continue;
    bool all = true;
    for (int j = 0; all && j < x.n[1]; j++)
      for (int k = 0; all && k < y.n[1]; k++)
        all = apart(x.at + j * x.step[1], x.size, y.at + k * y.step[1], y.size, period);
    if (all) return true;
  }
  return false;
}

static bool same(const Place& x, const Place& y) {
  return x.at == y.at && x.size == y.size && x.n[0] == y.n[0] && x.n[1] == y.n[1] &&
         x.step[0] == y.step[0] && x.step[1] == y.step[1];
}

static Place pool(const mk_kv_view* kv, const void* p) {
  return place(p, (wide)kv->n_blocks * kv->n_kv_heads * kv->block * kv->head_dim * 2);
}

static Rows rows(const mk_rows* r) { return Rows{r->p, r->token_stride, r->head_stride}; }

// Fills the device structs; MK_OK, or why not.
static int check(const mk_kv_view* kv, const mk_kv_batch* bt, KvView& v, KvBatch& b) {
  if (!kv || !bt) return MK_ERR_INVALID_ARG;
  if (!kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16) || kv->n_blocks < 1 ||
      kv->n_kv_heads < 1 || kv->block < 1)
    return MK_ERR_INVALID_ARG;
  if (bt->batch < 0 || bt->n_tokens < 0 || (bt->batch > 0 && !bt->d_lens) ||
      (!bt->d_cu && bt->n_tokens != bt->batch) || !aligned(bt->d_lens, 4) || !aligned(bt->d_cu, 4) ||
      !aligned(kv->d_table, 4))
    return MK_ERR_INVALID_ARG;
  int shift = 0;
  if (kv->d_table) {
    if (kv->block < 16 || kv->block > 4096 || (kv->block & (kv->block - 1)) || kv->table_stride < 1)
      return MK_ERR_INVALID_ARG;
    while ((1 << shift) < kv->block) shift++;
  } else if (kv->n_blocks < bt->batch) {
    return MK_ERR_INVALID_ARG;
  }
  if (kv->head_dim != 64 && kv->head_dim != 128) return MK_ERR_UNSUPPORTED;
  v = KvView{(const uint16_t*)kv->k, (const uint16_t*)kv->v, kv->d_table, kv->table_stride,
             kv->n_blocks, kv->n_kv_heads, kv->block, shift,
             std::min(kv->d_table ? (long long)kv->table_stride * kv->block : (long long)kv->block,
                      0x7FFFF000ll)};  // (a length may be rounded up to units)
  b = KvBatch{bt->d_lens, bt->d_cu, bt->batch, bt->n_tokens};
  return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" int mk_kv_append(const mk_kv_view* kv, const mk_kv_batch* bt, int n_q_heads,
                            const mk_rows* q, const mk_rows* k, const mk_rows* v, int src_type,
                            const mk_rows* q_out, double rope_theta, void* stream) {
  AppendArgs a;
  const int rc = check(kv, bt, a.kv, a.bt);
  if (rc) return rc;
  if (src_type != MK_SRC_BF16 && src_type != MK_SRC_F32) return MK_ERR_INVALID_ARG;
  const size_t size = src_type == MK_SRC_F32 ? 4 : 2;
  if (n_q_heads < 0 || !(rope_theta == 0.0 || (rope_theta >= 1.0 && rope_theta <= 1e30)))
    return MK_ERR_INVALID_ARG;
  if (bt->n_tokens == 0 || bt->batch == 0) return MK_OK;
  if (!rows_ok(k, size) || !rows_ok(v, size) ||
      (n_q_heads > 0 && (!rows_ok(q, size) || !out_ok(q_out, bt->n_tokens, n_q_heads, kv->head_dim))))
    return MK_ERR_INVALID_ARG;
  // What is written may not be read or written by another thread's piece: queries turn
  // in place (a thread reads its pieces before it writes them) or go elsewhere.
  const int n = bt->n_tokens, D = kv->head_dim;
  const Place kp = pool(kv, kv->k), vp = pool(kv, kv->v);
  if (!disjoint(kp, vp)) return MK_ERR_INVALID_ARG;
  if (n_q_heads > 0) {
    const Place to = place(q_out, n, n_q_heads, D, 2), from = place(q, n, n_q_heads, D, size);
    if (!(same(to, from) || disjoint(to, from)) || !disjoint(to, place(k, n, kv->n_kv_heads, D, size)) ||
        !disjoint(to, place(v, n, kv->n_kv_heads, D, size)) || !disjoint(to, kp) || !disjoint(to, vp))
      return MK_ERR_INVALID_ARG;
  }
  a.k = rows(k);
  a.v = rows(v);
  if (n_q_heads > 0) {
    a.q = rows(q);
    a.qo = rows(q_out);
  } else {
    a.q = a.qo = Rows{};
  }
  a.Hq = n_q_heads;
  a.rotate = rope_theta != 0.0;
  if (a.rotate) {
    // theta^(-2t/D) / 2 pi as a fraction of 2^64, from the powers of two of t
    double pw[6];
    for (int i = 0; i < 6; i++) pw[i] = std::pow(rope_theta, -2.0 * (1 << i) / D);
    for (int t = 0; t < D / 2; t++) {
      double f = 0.15915494309189533577;  // 1 / 2 pi
      for (int i = 0; i < 6; i++)
        if (t & (1 << i)) f *= pw[i];
      a.freq[t] = (unsigned long long)std::ldexp(f, 64);
    }
  }
  const int n_sm = sm_count();
  if (n_sm == 0) return cuda_failed();
  cudaStream_t s = (cudaStream_t)stream;
  if (D == 64) return status_of(size == 4 ? append_launch<64, true>(a, n_sm, s) : append_launch<64, false>(a, n_sm, s));
  return status_of(size == 4 ? append_launch<128, true>(a, n_sm, s) : append_launch<128, false>(a, n_sm, s));
}

extern "C" int mk_attn_workspace_bytes(int decode, int n_tokens, int batch, int n_q_heads,
                                       int n_kv_heads, int head_dim, size_t* bytes) {
  if (!bytes || decode < 0 || decode > 1 || n_tokens < 0 || batch < 0 || n_q_heads < 1 ||
      n_kv_heads < 1 || n_q_heads % n_kv_heads)
    return MK_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MK_ERR_UNSUPPORTED;
  *bytes = 0;
  const int n = sm_count(), nt = decode_tiles(n_q_heads / n_kv_heads);
  if (n == 0) return cuda_failed();
  if (!decode) {
    *bytes = ((head_dim == 64 ? PfShape<64>::STATE : PfShape<128>::STATE) * sizeof(float) * 2 +
              sizeof(PfPart)) * n;
  } else {
    *bytes = head_dim == 64 ? (nt == 1 ? decode_ws<64, 1>(n) : decode_ws<64, 2>(n))
                            : (nt == 1 ? decode_ws<128, 1>(n) : decode_ws<128, 2>(n));
  }
  return MK_OK;
}

static int attention(bool decode, const mk_kv_view* kv, const mk_kv_batch* bt, int n_q_heads,
                     const mk_rows* q, float scale, const mk_rows* out, float* d_lse, void* d_ws,
                     size_t ws_bytes, void* stream) {
  AttnArgs a;
  const int rc = check(kv, bt, a.kv, a.bt);
  if (rc) return rc;
  if ((bt->d_cu != nullptr) == decode) return MK_ERR_INVALID_ARG;
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads) return MK_ERR_INVALID_ARG;
  if (bt->n_tokens == 0 || bt->batch == 0) return MK_OK;
  if (!std::isfinite(scale * LOG2E) || !rows_ok(q, 2) ||
      !out_ok(out, bt->n_tokens, n_q_heads, kv->head_dim) || (d_lse && !aligned(d_lse, 4)))
    return MK_ERR_INVALID_ARG;
  // other blocks, and rows that are redone, read q and the cache after out is written
  const Place to = place(out, bt->n_tokens, n_q_heads, kv->head_dim, 2),
              from = place(q, bt->n_tokens, n_q_heads, kv->head_dim, 2),
              lse = place(d_lse, d_lse ? (wide)bt->n_tokens * n_q_heads * 4 : 0);
  const Place kp = pool(kv, kv->k), vp = pool(kv, kv->v);
  if (!disjoint(to, from) || !disjoint(to, kp) || !disjoint(to, vp)) return MK_ERR_INVALID_ARG;
  if (d_lse && !(disjoint(lse, from) && disjoint(lse, to) && disjoint(lse, kp) && disjoint(lse, vp)))
    return MK_ERR_INVALID_ARG;
  size_t need = 0;
  const int wrc = mk_attn_workspace_bytes(decode, bt->n_tokens, bt->batch, n_q_heads,
                                          kv->n_kv_heads, kv->head_dim, &need);
  if (wrc) return wrc;
  if (need > 0) {
    if (!d_ws || !aligned(d_ws, 256) || ws_bytes < need) return MK_ERR_INVALID_ARG;
    const Place ws = place(d_ws, need);
    if (!(disjoint(ws, from) && disjoint(ws, to) && disjoint(ws, kp) && disjoint(ws, vp)) ||
        (d_lse && !disjoint(ws, lse)))
      return MK_ERR_INVALID_ARG;
  }
  a.q = rows(q);
  a.o = rows(out);
  a.lse = d_lse;
  a.scale = scale;
  a.Hq = n_q_heads;
  a.G = n_q_heads / kv->n_kv_heads;
  a.ws = (float*)d_ws;
  const int n = sm_count(), nt = decode_tiles(a.G);
  cudaStream_t s = (cudaStream_t)stream;
  if (!decode) {
    if (a.G > PF_ROWS / 2) return MK_ERR_UNSUPPORTED;
    return kv->head_dim == 64 ? prefill_launch<64>(a, n, s) : prefill_launch<128>(a, n, s);
  }
  if (kv->head_dim == 64)
    return nt == 1 ? decode_launch<64, 1>(a, n, s) : decode_launch<64, 2>(a, n, s);
  return nt == 1 ? decode_launch<128, 1>(a, n, s) : decode_launch<128, 2>(a, n, s);
}

extern "C" int mk_attn_decode(const mk_kv_view* kv, const mk_kv_batch* bt, int n_q_heads,
                              const mk_rows* q, float scale, const mk_rows* out, float* d_lse,
                              void* d_ws, size_t ws_bytes, void* stream) {
  return attention(true, kv, bt, n_q_heads, q, scale, out, d_lse, d_ws, ws_bytes, stream);
}

extern "C" int mk_attn_prefill(const mk_kv_view* kv, const mk_kv_batch* bt, int n_q_heads,
                               const mk_rows* q, float scale, const mk_rows* out, float* d_lse,
                               void* d_ws, size_t ws_bytes, void* stream) {
  return attention(false, kv, bt, n_q_heads, q, scale, out, d_lse, d_ws, ws_bytes, stream);
}

extern "C" int mk_kv_set_wait_timeout(uint64_t ns) {
  if (ns > 1ull << 62) return MK_ERR_INVALID_ARG;  // (a limit is a time of the clock, in 64 bits)
  wait_ns.store(ns == 0 ? WAIT_NS : ns, std::memory_order_relaxed);
  return MK_OK;
}

extern "C" int mk_kv_status(void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  // (the caller's work outside the lock: it may take long, or wait for another thread)
  if (cudaStreamSynchronize(s) != cudaSuccess) return cuda_failed();
  static std::mutex one_at_a_time;  // kv_status_taken is one per device
  std::lock_guard<std::mutex> guard(one_at_a_time);
  int found = 0;
  if (launch(false, kv_status_take, dim3(1), 1, 0, s) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&found, kv_status_taken, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return cuda_failed();
  return found & KV_FOUND_TIMEOUT ? MK_ERR_TIMEOUT : found ? MK_ERR_INVALID_ARG : MK_OK;
}
