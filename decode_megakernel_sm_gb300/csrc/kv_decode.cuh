// kv_decode.cuh -- attention of one new token per sequence over its cache rows,
// split over the length and joined.
//
// Bound: the cache's bytes, each read once (query heads that share a kv head
// are one work item, up to 8 NT of them).  So the split is over bytes, not
// over sequences: the units (64 cache rows of one item) of the whole batch
// form one line, every block takes an equal piece of it, and a second kernel
// joins the states of items that more than one block has a part of.  Lengths
// are read on the device, so one captured graph serves growing sequences.
// Caches that can only hold little take a cluster of blocks per item instead, in
// one launch.  32 sequences of 16384-32768 rows, 8 kv heads of 64 (1.56 GB): 241.6 us,
// 6.48 TB/s; one of 1024 rows 5.0 us (clusters; 6.3 by the line).
//
// A block has four warps; a warp takes 16 rows of a unit straight from global
// memory into registers in the tensor cores' fragment layout, the next unit's
// loads issued before the current one is computed (no shared memory, no
// barrier inside an item):
//   S[heads x 16 rows] = Q K^T   mma.m16n8k16.  Which head dimension sits at
//     which k index is free as long as Q and K agree: lane 4r + c takes 16-byte
//     chunks c, c + 4, .. of row r's key, so a load touches whole sectors.
//   O^T[dims x heads] += V^T P^T  The S accumulator of head r, rows 2c, 2c + 1
//     is the B operand as it stands; lane 4r + c loads chunk r of its four rows
//     2c, 2c + 1, 2c + 8, 2c + 9, and one byte permute per register pairs rows.
// The weights enter the second product as bf16 high part and remainder (16
// mantissa bits; the tensor cores have time to spare here), sums and maxima
// stay fp32.  A running maximum is raised only when a score passes it by 2^8.
// A remainder of 0 times an infinite value would be NaN: heads whose result is
// not finite although their weights are, are redone by attn_row.
#pragma once
#include "kv_attn.cuh"

namespace mk {

constexpr int DEC_WARPS = 4, DEC_THREADS = 32 * DEC_WARPS;
constexpr int DEC_UNIT = 16 * DEC_WARPS;  // cache rows per unit

template <int D, int NT>
struct DecShape {
  static constexpr int HB = 8 * NT;                          // heads per item
  static constexpr int BLOCKS = D == 64 ? (NT == 1 ? 4 : 3) : 2;  // per SM (registers)
  static constexpr int STATE = HB * (D + 2);                 // floats of one partial state
};

// Where a block is in the line of units.
struct DecPlace {
  int b, len, units;  // sequence, its rows and units (one where it has no rows)
  int item, unit;     // item of the sequence (kv head, head block), unit of it
};

MK_DEV int dec_units(int len) { return max(1, (len + DEC_UNIT - 1) / DEC_UNIT); }

// Units of the whole batch, one item per sequence (one warp, all lanes).
MK_DEV long long dec_total(const KvView& kv, const KvBatch& bt, int lane) {
  long long n = 0;
  for (int b = lane; b < bt.batch; b += 32) n += dec_units(kv_len(kv, bt, b));
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, w);
  return n;
}

// The place of unit u of the line (one warp, all lanes).
MK_DEV DecPlace dec_find(const KvView& kv, const KvBatch& bt, int items, long long u, int lane) {
  long long before = 0;
  DecPlace p{};
  for (int b0 = 0; b0 < bt.batch; b0 += 32) {
    const int b = b0 + lane;
    const int len = b < bt.batch ? kv_len(kv, bt, b) : 0;
    const int n = b < bt.batch ? dec_units(len) : 0;
    int incl = n;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, w);
      if (lane >= w) incl += y;
    }
    const bool past = (before + incl) * items > u;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, past && n > 0);
    if (hit) {
      const int src = __ffs(hit) - 1;
      p.b = b0 + src;
      p.len = __shfl_sync(0xFFFFFFFFu, len, src);
      p.units = __shfl_sync(0xFFFFFFFFu, n, src);
      const long long rem = u - (before + __shfl_sync(0xFFFFFFFFu, incl - n, src)) * items;
      p.item = (int)(rem / p.units);
      p.unit = (int)(rem % p.units);
      return p;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return p;  // not reached for u < total * items
}

MK_DEV uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

MK_DEV uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// One warp's 16 rows of a unit in registers.
template <int D>
struct DecRows {
  static constexpr int C = D / 64;
  uint4 k[2][2 * C];  // key of row 8t + r: chunks c, c + 4, ..
  uint4 v[4][C];      // values of rows 2c, 2c + 1, 2c + 8, 2c + 9: chunks r, r + 8

  // row0: pool row of the first of the 16 rows (-1: none to read); n: how many exist.
  MK_DEV void load(const KvView& kv, long long row0, int n, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const bool in = row0 >= 0 && 8 * t + r < n;
      const uint4* p = (const uint4*)(kv.k + (row0 + 8 * t + r) * D) + c;
#pragma unroll
      for (int i = 0; i < 2 * C; i++) k[t][i] = in ? ldg_stream(p + 4 * i) : zero;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int row = 2 * c + (j & 1) + 8 * (j >> 1);
      const bool in = row0 >= 0 && row < n;
      const uint4* p = (const uint4*)(kv.v + (row0 + row) * D) + r;
#pragma unroll
      for (int i = 0; i < C; i++) v[j][i] = in ? ldg_stream(p + 8 * i) : zero;
    }
  }
};

template <int D, int NT>
struct DecWarp {
  static constexpr int C = D / 64, S = D / 16;
  uint32_t q[S][2 * NT];  // A fragments (NT 1: rows 8..15 are zero)
  float m[NT], l[NT];     // of head r (+ 8); l: this lane's share
  float o[S][NT][4];      // O^T: tile i, head tile n

  // q0: the item's first query head's row; n_heads of them.
  MK_DEV void init(const uint16_t* q0, long long hs, int n_heads, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; n++) {
      m[n] = -INFINITY;
      l[n] = 0.f;
      const bool in = 8 * n + r < n_heads;
      const uint4* p = (const uint4*)(q0 + (8 * n + r) * hs) + c;
#pragma unroll
      for (int i = 0; i < 2 * C; i++) {
        const uint4 w = in ? __ldg(p + 4 * i) : make_uint4(0, 0, 0, 0);
        q[2 * i][n] = w.x;
        q[2 * i][NT + n] = w.y;
        q[2 * i + 1][n] = w.z;
        q[2 * i + 1][NT + n] = w.w;
      }
    }
#pragma unroll
    for (int i = 0; i < S; i++)
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[i][n][e] = 0.f;
  }

  // 16 rows, of which the first nv count.
  MK_DEV void step(const DecRows<D>& kv, int nv, float scale2, int lane) {
    const int c = lane & 3;
    float x[2][4];
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int e = 0; e < 4; e++) x[t][e] = 0.f;
#pragma unroll
      for (int s = 0; s < S; s++) {
        const uint32_t a[4] = {q[s][0], NT == 2 ? q[s][1] : 0u, q[s][NT], NT == 2 ? q[s][NT + 1] : 0u};
        mma_16816(x[t], a, word(kv.k[t][s >> 1], 2 * (s & 1)), word(kv.k[t][s >> 1], 2 * (s & 1) + 1));
      }
#pragma unroll
      for (int e = 0; e < 4; e++)
        x[t][e] = 8 * t + 2 * c + (e & 1) < nv ? x[t][e] * scale2 : -INFINITY;
    }
    uint32_t hi[2][NT], lo[2][NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      float mx = fmaxf(fmaxf(x[0][2 * n], x[0][2 * n + 1]), fmaxf(x[1][2 * n], x[1][2 * n + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const bool higher = mx > m[n] + 8.f;
      if (__any_sync(0xFFFFFFFFu, higher)) {  // (each head by its own scores alone)
        const float f = higher ? join_weight(m[n], mx) : 1.f;
        if (higher) m[n] = mx;
        l[n] *= f;
        const float f0 = __shfl_sync(0xFFFFFFFFu, f, 8 * c), f1 = __shfl_sync(0xFFFFFFFFu, f, 8 * c + 4);
#pragma unroll
        for (int i = 0; i < S; i++) {
          o[i][n][0] *= f0;
          o[i][n][1] *= f1;
          o[i][n][2] *= f0;
          o[i][n][3] *= f1;
        }
      }
      const float base = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const float p0 = exp2f(x[t][2 * n] - base), p1 = exp2f(x[t][2 * n + 1] - base);
        l[n] += p0 + p1;
        hi[t][n] = bf2(p0, p1);
        lo[t][n] = bf2(p0 - bf_lo(hi[t][n]), p1 - bf_hi(hi[t][n]));
      }
    }
#pragma unroll
    for (int i = 0; i < S; i++) {
      const int ch = i >> 2, w = i & 3;  // dims 64 ch + 8 r + 2 w, + 1
      const uint32_t v0 = word(kv.v[0][ch], w), v1 = word(kv.v[1][ch], w), v2 = word(kv.v[2][ch], w),
                     v3 = word(kv.v[3][ch], w);
      const uint32_t a[4] = {__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632),
                             __byte_perm(v2, v3, 0x5410), __byte_perm(v2, v3, 0x7632)};
#pragma unroll
      for (int n = 0; n < NT; n++) {
        mma_16816(o[i][n], a, hi[0][n], hi[1][n]);
        mma_16816(o[i][n], a, lo[0][n], lo[1][n]);
      }
    }
  }
};

// Lane's output dims e = 0, 1 of tile i.
MK_DEV int dec_dim(int i, int r) { return 64 * (i >> 2) + 8 * r + 2 * (i & 3); }

// Writes a finished row: out = o / l (0 where nothing was seen).
MK_DEV void attn_store2(const AttnArgs& a, long long t, int head, int dim, float o0, float o1, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(uint32_t*)((uint16_t*)a.o.p + t * a.o.ts + head * a.o.hs + dim) =
      l == 0.f ? 0u : bf2(o0 * inv, o1 * inv);
}

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, DecShape<D, NT>::BLOCKS)
kv_decode_kernel(const __grid_constant__ AttnArgs a) {
  using Sh = DecShape<D, NT>;
  constexpr int HB = Sh::HB, S = D / 16, LD = D + 4;
  __shared__ __align__(16) float so[DEC_WARPS][HB][LD];
  __shared__ float sm[DEC_WARPS][HB], sl[DEC_WARPS][HB];
  __shared__ unsigned redo;
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int blocks_of_heads = (a.G + HB - 1) / HB, items = a.kv.Hkv * blocks_of_heads;
  const long long total = dec_total(a.kv, a.bt, lane) * items;
  const int parts = (int)min((long long)gridDim.x, total);
  if ((int)blockIdx.x >= parts) return;
  const long long u0 = part_begin(total, parts, blockIdx.x), u1 = part_begin(total, parts, blockIdx.x + 1);
  const float scale2 = a.scale * LOG2E;
  if (threadIdx.x == 0) redo = 0;

  // Advance a place by one unit.
  auto next = [&](DecPlace& p) {
    if (++p.unit < p.units) return;
    p.unit = 0;
    if (++p.item < items) return;
    p.item = 0;
    if (++p.b < a.bt.batch) {
      p.len = kv_len(a.kv, a.bt, p.b);
      p.units = dec_units(p.len);
    }
  };
  // This warp's first row of a unit, and how many of the 16 exist.
  auto rows_of = [&](const DecPlace& p, int& j) {
    j = p.unit * DEC_UNIT + 16 * warp;
    return min(16, p.len - j);
  };
  auto block_of = [&](const DecPlace& p) {
    int j;
    return rows_of(p, j) > 0 ? kv_block_of(a.kv, p.b, j) : -1;
  };
  auto load = [&](DecRows<D>& rows, const DecPlace& p, int blk) {
    int j;
    const int n = rows_of(p, j), h = p.item / blocks_of_heads;
    const int in = a.kv.table ? (j & (a.kv.block - 1)) : j;
    rows.load(a.kv, blk < 0 ? -1 : ((long long)blk * a.kv.Hkv + h) * a.kv.block + in, n, lane);
    return blk < 0 ? 0 : n;
  };

  DecPlace p = dec_find(a.kv, a.bt, items, u0, lane), p1 = p, p2 = p;
  DecWarp<D, NT> w;
  DecRows<D> rows, ahead;
  int nv = load(rows, p, block_of(p)), nv1 = 0, blk2 = -1;
  if (u0 + 1 < u1) {
    next(p1);
    p2 = p1;
    blk2 = block_of(p2);
  }
  bool fresh = true;
  int from = p.unit;  // first unit of the item in this block
  for (long long u = u0; u < u1; u++) {
    const int h = p.item / blocks_of_heads, hb = p.item % blocks_of_heads;
    const int head0 = h * a.G + hb * HB, n_heads = min(HB, a.G - hb * HB);
    if (fresh) {
      w.init((const uint16_t*)a.q.p + p.b * a.q.ts + head0 * a.q.hs, a.q.hs, n_heads, lane);
      fresh = false;
      from = p.unit;
    }
    if (u + 1 < u1) nv1 = load(ahead, p1, blk2);
    if (u + 2 < u1) {
      next(p2);
      blk2 = block_of(p2);
    }
    w.step(rows, nv, scale2, lane);
    if (p.unit == p.units - 1 || u == u1 - 1) {  // the item's end, or this block's
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float l = w.l[n];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (c == 0) {
          sm[warp][8 * n + r] = w.m[n];
          sl[warp][8 * n + r] = l;
        }
#pragma unroll
        for (int i = 0; i < S; i++) {
          const int dim = dec_dim(i, r);
          *(float2*)&so[warp][8 * n + 2 * c][dim] = make_float2(w.o[i][n][0], w.o[i][n][2]);
          *(float2*)&so[warp][8 * n + 2 * c + 1][dim] = make_float2(w.o[i][n][1], w.o[i][n][3]);
        }
      }
      __syncthreads();
      const bool whole = from == 0 && p.unit == p.units - 1;
      // the block's first item's state goes to slot 0, another last one's to slot 1
      const bool first = u - (p.unit - from) == u0;
      float* st = a.ws + ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * Sh::STATE;
      for (int i = threadIdx.x; i < n_heads * (D / 2); i += DEC_THREADS) {
        const int head = i / (D / 2), dim = 2 * (i % (D / 2));
        float top = -INFINITY, l = 0.f;
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < DEC_WARPS; v++) top = fmaxf(top, sm[v][head]);
#pragma unroll
        for (int v = 0; v < DEC_WARPS; v++) {
          const float f = join_weight(sm[v][head], top);
          const float2 y = *(const float2*)&so[v][head][dim];
          l = fmaf(sl[v][head], f, l);
          o.x = fmaf(y.x, f, o.x);
          o.y = fmaf(y.y, f, o.y);
        }
        if (!isfinite(o.x + o.y) && isfinite(l)) atomicOr(&redo, 1u << head);
        if (whole) {
          attn_store2(a, p.b, head0 + head, dim, o.x, o.y, l);
          if (a.lse && dim == 0) a.lse[(long long)p.b * a.Hq + head0 + head] = state_lse(top, l);
        } else {
          *(float2*)(st + head * D + dim) = o;
          if (dim == 0) {
            st[HB * D + head] = top;
            st[HB * D + HB + head] = l;
          }
        }
      }
      __syncthreads();
      if (redo) {
        const unsigned mask = redo;
        for (int head = warp; head < n_heads; head += DEC_WARPS) {
          if (!(mask >> head & 1u)) continue;
          float m, l, o[D / 32];
          attn_row<D>(a.kv, p.b, h, (const uint16_t*)a.q.p + p.b * a.q.ts + (head0 + head) * a.q.hs,
                      a.scale, from * DEC_UNIT, min(p.len, (p.unit + 1) * DEC_UNIT), m, l, o);
#pragma unroll
          for (int e = 0; e < D / 32; e += 2) {
            const int dim = lane * (D / 32) + e;
            if (whole) {
              attn_store2(a, p.b, head0 + head, dim, o[e], o[e + 1], l);
            } else {
              st[head * D + dim] = o[e];
              st[head * D + dim + 1] = o[e + 1];
            }
          }
          if (!whole && lane == 0) {
            st[HB * D + head] = m * LOG2E;
            st[HB * D + HB + head] = l;
          }
        }
        __syncthreads();
        if (threadIdx.x == 0) redo = 0;
      }
      fresh = true;
    }
    rows = ahead;
    nv = nv1;
    p = p1;
    p1 = p2;
  }
}

// ---- few rows: a cluster per item ---------------------------------------------
// Where even full sequences are a few units for each block of a cluster, a cluster
// takes an item: each block an equal share of its units, no search of a line, and
// the blocks' states joined through distributed shared memory, in the same launch.

MK_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MK_DEV uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; what they wrote before is there after it.
MK_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// Block `rank`'s copy of a shared variable, two floats of it.
MK_DEV uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
MK_DEV float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, DecShape<D, NT>::BLOCKS)
kv_decode_cluster_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int HB = DecShape<D, NT>::HB, S = D / 16, LD = D + 4;
  __shared__ __align__(16) float so[DEC_WARPS][HB][LD];
  __shared__ float sm[DEC_WARPS][HB], sl[DEC_WARPS][HB];
  __shared__ __align__(16) float po[HB][D];  // this block's state
  __shared__ float2 pml[HB];
  __shared__ unsigned redo;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int rank = (int)cluster_rank(), size = (int)cluster_size();
  const int blocks_of_heads = (a.G + HB - 1) / HB, items = a.kv.Hkv * blocks_of_heads;
  const int work = blockIdx.x / size, b = work / items, item = work % items;
  const int h = item / blocks_of_heads, hb = item % blocks_of_heads;
  const int head0 = h * a.G + hb * HB, n_heads = min(HB, a.G - hb * HB);
  const uint16_t* q0 = (const uint16_t*)a.q.p + b * a.q.ts + head0 * a.q.hs;
  const int len = kv_len(a.kv, a.bt, b);
  const long long units = (len + DEC_UNIT - 1) / DEC_UNIT;
  const int u0 = (int)(units * rank / size), u1 = (int)(units * (rank + 1) / size);
  const float scale2 = a.scale * LOG2E;
  if (threadIdx.x == 0) redo = 0;

  // This warp's rows of unit u: their block, then the rows; how many count.
  auto block_of = [&](int u) {
    const int j = u * DEC_UNIT + 16 * warp;
    return u < u1 && j < len ? kv_block_of(a.kv, b, j) : -1;
  };
  auto load = [&](DecRows<D>& rows, int u, int blk) {
    const int j = u * DEC_UNIT + 16 * warp, n = min(16, len - j);
    const int in = a.kv.table ? (j & (a.kv.block - 1)) : j;
    rows.load(a.kv, blk < 0 ? -1 : ((long long)blk * a.kv.Hkv + h) * a.kv.block + in, n, lane);
    return blk < 0 ? 0 : n;
  };
  DecWarp<D, NT> w;
  DecRows<D> rows, ahead;
  int blk = block_of(u0);
  int nv = load(rows, u0, blk), nv1 = 0;
  blk = block_of(u0 + 1);
  w.init(q0, a.q.hs, n_heads, lane);
  for (int u = u0; u < u1; u++) {
    if (u + 1 < u1) {
      nv1 = load(ahead, u + 1, blk);
      blk = block_of(u + 2);
    }
    w.step(rows, nv, scale2, lane);
    rows = ahead;
    nv = nv1;
  }
#pragma unroll
  for (int n = 0; n < NT; n++) {
    float l = w.l[n];
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    if (c == 0) {
      sm[warp][8 * n + r] = w.m[n];
      sl[warp][8 * n + r] = l;
    }
#pragma unroll
    for (int i = 0; i < S; i++) {
      const int dim = dec_dim(i, r);
      *(float2*)&so[warp][8 * n + 2 * c][dim] = make_float2(w.o[i][n][0], w.o[i][n][2]);
      *(float2*)&so[warp][8 * n + 2 * c + 1][dim] = make_float2(w.o[i][n][1], w.o[i][n][3]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_heads * (D / 2); i += DEC_THREADS) {
    const int head = i / (D / 2), dim = 2 * (i % (D / 2));
    float top = -INFINITY, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < DEC_WARPS; v++) top = fmaxf(top, sm[v][head]);
#pragma unroll
    for (int v = 0; v < DEC_WARPS; v++) {
      const float f = join_weight(sm[v][head], top);
      const float2 y = *(const float2*)&so[v][head][dim];
      l = fmaf(sl[v][head], f, l);
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
    }
    if (!isfinite(o.x + o.y) && isfinite(l)) atomicOr(&redo, 1u << head);
    *(float2*)&po[head][dim] = o;
    if (dim == 0) pml[head] = make_float2(top, l);
  }
  __syncthreads();
  if (const unsigned mask = redo) {
    for (int head = warp; head < n_heads; head += DEC_WARPS) {
      if (!(mask >> head & 1u)) continue;
      float m, l, o[D / 32];
      attn_row<D>(a.kv, b, h, q0 + head * a.q.hs, a.scale, u0 * DEC_UNIT, min(len, u1 * DEC_UNIT), m, l, o);
#pragma unroll
      for (int e = 0; e < D / 32; e++) po[head][lane * (D / 32) + e] = o[e];
      if (lane == 0) pml[head] = make_float2(m * LOG2E, l);
    }
  }
  cluster_sync();
  // pairs of dimensions, dealt out over the cluster; the states eight at a time
  for (int i = rank * DEC_THREADS + threadIdx.x; i < n_heads * (D / 2); i += size * DEC_THREADS) {
    const int head = i / (D / 2), dim = 2 * (i % (D / 2));
    float m = -INFINITY, l = 0.f;
    float2 o = make_float2(0.f, 0.f);
    for (int k0 = 0; k0 < size; k0 += 8) {
      float2 ml[8], y[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const bool in = k0 + k < size;
        ml[k] = in ? ld_cluster2(cluster_addr(&pml[head], k0 + k)) : make_float2(-INFINITY, 0.f);
        y[k] = in ? ld_cluster2(cluster_addr(&po[head][dim], k0 + k)) : make_float2(0.f, 0.f);
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < 8; k++) top = fmaxf(top, ml[k].x);
      const float f = join_weight(m, top);
      m = top;
      l *= f;
      o.x *= f;
      o.y *= f;
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float g = join_weight(ml[k].x, top);
        if (ml[k].y == 0.f) continue;  // no weight
        l = fmaf(ml[k].y, g, l);
        o.x = fmaf(y[k].x, g, o.x);
        o.y = fmaf(y[k].y, g, o.y);
      }
    }
    attn_store2(a, b, head0 + head, dim, o.x, o.y, l);
    if (a.lse && dim == 0) a.lse[(long long)b * a.Hq + head0 + head] = state_lse(m, l);
  }
  cluster_sync();  // the others may still read this block's state
}

// How the line of units is cut, for the join: block i of `parts` begins at begin(i),
// which is part_begin() in 32 bits (the launch refuses more units).
struct DecLine {
  unsigned total, quot, rest;
  int parts;
  MK_DEV unsigned begin(int i) const { return quot * i + rest * (unsigned)i / (unsigned)parts; }
  // The block whose range holds unit u < total.
  MK_DEV int part_of(unsigned u) const {
    int i = min((int)((float)u / (float)total * parts), parts - 1);
    while (i > 0 && begin(i) > u) i--;
    while (i + 1 < parts && begin(i + 1) <= u) i++;
    return i;
  }
};

// The line of the whole batch, and the units before sequence b (one warp, all
// lanes; len0: rows of this lane's sequence among the first 32).
MK_DEV DecLine dec_line(const KvView& kv, const KvBatch& bt, int items, int grid, int len0, int b,
                        unsigned& before, int lane) {
  unsigned n = 0, m = 0;
  for (int i = lane; i < bt.batch; i += 32) {
    const unsigned u = dec_units(i < 32 ? len0 : kv_len(kv, bt, i));
    n += u;
    if (i < b) m += u;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    n += __shfl_xor_sync(0xFFFFFFFFu, n, w);
    m += __shfl_xor_sync(0xFFFFFFFFu, m, w);
  }
  before = m * items;
  DecLine l;
  l.total = n * items;
  l.parts = (int)min((unsigned)grid, l.total);
  l.quot = l.total / l.parts;
  l.rest = l.total - l.quot * l.parts;
  return l;
}

// Joins the states of the blocks that shared a row's item, W warps to a (sequence,
// query head): each takes every W-th state, four at a time with all their loads in
// flight.  What a warp needs besides the states it finds before it waits for the
// first kernel.
constexpr int JOIN_WARPS = 8;

template <int D, int NT, int W>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
kv_decode_join_kernel(const __grid_constant__ AttnArgs a, int grid) {
  using Sh = DecShape<D, NT>;
  constexpr int HB = Sh::HB, E = D / 32, N = 4;
  __shared__ float so[JOIN_WARPS][D], sm[JOIN_WARPS], sl[JOIN_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks_of_heads = (a.G + HB - 1) / HB, items = a.kv.Hkv * blocks_of_heads;
  const int row = blockIdx.x * (JOIN_WARPS / W) + warp / W, me = warp % W;
  const bool live = row < a.bt.batch * a.Hq;
  const int b = live ? row / a.Hq : 0, hq = row - b * a.Hq;
  const int g = hq % a.G, hb = g / HB, head = g - hb * HB;
  const int item = hq / a.G * blocks_of_heads + hb;
  const int units = dec_units(kv_len(a.kv, a.bt, b));
  const int len0 = lane < a.bt.batch ? kv_len(a.kv, a.bt, lane) : 0;
  unsigned first;
  const DecLine line = dec_line(a.kv, a.bt, items, grid, len0, b, first, lane);
  first += item * units;
  const int i0 = live ? line.part_of(first) : 0, i1 = live ? line.part_of(first + units - 1) : 0;
  const int slot0 = line.begin(i0) == first ? 0 : 1;
  pdl_wait();
  const bool split = live && i0 != i1;  // (else one block wrote the result)
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; e++) o[e] = 0.f;
  for (int i = split ? i0 + me : 1 << 30; i <= i1; i += N * W) {
    float mi[N], li[N], oi[N][E];
#pragma unroll
    for (int n = 0; n < N; n++) {
      const int j = i + n * W;
      const bool in = j <= i1;
      const float* st = a.ws + ((size_t)j * 2 + (j == i0 ? slot0 : 0)) * Sh::STATE;
      mi[n] = in ? st[HB * D + head] : -INFINITY;
      li[n] = in ? st[HB * D + HB + head] : 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 y = in ? *(const float2*)(st + head * D + lane * E + e) : make_float2(0.f, 0.f);
        oi[n][e] = y.x;
        oi[n][e + 1] = y.y;
      }
    }
    float top = m;
#pragma unroll
    for (int n = 0; n < N; n++) top = fmaxf(top, mi[n]);
    const float f = join_weight(m, top);
    l *= f;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] *= f;
#pragma unroll
    for (int n = 0; n < N; n++) {
      const float y = join_weight(mi[n], top);
      l = fmaf(li[n], y, l);
#pragma unroll
      for (int e = 0; e < E; e++) o[e] = fmaf(oi[n][e], y, o[e]);
    }
    m = top;
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < E; e++) so[warp][lane * E + e] = o[e];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (!split || me != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; w++) top = fmaxf(top, sm[warp + w]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < W; w++) {
      const float f = join_weight(sm[warp + w], top);
      l = fmaf(sl[warp + w], f, l);
#pragma unroll
      for (int e = 0; e < E; e++) o[e] = fmaf(so[warp + w][lane * E + e], f, o[e]);
    }
    m = top;
  }
  if (!split) return;
#pragma unroll
  for (int e = 0; e < E; e += 2) attn_store2(a, b, hq, lane * E + e, o[e], o[e + 1], l);
  if (a.lse && lane == 0) a.lse[(long long)b * a.Hq + hq] = state_lse(m, l);
}

}  // namespace mk
