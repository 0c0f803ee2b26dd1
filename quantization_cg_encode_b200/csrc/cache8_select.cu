// Choosing blocks of the 8-bit block-scaled KV cache: by a cheap score for each query token
// (sparse attention), or by the attention weight they have drawn (eviction).
//
// Score of a block for one query row: with q8 the row in whole numbers, |q8| <= 127 times a power
// of two 2^e,
//   2^e s_K sum_c max(q8_c lo_c, q8_c hi_c) = 2^e s_K (sum q8+ hi + sum q8- lo),
// the largest product that keys between the block's bounds can have with the rounded row; a
// block's score for a query token is its largest over the query heads of the KV head.  The sums
// are whole numbers below 2^21 and the factors powers of two: every step is exact in fp32 (within its
// normal range), so the choice does not depend on the order of the sums, and ties go to the lowest index.
//
// The scores are a product of the bounds (16 blocks a warp) with the rows (8 at a time) on the
// integer tensor path, mma.sync m16n8k32: the bytes go from memory to operands as they are.  A
// cluster scores the blocks of one KV head, and one of its CTAs chooses among them for each query
// token from the shared memory of all: one kernel, whose time is its latency where few blocks are
// scored and the reading of the bounds where many are.  Beyond kPickKeys blocks the scores go
// through the workspace to a second kernel.
//
// Measured (B200, d = 128): 128 of up to 1024 blocks for 32 sequences of 8 KV heads, 42 MB of bounds,
// 20 us, of which the choice is 6 (it is serial: its barriers and loads wait with little else in
// flight); 64 of 2048 blocks for one sequence 9 us, the choice 4; 128 of 8192 23 us, of 10240 through
// the second kernel 25.  Eviction of half of the blocks of
// 32 layers x 2 sequences x 8 heads, 262 MB of codes in and out, 93 us = 5.9 TB/s; of one layer of 4
// sequences 8.5 us, latency.
#include <cooperative_groups.h>

#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStep = kWarps * 16;     // blocks that a CTA scores at a time
constexpr int kPickRegs = 8 * kThreads;  // keys that a choosing CTA holds in registers
constexpr int kPickKeys = 8192;          // and in the shared memory of its cluster
constexpr int kListed = 8192;            // blocks that an evicting CTA lists in shared memory
constexpr int kSms = 148;

// fp32 as an unsigned key of the same order; -0 is 0, NaN comes below everything
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Blocks [0, nb) a query token sees
__device__ __forceinline__ int seen_blocks(int n, int nq, int i, int tb) { return (max(0, n - nq + 1 + i) + tb - 1) / tb; }

__device__ __forceinline__ void imma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kFew = 32;  // keys among which a warp finds the threshold by counting

struct PickShared {
  uint4 hist[4][64];  // 256 bins a pass
  uint32_t few[kFew];
  uint32_t warp_sum[2][kWarps];
  uint32_t least, most, n_few;
};
// Before pick_blocks, with a barrier between
__device__ __forceinline__ void pick_prepare(PickShared& sh) {
  sh.hist[threadIdx.x >> 6][threadIdx.x & 63] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) sh.least = 0xffffffffu, sh.most = 0, sh.n_few = 0;
}
static_assert(kThreads == 256, "four histograms of 64 words of 16 bytes");

// The k chosen of nb blocks (nb > k), ascending, into `out`: the first `sink`, the last
// `recent`, and of the others those of the highest keys, ties to the lowest index.  Whole CTA.
// Radix selection finds the key of the last one taken, eight bits a pass from the first bit in
// which the keys differ, until few keys are left, which are counted against one another; then one
// ordered pass writes the list.  Every warp reads the histogram for itself: one barrier a pass.
// A thread has KPT consecutive keys in registers (keys.load gives them, of whatever stands behind
// the last one), keys(i) gives key i (KPT 0: a run of them, read each time).
template <int KPT, typename Keys>
__device__ void pick_blocks(const Keys& keys, int nb, unsigned k, int sink, int recent, int* out, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = sink, hi = nb - recent;
  uint32_t u[KPT ? KPT : 1];
  if constexpr (KPT > 0) {
    if (tid * KPT < nb) keys.load(tid * KPT, nb, u);
  }
  auto each = [&](auto f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const int i = tid * KPT + j;
        if (i >= lo && i < hi) f(u[j]);
      }
    } else {
      for (int i = lo + tid; i < hi; i += kThreads) f(keys(i));
    }
  };
  uint32_t least = 0xffffffffu, most = 0;
  each([&](uint32_t v) { least = min(least, v), most = max(most, v); });
  least = __reduce_min_sync(0xffffffffu, least), most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMin(&sh.least, least), atomicMax(&sh.most, most);
  __syncthreads();
  // keys > thr are taken, and of those == thr the first `need`
  uint32_t need = (uint32_t)(k - sink - recent), thr = 0xffffffffu;  // (no key is as high)
  if (need) {
    const uint32_t differ = sh.least ^ sh.most;
    int shift = differ ? 32 - __clz(differ) : 0;       // the bits below it differ
    thr = shift < 32 ? sh.most >> shift << shift : 0;   // the bits above it are common
    uint32_t inside = (uint32_t)(hi - lo);              // keys with those bits
    for (int pass = 0; shift > 0; ++pass) {
      const int high = shift;
      if (inside <= kFew) {
        each([&](uint32_t v) {
          if (high == 32 || (v >> high) == (thr >> high)) {
            const uint32_t at = atomicAdd(&sh.n_few, 1u);
            if (at < kFew) sh.few[at] = v;  // (always, unless the values change meanwhile)
          }
        });
        __syncthreads();
        const uint32_t mine = lane < inside ? sh.few[lane] : 0u;
        uint32_t above = 0, same = 0;
        for (uint32_t j = 0; j < inside; ++j) {
          const uint32_t v = sh.few[j];
          above += v > mine, same += v == mine;
        }
        const unsigned got = __ballot_sync(0xffffffffu, lane < inside && above < need && above + same >= need);
        thr = __shfl_sync(0xffffffffu, mine, __ffs(got) - 1);
        need -= __shfl_sync(0xffffffffu, above, __ffs(got) - 1);
        break;
      }
      const int width = min(8, shift);
      shift -= width;
      uint32_t* hist = reinterpret_cast<uint32_t*>(sh.hist[pass]);
      each([&](uint32_t v) {
        if (high == 32 || (v >> high) == (thr >> high)) atomicAdd(&hist[(v >> shift) & ((1u << width) - 1)], 1u);
      });
      __syncthreads();
      // the bin in which the need-th highest lies: a lane's bins are 255 - 8 lane and the seven below
      const uint4 x = sh.hist[pass][63 - 2 * lane], y = sh.hist[pass][62 - 2 * lane];
      const uint32_t c[8] = {x.w, x.z, x.y, x.x, y.w, y.z, y.y, y.x};
      const uint32_t sum = c[0] + c[1] + c[2] + c[3] + c[4] + c[5] + c[6] + c[7];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      uint32_t above = incl - sum, bin = 255 - 8 * lane, in_bin = 0;
      const bool mine = above < need && incl >= need;
      bool found = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!found && above + c[j] >= need) found = true, in_bin = c[j], bin -= j;
        if (!found) above += c[j];
      }
      const int owner = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      thr |= __shfl_sync(0xffffffffu, bin, owner) << shift;
      need -= __shfl_sync(0xffffffffu, above, owner);
      inside = __shfl_sync(0xffffffffu, in_bin, owner);
    }
  }
  // 0: not taken, 1: taken, 2: equal to the threshold; a thread has consecutive keys
  const int per = KPT ? KPT : (nb + kThreads - 1) / kThreads | 1;  // (odd: no two threads of a warp meet in a bank)
  const int i0 = min(nb, tid * per), i1 = min(nb, i0 + per);
  auto kind = [&](int i, uint32_t v) { return i < lo || i >= hi || v > thr ? 1 : v == thr ? 2 : 0; };
  auto ordered = [&](auto f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (tid * KPT + j < nb) f(tid * KPT + j, kind(tid * KPT + j, u[j]));
    } else {
      for (int i = i0; i < i1; ++i) f(i, kind(i, keys(i)));
    }
  };
  uint32_t sure = 0, equal = 0;
  ordered([&](int, int t) { sure += t == 1, equal += t == 2; });
  // sums over the threads before this one
  uint32_t s_incl = sure, e_incl = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, s_incl, o), y = __shfl_up_sync(0xffffffffu, e_incl, o);
    if (lane >= o) s_incl += x, e_incl += y;
  }
  if (lane == 31) sh.warp_sum[0][warp] = s_incl, sh.warp_sum[1][warp] = e_incl;
  __syncthreads();
  sure = s_incl - sure, equal = e_incl - equal;
  for (int w = 0; w < warp; ++w) sure += sh.warp_sum[0][w], equal += sh.warp_sum[1][w];
  ordered([&](int i, int t) {
    const uint32_t at = sure + min(equal, need);
    if ((t == 1 || (t == 2 && equal < need)) && at < k) out[at] = i;  // (at < k unless the values change meanwhile)
    sure += t == 1, equal += t == 2;
  });
}
template <typename Keys>
__device__ __forceinline__ void pick_any(const Keys& keys, int nb, int k, int sink, int recent, int* out, PickShared& sh) {
  if (nb <= 2 * kThreads)
    pick_blocks<2>(keys, nb, k, sink, recent, out, sh);
  else if (nb <= kPickRegs)
    pick_blocks<8>(keys, nb, k, sink, recent, out, sh);
  else
    pick_blocks<0>(keys, nb, k, sink, recent, out, sh);
}
// Keys of fp32 values in global memory
struct ValueKeys {
  const float* v;
  __device__ uint32_t operator()(int i) const { return order_key(v[i]); }
  template <int N>
  __device__ void load(int i, int nb, uint32_t (&u)[N]) const {
    float x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = i + j < nb ? v[i + j] : 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) u[j] = order_key(x[j]);
  }
};
// Keys that the CTAs of a cluster hold, `per` (a multiple of 16) each
struct ClusterKeys {
  const uint32_t* mine;
  int per;
  unsigned per_inv;  // i / per = umulhi(i, per_inv) for i < 2^16
  __device__ const uint32_t* of(int i) const {
    const int k = __umulhi((unsigned)i, per_inv);
    return cooperative_groups::this_cluster().map_shared_rank(mine, k) + (i - k * per);
  }
  __device__ uint32_t operator()(int i) const { return *of(i); }
  __device__ void load(int i, int, uint32_t (&u)[2]) const {
    const uint2 x = *reinterpret_cast<const uint2*>(of(i));
    u[0] = x.x, u[1] = x.y;
  }
  __device__ void load(int i, int, uint32_t (&u)[8]) const {
    const uint4* p = reinterpret_cast<const uint4*>(of(i));
    const uint4 x = p[0], y = p[1];
    u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w, u[4] = y.x, u[5] = y.y, u[6] = y.z, u[7] = y.w;
  }
};
// Keys in this CTA's shared memory
struct HeldKeys {
  const uint32_t* v;
  __device__ uint32_t operator()(int i) const { return v[i]; }
};

// Query rows in tiles of eight operand columns: up to eight heads make a group of 1, 2, 4 or 8
// columns, as many query tokens to a tile as fit; more heads take two tiles a token.
struct RowTiles {
  int group;      // log2 of the columns of a token in a tile (a tile has 8 >> group tokens)
  int per_token;  // log2 of the tiles of a token (0, or 1 where group is 3)
  int count;
};
__host__ __device__ inline RowTiles row_tiles(int gq, int nq) {
  RowTiles r;
  r.group = gq <= 1 ? 0 : gq <= 2 ? 1 : gq <= 4 ? 2 : 3;
  r.per_token = gq > 8;
  r.count = (nq + (8 >> r.group) - 1) >> (3 - r.group) << r.per_token;
  return r;
}

}  // namespace

// A CTA scores `per` blocks of one (layer, batch, KV head).  FUSED: the CTAs of a cluster share the
// unit, each keeps its scores as keys, and the choice follows; else the scores go to a.scores.
// CTAS: how many of them an SM has to hold.
template <int D, bool FUSED, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) cache8_score_kernel(Cache8SelectArgs a, int chunks, int per, int nb_max) {
  constexpr int Q = D / 64;               // 16-byte pieces of a lane, of one bound of one block
  __shared__ PickShared sh;
  __shared__ int s_n;
  extern __shared__ uint4 sq[];           // [tile][column][q8 <= 0, q8 >= 0][D / 16]
  const RowTiles rt = row_tiles(a.gq, a.nq);
  float* unit = reinterpret_cast<float*>(sq + rt.count * 8 * (D / 8));  // [tile][column] 2^e, negative: no row
  uint32_t* keys = reinterpret_cast<uint32_t*>(unit + rt.count * 8);     // [nq][per]
  const unsigned H = a.c.k.H, B = a.c.k.B, u = blockIdx.x / chunks, bh = u / H;
  const int chunk = blockIdx.x % chunks, h = u - bh * H, b = bh % B, lz = bh / B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const long long slice = ((long long)(a.l0 + lz) * B + b) * H + h;
  const uint4* bounds = reinterpret_cast<const uint4*>(a.bounds + slice * a.c.blocks() * 2 * D) + c;
  const float* scales = a.scales + (((long long)(a.l0 + lz) * 2 * B + b) * H + h) * a.c.blocks();
  previous_kernel_done();
  const int n = max(0, min(a.lens[b], a.max_tokens));
  if (threadIdx.x == 0) s_n = n;  // for the choice: its barriers depend on it, so one reading for all
  const int nb = (n + a.c.tb - 1) / a.c.tb;
  const int begin = chunk * per, end = min(nb, begin + per);
  if (!FUSED && begin >= nb) return;
  uint4 x[2][2][Q];  // [block g, g + 8][low, high][piece]
  float scale[2];
  auto load = [&](int at) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int blk = at + g + 8 * r;
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        x[r][0][j] = blk < end ? bounds[(long long)blk * (D / 8) + 4 * j] : make_uint4(0, 0, 0, 0);
        x[r][1][j] = blk < end ? bounds[(long long)blk * (D / 8) + D / 16 + 4 * j] : make_uint4(0, 0, 0, 0);
      }
      scale[r] = blk < end ? scales[blk] : 0.0f;
    }
  };
  load(begin + warp * 16);
  for (int r = warp; r < rt.count * 8; r += kWarps) {
    const int tile = r >> 3, col = r & 7;
    const int i = (tile >> rt.per_token << (3 - rt.group)) + (col >> rt.group);
    const int j = (tile & rt.per_token) * 8 + (col & ((1 << rt.group) - 1));
    const bool on = i < a.nq && j < a.gq;
    uint2 y = make_uint2(0, 0);
    if (on && lane < D / 4) y = *reinterpret_cast<const uint2*>(a.q + (((long long)u * a.gq + j) * a.nq + i) * D + 4 * lane);
    const float v[4] = {bf16lo(y.x), bf16hi(y.x), bf16lo(y.y), bf16hi(y.y)};
    const float m = warp_max_f32(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const int e = cache8_exponent<kCache8Int8>(m);
    const float inv = two_to(-e);
    uint32_t dn = 0, up = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int q = max(-127, min(127, __float2int_rn(v[k] * inv)));
      dn |= ((uint32_t)min(q, 0) & 255u) << (8 * k);
      up |= ((uint32_t)max(q, 0) & 255u) << (8 * k);
    }
    uint32_t* w = reinterpret_cast<uint32_t*>(sq + r * (D / 8));
    if (lane < D / 4) w[lane] = dn, w[D / 4 + lane] = up;
    if (lane == 0) unit[r] = on ? two_to(e) : -1.0f;
  }
  __syncthreads();
  for (int at = begin + warp * 16; at < end; at += kStep) {  // warp-uniform
    float best[4];  // (block g, columns 2c, 2c + 1), then block g + 8
    for (int tile = 0; tile < rt.count; ++tile) {
      int dot[4] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const uint4 q = sq[(tile * 8 + g) * (D / 8) + s * (D / 16) + 4 * j + c];
          imma(dot, x[0][s][j].x, x[1][s][j].x, x[0][s][j].y, x[1][s][j].y, q.x, q.y);
          imma(dot, x[0][s][j].z, x[1][s][j].z, x[0][s][j].w, x[1][s][j].w, q.z, q.w);
        }
      const float2 un = *reinterpret_cast<const float2*>(unit + tile * 8 + 2 * c);
      const float v0 = un.x > 0.0f ? (float)dot[0] * un.x : -INFINITY, v1 = un.y > 0.0f ? (float)dot[1] * un.y : -INFINITY;
      const float v2 = un.x > 0.0f ? (float)dot[2] * un.x : -INFINITY, v3 = un.y > 0.0f ? (float)dot[3] * un.y : -INFINITY;
      if (!(tile & rt.per_token)) {
        best[0] = v0, best[1] = v1, best[2] = v2, best[3] = v3;
      } else {
        best[0] = fmaxf(best[0], v0), best[1] = fmaxf(best[1], v1), best[2] = fmaxf(best[2], v2), best[3] = fmaxf(best[3], v3);
      }
      if (rt.per_token && !(tile & 1)) continue;
      // the largest of a token's columns
      if (rt.group >= 1) best[0] = best[1] = fmaxf(best[0], best[1]), best[2] = best[3] = fmaxf(best[2], best[3]);
      for (int o = 1; o < 1 << rt.group >> 1; o <<= 1) {
        best[0] = fmaxf(best[0], __shfl_xor_sync(0xffffffffu, best[0], o));
        best[2] = fmaxf(best[2], __shfl_xor_sync(0xffffffffu, best[2], o));
      }
      const int i0 = tile >> rt.per_token << (3 - rt.group);
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // column 2c + k writes if it is its token's first
        const int col = 2 * c + k, i = i0 + (col >> rt.group);
        if ((col & ((1 << rt.group) - 1)) == 0 && i < a.nq) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int blk = at + g + 8 * r;
            const float score = best[2 * r + k] * scale[r];
            if (blk < end) {
              if (FUSED)
                keys[i * per + blk - begin] = order_key(score);
              else
                a.scores[((long long)u * a.nq + i) * nb_max + blk] = score;
            }
          }
        }
      }
    }
    load(at + kStep);
  }
  if constexpr (FUSED) {
    namespace cgs = cooperative_groups;
    cgs::cluster_group cluster = cgs::this_cluster();
    pick_prepare(sh);
    cluster.sync();
    uint32_t* all = keys + a.nq * per;  // [nb] where a choice among more than kPickRegs needs them all
    const unsigned per_inv = 0xffffffffu / per + 1;  // i / per for i < 2^16, per > 1
    for (int i = chunk; i < a.nq; i += chunks) {
      const int seen = seen_blocks(s_n, a.nq, i, a.c.tb);
      int* out = a.sel + ((long long)u * a.nq + i) * a.n_select;
      if (seen <= a.n_select) {
        for (int j = threadIdx.x; j < a.n_select; j += kThreads) out[j] = j < seen ? j : -1;
        continue;
      }
      const ClusterKeys theirs{keys + i * per, per, per_inv};
      if (i != chunk) {  // another token of this CTA's
        __syncthreads();
        pick_prepare(sh);
      }
      if (seen > kPickRegs) {
#pragma unroll 4
        for (int j = threadIdx.x; j < seen; j += kThreads) all[j] = theirs(j);
      }
      __syncthreads();
      if (seen > kPickRegs)
        pick_blocks<0>(HeldKeys{all}, seen, a.n_select, a.sink, a.recent, out, sh);
      else if (seen > 2 * kThreads)
        pick_blocks<8>(theirs, seen, a.n_select, a.sink, a.recent, out, sh);
      else
        pick_blocks<2>(theirs, seen, a.n_select, a.sink, a.recent, out, sh);
    }
    cluster.sync();  // no CTA ends while another reads its keys
  }
}

__global__ void __launch_bounds__(kThreads) cache8_pick_kernel(Cache8SelectArgs a, int nb_max) {
  __shared__ PickShared sh;
  const long long row = blockIdx.x;  // [nl][B][H][nq]
  const int i = (int)(row % a.nq), b = (int)(row / a.nq / a.c.k.H % a.c.k.B);
  __shared__ int s_n;
  previous_kernel_done();
  if (threadIdx.x == 0) s_n = max(0, min(a.lens[b], a.max_tokens));
  __syncthreads();
  const int nb = seen_blocks(s_n, a.nq, i, a.c.tb);
  int* out = a.sel + row * a.n_select;
  if (nb <= a.n_select) {
    for (int j = threadIdx.x; j < a.n_select; j += kThreads) out[j] = j < nb ? j : -1;
    return;
  }
  pick_prepare(sh);
  __syncthreads();
  pick_any(ValueKeys{a.scores + row * nb_max}, nb, a.n_select, a.sink, a.recent, out, sh);
}

// Eviction: a CTA chooses the blocks of one (layer, batch, KV head) and moves a part of them.  The
// choice is made again by every CTA of the unit, which costs less than a second kernel or a wait;
// the first one writes it down.
// LISTED: the choice (more than kListed blocks stay) has been written by cache8_keep_kernel.
__device__ void keep_blocks(const Cache8EvictArgs& a, int u, int b, int lz, int h, bool write, int* list, PickShared& sh) {
  __shared__ int s_n;
  if (threadIdx.x == 0) s_n = max(0, min(a.lens[b], a.c.k.T));
  __syncthreads();  // one reading for all: barriers depend on it
  const int n = s_n, tb = a.c.tb, nb = (n + tb - 1) / tb;
  const long long slice = ((long long)(a.l0 + lz) * a.c.k.B + b) * a.c.k.H + h;
  const float* mass = a.mass + slice * a.c.blocks();
  if (nb <= a.keep) {
    for (int j = threadIdx.x; j < a.keep; j += kThreads) list[j] = j < nb ? j : -1;
  } else {
    pick_prepare(sh);
    __syncthreads();
    pick_any(ValueKeys{mass}, nb, a.keep, a.sink, a.recent, list, sh);
  }
  __syncthreads();
  if (!write) return;
  int* kept = a.kept + (long long)u * a.keep;
  float* to_mass = a.to_mass + slice * a.to.blocks();
  const int m = min(nb, a.keep);
  if (lz == 0 && h == 0 && threadIdx.x == 0) a.to_lens[b] = nb > a.keep ? n - (nb - a.keep) * tb : n;
  for (int j = threadIdx.x; j < a.to.blocks(); j += kThreads) to_mass[j] = j < m && (unsigned)list[j] < (unsigned)a.c.blocks() ? mass[list[j]] : 0.0f;
  if (kept != list)
    for (int j = threadIdx.x; j < a.keep; j += kThreads) kept[j] = list[j];
}

__global__ void __launch_bounds__(kThreads) cache8_keep_kernel(Cache8EvictArgs a) {
  __shared__ PickShared sh;
  const unsigned H = a.c.k.H, B = a.c.k.B, u = blockIdx.x, bh = u / H;
  previous_kernel_done();
  const int b = bh % B;
  keep_blocks(a, u, b, bh / B, u - bh * H, true, a.kept + (long long)u * a.keep, sh);
}

template <bool LISTED>
__global__ void __launch_bounds__(kThreads, 4) cache8_evict_kernel(Cache8EvictArgs a, int parts) {
  constexpr int kPiece = 4096;  // bytes of codes that a warp moves at a time, all loads before the stores
  __shared__ PickShared sh;
  extern __shared__ int s_list[];  // [keep]
  const unsigned H = a.c.k.H, B = a.c.k.B, u = blockIdx.x / parts, bh = u / H;
  const int part = blockIdx.x % parts, h = u - bh * H, b = bh % B, lz = bh / B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.c.k.d;
  const int* kept = LISTED ? a.kept + (long long)u * a.keep : s_list;
  previous_kernel_done();
  if (!LISTED) keep_blocks(a, u, b, lz, h, part == 0, s_list, sh);
  const int shift = 31 - __clz(a.c.tb * d);  // bytes of a block: 2^10 .. 2^13
  const int pieces = (int)((((long long)a.keep << shift) + kPiece - 1) / kPiece);  // of the keys, and of the values
  for (int item = part * kWarps + warp; item < 2 * pieces; item += parts * kWarps) {
    const int s = item >= pieces, piece = item - s * pieces;
    const long long slice = (((long long)(a.l0 + lz) * 2 + s) * B + b) * H + h;
    const uint8_t* src = a.codes + slice * a.c.k.T * d;
    uint8_t* dst = a.to_codes + slice * a.to.k.T * d;
    const long long p0 = (long long)piece * kPiece + 16 * lane;
    uint4 v[kPiece / 512];
    bool there[kPiece / 512];
#pragma unroll
    for (int i = 0; i < kPiece / 512; ++i) {
      const int j = (int)((p0 + 512 * i) >> shift), blk = j < a.keep ? kept[j] : -1;
      there[i] = (unsigned)blk < (unsigned)a.c.blocks();
      if (there[i]) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + ((long long)blk << shift) + ((p0 + 512 * i) & ((1 << shift) - 1))));
    }
#pragma unroll
    for (int i = 0; i < kPiece / 512; ++i)
      if (there[i]) *reinterpret_cast<uint4*>(dst + p0 + 512 * i) = v[i];
    // scales and bounds of the blocks whose codes begin in the piece
    const long long unit = ((long long)(a.l0 + lz) * B + b) * H + h;
    const int last = (int)(((long long)piece * kPiece + kPiece - 1) >> shift);
    for (int j = (int)((((long long)piece * kPiece - 1) >> shift) + 1); j <= last && j < a.keep; ++j) {
      const int blk = kept[j];
      if ((unsigned)blk >= (unsigned)a.c.blocks()) break;
      if (lane == 31) a.to_scales[slice * a.to.blocks() + j] = a.scales[slice * a.c.blocks() + blk];
      if (s == 0 && a.bounds && lane < d / 8)
        reinterpret_cast<uint4*>(a.to_bounds)[(unit * a.to.blocks() + j) * (d / 8) + lane] =
            reinterpret_cast<const uint4*>(a.bounds)[(unit * a.c.blocks() + blk) * (d / 8) + lane];
    }
  }
}

namespace {

long long select_units(const Cache8SelectArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H; }
int select_nb(const Cache8SelectArgs& a) { return (a.max_tokens + a.c.tb - 1) / a.c.tb; }
bool select_fused(const Cache8SelectArgs& a) { return select_nb(a) <= kPickKeys; }
// CTAs of a unit.  Fused: a cluster of up to eight, no more than the GPU holds at once beyond two
// unless the keys of all query tokens would not fit.  Else as many as keep the rows' rounding to one
// in eight steps.
int score_chunks(const Cache8SelectArgs& a) {
  const int steps = (select_nb(a) + kStep - 1) / kStep;
  if (!select_fused(a)) return (steps + 7) / 8;
  int c = 1;
  while (c < 8 && c < steps && (c < 2 || select_units(a) * c * 2 <= 5 * kSms || (long long)a.nq * select_nb(a) / c > 8192)) c *= 2;
  return c;
}
int score_per(const Cache8SelectArgs& a) {
  const int c = score_chunks(a);
  return ((select_nb(a) + c - 1) / c + 15) / 16 * 16;
}
size_t score_smem(const Cache8SelectArgs& a) {
  const RowTiles rt = row_tiles(a.gq, a.nq);
  return (size_t)rt.count * 8 * (2 * a.c.k.d + sizeof(float)) + (select_fused(a) ? (size_t)a.nq * score_per(a) * 4 : 0) +
         (select_fused(a) && select_nb(a) > kPickRegs ? (size_t)select_nb(a) * 4 : 0);
}
long long evict_units(const Cache8EvictArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H; }
// CTAs of a unit: enough for the GPU, but at least 64 KB of codes to move for each choice made
int evict_parts(const Cache8EvictArgs& a) {
  const long long bytes = 2LL * a.keep * a.c.tb * a.c.k.d, most = (bytes + 65535) / 65536;
  const long long want = (4 * kSms + evict_units(a) - 1) / evict_units(a);
  return (int)(want < most ? want : most);
}
bool evict_listed(const Cache8EvictArgs& a) { return a.keep > kListed; }

}  // namespace

uint64_t cache8_select_workspace(const Cache8SelectArgs& a) {
  return select_fused(a) ? 16 : ((uint64_t)select_units(a) * a.nq * select_nb(a) * sizeof(float) + 15) & ~15ull;
}
bool cache8_select_fits(const Cache8SelectArgs& a) {
  return select_units(a) * score_chunks(a) < (1LL << 31) && select_units(a) * a.nq < (1LL << 31);
}
cudaError_t launch_cache8_select(const Cache8SelectArgs& a, cudaStream_t st) {
  const int chunks = score_chunks(a), per = score_per(a), nb = select_nb(a);
  const bool fused = select_fused(a), wide = a.c.k.d == 128;
  static std::atomic<uint64_t> ready[6];
  // Two CTAs an SM leave registers for all loads at once, four the more CTAs: one sequence of 2048
  // blocks and its attention took 16.4 us with two and 18.2 with four, 32 sequences 74.8 and 71.9.
  const bool many = fused && select_units(a) * chunks > 2 * kSms;
  auto kern = many ? (wide ? cache8_score_kernel<128, true, 4> : cache8_score_kernel<64, true, 4>)
              : fused ? (wide ? cache8_score_kernel<128, true, 2> : cache8_score_kernel<64, true, 2>)
                      : (wide ? cache8_score_kernel<128, false, 2> : cache8_score_kernel<64, false, 2>);
  // 256 rows of 256 bytes, the keys of 16 tokens and 1024 blocks, and those of one token and all
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 176 * 1024, ready[2 * (fused + many) + wide]);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, dim3((unsigned)(select_units(a) * chunks)), kThreads, score_smem(a), st, fused ? chunks : 1, a, chunks, per, nb);
  if (e != cudaSuccess || fused) return e;
  return launch_after(cache8_pick_kernel, dim3((unsigned)(select_units(a) * a.nq)), kThreads, 0, st, 1, a, nb);
}

bool cache8_evict_fits(const Cache8EvictArgs& a) {
  const long long most = (1LL << 31) - 1;
  return evict_units(a) * evict_parts(a) <= most && ((long long)a.keep * a.c.tb * a.c.k.d + 4095) / 4096 <= most / 2;
}
cudaError_t launch_cache8_evict(const Cache8EvictArgs& a, cudaStream_t st) {
  const int parts = evict_parts(a);
  const unsigned ctas = (unsigned)(evict_units(a) * parts);
  if (!evict_listed(a)) {
    static std::atomic<uint64_t> ready;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(cache8_evict_kernel<false>), kListed * 4, ready);
    if (e != cudaSuccess) return e;
    return launch_after(cache8_evict_kernel<false>, dim3(ctas), kThreads, a.keep * sizeof(int), st, 1, a, parts);
  }
  const cudaError_t e = launch_after(cache8_keep_kernel, dim3((unsigned)evict_units(a)), kThreads, 0, st, 1, a);
  if (e != cudaSuccess) return e;
  return launch_after(cache8_evict_kernel<true>, dim3(ctas), kThreads, 0, st, 1, a, parts);
}

}  // namespace cg
