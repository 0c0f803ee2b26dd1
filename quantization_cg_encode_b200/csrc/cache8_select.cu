// Choosing blocks of the 8-bit block-scaled KV cache: by a cheap score for each query token
// (sparse attention), or by the attention weight they have drawn (eviction).
//
// Score of a block for one query row: with q8 the row in whole numbers, |q8| <= 127 times a power
// of two 2^e,
//   2^e s_K sum_c max(q8_c lo_c, q8_c hi_c) = 2^e s_K (sum q8+ hi + sum q8- lo),
// the largest product that keys between the block's bounds can have with the rounded row; a
// block's score for a query token is its largest over the query heads of the KV head.  The sums
// are whole numbers below 2^21 and the factors powers of two: every step is exact in fp32, so the
// choice does not depend on the order of the sums, and ties go to the lowest index.
#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreBlocks = kScoreThreads / 4;  // blocks of the cache that a CTA scores at a time
constexpr int kPickThreads = 512;
constexpr int kPickKeys = 8192;                  // keys that the choosing CTA holds in shared memory
constexpr int kSms = 148;

// fp32 as an unsigned key of the same order; -0 is 0, NaN comes below everything
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Blocks [0, nb) a query token sees
__device__ __forceinline__ int seen_blocks(int n, int nq, int i, int tb) { return (max(0, n - nq + 1 + i) + tb - 1) / tb; }

}  // namespace

// scores[unit][i][block]: four lanes share a block (d / 4 channels each, both bounds), eight blocks a
// warp; the bounds stay in registers for all rows of the unit, and those of the CTA's next blocks
// are on their way meanwhile.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) cache8_score_kernel(Cache8SelectArgs a, int chunks, int per, int nb_max) {
  constexpr int Q = D / 64;               // 16-byte words of a lane's channels
  extern __shared__ uint4 sq[];           // [rows][2][D / 16]: q8 >= 0, q8 <= 0
  const int rows = a.gq * a.nq;
  float* unit = reinterpret_cast<float*>(sq + rows * (D / 8));  // [rows] 2^e
  const int H = a.c.k.H, B = a.c.k.B;
  const int u = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int h = u % H, b = u / H % B, lz = u / H / B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 3;
  const long long slice = ((long long)(a.l0 + lz) * B + b) * H + h;
  const uint4* bounds = reinterpret_cast<const uint4*>(a.bounds + slice * a.c.blocks() * 2 * D) + part;
  const float* scales = a.scales + (((long long)(a.l0 + lz) * 2 * B + b) * H + h) * a.c.blocks();
  previous_kernel_done();
  const int n = max(0, min(a.lens[b], a.max_tokens));
  const int nb = (n + a.c.tb - 1) / a.c.tb;
  const int end = min(nb, (chunk + 1) * per);
  int blk = chunk * per + warp * 8 + (lane >> 2);
  if (chunk * per >= nb) return;
  uint4 lo[Q], hi[Q];
  float sk = 0.0f;
  auto load = [&](int at) {
#pragma unroll
    for (int j = 0; j < Q; ++j) lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
    if (at < end) {
#pragma unroll
      for (int j = 0; j < Q; ++j) lo[j] = bounds[(long long)at * (D / 8) + 4 * j], hi[j] = bounds[(long long)at * (D / 8) + D / 16 + 4 * j];
      sk = scales[at];
    }
  };
  load(blk);
  for (int r = warp; r < rows; r += kScoreThreads / 32) {
    const uint16_t* q = a.q + ((long long)u * rows + r) * D;
    uint2 x = make_uint2(0, 0);
    if (lane < D / 4) x = *reinterpret_cast<const uint2*>(q + 4 * lane);
    const float v[4] = {bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y)};
    const float m = warp_max_f32(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const int e = cache8_exponent<kCache8Int8>(m);
    const float inv = two_to(-e);
    uint32_t up = 0, dn = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = max(-127, min(127, __float2int_rn(v[j] * inv)));
      up |= ((uint32_t)max(i, 0) & 255u) << (8 * j);
      dn |= ((uint32_t)min(i, 0) & 255u) << (8 * j);
    }
    uint32_t* w = reinterpret_cast<uint32_t*>(sq + r * (D / 8));
    if (lane < D / 4) w[lane] = up, w[D / 4 + lane] = dn;
    if (lane == 0) unit[r] = two_to(e);
  }
  __syncthreads();
  auto dot4 = [](const uint4& x, const uint4& y, int acc) {
    acc = __dp4a((int)x.x, (int)y.x, acc);
    acc = __dp4a((int)x.y, (int)y.y, acc);
    acc = __dp4a((int)x.z, (int)y.z, acc);
    return __dp4a((int)x.w, (int)y.w, acc);
  };
  float* out = a.scores + (long long)u * a.nq * nb_max;
  for (; blk - (lane >> 2) < end; blk += kScoreBlocks) {  // warp-uniform
    uint4 l[Q], g[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) l[j] = lo[j], g[j] = hi[j];
    const float scale = sk;
    load(blk + kScoreBlocks);
    for (int i = 0; i < a.nq; ++i) {
      float best = -INFINITY;
      for (int r = i; r < rows; r += a.nq) {
        const uint4* q = sq + r * (D / 8) + part;
        int dot = 0;
#pragma unroll
        for (int j = 0; j < Q; ++j) dot = dot4(g[j], q[4 * j], dot4(l[j], q[D / 16 + 4 * j], dot));
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        best = fmaxf(best, (float)dot * unit[r]);
      }
      if (part == 0 && blk < end) out[(long long)i * nb_max + blk] = best * scale;
    }
  }
}

namespace {

struct PickShared {
  uint32_t key[kPickKeys];
  uint32_t hist[2][256];
  uint32_t warp_sum[kPickThreads / 32];
  uint32_t least, most, found, need, whole;
};

// The k chosen of nb blocks (nb > k), ascending, into `out`: the first `sink`, the last
// `recent`, and of the others those of the highest keys, ties to the lowest index.  Whole CTA.
// Radix selection finds the key of the last one taken, eight bits a pass from the first bit in
// which the keys differ, until a pass ends with a whole bin; then one ordered pass writes the list.
// Keys wait in shared memory, or stay where they are if there are more than kPickKeys.
__device__ void pick_blocks(const float* key, int nb, int k, int sink, int recent, int* out, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = sink, hi = nb - recent;
  const bool held = nb <= kPickKeys;
  auto key_at = [&](int i) { return held ? sh.key[i] : order_key(key[i]); };
  if (tid == 0) sh.least = 0xffffffffu, sh.most = 0;
  if (tid < 256) sh.hist[0][tid] = 0;
  __syncthreads();
  uint32_t least = 0xffffffffu, most = 0;
  for (int i = lo + tid; i < hi; i += kPickThreads) {
    const uint32_t u = order_key(key[i]);
    if (held) sh.key[i] = u;
    least = min(least, u), most = max(most, u);
  }
  least = __reduce_min_sync(0xffffffffu, least), most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMin(&sh.least, least), atomicMax(&sh.most, most);
  __syncthreads();
  // keys >= thr are taken for sure, of those == thr the first `need` if it is not 0
  uint32_t need = (uint32_t)(k - sink - recent), thr = 0xffffffffu;
  bool exact = false;  // thr is one key's value
  if (need) {
    const uint32_t differ = sh.least ^ sh.most;
    int shift = differ ? 32 - __clz(differ) : 0;             // bits below it differ
    thr = shift < 32 ? sh.most >> shift << shift : 0;         // the bits above it are common
    for (int pass = 0; shift > 0; ++pass) {
      const int width = min(8, shift), high = shift;
      shift -= width;
      uint32_t* hist = sh.hist[pass & 1];
      for (int i = lo + tid; i < hi; i += kPickThreads) {
        const uint32_t u = key_at(i);
        if (high == 32 || (u >> high) == (thr >> high)) atomicAdd(&hist[(u >> shift) & ((1u << width) - 1)], 1u);
      }
      if (tid < 256) sh.hist[(pass + 1) & 1][tid] = 0;
      __syncthreads();
      if (warp == 0) {  // the bin in which the need-th highest lies
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - (8 * lane + j)];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        uint32_t above = incl - sum;
        if (above < need && incl >= need) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above + c[j] >= need) {
              sh.found = 255 - (8 * lane + j);
              sh.need = need - above;
              sh.whole = above + c[j] == need;
              break;
            }
            above += c[j];
          }
        }
      }
      __syncthreads();
      thr |= sh.found << shift;
      need = sh.need;
      if (sh.whole) break;
    }
    // a whole bin: every key from its lower end is taken; else the bits are used up and thr is a key
    exact = shift == 0 && !(sh.least != sh.most && sh.whole);
    if (!exact) need = 0;
  }
  // runs of an odd length for each thread (no two threads of a warp meet in a bank)
  const int per = (nb + kPickThreads - 1) / kPickThreads | 1;
  const int i0 = min(nb, tid * per), i1 = min(nb, i0 + per);
  auto kind = [&](int i) {  // 0: not taken, 1: taken, 2: equal to the threshold
    if (i < lo || i >= hi) return 1;
    if (thr == 0xffffffffu && !exact) return 0;
    const uint32_t u = key_at(i);
    return exact ? (u > thr ? 1 : u == thr ? 2 : 0) : (u >= thr ? 1 : 0);
  };
  uint32_t sure = 0, equal = 0;
  for (int i = i0; i < i1; ++i) {
    const int t = kind(i);
    sure += t == 1, equal += t == 2;
  }
  auto before = [&](uint32_t v) {  // sum over the threads before this one
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t sum = incl - v;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w)
      if (w < warp) sum += sh.warp_sum[w];
    return sum;
  };
  uint32_t at_sure = before(sure), at_equal = exact ? before(equal) : 0;  // `exact` is uniform
  for (int i = i0; i < i1; ++i) {
    const int t = kind(i);
    if (t == 1) out[at_sure++ + min(at_equal, need)] = i;
    if (t == 2) {
      if (at_equal < need) out[at_sure + at_equal] = i;
      ++at_equal;
    }
  }
}

}  // namespace

__global__ void __launch_bounds__(kPickThreads) cache8_pick_kernel(Cache8SelectArgs a, int nb_max) {
  __shared__ PickShared sh;
  const long long row = blockIdx.x;  // [nl][B][H][nq]
  const int i = (int)(row % a.nq), b = (int)(row / a.nq / a.c.k.H % a.c.k.B);
  previous_kernel_done();
  const int n = max(0, min(a.lens[b], a.max_tokens));
  const int nb = seen_blocks(n, a.nq, i, a.c.tb);
  int* out = a.sel + row * a.n_select;
  if (nb <= a.n_select) {
    for (int j = threadIdx.x; j < a.n_select; j += kPickThreads) out[j] = j < nb ? j : -1;
    return;
  }
  pick_blocks(a.scores + row * nb_max, nb, a.n_select, a.sink, a.recent, out, sh);
}

__global__ void __launch_bounds__(kPickThreads) cache8_keep_kernel(Cache8EvictArgs a) {
  __shared__ PickShared sh;
  const int u = blockIdx.x;  // [nl][B][H]
  const int H = a.c.k.H, B = a.c.k.B;
  const int h = u % H, b = u / H % B, lz = u / H / B;
  previous_kernel_done();
  const int n = max(0, min(a.lens[b], a.c.k.T)), tb = a.c.tb, nb = (n + tb - 1) / tb;
  const long long slice = ((long long)(a.l0 + lz) * B + b) * H + h;
  const float* mass = a.mass + slice * a.c.blocks();
  float* to_mass = a.to_mass + slice * a.to.blocks();
  int* kept = a.kept + (long long)u * a.keep;
  if (lz == 0 && h == 0 && threadIdx.x == 0) a.to_lens[b] = nb > a.keep ? n - (nb - a.keep) * tb : n;
  if (nb <= a.keep) {
    for (int j = threadIdx.x; j < a.keep; j += kPickThreads) kept[j] = j < nb ? j : -1;
  } else {
    pick_blocks(mass, nb, a.keep, a.sink, a.recent, kept, sh);
  }
  __syncthreads();
  const int m = min(nb, a.keep);
  for (int j = threadIdx.x; j < a.to.blocks(); j += kPickThreads) to_mass[j] = j < m ? mass[kept[j]] : 0.0f;
}

// Kept blocks of one (layer, K or V, batch, head): a warp moves 4096 bytes of codes, all its loads
// before its stores, and what belongs to the blocks that begin there.
__global__ void __launch_bounds__(256) cache8_move_kernel(Cache8EvictArgs a, int pieces) {
  constexpr int kPiece = 4096;
  const int H = a.c.k.H, B = a.c.k.B, d = a.c.k.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 8 + warp;  // (slice, piece)
  previous_kernel_done();
  const int piece = (int)(item % pieces);
  const int sl = (int)(item / pieces);
  if (sl >= a.nl * 2 * B * H) return;
  const int h = sl % H, b = sl / H % B, s = sl / H / B & 1, lz = sl / H / B >> 1;
  const int* kept = a.kept + (((long long)lz * B + b) * H + h) * a.keep;
  const long long slice = (((long long)(a.l0 + lz) * 2 + s) * B + b) * H + h;
  const int shift = 31 - __clz(a.c.tb * d);  // bytes of a block: 2^10 .. 2^13
  const uint8_t* src = a.codes + slice * a.c.k.T * d;
  uint8_t* dst = a.to_codes + slice * a.to.k.T * d;
  uint4 v[kPiece / 512];
  int from[kPiece / 512];
#pragma unroll
  for (int i = 0; i < kPiece / 512; ++i) {
    const long long at = (long long)piece * kPiece + 512 * i + 16 * lane;
    const int j = (int)(at >> shift);
    from[i] = j < a.keep ? kept[j] : -1;
  }
#pragma unroll
  for (int i = 0; i < kPiece / 512; ++i) {
    const long long at = (long long)piece * kPiece + 512 * i + 16 * lane;
    if (from[i] >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + ((long long)from[i] << shift) + (at & ((1 << shift) - 1))));
  }
#pragma unroll
  for (int i = 0; i < kPiece / 512; ++i) {
    const long long at = (long long)piece * kPiece + 512 * i + 16 * lane;
    if (from[i] >= 0) *reinterpret_cast<uint4*>(dst + at) = v[i];
  }
  // scales and bounds of the blocks whose codes begin in the piece
  const long long first = (((long long)piece * kPiece - 1) >> shift) + 1, last = ((long long)piece * kPiece + kPiece - 1) >> shift;
  const long long unit = ((long long)(a.l0 + lz) * B + b) * H + h;
  for (long long j = first; j <= last && j < a.keep; ++j) {
    const int blk = kept[j];
    if (blk < 0) break;
    if (lane == 31) a.to_scales[slice * a.to.blocks() + j] = a.scales[slice * a.c.blocks() + blk];
    if (s == 0 && a.bounds && lane < d / 8)
      reinterpret_cast<uint4*>(a.to_bounds)[(unit * a.to.blocks() + j) * (d / 8) + lane] =
          reinterpret_cast<const uint4*>(a.bounds)[(unit * a.c.blocks() + blk) * (d / 8) + lane];
  }
}

namespace {

long long select_units(const Cache8SelectArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H; }
int select_nb(const Cache8SelectArgs& a) { return (a.max_tokens + a.c.tb - 1) / a.c.tb; }
// blocks that a CTA scores: enough CTAs for the GPU, but up to eight times kScoreBlocks each, so that
// the query rows are rounded for many blocks
int score_per(const Cache8SelectArgs& a) {
  const long long want = (select_units(a) * select_nb(a) + 8 * kSms - 1) / (8 * kSms);
  const long long steps = (want + kScoreBlocks - 1) / kScoreBlocks;
  return kScoreBlocks * (int)(steps > 8 ? 8 : steps);
}
int score_chunks(const Cache8SelectArgs& a) { return (select_nb(a) + score_per(a) - 1) / score_per(a); }
int move_pieces(const Cache8EvictArgs& a) { return (int)(((long long)a.keep * a.c.tb * a.c.k.d + 4095) / 4096); }
long long move_ctas(const Cache8EvictArgs& a) { return ((long long)a.nl * 2 * a.c.k.B * a.c.k.H * move_pieces(a) + 7) / 8; }

}  // namespace

uint64_t cache8_select_workspace(const Cache8SelectArgs& a) {
  return ((uint64_t)select_units(a) * a.nq * select_nb(a) * sizeof(float) + 15) & ~15ull;
}
bool cache8_select_fits(const Cache8SelectArgs& a) {
  return select_units(a) * score_chunks(a) < (1LL << 31) && select_units(a) * a.nq < (1LL << 31);
}
cudaError_t launch_cache8_select(const Cache8SelectArgs& a, cudaStream_t st) {
  const int rows = a.gq * a.nq, d = a.c.k.d, per = score_per(a), chunks = score_chunks(a), nb = select_nb(a);
  const size_t smem = (size_t)rows * (2 * d + sizeof(float)), most = (size_t)kMaxGroup * kMaxQTokens * (2 * d + sizeof(float));
  static std::atomic<uint64_t> ready[2];
  auto kern = d == 128 ? cache8_score_kernel<128> : cache8_score_kernel<64>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), most, ready[d == 128]);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, dim3((unsigned)(select_units(a) * chunks)), kScoreThreads, smem, st, 1, a, chunks, per, nb);
  if (e != cudaSuccess) return e;
  return launch_after(cache8_pick_kernel, dim3((unsigned)(select_units(a) * a.nq)), kPickThreads, 0, st, 1, a, nb);
}

bool cache8_evict_fits(const Cache8EvictArgs& a) {
  return move_ctas(a) < (1LL << 31) && (long long)a.nl * 2 * a.c.k.B * a.c.k.H < (1LL << 31);
}
cudaError_t launch_cache8_evict(const Cache8EvictArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_after(cache8_keep_kernel, dim3((unsigned)(a.nl * a.c.k.B * a.c.k.H)), kPickThreads, 0, st, 1, a);
  if (e != cudaSuccess) return e;
  return launch_after(cache8_move_kernel, dim3((unsigned)move_ctas(a)), 256, 0, st, 1, a, move_pieces(a));
}

}  // namespace cg
