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
constexpr int kPickThreads = 512;

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
// warp; the bounds stay in registers for all rows of the unit.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) cache8_score_kernel(Cache8SelectArgs a, int chunks, int nb_max) {
  constexpr int W = D / 16;               // words (of four channels) of a lane
  extern __shared__ uint32_t sq[];        // [rows][2][D / 4]: q8 >= 0, q8 <= 0
  const int rows = a.gq * a.nq;
  float* unit = reinterpret_cast<float*>(sq + rows * (D / 2));  // [rows] 2^e
  const int H = a.c.k.H, B = a.c.k.B;
  const long long u = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int h = (int)(u % H), b = (int)((u / H) % B), lz = (int)(u / H / B);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = max(0, min(a.lens[b], a.max_tokens));
  const int nb = (n + a.c.tb - 1) / a.c.tb;
  if (chunk * kScoreThreads / 4 >= nb) return;
  for (int r = warp; r < rows; r += kScoreThreads / 32) {
    const uint16_t* q = a.q + (u * rows + r) * D;
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
    if (lane < D / 4) sq[r * (D / 2) + lane] = up, sq[r * (D / 2) + D / 4 + lane] = dn;
    if (lane == 0) unit[r] = two_to(e);
  }
  __syncthreads();
  const int part = lane & 3;
  const int blk = chunk * (kScoreThreads / 4) + warp * 8 + (lane >> 2);
  const bool live = blk < nb;
  const long long slice = ((long long)(a.l0 + lz) * B + b) * H + h;
  uint32_t lo[W], hi[W];
  if (live) {
    const uint4* p = reinterpret_cast<const uint4*>(a.bounds + (slice * a.c.blocks() + blk) * 2 * D);
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const uint4 x = p[part * (W / 4) + j], y = p[D / 16 + part * (W / 4) + j];
      lo[4 * j] = x.x, lo[4 * j + 1] = x.y, lo[4 * j + 2] = x.z, lo[4 * j + 3] = x.w;
      hi[4 * j] = y.x, hi[4 * j + 1] = y.y, hi[4 * j + 2] = y.z, hi[4 * j + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j) lo[j] = hi[j] = 0;
  }
  const float sk = live ? a.scales[((((long long)(a.l0 + lz) * 2) * B + b) * H + h) * a.c.blocks() + blk] : 0.0f;
  for (int i = 0; i < a.nq; ++i) {
    float best = -INFINITY;
    for (int j = 0; j < a.gq; ++j) {
      const int r = j * a.nq + i;
      const uint32_t* up = sq + r * (D / 2) + part * W;
      int dot = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) dot = __dp4a((int)hi[w], (int)up[w], dot);
#pragma unroll
      for (int w = 0; w < W; ++w) dot = __dp4a((int)lo[w], (int)up[D / 4 + w], dot);
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      best = fmaxf(best, (float)dot * unit[r]);
    }
    if (live && part == 0) a.scores[(u * a.nq + i) * nb_max + blk] = best * sk;
  }
}

namespace {

struct PickShared {
  uint32_t hist[256];
  uint32_t warp_sum[kPickThreads / 32];
  uint32_t prefix, need, found;
};

// The k chosen of nb blocks (nb > k), ascending, into `out`: the first `sink`, the last
// `recent`, and of the others those of the highest keys, ties to the lowest index.  Whole CTA.
// Radix selection finds the key of the last one taken (four passes of eight bits), then one
// ordered pass writes the list.
__device__ void pick_blocks(const float* key, int nb, int k, int sink, int recent, int* out, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = sink, hi = nb - recent;
  uint32_t thr = 0, need = (uint32_t)(k - sink - recent);
  if (need) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kPickThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kPickThreads) {
        const uint32_t u = order_key(key[i]);
        if (shift == 24 || (u >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&sh.hist[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // the bin in which the need-th highest lies
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = sh.hist[255 - (8 * lane + j)];
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
            if (above < need && above + c[j] >= need) {
              sh.found = 255 - (8 * lane + j);
              sh.need = need - above;
              break;
            }
            above += c[j];
          }
        }
      }
      __syncthreads();
      thr |= sh.found << shift;
      need = sh.need;
      __syncthreads();
    }
  }
  // `need` of the keys equal to thr are taken, the lowest indices first
  uint32_t taken = 0, equal = 0;  // before the current run
  for (int base = 0; base < nb; base += kPickThreads) {
    const int i = base + tid;
    uint32_t flag = 0;  // low half: taken for sure, high half: equal to the threshold
    if (i < nb) {
      if (i < lo || i >= hi) {
        flag = 1;
      } else if (k > sink + recent) {
        const uint32_t u = order_key(key[i]);
        flag = u > thr ? 1u : u == thr ? 0x10000u : 0u;
      }
    }
    uint32_t incl = flag;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) {
      const uint32_t v = sh.warp_sum[w];
      if (w < warp) before += v;
      all += v;
    }
    const uint32_t excl = before + incl - flag;
    const uint32_t eq = equal + (excl >> 16), sure = taken + (excl & 0xffffu);
    if (flag == 1u || (flag == 0x10000u && eq < need)) out[sure + min(eq, need)] = i;
    taken += all & 0xffffu;
    equal += all >> 16;
    __syncthreads();
  }
}

}  // namespace

__global__ void __launch_bounds__(kPickThreads) cache8_pick_kernel(Cache8SelectArgs a, int nb_max) {
  __shared__ PickShared sh;
  const long long row = blockIdx.x;  // [nl][B][H][nq]
  const int i = (int)(row % a.nq), b = (int)(row / a.nq / a.c.k.H % a.c.k.B);
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
  const long long u = blockIdx.x;  // [nl][B][H]
  const int H = a.c.k.H, B = a.c.k.B;
  const int h = (int)(u % H), b = (int)((u / H) % B), lz = (int)(u / H / B);
  const int n = max(0, min(a.lens[b], a.c.k.T)), tb = a.c.tb, nb = (n + tb - 1) / tb;
  const long long slice = ((long long)(a.l0 + lz) * B + b) * H + h;
  const float* mass = a.mass + slice * a.c.blocks();
  float* to_mass = a.to_mass + slice * a.to.blocks();
  int* kept = a.kept + u * a.keep;
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

// Kept blocks of one (layer, K or V, batch, head), 4096 bytes of codes a CTA
__global__ void __launch_bounds__(256) cache8_move_kernel(Cache8EvictArgs a, int per, int chunks) {
  const int H = a.c.k.H, B = a.c.k.B, d = a.c.k.d, tb = a.c.tb;
  const int chunk = blockIdx.x % chunks;
  const long long sl = blockIdx.x / chunks;
  const int h = (int)(sl % H), b = (int)((sl / H) % B), s = (int)((sl / H / B) & 1), lz = (int)(sl / H / B / 2);
  const int* kept = a.kept + (((long long)lz * B + b) * H + h) * a.keep;
  const long long slice = (((long long)(a.l0 + lz) * 2 + s) * B + b) * H + h;
  const long long unit = ((long long)(a.l0 + lz) * B + b) * H + h;
  const int v = tb * d / 16;  // 16-byte words of a block
  const uint4* src = reinterpret_cast<const uint4*>(a.codes + slice * a.c.k.T * d);
  uint4* dst = reinterpret_cast<uint4*>(a.to_codes + slice * a.to.k.T * d);
  const int j0 = chunk * per, j1 = min(a.keep, j0 + per);
  for (int e = threadIdx.x; e < (j1 - j0) * v; e += 256) {
    const int j = j0 + e / v, blk = kept[j];
    if (blk >= 0) dst[(long long)j * v + e % v] = src[(long long)blk * v + e % v];
  }
  for (int j = j0 + threadIdx.x; j < j1; j += 256)
    if (kept[j] >= 0) a.to_scales[slice * a.to.blocks() + j] = a.scales[slice * a.c.blocks() + kept[j]];
  if (s == 0 && a.bounds) {
    const int w = 2 * d / 16;
    const uint4* bs = reinterpret_cast<const uint4*>(a.bounds + unit * a.c.blocks() * 2 * d);
    uint4* bd = reinterpret_cast<uint4*>(a.to_bounds + unit * a.to.blocks() * 2 * d);
    for (int e = threadIdx.x; e < (j1 - j0) * w; e += 256) {
      const int j = j0 + e / w, blk = kept[j];
      if (blk >= 0) bd[(long long)j * w + e % w] = bs[(long long)blk * w + e % w];
    }
  }
}

namespace {

long long select_units(const Cache8SelectArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H; }
int select_nb(const Cache8SelectArgs& a) { return (a.max_tokens + a.c.tb - 1) / a.c.tb; }
int score_chunks(const Cache8SelectArgs& a) { return (select_nb(a) + kScoreThreads / 4 - 1) / (kScoreThreads / 4); }
int move_per(const Cache8EvictArgs& a) {
  const int per = 4096 / (a.c.tb * a.c.k.d);
  return per < 1 ? 1 : per;
}
long long move_ctas(const Cache8EvictArgs& a) {
  const int per = move_per(a);
  return (long long)a.nl * 2 * a.c.k.B * a.c.k.H * ((a.keep + per - 1) / per);
}

}  // namespace

uint64_t cache8_select_workspace(const Cache8SelectArgs& a) {
  return ((uint64_t)select_units(a) * a.nq * select_nb(a) * sizeof(float) + 15) & ~15ull;
}
bool cache8_select_fits(const Cache8SelectArgs& a) {
  return select_units(a) * score_chunks(a) < (1LL << 31) && select_units(a) * a.nq < (1LL << 31);
}
cudaError_t launch_cache8_select(const Cache8SelectArgs& a, cudaStream_t st) {
  const int rows = a.gq * a.nq, d = a.c.k.d, chunks = score_chunks(a), nb = select_nb(a);
  const size_t smem = (size_t)rows * (2 * d + sizeof(float));
  auto kern = d == 128 ? cache8_score_kernel<128> : cache8_score_kernel<64>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(select_units(a) * chunks), kScoreThreads, smem, st>>>(a, chunks, nb);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache8_pick_kernel<<<(unsigned)(select_units(a) * a.nq), kPickThreads, 0, st>>>(a, nb);
  return cudaGetLastError();
}

bool cache8_evict_fits(const Cache8EvictArgs& a) { return move_ctas(a) < (1LL << 31); }
cudaError_t launch_cache8_evict(const Cache8EvictArgs& a, cudaStream_t st) {
  cache8_keep_kernel<<<(unsigned)((long long)a.nl * a.c.k.B * a.c.k.H), kPickThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per = move_per(a);
  cache8_move_kernel<<<(unsigned)move_ctas(a), 256, 0, st>>>(a, per, (a.keep + per - 1) / per);
  return cudaGetLastError();
}

}  // namespace cg
