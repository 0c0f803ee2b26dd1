// Decode-step attention over the 8-bit block-scaled KV cache, over every token or over listed
// blocks, with the attention weight of every block on request.
//
// For the query rows of one KV head (row = query head of its group, query token) and tokens t:
//   x_t = scale log2(e) (q . k_t) s_K,  p_t = 2^(x_t - M),  out = sum p_t s_V v_t / sum p_t,
// k_t, v_t the codes and s_K, s_V the scales of the token's block.
//
// One pass over the cache, which is what bounds it (2 d bytes a token): the codes go from
// memory to tensor-core operands (mma.sync m16n8k16: the few query rows are the 8 columns; the
// fifth-generation MMA would leave 120 of its 128 rows empty, and this pass waits for memory).
//   scores  A = 16 tokens x 16 channels of key codes, exact in fp16; B = q, times a power of two
//           per row that puts its largest element into [2^14, 2^15): bf16 values are exact in
//           fp16 down to 2^-29 of the row's largest;
//   values  A = 16 channels x 16 tokens of value codes; B = p as two fp16 terms (2^-22).
// The order of channels within a contraction is free, so a thread's codes come as 16-byte
// pieces of the cache's rows, with no exchange between threads; B of the second product is the
// scores' layout transposed (movmatrix).
//
// The value scale is a power of two, 2^v: p s_V = 2^(x + v) is kept relative to its own running
// maximum M', so that no ratio of scales costs fp16 range, and the sum of p relative to M:
//   out = (sum 2^(x + v - M') code) / (sum 2^(x - M)) 2^(M' - M).
// M and M' follow the maxima lazily (they move when a value is 2^8 above).
//
// A warp owns 16-token tiles; the warps of a CTA share a run of tiles (a split) and merge in
// shared memory; a second kernel merges the splits.
#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxSplits = 256;
constexpr int kSms = 148;               // what the split is sized for
constexpr float kNone = -1.0e30f;       // a running maximum that has seen nothing
constexpr float kLag = 8.0f;            // how far a value may lie above the running maximum
constexpr float kShift = 7.0f;          // 2^kShift p' <= 2^15 fits fp16

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// maximum over the eight lanes that share lane % 4
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float column_sum(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int clamped_len(const Cache8AttnArgs& a, int b) { return max(0, min(a.lens[b], a.max_tokens)); }
// 16-token tiles that the rows of a unit have to look at
__device__ __forceinline__ int live_tiles(const Cache8AttnArgs& a, int n) {
  return a.n_select ? (n ? a.n_select * (a.c.tb >> 4) : 0) : (n + 15) >> 4;
}

}  // namespace

template <int D, int CODE, int NT, bool SPARSE, bool MASS>
__global__ void __launch_bounds__(kWarps * 32) cache8_attn_kernel(Cache8AttnArgs a) {
  constexpr int R = 8 * NT, HALVES = D / 64, VW = D / 32;  // VW: words of a thread's value codes of one token
  __shared__ float s_m[kWarps][R], s_mv[kWarps][R], s_l[kWarps][R];
  extern __shared__ float s_o[];  // [kWarps][R][D]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x % a.splits;
  long long u = blockIdx.x / a.splits;
  const int rt = (int)(u % a.row_tiles);
  u /= a.row_tiles;
  const int qi = SPARSE ? (int)(u % a.nq) : 0;  // the query token of a sparse unit
  if (SPARSE) u /= a.nq;
  const int H = a.c.k.H, B = a.c.k.B;
  const int h = (int)(u % H), b = (int)((u / H) % B), lz = (int)(u / H / B);
  const int rows = SPARSE ? a.gq : a.gq * a.nq;
  const int n = clamped_len(a, b);
  const int tiles = live_tiles(a, n);
  const int tile0 = split * a.tiles_per_split, tile1 = min(tiles, tile0 + a.tiles_per_split);
  // row r of the unit is row `first + r step` of the [nl][B][hq][nq] rows
  const long long first = (u * a.gq) * a.nq + qi, step = SPARSE ? a.nq : 1;
  if (tile0 >= tile1) {
    if (a.splits == 1)  // nothing to see: zeros
      for (int e = threadIdx.x; e < R * D; e += kWarps * 32) {
        const int r = rt * R + e / D;
        if (r < rows) a.out[(first + r * step) * D + e % D] = 0.0f;
        if (MASS && r < rows && e % D == 0) a.stats[first + r * step] = make_float2(0.0f, 0.0f);
      }
    return;
  }
  const long long ks_slice = (((long long)(a.l0 + lz) * 2 + 0) * B + b) * H + h;
  const long long vs_slice = (((long long)(a.l0 + lz) * 2 + 1) * B + b) * H + h;
  const uint8_t* kc = a.codes + ks_slice * a.c.k.T * D;
  const uint8_t* vc = a.codes + vs_slice * a.c.k.T * D;
  const float* ks = a.scales + ks_slice * a.c.blocks();
  const float* vs = a.scales + vs_slice * a.c.blocks();
  const int tb_shift = 31 - __clz(a.c.tb);

  // q as the scores' B operand, its row's power of two, and what each column's rows see
  uint32_t bq[NT][4 * HALVES][2];
  float qs[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rt * R + nt * 8 + g;
    const uint16_t* qrow = a.q + (first + (long long)min(r, rows - 1) * step) * D;
    uint4 raw[HALVES][2];
    float m = 0.0f;
#pragma unroll
    for (int hh = 0; hh < HALVES; ++hh)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        raw[hh][j] = r < rows ? *reinterpret_cast<const uint4*>(qrow + 64 * hh + 16 * c + 8 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16lo(word(raw[hh][j], i))), fabsf(bf16hi(word(raw[hh][j], i)))));
      }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100) - 14;  // m 2^-e in [2^14, 2^15)
    const float up = two_to(-e);
#pragma unroll
    for (int hh = 0; hh < HALVES; ++hh)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t p0 = word(raw[hh][w >> 1], 2 * (w & 1)), p1 = word(raw[hh][w >> 1], 2 * (w & 1) + 1);
        const float v0 = bf16lo(p0) * up, v1 = bf16hi(p0) * up, v2 = bf16lo(p1) * up, v3 = bf16hi(p1) * up;
        __half2 f0, f1;
        if (CODE == kCache8Int8) {
          f0 = __floats2half2_rn(v0, v2), f1 = __floats2half2_rn(v1, v3);
        } else {
          f0 = __floats2half2_rn(v0, v1), f1 = __floats2half2_rn(v2, v3);
        }
        bq[nt][4 * hh + w][0] = *reinterpret_cast<uint32_t*>(&f0);
        bq[nt][4 * hh + w][1] = *reinterpret_cast<uint32_t*>(&f1);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = 2 * c + j, rc = rt * R + nt * 8 + col;
      qs[nt][j] = two_to(max(__shfl_sync(0xffffffffu, e, 4 * col), -126)) * (a.scale * 1.4426950408889634f);
      const int i = SPARSE ? qi : rc % a.nq;
      lim[nt][j] = rc < rows ? max(0, n - a.nq + 1 + i) : 0x7fffffff;  // columns beyond the rows are not stored
    }
  }
  const int all_see = max(0, n - a.nq + 1 + (SPARSE ? qi : 0));  // tokens that every row sees
  const int end = SPARSE ? all_see : n;                          // tokens that some row sees

  float o[NT][D / 16][4];
  float m_run[NT][2], mv_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) m_run[nt][j] = mv_run[nt][j] = kNone, l_run[nt][j] = 0.0f;
  }

  const int* list = SPARSE ? a.sel + (u * a.nq + qi) * a.n_select : nullptr;
  for (int tile = tile0 + warp; tile < tile1; tile += kWarps) {
    int t0 = tile * 16;
    if (SPARSE) {
      const int blk = list[t0 >> tb_shift];
      if (blk < 0 || blk > (end - 1) >> tb_shift || end == 0) continue;  // warp-uniform
      t0 = (blk << tb_shift) + (t0 & (a.c.tb - 1));
      if (t0 >= end) continue;
    }
    const bool full = t0 + 16 <= end;  // else the codes behind the end may be anything: not read
    uint4 kr[2][HALVES];
    uint32_t vr[4][VW];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int hh = 0; hh < HALVES; ++hh) {
        const int t = t0 + g + 8 * j;
        kr[j][hh] = full || t < end ? *reinterpret_cast<const uint4*>(kc + (long long)t * D + 64 * hh + 16 * c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + 2 * c + (j & 1) + 8 * (j >> 1);
      const uint8_t* p = vc + (long long)t * D + (D / 8) * g;
      if constexpr (VW == 4) {
        const uint4 v = full || t < end ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        vr[j][0] = v.x, vr[j][1] = v.y, vr[j][2] = v.z, vr[j][3] = v.w;
      } else {
        const uint2 v = full || t < end ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
        vr[j][0] = v.x, vr[j][1] = v.y;
      }
    }
    const float kscale = ks[t0 >> tb_shift];
    const float vexp = (float)((int)(__float_as_uint(vs[t0 >> tb_shift]) >> 23) - 127);

    // scores of 16 tokens x R rows
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
    for (int hh = 0; hh < HALVES; ++hh)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t af[4];
        codes_to_f16<CODE>(word(kr[0][hh], w), af[0], af[2]);
        codes_to_f16<CODE>(word(kr[1][hh], w), af[1], af[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt], af, bq[nt][4 * hh + w][0], bq[nt][4 * hh + w][1]);
      }
    // s[nt][0..3]: token g (0, 1) or g + 8 (2, 3), row 2c + (index & 1)
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + g + 8 * (j >> 1);
        float x = s[nt][j] * (kscale * qs[nt][j & 1]);
        if (t0 + 16 > all_see) x = t < lim[nt][j & 1] && t < end ? x : -INFINITY;
        s[nt][j] = x;
        over |= x > m_run[nt][j & 1] + kLag || x + vexp > mv_run[nt][j & 1] + kLag;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float top = column_max(fmaxf(s[nt][j], s[nt][j + 2]));
          const float m = fmaxf(m_run[nt][j], top), mv = fmaxf(mv_run[nt][j], top + vexp);
          const float f = ex2(m_run[nt][j] - m), fv = ex2(mv_run[nt][j] - mv);
          m_run[nt][j] = m, mv_run[nt][j] = mv;
          l_run[nt][j] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[nt][i][j] *= fv, o[nt][i][j + 2] *= fv;
        }
    }
    uint32_t bhi[NT][2], blo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4];
      float tile_sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2(s[nt][j] - m_run[nt][j & 1]);
        tile_sum[j & 1] += p;
        pv[j] = ex2(s[nt][j] + (vexp + kShift) - mv_run[nt][j & 1]);
      }
      l_run[nt][0] += tile_sum[0], l_run[nt][1] += tile_sum[1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 hi = __floats2half2_rn(pv[2 * j], pv[2 * j + 1]);
        const float2 back = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(pv[2 * j] - back.x, pv[2 * j + 1] - back.y);
        bhi[nt][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&hi));
        blo[nt][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
      }
      if (MASS) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float sum = column_sum(tile_sum[j]);
          const int r = rt * R + nt * 8 + 2 * c + j;
          if (g == 0 && r < rows)
            a.tile_mass[(first + r) * ((a.max_tokens + 15) >> 4) + tile] = make_float2(sum, m_run[nt][j]);
        }
      }
    }
    // o[channel][row] += codes^T p
#pragma unroll
    for (int w = 0; w < VW; ++w)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t af[4];
        const uint32_t pick = CODE == kCache8Int8 ? (p ? 0x7632u : 0x5410u) : (p ? 0x7362u : 0x5140u);
        codes_to_f16<CODE>(__byte_perm(vr[0][w], vr[1][w], pick), af[0], af[1]);
        codes_to_f16<CODE>(__byte_perm(vr[2][w], vr[3][w], pick), af[2], af[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(o[nt][2 * w + p], af, bhi[nt][0], bhi[nt][1]);
          mma_f16_16816(o[nt][2 * w + p], af, blo[nt][0], blo[nt][1]);
        }
      }
  }

  // merge the warps: o relative to the CTA's maxima
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float l = column_sum(l_run[nt][j]);
      const int r = nt * 8 + 2 * c + j;
      if (g == 0) s_m[warp][r] = m_run[nt][j], s_mv[warp][r] = mv_run[nt][j], s_l[warp][r] = l;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int ch = (D / 8) * g + 2 * i;  // tile i = 2 w + p: channels 4 w + 2 p and the next
        s_o[(warp * R + r) * D + ch] = o[nt][i][j];
        s_o[(warp * R + r) * D + ch + 1] = o[nt][i][j + 2];
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < R * D; e += kWarps * 32) {
    const int r = e / D, ch = e % D;
    if (rt * R + r >= rows) continue;
    float m = kNone, mv = kNone, l = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][r]), mv = fmaxf(mv, s_mv[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      l = __fmaf_rn(s_l[w][r], ex2(s_m[w][r] - m), l);
      acc = __fmaf_rn(s_o[(w * R + r) * D + ch], ex2(s_mv[w][r] - mv), acc);
    }
    const long long row = first + (rt * R + r) * step;
    if (a.splits == 1) {
      a.out[row * D + ch] = l > 0.0f ? acc * ex2(mv - m - kShift) / l : 0.0f;
      if (MASS && ch == 0) a.stats[row] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
    } else {
      float* p = a.part + (row * a.splits + split) * (D + 4);
      p[4 + ch] = acc;
      if (ch == 0) p[0] = m, p[1] = mv, p[2] = l;
    }
  }
}

// One row of the output from its splits.
template <int D>
__global__ void __launch_bounds__(D) cache8_combine_kernel(Cache8AttnArgs a, bool mass) {
  __shared__ float wo[kMaxSplits];
  __shared__ float red[3][D / 32];
  const long long row = blockIdx.x;
  const int b = (int)(row / ((long long)a.hq * a.nq) % a.c.k.B);
  const int live = (live_tiles(a, clamped_len(a, b)) + a.tiles_per_split - 1) / a.tiles_per_split;
  const float* part = a.part + row * a.splits * (D + 4);
  const int ch = threadIdx.x, warp = ch >> 5;
  float m = kNone, mv = kNone, l = 0.0f;
  for (int i = ch; i < live; i += D) m = fmaxf(m, part[i * (D + 4)]), mv = fmaxf(mv, part[i * (D + 4) + 1]);
  m = warp_max_f32(m), mv = warp_max_f32(mv);
  if ((ch & 31) == 0) red[0][warp] = m, red[1][warp] = mv;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < D / 32; ++i) m = fmaxf(m, red[0][i]), mv = fmaxf(mv, red[1][i]);
  for (int i = ch; i < live; i += D) {
    l = __fmaf_rn(part[i * (D + 4) + 2], ex2(part[i * (D + 4)] - m), l);
    wo[i] = ex2(part[i * (D + 4) + 1] - mv);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((ch & 31) == 0) red[2][warp] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) l += red[2][i];
  float acc = 0.0f;
#pragma unroll 4
  for (int i = 0; i < live; ++i) acc = __fmaf_rn(part[i * (D + 4) + 4 + ch], wo[i], acc);
  a.out[row * D + ch] = l > 0.0f ? acc * ex2(mv - m - kShift) / l : 0.0f;
  if (mass && ch == 0) a.stats[row] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
}

// mass[block] (+)= sum over the unit's rows and the block's tiles of p
__global__ void __launch_bounds__(256) cache8_mass_kernel(Cache8AttnArgs a, int chunks) {
  const int H = a.c.k.H, B = a.c.k.B, nb = a.c.blocks();
  const long long u = blockIdx.x / chunks;
  const int blk = (blockIdx.x % chunks) * 256 + threadIdx.x;
  if (blk >= nb) return;
  const int h = (int)(u % H), b = (int)((u / H) % B), lz = (int)(u / H / B);
  const int n = clamped_len(a, b), tpb = a.c.tb >> 4, tiles = (a.max_tokens + 15) >> 4, live = (n + 15) >> 4;
  const int rows = a.gq * a.nq;
  float* at = a.mass + (((long long)(a.l0 + lz) * B + b) * H + h) * nb + blk;
  float sum = 0.0f;
  const int i1 = min(live, (blk + 1) * tpb);
  for (int r = 0; r < rows; ++r) {
    const float2 st = a.stats[u * rows + r];
    const float2* tm = a.tile_mass + (u * rows + r) * tiles;
    float part = 0.0f;
    for (int i = blk * tpb; i < i1; ++i) part = __fmaf_rn(tm[i].x, ex2(tm[i].y - st.x), part);
    sum = __fmaf_rn(part, st.y, sum);
  }
  if (!a.accumulate) {
    *at = sum;
  } else if (blk * tpb < live) {
    *at += sum;
  }
}

namespace {

long long total_rows(const Cache8AttnArgs& a) { return (long long)a.nl * a.c.k.B * a.hq * a.nq; }
long long units(const Cache8AttnArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H * (a.n_select ? a.nq : 1) * a.row_tiles; }

// Rows of a CTA: 8 where they are enough, else 16 (two operand columns for one reading of the
// codes).  Splits: as many CTAs as fill the GPU a few times over, so that ragged lengths even
// out, but no run of fewer than 16 tiles (two a warp).
void plan(Cache8AttnArgs& a) {
  const int rows = a.n_select ? a.gq : a.gq * a.nq;
  a.nt = rows > 8 ? 2 : 1;
  a.row_tiles = (rows + 8 * a.nt - 1) / (8 * a.nt);
  const int tiles = a.n_select ? a.n_select * (a.c.tb / 16) : (a.max_tokens + 15) / 16;
  const long long want = (8LL * kSms + units(a) - 1) / units(a);
  long long per = (tiles + want - 1) / want;
  per = per < 16 ? 16 : per > 64 ? 64 : per;
  if ((tiles + per - 1) / per > kMaxSplits) per = (tiles + kMaxSplits - 1) / kMaxSplits;
  a.tiles_per_split = (int)per;
  a.splits = (int)((tiles + per - 1) / per);
}

uint64_t round16(uint64_t b) { return (b + 15) & ~15ull; }

void layout(Cache8AttnArgs& a, char* base, bool want_mass, uint64_t& bytes) {
  const uint64_t rows = (uint64_t)total_rows(a);
  uint64_t at = 0;
  a.part = reinterpret_cast<float*>(base);
  if (a.splits > 1) at += round16(rows * a.splits * (a.c.k.d + 4) * sizeof(float));
  if (want_mass) {
    a.tile_mass = reinterpret_cast<float2*>(base + at);
    at += round16(rows * ((a.max_tokens + 15) / 16) * sizeof(float2));
    a.stats = reinterpret_cast<float2*>(base + at);
    at += round16(rows * sizeof(float2));
  }
  bytes = at ? at : 16;
}

template <int D, int CODE, int NT, bool SPARSE, bool MASS>
cudaError_t launch_one(const Cache8AttnArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * kWarps * 8 * NT * D;
  auto kern = cache8_attn_kernel<D, CODE, NT, SPARSE, MASS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(units(a) * a.splits), kWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}
template <int D, int CODE, int NT>
cudaError_t launch_kind(const Cache8AttnArgs& a, cudaStream_t st) {
  if (a.n_select) return launch_one<D, CODE, NT, true, false>(a, st);
  return a.mass ? launch_one<D, CODE, NT, false, true>(a, st) : launch_one<D, CODE, NT, false, false>(a, st);
}
template <int D>
cudaError_t launch_d(const Cache8AttnArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.c.code == kCache8Int8)
    e = a.nt == 1 ? launch_kind<D, kCache8Int8, 1>(a, st) : launch_kind<D, kCache8Int8, 2>(a, st);
  else
    e = a.nt == 1 ? launch_kind<D, kCache8E4m3, 1>(a, st) : launch_kind<D, kCache8E4m3, 2>(a, st);
  if (e != cudaSuccess || a.splits == 1) return e;
  cache8_combine_kernel<D><<<(unsigned)total_rows(a), D, 0, st>>>(a, a.mass != nullptr);
  return cudaGetLastError();
}

int mass_chunks(const Cache8AttnArgs& a) { return (a.c.blocks() + 255) / 256; }

}  // namespace

uint64_t cache8_attn_workspace(Cache8AttnArgs a, bool want_mass) {
  plan(a);
  uint64_t bytes = 0;
  layout(a, nullptr, want_mass, bytes);
  return bytes;
}

bool cache8_attn_fits(Cache8AttnArgs a) {
  plan(a);
  const long long most = (1LL << 31) - 1;
  return units(a) * a.splits <= most && total_rows(a) <= most &&
         (long long)a.nl * a.c.k.B * a.c.k.H * mass_chunks(a) <= most;
}

cudaError_t launch_cache8_attention(Cache8AttnArgs a, void* workspace, cudaStream_t st) {
  plan(a);
  uint64_t bytes = 0;
  layout(a, reinterpret_cast<char*>(workspace), a.mass != nullptr, bytes);
  cudaError_t e = a.c.k.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
  if (e != cudaSuccess || !a.mass) return e;
  const int chunks = mass_chunks(a);
  cache8_mass_kernel<<<(unsigned)((long long)a.nl * a.c.k.B * a.c.k.H * chunks), 256, 0, st>>>(a, chunks);
  return cudaGetLastError();
}

}  // namespace cg
