// Store of new tokens into the 8-bit block-scaled KV cache.
//
// Every block of tb tokens of one head has one scale s = 2^e, e the least with
// amax |x| <= top 2^e over what the block holds (top = 127 for int8, 448 for e4m3).  New tokens
// that fall into a block with older ones raise its scale when they are larger, and then the
// older codes are rounded anew, c <- rnd(c s_old / s): with powers of two every step is one
// rounding of an exact number, so the codes do not depend on how the arithmetic is done, and an
// e4m3 code loses nothing unless it falls below the normal range.
//
// Memory bound: 2 bytes read and 1 written a value.  One CTA takes 64 tokens of one or more
// blocks, a warp 16 of them, which it holds in registers between the maximum and the rounding,
// so that the input is read once; a lane has the same four channels of every token, so that the
// per-channel bounds need no exchange within a warp (d = 128).
#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t pack_codes_i8(float a, float b, float c, float d) {
  const uint32_t ia = (uint32_t)__float2int_rn(a) & 255u, ib = (uint32_t)__float2int_rn(b) & 255u;
  const uint32_t ic = (uint32_t)__float2int_rn(c) & 255u, id = (uint32_t)__float2int_rn(d) & 255u;
  return ia | (ib << 8) | (ic << 16) | (id << 24);
}
__device__ __forceinline__ uint32_t pack_codes_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
template <int CODE>
__device__ __forceinline__ uint32_t pack_codes(const float (&v)[4]) {
  return CODE == kCache8Int8 ? pack_codes_i8(v[0], v[1], v[2], v[3]) : pack_codes_e4m3(v[0], v[1], v[2], v[3]);
}
template <int CODE>
__device__ __forceinline__ void unpack_codes(uint32_t w, float (&v)[4]) {
  if constexpr (CODE == kCache8Int8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int)(int8_t)(w >> (8 * i));
  } else {
    uint32_t lo, hi;
    codes_to_f16<CODE>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
}
// Bounds of four channels as int8.  e4m3 values are multiples of 2^-9, so the quotient by
// 448 / 127 is rounded outwards in whole numbers.
__device__ __forceinline__ int floor_div(int a, int b) {
  const int q = a / b;
  return q - (a % b < 0);
}
template <int CODE>
__device__ __forceinline__ int low_bound(float v) {
  return CODE == kCache8Int8 ? (int)v : floor_div((int)(v * 512.0f) * 127, 448 * 512);
}
template <int CODE>
__device__ __forceinline__ int high_bound(float v) {
  return CODE == kCache8Int8 ? (int)v : -floor_div((int)(-v * 512.0f) * 127, 448 * 512);
}

template <int D, int CODE>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(Cache8AppendArgs a) {
  constexpr int LPT = D / 4;         // lanes a token
  constexpr int TPL = 32 / LPT;      // tokens a warp loads at once
  constexpr int NL = 16 / TPL;       // loads of a warp
  __shared__ float s_max[kWarps];
  __shared__ float s_lo[kWarps][D], s_hi[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tb = a.c.tb, wpb = tb >> 4;               // warps of a block: 1, 2 or 4
  const int window = (a.n + tb - 2) / tb + 1;         // blocks that n tokens touch at most
  const long long slices = (long long)a.nl * 2 * a.c.k.B * a.c.k.H;
  const long long item = (long long)blockIdx.x * (kWarps / wpb) + warp / wpb;  // (slice, block of the window)
  const int part = warp % wpb;
  const bool inside = item < slices * window;
  const long long sl = inside ? item / window : 0;
  const int w = inside ? (int)(item % window) : 0;
  int h, b, s, lz;
  {
    long long r = sl;
    h = (int)(r % a.c.k.H), r /= a.c.k.H;
    b = (int)(r % a.c.k.B), r /= a.c.k.B;
    s = (int)(r & 1), lz = (int)(r >> 1);
  }
  const int pos = a.pos[b];
  const int cnt = min(a.n, a.counts ? a.counts[b] : a.n);
  // tokens [pos, end) are new; positions off the cache are not written
  const long long end = pos < 0 || cnt <= 0 ? 0 : min((long long)pos + cnt, (long long)a.c.k.T);
  const int blk = inside && pos >= 0 ? pos / tb + w : 0;
  const long long b0 = (long long)blk * tb;
  const bool live = inside && pos >= 0 && b0 < end;
  bool has_old = live && b0 < pos;
  const long long slice = (((long long)(a.l0 + lz) * 2 + s) * a.c.k.B + b) * a.c.k.H + h;

  const int ch = 4 * (lane % LPT), sub = lane / LPT;  // channels [ch, ch + 4), token of the pair
  const int t0 = (int)b0 + 16 * part + sub;
  uint2 x[NL];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int t = t0 + i * TPL;
    x[i] = make_uint2(0, 0);
    if (live && t >= pos && t < end)
      x[i] = *reinterpret_cast<const uint2*>(a.x + (sl * a.n + (t - pos)) * D + ch);
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    m = fmaxf(m, fmaxf(fabsf(bf16lo(x[i].x)), fabsf(bf16hi(x[i].x))));
    m = fmaxf(m, fmaxf(fabsf(bf16lo(x[i].y)), fabsf(bf16hi(x[i].y))));
  }
  m = warp_max_f32(m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  for (int i = 0; i < wpb; ++i) m = fmaxf(m, s_max[warp - part + i]);
  int e = cache8_exponent<CODE>(m);
  float ratio = 1.0f;
  bool grew = false;
  float* sp = a.scales + slice * a.c.blocks() + blk;
  const float was = has_old ? *sp : 0.0f;
  has_old = was > 0.0f && was < INFINITY;  // anything else was never stored: the block is empty
  if (has_old) {
    grew = two_to(e) > was;
    if (grew) {
      ratio = was * two_to(-e);
    } else {
      e = (int)(__float_as_uint(was) >> 23) - 127;
    }
  }
  const float inv = two_to(-e);
  float lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) lo[j] = 448.0f, hi[j] = -448.0f;
  uint8_t* row = a.codes + slice * a.c.k.T * D + ch;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int t = t0 + i * TPL;
    const bool is_new = live && t >= pos && t < end;
    if (is_new || (grew && t < pos)) {
      float v[4];
      uint32_t* at = reinterpret_cast<uint32_t*>(row + (long long)t * D);
      if (is_new) {
        v[0] = bf16lo(x[i].x) * inv, v[1] = bf16hi(x[i].x) * inv, v[2] = bf16lo(x[i].y) * inv, v[3] = bf16hi(x[i].y) * inv;
      } else {
        unpack_codes<CODE>(*at, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= ratio;
      }
      const uint32_t c = pack_codes<CODE>(v);
      *at = c;
      unpack_codes<CODE>(c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) lo[j] = fminf(lo[j], v[j]), hi[j] = fmaxf(hi[j], v[j]);
    }
  }
  const bool keys = a.bounds != nullptr && s == 0;
  // the block's warps share their extremes; every warp of the CTA comes this way
  if constexpr (TPL == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s_lo[warp][ch + j] = lo[j], s_hi[warp][ch + j] = hi[j];
  }
  __syncthreads();  // also: every warp of the block has read the old scale
  if (live && part == 0 && sub == 0) {
    if (lane == 0) *sp = two_to(e);
    if (keys) {
      for (int i = 1; i < wpb; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = fminf(lo[j], s_lo[warp + i][ch + j]), hi[j] = fmaxf(hi[j], s_hi[warp + i][ch + j]);
      }
      const long long unit = ((long long)(a.l0 + lz) * a.c.k.B + b) * a.c.k.H + h;
      char4* at = reinterpret_cast<char4*>(a.bounds + (unit * a.c.blocks() + blk) * 2 * D + ch);
      int l4[4], h4[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) l4[j] = low_bound<CODE>(lo[j]), h4[j] = high_bound<CODE>(hi[j]);
      if (has_old && !grew) {
        const char4 pl = at[0], ph = at[D / 4];
        l4[0] = min(l4[0], (int)pl.x), l4[1] = min(l4[1], (int)pl.y), l4[2] = min(l4[2], (int)pl.z), l4[3] = min(l4[3], (int)pl.w);
        h4[0] = max(h4[0], (int)ph.x), h4[1] = max(h4[1], (int)ph.y), h4[2] = max(h4[2], (int)ph.z), h4[3] = max(h4[3], (int)ph.w);
      }
      at[0] = make_char4(l4[0], l4[1], l4[2], l4[3]);
      at[D / 4] = make_char4(h4[0], h4[1], h4[2], h4[3]);
    }
  }
}

long long append_ctas(const Cache8AppendArgs& a) {
  const int per = kWarps / (a.c.tb / 16), window = (a.n + a.c.tb - 2) / a.c.tb + 1;
  const long long items = (long long)a.nl * 2 * a.c.k.B * a.c.k.H * window;
  return (items + per - 1) / per;
}

}  // namespace

bool cache8_append_fits(const Cache8AppendArgs& a) { return append_ctas(a) < (1LL << 31); }

cudaError_t launch_cache8_append(const Cache8AppendArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)append_ctas(a);
  const bool i8 = a.c.code == kCache8Int8;
  if (a.c.k.d == 128)
    i8 ? append_kernel<128, kCache8Int8><<<grid, kWarps * 32, 0, st>>>(a) : append_kernel<128, kCache8E4m3><<<grid, kWarps * 32, 0, st>>>(a);
  else
    i8 ? append_kernel<64, kCache8Int8><<<grid, kWarps * 32, 0, st>>>(a) : append_kernel<64, kCache8E4m3><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace cg
