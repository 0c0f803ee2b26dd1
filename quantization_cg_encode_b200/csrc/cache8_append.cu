// Store of new tokens into the 8-bit block-scaled KV cache.
//
// Every block of tb tokens of one head has one scale s = 2^e, e the least with
// amax |x| <= top 2^e over what the block holds (top = 127 for int8, 448 for e4m3).  New tokens
// that fall into a block with older ones raise its scale when they are larger, and then the
// older codes are rounded anew, c <- rnd(c s_old / s): with powers of two every step is one
// rounding of an exact number, so the codes do not depend on how the arithmetic is done, and an
// e4m3 code loses nothing unless it falls below the normal range.
//
// Memory bound: 2 bytes read and 1 written a value.  A warp takes 16 tokens, which it holds in
// registers between the maximum and the rounding, so that the input is read once (16-byte loads,
// eight in flight); a lane has the same eight channels of every second (fourth) token, so the
// extremes of its channels are packed bf16 operations on the input as it is, and everything else
// that needs them, the block's maximum and the bounds, comes from those: the rounding keeps order.
// Registers are held to eight CTAs an SM, which the loads in flight need, at 16 bytes of spills for
// d = 128 (five CTAs: 150 us, ten: 166 us, where eight took 132).
// Measured (B200, d = 128): 4096 tokens to 32 layers of 8 heads, 268 M values, 118 us = 6.9 TB/s of
// the 3 bytes a value (the last writes stay in L2); one token of 8 sequences to the same layers
// 4.8 us, latency.
#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kWarps = 4;

// c = rnd(v) of four values as bytes.  int8: 1.5 2^23 + v is rounded to a whole number, whose low
// byte is the code.
template <int CODE>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  if constexpr (CODE == kCache8Int8) {
    const float k = 12582912.0f;
    const uint32_t ab = __byte_perm(__float_as_uint(a + k), __float_as_uint(b + k), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c + k), __float_as_uint(d + k), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
  } else {
    uint32_t r;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
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
// Bounds of a channel from its least and largest code value.  e4m3 values are multiples of 2^-9,
// so the quotient by 448 / 127 is rounded outwards in whole numbers.
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
__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
constexpr uint32_t kBf16Inf2 = 0x7F807F80u, kBf16NegInf2 = 0xFF80FF80u;

template <int D, int CODE>
__global__ void __launch_bounds__(kWarps * 32, 8) append_kernel(Cache8AppendArgs a, unsigned window, int tb_shift) {
  constexpr int LPT = D / 8;         // lanes a token
  constexpr int TPL = 32 / LPT;      // tokens a warp loads at once: 2 or 4
  constexpr int NL = 16 / TPL;       // loads of a warp
  __shared__ float s_max[kWarps];
  __shared__ uint4 s_ext[kWarps][LPT][2];         // extremes of the new tokens, bf16 pairs: low, high
  __shared__ float s_old[kWarps][2][D];           // and of the code values of older tokens rounded anew
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpb = 1 << (tb_shift - 4);                // warps of a block: 1, 2 or 4
  // (slice, block of the window: the blocks that n tokens touch at most)
  const unsigned item = blockIdx.x * (kWarps >> (tb_shift - 4)) + (warp >> (tb_shift - 4));
  const int part = warp & (wpb - 1);
  const unsigned H = a.c.k.H, B = a.c.k.B, slices = a.nl * 2 * B * H;
  unsigned sl = item / window;
  const bool inside = sl < slices;
  if (!inside) sl = 0;
  const int w = inside ? (int)(item - sl * window) : 0;
  const unsigned bh = sl / H, ls = bh / B;
  const int h = (int)(sl - bh * H), b = (int)(bh - ls * B), s = (int)(ls & 1u), lz = (int)(ls >> 1);
  previous_kernel_done();
  const int pos = a.pos[b];
  const int cnt = min(a.n, a.counts ? a.counts[b] : a.n);
  // tokens [pos, end) are new; positions off the cache are not written
  const int end = pos < 0 || cnt <= 0 ? 0 : (int)min((long long)pos + cnt, (long long)a.c.k.T);
  const long long b0 = pos < 0 ? 0 : ((long long)(pos >> tb_shift) + w) << tb_shift;  // the block's first token
  const bool live = inside && pos >= 0 && b0 < end;
  if (__syncthreads_or(live) == 0) return;
  const int blk = live ? (int)(b0 >> tb_shift) : 0;
  const long long slice = (((long long)(a.l0 + lz) * 2 + s) * a.c.k.B + b) * a.c.k.H + h;

  const int ch = 8 * (lane % LPT), sub = lane / LPT;  // channels [ch, ch + 8), token of the load
  const int t0 = (live ? (int)b0 : 0) + 16 * part + sub;
  // tokens t0, t0 + TPL, ... of the lane; `all`: the warp's 16 tokens are new
  const int first = (live ? (int)b0 : 0) + 16 * part;
  const bool all = live && first >= pos && first + 16 <= end;
  const uint4* from = reinterpret_cast<const uint4*>(a.x + ((long long)sl * a.n + (t0 - pos)) * D + ch);
  uint4 x[NL];
  unsigned fresh = 0;  // bit i: the lane's token i is new
  if (all) {
#pragma unroll
    for (int i = 0; i < NL; ++i) x[i] = from[i * 32];  // 32 lanes of 16 bytes: TPL tokens
    fresh = (1u << NL) - 1;
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int t = t0 + i * TPL;
      x[i] = make_uint4(0, 0, 0, 0);
      if (live && t >= pos && t < end) x[i] = from[i * 32], fresh |= 1u << i;
    }
  }
  float* sp = a.scales + slice * a.c.blocks() + blk;
  const float was = live && b0 < pos ? *sp : 0.0f;
  const bool has_old = was > 0.0f && was < INFINITY;  // anything else was never stored: the block is empty
  // extremes of the lane's channels over the new tokens
  __nv_bfloat162 lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) lo[j] = as_bf16x2(kBf16Inf2), hi[j] = as_bf16x2(kBf16NegInf2);
  auto widen = [&](const uint4& y) {
    const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) lo[j] = __hmin2(lo[j], as_bf16x2(v[j])), hi[j] = __hmax2(hi[j], as_bf16x2(v[j]));
  };
  if (all) {
#pragma unroll
    for (int i = 0; i < NL; ++i) widen(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (fresh >> i & 1u) widen(x[i]);
  }
  float m = 0.0f;
  if (fresh) {  // (a lane without new tokens has inf and -inf)
    const __nv_bfloat162 x0 = __hmax2(__hmax2(__habs2(lo[0]), __habs2(hi[0])), __hmax2(__habs2(lo[1]), __habs2(hi[1])));
    const __nv_bfloat162 x1 = __hmax2(__hmax2(__habs2(lo[2]), __habs2(hi[2])), __hmax2(__habs2(lo[3]), __habs2(hi[3])));
    const float2 f = __bfloat1622float2(__hmax2(x0, x1));
    m = fmaxf(f.x, f.y);
  }
  m = warp_max_f32(m);
  if (wpb > 1) {
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    for (int i = 0; i < wpb; ++i) m = fmaxf(m, s_max[warp - part + i]);
  }
  int e = cache8_exponent<CODE>(m);
  const bool grew = has_old && two_to(e) > was;
  const float ratio = grew ? was * two_to(-e) : 1.0f;
  if (has_old && !grew) e = (int)(__float_as_uint(was) >> 23) - 127;
  const float inv = two_to(-e);
  uint8_t* row = a.codes + slice * a.c.k.T * D + ch;
  uint2* to = reinterpret_cast<uint2*>(row + (long long)t0 * D);
  auto coded = [&](const uint4& y) {
    uint2 c;
    c.x = pack_codes<CODE>(bf16lo(y.x) * inv, bf16hi(y.x) * inv, bf16lo(y.y) * inv, bf16hi(y.y) * inv);
    c.y = pack_codes<CODE>(bf16lo(y.z) * inv, bf16hi(y.z) * inv, bf16lo(y.w) * inv, bf16hi(y.w) * inv);
    return c;
  };
  if (all) {
#pragma unroll
    for (int i = 0; i < NL; ++i) to[i * 32] = coded(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (fresh >> i & 1u) to[i * 32] = coded(x[i]);
  }
  const bool keys = a.bounds != nullptr && s == 0;
  if (keys) {
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = __hmin2(lo[j], as_bf16x2(__shfl_xor_sync(0xffffffffu, as_u32(lo[j]), o)));
        hi[j] = __hmax2(hi[j], as_bf16x2(__shfl_xor_sync(0xffffffffu, as_u32(hi[j]), o)));
      }
    if (wpb > 1 && sub == 0) {
      s_ext[warp][lane][0] = make_uint4(as_u32(lo[0]), as_u32(lo[1]), as_u32(lo[2]), as_u32(lo[3]));
      s_ext[warp][lane][1] = make_uint4(as_u32(hi[0]), as_u32(hi[1]), as_u32(hi[2]), as_u32(hi[3]));
    }
  }
  if (__syncthreads_or(grew)) {  // the older codes of a block, rounded anew (every warp has read its scale)
    float vlo[8], vhi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) vlo[j] = 448.0f, vhi[j] = -448.0f;
    if (grew) {
      for (int t = t0; t < min(pos, first + 16); t += TPL) {
        uint2* at = reinterpret_cast<uint2*>(row + (long long)t * D);
        uint2 c = *at;
        float v[8];
        unpack_codes<CODE>(c.x, *reinterpret_cast<float(*)[4]>(v));
        unpack_codes<CODE>(c.y, *reinterpret_cast<float(*)[4]>(v + 4));
        c.x = pack_codes<CODE>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
        c.y = pack_codes<CODE>(v[4] * ratio, v[5] * ratio, v[6] * ratio, v[7] * ratio);
        *at = c;
        unpack_codes<CODE>(c.x, *reinterpret_cast<float(*)[4]>(v));
        unpack_codes<CODE>(c.y, *reinterpret_cast<float(*)[4]>(v + 4));
#pragma unroll
        for (int j = 0; j < 8; ++j) vlo[j] = fminf(vlo[j], v[j]), vhi[j] = fmaxf(vhi[j], v[j]);
      }
    }
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        vlo[j] = fminf(vlo[j], __shfl_xor_sync(0xffffffffu, vlo[j], o));
        vhi[j] = fmaxf(vhi[j], __shfl_xor_sync(0xffffffffu, vhi[j], o));
      }
    if (sub == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s_old[warp][0][ch + j] = vlo[j], s_old[warp][1][ch + j] = vhi[j];
    }
    __syncthreads();
  }
  if (live && part == 0) {
    if (lane == 0) *sp = two_to(e);
    if (keys && sub == 0) {
      for (int i = 1; i < wpb; ++i) {
        const uint4 l = s_ext[warp + i][lane][0], h4 = s_ext[warp + i][lane][1];
        const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, hw[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = __hmin2(lo[j], as_bf16x2(lw[j])), hi[j] = __hmax2(hi[j], as_bf16x2(hw[j]));
      }
      // their code values, by the same rounding
      float vlo[8], vhi[8];
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 l0 = __bfloat1622float2(lo[j]), l1 = __bfloat1622float2(lo[j + 1]);
        const float2 h0 = __bfloat1622float2(hi[j]), h1 = __bfloat1622float2(hi[j + 1]);
        unpack_codes<CODE>(pack_codes<CODE>(l0.x * inv, l0.y * inv, l1.x * inv, l1.y * inv), *reinterpret_cast<float(*)[4]>(vlo + 2 * j));
        unpack_codes<CODE>(pack_codes<CODE>(h0.x * inv, h0.y * inv, h1.x * inv, h1.y * inv), *reinterpret_cast<float(*)[4]>(vhi + 2 * j));
      }
      if (grew) {
        for (int i = 0; i < wpb; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) vlo[j] = fminf(vlo[j], s_old[warp + i][0][ch + j]), vhi[j] = fmaxf(vhi[j], s_old[warp + i][1][ch + j]);
        }
      }
      const long long unit = ((long long)(a.l0 + lz) * a.c.k.B + b) * a.c.k.H + h;
      uint2* at = reinterpret_cast<uint2*>(a.bounds + (unit * a.c.blocks() + blk) * 2 * D + ch);
      int l8[8], h8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) l8[j] = low_bound<CODE>(vlo[j]), h8[j] = high_bound<CODE>(vhi[j]);
      if (has_old && !grew) {
        const uint2 pl = at[0], ph = at[D / 8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          l8[j] = min(l8[j], (int)(int8_t)((j < 4 ? pl.x : pl.y) >> (8 * (j & 3))));
          h8[j] = max(h8[j], (int)(int8_t)((j < 4 ? ph.x : ph.y) >> (8 * (j & 3))));
        }
      }
      uint32_t l[2] = {0, 0}, hh[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        l[j >> 2] |= ((uint32_t)l8[j] & 255u) << (8 * (j & 3));
        hh[j >> 2] |= ((uint32_t)h8[j] & 255u) << (8 * (j & 3));
      }
      at[0] = make_uint2(l[0], l[1]);
      at[D / 8] = make_uint2(hh[0], hh[1]);
    }
  }
}

long long append_window(const Cache8AppendArgs& a) { return (a.n + a.c.tb - 2) / a.c.tb + 1; }
long long append_ctas(const Cache8AppendArgs& a) {
  const int per = kWarps / (a.c.tb / 16);
  const long long items = (long long)a.nl * 2 * a.c.k.B * a.c.k.H * append_window(a);
  return (items + per - 1) / per;
}

}  // namespace

bool cache8_append_fits(const Cache8AppendArgs& a) {
  return append_ctas(a) * (kWarps / (a.c.tb / 16)) < (1LL << 31);
}

cudaError_t launch_cache8_append(const Cache8AppendArgs& a, cudaStream_t st) {
  const bool i8 = a.c.code == kCache8Int8;
  auto kern = a.c.k.d == 128 ? (i8 ? append_kernel<128, kCache8Int8> : append_kernel<128, kCache8E4m3>)
                             : (i8 ? append_kernel<64, kCache8Int8> : append_kernel<64, kCache8E4m3>);
  const int tb_shift = a.c.tb == 16 ? 4 : a.c.tb == 32 ? 5 : 6;
  return launch_after(kern, dim3((unsigned)append_ctas(a)), kWarps * 32, 0, st, 1, a, (unsigned)append_window(a), tb_shift);
}

}  // namespace cg
