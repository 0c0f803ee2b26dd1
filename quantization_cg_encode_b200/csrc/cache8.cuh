// The 8-bit KV cache with a scale for each block of tokens and head: what its kernels and
// entry points share.
//
// codes  [L][2][B][H][T][d]      one byte a value: int8, or e4m3
// scales fp32 [L][2][B][H][T/tb] powers of two; a code c of the block stands for s c
// bounds s8 [L][B][H][T/tb][2][d] the least and the largest key code of every channel of the
//        block: int8 codes as they are, e4m3 codes in units of 448 / 127 rounded outwards
// mass   fp32 [L][B][H][T/tb]    the attention weight that the block has drawn
#pragma once
#include <atomic>

#include "cg_kernels.cuh"

namespace cg {

constexpr int kCache8Int8 = 0, kCache8E4m3 = 1;
constexpr int kMaxGroup = 16;    // query heads of one KV head
constexpr int kMaxQTokens = 16;  // query tokens of one sequence

struct Cache8 {
  KvGeom k;
  int code, tb;
  __host__ __device__ int blocks() const { return k.T / tb; }
};

struct Cache8AppendArgs {
  Cache8 c;
  int l0, nl, n;           // layers [l0, l0 + nl), new tokens of every sequence
  const uint16_t* x;       // bf16 [nl][2][B][H][n][d]
  const int* pos;          // [B] where each sequence's new tokens begin
  const int* counts;       // [B] how many of the n it takes, or null: all
  uint8_t* codes;
  float* scales;
  int8_t* bounds;          // or null
};
cudaError_t launch_cache8_append(const Cache8AppendArgs& a, cudaStream_t st);
bool cache8_append_fits(const Cache8AppendArgs& a);

struct Cache8AttnArgs {
  Cache8 c;
  int hq, gq, nq;          // query heads, heads of one KV head, query tokens
  int l0, nl, max_tokens;
  int n_select;            // 0: every token; else blocks listed for each query token
  int accumulate;
  float scale;
  const uint16_t* q;       // bf16 [nl][B][hq][nq][d]
  const uint8_t* codes;
  const float* scales;
  const int* lens;         // [B]
  const int* sel;          // [nl][B][H][nq][n_select]
  float* out;              // fp32 [nl][B][hq][nq][d]
  float* mass;             // or null
  // set by the launcher
  int nt;                  // query rows of a CTA / 8
  int row_tiles, ctas;
  int cluster;             // CTAs that share one unit, 0: every CTA takes an equal run of all tiles
  float* part;             // [cta][2][8 nt][d + 4] {max, max with value scale, sum, -, o[d]}
  void* tails;             // [cta]
  float2* tile_mass;       // [row][16-token tile] {sum, its reference}
  float2* stats;           // [row] {max, 1 / sum}
};
uint64_t cache8_attn_workspace(Cache8AttnArgs a, bool want_mass);
bool cache8_attn_fits(Cache8AttnArgs a, bool want_mass);
cudaError_t launch_cache8_attention(Cache8AttnArgs a, void* workspace, cudaStream_t st);

struct Cache8SelectArgs {
  Cache8 c;
  int hq, gq, nq;
  int l0, nl, max_tokens;
  int n_select, sink, recent;
  const uint16_t* q;
  const float* scales;
  const int8_t* bounds;
  const int* lens;
  int* sel;
  float* scores;           // workspace [nl][B][H][nq][ceil(max_tokens / tb)]
};
uint64_t cache8_select_workspace(const Cache8SelectArgs& a);
bool cache8_select_fits(const Cache8SelectArgs& a);
cudaError_t launch_cache8_select(const Cache8SelectArgs& a, cudaStream_t st);

struct Cache8EvictArgs {
  Cache8 c, to;
  int l0, nl, keep, sink, recent;
  const int* lens;
  const uint8_t* codes;
  const float* scales;
  const int8_t* bounds;    // or null, then to_bounds too
  const float* mass;
  uint8_t* to_codes;
  float* to_scales;
  int8_t* to_bounds;
  float* to_mass;
  int* to_lens;
  int* kept;               // [nl][B][H][keep]
};
bool cache8_evict_fits(const Cache8EvictArgs& a);
cudaError_t launch_cache8_evict(const Cache8EvictArgs& a, cudaStream_t st);

// Lets a kernel use `bytes` of dynamic shared memory, once for each device
inline cudaError_t allow_smem(const void* kern, size_t bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch that may begin while the kernel before it on the stream still runs; such a kernel calls
// previous_kernel_done() in every thread before it touches memory.  `cluster` CTAs form a cluster.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster > 1 ? cluster : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
__device__ __forceinline__ void previous_kernel_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The least e >= -126 with amax <= top 2^e, top = 127 (int8) or 448 (e4m3), for finite amax >= 0.
// With amax = m 2^x, m in [1, 2): 127 = (127/64) 2^6 and 448 = (7/4) 2^8.
template <int CODE>
__device__ __forceinline__ int cache8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = (int)(u >> 23) - 127;  // subnormal amax: -127, and the clamp decides
  const uint32_t man = u & 0x7fffffu;
  const int e = CODE == kCache8Int8 ? x - 6 + (man > 0x7e0000u) : x - 8 + (man > 0x600000u);
  return max(e, -126);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// Four codes of a word as two fp16 pairs, exact.  int8: `lo` holds bytes 0 and 2, `hi` bytes 1
// and 3 (0x6400 | (c + 128) is 1152 + c, from which 1152 goes); e4m3: bytes 0 and 1, 2 and 3.
template <int CODE>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == kCache8Int8) {
    // one logic operation each: (w & m) ^ k with the mask in a register
    uint32_t a, b, m;
    asm("mov.b32 %0, 0x00FF00FF;" : "=r"(m));
    asm("lop3.b32 %0, %1, %2, 0x64806480, 0x6A;" : "=r"(a) : "r"(w), "r"(m));
    asm("lop3.b32 %0, %1, %2, 0x64806480, 0x6A;" : "=r"(b) : "r"(w >> 8), "r"(m));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

}  // namespace cg
