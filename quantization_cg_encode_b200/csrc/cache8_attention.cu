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
//           fp16 down to 2^-31 of the row's largest;
//   values  A = 16 channels x 16 tokens of value codes; B = p s_V as two fp16 terms, which are two
//           products, or, for up to four rows (PAIR), columns 0-3 and 4-7 of one, the second term
//           times 2^11.  A weight is off by at most 2^-22 of itself or, where that is more, 2^-37
//           (PAIR: 2^-48) of its row's largest p s_V: half a step of fp16's subnormals.  (Three
//           bf16 terms, which keep all bits of every weight, took 53 us where these take 48, and 85
//           with 16 rows where these take 73.)
// The order of channels within a contraction is free, so ldmatrix moves the bytes as 16-bit
// pairs and no thread exchanges codes with another; B of the second product is the scores'
// layout transposed (movmatrix).
//
// The value scale is a power of two, 2^v: p s_V = 2^(x + v) is kept relative to its own running
// maximum M', so that a row's largest p s_V stands high in fp16's range whatever the scales are, and
// the sum of p relative to M:
//   out = (sum 2^(x + v - M') code) / (sum 2^(x - M)) 2^(M' - M).
// M and M' are whole numbers, so that M' - M is exact; they follow the maxima lazily (they move when
// a value is 2^2 above).
//
// All tiles of the call (every unit's, a unit being the query rows of one layer, sequence and KV
// head, 8 or 16 of them) stand in one row, of which every CTA takes an equal run, so that ragged
// lengths and odd head counts leave no CTA waiting.  Within a run a warp fetches its tiles by
// itself (cp.async, a ring of kStages tiles); at a unit's end the warps merge in shared memory.
// A unit that lies in one run goes out as it is; the pieces of the others go to the workspace
// and a second kernel merges them.  Where units are few and short, a cluster of CTAs takes each
// instead and merges through its shared memory: no looking for a place, no second kernel.
//
// Measured (B200, d = 128, 4 query heads a KV head): 32 layers x 8 heads of 4096 tokens, int8,
// 48 us = 5.6 TB/s; 64 ragged sequences of up to 8192 tokens, e4m3, 114 us = 5.9 TB/s.  A tile costs
// 382 instructions of a warp, of which the codes' conversion is 174 (int8) and products 16.  With
// 16 rows it is 48 products and 470 others, and what bounds it is their latency: the registers leave
// two warps a scheduler, which do not cover the chain from ldmatrix over conversion, product,
// exponential and transposition to the second product (46% of the issue slots, 36% of the tensor
// pipe, 28% of DRAM); 32 rows, 12 sequences of up to 16001 tokens, 73 us with block weights, 1.6 TB/s.
#include <cooperative_groups.h>

#include "cache8.cuh"

namespace cg {

namespace {

constexpr int kWarps = 8;
// CTAs an SM: 16 query rows at d = 128 leave registers for one (at d = 64, without block weights, two
// spill 44 to 56 bytes).  (With their q in shared memory 12
// and 16 warps fit; four draft tokens with block weights took 74 us with 8, 88 with 12, 96 with 16.)
constexpr int ctas_per_sm(int d, int nt) { return d == 128 && nt == 2 ? 1 : 2; }
constexpr int kStages = 3;
constexpr int kSms = 148;               // what the number of CTAs is sized for
constexpr int kLeastRun = 8;            // tiles of a run at least, if units have as many
constexpr int kFewPieces = 4;            // of a unit that are read one after another
constexpr int kMaxCluster = 8;
constexpr int kClusterTiles = 16;       // tiles of a warp in a unit that a cluster takes
// Clusters of a size that a B200 holds at once, at one or two CTAs an SM: its parts' numbers of SMs are no
// multiples of 4 or 8.  Constants, because the workspace size is asked for without a device; where fewer fit, the
// others wait their turn.  (16 units on 8 CTAs each, one an SM, took two turns: 17.2 us, on 4 each 10.2.)
constexpr long long clusters_at_once(int size, int per_sm) {
  return size == 8 ? (per_sm == 2 ? 33 : 15) : size == 4 ? (per_sm == 2 ? 71 : 33) : kSms / size * per_sm;
}
constexpr float kNone = -1.0e30f;       // a running maximum that has seen nothing
constexpr float kDeep = -80.0f;         // the least power of two that a result is multiplied with at once
// p' = 2^kShift p s_V relative to M' is at most 2^(kLag + kShift) = 2^15, as far as fp16 reaches, and the row's
// largest at least 2^12: the farther up, the more bits the weights far below it keep (2^8 and 2^7 lost six, in
// the same time)
constexpr float kLag = 2.0f;            // how far a value may lie above the running maximum
constexpr float kShift = 13.0f;
constexpr float kLow = 2048.0f;         // what the second term is times where it has columns of its own

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
// 2^e / l (0 where l is) in two factors: a result that fp32 holds may need a power of two that it does not
__device__ __forceinline__ float2 last_factor(float e, float l) {
  return make_float2(l > 0.0f ? ex2(fmaxf(e, kDeep)) / l : 0.0f, ex2(fminf(e - kDeep, 0.0f)));
}
// 16 bytes (or 4) from global to shared memory, asynchronously; `bytes` 0 writes zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Where 16-byte piece `ch` of row `row` of a tile stands: rows of 128 (64) bytes, the pieces permuted
// so that the same piece of eight rows falls into different banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int ch) {
  return (uint32_t)(row * D + ((ch ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4));
}
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
// 16-token tiles of a unit of a sequence of n tokens: all that it may see, or all that are listed
__device__ __forceinline__ int unit_tiles(const Cache8AttnArgs& a, int n) {
  return a.n_select ? (n ? a.n_select * (a.c.tb >> 4) : 0) : (n + 15) >> 4;
}

// A unit, its first tile in this CTA, and the CTA's run
struct Place {
  int lz, b, idx, n;             // layer of the call, sequence, unit of the two, tokens of the sequence
  int tile0, tiles;              // first tile, tiles of the unit
  int unit_at;                   // the unit's first tile in the row of all tiles
  int begin, end, run;
};

// A unit whose last piece is in this CTA's run and whose first is not
struct Tail {
  long long row0;  // its first output row
  int step;        // distance of its rows
  int rows;
  int pieces;      // this one included; 0: the CTA has no such unit
  int pad;
};

}  // namespace

template <int D, int CODE, int NT, bool PAIR, bool SPARSE, bool MASS>
__global__ void __launch_bounds__(kWarps * 32, ctas_per_sm(D, NT)) cache8_attn_kernel(Cache8AttnArgs a) {
  constexpr int R = 8 * NT, CH = D / 16, TILE = 16 * D;  // CH: 16-byte pieces of a row
  __shared__ float s_m[kWarps][R], s_mv[kWarps][R], s_l[kWarps][R];
  __shared__ float s_w[kWarps][R], s_fin[R][3];
  __shared__ float s_scale[kWarps][kStages][2];
  __shared__ Place s_place;
  // the warps' tiles [kWarps][kStages][key, value][TILE], then their outputs fp32 [kWarps][R][D]
  extern __shared__ __align__(128) unsigned char dyn[];
  float* s_o = reinterpret_cast<float*>(dyn);
  float* s_part = s_o + kWarps * R * D;  // [R][D + 4]: the CTA's piece of its cluster's unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int H = a.c.k.H, B = a.c.k.B;
  const int rows = SPARSE ? a.gq : a.gq * a.nq;
  const int per_batch = H * (SPARSE ? a.nq : 1) * a.row_tiles;  // units of one layer and sequence
  const int tb_shift = 31 - __clz(a.c.tb);
  // where this lane's pieces stand in a tile: of its copies (32 / CH rows apart: the permutation
  // repeats every second copy), and of its ldmatrix row (rows 0-7, 8-15 of a piece, then of the next)
  const uint32_t ring = smem_u32(dyn) + warp * (kStages * 2 * TILE), scales_at = smem_u32(s_scale[warp]);
  const int lane_row = lane / CH, lane_ch = lane % CH;
  const uint32_t lane_piece[2] = {piece_at<D>(lane_row, lane_ch), piece_at<D>(lane_row + 32 / CH, lane_ch) - 512};
  uint32_t matrix_piece[CH / 2];
#pragma unroll
  for (int jj = 0; jj < CH / 2; ++jj) matrix_piece[jj] = piece_at<D>(lane & 15, 2 * jj + (lane >> 4));
  previous_kernel_done();
  dependents_may_launch();

  // Where the CTA begins: found by one warp and taken from shared memory by all, so that lengths
  // that change meanwhile (they should not) cannot part the threads of a CTA.
  if (warp == 0) {
    Place p = {0, 0, 0, 0, 0, 0, 0, 0, 0, 1};
    if (a.cluster) {  // a cluster is a unit: an equal part of its tiles to every CTA
      const int unit = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
      p.idx = unit % per_batch, p.b = unit / per_batch % B, p.lz = unit / per_batch / B;
      p.n = clamped_len(a, p.b);
      p.tiles = unit_tiles(a, p.n);
      const int part = (p.tiles + a.cluster - 1) / a.cluster;
      p.begin = p.tile0 = min(p.tiles, rank * part);
      p.end = min(p.tiles, p.begin + part);
    } else {
      // The run in the row of all tiles, and the unit in which it begins: the warp sums the batch's
      // tiles, 32 sequences at a time, and finds the place on a second way.
      int batch_tiles = 0, live = 0;  // of one unit of every sequence; sequences that have tokens
      for (int b0 = lane; b0 < B; b0 += 32) {
        const int t = unit_tiles(a, clamped_len(a, b0));
        batch_tiles += t, live += t > 0;
      }
      batch_tiles = __reduce_add_sync(0xffffffffu, batch_tiles), live = __reduce_add_sync(0xffffffffu, live);
      const int layer_tiles = batch_tiles * per_batch, total = layer_tiles * a.nl;
      // A tile for every warp, but no more units to a run than one, on the average, while there are CTAs: units begin
      // and end with latency.  (8 sequences of 16 tokens, 8 heads, in a call for up to 32768: 7.7 us, with 8 units a run 28.4.)
      p.run = max(min(kLeastRun, batch_tiles / max(live, 1)), (total + (int)gridDim.x - 1) / (int)gridDim.x);
      p.begin = (int)min((long long)total, (long long)blockIdx.x * p.run);
      p.end = min(total, p.begin + p.run);
      p.lz = p.begin < p.end ? p.begin / layer_tiles : 0;
      const int rem = p.begin - p.lz * layer_tiles;
      int passed = 0;
      for (int b0 = 0; b0 < B && p.begin < p.end; b0 += 32) {
        const int n = b0 + lane < B ? clamped_len(a, b0 + lane) : 0, v = unit_tiles(a, n) * per_batch;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned in = __ballot_sync(0xffffffffu, rem < passed + incl);
        if (in) {
          const int first = __ffs(in) - 1;  // the first sequence whose tiles end behind the place
          p.b = b0 + first;
          p.n = __shfl_sync(0xffffffffu, n, first);
          p.tiles = unit_tiles(a, p.n);
          passed += __shfl_sync(0xffffffffu, incl - v, first);
          break;
        }
        passed += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (p.tiles) {
        p.idx = (rem - passed) / p.tiles;
        p.unit_at = p.lz * layer_tiles + passed + p.idx * p.tiles;
        p.tile0 = p.begin - p.unit_at;
      } else {
        p.end = p.begin;
      }
    }
    if (lane == 0) s_place = p;
  }
  __syncthreads();
  const int begin = s_place.begin, end_all = s_place.end, run = s_place.run, first_tiles = s_place.tiles;
  if (a.cluster > 1 && begin == end_all)  // a piece without weight
    for (int e = tid; e < R * (D + 4); e += kWarps * 32) s_part[e] = e % (D + 4) < 2 ? kNone : 0.0f;

  Tail tail = {0, 0, 0, 0, 0};
  for (int at = begin; at < end_all;) {
    const int lz = s_place.lz, b = s_place.b, idx = s_place.idx, n = s_place.n;
    const int tile0 = s_place.tile0, tiles = s_place.tiles, unit_at = s_place.unit_at;
    const int rt = idx % a.row_tiles;
    const int qi = SPARSE ? idx / a.row_tiles % a.nq : 0;  // the query token of a sparse unit
    const int h = idx / a.row_tiles / (SPARSE ? a.nq : 1);
    const long long u = ((long long)lz * B + b) * H + h;
    const int tile1 = min(tiles, tile0 + (end_all - at));
    // row r of the unit is row `first + r step` of the [nl][B][hq][nq] rows
    const long long first = u * a.gq * a.nq + qi, step = SPARSE ? a.nq : 1;
    const long long ks_slice = (((long long)(a.l0 + lz) * 2 + 0) * B + b) * H + h;
    const long long vs_slice = (((long long)(a.l0 + lz) * 2 + 1) * B + b) * H + h;
    const uint8_t* kc = a.codes + ks_slice * a.c.k.T * D;
    const uint8_t* vc = a.codes + vs_slice * a.c.k.T * D;
    const float* ks = a.scales + ks_slice * a.c.blocks();
    const float* vs = a.scales + vs_slice * a.c.blocks();
    const int all_see = max(0, n - a.nq + 1 + (SPARSE ? qi : 0));  // tokens that every row sees
    const int end = SPARSE ? all_see : n;                          // tokens that some row sees

    const int* list = SPARSE ? a.sel + (u * a.nq + qi) * a.n_select : nullptr;
    const int n_mine = (tile1 - tile0 - warp + kWarps - 1) / kWarps;  // this warp's tiles: tile0 + warp + i kWarps
    // the block that tile i lies in, and the tile's first token, -1 if it has none to see
    auto listed = [&](int i) { return i < n_mine ? list[((tile0 + warp + i * kWarps) * 16) >> tb_shift] : -1; };
    auto first_token = [&](int i, int blk) {
      const int t = (tile0 + warp + i * kWarps) * 16;
      if (!SPARSE) return t;
      if (blk < 0 || end == 0 || blk > (end - 1) >> tb_shift) return -1;
      const int t0 = (blk << tb_shift) + (t & (a.c.tb - 1));
      return t0 < end ? t0 : -1;
    };
    // A tile to a stage: lane pieces (row, ch), (row + 32 / CH, ch), ...  Codes behind the end may
    // be anything: zeros stand for them.
    const uint8_t* k_lane = kc + lane_row * D + 16 * lane_ch;
    const uint8_t* v_lane = vc + lane_row * D + 16 * lane_ch;
    const float* scale_lane = lane ? vs : ks;
    auto fetch = [&](int i, int t0, int st) {
      if (i < n_mine && t0 >= 0) {
        const uint32_t dst = ring + st * (2 * TILE);
        const long long from = (long long)t0 * D;
        if (t0 + 16 <= end) {
#pragma unroll
          for (int j = 0; j < CH / 2; ++j) {
            copy16(dst + lane_piece[j & 1] + j * 512, k_lane + from + j * 512);
            copy16(dst + lane_piece[j & 1] + j * 512 + TILE, v_lane + from + j * 512);
          }
        } else {
#pragma unroll
          for (int j = 0; j < CH / 2; ++j) {
            const int bytes = t0 + lane_row + j * (32 / CH) < end ? 16 : 0;
            const long long there = bytes ? from + j * 512 : from - lane_row * D;  // else a row that exists
            copy16_or_zero(dst + lane_piece[j & 1] + j * 512, k_lane + there, bytes);
            copy16_or_zero(dst + lane_piece[j & 1] + j * 512 + TILE, v_lane + there, bytes);
          }
        }
        if (lane < 2) copy4(scales_at + st * 8 + lane * 4, scale_lane + (t0 >> tb_shift));
      }
      copies_commit();
    };
    int starts[kStages];  // first tokens of the tiles in flight, by stage
#pragma unroll
    for (int i = 0; i < kStages; ++i) starts[i] = first_token(i, SPARSE ? listed(i) : 0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i, starts[i], i);
    int blk_ahead = SPARSE ? listed(kStages) : 0;

    // q as the scores' B operand, its row's power of two, and what each column's rows see
    uint32_t bq[NT][CH][2];
    float qs[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rt * R + nt * 8 + g;
      const uint16_t* qrow = a.q + (first + (long long)min(r, rows - 1) * step) * D;
      uint2 raw[CH];  // four channels of every piece
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        raw[j] = r < rows ? *reinterpret_cast<const uint2*>(qrow + 16 * j + 4 * c) : make_uint2(0, 0);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(bf16lo(raw[j].x)), fabsf(bf16hi(raw[j].x))), fmaxf(fabsf(bf16lo(raw[j].y)), fabsf(bf16hi(raw[j].y)))));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100) - 14;  // m 2^-e in [2^14, 2^15)
      const float up = two_to(-e);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const float v0 = bf16lo(raw[j].x) * up, v1 = bf16hi(raw[j].x) * up, v2 = bf16lo(raw[j].y) * up, v3 = bf16hi(raw[j].y) * up;
        __half2 f0, f1;  // the order in which codes_to_f16 gives the four codes
        if (CODE == kCache8Int8) {
          f0 = __floats2half2_rn(v0, v2), f1 = __floats2half2_rn(v1, v3);
        } else {
          f0 = __floats2half2_rn(v0, v1), f1 = __floats2half2_rn(v2, v3);
        }
        bq[nt][j][0] = *reinterpret_cast<uint32_t*>(&f0);
        bq[nt][j][1] = *reinterpret_cast<uint32_t*>(&f1);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = 2 * c + j, rc = rt * R + nt * 8 + col;
        qs[nt][j] = two_to(max(__shfl_sync(0xffffffffu, e, 4 * col), -126)) * (a.scale * 1.4426950408889634f);
        const int i = SPARSE ? qi : rc % a.nq;
        lim[nt][j] = rc < rows ? max(0, n - a.nq + 1 + i) : 0x7fffffff;  // columns beyond the rows are not stored
      }
    }

    float o[NT][CH][4];
    float m_run[NT][2], mv_run[NT][2], mv_m[NT][2], l_run[NT][2];  // mv_m: M' - M
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) m_run[nt][j] = mv_run[nt][j] = kNone, mv_m[nt][j] = l_run[nt][j] = 0.0f;
    }

    for (int i0 = 0; i0 < n_mine; i0 += kStages) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        const int i = i0 + st;
        if (i >= n_mine) break;
        const int t0 = starts[st], ahead = (st + kStages - 1) % kStages;
        fetch(i + kStages - 1, starts[ahead], ahead);
        starts[st] = first_token(i + kStages, blk_ahead);
        if (SPARSE) blk_ahead = listed(i + kStages + 1);
        copies_wait<kStages - 1>();
        __syncwarp();
        if (SPARSE && t0 < 0) continue;  // warp-uniform
        uint32_t pieces[CH / 2];  // pieces 2 jj, 2 jj + 1 of this lane's ldmatrix row
#pragma unroll
        for (int jj = 0; jj < CH / 2; ++jj) pieces[jj] = ring + st * (2 * TILE) + matrix_piece[jj];
        const float kscale = s_scale[warp][st][0];
        const float vexp = (float)((int)(__float_as_uint(s_scale[warp][st][1]) >> 23) - 127);

        // scores of 16 tokens x R rows
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
        for (int jj = 0; jj < CH / 2; ++jj) {
          uint32_t w[4];  // token g, g + 8 of piece 2 jj, then of the next
          ldmatrix_x4(w, pieces[jj]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t af[4];
            codes_to_f16<CODE>(w[2 * k], af[0], af[2]);
            codes_to_f16<CODE>(w[2 * k + 1], af[1], af[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt], af, bq[nt][2 * jj + k][0], bq[nt][2 * jj + k][1]);
          }
        }
        // s[nt][0..3]: token g (0, 1) or g + 8 (2, 3), row 2c + (index & 1); x = factor s
        float factor[NT][2], x[NT][4];  // x - M
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            factor[nt][j] = fmaxf(kscale * qs[nt][j], 1.0e-37f);  // (0 times -inf is no -inf)
            if (t0 + 16 > all_see) {
              const int t = t0 + g, see = min(lim[nt][j], end);
              s[nt][j] = t < see ? s[nt][j] : -INFINITY;
              s[nt][j + 2] = t + 8 < see ? s[nt][j + 2] : -INFINITY;
            }
            x[nt][j] = __fmaf_rn(s[nt][j], factor[nt][j], -m_run[nt][j]);
            x[nt][j + 2] = __fmaf_rn(s[nt][j + 2], factor[nt][j], -m_run[nt][j]);
            over |= (!PAIR || c < 2) && fmaxf(x[nt][j], x[nt][j + 2]) > fminf(kLag, mv_m[nt][j] + (kLag - vexp));
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float top = column_max(fmaxf(s[nt][j], s[nt][j + 2])) * factor[nt][j];
              const float m_old = m_run[nt][j], mv_old = mv_run[nt][j];
              const float m = fmaxf(m_old, ceilf(top)), mv = fmaxf(mv_old, ceilf(top) + vexp);
              float fv = ex2(mv_old - mv);
              if (PAIR) {  // columns 4-7 go with 0-3
                const float other = __shfl_xor_sync(0xffffffffu, fv, 2);
                fv = c < 2 ? fv : other;
              }
              m_run[nt][j] = m, mv_run[nt][j] = mv, mv_m[nt][j] = mv - m;
              l_run[nt][j] *= ex2(m_old - m);
              x[nt][j] = __fmaf_rn(s[nt][j], factor[nt][j], -m);
              x[nt][j + 2] = __fmaf_rn(s[nt][j + 2], factor[nt][j], -m);
#pragma unroll
              for (int k = 0; k < CH; ++k) o[nt][k][j] *= fv, o[nt][k][j + 2] *= fv;
            }
        }
        uint32_t bhi[NT][2], blo[NT][2];
        float tile_sum[2 * NT];  // of this lane's two tokens: column (nt, j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float p0 = ex2(x[nt][j]), p1 = ex2(x[nt][j + 2]);
            tile_sum[2 * nt + j] = p0 + p1;
            l_run[nt][j] += tile_sum[2 * nt + j];
            // p s_V relative to M' has an exponential of its own: p times 2^e would be nothing where fp32 has lost p,
            // yet such a token is the row's output where the tokens of weight have values of a far smaller scale
            const float e = (vexp + kShift) - mv_m[nt][j];
            pv[j] = ex2(x[nt][j] + e), pv[j + 2] = ex2(x[nt][j + 2] + e);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const __half2 hi = __floats2half2_rn(pv[2 * j], pv[2 * j + 1]);
            const float2 back = __half22float2(hi);
            const float up = PAIR ? kLow : 1.0f;
            const __half2 lo = __floats2half2_rn((pv[2 * j] - back.x) * up, (pv[2 * j + 1] - back.y) * up);
            if (PAIR) {
              const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&lo), 2);
              bhi[nt][j] = transpose_8x8(c < 2 ? *reinterpret_cast<const uint32_t*>(&hi) : other);
            } else {
              bhi[nt][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&hi));
              blo[nt][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&lo));
            }
          }
        }
        if (MASS) {
          // over the eight lanes of a column, each step halving the columns that a lane keeps: lane g
          // ends with one
          float ref[2 * NT];
#pragma unroll
          for (int k = 0; k < 2 * NT; ++k) ref[k] = m_run[k >> 1][k & 1];
          int o = 4;
#pragma unroll
          for (int half = NT; half >= 1; half >>= 1, o <<= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int k = 0; k < half; ++k) {
              const float keep = up ? tile_sum[half + k] : tile_sum[k], give = up ? tile_sum[k] : tile_sum[half + k];
              tile_sum[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              ref[k] = up ? ref[half + k] : ref[k];
            }
          }
#pragma unroll
          for (; o <= 16; o <<= 1) tile_sum[0] += __shfl_xor_sync(0xffffffffu, tile_sum[0], o);
          // the column that the halving left: its high bit was decided first
          const int col = NT == 2 ? (g & 1) * 2 + (g >> 1 & 1) : g & 1;
          const int r = rt * R + (col >> 1) * 8 + 2 * c + (col & 1);
          if (g < 2 * NT && r < rows)
            a.tile_mass[(first + r) * ((a.max_tokens + 15) >> 4) + (tile0 + warp + i * kWarps)] = make_float2(tile_sum[0], ref[0]);
        }
        // o[channel][row] += codes^T p
#pragma unroll
        for (int jj = 0; jj < CH / 2; ++jj) {
          uint32_t w[4];  // tokens 2c, 2c + 1, then 2c + 8, 2c + 9, of channels 2g, 2g + 1 of piece 2 jj; of the next
          ldmatrix_x4_trans(w, pieces[jj] + TILE);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t af[4];
            if (CODE == kCache8E4m3) w[2 * k] = __byte_perm(w[2 * k], 0, 0x3120), w[2 * k + 1] = __byte_perm(w[2 * k + 1], 0, 0x3120);
            codes_to_f16<CODE>(w[2 * k], af[0], af[1]);
            codes_to_f16<CODE>(w[2 * k + 1], af[2], af[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(o[nt][2 * jj + k], af, bhi[nt][0], bhi[nt][1]);
              if (!PAIR) mma_f16_16816(o[nt][2 * jj + k], af, blo[nt][0], blo[nt][1]);
            }
          }
        }
        __syncwarp();  // the stage is free for the next fetch
      }
    }

    // merge the warps: o relative to the CTA's maxima
    copies_wait<0>();
    __syncthreads();  // the tiles' memory now takes the outputs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float l = column_sum(l_run[nt][j]);
        const int r = nt * 8 + 2 * c + j;
        if (g == 0) s_m[warp][r] = m_run[nt][j], s_mv[warp][r] = mv_run[nt][j], s_l[warp][r] = l;
#pragma unroll
        for (int i = 0; i < CH; ++i)
          *reinterpret_cast<float2*>(&s_o[(warp * R + r) * D + 16 * i + 2 * g]) = make_float2(o[nt][i][j], o[nt][i][j + 2]);
      }
    __syncthreads();
    const bool ends = tile1 == tiles, whole = ends && tile0 == 0 && a.cluster <= 1;
    if (tid < R) {
      float m = kNone, mv = kNone, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][tid]), mv = fmaxf(mv, s_mv[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l = __fmaf_rn(s_l[w][tid], ex2(s_m[w][tid] - m), l);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s_w[w][tid] = ex2(s_mv[w][tid] - mv);
      const float2 last = last_factor(mv - m - kShift, l);
      s_fin[tid][0] = whole ? last.x : m, s_fin[tid][1] = whole ? last.y : mv, s_fin[tid][2] = l;
      if (MASS && whole && rt * R + tid < rows) a.stats[first + rt * R + tid] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
    }
    __syncthreads();
    const int my_rows = min(R, rows - rt * R);
    const long long row0 = first + (long long)rt * R * step;
    // a unit that ends here has its last piece in slot 0, one that does not end its piece in slot 1
    float* part = a.cluster ? s_part : a.part + (long long)(blockIdx.x * 2 + (ends ? 0 : 1)) * R * (D + 4);
    for (int e = tid; e < my_rows * (D / 4); e += kWarps * 32) {
      const int r = e / (D / 4), ch = 4 * (e % (D / 4));
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        float4 v = *reinterpret_cast<const float4*>(&s_o[(w * R + r) * D + ch]);
        if (PAIR) {
          const float4 lo = *reinterpret_cast<const float4*>(&s_o[(w * R + r + 4) * D + ch]);
          constexpr float down = 1.0f / kLow;
          v.x = __fmaf_rn(lo.x, down, v.x), v.y = __fmaf_rn(lo.y, down, v.y), v.z = __fmaf_rn(lo.z, down, v.z), v.w = __fmaf_rn(lo.w, down, v.w);
        }
        const float f = s_w[w][r];
        acc.x = __fmaf_rn(v.x, f, acc.x), acc.y = __fmaf_rn(v.y, f, acc.y), acc.z = __fmaf_rn(v.z, f, acc.z), acc.w = __fmaf_rn(v.w, f, acc.w);
      }
      if (whole) {
        const float f0 = s_fin[r][0], f1 = s_fin[r][1];
        acc.x = acc.x * f0 * f1, acc.y = acc.y * f0 * f1, acc.z = acc.z * f0 * f1, acc.w = acc.w * f0 * f1;
      }
      float* to = whole ? a.out + (row0 + r * step) * D + ch : part + r * (D + 4) + 4 + ch;
      *reinterpret_cast<float4*>(to) = acc;
      if (!whole && ch == 0) *reinterpret_cast<float4*>(part + r * (D + 4)) = make_float4(s_fin[r][0], s_fin[r][1], s_fin[r][2], 0.0f);
    }
    if (ends && !whole) {
      tail.row0 = row0, tail.step = (int)step, tail.rows = my_rows;
      tail.pieces = (int)blockIdx.x - unit_at / run + 1;
    }
    at += tile1 - tile0;
    if (tid == 0 && at < end_all) {  // the next unit
      Place p = s_place;
      p.unit_at += tiles;
      p.tile0 = 0;
      if (++p.idx == per_batch) {
        p.idx = 0;
        do {
          if (++p.b == B) p.b = 0, ++p.lz;
          p.n = p.lz < a.nl ? clamped_len(a, p.b) : 0;
          p.tiles = unit_tiles(a, p.n);
        } while (p.tiles == 0 && p.lz < a.nl);
      }
      s_place = p;
    }
    __syncthreads();  // the outputs' memory takes tiles again, and the next unit is in its place
    if (s_place.tiles == 0) break;
  }
  if (a.cluster > 1) {
    namespace cgs = cooperative_groups;
    cgs::cluster_group cluster = cgs::this_cluster();
    cluster.sync();
    if (first_tiles) {  // the rows in turn, a warp each
      const int lz = s_place.lz, b = s_place.b, unit = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
      const int at = unit % per_batch, rt = at % a.row_tiles, qi = SPARSE ? at / a.row_tiles % a.nq : 0;
      const long long u = ((long long)lz * B + b) * H + at / a.row_tiles / (SPARSE ? a.nq : 1);
      const long long first = u * a.gq * a.nq + qi, step = SPARSE ? a.nq : 1;
      for (int r = rank * kWarps + warp; r < min(R, rows - rt * R); r += a.cluster * kWarps) {
        float m = kNone, mv = kNone, l = 0.0f, acc[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] = 0.0f;
        for (int i = 0; i < a.cluster; ++i) {
          const float* p = cluster.map_shared_rank(s_part, i) + r * (D + 4);
          const float4 st = *reinterpret_cast<const float4*>(p);
          const float m2 = fmaxf(m, st.x), mv2 = fmaxf(mv, st.y), f = ex2(mv - mv2), fi = ex2(st.y - mv2);
          l = l * ex2(m - m2) + st.z * ex2(st.x - m2);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) acc[j] = acc[j] * f + p[4 + 32 * j + lane] * fi;
          m = m2, mv = mv2;
        }
        const long long row = first + (long long)(rt * R + r) * step;
        const float2 last = last_factor(mv - m - kShift, l);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) a.out[row * D + 32 * j + lane] = acc[j] * last.x * last.y;
        if (MASS && lane == 0) a.stats[row] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
      }
    }
    cluster.sync();  // no CTA ends while another reads its piece
  }
  if (tid == 0 && !a.cluster) reinterpret_cast<Tail*>(a.tails)[blockIdx.x] = tail;

  // sequences that are empty: zeros
  const int seq_rows = a.hq * a.nq;
  for (long long e = blockIdx.x; e < (long long)a.nl * B; e += gridDim.x) {
    if (clamped_len(a, (int)(e % B))) continue;
    float4* to = reinterpret_cast<float4*>(a.out + e * seq_rows * D);
    for (int i = tid; i < seq_rows * (D / 4); i += kWarps * 32) to[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
}

// The units whose pieces lie in several runs, from the run in which a unit ends back to the one in
// which it begins.  One CTA a run and row.  How many pieces there are is known here alone (lengths
// live on the device, and a batch may hold one long sequence beside vacant slots).  A few are read one
// after another, a channel a thread; more side by side, first all maxima and sums, a piece a thread,
// then the outputs, which the warps take in turn.  (One head of 32768 tokens, 256 pieces, alone or
// beside 79 vacant slots: 16 us with the attention, 57 one after another.)
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) cache8_combine_kernel(Cache8AttnArgs a, bool mass) {
  constexpr int N = D / 32;
  __shared__ float s_stat[WARPS][3], s_o[WARPS][D];
  const int R = 8 * a.nt, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = blockIdx.y;
  previous_kernel_done();
  dependents_may_launch();
  const Tail tail = reinterpret_cast<const Tail*>(a.tails)[blockIdx.x];
  if (r >= tail.rows || tail.pieces == 0) return;
  auto piece = [&](int i) {  // 0: the last
    return a.part + ((long long)(blockIdx.x - i) * 2 + (i ? 1 : 0)) * R * (D + 4) + r * (D + 4);
  };
  const long long row = tail.row0 + (long long)r * tail.step;
  float m = kNone, mv = kNone, l = 0.0f;
  if (tail.pieces <= kFewPieces) {
    if (tid >= D) return;
    float acc = 0.0f;
    for (int i = 0; i < tail.pieces; ++i) {
      const float4 st = *reinterpret_cast<const float4*>(piece(i));
      const float v = piece(i)[4 + tid];
      const float m2 = fmaxf(m, st.x), mv2 = fmaxf(mv, st.y);
      l = l * ex2(m - m2) + st.z * ex2(st.x - m2);
      acc = acc * ex2(mv - mv2) + v * ex2(st.y - mv2);
      m = m2, mv = mv2;
    }
    const float2 last = last_factor(mv - m - kShift, l);
    a.out[row * D + tid] = acc * last.x * last.y;
    if (mass && tid == 0) a.stats[row] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
    return;
  }
  // a thread's pieces, then a warp's, then all: m, m' and the sum relative to m
  for (int i = tid; i < tail.pieces; i += WARPS * 32) {
    const float4 st = *reinterpret_cast<const float4*>(piece(i));
    const float m2 = fmaxf(m, st.x);
    l = l * ex2(m - m2) + st.z * ex2(st.x - m2);
    m = m2, mv = fmaxf(mv, st.y);
  }
  const float m_warp = warp_max_f32(m), mv_warp = warp_max_f32(mv);
  l *= ex2(m - m_warp);
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_stat[warp][0] = m_warp, s_stat[warp][1] = mv_warp, s_stat[warp][2] = l;
  __syncthreads();
  m = mv = kNone, l = 0.0f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_stat[w][0]), mv = fmaxf(mv, s_stat[w][1]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) l = __fmaf_rn(s_stat[w][2], ex2(s_stat[w][0] - m), l);
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
#pragma unroll 8
  for (int i = warp; i < tail.pieces; i += WARPS) {
    const float* v = piece(i);
    const float f = ex2(v[1] - mv);
    if constexpr (N == 4) {
      const float4 o = *reinterpret_cast<const float4*>(v + 4 + 4 * lane);
      acc[0] = __fmaf_rn(o.x, f, acc[0]), acc[1] = __fmaf_rn(o.y, f, acc[1]), acc[2] = __fmaf_rn(o.z, f, acc[2]), acc[3] = __fmaf_rn(o.w, f, acc[3]);
    } else {
      const float2 o = *reinterpret_cast<const float2*>(v + 4 + 2 * lane);
      acc[0] = __fmaf_rn(o.x, f, acc[0]), acc[1] = __fmaf_rn(o.y, f, acc[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) s_o[warp][N * lane + j] = acc[j];
  __syncthreads();
  const float2 last = last_factor(mv - m - kShift, l);
  for (int ch = tid; ch < D; ch += WARPS * 32) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += s_o[w][ch];
    a.out[row * D + ch] = sum * last.x * last.y;
  }
  if (mass && tid == 0) a.stats[row] = make_float2(m, l > 0.0f ? 1.0f / l : 0.0f);
}

// mass[block] (+)= sum over the unit's rows and the block's tiles of p: 32 blocks a CTA, its warps
// take rows in turn
__global__ void __launch_bounds__(256) cache8_mass_kernel(Cache8AttnArgs a, int chunks) {
  __shared__ float s_sum[8][32];
  const int H = a.c.k.H, B = a.c.k.B, nb = a.c.blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  previous_kernel_done();
  dependents_may_launch();
  const long long u = blockIdx.x / chunks;
  const int blk = (blockIdx.x % chunks) * 32 + lane;
  const int h = (int)(u % H), b = (int)((u / H) % B), lz = (int)(u / H / B);
  const int n = clamped_len(a, b), tpb = a.c.tb >> 4, tiles = (a.max_tokens + 15) >> 4, live = (n + 15) >> 4;
  const int rows = a.gq * a.nq;
  const int i0 = blk * tpb, i1 = min(live, i0 + tpb);
  float sum = 0.0f;
  if (i0 < i1) {
    // four rows' loads together
    for (int r = warp; r < rows; r += 32) {
      float2 st[4], tm[4][4];  // a block has four tiles at most
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool on = r + 8 * k < rows;
        const float2* row = a.tile_mass + (u * rows + (on ? r + 8 * k : r)) * tiles;
        st[k] = on ? a.stats[u * rows + r + 8 * k] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) tm[k][i] = i0 + i < i1 ? row[i0 + i] : make_float2(0.0f, kNone);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) part = __fmaf_rn(tm[k][i].x, ex2(fminf(tm[k][i].y - st[k].x, kLag)), part);
        sum = __fmaf_rn(part, st[k].y, sum);
      }
    }
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (warp || blk >= nb) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) sum += s_sum[w][lane];
  float* at = a.mass + (((long long)(a.l0 + lz) * B + b) * H + h) * nb + blk;
  if (!a.accumulate) {
    *at = sum;
  } else if (i0 < i1) {
    *at += sum;
  }
}

namespace {

long long total_rows(const Cache8AttnArgs& a) { return (long long)a.nl * a.c.k.B * a.hq * a.nq; }
long long units(const Cache8AttnArgs& a) { return (long long)a.nl * a.c.k.B * a.c.k.H * (a.n_select ? a.nq : 1) * a.row_tiles; }

// tiles of the call if every sequence had the longest length
long long tiles_of(const Cache8AttnArgs& a) {
  const double u = (double)units(a), t = a.n_select ? (double)a.n_select * (a.c.tb / 16) : (double)((a.max_tokens + 15) / 16);
  return u * t < 9.0e18 ? units(a) * (long long)t : 1LL << 62;
}

// Rows of a unit: 8 where they are enough, else 16 (two operand columns for one reading of the
// codes).  CTAs: as many as the GPU holds at once, but none with a run shorter than kLeastRun if
// every sequence were of the longest length.
void plan(Cache8AttnArgs& a) {
  const int rows = a.n_select ? a.gq : a.gq * a.nq;
  a.nt = rows > 8 ? 2 : 1;
  a.row_tiles = (rows + 8 * a.nt - 1) / (8 * a.nt);
  const long long most = kSms * ctas_per_sm(a.c.k.d, a.nt);
  const long long runs = (tiles_of(a) + kLeastRun - 1) / kLeastRun;
  a.ctas = (int)(runs < most ? runs : most);
  // clusters: as many CTAs as give each warp one tile of the longest unit, where the GPU holds them
  // all at once.  A unit that is shorter than the others leaves its CTAs idle, so no warp may get
  // more than kClusterTiles, unless all units are of one length (one sequence, or lists) and fill the
  // GPU: there 32 layers of 1024 (2048, 4096) tokens took 18.2 (27.9, 48.1) us, with equal runs and
  // the second kernel 24.3 (33.5, 50.9).
  const long long unit = a.n_select ? (long long)a.n_select * (a.c.tb / 16) : (a.max_tokens + 15) / 16;
  int size = 1;
  while (size < kMaxCluster && size * kWarps < unit && units(a) <= clusters_at_once(2 * size, ctas_per_sm(a.c.k.d, a.nt))) size *= 2;
  const bool even = (a.c.k.B == 1 || a.n_select) && 4 * units(a) * size >= 3 * most;
  // One or two units' clusters leave most SMs idle: equal runs from four tiles a warp on (two heads of 4096,
  // 8192, 16384 tokens: clusters 10.0, 12.8, 18.4 us, runs 9.7, 10.0, 13.0).
  const int tiles = units(a) * size * 8 <= kSms ? kClusterTiles / 4 : kClusterTiles;
  a.cluster = units(a) <= most && (even || unit <= (long long)size * kWarps * tiles) ? size : 0;
  if (a.cluster) a.ctas = (int)units(a) * size;
}

uint64_t round16(uint64_t b) { return (b + 15) & ~15ull; }

void layout(Cache8AttnArgs& a, char* base, bool want_mass, uint64_t& bytes) {
  const uint64_t rows = (uint64_t)total_rows(a);
  uint64_t at = 0;
  a.part = reinterpret_cast<float*>(base);
  at += round16((uint64_t)a.ctas * 2 * 8 * a.nt * (a.c.k.d + 4) * sizeof(float));
  a.tails = base + at;
  at += round16(a.ctas * sizeof(Tail));
  if (want_mass) {
    a.tile_mass = reinterpret_cast<float2*>(base + at);
    at += round16(rows * ((a.max_tokens + 15) / 16) * sizeof(float2));
    a.stats = reinterpret_cast<float2*>(base + at);
    at += round16(rows * sizeof(float2));
  }
  bytes = at;
}

template <int D, int CODE, int NT, bool PAIR, bool SPARSE, bool MASS>
cudaError_t launch_one(const Cache8AttnArgs& a, cudaStream_t st) {
  const size_t tiles = (size_t)kWarps * kStages * 32 * D, outputs = sizeof(float) * 8 * NT * (kWarps * D + D + 4);
  const size_t smem = tiles > outputs ? tiles : outputs;
  auto kern = cache8_attn_kernel<D, CODE, NT, PAIR, SPARSE, MASS>;
  static std::atomic<uint64_t> ready{0};  // a bit a device
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(a.ctas), kWarps * 32, smem, st, a.cluster, a);
}
template <int D, int CODE, int NT, bool PAIR>
cudaError_t launch_kind(const Cache8AttnArgs& a, cudaStream_t st) {
  if (a.n_select) return launch_one<D, CODE, NT, PAIR, true, false>(a, st);
  return a.mass ? launch_one<D, CODE, NT, PAIR, false, true>(a, st) : launch_one<D, CODE, NT, PAIR, false, false>(a, st);
}
template <int D, int CODE>
cudaError_t launch_rows(const Cache8AttnArgs& a, cudaStream_t st) {
  if (a.nt == 2) return launch_kind<D, CODE, 2, false>(a, st);
  return (a.n_select ? a.gq : a.gq * a.nq) <= 4 ? launch_kind<D, CODE, 1, true>(a, st) : launch_kind<D, CODE, 1, false>(a, st);
}
template <int D>
cudaError_t launch_d(const Cache8AttnArgs& a, cudaStream_t st) {
  const cudaError_t e = a.c.code == kCache8Int8 ? launch_rows<D, kCache8Int8>(a, st) : launch_rows<D, kCache8E4m3>(a, st);
  if (e != cudaSuccess || a.cluster) return e;
  const int rows = a.n_select ? a.gq : a.gq * a.nq;
  const dim3 grid(a.ctas, rows < 8 * a.nt ? rows : 8 * a.nt);
  // Eight warps for the merge where sequences of one length, or one that alone holds tokens, are cut into many pieces.
  // (One head of 32768 tokens: eight 16 us, four 27; eight heads 21.8, 22.5; 512 units of 64 ragged sequences 114.2, 113.8;
  // 96 units of 16 rows 73.8, 73.2.)
  const bool many = a.ctas > kFewPieces * units(a) || a.ctas > 64 * (units(a) / a.c.k.B);
  return launch_after(many ? cache8_combine_kernel<D, 8> : cache8_combine_kernel<D, 4>, grid, many ? 256 : 128, 0, st, 1, a, a.mass != nullptr);
}

int mass_chunks(const Cache8AttnArgs& a) { return (a.c.blocks() + 31) / 32; }

}  // namespace

uint64_t cache8_attn_workspace(Cache8AttnArgs a, bool want_mass) {
  plan(a);
  uint64_t bytes = 0;
  layout(a, nullptr, want_mass, bytes);
  return bytes;
}

bool cache8_attn_fits(Cache8AttnArgs a, bool want_mass) {
  const long long most = (1LL << 31) - 1;
  plan(a);
  return tiles_of(a) <= most - (1 << 16) && total_rows(a) <= most && (!want_mass || (long long)a.nl * a.c.k.B * a.c.k.H * mass_chunks(a) <= most);
}

cudaError_t launch_cache8_attention(Cache8AttnArgs a, void* workspace, cudaStream_t st) {
  plan(a);
  uint64_t bytes = 0;
  layout(a, reinterpret_cast<char*>(workspace), a.mass != nullptr, bytes);
  cudaError_t e = a.c.k.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
  if (e != cudaSuccess || !a.mass) return e;
  const int chunks = mass_chunks(a);
  return launch_after(cache8_mass_kernel, dim3((unsigned)((long long)a.nl * a.c.k.B * a.c.k.H * chunks)), 256, 0, st, 1, a, chunks);
}

}  // namespace cg
