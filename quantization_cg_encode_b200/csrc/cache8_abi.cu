// C entry points of the 8-bit block-scaled KV cache (declared in include/cg.h): argument
// validation and dispatch.
#include <cstring>

#include "cache8.cuh"

using namespace cg;

namespace {

cg_status check_cache8(const cg_kv_desc* kv, const cg_cache8_desc* c8) {
  const cg_status st = check_kv(kv);
  if (st != CG_OK) return st;
  if (!c8) return CG_ERR_INVALID;
  if (c8->code != CG_CACHE8_INT8 && c8->code != CG_CACHE8_E4M3) return CG_ERR_INVALID;
  if (c8->tb != 16 && c8->tb != 32 && c8->tb != 64) return CG_ERR_UNSUPPORTED;
  if (kv->tokens % c8->tb != 0) return CG_ERR_INVALID;
  return CG_OK;
}

Cache8 cache8_of(const cg_kv_desc* kv, const cg_cache8_desc* c8) {
  return Cache8{KvGeom{kv->layers, kv->batch, kv->heads, kv->tokens, kv->d_head}, c8->code, c8->tb};
}

cg_status check_layers(const cg_kv_desc* kv, int layer0, int n_layers) {
  return layer0 < 0 || n_layers < 1 || (long long)layer0 + n_layers > kv->layers ? CG_ERR_INVALID : CG_OK;
}

// Query heads and tokens, layers and the longest length of an attention or selection call.
cg_status check_queries(const cg_kv_desc* kv, int q_heads, int q_tokens, int layer0, int n_layers, int max_tokens) {
  if (q_heads <= 0 || q_heads % kv->heads != 0) return CG_ERR_INVALID;
  if (q_heads / kv->heads > kMaxGroup) return CG_ERR_UNSUPPORTED;
  if (q_tokens < 1) return CG_ERR_INVALID;
  if (q_tokens > kMaxQTokens) return CG_ERR_UNSUPPORTED;
  if (max_tokens < 1 || max_tokens > kv->tokens) return CG_ERR_INVALID;
  return check_layers(kv, layer0, n_layers);
}

cg_status check_attn8(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_attn_desc* at, bool want_mass,
                      Cache8AttnArgs& a) {
  cg_status s = check_cache8(kv, c8);
  if (s != CG_OK) return s;
  if (!at) return CG_ERR_INVALID;
  s = check_queries(kv, at->q_heads, at->q_tokens, at->layer0, at->n_layers, at->max_tokens);
  if (s != CG_OK) return s;
  if (!(at->scale > 0.0f) || !(at->scale < 3.0e38f)) return CG_ERR_INVALID;
  if (at->n_select < 0 || at->n_select > kv->tokens / c8->tb) return CG_ERR_INVALID;
  if (at->accumulate != 0 && at->accumulate != 1) return CG_ERR_INVALID;
  if (want_mass && at->n_select) return CG_ERR_UNSUPPORTED;
  std::memset(&a, 0, sizeof(a));
  a.c = cache8_of(kv, c8);
  a.hq = at->q_heads;
  a.gq = at->q_heads / kv->heads;
  a.nq = at->q_tokens;
  a.l0 = at->layer0;
  a.nl = at->n_layers;
  a.max_tokens = at->max_tokens;
  a.n_select = at->n_select;
  a.accumulate = at->accumulate;
  a.scale = at->scale;
  return cache8_attn_fits(a, want_mass) ? CG_OK : CG_ERR_TOO_LARGE;
}

cg_status check_select8(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_select_desc* sd, Cache8SelectArgs& a) {
  cg_status s = check_cache8(kv, c8);
  if (s != CG_OK) return s;
  if (!sd) return CG_ERR_INVALID;
  s = check_queries(kv, sd->q_heads, sd->q_tokens, sd->layer0, sd->n_layers, sd->max_tokens);
  if (s != CG_OK) return s;
  if (sd->n_select < 1 || sd->n_select > kv->tokens / c8->tb) return CG_ERR_INVALID;
  if (sd->sink_blocks < 0 || sd->recent_blocks < 0 || (long long)sd->sink_blocks + sd->recent_blocks > sd->n_select)
    return CG_ERR_INVALID;
  std::memset(&a, 0, sizeof(a));
  a.c = cache8_of(kv, c8);
  a.hq = sd->q_heads;
  a.gq = sd->q_heads / kv->heads;
  a.nq = sd->q_tokens;
  a.l0 = sd->layer0;
  a.nl = sd->n_layers;
  a.max_tokens = sd->max_tokens;
  a.n_select = sd->n_select;
  a.sink = sd->sink_blocks;
  a.recent = sd->recent_blocks;
  return cache8_select_fits(a) ? CG_OK : CG_ERR_TOO_LARGE;
}

bool bad(const void* p) { return !p || !aligned16(p); }

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

cg_cache8_sizes sizes_of(const Cache8& c) {
  cg_cache8_sizes z;
  const uint64_t heads = (uint64_t)c.k.L * c.k.B * c.k.H, nb = (uint64_t)c.blocks();
  z.code_bytes = heads * 2 * c.k.T * c.k.d;
  z.scale_count = heads * 2 * nb;
  z.bound_bytes = heads * nb * 2 * c.k.d;
  z.mass_count = heads * nb;
  return z;
}

}  // namespace

extern "C" {

cg_status cg_cache8_sizes_for(const cg_kv_desc* kv, const cg_cache8_desc* c8, cg_cache8_sizes* out) {
  const cg_status s = check_cache8(kv, c8);
  if (s != CG_OK) return s;
  if (!out) return CG_ERR_INVALID;
  *out = sizes_of(cache8_of(kv, c8));
  return CG_OK;
}

cg_status cg_cache8_append(const cg_kv_desc* kv, const cg_cache8_desc* c8, int32_t layer0, int32_t n_layers, int32_t n_new,
                           const void* new_dev, const int32_t* pos_dev, const int32_t* counts_dev, uint8_t* codes_dev,
                           float* scales_dev, int8_t* bounds_dev, void* stream) {
  cg_status s = check_cache8(kv, c8);
  if (s != CG_OK) return s;
  s = check_layers(kv, layer0, n_layers);
  if (s != CG_OK) return s;
  if (n_new < 0 || n_new > kv->tokens) return CG_ERR_INVALID;
  if (n_new == 0) return CG_OK;
  if (bad(new_dev) || bad(pos_dev) || bad(codes_dev) || bad(scales_dev)) return CG_ERR_INVALID;
  if ((counts_dev && !aligned16(counts_dev)) || (bounds_dev && !aligned16(bounds_dev))) return CG_ERR_INVALID;
  Cache8AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache8_of(kv, c8);
  a.l0 = layer0;
  a.nl = n_layers;
  a.n = n_new;
  a.x = (const uint16_t*)new_dev;
  a.pos = pos_dev;
  a.counts = counts_dev;
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.bounds = bounds_dev;
  if (!cache8_append_fits(a)) return CG_ERR_TOO_LARGE;
  return from_cuda(launch_cache8_append(a, (cudaStream_t)stream));
}

cg_status cg_cache8_attention_workspace_size(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_attn_desc* at,
                                             int32_t want_mass, uint64_t* bytes) {
  Cache8AttnArgs a;
  const cg_status s = check_attn8(kv, c8, at, want_mass != 0, a);
  if (s != CG_OK) return s;
  if (!bytes) return CG_ERR_INVALID;
  *bytes = cache8_attn_workspace(a, want_mass != 0);
  return CG_OK;
}

cg_status cg_cache8_attention(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_attn_desc* at,
                              const void* q_dev, const uint8_t* codes_dev, const float* scales_dev, const int32_t* lens_dev,
                              const int32_t* sel_dev, float* out_dev, float* mass_dev, void* workspace_dev,
                              uint64_t workspace_bytes, void* stream) {
  Cache8AttnArgs a;
  const cg_status s = check_attn8(kv, c8, at, mass_dev != nullptr, a);
  if (s != CG_OK) return s;
  if ((at->n_select != 0) != (sel_dev != nullptr)) return CG_ERR_INVALID;
  if (bad(q_dev) || bad(codes_dev) || bad(scales_dev) || bad(lens_dev) || bad(out_dev) || bad(workspace_dev)) return CG_ERR_INVALID;
  if ((sel_dev && !aligned16(sel_dev)) || (mass_dev && !aligned16(mass_dev))) return CG_ERR_INVALID;
  if (workspace_bytes < cache8_attn_workspace(a, mass_dev != nullptr)) return CG_ERR_INVALID;
  a.q = (const uint16_t*)q_dev;
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.lens = lens_dev;
  a.sel = sel_dev;
  a.out = out_dev;
  a.mass = mass_dev;
  return from_cuda(launch_cache8_attention(a, workspace_dev, (cudaStream_t)stream));
}

cg_status cg_cache8_select_workspace_size(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_select_desc* sd,
                                          uint64_t* bytes) {
  Cache8SelectArgs a;
  const cg_status s = check_select8(kv, c8, sd, a);
  if (s != CG_OK) return s;
  if (!bytes) return CG_ERR_INVALID;
  *bytes = cache8_select_workspace(a);
  return CG_OK;
}

cg_status cg_cache8_select(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_select_desc* sd, const void* q_dev,
                           const float* scales_dev, const int8_t* bounds_dev, const int32_t* lens_dev, int32_t* sel_dev,
                           void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  Cache8SelectArgs a;
  const cg_status s = check_select8(kv, c8, sd, a);
  if (s != CG_OK) return s;
  if (bad(q_dev) || bad(scales_dev) || bad(bounds_dev) || bad(lens_dev) || bad(sel_dev) || bad(workspace_dev)) return CG_ERR_INVALID;
  if (workspace_bytes < cache8_select_workspace(a)) return CG_ERR_INVALID;
  a.q = (const uint16_t*)q_dev;
  a.scales = scales_dev;
  a.bounds = bounds_dev;
  a.lens = lens_dev;
  a.sel = sel_dev;
  a.scores = (float*)workspace_dev;
  return from_cuda(launch_cache8_select(a, (cudaStream_t)stream));
}

cg_status cg_cache8_evict(const cg_kv_desc* kv, const cg_cache8_desc* c8, const cg_cache8_evict_desc* ev, const int32_t* lens_dev,
                          const uint8_t* codes_dev, const float* scales_dev, const int8_t* bounds_dev, const float* mass_dev,
                          const cg_kv_desc* to_kv, uint8_t* to_codes_dev, float* to_scales_dev, int8_t* to_bounds_dev,
                          float* to_mass_dev, int32_t* to_lens_dev, int32_t* kept_dev, void* stream) {
  cg_status s = check_cache8(kv, c8);
  if (s != CG_OK) return s;
  s = check_cache8(to_kv, c8);
  if (s != CG_OK) return s;
  if (!ev) return CG_ERR_INVALID;
  if (to_kv->layers != kv->layers || to_kv->batch != kv->batch || to_kv->heads != kv->heads || to_kv->d_head != kv->d_head)
    return CG_ERR_INVALID;
  s = check_layers(kv, ev->layer0, ev->n_layers);
  if (s != CG_OK) return s;
  if (ev->keep_blocks < 1 || ev->keep_blocks > to_kv->tokens / c8->tb) return CG_ERR_INVALID;
  if (ev->sink_blocks < 0 || ev->recent_blocks < 1 || (long long)ev->sink_blocks + ev->recent_blocks > ev->keep_blocks)
    return CG_ERR_INVALID;
  if (bad(lens_dev) || bad(codes_dev) || bad(scales_dev) || bad(mass_dev) || bad(to_codes_dev) || bad(to_scales_dev) ||
      bad(to_mass_dev) || bad(to_lens_dev) || bad(kept_dev))
    return CG_ERR_INVALID;
  if ((bounds_dev == nullptr) != (to_bounds_dev == nullptr)) return CG_ERR_INVALID;
  if (bounds_dev && (!aligned16(bounds_dev) || !aligned16(to_bounds_dev))) return CG_ERR_INVALID;
  Cache8EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache8_of(kv, c8);
  a.to = cache8_of(to_kv, c8);
  const cg_cache8_sizes z = sizes_of(a.c), tz = sizes_of(a.to);
  // blocks move in parallel: the two caches must be apart
  if (overlap(codes_dev, z.code_bytes, to_codes_dev, tz.code_bytes) ||
      overlap(scales_dev, z.scale_count * 4, to_scales_dev, tz.scale_count * 4) ||
      overlap(mass_dev, z.mass_count * 4, to_mass_dev, tz.mass_count * 4) ||
      overlap(lens_dev, (uint64_t)kv->batch * 4, to_lens_dev, (uint64_t)kv->batch * 4) ||
      (bounds_dev && overlap(bounds_dev, z.bound_bytes, to_bounds_dev, tz.bound_bytes)))
    return CG_ERR_INVALID;
  a.l0 = ev->layer0;
  a.nl = ev->n_layers;
  a.keep = ev->keep_blocks;
  a.sink = ev->sink_blocks;
  a.recent = ev->recent_blocks;
  a.lens = lens_dev;
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.bounds = bounds_dev;
  a.mass = mass_dev;
  a.to_codes = to_codes_dev;
  a.to_scales = to_scales_dev;
  a.to_bounds = to_bounds_dev;
  a.to_mass = to_mass_dev;
  a.to_lens = to_lens_dev;
  a.kept = kept_dev;
  if (!cache8_evict_fits(a)) return CG_ERR_TOO_LARGE;
  return from_cuda(launch_cache8_evict(a, (cudaStream_t)stream));
}

}  // extern "C"
