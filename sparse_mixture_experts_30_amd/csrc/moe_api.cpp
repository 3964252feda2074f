// C ABI of libmoe: argument validation, workspace layout and launch order.
// Every check happens on the host before anything is enqueued.
#include "moe.h"

#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <mutex>
#include <new>

#include "moe_internal.hpp"
#include "backward.hpp"
#include "block.hpp"
#include "dense.hpp"
#include "grads.hpp"

namespace {

thread_local char g_msg[512] = "";

moe_status fail(moe_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

moe_status hip_fail(hipError_t e, const char* where) {
  return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// e4m3 weights, with block scales a / 448 or powers of two.
bool is_fp8(moe_dtype w) { return w == MOE_FP8_E4M3 || w == MOE_FP8_E4M3_E8M0; }

// 4-bit weights with bf16 scales per group of 128 or 32 inputs.
bool is_int4(moe_dtype w) { return w == MOE_INT4_G128 || w == MOE_INT4_G32; }
int int4_group(moe_dtype w) { return w == MOE_INT4_G32 ? 32 : 128; }

// 8-bit integer weights with an fp32 scale per output channel.
bool is_int8(moe_dtype w) { return w == MOE_INT8; }
constexpr int kInt8MaxK = 131072;   // 127^2 k stays below 2^31

// Weight types whose kernels read tokens quantised beforehand.
bool quantises_act(moe_dtype w) { return is_fp8(w) || is_int8(w); }

// Configurations of the expert and layer backward: integer weights are for
// serving and have none.
bool has_backward(const moe_config* c) {
  return c->act_dtype == MOE_BF16 && (c->weight_dtype == MOE_BF16 || is_fp8(c->weight_dtype));
}

// Shape checks shared by every entry point.
moe_status check_cfg(const moe_config* c) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
  const int H = c->hidden_size, E = c->n_routed_experts, G = c->n_group, TG = c->topk_group,
            K = c->num_experts_per_tok, I = c->moe_intermediate_size,
            Is = c->shared_intermediate_size;
  if (H <= 0 || E <= 0 || G <= 0 || I <= 0 || Is < 0)
    return fail(MOE_ERR_INVALID_ARG, "sizes must be positive (H=%d E=%d G=%d I=%d Is=%d)", H, E, G,
                I, Is);
  if (E % G != 0 || E / G < 2)
    return fail(MOE_ERR_INVALID_ARG, "n_routed_experts %% n_group must be 0 with >= 2 experts per "
                "group (E=%d G=%d)", E, G);
  if (TG < 1 || TG > G)
    return fail(MOE_ERR_INVALID_ARG, "topk_group must be in [1, n_group] (TG=%d G=%d)", TG, G);
  if (K < 1 || K > E)
    return fail(MOE_ERR_INVALID_ARG, "num_experts_per_tok must be in [1, E] (K=%d E=%d)", K, E);
  if (!(isfinite(c->routed_scaling_factor) && c->routed_scaling_factor > 0.0f))
    return fail(MOE_ERR_INVALID_ARG, "routed_scaling_factor must be finite and > 0");
  const moe_dtype a = c->act_dtype, w = c->weight_dtype;
  if (a != MOE_F32 && a != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "act_dtype must be MOE_F32 or MOE_BF16");
  if (w != MOE_F32 && w != MOE_BF16 && !is_fp8(w) && !is_int4(w) && !is_int8(w))
    return fail(MOE_ERR_INVALID_ARG, "unknown weight_dtype");
  // Valid for the method, not handled by these kernels:
  if (E > 512) return fail(MOE_ERR_UNSUPPORTED, "n_routed_experts > 512");
  if (G > 64) return fail(MOE_ERR_UNSUPPORTED, "n_group > 64");
  if (K > 64) return fail(MOE_ERR_UNSUPPORTED, "num_experts_per_tok > 64");
  if ((a == MOE_F32) != (w == MOE_F32))
    return fail(MOE_ERR_UNSUPPORTED, "fp32 activations need fp32 weights and vice versa");
  const int mult = is_fp8(w) || is_int4(w) || is_int8(w) ? 128 : 64;
  if (H % mult || I % mult || Is % mult)
    return fail(MOE_ERR_UNSUPPORTED, "hidden and FFN sizes must be multiples of %d", mult);
  if (is_int8(w) && (H > kInt8MaxK || I > kInt8MaxK || Is > kInt8MaxK))
    return fail(MOE_ERR_UNSUPPORTED, "8-bit integer products take sizes up to %d", kInt8MaxK);
  return MOE_OK;
}

moe_status check_T(int64_t T, const moe_config* c) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T < 0");
  if (T * (int64_t)c->num_experts_per_tok > 0x7fffffffLL || T > 0x7fffffffLL)
    return fail(MOE_ERR_UNSUPPORTED, "T * top_k exceeds int32 indexing");
  if (is_int8(c->weight_dtype) &&
      T * ((int64_t)c->num_experts_per_tok + 1) > moe::quantize_rows_int8_max())
    return fail(MOE_ERR_UNSUPPORTED, "T * (top_k + 1): one launch quantises %lld rows",
                (long long)moe::quantize_rows_int8_max());
  return MOE_OK;
}

size_t act_bytes(const moe_config* c) { return c->act_dtype == MOE_BF16 ? 2 : 4; }

// Workspace segments (byte offsets, 256-aligned).
struct Layout {
  size_t err, part, gsplit, idx, w, counts, offsets, perm, pos, hist, tiles, tiles2, h, hq, hs,
      xq, xs, y, ys, flags, total;
  int ksplit;
  bool decode;   // decode routing (gate, selection, permutation, tile list in three launches)
};

// The segments of the expert products themselves: h of N routed and T shared
// rows, its codes and scales, the tokens' codes and scales.
template <class Take>
void ffn_segments(Layout& L, const moe_config* c, int64_t N, int64_t T, Take take) {
  const int64_t H = c->hidden_size, I = c->moe_intermediate_size, Is = c->shared_intermediate_size;
  const size_t hel = (size_t)(N * I + T * Is);
  L.hq = L.hs = L.xq = L.xs = 0;
  if (is_fp8(c->weight_dtype)) {
    L.h = take(hel);
    L.hs = take(hel / 128 * 4);
    L.xq = take((size_t)T * H);
    L.xs = take((size_t)T * H / 128 * 4);
  } else if (is_int8(c->weight_dtype)) {
    L.h = take(hel * 4);   // fp32
    L.hq = take(hel);
    L.hs = take((size_t)(N + T) * 4);
    L.xq = take((size_t)T * H);
    L.xs = take((size_t)T * 4);
  } else {
    L.h = take(hel * act_bytes(c));
  }
}

Layout layout(const moe_config* c, int64_t T) {
  Layout L{};
  const int64_t H = c->hidden_size, E = c->n_routed_experts, K = c->num_experts_per_tok,
                I = c->moe_intermediate_size, Is = c->shared_intermediate_size;
  const int64_t N = T * K;
  L.ksplit = c->act_dtype == MOE_BF16 ? moe::gate_ksplit(T, (int)H, (int)E) : 1;
  L.decode = moe::decode_route_ok(T, (int)H, (int)E, (int)K);
  const int64_t nparts = std::max<int64_t>(L.ksplit, L.decode ? moe::decode_ksplit((int)H, (int)E) : 1);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o += up(bytes);
    return at;
  };
  L.err = take(sizeof(int32_t));
  L.part = take((size_t)nparts * T * E * 4);
  L.gsplit = c->act_dtype == MOE_BF16 ? take(moe::gate_split_bytes((int)H, (int)E)) : o;
  L.idx = take((size_t)N * 4);
  L.w = take((size_t)N * 4);
  L.counts = take((size_t)E * 4);
  L.offsets = take((size_t)(E + 1) * 4);
  L.perm = take((size_t)N * 4);
  L.pos = take((size_t)N * 4);
  L.hist = take((size_t)moe::permute_nblk(N) * (E + 1) * 4);
  moe::FfnDims d{T, N, (int)H, (int)I, (int)Is, (int)E, (int)K};
  const size_t tiles = moe::ffn_tiles_bytes(d);
  L.tiles = take(tiles);
  L.tiles2 = take(tiles);   // the shared expert's list on a second stream
  ffn_segments(L, c, N, T, take);
  L.y = take((size_t)N * H * act_bytes(c));
  L.ys = take((size_t)T * H * act_bytes(c));
  // completion flags of the one-launch decode layer (bf16)
  L.flags = (L.decode && c->act_dtype == MOE_BF16 && c->weight_dtype == MOE_BF16)
                ? take(moe::decode_layer_flags_bytes((int)H, (int)E, (int)K, (int)I, (int)Is))
                : o;
  L.total = o;
  return L;
}

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

moe_status check_ws(void* ws, size_t ws_bytes, const Layout& L) {
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign)
    return fail(MOE_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kAlign);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, L.total);
  return MOE_OK;
}

#define CHECK(expr)                  \
  do {                               \
    moe_status _s = (expr);          \
    if (_s != MOE_OK) return _s;     \
  } while (0)
#define NONNULL(p)                                                     \
  do {                                                                 \
    if (!(p)) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);      \
  } while (0)
// Rows and packed weights are read 16 bytes at a time.
#define ALIGNED16(p)                                                                \
  do {                                                                              \
    if ((uintptr_t)(p) % 16)                                                        \
      return fail(MOE_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p);           \
  } while (0)
#define HIPCALL(expr, where)                              \
  do {                                                    \
    hipError_t _e = (expr);                               \
    if (_e != hipSuccess) return hip_fail(_e, where);     \
  } while (0)

// ---- the pieces, after validation -------------------------------------------

moe_status run_gate(const moe_config* c, int64_t T, const void* x, const float* gate_w,
                    const float* bias, float* logits, int32_t* idx, float* w, void* ws,
                    const Layout& L, hipStream_t s) {
  float* part = at<float>(ws, L.part);
  const bool bf16 = c->act_dtype == MOE_BF16;
  if (bf16 && moe::gate_use_fused(T, c->hidden_size, c->n_routed_experts, c->n_group,
                                  c->topk_group, c->num_experts_per_tok)) {
    HIPCALL(moe::launch_gate_select_fused((const uint16_t*)x, gate_w, at<void>(ws, L.gsplit), bias,
                                          logits, idx, w, T, c->hidden_size,
                                          c->n_routed_experts, c->n_group, c->topk_group,
                                          c->num_experts_per_tok, c->routed_scaling_factor, s),
            "gate and selection");
    return MOE_OK;
  }
  HIPCALL(moe::launch_gate_logits(x, bf16, gate_w, at<void>(ws, L.gsplit), part, T,
                                  c->hidden_size, c->n_routed_experts, L.ksplit, s),
          "gate logits");
  HIPCALL(moe::launch_select(part, L.ksplit, bias, logits, idx, w, T, c->n_routed_experts,
                             c->n_group, c->topk_group, c->num_experts_per_tok,
                             c->routed_scaling_factor, s),
          "select");
  return MOE_OK;
}

moe_status run_permute(const moe_config* c, int64_t T, const int32_t* idx, int32_t* counts,
                       int32_t* offsets, int32_t* perm, int32_t* pos, void* ws, const Layout& L,
                       hipStream_t s) {
  HIPCALL(moe::launch_permute(idx, T * c->num_experts_per_tok, c->n_routed_experts,
                              at<int32_t>(ws, L.hist), counts, offsets, perm, pos,
                              at<int32_t>(ws, L.err), s),
          "permute");
  return MOE_OK;
}

// Quantises T token rows of x into the workspace, as the weights' kernels read them.
moe_status quantise_tokens(const moe_config* c, int64_t T, const void* x, void* ws,
                           const Layout& L, hipStream_t s) {
  if (is_int8(c->weight_dtype))
    HIPCALL(moe::launch_quantize_rows_int8((const uint16_t*)x, T, c->hidden_size, at<int8_t>(ws, L.xq),
                                           at<float>(ws, L.xs), s),
            "quantise x");
  else
    HIPCALL(moe::launch_quant_rows((const uint16_t*)x, T, c->hidden_size, at<uint8_t>(ws, L.xq),
                                   at<float>(ws, L.xs), c->weight_dtype == MOE_FP8_E4M3_E8M0, s),
            "quantise x");
  return MOE_OK;
}

// groups: which groups to compute (moe::kGroupRouted / kGroupShared);
// tiles: the tile list to use (built here unless tiles_ready); quantize: e4m3
// and 8-bit integer weights only, quantise x first (else the workspace's xq /
// xs already hold it, or given_q / given_s do).
moe_status run_ffn(const moe_config* c, int64_t T, const void* x, const int32_t* perm,
                   const int32_t* offsets, const moe_weights* wt, void* y, void* ys, void* ws,
                   const Layout& L, hipStream_t s, int groups = moe::kGroupsAll,
                   int32_t* tiles = nullptr, bool tiles_ready = false, bool quantize = true,
                   const uint8_t* given_q = nullptr, const float* given_s = nullptr) {
  moe::FfnDims d{T, T * c->num_experts_per_tok, c->hidden_size, c->moe_intermediate_size,
                 c->shared_intermediate_size, c->n_routed_experts, c->num_experts_per_tok};
  if (!(groups & moe::kGroupRouted) && !perm) d.N = 0;   // a dense layer: no routed rows at all
  d.groups = groups;
  d.tiles_ready = tiles_ready;
  if (!tiles) tiles = at<int32_t>(ws, L.tiles);
  switch (c->weight_dtype) {
    case MOE_F32:
      HIPCALL(moe::launch_ffn_f32(d, (const float*)x, perm, offsets, (const float*)wt->w13,
                                  (const float*)wt->w2, (const float*)wt->ws13,
                                  (const float*)wt->ws2, at<float>(ws, L.h), (float*)y,
                                  (float*)ys, s),
              "ffn f32");
      break;
    case MOE_BF16:
      if (wt->packed) {
        HIPCALL(moe::launch_ffn_bf16_packed(d, (const uint16_t*)x, perm, offsets, wt->w13, wt->w2,
                                            wt->ws13, wt->ws2, at<uint16_t>(ws, L.h),
                                            tiles, (uint16_t*)y,
                                            (uint16_t*)ys, s),
                "ffn bf16 packed");
      } else {
        HIPCALL(moe::launch_ffn_bf16(d, (const uint16_t*)x, perm, offsets,
                                     (const uint16_t*)wt->w13, (const uint16_t*)wt->w2,
                                     (const uint16_t*)wt->ws13, (const uint16_t*)wt->ws2,
                                     at<uint16_t>(ws, L.h), tiles,
                                     (uint16_t*)y, (uint16_t*)ys, s),
                "ffn bf16");
      }
      break;
    case MOE_INT4_G128:
    case MOE_INT4_G32:
      HIPCALL(moe::launch_ffn_int4(d, int4_group(c->weight_dtype), (const uint16_t*)x, perm,
                                   offsets, wt->w13, wt->w2, wt->ws13, wt->ws2,
                                   at<uint16_t>(ws, L.h), (uint16_t*)y, (uint16_t*)ys, s),
              "ffn int4");
      break;
    case MOE_INT8: {
      const uint8_t* xq = given_q ? given_q : at<uint8_t>(ws, L.xq);
      const float* xs = given_q ? given_s : at<float>(ws, L.xs);
      if (quantize) CHECK(quantise_tokens(c, T, x, ws, L, s));
      HIPCALL(moe::launch_ffn_int8(d, (const int8_t*)xq, xs, perm, offsets, wt->w13, wt->w13_scale,
                                   wt->w2, wt->w2_scale, wt->ws13, wt->ws13_scale, wt->ws2,
                                   wt->ws2_scale, at<float>(ws, L.h), at<int8_t>(ws, L.hq),
                                   at<float>(ws, L.hs), (uint16_t*)y, (uint16_t*)ys, s),
              "ffn int8");
      break;
    }
    case MOE_FP8_E4M3_E8M0: {
      const uint8_t* xq = given_q ? given_q : at<uint8_t>(ws, L.xq);
      const float* xs = given_q ? given_s : at<float>(ws, L.xs);
      if (quantize) CHECK(quantise_tokens(c, T, x, ws, L, s));
      HIPCALL(moe::launch_ffn_fp8_mx(d, xq, xs, perm, offsets, wt->w13, wt->w13_scale, wt->w2,
                                     wt->w2_scale, wt->ws13, wt->ws13_scale, wt->ws2,
                                     wt->ws2_scale, at<uint8_t>(ws, L.h), at<float>(ws, L.hs),
                                     tiles, (uint16_t*)y, (uint16_t*)ys, s),
              "ffn fp8 (power-of-two scales)");
      break;
    }
    case MOE_FP8_E4M3: {
      const uint8_t* xq = given_q ? given_q : at<uint8_t>(ws, L.xq);
      const float* xs = given_q ? given_s : at<float>(ws, L.xs);
      if (quantize) CHECK(quantise_tokens(c, T, x, ws, L, s));
      if (wt->packed) {
        HIPCALL(moe::launch_ffn_fp8_packed(d, xq, xs, perm, offsets, wt->w13, wt->w13_scale,
                                           wt->w2, wt->w2_scale, wt->ws13, wt->ws13_scale, wt->ws2,
                                           wt->ws2_scale, at<uint8_t>(ws, L.h), at<float>(ws, L.hs),
                                           tiles, (uint16_t*)y, (uint16_t*)ys,
                                           s),
                "ffn fp8 packed");
        break;
      }
      HIPCALL(moe::launch_ffn_fp8(d, xq, xs, perm, offsets, (const uint8_t*)wt->w13, wt->w13_scale,
                                  (const uint8_t*)wt->w2, wt->w2_scale, (const uint8_t*)wt->ws13,
                                  wt->ws13_scale, (const uint8_t*)wt->ws2, wt->ws2_scale,
                                  at<uint8_t>(ws, L.h), at<float>(ws, L.hs),
                                  tiles, (uint16_t*)y, (uint16_t*)ys, s),
              "ffn fp8");
      break;
    }
  }
  return MOE_OK;
}

// dense: the shared expert's matrices only.
moe_status check_weights(const moe_config* c, const moe_weights* w, bool need_gate,
                         bool dense = false) {
  NONNULL(w);
  if (w->packed != 0 && w->packed != 1)
    return fail(MOE_ERR_INVALID_ARG, "moe_weights.packed must be 0 or 1");
  if (w->packed && c->weight_dtype == MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "the packed weight layout is for bf16 and fp8 weights");
  if (!w->packed && is_int4(c->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "4-bit weights must be packed (moe_pack_quantized)");
  if (!w->packed && is_int8(c->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "8-bit integer weights must be packed (moe_pack_weight)");
  if (need_gate) {
    NONNULL(w->gate_w);
    NONNULL(w->bias);
  }
  if (!dense) {
    NONNULL(w->w13);
    NONNULL(w->w2);
  }
  const bool scaled = is_fp8(c->weight_dtype) || is_int8(c->weight_dtype);
  if (c->weight_dtype == MOE_FP8_E4M3_E8M0 && !w->packed)
    return fail(MOE_ERR_UNSUPPORTED, "e4m3 weights with power-of-two scales must be packed "
                "(moe_pack_weight)");
  if (scaled && !dense) {
    NONNULL(w->w13_scale);
    NONNULL(w->w2_scale);
  }
  if (c->shared_intermediate_size > 0) {
    NONNULL(w->ws13);
    NONNULL(w->ws2);
    if (scaled) {
      NONNULL(w->ws13_scale);
      NONNULL(w->ws2_scale);
    }
  }
  if (is_int4(c->weight_dtype) || is_int8(c->weight_dtype)) {
    if (!dense) {
      ALIGNED16(w->w13);
      ALIGNED16(w->w2);
    }
    if (c->shared_intermediate_size > 0) {
      ALIGNED16(w->ws13);
      ALIGNED16(w->ws2);
    }
  }
  if (is_int8(c->weight_dtype)) {   // four channels' scales are read together
    if (!dense) {
      ALIGNED16(w->w13_scale);
      ALIGNED16(w->w2_scale);
    }
    if (c->shared_intermediate_size > 0) {
      ALIGNED16(w->ws13_scale);
      ALIGNED16(w->ws2_scale);
    }
  }
  return MOE_OK;
}


// Events that order a call's work across its two streams, one pair per
// device and host thread (created on first use, reused by every later call:
// a wait takes the event's most recent record at the time it is enqueued).
struct ForkJoin {
  hipEvent_t fork = nullptr, join = nullptr;
};

hipError_t fork_join_events(ForkJoin** out) {
  constexpr int kMaxDevices = 64;
  thread_local ForkJoin ev[kMaxDevices];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  ForkJoin& f = ev[dev];
  if (!f.fork && (e = hipEventCreateWithFlags(&f.fork, hipEventDisableTiming)) != hipSuccess)
    return e;
  if (!f.join && (e = hipEventCreateWithFlags(&f.join, hipEventDisableTiming)) != hipSuccess)
    return e;
  *out = &f;
  return hipSuccess;
}

// The layer on stream s.  With s2 (not null), the shared expert's GEMMs run
// on s2, forked from s at the start and joined back before the combine.
moe_status forward_impl(const moe_config* cfg, int64_t T, const void* x, const moe_weights* w,
                        void* out, float* logits, int32_t* topk_idx, float* topk_w,
                        int32_t* counts, int32_t* perm, void* ws, size_t ws_bytes,
                        hipStream_t s, hipStream_t s2, bool one_launch = false) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(out);
  CHECK(check_weights(cfg, w, true));
  if (is_int4(cfg->weight_dtype) || is_int8(cfg->weight_dtype)) ALIGNED16(x);
  const Layout L = layout(cfg, T);
  CHECK(check_ws(ws, ws_bytes, L));
  if (one_launch &&
      !(L.decode && cfg->act_dtype == MOE_BF16 && cfg->weight_dtype == MOE_BF16 && w->packed &&
        moe::decode_layer_ok(T, cfg->hidden_size, cfg->n_routed_experts,
                             cfg->num_experts_per_tok, cfg->moe_intermediate_size,
                             cfg->shared_intermediate_size)))
    return fail(MOE_ERR_UNSUPPORTED,
                "the one-launch decode layer takes 1 <= T <= %d bf16 tokens and packed bf16 "
                "weights", moe::kDecodeMaxT);
  int32_t* idx = topk_idx ? topk_idx : at<int32_t>(ws, L.idx);
  float* wt = topk_w ? topk_w : at<float>(ws, L.w);
  int32_t* cnt = counts ? counts : at<int32_t>(ws, L.counts);
  int32_t* pm = perm ? perm : at<int32_t>(ws, L.perm);
  int32_t* offs = at<int32_t>(ws, L.offsets);
  int32_t* pos = at<int32_t>(ws, L.pos);
  int32_t* tiles = at<int32_t>(ws, L.tiles);
  void* y = at<void>(ws, L.y);
  const bool sh = cfg->shared_intermediate_size > 0;
  void* ys = sh ? at<void>(ws, L.ys) : nullptr;
  // The fp32 expert kernels compute every group in one launch.
  const bool split = s2 && sh && cfg->weight_dtype != MOE_F32;

  ForkJoin* ev = nullptr;
  if (split) {
    HIPCALL(fork_join_events(&ev), "fork/join events");
    if (quantises_act(cfg->weight_dtype))   // once, before the fork, for both streams
      CHECK(quantise_tokens(cfg, T, x, ws, L, s));
    HIPCALL(hipEventRecord(ev->fork, s), "fork");
    HIPCALL(hipStreamWaitEvent(s2, ev->fork, 0), "fork");
    CHECK(run_ffn(cfg, T, x, pm, offs, w, y, ys, ws, L, s2, moe::kGroupShared,
                  at<int32_t>(ws, L.tiles2), false, false));
    HIPCALL(hipEventRecord(ev->join, s2), "join");
  }
  const int groups = split ? moe::kGroupRouted : moe::kGroupsAll;
  if (one_launch) {
    HIPCALL(moe::launch_decode_layer(
                (const uint16_t*)x, w->gate_w, w->bias, w->w13, w->w2, w->ws13, w->ws2, T,
                cfg->hidden_size, cfg->n_routed_experts, cfg->n_group, cfg->topk_group,
                cfg->num_experts_per_tok, cfg->moe_intermediate_size,
                cfg->shared_intermediate_size, cfg->routed_scaling_factor,
                at<float>(ws, L.part), logits, idx, wt, cnt, offs, pm, pos,
                at<int32_t>(ws, L.err), tiles, at<uint16_t>(ws, L.h), (uint16_t*)y,
                (uint16_t*)ys, (uint16_t*)out, at<void>(ws, L.flags), s),
            "decode layer");
    return MOE_OK;
  }
  if (L.decode) {
    HIPCALL(moe::launch_decode_route(x, cfg->act_dtype == MOE_BF16, w->gate_w, w->bias,
                                     at<float>(ws, L.part), logits, idx, wt, T, cfg->hidden_size,
                                     cfg->n_routed_experts, cfg->n_group, cfg->topk_group,
                                     cfg->num_experts_per_tok, cfg->routed_scaling_factor, cnt,
                                     offs, pm, pos, at<int32_t>(ws, L.err), tiles, true,
                                     (groups & moe::kGroupShared) && sh, s),
            "decode routing");
  } else {
    CHECK(run_gate(cfg, T, x, w->gate_w, w->bias, logits, idx, wt, ws, L, s));
    CHECK(run_permute(cfg, T, idx, cnt, offs, pm, pos, ws, L, s));
  }
  CHECK(run_ffn(cfg, T, x, pm, offs, w, y, ys, ws, L, s, groups, tiles, L.decode, !split));
  if (split) HIPCALL(hipStreamWaitEvent(s, ev->join, 0), "join");
  HIPCALL(moe::launch_combine(y, ys, pos, wt, out, T, cfg->hidden_size, cfg->num_experts_per_tok,
                              cfg->act_dtype == MOE_BF16, s),
          "combine");
  return MOE_OK;
}

// One expert weight matrix: its experts, output columns n (of gate and up
// each, for gate_up) and input columns kd.
struct Matrix {
  bool gate_up;
  int64_t experts;
  int n, kd;
};

moe_status weight_matrix(const moe_config* c, moe_weight_id which, Matrix* m) {
  if (which < MOE_W13 || which > MOE_WS2) return fail(MOE_ERR_INVALID_ARG, "unknown weight id");
  const bool shared = which == MOE_WS13 || which == MOE_WS2;
  if (shared && c->shared_intermediate_size == 0)
    return fail(MOE_ERR_INVALID_ARG, "no shared expert (shared_intermediate_size == 0)");
  const int inter = shared ? c->shared_intermediate_size : c->moe_intermediate_size;
  m->gate_up = which == MOE_W13 || which == MOE_WS13;
  m->experts = shared ? 1 : c->n_routed_experts;
  m->n = m->gate_up ? inter : c->hidden_size;
  m->kd = m->gate_up ? c->hidden_size : inter;
  return MOE_OK;
}

// rstd of a zero row is 1 / sqrt(eps): eps must be > 0.
moe_status check_norm(const moe_config* c, int64_t rows, float eps) {
  CHECK(check_cfg(c));
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows < 0");
  if (rows > 0x7fffffffLL) return fail(MOE_ERR_UNSUPPORTED, "rows exceeds int32 indexing");
  if (!(isfinite(eps) && eps > 0.0f))
    return fail(MOE_ERR_INVALID_ARG, "eps must be finite and > 0");
  return MOE_OK;
}

// The row kernels have a workgroup per token.
moe_status check_tokens(const moe_config* c, int64_t T, int64_t row_bytes) {
  CHECK(check_T(T, c));
  const int64_t most = moe::dispatch_max_tokens(row_bytes);
  if (T > most)
    return fail(MOE_ERR_UNSUPPORTED, "%lld tokens: one launch takes %lld rows of %lld bytes",
                (long long)T, (long long)most, (long long)row_bytes);
  return MOE_OK;
}

// The 4-bit quantiser and packer, workgroups of 256 threads.
moe_status check_matrix_threads(int64_t threads) {
  if (threads > moe::kMaxGridThreads / 256 * 256)
    return fail(MOE_ERR_UNSUPPORTED, "the matrix is too large for one launch (take its experts in "
                "parts, with fewer n_routed_experts)");
  return MOE_OK;
}

// ---- dense layers -----------------------------------------------------------
// The shared expert's matrices alone: `c` is cfg without its routed part, whose
// sizes then decide about nothing (what is refused, the workspace, the choice of
// kernels).
moe_status check_dense(const moe_config* cfg, int64_t T, moe_config* c) {
  NONNULL(cfg);
  *c = *cfg;
  c->n_routed_experts = 2;
  c->n_group = c->topk_group = c->num_experts_per_tok = 1;
  c->moe_intermediate_size = 128;
  c->routed_scaling_factor = 1.0f;
  CHECK(check_cfg(c));
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T < 0");
  const int64_t most = is_int8(c->weight_dtype) ? moe::quantize_rows_int8_max() : 0x7fffffffLL;
  if (T > most)
    return fail(MOE_ERR_UNSUPPORTED, "%lld tokens: a dense layer takes %lld", (long long)T,
                (long long)most);
  if (c->shared_intermediate_size <= 0)
    return fail(MOE_ERR_INVALID_ARG, "a dense layer needs shared_intermediate_size > 0");
  if (c->weight_dtype == MOE_BF16 &&
      !moe::dense_fits(T, c->hidden_size, c->shared_intermediate_size))
    return fail(MOE_ERR_UNSUPPORTED, "T, hidden_size or shared_intermediate_size is too large for "
                "one launch of the dense layer");
  return MOE_OK;
}

// Either form of the weights (row-major, packed) fits.
Layout dense_layout(const moe_config* c, int64_t T) {
  Layout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o += up(bytes);
    return at;
  };
  moe::FfnDims d{T, 0, c->hidden_size, c->moe_intermediate_size, c->shared_intermediate_size,
                 c->n_routed_experts, c->num_experts_per_tok};
  L.tiles = take(moe::ffn_tiles_bytes(d));
  ffn_segments(L, c, 0, T, take);
  if (c->weight_dtype == MOE_BF16)
    L.part = take(moe::dense_part_bytes(T, c->hidden_size, c->shared_intermediate_size, false));
  L.total = o;
  return L;
}

struct DenseBackwardLayout {
  size_t gu, da, h, part, total;
};
DenseBackwardLayout dense_backward_layout(const moe_config* c, int64_t T) {
  const size_t row = up((size_t)T * c->shared_intermediate_size * 2);
  return {0, 4 * row, 6 * row, 7 * row,
          7 * row + up(moe::dense_part_bytes(T, c->hidden_size, c->shared_intermediate_size, true))};
}

// ---- gradients --------------------------------------------------------------
struct GradArrays {
  std::unique_ptr<uint8_t[]> bf16;
  moe::GradList list(const moe_gradients* g) const {
    return {g->n, g->grad, g->out, g->count, bf16.get()};
  }
};

moe_status check_overlap(const moe_gradients* g) {
  struct Range {
    uintptr_t a, b;
    int i;
    bool out;
  };
  // Outputs that follow one another, on the gradients themselves or all behind
  // or before them, as the pieces of flat buffers do, need no sorting.
  uintptr_t end = 0, lo = UINTPTR_MAX, hi = 0, olo = UINTPTR_MAX;
  bool ordered = true, same = true;
  for (int i = 0; i < g->n; ++i) {
    if (!g->count[i]) continue;
    const uintptr_t bytes = g->count[i] * (g->dtype[i] == MOE_BF16 ? 2 : 4);
    const uintptr_t in = (uintptr_t)g->grad[i], out = (uintptr_t)g->out[i];
    ordered = ordered && out >= end;
    same = same && in == out;
    end = out + bytes;
    lo = std::min(lo, in);
    hi = std::max(hi, in + bytes);
    olo = std::min(olo, out);
  }
  if (ordered && (same || end <= lo || olo >= hi)) return MOE_OK;
  const std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)g->n]);
  if (!r) return fail(MOE_ERR_INVALID_ARG, "n = %d: no host memory", g->n);
  size_t m = 0;
  for (int i = 0; i < g->n; ++i) {
    if (!g->count[i]) continue;
    const uintptr_t bytes = g->count[i] * (g->dtype[i] == MOE_BF16 ? 2 : 4);
    const uintptr_t in = (uintptr_t)g->grad[i], out = (uintptr_t)g->out[i];
    r[m++] = {out, out + bytes, i, true};
    if (in != out) r[m++] = {in, in + bytes, i, false};
  }
  std::sort(r.get(), r.get() + m, [](const Range& x, const Range& y) { return x.a < y.a; });
  // Ends of the ranges so far: of the outputs, and of all.
  uintptr_t out_end = 0, all_end = 0;
  int out_i = 0, all_i = 0;
  for (size_t k = 0; k < m; ++k) {
    const bool bad = r[k].out ? r[k].a < all_end : r[k].a < out_end;
    if (bad)
      return fail(MOE_ERR_INVALID_ARG, "output of gradient %d overlaps gradient or output %d",
                  r[k].out ? r[k].i : out_i, r[k].out ? all_i : r[k].i);
    if (r[k].out && r[k].b > out_end) out_end = r[k].b, out_i = r[k].i;
    if (r[k].b > all_end) all_end = r[k].b, all_i = r[k].i;
  }
  return MOE_OK;
}

// With `writes`, no output may overlap another gradient or output; a gradient
// may be its own output.
moe_status check_gradients(const moe_gradients* g, bool writes, GradArrays* a) {
  NONNULL(g);
  if (g->n < 0) return fail(MOE_ERR_INVALID_ARG, "n < 0");
  if (g->n == 0) return MOE_OK;   // its arrays may be NULL
  NONNULL(g->grad);
  NONNULL(g->count);
  NONNULL(g->dtype);
  if (writes) NONNULL(g->out);
  a->bf16.reset(new (std::nothrow) uint8_t[g->n]);
  if (!a->bf16) return fail(MOE_ERR_INVALID_ARG, "n = %d: no host memory", g->n);
  double bytes = 0;
  for (int i = 0; i < g->n; ++i) {
    const int32_t t = g->dtype[i];
    if (t != MOE_F32 && t != MOE_BF16)
      return fail(MOE_ERR_UNSUPPORTED, "gradient %d: dtype must be MOE_F32 or MOE_BF16", i);
    const int size = t == MOE_BF16 ? 2 : 4;
    a->bf16[i] = t == MOE_BF16;
    if (g->count[i] < 0) return fail(MOE_ERR_INVALID_ARG, "gradient %d: count < 0", i);
    if (g->count[i] == 0) continue;
    bytes += (double)g->count[i] * size;
    if (!g->grad[i] || (writes && !g->out[i]))
      return fail(MOE_ERR_INVALID_ARG, "gradient %d is NULL", i);
    if ((uintptr_t)g->grad[i] % size || (writes && (uintptr_t)g->out[i] % size))
      return fail(MOE_ERR_INVALID_ARG, "gradient %d is not aligned to its type", i);
  }
  if (bytes > 4e12) return fail(MOE_ERR_UNSUPPORTED, "more than 4e12 bytes of gradients");
  return writes ? check_overlap(g) : MOE_OK;
}

moe_status check_grad_ws(const moe::GradList& l, void* ws, size_t ws_bytes) {
  const size_t need = moe::grad_norm_ws_bytes(l);
  if (l.n && (!ws || ws_bytes < need || ((uintptr_t)ws & 255)))
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned and >= %zu bytes", need);
  return MOE_OK;
}

// ---- the no-allocation forward ----------------------------------------------
// Workspace of moe_forward_noalloc: one static device array, of which every GPU
// that runs the library holds its own copy until the process ends.  In host
// code `scratch` names a host-side stand-in, not device memory: its device
// address comes from hipGetSymbolAddress, looked up once per device with
// that device current, and only that address is ever handed to kernels.
constexpr size_t kScratchBytes = MOE_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char scratch[kScratchBytes];

hipError_t scratch_address(void** out) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static void* addr[kMaxDevices] = {};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    addr[dev] = p;
  }
  *out = addr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

size_t moe_workspace_bytes(const moe_config* cfg, int64_t T) {
  if (check_cfg(cfg) != MOE_OK || T < 0 || check_T(T, cfg) != MOE_OK) return 0;
  return layout(cfg, T).total;
}

moe_status moe_set_gate_mode(int mode) {
  if (mode != MOE_GATE_SPLIT && mode != MOE_GATE_FUSED)
    return fail(MOE_ERR_INVALID_ARG, "gate mode %d is neither 0 (split) nor 1 (fused)", mode);
  moe::set_gate_mode(mode);
  return MOE_OK;
}

moe_status moe_gate(const moe_config* cfg, int64_t T, const void* x, const float* gate_w,
                    const float* bias, float* logits, int32_t* topk_idx, float* topk_w, void* ws,
                    size_t ws_bytes, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(gate_w);
  NONNULL(bias);
  NONNULL(topk_idx);
  NONNULL(topk_w);
  const Layout L = layout(cfg, T);
  CHECK(check_ws(ws, ws_bytes, L));
  return run_gate(cfg, T, x, gate_w, bias, logits, topk_idx, topk_w, ws, L, (hipStream_t)stream);
}

moe_status moe_permute(const moe_config* cfg, int64_t T, const int32_t* topk_idx, int32_t* counts,
                       int32_t* offsets, int32_t* perm, int32_t* pos, void* ws, size_t ws_bytes,
                       void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  NONNULL(topk_idx);
  NONNULL(counts);
  NONNULL(offsets);
  NONNULL(perm);
  NONNULL(pos);
  const Layout L = layout(cfg, T);
  CHECK(check_ws(ws, ws_bytes, L));
  return run_permute(cfg, T, topk_idx, counts, offsets, perm, pos, ws, L, (hipStream_t)stream);
}

moe_status moe_expert_ffn(const moe_config* cfg, int64_t T, const void* x, const int32_t* perm,
                          const int32_t* offsets, const moe_weights* w, void* y, void* y_shared,
                          void* ws, size_t ws_bytes, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(perm);
  NONNULL(offsets);
  NONNULL(y);
  CHECK(check_weights(cfg, w, false));
  if (cfg->shared_intermediate_size > 0) NONNULL(y_shared);
  if (is_int4(cfg->weight_dtype) || is_int8(cfg->weight_dtype)) {
    ALIGNED16(x);
    ALIGNED16(y);
    if (cfg->shared_intermediate_size > 0) ALIGNED16(y_shared);
  }
  const Layout L = layout(cfg, T);
  CHECK(check_ws(ws, ws_bytes, L));
  return run_ffn(cfg, T, x, perm, offsets, w, y,
                 cfg->shared_intermediate_size > 0 ? y_shared : nullptr, ws, L,
                 (hipStream_t)stream);
}

moe_status moe_combine(const moe_config* cfg, int64_t T, const void* y, const void* y_shared,
                       const int32_t* pos, const float* topk_w, void* out, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  NONNULL(y);
  NONNULL(pos);
  NONNULL(topk_w);
  NONNULL(out);
  if (cfg->shared_intermediate_size > 0) NONNULL(y_shared);
  if (cfg->hidden_size % 8)
    return fail(MOE_ERR_UNSUPPORTED, "hidden_size must be a multiple of 8");
  HIPCALL(moe::launch_combine(y, cfg->shared_intermediate_size > 0 ? y_shared : nullptr, pos,
                              topk_w, out, T, cfg->hidden_size, cfg->num_experts_per_tok,
                              cfg->act_dtype == MOE_BF16, (hipStream_t)stream),
          "combine");
  return MOE_OK;
}

moe_status moe_forward(const moe_config* cfg, int64_t T, const void* x, const moe_weights* w,
                       void* out, float* logits, int32_t* topk_idx, float* topk_w,
                       int32_t* counts, int32_t* perm, void* ws, size_t ws_bytes, void* stream) {
  return forward_impl(cfg, T, x, w, out, logits, topk_idx, topk_w, counts, perm, ws, ws_bytes,
                      (hipStream_t)stream, nullptr);
}

moe_status moe_forward_noalloc(const moe_config* cfg, int64_t T, const void* x,
                               const moe_weights* w, void* out, float* logits, int32_t* topk_idx,
                               float* topk_w, int32_t* counts, int32_t* perm, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (T == 0) return MOE_OK;
  const size_t need = layout(cfg, T).total;
  if (need > kScratchBytes)
    return fail(MOE_ERR_UNSUPPORTED,
                "moe_forward_noalloc: %lld tokens need %zu bytes of workspace, the static "
                "scratch holds %zu (use moe_forward with a caller workspace)",
                (long long)T, need, kScratchBytes);
  void* ws = nullptr;
  HIPCALL(scratch_address(&ws), "static scratch address");
  return forward_impl(cfg, T, x, w, out, logits, topk_idx, topk_w, counts, perm, ws,
                      kScratchBytes, (hipStream_t)stream, nullptr);
}

moe_status moe_forward_decode_fused(const moe_config* cfg, int64_t T, const void* x,
                                    const moe_weights* w, void* out, float* logits,
                                    int32_t* topk_idx, float* topk_w, int32_t* counts,
                                    int32_t* perm, void* ws, size_t ws_bytes, void* stream) {
  return forward_impl(cfg, T, x, w, out, logits, topk_idx, topk_w, counts, perm, ws, ws_bytes,
                      (hipStream_t)stream, nullptr, true);
}

moe_status moe_forward_overlap(const moe_config* cfg, int64_t T, const void* x,
                               const moe_weights* w, void* out, float* logits, int32_t* topk_idx,
                               float* topk_w, int32_t* counts, int32_t* perm, void* ws,
                               size_t ws_bytes, void* stream, void* shared_stream) {
  if (!shared_stream || shared_stream == stream)
    return fail(MOE_ERR_INVALID_ARG, "shared_stream must be a stream other than stream");
  return forward_impl(cfg, T, x, w, out, logits, topk_idx, topk_w, counts, perm, ws, ws_bytes,
                      (hipStream_t)stream, (hipStream_t)shared_stream);
}

size_t moe_expert_ffn_backward_workspace_bytes(const moe_config* cfg, int64_t T) {
  if (check_cfg(cfg) != MOE_OK || check_T(T, cfg) != MOE_OK) return 0;
  if (!has_backward(cfg)) return 0;
  moe::FfnDims d{T, T * cfg->num_experts_per_tok, cfg->hidden_size, cfg->moe_intermediate_size,
                 cfg->shared_intermediate_size, cfg->n_routed_experts,
                 cfg->num_experts_per_tok};
  return is_fp8(cfg->weight_dtype) ? moe::ffn_backward_fp8_ws_bytes(d)
                                   : moe::ffn_backward_ws_bytes(d);
}

moe_status moe_expert_ffn_backward(const moe_config* cfg, int64_t T, const void* x,
                                   const int32_t* perm, const int32_t* offsets,
                                   const moe_weights* w, const void* dy, const void* dy_shared,
                                   void* dx, void* dx_shared, void* dw13, void* dw2,
                                   void* dws13, void* dws2, void* ws, size_t ws_bytes,
                                   void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  const bool fp8 = is_fp8(cfg->weight_dtype);
  if (!has_backward(cfg))
    return fail(MOE_ERR_UNSUPPORTED,
                "the expert backward takes bf16 activations with bf16 or e4m3 weights");
  if (T == 0) return MOE_OK;
  NONNULL(w);
  if (w->packed)
    return fail(MOE_ERR_UNSUPPORTED, "the expert backward reads row-major weights (packed = 0)");
  NONNULL(x);
  NONNULL(perm);
  NONNULL(offsets);
  NONNULL(w->w13);
  NONNULL(w->w2);
  NONNULL(dy);
  NONNULL(dw13);
  NONNULL(dw2);
  const bool sh = cfg->shared_intermediate_size > 0;
  if (sh) {
    NONNULL(w->ws13);
    NONNULL(w->ws2);
    NONNULL(dy_shared);
    NONNULL(dws13);
    NONNULL(dws2);
  }
  if (fp8) {
    NONNULL(w->w13_scale);
    NONNULL(w->w2_scale);
    if (sh) {
      NONNULL(w->ws13_scale);
      NONNULL(w->ws2_scale);
    }
  }
  moe::FfnDims d{T, T * cfg->num_experts_per_tok, cfg->hidden_size, cfg->moe_intermediate_size,
                 cfg->shared_intermediate_size, cfg->n_routed_experts,
                 cfg->num_experts_per_tok};
  const size_t need = fp8 ? moe::ffn_backward_fp8_ws_bytes(d) : moe::ffn_backward_ws_bytes(d);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255))
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned and >= %zu bytes", need);
  if (fp8) {
    HIPCALL(moe::launch_ffn_backward_fp8(
                d, cfg->weight_dtype == MOE_FP8_E4M3_E8M0, (const uint16_t*)x, perm, offsets,
                (const uint8_t*)w->w13, w->w13_scale, (const uint8_t*)w->w2, w->w2_scale,
                (const uint8_t*)(sh ? w->ws13 : nullptr), sh ? w->ws13_scale : nullptr,
                (const uint8_t*)(sh ? w->ws2 : nullptr), sh ? w->ws2_scale : nullptr,
                (const uint16_t*)dy, (const uint16_t*)(sh ? dy_shared : nullptr), (uint16_t*)dx,
                (uint16_t*)(sh ? dx_shared : nullptr), (uint16_t*)dw13, (uint16_t*)dw2,
                (uint16_t*)(sh ? dws13 : nullptr), (uint16_t*)(sh ? dws2 : nullptr), ws,
                (hipStream_t)stream),
            "expert backward (e4m3)");
    return MOE_OK;
  }
  HIPCALL(moe::launch_ffn_backward(d, (const uint16_t*)x, perm, offsets,
                                   (const uint16_t*)w->w13, (const uint16_t*)w->w2,
                                   (const uint16_t*)(sh ? w->ws13 : nullptr),
                                   (const uint16_t*)(sh ? w->ws2 : nullptr), (const uint16_t*)dy,
                                   (const uint16_t*)(sh ? dy_shared : nullptr), (uint16_t*)dx,
                                   (uint16_t*)(sh ? dx_shared : nullptr), (uint16_t*)dw13,
                                   (uint16_t*)dw2, (uint16_t*)(sh ? dws13 : nullptr),
                                   (uint16_t*)(sh ? dws2 : nullptr), ws, (hipStream_t)stream),
          "expert backward");
  return MOE_OK;
}

size_t moe_backward_workspace_bytes(const moe_config* cfg, int64_t T) {
  if (check_cfg(cfg) != MOE_OK || check_T(T, cfg) != MOE_OK) return 0;
  if (!has_backward(cfg)) return 0;
  moe::FfnDims d{T, T * cfg->num_experts_per_tok, cfg->hidden_size, cfg->moe_intermediate_size,
                 cfg->shared_intermediate_size, cfg->n_routed_experts,
                 cfg->num_experts_per_tok};
  return moe::layer_backward_ws_bytes(d, is_fp8(cfg->weight_dtype));
}

moe_status moe_backward(const moe_config* cfg, int64_t T, const void* x, const moe_weights* w,
                        const float* logits, const int32_t* topk_idx, const float* topk_w,
                        const int32_t* perm, const int32_t* offsets, const int32_t* pos,
                        const void* y, const void* dout, void* dx, float* dgate_w, void* dw13,
                        void* dw2, void* dws13, void* dws2, void* ws, size_t ws_bytes,
                        void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  const bool fp8 = is_fp8(cfg->weight_dtype);
  if (!has_backward(cfg))
    return fail(MOE_ERR_UNSUPPORTED,
                "the layer backward takes bf16 activations with bf16 or e4m3 weights");
  if (T == 0) return MOE_OK;
  NONNULL(w);
  if (w->packed)
    return fail(MOE_ERR_UNSUPPORTED, "the layer backward reads row-major weights (packed = 0)");
  NONNULL(x);
  NONNULL(w->gate_w);
  NONNULL(w->w13);
  NONNULL(w->w2);
  NONNULL(logits);
  NONNULL(topk_idx);
  NONNULL(topk_w);
  NONNULL(perm);
  NONNULL(offsets);
  NONNULL(pos);
  NONNULL(y);
  NONNULL(dout);
  NONNULL(dx);
  NONNULL(dgate_w);
  NONNULL(dw13);
  NONNULL(dw2);
  const bool sh = cfg->shared_intermediate_size > 0;
  if (sh) {
    NONNULL(w->ws13);
    NONNULL(w->ws2);
    NONNULL(dws13);
    NONNULL(dws2);
  }
  if (fp8) {
    NONNULL(w->w13_scale);
    NONNULL(w->w2_scale);
    if (sh) {
      NONNULL(w->ws13_scale);
      NONNULL(w->ws2_scale);
    }
  }
  moe::FfnDims d{T, T * cfg->num_experts_per_tok, cfg->hidden_size, cfg->moe_intermediate_size,
                 cfg->shared_intermediate_size, cfg->n_routed_experts,
                 cfg->num_experts_per_tok};
  const size_t need = moe::layer_backward_ws_bytes(d, fp8);
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 255))
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned and >= %zu bytes", need);
  moe::ExpertWeights ew{w->w13, w->w2, sh ? w->ws13 : nullptr, sh ? w->ws2 : nullptr};
  if (fp8) {
    ew.w13s = w->w13_scale;
    ew.w2s = w->w2_scale;
    ew.ws13s = sh ? w->ws13_scale : nullptr;
    ew.ws2s = sh ? w->ws2_scale : nullptr;
    ew.fp8 = true;
    ew.pow2 = cfg->weight_dtype == MOE_FP8_E4M3_E8M0;
  }
  HIPCALL(moe::launch_layer_backward(
              d, (const uint16_t*)x, w->gate_w, logits, topk_idx, topk_w, perm, offsets, pos,
              (const uint16_t*)y, (const uint16_t*)dout, ew, cfg->routed_scaling_factor,
              (uint16_t*)dx, dgate_w, (uint16_t*)dw13, (uint16_t*)dw2,
              (uint16_t*)(sh ? dws13 : nullptr), (uint16_t*)(sh ? dws2 : nullptr), ws,
              (hipStream_t)stream),
          "layer backward");
  return MOE_OK;
}

moe_status moe_expert_ffn_quantized(const moe_config* cfg, int64_t T, const uint8_t* xq,
                                    const float* xs, const int32_t* perm, const int32_t* offsets,
                                    const moe_weights* w, void* y, void* y_shared, void* ws,
                                    size_t ws_bytes, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_T(T, cfg));
  if (!quantises_act(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "quantised rows need e4m3 or 8-bit integer weights");
  if (T == 0) return MOE_OK;
  NONNULL(xq);
  NONNULL(xs);
  ALIGNED16(xq);
  NONNULL(perm);
  NONNULL(offsets);
  NONNULL(y);
  CHECK(check_weights(cfg, w, false));
  if (cfg->shared_intermediate_size > 0) NONNULL(y_shared);
  if (is_int8(cfg->weight_dtype)) {
    ALIGNED16(y);
    if (cfg->shared_intermediate_size > 0) ALIGNED16(y_shared);
  }
  const Layout L = layout(cfg, T);
  CHECK(check_ws(ws, ws_bytes, L));
  return run_ffn(cfg, T, nullptr, perm, offsets, w, y,
                 cfg->shared_intermediate_size > 0 ? y_shared : nullptr, ws, L,
                 (hipStream_t)stream, moe::kGroupsAll, nullptr, false, false, xq, xs);
}

moe_status moe_add_rmsnorm(const moe_config* cfg, int64_t rows, const void* x,
                           const void* residual, const float* weight, float eps, void* sum,
                           void* y, uint8_t* yq, float* ys, void* stream) {
  CHECK(check_norm(cfg, rows, eps));
  if (!yq != !ys) return fail(MOE_ERR_INVALID_ARG, "yq and ys go together");
  if (yq && cfg->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "the e4m3 output takes bf16 activations");
  if (yq && is_int8(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "the norm writes no 8-bit integer rows (moe_quantize_act)");
  if (yq && cfg->hidden_size % 128) return fail(MOE_ERR_UNSUPPORTED, "hidden_size %% 128 != 0");
  const int64_t most = moe::add_rmsnorm_max_rows(cfg->hidden_size, cfg->act_dtype == MOE_BF16);
  if (rows > most)
    return fail(MOE_ERR_UNSUPPORTED, "%lld rows: one launch takes %lld of this width",
                (long long)rows, (long long)most);
  if (rows == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(weight);
  if (!y && !yq) return fail(MOE_ERR_INVALID_ARG, "y and yq are both NULL");
  ALIGNED16(x);
  ALIGNED16(residual);
  ALIGNED16(weight);
  ALIGNED16(sum);
  ALIGNED16(y);
  ALIGNED16(yq);
  HIPCALL(moe::launch_add_rmsnorm(x, residual, weight, eps, rows, cfg->hidden_size,
                                  cfg->act_dtype == MOE_BF16, sum, y, yq, ys,
                                  cfg->weight_dtype == MOE_FP8_E4M3_E8M0, (hipStream_t)stream),
          "rmsnorm");
  return MOE_OK;
}

size_t moe_add_rmsnorm_backward_workspace_bytes(const moe_config* cfg, int64_t rows) {
  if (check_norm(cfg, rows, 1.0f) != MOE_OK) return 0;
  return moe::rmsnorm_backward_ws_bytes(rows, cfg->hidden_size);
}

moe_status moe_add_rmsnorm_backward(const moe_config* cfg, int64_t rows, const void* sum,
                                    const float* weight, float eps, const void* dy,
                                    const void* dsum, void* dx, float* dweight, void* ws,
                                    size_t ws_bytes, void* stream) {
  CHECK(check_norm(cfg, rows, eps));
  NONNULL(dweight);
  ALIGNED16(sum);
  ALIGNED16(weight);
  ALIGNED16(dy);
  ALIGNED16(dsum);
  ALIGNED16(dx);
  ALIGNED16(dweight);
  if (rows) {
    NONNULL(sum);
    NONNULL(weight);
    NONNULL(dy);
    NONNULL(dx);
    const size_t need = moe::rmsnorm_backward_ws_bytes(rows, cfg->hidden_size);
    if (!ws || ws_bytes < need || ((uintptr_t)ws & 255))
      return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned and >= %zu bytes", need);
  }
  HIPCALL(moe::launch_add_rmsnorm_backward(sum, weight, eps, dy, dsum, rows, cfg->hidden_size,
                                           cfg->act_dtype == MOE_BF16, dx, dweight, (float*)ws,
                                           (hipStream_t)stream),
          "rmsnorm backward");
  return MOE_OK;
}

moe_status moe_dispatch(const moe_config* cfg, int64_t T, const void* x, const int32_t* pos,
                        void* rows, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_tokens(cfg, T, (int64_t)cfg->hidden_size * act_bytes(cfg)));
  if (T == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(pos);
  NONNULL(rows);
  ALIGNED16(x);
  ALIGNED16(rows);
  HIPCALL(moe::launch_dispatch(x, (int64_t)cfg->hidden_size * act_bytes(cfg), nullptr, 0, pos, T,
                               cfg->num_experts_per_tok, rows, nullptr, (hipStream_t)stream),
          "dispatch");
  return MOE_OK;
}

moe_status moe_dispatch_quantized(const moe_config* cfg, int64_t T, const uint8_t* xq,
                                  const float* xs, const int32_t* pos, uint8_t* rows_q,
                                  float* rows_s, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_tokens(cfg, T, cfg->hidden_size));
  if (cfg->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "e4m3 rows belong to bf16 activations");
  if (is_int8(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "rows of e4m3 codes with 1x128 scales, not of 8-bit integers");
  if (cfg->hidden_size % 128) return fail(MOE_ERR_UNSUPPORTED, "hidden_size %% 128 != 0");
  if (T == 0) return MOE_OK;
  NONNULL(xq);
  NONNULL(xs);
  NONNULL(pos);
  NONNULL(rows_q);
  NONNULL(rows_s);
  ALIGNED16(xq);
  ALIGNED16(rows_q);
  HIPCALL(moe::launch_dispatch(xq, cfg->hidden_size, xs, cfg->hidden_size / 128, pos, T,
                               cfg->num_experts_per_tok, rows_q, rows_s, (hipStream_t)stream),
          "dispatch");
  return MOE_OK;
}

moe_status moe_dispatch_backward(const moe_config* cfg, int64_t T, const void* drows,
                                 const void* dx_add, const int32_t* pos, void* dx, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_tokens(cfg, T, (int64_t)cfg->hidden_size * act_bytes(cfg)));
  if (T == 0) return MOE_OK;
  NONNULL(drows);
  NONNULL(pos);
  NONNULL(dx);
  ALIGNED16(drows);
  ALIGNED16(dx_add);
  ALIGNED16(dx);
  HIPCALL(moe::launch_dispatch_backward(drows, dx_add, pos, T, cfg->hidden_size,
                                        cfg->num_experts_per_tok, cfg->act_dtype == MOE_BF16, dx,
                                        (hipStream_t)stream),
          "dispatch backward");
  return MOE_OK;
}

moe_status moe_combine_backward(const moe_config* cfg, int64_t T, const void* dout, const void* y,
                                const int32_t* pos, const float* topk_w, void* dy,
                                float* dtopk_w, void* stream) {
  CHECK(check_cfg(cfg));
  CHECK(check_tokens(cfg, T, (int64_t)cfg->hidden_size * act_bytes(cfg)));
  if (T == 0) return MOE_OK;
  NONNULL(dout);
  NONNULL(y);
  NONNULL(pos);
  NONNULL(topk_w);
  NONNULL(dy);
  NONNULL(dtopk_w);
  ALIGNED16(dout);
  ALIGNED16(y);
  ALIGNED16(dy);
  HIPCALL(moe::launch_combine_backward(dout, y, pos, topk_w, T, cfg->hidden_size,
                                       cfg->num_experts_per_tok, cfg->act_dtype == MOE_BF16, dy,
                                       dtopk_w, (hipStream_t)stream),
          "combine backward");
  return MOE_OK;
}

size_t moe_dense_ffn_workspace_bytes(const moe_config* cfg, int64_t T) {
  moe_config c;
  return check_dense(cfg, T, &c) == MOE_OK ? dense_layout(&c, T).total : 0;
}

moe_status moe_dense_ffn(const moe_config* cfg, int64_t T, const void* x, const moe_weights* w,
                         float* gu, void* y, void* ws, size_t ws_bytes, void* stream) {
  moe_config c;
  CHECK(check_dense(cfg, T, &c));
  NONNULL(w);
  const bool rowmajor = c.weight_dtype == MOE_BF16 && !w->packed;
  if (gu && !rowmajor)
    return fail(MOE_ERR_UNSUPPORTED, "gu is kept by row-major bf16 weights only");
  if (T == 0) return MOE_OK;
  NONNULL(x);
  NONNULL(y);
  CHECK(check_weights(&c, w, false, true));
  ALIGNED16(x);
  ALIGNED16(y);
  ALIGNED16(gu);
  const Layout L = dense_layout(&c, T);
  CHECK(check_ws(ws, ws_bytes, L));
  const hipStream_t s = (hipStream_t)stream;
  if (!rowmajor)
    return run_ffn(&c, T, x, nullptr, nullptr, w, nullptr, y, ws, L, s, moe::kGroupShared);
  ALIGNED16(w->ws13);
  ALIGNED16(w->ws2);
  const int H = c.hidden_size, I = c.shared_intermediate_size;
  uint16_t* h = at<uint16_t>(ws, L.h);
  HIPCALL(moe::launch_dense_gate_up((const uint16_t*)x, (const uint16_t*)w->ws13, T, H, I,
                                    gu, h, at<float>(ws, L.part), s),
          "dense gate/up");
  HIPCALL(moe::launch_dense_down(h, (const uint16_t*)w->ws2, T, H, I, (uint16_t*)y,
                                 at<float>(ws, L.part), s),
          "dense down");
  return MOE_OK;
}

size_t moe_dense_ffn_backward_workspace_bytes(const moe_config* cfg, int64_t T) {
  moe_config c;
  if (check_dense(cfg, T, &c) != MOE_OK || c.weight_dtype != MOE_BF16) return 0;
  return dense_backward_layout(&c, T).total;
}

moe_status moe_dense_ffn_backward(const moe_config* cfg, int64_t T, const void* x,
                                  const moe_weights* w, const float* gu, const void* dy, void* dx,
                                  void* dws13, void* dws2, void* ws, size_t ws_bytes,
                                  void* stream) {
  moe_config c;
  CHECK(check_dense(cfg, T, &c));
  if (c.weight_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "the dense backward takes bf16 weights");
  NONNULL(w);
  if (w->packed)
    return fail(MOE_ERR_UNSUPPORTED, "the dense backward reads row-major weights (packed = 0)");
  NONNULL(dws13);
  NONNULL(dws2);
  const int H = c.hidden_size, I = c.shared_intermediate_size;
  const DenseBackwardLayout L = dense_backward_layout(&c, T);
  if (T) {
    NONNULL(x);
    NONNULL(dy);
    NONNULL(w->ws13);
    NONNULL(w->ws2);
    if (!ws || ws_bytes < L.total || ((uintptr_t)ws & 255))
      return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned and >= %zu bytes",
                  L.total);
  }
  ALIGNED16(x);
  ALIGNED16(w->ws13);
  ALIGNED16(w->ws2);
  ALIGNED16(gu);
  ALIGNED16(dy);
  ALIGNED16(dx);
  ALIGNED16(dws13);
  ALIGNED16(dws2);
  const hipStream_t s = (hipStream_t)stream;
  const float* g = gu;
  if (T && !g) {   // computed again
    HIPCALL(moe::launch_dense_gate_up((const uint16_t*)x, (const uint16_t*)w->ws13, T, H, I,
                                      at<float>(ws, L.gu), nullptr, at<float>(ws, L.part), s),
            "dense gate/up");
    g = at<float>(ws, L.gu);
  }
  HIPCALL(moe::launch_dense_backward((const uint16_t*)x, (const uint16_t*)w->ws13,
                                     (const uint16_t*)w->ws2, g, (const uint16_t*)dy, T, H, I,
                                     at<uint16_t>(ws, L.da), at<uint16_t>(ws, L.h), (uint16_t*)dx,
                                     (uint16_t*)dws13, (uint16_t*)dws2, at<float>(ws, L.part), s),
          "dense backward");
  return MOE_OK;
}

size_t moe_grad_norm_workspace_bytes(const moe_gradients* g) {
  GradArrays a;
  return check_gradients(g, false, &a) == MOE_OK ? moe::grad_norm_ws_bytes(a.list(g)) : 0;
}

moe_status moe_grad_norm(const moe_gradients* g, float* norm, void* ws, size_t ws_bytes,
                         void* stream) {
  GradArrays a;
  CHECK(check_gradients(g, false, &a));
  NONNULL(norm);
  const moe::GradList l = a.list(g);
  CHECK(check_grad_ws(l, ws, ws_bytes));
  HIPCALL(moe::launch_grad_norm(l, (double*)ws, norm, (hipStream_t)stream),
          "gradient norm");
  return MOE_OK;
}

moe_status moe_clip_grads(const moe_gradients* g, float max_norm, float* norm, int norm_given,
                          void* ws, size_t ws_bytes, void* stream) {
  GradArrays a;
  CHECK(check_gradients(g, true, &a));
  if (!(max_norm >= 0.0f)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be >= 0");
  NONNULL(norm);
  const moe::GradList l = a.list(g);
  if (!norm_given) CHECK(check_grad_ws(l, ws, ws_bytes));
  const hipStream_t s = (hipStream_t)stream;
  HIPCALL(moe::launch_clip(l, (double*)ws, norm, norm_given != 0, max_norm, s),
          "gradient clipping");
  return MOE_OK;
}

moe_status moe_bias_update(const moe_config* cfg, const int32_t* counts, float gamma,
                           float* bias, void* stream) {
  CHECK(check_cfg(cfg));
  if (!(gamma >= 0.0f) || isinf(gamma))
    return fail(MOE_ERR_INVALID_ARG, "gamma must be finite and >= 0");
  NONNULL(counts);
  NONNULL(bias);
  HIPCALL(moe::launch_bias_update(counts, bias, cfg->n_routed_experts, gamma,
                                  (hipStream_t)stream),
          "bias update");
  return MOE_OK;
}

moe_status moe_quantize_act(const moe_config* cfg, int64_t rows, const void* x, uint8_t* xq,
                            float* xs, void* stream) {
  CHECK(check_cfg(cfg));
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows < 0");
  if (rows == 0) return MOE_OK;
  if (cfg->act_dtype != MOE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "the quantiser takes bf16 activations");
  if (cfg->hidden_size % 128) return fail(MOE_ERR_UNSUPPORTED, "hidden_size %% 128 != 0");
  if (is_int8(cfg->weight_dtype) && rows > moe::quantize_rows_int8_max())
    return fail(MOE_ERR_UNSUPPORTED, "%lld rows: one launch takes %lld", (long long)rows,
                (long long)moe::quantize_rows_int8_max());
  NONNULL(x);
  NONNULL(xq);
  NONNULL(xs);
  if (is_int8(cfg->weight_dtype)) {
    ALIGNED16(x);
    ALIGNED16(xq);
    HIPCALL(moe::launch_quantize_rows_int8((const uint16_t*)x, rows, cfg->hidden_size,
                                           (int8_t*)xq, xs, (hipStream_t)stream),
            "quantise");
    return MOE_OK;
  }
  HIPCALL(moe::launch_quant_rows((const uint16_t*)x, rows, cfg->hidden_size, xq, xs,
                                 cfg->weight_dtype == MOE_FP8_E4M3_E8M0,
                                 (hipStream_t)stream),
          "quantise");
  return MOE_OK;
}

size_t moe_packed_bytes(const moe_config* cfg, moe_weight_id which) {
  if (check_cfg(cfg) != MOE_OK || cfg->weight_dtype == MOE_F32) return 0;
  const int H = cfg->hidden_size, I = cfg->moe_intermediate_size,
            Is = cfg->shared_intermediate_size, E = cfg->n_routed_experts;
  auto bytes = [cfg](bool gate_up, int64_t experts, int n, int kd) {
    if (is_int4(cfg->weight_dtype))
      return moe::packed4_bytes(gate_up, experts, n, kd, int4_group(cfg->weight_dtype));
    if (is_int8(cfg->weight_dtype)) return moe::packed_int8_bytes(gate_up, experts, n, kd);
    return is_fp8(cfg->weight_dtype) ? moe::packed8_bytes(gate_up, experts, n, kd)
                                     : moe::packed_bytes(gate_up, experts, n, kd);
  };
  switch (which) {
    case MOE_W13: return bytes(true, E, I, H);
    case MOE_W2: return bytes(false, E, H, I);
    case MOE_WS13: return Is ? bytes(true, 1, Is, H) : 0;
    case MOE_WS2: return Is ? bytes(false, 1, H, Is) : 0;
  }
  return 0;
}

moe_status moe_pack_weight(const moe_config* cfg, moe_weight_id which, const void* src,
                           void* dst, void* stream) {
  CHECK(check_cfg(cfg));
  if (cfg->weight_dtype == MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "the packed weight layout is for bf16 and fp8 weights");
  if (is_int4(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "4-bit weights are packed with their scales by "
                "moe_pack_quantized");
  Matrix m;
  CHECK(weight_matrix(cfg, which, &m));
  NONNULL(src);
  NONNULL(dst);
  if (is_int8(cfg->weight_dtype)) {
    CHECK(check_matrix_threads((int64_t)(moe_packed_bytes(cfg, which) / 16)));
    ALIGNED16(src);
    ALIGNED16(dst);
    HIPCALL(moe::launch_pack_int8(m.gate_up, (const int8_t*)src, dst, m.experts, m.n, m.kd,
                                  (hipStream_t)stream),
            "pack weight");
  } else if (is_fp8(cfg->weight_dtype))
    HIPCALL(moe::launch_pack8(m.gate_up, (const uint8_t*)src, dst, m.experts, m.n, m.kd,
                              (hipStream_t)stream),
            "pack weight");
  else
    HIPCALL(moe::launch_pack(m.gate_up, (const uint16_t*)src, dst, m.experts, m.n, m.kd,
                             (hipStream_t)stream),
            "pack weight");
  return MOE_OK;
}

moe_status moe_quantize_weight(const moe_config* cfg, moe_weight_id which, const void* src,
                               uint8_t* codes, void* scales, void* stream) {
  CHECK(check_cfg(cfg));
  if (!is_int4(cfg->weight_dtype) && !is_int8(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED,
                "moe_quantize_weight makes integer weights (MOE_INT4_*, MOE_INT8)");
  Matrix m;
  CHECK(weight_matrix(cfg, which, &m));
  if (is_int8(cfg->weight_dtype)) {
    const int64_t rows = m.experts * (m.gate_up ? 2 : 1) * m.n;
    CHECK(check_matrix_threads(rows * 256));
    NONNULL(src);
    NONNULL(codes);
    NONNULL(scales);
    ALIGNED16(src);
    ALIGNED16(codes);
    HIPCALL(moe::launch_quantize_rows_int8((const uint16_t*)src, rows, m.kd, (int8_t*)codes,
                                           (float*)scales, (hipStream_t)stream),
            "quantise weight");
    return MOE_OK;
  }
  CHECK(check_matrix_threads(m.experts * (m.gate_up ? 2 : 1) * m.n * (m.kd / 8)));
  NONNULL(src);
  NONNULL(codes);
  NONNULL(scales);
  ALIGNED16(src);
  ALIGNED16(codes);
  HIPCALL(moe::launch_quantize_int4(int4_group(cfg->weight_dtype), (const uint16_t*)src,
                                    m.experts * (m.gate_up ? 2 : 1) * m.n, m.kd, codes,
                                    (uint16_t*)scales, (hipStream_t)stream),
          "quantise weight");
  return MOE_OK;
}

moe_status moe_pack_quantized(const moe_config* cfg, moe_weight_id which, const uint8_t* codes,
                              const void* scales, void* dst, void* stream) {
  CHECK(check_cfg(cfg));
  if (!is_int4(cfg->weight_dtype))
    return fail(MOE_ERR_UNSUPPORTED, "moe_pack_quantized packs 4-bit weights (MOE_INT4_*)");
  Matrix m;
  CHECK(weight_matrix(cfg, which, &m));
  CHECK(check_matrix_threads((int64_t)(moe_packed_bytes(cfg, which) / 16)));
  NONNULL(codes);
  NONNULL(scales);
  NONNULL(dst);
  ALIGNED16(dst);
  HIPCALL(moe::launch_pack_int4(m.gate_up, int4_group(cfg->weight_dtype), codes,
                                (const uint16_t*)scales, dst, m.experts, m.n, m.kd,
                                (hipStream_t)stream),
          "pack quantised weight");
  return MOE_OK;
}

moe_status moe_get_device_error(void* ws, size_t ws_bytes, void* stream) {
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  if (ws_bytes < sizeof(int32_t)) return fail(MOE_ERR_WORKSPACE, "workspace too small");
  int32_t flag = 0;
  hipStream_t s = (hipStream_t)stream;
  HIPCALL(hipMemcpyAsync(&flag, ws, sizeof(flag), hipMemcpyDeviceToHost, s), "read error flag");
  HIPCALL(hipStreamSynchronize(s), "synchronise");
  if (flag & 2)
    return fail(MOE_ERR_DEVICE_CHECK,
                "a completion wait of the one-launch decode layer timed out: outputs unreliable");
  if (flag) return fail(MOE_ERR_DEVICE_CHECK, "an expert index was outside [0, E)");
  return MOE_OK;
}

const char* moe_strerror(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_HIP: return "HIP runtime error";
    case MOE_ERR_DEVICE_CHECK: return "device check failed (expert index out of range)";
  }
  return "unknown status";
}

const char* moe_last_error(void) { return g_msg; }

}  // extern "C"
