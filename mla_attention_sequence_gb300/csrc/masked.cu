// C ABI of the operators around packed documents: key bounds, masked attention forward and
// backward, rotary positions, 8-bit checkpoints. Argument checks, workspace layout, dispatch.
//
// Where the bf16 calls round to fewer bits than the fp32 they sum in: K and V, the weights P and dS,
// because they are operands of bf16 products (as fp32 each would be split in two or three, and every
// product would take as many times as long); dK and dV, because they are the next products' operands and
// are stored between the kernels (twice the bytes in fp32); out, from which the backward takes D, because
// the caller keeps it in bf16. As in the plain calls: 0.003 to 0.004 from 64 bits where one rounding of
// the outputs gives 0.0017. The CUDA-core path rounds inputs and outputs alone.
#include "api_util.h"
#include "mask.h"
#include "rope.h"

#include <algorithm>
#include <cmath>

namespace laga {
LaunchResult pack8(bool is_bf16, long long rows, int cols, const void* x, uint8_t* codes, uint8_t* scales,
                   cudaStream_t st);
LaunchResult unpack8(bool is_bf16, long long rows, int cols, const Packed& p, void* x, cudaStream_t st);

namespace {

constexpr const char* kTensorPointers = "tensor pointers must be non-null and 16-byte aligned%s";
constexpr const char* kWorkspace = "workspace missing, misaligned (256 B) or too small%s";

// The masked calls' path: plan's, without what they do not take.
Path masked_plan(const laga_mla_desc* desc, Dims* d, laga_status* st, bool for_bwd) {
  const Path path = plan(desc, d, st, for_bwd);
  if (path == Path::Invalid) return path;
  if (path == Path::TensorCoreFused) {
    *st = fail(LAGA_ERR_UNSUPPORTED, "masked attention has no LAGA_VARIANT_FUSED_RECON%s");
    return Path::Invalid;
  }
  if (desc->flags & LAGA_FLAG_KV_PREBUILT) {
    *st = fail(LAGA_ERR_UNSUPPORTED, "masked attention rebuilds K and V itself (no LAGA_FLAG_KV_PREBUILT)%s");
    return Path::Invalid;
  }
  if (path == Path::Simt && (d->d_qk() > 256 || d->d_v > 256)) {
    *st = fail(LAGA_ERR_UNSUPPORTED, "masked attention supports d_nope + d_rope <= 256 and d_v <= 256%s");
    return Path::Invalid;
  }
  if (path == Path::Simt && static_cast<int64_t>(d->B) * d->S >= (int64_t(1) << 31)) {
    *st = fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
    return Path::Invalid;
  }
  if (d->B > 65535 || d->n_h > 65535 ||
      static_cast<int64_t>(d->B) * d->n_h * (d->sq_pad / 128) >= (int64_t(1) << 31) - 65536) {
    *st = fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
    return Path::Invalid;
  }
  return path;
}

int elem_size(const laga_mla_desc* desc) { return desc->dtype == LAGA_DTYPE_BF16 ? 2 : 4; }

// Heads per dK/dV CTA: as in the plain backward, fewer where that would leave the 152 SMs fewer
// than six CTAs each. Documents make CTAs of very different length, and a walk over four heads
// of the longest sets the time (2 x 4096 rows of 16 heads, 5 documents: 184 us with four heads,
// 158 with two, 150 with one; 2999 rows of 32 heads, 6 documents, capped: 182 and 119).
int masked_heads_per_cta(const Dims& d) {
  int G = dkdv_heads_per_cta(d.n_h);
  while (G > 1 && static_cast<int64_t>(d.skv_pad / 128) * d.B * (d.n_h / G) < 6 * 152) G /= 2;
  return G;
}

size_t tc_clean_q_bytes(const Dims& d) { return align_up(static_cast<size_t>(d.B) * d.Sq * d.n_h * 192 * 2, 256); }
size_t tc_clean_dout_bytes(const Dims& d) { return align_up(static_cast<size_t>(d.B) * d.Sq * d.n_h * 128 * 2, 256); }

size_t fwd_bytes(const Dims& d, Path path, int elem) {
  return path == Path::Simt ? simt_masked_fwd_workspace(d, elem) : tc_fwd_workspace(d) + mask_bytes(d, elem);
}
size_t bwd_bytes(const Dims& d, Path path, int elem) {
  return path == Path::Simt ? simt_masked_bwd_workspace(d, elem)
                            : tc_bwd_workspace(d, masked_heads_per_cta(d)) + mask_bytes(d, elem) + tc_clean_q_bytes(d) + tc_clean_dout_bytes(d);
}

// ---- the rotation's frequencies. Positions multiply a frequency's error, so that a double's 53 bits
// would be 2^-25 turns off at position 2^31; a pair of doubles (their exact sum, some 106 bits) leaves
// nothing but the rounding of the 64-bit fraction itself.
struct Pair {
  double hi, lo;
};
Pair sum_of(double a, double b) {  // exact for |a| >= |b|
  const double s = a + b;
  return Pair{s, b - (s - a)};
}
Pair operator*(Pair a, Pair b) {
  const double p = a.hi * b.hi;
  return sum_of(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

// theta^(-1/n): a double's guess x, and one Newton step for x^n theta = 1.
Pair root_step(double theta, int n) {
  const double x = std::pow(theta, -1.0 / n);
  Pair r{theta, 0.0}, square{x, 0.0};
  for (int k = n; k > 0; k >>= 1, square = square * square)
    if (k & 1) r = r * square;
  return sum_of(x, x * ((1.0 - r.hi) - r.lo) / n);
}

// Turns per position step as a fraction of 2^64, to the nearest: f / (2 pi), at most 0.16.
uint64_t turns_of(Pair f) {
  const Pair t = f * Pair{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
  const double h = std::ldexp(t.hi, 64), whole = std::floor(h);
  return static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint((h - whole) + std::ldexp(t.lo, 64)));
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

}  // namespace

laga_status check_mods(const laga_mla_mods* mods, ScoreMods* out) {
  *out = ScoreMods{0.f, nullptr};
  if (!mods) return LAGA_OK;
  // outside this range cap or 1 / cap, times the other factors of a score, leaves fp32
  if (mods->softcap != 0.f && !(mods->softcap >= 1e-20f && mods->softcap <= 1e30f))
    return fail(LAGA_ERR_INVALID_ARG, "softcap must be 0 (none) or between 1e-20 and 1e30%s");
  auto aligned4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if (!aligned4(mods->key_lo) || !aligned4(mods->key_hi) || !aligned4(mods->slopes))
    return fail(LAGA_ERR_INVALID_ARG, "key_lo, key_hi and slopes must be 4-byte aligned%s");
  out->cap = mods->softcap;
  out->slopes = mods->slopes;
  return LAGA_OK;
}

laga_status rope_plan(const laga_mla_rope_desc* desc, const void* pos, RopeArgs* args, const RopeTable** table) {
  if (!desc) return fail(LAGA_ERR_INVALID_ARG, "null descriptor%s");
  const laga_mla_rope_desc& x = *desc;
  const int64_t lim = int64_t(1) << 40;
  if (x.tokens < 1 || x.n_h < 1 || x.d_nope < 0 || x.d_rope < 2 || x.d_rope % 2 != 0 || x.n_axes < 1 ||
      x.n_axes > LAGA_ROPE_MAX_AXES)
    return fail(LAGA_ERR_INVALID_ARG, "rope: tokens, n_h >= 1, d_nope >= 0, even d_rope >= 2, 1 <= n_axes <= 4%s");
  if (x.dtype != LAGA_DTYPE_F32 && x.dtype != LAGA_DTYPE_BF16)
    return fail(LAGA_ERR_UNSUPPORTED, "dtype must be LAGA_DTYPE_F32 or LAGA_DTYPE_BF16%s");
  if (x.tokens >= (int64_t(1) << 31) || x.n_h >= 65536 || x.d_nope >= 65536 || x.d_rope > 2 * kRopePairs ||
      x.tokens * x.n_h * (x.d_nope + x.d_rope) >= lim || x.n_h * (x.d_nope + x.d_rope) >= (int64_t(1) << 26))
    return fail(LAGA_ERR_UNSUPPORTED, "rope: problem too large (d_rope <= 256)%s");
  if (!(x.theta >= 1.0) || !std::isfinite(x.theta))
    return fail(LAGA_ERR_INVALID_ARG, "rope: theta must be finite and >= 1%s");
  int64_t pairs = 0;
  for (int a = 0; a < x.n_axes; ++a) {
    if (x.sections[a] < 0) return fail(LAGA_ERR_INVALID_ARG, "rope: sections must be >= 0%s");
    pairs += x.sections[a];
  }
  if (pairs != x.d_rope / 2) return fail(LAGA_ERR_INVALID_ARG, "rope: the sections must add up to d_rope / 2%s");
  const uintptr_t pe = x.pos64 ? 8 : 4;
  if (!pos || (reinterpret_cast<uintptr_t>(pos) & (pe - 1)))
    return fail(LAGA_ERR_INVALID_ARG, "rope: pos must be non-null and aligned to its type%s");
  // The table of the last call's frequencies, per thread: a program's calls share theta and the
  // sections, and its powers are half of a small call's host time.
  static thread_local RopeTable t;
  static thread_local laga_mla_rope_desc made;  // n_axes 0: none
  if (made.n_axes != x.n_axes || made.d_rope != x.d_rope || made.theta != x.theta ||
      !std::equal(x.sections, x.sections + x.n_axes, made.sections)) {
    const Pair step = root_step(x.theta, static_cast<int>(x.d_rope / 2));
    Pair f{1.0, 0.0};
    int i = 0;
    for (int a = 0; a < x.n_axes; ++a)
      for (int k = 0; k < x.sections[a]; ++k, ++i, f = f * step) {
        t.turns[i] = turns_of(f);
        t.axis[i] = static_cast<uint8_t>(a);
      }
    made = x;
  }
  RopeArgs& g = *args;
  g.tokens = x.tokens;
  g.n_h = static_cast<int>(x.n_h);
  g.d_nope = static_cast<int>(x.d_nope);
  g.d_rope = static_cast<int>(x.d_rope);
  g.interleaved = x.interleaved != 0;
  g.inverse = x.inverse != 0;
  g.pos64 = x.pos64 != 0;
  g.is_bf16 = x.dtype == LAGA_DTYPE_BF16;
  g.pos = pos;
  *table = &t;
  return LAGA_OK;
}

}  // namespace laga

using namespace laga;

extern "C" {

size_t laga_mla_masked_fwd_workspace_size(const laga_mla_desc* desc) {
  Dims d{};
  laga_status st;
  const Path path = masked_plan(desc, &d, &st, false);
  return path == Path::Invalid ? 0 : fwd_bytes(d, path, elem_size(desc));
}

size_t laga_mla_masked_bwd_workspace_size(const laga_mla_desc* desc) {
  Dims d{};
  laga_status st;
  const Path path = masked_plan(desc, &d, &st, true);
  return path == Path::Invalid ? 0 : bwd_bytes(d, path, elem_size(desc));
}

laga_status laga_mla_masked_fwd(const laga_mla_desc* desc, const laga_mla_mods* mods, const void* q, const void* c_kv,
                                const void* k_rope, const void* W_UK, const void* W_UV, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, laga_stream_t stream) {
  Dims d{};
  laga_status st;
  const Path path = masked_plan(desc, &d, &st, false);
  if (path == Path::Invalid) return st;
  ScoreMods sm;
  st = check_mods(mods, &sm);
  if (st != LAGA_OK) return st;
  for (const void* p : {q, c_kv, W_UK, W_UV, static_cast<const void*>(out), static_cast<const void*>(lse)})
    if (!p || !aligned16(p)) return fail(LAGA_ERR_INVALID_ARG, kTensorPointers);
  if (d.d_rope > 0 && (!k_rope || !aligned16(k_rope)))
    return fail(LAGA_ERR_INVALID_ARG, "k_rope must be non-null and 16-byte aligned%s");
  const int elem = elem_size(desc);
  if (!workspace_ok(workspace, workspace_bytes, fwd_bytes(d, path, elem))) return fail(LAGA_ERR_WORKSPACE, kWorkspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int32_t* lo = mods ? mods->key_lo : nullptr;
  const int32_t* hi = mods ? mods->key_hi : nullptr;
  if (path == Path::Simt)
    return from_launch(timed("simt_masked_fwd", s, [&] {
      return simt_masked_fwd(d, elem == 2, sm, lo, hi, q, c_kv, k_rope, W_UK, W_UV, out, lse, workspace, s);
    }));
  auto cb = [](const void* p) { return static_cast<const bf16*>(p); };
  bf16* k_ws = static_cast<bf16*>(workspace);
  bf16* v_ws = k_ws + static_cast<size_t>(d.B) * d.skv_pad * d.n_h * 128;
  char* at = static_cast<char*>(workspace) + tc_fwd_workspace(d);
  const MaskBuffers m = mask_carve(d, elem, at);
  const MaskArgs mask{m.meta(), sm};
  const KeyList list{m.seen_list, m.counters};
  LaunchResult r =
      timed("mask_prepare", s, [&] { return mask_prepare(d, true, lo, hi, c_kv, k_rope, m, true, s); });
  if (r.ok())
    r = timed("recon_fwd_gemm", s,
              [&] { return tc_recon_fwd(d, cb(m.c_kv), cb(W_UK), cb(W_UV), k_ws, v_ws, d.skv_pad, s, 0, -1, &list); });
  // Without a cap or bias a long walk is better off with one CTA per query tile (2048 rows of 128
  // heads over up to 16384 keys: 1.04 ms against 1.23), short ones with CTAs that stay (2 x 4096
  // rows of 16 heads, documents of ~100 keys: 52 us against 67; of ~800: 90 against 92; but one
  // document of 4096: 179 against 143). How long the walks are only the device knows; how long they
  // can be, the sizes say.
  const bool long_walks = mod_of(sm) == 0 && d.skv_pad >= 64 * 128;
  if (r.ok())
    r = timed("masked_attn_fwd", s, [&] {
      if (long_walks)
        return tc_attn_fwd(d, cb(q), k_ws, v_ws, cb(m.k_rope), static_cast<bf16*>(out), lse, s, &mask);
      return tc_masked_attn_fwd(d, mask, cb(q), k_ws, v_ws, cb(m.k_rope), static_cast<bf16*>(out), lse, s);
    });
  return from_launch(r);
}

laga_status laga_mla_masked_bwd(const laga_mla_desc* desc, const laga_mla_mods* mods, const void* q, const void* c_kv,
                                const void* k_rope, const void* W_UK, const void* W_UV, const void* out,
                                const float* lse, const void* dout, const laga_mla_packed* q8,
                                const laga_mla_packed* out8, void* dq, void* dc_kv, void* dk_rope, void* dW_UK,
                                void* dW_UV, void* workspace, size_t workspace_bytes, laga_stream_t stream) {
  Dims d{};
  laga_status st;
  const Path path = masked_plan(desc, &d, &st, true);
  if (path == Path::Invalid) return st;
  ScoreMods sm;
  st = check_mods(mods, &sm);
  if (st != LAGA_OK) return st;
  const bool packed = q8 != nullptr || out8 != nullptr;
  if (packed) {
    if (!q8 || !out8 || q || out)
      return fail(LAGA_ERR_INVALID_ARG, "q and out come either both as tensors or both as 8-bit checkpoints%s");
    for (const laga_mla_packed* p : {q8, out8})
      if (!p->codes || !p->scales || !aligned16(p->codes))
        return fail(LAGA_ERR_INVALID_ARG, "checkpoint pointers must be non-null and the codes 16-byte aligned%s");
  } else if (!q || !out || !aligned16(q) || !aligned16(out)) {
    return fail(LAGA_ERR_INVALID_ARG, kTensorPointers);
  }
  for (const void* p : {c_kv, W_UK, W_UV, static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dc_kv), static_cast<const void*>(dW_UK),
                        static_cast<const void*>(dW_UV)})
    if (!p || !aligned16(p)) return fail(LAGA_ERR_INVALID_ARG, kTensorPointers);
  if (d.d_rope > 0 && (!k_rope || !aligned16(k_rope) || !dk_rope || !aligned16(dk_rope)))
    return fail(LAGA_ERR_INVALID_ARG, "k_rope/dk_rope must be non-null and 16-byte aligned%s");
  const int elem = elem_size(desc);
  if (!workspace_ok(workspace, workspace_bytes, bwd_bytes(d, path, elem))) return fail(LAGA_ERR_WORKSPACE, kWorkspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int32_t* lo = mods ? mods->key_lo : nullptr;
  const int32_t* hi = mods ? mods->key_hi : nullptr;
  const bool reuse = (desc->flags & LAGA_FLAG_REUSE_KV) != 0;
  const Packed pq = packed ? Packed{q8->codes, q8->scales} : Packed{};
  const Packed po = packed ? Packed{out8->codes, out8->scales} : Packed{};
  if (path == Path::Simt)
    return from_launch(timed("simt_masked_bwd", s, [&] {
      return simt_masked_bwd(d, elem == 2, sm, lo, hi, q, c_kv, k_rope, W_UK, W_UV, out, packed ? &pq : nullptr,
                             packed ? &po : nullptr, lse, dout, BwdGrads{dq, dc_kv, dk_rope, dW_UK, dW_UV}, workspace,
                             reuse, s);
    }));
  auto cb = [](const void* p) { return static_cast<const bf16*>(p); };
  // K, V and the mask's buffers where the forward has them, then the rest of the plain layout
  char* at = static_cast<char*>(workspace) + tc_fwd_workspace(d);
  const MaskBuffers m = mask_carve(d, elem, at);
  const int G = masked_heads_per_cta(d);
  BwdWorkspace w = tc_bwd_carve(d, at - tc_fwd_workspace(d), G);
  w.k_ws = static_cast<bf16*>(workspace);
  w.v_ws = w.k_ws + static_cast<size_t>(d.B) * d.skv_pad * d.n_h * 128;
  at += tc_bwd_workspace(d, G) - tc_fwd_workspace(d);
  bf16* q_clean = reinterpret_cast<bf16*>(at);
  bf16* dout_clean = reinterpret_cast<bf16*>(at + tc_clean_q_bytes(d));
  const MaskArgs mask{m.meta(), sm};
  const KeyList list{m.seen_list, m.counters};
  const bf16* qr = packed ? q_clean : cb(q);  // what the kernels read as q
  const bf16 *c = cb(m.c_kv), *kr = cb(m.k_rope);
  LaunchResult r;
  if (!reuse) {
    r = timed("mask_prepare", s, [&] { return mask_prepare(d, true, lo, hi, c_kv, k_rope, m, true, s); });
    if (r.ok())
      r = timed("recon_fwd_gemm", s, [&] { return tc_recon_fwd(d, c, cb(W_UK), cb(W_UV), w.k_ws, w.v_ws, d.skv_pad, s, 0, -1, &list); });
  }
  if (r.ok())
    r = timed("masked_bwd_pre", s, [&] {
      return tc_mask_bwd_pre(d, cb(q), cb(out), packed ? &pq : nullptr, packed ? &po : nullptr, cb(dout), lse, w, q_clean,
                             dout_clean, m.q_bad, sm.cap > 0.f, !reuse, s);
    });
  if (r.ok())
    r = timed("masked_attn_bwd_dkdv", s,
              [&] { return tc_attn_bwd_dkdv(d, qr, kr, cb(dout), w, s, &mask, q_clean, dout_clean); });
  if (r.ok())
    r = timed("masked_attn_bwd_dq", s,
              [&] { return tc_attn_bwd_dq(d, qr, kr, cb(dout), w, static_cast<bf16*>(dq), s, &mask); });
  if (r.ok())
    r = timed("recon_bwd_dc_gemm", s, [&] {
      return tc_recon_bwd_dc(d, w.dk_ws, w.dv_ws, cb(W_UK), cb(W_UV), static_cast<bf16*>(dc_kv), s, &list);
    });
  if (r.ok())
    r = timed("recon_bwd_dw_gemm", s, [&] {
      return tc_recon_bwd_dw(d, c, w.dk_ws, w.dv_ws, static_cast<bf16*>(dW_UK), static_cast<bf16*>(dW_UV), s, &list);
    });
  if (r.ok()) r = timed("bwd_post", s, [&] { return tc_bwd_post(d, w, static_cast<bf16*>(dk_rope), s, m.seen, static_cast<bf16*>(dc_kv)); });
  return from_launch(r);
}

laga_status laga_mla_key_bounds(int64_t batch, int64_t sq, int64_t skv, int64_t q_offset, int64_t q_split,
                                int64_t q_offset2, const int32_t* doc_starts, int64_t n_docs, const int32_t* prefix,
                                int64_t window, int32_t* key_lo, int32_t* key_hi, laga_stream_t stream) {
  const int64_t lim = int64_t(1) << 30;
  if (batch < 1 || sq < 1 || skv < 1 || n_docs < 1 || q_offset < 0 || q_split < 0 || q_split >= sq || window < 0 ||
      (q_split > 0 && q_offset2 < 0))
    return fail(LAGA_ERR_INVALID_ARG, "key bounds: batch, sq, skv, n_docs >= 1, 0 <= q_split < sq, offsets and window >= 0%s");
  if (prefix && window > 0)
    return fail(LAGA_ERR_INVALID_ARG, "key bounds: a prefix outside the window is no interval; give one of the two%s");
  if (batch > 65535 || sq >= lim || skv >= lim || n_docs >= lim || q_offset >= lim || (q_split > 0 && q_offset2 >= lim))
    return fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
  for (const void* p : {static_cast<const void*>(doc_starts), static_cast<const void*>(key_lo),
                        static_cast<const void*>(key_hi)})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u))
      return fail(LAGA_ERR_INVALID_ARG, "doc_starts, key_lo and key_hi must be non-null and 4-byte aligned%s");
  if (reinterpret_cast<uintptr_t>(prefix) & 3u) return fail(LAGA_ERR_INVALID_ARG, "prefix must be 4-byte aligned%s");
  Dims d{};
  d.B = static_cast<int>(batch);
  d.Sq = static_cast<int>(sq);
  d.S = static_cast<int>(skv);
  d.q_offset = static_cast<int>(q_offset);
  d.q_split = static_cast<int>(q_split);
  d.q_offset2 = q_split > 0 ? static_cast<int>(q_offset2) : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("key_bounds", s, [&] {
    return mask_key_bounds(d, doc_starts, static_cast<int>(n_docs), prefix, static_cast<int>(std::min(window, lim)), key_lo,
                           key_hi, s);
  }));
}

laga_status laga_mla_rope(const laga_mla_rope_desc* desc, const void* pos, const void* q, const void* k_rope, void* q_out,
                          void* k_out, laga_stream_t stream) {
  RopeArgs g{};
  const RopeTable* t = nullptr;
  const laga_status st = rope_plan(desc, pos, &g, &t);
  if (st != LAGA_OK) return st;
  if ((!q && !k_rope) || !q != !q_out || !k_rope != !k_out)
    return fail(LAGA_ERR_INVALID_ARG, "rope: q or k_rope, each with its output%s");
  const uintptr_t e = g.is_bf16 ? 2 : 4;
  for (const void* p : {q, k_rope, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (reinterpret_cast<uintptr_t>(p) & (e - 1))
      return fail(LAGA_ERR_INVALID_ARG, "rope: tensors must be aligned to their type%s");
  g.q = q;
  g.k = k_rope;
  g.q_out = q_out;
  g.k_out = k_out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("rope", s, [&] { return rope(g, *t, s); }));
}

static laga_status check_pack(int32_t dtype, int64_t rows, int64_t cols, const void* x, const void* codes,
                              const void* scales) {
  if (dtype != LAGA_DTYPE_F32 && dtype != LAGA_DTYPE_BF16)
    return fail(LAGA_ERR_UNSUPPORTED, "dtype must be LAGA_DTYPE_F32 or LAGA_DTYPE_BF16%s");
  if (rows < 1 || cols < 1) return fail(LAGA_ERR_INVALID_ARG, "pack8: rows and cols must be positive%s");
  if (cols >= (int64_t(1) << 30) || rows >= (int64_t(1) << 36) || rows * ((cols + 31) / 32) >= (int64_t(1) << 33))
    return fail(LAGA_ERR_UNSUPPORTED, "pack8: problem too large%s");
  const uintptr_t e = dtype == LAGA_DTYPE_BF16 ? 2 : 4;
  if (!x || !codes || !scales || (reinterpret_cast<uintptr_t>(x) & (e - 1)))
    return fail(LAGA_ERR_INVALID_ARG, "pack8: pointers must be non-null and aligned to their type%s");
  return LAGA_OK;
}

laga_status laga_mla_pack8(int32_t dtype, int64_t rows, int64_t cols, const void* x, uint8_t* codes, uint8_t* scales,
                           laga_stream_t stream) {
  const laga_status st = check_pack(dtype, rows, cols, x, codes, scales);
  if (st != LAGA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed(
      "pack8", s, [&] { return pack8(dtype == LAGA_DTYPE_BF16, rows, static_cast<int>(cols), x, codes, scales, s); }));
}

laga_status laga_mla_unpack8(int32_t dtype, int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales,
                             void* x, laga_stream_t stream) {
  const laga_status st = check_pack(dtype, rows, cols, x, codes, scales);
  if (st != LAGA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("unpack8", s, [&] {
    return unpack8(dtype == LAGA_DTYPE_BF16, rows, static_cast<int>(cols), Packed{codes, scales}, x, s);
  }));
}

}  // extern "C"
