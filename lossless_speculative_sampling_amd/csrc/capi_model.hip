// The C ABI's entry points on either side of the verification: verification from given
// probabilities, draft-tree rows, the rotary append and the attention over a shared prefix.
// Argument validation, workspace layout and kernel launches.
#include <cmath>

#include "attention.h"
#include "kvcache.h"
#include "probs.h"

using namespace sv;

namespace {

size_t up_to(size_t x, size_t a) { return (x + a - 1) / a * a; }

int launched() { return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A grid's threads are counted in 32 bits: at most this many workgroups of 256.
constexpr int64_t kMaxGroups = (1ll << 24) - 1;
constexpr int kMaxHeadDim = 1024;
// Tokens of a vocabulary or a prefix: positions a few tiles past the end still fit in 32 bits.
constexpr int64_t kMaxLen = 0x7fff0000;

// What every user of a paged cache needs of its description; SPEC_OK or an error.
int check_cache(const spec_kv_cache* c, int dtype) {
    if (!c || !c->k || !c->v || c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1) return SPEC_EINVAL;
    if ((int64_t)c->num_pages * c->page_size > 0x7fffffffll) return SPEC_EINVAL;
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return SPEC_EINVAL;
    if (c->dtype != dtype && c->dtype != SPEC_E4M3) return SPEC_EDTYPE;
    return SPEC_OK;
}

bool half_type(int dtype) { return dtype == SPEC_BF16 || dtype == SPEC_FP16; }

}  // namespace

extern "C" {

size_t spec_verify_probs_workspace_bytes(int B, int V) {
    if (B < 1 || V <= probs::kOneLaunchV || V > kMaxLen) return 0;
    const int64_t cell = probs::cell_of(V), cells = (V + cell - 1) / cell;
    if (B * cells > kMaxGroups) return 0;
    return up_to((size_t)B * sizeof(probs::Rec), 256) + up_to((size_t)(B * cells) * sizeof(double), 256);
}

int spec_verify_probs(const void* draft_probs, int64_t draft_request_stride, int64_t draft_row_stride,
                      const void* target_probs, int64_t target_request_stride, int64_t target_row_stride, int dtype,
                      int B, int K, int V, const int32_t* draft_tokens, const int32_t* draft_lens, const void* accept_u,
                      const void* sample_v, int uniform_dtype, uint32_t flags, int32_t* out_k, int32_t* out_tstar,
                      int32_t* out_emitted, float* out_resid_mass, uint32_t* out_status, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    const uint32_t kinds = SPEC_UNIFORM_DRAFT | SPEC_POINT_DRAFT;
    if ((flags & ~kinds) != 0 || (flags & kinds) == kinds) return SPEC_EINVAL;
    if ((!draft_probs && !flags) || !target_probs || !draft_tokens || !accept_u || !sample_v || !out_k || !out_tstar)
        return SPEC_EINVAL;
    if (B < 1 || K < 1 || V < 1) return SPEC_EINVAL;
    if (dtype != SPEC_FP32 && !half_type(dtype)) return SPEC_EDTYPE;
    if (uniform_dtype != SPEC_FP32 && uniform_dtype != SPEC_FP64) return SPEC_EDTYPE;
    const uintptr_t e = dtype == SPEC_FP32 ? 4 : 2, u = uniform_dtype == SPEC_FP64 ? 8 : 4;
    if (!aligned(target_probs, e) || (!flags && !aligned(draft_probs, e)) || !aligned(accept_u, u) || !aligned(sample_v, u))
        return SPEC_EINVAL;
    const size_t need = spec_verify_probs_workspace_bytes(B, V);
    if (V > probs::kOneLaunchV) {
        if (need == 0) return SPEC_EINVAL;
        if (!workspace || !aligned(workspace, 8) || workspace_bytes < need) return SPEC_EWORKSPACE;
    } else if (B > kMaxGroups) {
        return SPEC_EINVAL;
    }
    probs::Args a{};
    a.draft = flags ? nullptr : draft_probs;
    a.draft_req = draft_request_stride;
    a.draft_row = draft_row_stride;
    a.target = target_probs;
    a.target_req = target_request_stride;
    a.target_row = target_row_stride;
    a.B = B;
    a.K = K;
    a.V = V;
    a.tokens = draft_tokens;
    a.lens = draft_lens;
    a.u = accept_u;
    a.v = sample_v;
    a.u64 = uniform_dtype == SPEC_FP64;
    a.flags = flags;
    a.out_k = out_k;
    a.out_tstar = out_tstar;
    a.out_emitted = out_emitted;
    a.out_mass = out_resid_mass;
    a.out_status = out_status;
    a.cell = probs::cell_of(V);
    a.cells = (int)(((int64_t)V + a.cell - 1) / a.cell);
    a.per = probs::per_of(B, a.cells);
    if (need) {
        a.recs = static_cast<probs::Rec*>(workspace);
        a.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + up_to((size_t)B * sizeof(probs::Rec), 256));
    }
    probs::launch(a, dtype, stream);
    return launched();
}

int spec_tree_rows(const int32_t* tree_tokens, const int32_t* tree_parents, const int32_t* node_slots,
                   const int32_t* ctx_len, int B, int N, int max_depth, int32_t* out_positions,
                   int32_t* out_append_slots, int32_t* out_suffix_slots, int32_t* out_suffix_len, hipStream_t stream) {
    if (!tree_tokens || !tree_parents || !node_slots || !ctx_len || !out_positions || !out_append_slots ||
        !out_suffix_slots || !out_suffix_len)
        return SPEC_EINVAL;
    if (B < 1 || N < 1 || max_depth < 1 || N > kMaxLen || max_depth > kMaxLen || B > kMaxGroups) return SPEC_EINVAL;
    kv::RowsArgs a{tree_tokens, tree_parents, node_slots, ctx_len, B, N, max_depth, out_positions, out_append_slots,
                   out_suffix_slots, out_suffix_len};
    kv::launch_rows(a, stream);
    return launched();
}

int spec_rope_frequencies(int rot_dim, double base, double factor, double low, double high, int original_len,
                          double* out) {
    if (!out || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > kMaxHeadDim || original_len < 1) return SPEC_EINVAL;
    if (!(base > 0.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) || !(low <= high) ||
        low == -HUGE_VAL)
        return SPEC_EINVAL;
    const double two_pi = 6.283185307179586477;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        const double n = original_len * f / two_pi;
        const double g = low == high ? (n >= low ? 1.0 : 0.0) : std::fmin(std::fmax((n - low) / (high - low), 0.0), 1.0);
        out[i] = f * (g + (1.0 - g) / factor);
    }
    return SPEC_OK;
}

int spec_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                   int64_t q_out_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                   const void* v, int64_t v_token_stride, int64_t v_head_stride, int dtype, int T, int q_heads,
                   int heads, int head_dim, const int32_t* positions, const int32_t* slots, const double* freqs,
                   int rot_dim, float rope_scale, uint32_t rope_flags, const spec_kv_cache* cache, uint32_t* out_status,
                   hipStream_t stream) {
    if (T == 0) return SPEC_OK;  // (empty arrays may be null)
    if ((!q && !k) || (q && !q_out) || (!k != !v) || (!k != !cache) || (k && !slots)) return SPEC_EINVAL;
    if (T < 0 || T > kMaxGroups || head_dim < 1 || head_dim > kMaxHeadDim) return SPEC_EINVAL;
    if ((q && q_heads < 1) || (k && heads < 1) || q_heads > (1 << 16) || heads > (1 << 16)) return SPEC_EINVAL;
    if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > head_dim || (rot_dim && (!positions || !freqs))) return SPEC_EINVAL;
    if ((rope_flags & ~(uint32_t)SPEC_ROPE_INTERLEAVED) != 0 || !std::isfinite(rope_scale)) return SPEC_EINVAL;
    if (!half_type(dtype)) return SPEC_EDTYPE;
    if (!aligned(q, 2) || !aligned(q_out, 2) || !aligned(k, 2) || !aligned(v, 2)) return SPEC_EINVAL;
    if (q && q == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride)) return SPEC_EINVAL;
    kv::AppendArgs a{};
    if (k) {
        const int rc = check_cache(cache, dtype);
        if (rc != SPEC_OK) return rc;
        if (cache->heads != heads || cache->head_dim != head_dim) return SPEC_EINVAL;
        if (cache->dtype != SPEC_E4M3 && (!aligned(cache->k, 2) || !aligned(cache->v, 2))) return SPEC_EINVAL;
        a.cache = *cache;
        if (cache->dtype != SPEC_E4M3) a.cache.k_scale = a.cache.v_scale = nullptr;
    }
    a.q = q;
    a.q_out = q_out;
    a.k = k;
    a.v = v;
    a.qs = {q_token_stride, q_head_stride};
    a.qo = {q_out_token_stride, q_out_head_stride};
    a.ks = {k_token_stride, k_head_stride};
    a.vs = {v_token_stride, v_head_stride};
    a.T = T;
    a.q_heads = q ? q_heads : 0;
    a.heads = k ? heads : 0;
    a.D = head_dim;
    a.positions = positions;
    a.slots = k ? slots : nullptr;
    a.freqs = freqs;
    a.rot = rot_dim;
    a.rope_scale = rope_scale;
    a.interleaved = (rope_flags & SPEC_ROPE_INTERLEAVED) != 0;
    a.out_status = out_status;
    // whole vectors of eight elements on both sides
    bool vec = head_dim % 8 == 0 && rot_dim % (a.interleaved ? 8 : 16) == 0;
    if (q)
        vec = vec && aligned(q, 16) && aligned(q_out, 16) &&
              ((q_token_stride | q_head_stride | q_out_token_stride | q_out_head_stride) & 7) == 0;
    if (k)
        vec = vec && aligned(k, 16) && aligned(v, 16) &&
              ((k_token_stride | k_head_stride | v_token_stride | v_head_stride | cache->page_stride |
                cache->token_stride | cache->head_stride) & 7) == 0 &&
              aligned(cache->k, cache->dtype == SPEC_E4M3 ? 8 : 16) && aligned(cache->v, cache->dtype == SPEC_E4M3 ? 8 : 16);
    kv::launch_append(a, dtype, vec, stream);
    return launched();
}

size_t spec_prefix_attention_workspace_bytes(int R, int G, int q_heads, int heads, int head_dim, int64_t max_prefix,
                                             int max_suffix) {
    if (R < 0 || G < 1 || heads < 1 || q_heads < heads || q_heads % heads != 0 || q_heads > (1 << 16)) return 0;
    if (head_dim < 8 || head_dim > attn::kMaxD || head_dim % 8 != 0 || max_prefix < 0 || max_prefix > kMaxLen ||
        max_suffix < 0 || G > kMaxGroups || (int64_t)R * q_heads > 4 * kMaxGroups)
        return 0;
    const attn::Plan p = attn::plan_of(R, G, q_heads, heads, head_dim, max_prefix, max_suffix);
    if ((int64_t)p.slots * heads + p.suffix_blocks > kMaxGroups) return 0;
    return p.bytes;
}

int spec_prefix_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride, int dtype, int R, int q_heads,
                          const spec_kv_cache* cache, int G, const int32_t* row_start, const int32_t* page_table,
                          int max_pages, const int32_t* prefix_len, const int32_t* suffix_slots, int max_suffix,
                          const int32_t* suffix_len, float scale, void* out, int64_t out_row_stride,
                          int64_t out_head_stride, float* out_lse, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    if (R == 0) return SPEC_OK;  // (empty arrays may be null)
    if (!q || !cache || !row_start || !out || q == out || max_pages < 0 || max_suffix < 0) return SPEC_EINVAL;
    if (max_pages && (!page_table || !prefix_len)) return SPEC_EINVAL;
    if (max_suffix && (!suffix_slots || !suffix_len)) return SPEC_EINVAL;
    if (!std::isfinite(scale)) return SPEC_EINVAL;
    if (!half_type(dtype)) return SPEC_EDTYPE;
    const int rc = check_cache(cache, dtype);
    if (rc != SPEC_OK) return rc;
    const int64_t most = (int64_t)max_pages * cache->page_size;
    const size_t need = spec_prefix_attention_workspace_bytes(R, G, q_heads, cache->heads, cache->head_dim, most,
                                                             max_suffix);
    if (need == 0) return SPEC_EINVAL;
    const uintptr_t kv_align = cache->dtype == SPEC_E4M3 ? 8 : 16;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache->k, kv_align) || !aligned(cache->v, kv_align) ||
        ((q_row_stride | q_head_stride | out_row_stride | out_head_stride | cache->page_stride | cache->token_stride |
          cache->head_stride) & 7) != 0)
        return SPEC_EINVAL;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return SPEC_EWORKSPACE;
    attn::Args a{};
    a.q = q;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.R = R;
    a.q_heads = q_heads;
    a.heads = cache->heads;
    a.D = cache->head_dim;
    a.per = q_heads / cache->heads;
    a.cache = *cache;
    if (cache->dtype != SPEC_E4M3) a.cache.k_scale = a.cache.v_scale = nullptr;
    a.G = G;
    a.row_start = row_start;
    a.table = page_table;
    a.max_pages = max_pages;
    a.prefix_len = prefix_len;
    a.lists = suffix_slots;
    a.max_suffix = max_suffix;
    a.suffix_len = suffix_len;
    a.scale = scale;
    a.out = out;
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.lse = out_lse;
    const int page = cache->page_size;
    a.page_shift = (page & (page - 1)) == 0 ? __builtin_ctz((unsigned)page) : -1;
    const attn::Plan p = attn::plan_of(R, G, q_heads, cache->heads, cache->head_dim, most, max_suffix);
    char* ws = static_cast<char*>(workspace);
    a.want = p.want;
    a.slots = p.slots;
    a.suffix_blocks = (int)p.suffix_blocks;
    a.piece_o = reinterpret_cast<float*>(ws + p.piece_o);
    a.piece_ml = reinterpret_cast<float2*>(ws + p.piece_ml);
    a.suffix_o = reinterpret_cast<float*>(ws + p.suffix_o);
    a.suffix_ml = reinterpret_cast<float2*>(ws + p.suffix_ml);
    a.groups = reinterpret_cast<int2*>(ws + p.groups);
    attn::launch(a, p.tile, dtype, stream);
    return launched();
}

}  // extern "C"
