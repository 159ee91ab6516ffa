// Host implementation of the rotary and paged-cache part of the C ABI (flexattn.h):
// argument validation and kernel launches.  Nothing here allocates device memory or
// synchronises the host.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_common.cuh"
#include "flexattn.h"
#include "paged_decode.cuh"
#include "rope.cuh"
#include "serving_rules.h"
#include "shared_prefix.cuh"

using fa::aligned16;
using fa::check_tensor;
using fa::kMaxLen;
using fa::kWorkspaceBytes;
using fa::sm_count;
using fa::tmap_for;

namespace {

bool same_dims(const fa_tensor* a, const fa_tensor* b)
{
    for (int i = 0; i < 4; ++i)
        if (a->dims[i] != b->dims[i]) return false;
    return true;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int check_rope(const fa_rope* r, int64_t D)
{
    if (r->rotary_dim < 0 || r->rotary_dim > D) return FA_ERR_INVALID_ARG;
    if (r->rotary_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (r->rotary_dim > 0 && !r->inv_freq) return FA_ERR_INVALID_ARG;
    if (!(r->amplitude >= 0.f) || std::isinf(r->amplitude)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

void set_rope(fa::RopeParams& P, const fa_rope* r, bool inverse)
{
    P.inv_freq = r ? r->inv_freq : nullptr;
    P.rotary = r ? r->rotary_dim : 0;
    P.interleaved = r && r->interleaved ? 1 : 0;
    P.amplitude = r && r->amplitude != 0.f ? r->amplitude : 1.f;
    P.sin_sign = inverse ? -1.f : 1.f;
}

fa::RopeGroup rope_group(const fa_tensor* x, const fa_tensor* y, bool rotate, bool paged)
{
    fa::RopeGroup g;
    g.x = static_cast<const uint16_t*>(x->data);
    g.x_st0 = x->strides[0]; g.x_st1 = x->strides[1]; g.x_st2 = x->strides[2];
    g.y = static_cast<uint16_t*>(y->data);
    g.y_st0 = y->strides[0]; g.y_st1 = y->strides[1]; g.y_st2 = y->strides[2];
    g.H = (int32_t)x->dims[1];
    g.rotate = rotate ? 1 : 0;
    g.paged = paged ? 1 : 0;
    return g;
}

// The status of a launch; nothing is thrown through the C ABI.
template <class Launch>
int launched(Launch launch)
{
    try {
        return launch() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    } catch (...) {
        return FA_ERR_CUDA;
    }
}

// Pools [num_pages, Hkv, FA_BLOCK_SIZE, D] of the same shape.
int check_pools(const fa_tensor* k, const fa_tensor* v)
{
    int rc;
    if ((rc = check_tensor(k)) || (rc = check_tensor(v))) return rc;
    if (!same_dims(k, v) || k->dims[2] != FA_BLOCK_SIZE) return FA_ERR_INVALID_ARG;
    if (k->dims[0] > INT32_MAX) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

} // namespace

extern "C" {

int fa_rope_frequencies(int rotary_dim, double base, const fa_rope_scaling* scaling, double* inv_freq,
                        float* amplitude)
{
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || !(base > 1.0) || std::isinf(base) || !inv_freq)
        return FA_ERR_INVALID_ARG;
    const int kind = scaling ? scaling->kind : FA_ROPE_UNSCALED;
    if (kind < FA_ROPE_UNSCALED || kind > FA_ROPE_YARN) return FA_ERR_INVALID_ARG;
    const double s = kind == FA_ROPE_UNSCALED ? 1.0 : scaling->factor;
    if (!(s >= 1.0) || std::isinf(s)) return FA_ERR_INVALID_ARG;
    const bool bands = kind == FA_ROPE_BANDS || kind == FA_ROPE_YARN;
    if (bands && (!(scaling->original_len > 0) || !(scaling->rot_lo > 0) || !(scaling->rot_hi > scaling->rot_lo) ||
                  std::isinf(scaling->rot_hi) || std::isinf(scaling->original_len)))
        return FA_ERR_INVALID_ARG;
    if (kind == FA_ROPE_BASE && rotary_dim == 2) return FA_ERR_INVALID_ARG;
    const double r = rotary_dim, pi2 = 6.283185307179586476925;
    const double b = kind == FA_ROPE_BASE ? base * std::pow(s, r / (r - 2)) : base;
    double lo = 0, hi = 0;
    if (kind == FA_ROPE_YARN) {
        // index of the pair that turns n times over original_len positions
        auto index = [&](double n) { return r * std::log(scaling->original_len / (n * pi2)) / (2 * std::log(base)); };
        lo = std::floor(index(scaling->rot_hi));
        hi = std::ceil(index(scaling->rot_lo));
        lo = lo < 0 ? 0 : lo;
        hi = hi > r - 1 ? r - 1 : hi;
        if (hi <= lo) hi = lo + 0.001;  // one index: a step
    }
    for (int j = 0; j < rotary_dim / 2; ++j) {
        const double f = std::pow(b, -2.0 * j / r);
        double share = 0;  // how far towards f / factor
        if (kind == FA_ROPE_LINEAR) share = 1;
        if (kind == FA_ROPE_BANDS) {
            const double turns = scaling->original_len * f / pi2;
            share = (scaling->rot_hi - turns) / (scaling->rot_hi - scaling->rot_lo);
        }
        if (kind == FA_ROPE_YARN) share = (j - lo) / (hi - lo);
        share = share < 0 ? 0 : share > 1 ? 1 : share;
        inv_freq[j] = f / s * share + f * (1 - share);
    }
    if (amplitude) *amplitude = kind == FA_ROPE_YARN ? (float)(0.1 * std::log(s) + 1.0) : 1.f;
    return FA_OK;
}

int fa_rope_apply(const fa_tensor* q, const fa_tensor* k, const fa_rope* rope, const int32_t* positions,
                  int64_t positions_stride, int64_t position_offset, int inverse, const fa_tensor* q_out,
                  const fa_tensor* k_out, void* stream)
{
    if (!rope || (!q && !k) || !q != !q_out || !k != !k_out) return FA_ERR_INVALID_ARG;
    int rc;
    const fa_tensor* in[2] = {q, k};
    const fa_tensor* out[2] = {q_out, k_out};
    const fa_tensor* any = q ? q : k;
    const int64_t B = any->dims[0], S = any->dims[2], D = any->dims[3];
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        if ((rc = check_tensor(in[i])) || (rc = check_tensor(out[i]))) return rc;
        if (!same_dims(in[i], out[i])) return FA_ERR_INVALID_ARG;
        if (in[i]->dims[0] != B || in[i]->dims[2] != S || in[i]->dims[3] != D) return FA_ERR_INVALID_ARG;
        if (in[i]->dims[1] > 65535) return FA_ERR_INVALID_ARG;
    }
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if ((rc = check_rope(rope, D)) != FA_OK) return rc;
    if (B > 65535 || S > kMaxLen || positions_stride < 0) return FA_ERR_INVALID_ARG;
    if (!positions && (position_offset < -kMaxLen || position_offset > kMaxLen)) return FA_ERR_INVALID_ARG;
    fa::RopeParams P;
    std::memset(&P, 0, sizeof P);
    for (int i = 0; i < 2; ++i)
        if (in[i]) P.g[i] = rope_group(in[i], out[i], true, false);
    if (B == 0 || S == 0 || P.g[0].H + P.g[1].H == 0) return FA_OK;
    if (B * S > kMaxLen) return FA_ERR_UNSUPPORTED;
    set_rope(P, rope, inverse != 0);
    P.B = (int32_t)B;
    P.S = S;
    P.tokens = B * S;
    P.positions = positions;
    P.pos_stride = positions_stride;
    P.pos_offset = position_offset;
    const int sms = sm_count();
    if (sms <= 0) return FA_ERR_CUDA;
    return fa::launch_rope(P, (int)D, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_paged_append(const fa_tensor* k, const fa_tensor* v, const fa_tensor* q, const fa_rope* rope,
                    const int32_t* cache_lens, const int32_t* new_lens, const int32_t* page_table,
                    int64_t page_table_stride, int64_t pages_per_seq, const fa_tensor* k_pages,
                    const fa_tensor* v_pages, const fa_tensor* q_out, void* workspace, size_t workspace_bytes,
                    void* stream)
{
    if (!q != !q_out) return FA_ERR_INVALID_ARG;
    int rc;
    if ((rc = check_tensor(k)) || (rc = check_tensor(v)) || (rc = check_pools(k_pages, v_pages))) return rc;
    const int64_t B = k->dims[0], Hkv = k->dims[1], S = k->dims[2], D = k->dims[3];
    if (!same_dims(k, v)) return FA_ERR_INVALID_ARG;
    if (k_pages->dims[1] != Hkv || k_pages->dims[3] != D) return FA_ERR_INVALID_ARG;
    if (q) {
        if ((rc = check_tensor(q)) || (rc = check_tensor(q_out))) return rc;
        if (!same_dims(q, q_out)) return FA_ERR_INVALID_ARG;
        if (q->dims[0] != B || q->dims[2] != S || q->dims[3] != D || q->dims[1] > 65535) return FA_ERR_INVALID_ARG;
    }
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (rope && (rc = check_rope(rope, D)) != FA_OK) return rc;
    if (B > 65535 || Hkv > 65535 || S > kMaxLen) return FA_ERR_INVALID_ARG;
    if (pages_per_seq < 0 || pages_per_seq > kMaxLen / FA_BLOCK_SIZE || page_table_stride < 0) return FA_ERR_INVALID_ARG;
    if (B > 1 && page_table_stride < pages_per_seq) return FA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kWorkspaceBytes || !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    if (B == 0 || S == 0 || (Hkv == 0 && (!q || q->dims[1] == 0))) return FA_OK;
    if (!cache_lens || (pages_per_seq > 0 && !page_table)) return FA_ERR_INVALID_ARG;
    if (B * S > kMaxLen) return FA_ERR_UNSUPPORTED;
    fa::RopeParams P;
    std::memset(&P, 0, sizeof P);
    set_rope(P, rope, false);
    if (q) P.g[0] = rope_group(q, q_out, true, false);
    P.g[1] = rope_group(k, k_pages, true, true);
    P.g[2] = rope_group(v, v_pages, false, true);
    P.B = (int32_t)B;
    P.S = S;
    P.tokens = B * S;
    P.cache_lens = cache_lens;
    P.new_lens = new_lens;
    P.page_table = page_table;
    P.pt_stride = page_table_stride;
    P.pt_width = pages_per_seq;
    P.num_pages = (int32_t)k_pages->dims[0];
    P.status = static_cast<int*>(workspace);
    const int sms = sm_count();
    if (sms <= 0) return FA_ERR_CUDA;
    return fa::launch_rope(P, (int)D, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

} // extern "C"

namespace {

// Workspace of a paged decode: the status word, a counter per team, then per partial
// result (two per team) the (running max, sum) and the unnormalised O of every packed
// query row, each part 256-byte aligned.  The counters lie at the same place for every
// shape, since they alone must be zero when a call starts.  With a shared prefix, the
// prefix's partial results and every row's own state follow.
struct PdLayout {
    size_t arrived, ml, o, split, pre_ml, pre_o, own_ml, own_o, end;
    int sms;
};

PdLayout pd_layout(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t prefix_pages)
{
    PdLayout L;
    L.sms = sm_count();
    const size_t ctas = L.sms > 0 ? L.sms : 1, teams = ctas * fa::kPdTeams, parts = 2 * teams * (size_t)rows;
    L.arrived = kWorkspaceBytes;
    L.ml = L.arrived + align256(teams * sizeof(uint32_t));
    L.o = L.ml + align256(parts * 2 * sizeof(float));
    L.end = L.o + parts * D * sizeof(float);
    L.split = L.pre_ml = L.pre_o = L.own_ml = L.own_o = 0;
    if (prefix_pages > 0) {
        const fa::SpGeom g = fa::sp_geom(B * rows, (int32_t)prefix_pages);
        const int64_t entries = Hkv * g.per_head;
        const size_t pre_ctas = entries < (int64_t)ctas ? (size_t)entries : ctas;
        const size_t slots = 2 * ((size_t)Hkv * fa::sp_cols(g) + pre_ctas) * fa::kSpRows;
        const size_t own = (size_t)(B * Hkv * rows);
        L.split = align256(L.end);
        L.pre_ml = L.split + 256;
        L.pre_o = L.pre_ml + align256(slots * 2 * sizeof(float));
        L.own_ml = L.pre_o + slots * D * sizeof(float);
        L.own_o = L.own_ml + align256(own * 2 * sizeof(float));
        L.end = L.own_o + own * D * sizeof(float);
    }
    return L;
}

// Head counts, rows and a prefix that the calls take: 0, or the status they are refused with.
int check_shape(int64_t B, int64_t Hq, int64_t Hkv, int64_t q_len, int64_t D, int64_t prefix_pages)
{
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (Hkv < 1 || Hq % Hkv != 0 || B > 65535 || Hkv > 65535) return FA_ERR_INVALID_ARG;
    const int64_t G = Hq / Hkv, most = fa::kPdMaxRows;
    if (q_len > most || (q_len > 0 && G > most) || G * q_len > most) return FA_ERR_UNSUPPORTED;
    const int64_t rows = G * q_len;
    // the prefix's work list
    if (B * rows > 0 && Hkv * (B * rows / (2 * fa::kSpRows) + 2) * prefix_pages > kMaxLen) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// fa_decode_paged and fa_decode_shared (prefix_len > 0).
int decode_paged(const fa_tensor* q, const fa_tensor* k_pages, const fa_tensor* v_pages, const int32_t* page_table,
                 int64_t page_table_stride, int64_t pages_per_seq, const int32_t* seq_lens, int64_t window,
                 int64_t prefix_pages, const fa_score_mod* sm, float scale, const fa_tensor* o, float* lse,
                 void* workspace, size_t workspace_bytes, void* stream)
{
    int rc;
    if ((rc = check_tensor(q)) || (rc = check_tensor(o)) || (rc = check_pools(k_pages, v_pages))) return rc;
    const int64_t B = q->dims[0], Hq = q->dims[1], q_len = q->dims[2], D = q->dims[3];
    const int64_t Hkv = k_pages->dims[1], num_pages = k_pages->dims[0];
    if (!same_dims(q, o) || k_pages->dims[3] != D) return FA_ERR_INVALID_ARG;
    if (pages_per_seq < 0 || pages_per_seq > kMaxLen / FA_BLOCK_SIZE || page_table_stride < 0) return FA_ERR_INVALID_ARG;
    if (B > 1 && page_table_stride < pages_per_seq) return FA_ERR_INVALID_ARG;
    if ((rc = check_shape(B, Hq, Hkv, q_len, D, prefix_pages)) != FA_OK) return rc;
    const int kind = sm ? sm->kind : FA_SCORE_NONE;
    if (kind < FA_SCORE_NONE || kind > FA_SCORE_BIAS_SOFTCAP) return FA_ERR_INVALID_ARG;
    if (kind == FA_SCORE_BIAS || kind == FA_SCORE_BIAS_SOFTCAP) return FA_ERR_UNSUPPORTED;
    if (kind == FA_SCORE_ALIBI && !sm->alibi_slopes) return FA_ERR_INVALID_ARG;
    const float factor = scale > 0.f ? scale : 1.0f / std::sqrt((float)D);
    // cap tanh(s / cap) with the cap and its inverse taken into the scores' factors
    if (kind == FA_SCORE_SOFTCAP &&
        (!(sm->softcap > 0.f) || !std::isfinite(factor / sm->softcap) || !std::isfinite(sm->softcap * 1.5f)))
        return FA_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return FA_ERR_INVALID_ARG;
    if (B * Hq * q_len == 0) return FA_OK;
    if (!seq_lens || (pages_per_seq > 0 && (!page_table || num_pages < 1))) return FA_ERR_INVALID_ARG;
    if (B * Hkv * pages_per_seq > kMaxLen) return FA_ERR_UNSUPPORTED;  // the work list
    const int64_t row0_pages = fa::takes_prefix_once(B, Hkv, (Hq / Hkv) * q_len, D, prefix_pages) ? 0 : prefix_pages;
    if (row0_pages) prefix_pages = 0;
    const PdLayout lay = pd_layout(B, Hkv, (Hq / Hkv) * q_len, D, prefix_pages);
    if (lay.sms <= 0) return FA_ERR_CUDA;
    if (workspace_bytes < lay.end) return FA_ERR_INVALID_ARG;

    fa::PdParams P;
    std::memset(&P, 0, sizeof P);
    // without pages no sequence has a key and the maps are never read
    if (num_pages > 0 && (!tmap_for(&P.tm_k, k_pages) || !tmap_for(&P.tm_v, v_pages))) return FA_ERR_INVALID_ARG;
    P.q = static_cast<const uint16_t*>(q->data);
    P.q_st0 = q->strides[0]; P.q_st1 = q->strides[1]; P.q_st2 = q->strides[2];
    P.o = static_cast<uint16_t*>(o->data);
    P.o_st0 = o->strides[0]; P.o_st1 = o->strides[1]; P.o_st2 = o->strides[2];
    P.lse = lse;
    P.B = (int32_t)B;
    P.Hq = (int32_t)Hq;
    P.Hkv = (int32_t)Hkv;
    P.G = (int32_t)(Hq / Hkv);
    P.q_len = (int32_t)q_len;
    P.rows = P.G * P.q_len;
    P.seq_lens = seq_lens;
    P.page_table = page_table;
    P.pt_stride = page_table_stride;
    P.pt_width = (int32_t)pages_per_seq;
    P.num_pages = (int32_t)num_pages;
    P.prefix_pages = (int32_t)prefix_pages;
    P.row0_pages = (int32_t)row0_pages;
    P.has_window = window >= 0 ? 1 : 0;
    P.window = window >= 0 ? (window < kMaxLen ? window : kMaxLen) : 0;
    P.scale = factor;
    if (kind == FA_SCORE_SOFTCAP) {
        P.softcap = sm->softcap;
        P.softcap_in = P.scale / sm->softcap;
    }
    P.slopes = kind == FA_SCORE_ALIBI ? sm->alibi_slopes : nullptr;
    const int64_t most = B * Hkv * pages_per_seq;  // one CTA per SM, never more than pages in all
    P.grid = (int32_t)(most < 1 ? 1 : most < lay.sms ? most : lay.sms);
    P.teams = fa::teams_that_pay(B * Hkv, fa::pages_of_a_segment(pages_per_seq, window, q_len), P.rows, D,
                                 lay.sms * fa::kPdTeams);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    P.arrived = reinterpret_cast<unsigned*>(ws + lay.arrived);
    P.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    P.part_o = reinterpret_cast<float*>(ws + lay.o);
    P.status = reinterpret_cast<int*>(ws);
    P.watchdog_ns = fa::watchdog_ns();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (prefix_pages == 0) return launched([&] { return fa::launch_paged_decode(P, (int)D, kind, st); });

    if (lay.sms < 2) return FA_ERR_UNSUPPORTED;
    P.own_ml = reinterpret_cast<float*>(ws + lay.own_ml);
    P.own_o = reinterpret_cast<float*>(ws + lay.own_o);
    fa::SpParams S;
    std::memset(&S, 0, sizeof S);
    S.tm_k = P.tm_k;
    S.tm_v = P.tm_v;
    S.q = P.q;
    S.q_st0 = P.q_st0; S.q_st1 = P.q_st1; S.q_st2 = P.q_st2;
    S.B = P.B; S.Hkv = P.Hkv; S.G = P.G; S.q_len = P.q_len; S.rows = P.rows;
    S.seq_lens = seq_lens;
    S.prefix_row = page_table;
    S.num_pages = P.num_pages;
    S.scale = P.scale; S.softcap = P.softcap; S.softcap_in = P.softcap_in;
    S.slopes = P.slopes;
    S.geom = fa::sp_geom(B * P.rows, (int32_t)prefix_pages);
    S.sms = lay.sms;
    S.split = reinterpret_cast<int32_t*>(ws + lay.split);
    S.part_ml = reinterpret_cast<float*>(ws + lay.pre_ml);
    S.part_o = reinterpret_cast<float*>(ws + lay.pre_o);
    S.o = P.o;
    S.o_st0 = P.o_st0; S.o_st1 = P.o_st1; S.o_st2 = P.o_st2;
    S.lse = lse;
    S.own_o = P.own_o;
    S.own_ml = P.own_ml;
    S.pt_width = P.pt_width;
    S.status = P.status;
    S.watchdog_ns = P.watchdog_ns;
    if ((rc = launched([&] { return fa::launch_shared_decode(S, P, (int)D, kind, st); })) != FA_OK) return rc;
    return launched([&] { return fa::launch_shared_join(S, (int)D, st); });
}

} // namespace

extern "C" {

size_t fa_decode_paged_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t q_len, int64_t D)
{
    if (B < 0 || Hq < 0 || q_len < 0 || check_shape(B, Hq, Hkv, q_len, D, 0) != FA_OK) return 0;
    if (B * Hq * q_len == 0) return kWorkspaceBytes;
    return pd_layout(B, Hkv, (Hq / Hkv) * q_len, D, 0).end;
}

int fa_decode_paged(const fa_tensor* q, const fa_tensor* k_pages, const fa_tensor* v_pages, const int32_t* page_table,
                    int64_t page_table_stride, int64_t pages_per_seq, const int32_t* seq_lens, int64_t window,
                    const fa_score_mod* sm, float scale, const fa_tensor* o, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream)
{
    return decode_paged(q, k_pages, v_pages, page_table, page_table_stride, pages_per_seq, seq_lens, window, 0, sm,
                        scale, o, lse, workspace, workspace_bytes, stream);
}

size_t fa_decode_shared_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t q_len, int64_t D,
                                       int64_t prefix_len)
{
    if (prefix_len < 0 || prefix_len > kMaxLen || B < 0 || Hq < 0 || q_len < 0) return 0;
    const int64_t pages = prefix_len / FA_BLOCK_SIZE;
    if (check_shape(B, Hq, Hkv, q_len, D, pages) != FA_OK) return 0;
    if (B * Hq * q_len == 0) return kWorkspaceBytes;
    return pd_layout(B, Hkv, (Hq / Hkv) * q_len, D, fa::takes_prefix_once(B, Hkv, (Hq / Hkv) * q_len, D, pages) ? pages : 0).end;
}

int fa_decode_shared(const fa_tensor* q, const fa_tensor* k_pages, const fa_tensor* v_pages,
                     const int32_t* page_table, int64_t page_table_stride, int64_t pages_per_seq,
                     const int32_t* seq_lens, int64_t prefix_len, const fa_score_mod* sm, float scale,
                     const fa_tensor* o, float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    if (prefix_len < 0 || prefix_len % FA_BLOCK_SIZE != 0) return FA_ERR_INVALID_ARG;
    if (prefix_len / FA_BLOCK_SIZE > pages_per_seq) return FA_ERR_INVALID_ARG;
    return decode_paged(q, k_pages, v_pages, page_table, page_table_stride, pages_per_seq, seq_lens, -1,
                        prefix_len / FA_BLOCK_SIZE, sm, scale, o, lse, workspace, workspace_bytes, stream);
}

} // extern "C"
