// Host side of the C ABI of head norms and rotary positions: checks and launches (nr_internal.h has the operator).
#include <cmath>

#include "nr_internal.h"

namespace dplr {
namespace nr {
namespace {

constexpr size_t kAlign = 256;
constexpr size_t kHeader = 1024;       // of a workspace: counters
static_assert(64 + 2 * (1 + kGradGroups) * sizeof(unsigned) <= kHeader, "the counters fit");

int esize(int dtype) { return dtype == DPLR_BF16 ? 2 : 4; }
bool type_ok(int t) { return t == DPLR_F32 || t == DPLR_BF16; }

dplr_status check_desc(const dplr_nr_desc* d) {
    if (!d || !type_ok(d->in_dtype) || !type_ok(d->grad_dtype)) return DPLR_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->Hk < 0 || d->d < 1) return DPLR_ERR_INVALID_ARG;
    if (d->rot < 0 || d->rot > d->d || (d->interleaved != 0 && d->interleaved != 1)) return DPLR_ERR_INVALID_ARG;
    if (d->norm != kNone && d->norm != kRms && d->norm != kL2) return DPLR_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->q_scale) || !std::isfinite(d->rot_scale))
        return DPLR_ERR_INVALID_ARG;
    if (d->in_dtype == DPLR_F32 && d->grad_dtype == DPLR_BF16) return DPLR_ERR_UNSUPPORTED;
    if ((d->d != 32 && d->d != 64 && d->d != 128 && d->d != 256) || d->rot % 16 != 0) return DPLR_ERR_UNSUPPORTED;
    if ((long long)d->B * d->T >= (1LL << 31) || d->Hq > (1 << 16) || d->Hk > (1 << 16)) return DPLR_ERR_UNSUPPORTED;
    return DPLR_OK;
}

// Rows [B,heads,T,d]; `out`: they must not overlap either.
dplr_status rows_of(const dplr_nr_desc* d, const dplr_hd_tensor* t, int heads, int dtype, bool out, Rows* r) {
    *r = Rows{nullptr, d->d, d->d, d->d};
    if (d->T == 0 || heads == 0) return DPLR_OK;
    if (!t || !t->data || (reinterpret_cast<uintptr_t>(t->data) & 15u)) return DPLR_ERR_INVALID_ARG;
    const int es = esize(dtype);
    const long long n[3] = {d->B, heads, d->T};
    long long st[3] = {t->sb, t->sh, t->st};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) { st[i] = d->d; continue; }
        if (st[i] <= 0 || (st[i] * es) % 16 != 0) return DPLR_ERR_INVALID_ARG;
        if (st[i] >= (1LL << 40) / es) return DPLR_ERR_UNSUPPORTED;
    }
    if (out) {                             // ascending strides, each past what lies inside it
        int o[3] = {0, 1, 2};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (st[o[j]] > st[o[j + 1]]) { const int x = o[j]; o[j] = o[j + 1]; o[j + 1] = x; }
        long long span = d->d;
        for (int i = 0; i < 3; ++i) {
            if (n[o[i]] == 1) continue;
            if (st[o[i]] < span) return DPLR_ERR_INVALID_ARG;
            span += (n[o[i]] - 1) * st[o[i]];
        }
    }
    *r = Rows{t->data, st[0], st[1], st[2]};
    return DPLR_OK;
}

bool aligned(const void* p, unsigned n, bool needed) { return p ? (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0 : !needed; }

// Positions, frequencies and weights, the same in both directions.
dplr_status common(const dplr_nr_desc* d, const int32_t* positions, int64_t pos_sb, int64_t pos_st, int32_t first,
                   const uint64_t* turns, const float* wq, const float* wk, Args* a) {
    if (!aligned(positions, 4, false) || !aligned(turns, 8, d->rot > 0)) return DPLR_ERR_INVALID_ARG;
    if (positions ? (d->B > 1 && pos_sb < 0) || (d->T > 1 && pos_st < 0)
                  : first < 0 || (long long)first + d->T > (1LL << 31))
        return DPLR_ERR_INVALID_ARG;
    if (!aligned(wq, 4, false) || !aligned(wk, 4, false) || (d->norm == kNone && (wq || wk))) return DPLR_ERR_INVALID_ARG;
    a->pos = positions; a->psb = d->B > 1 ? pos_sb : 0; a->pst = d->T > 1 ? pos_st : 0; a->first = first;
    a->turns = reinterpret_cast<const unsigned long long*>(turns);
    a->wq = wq; a->wk = wk;
    a->B = d->B; a->T = d->T; a->Hq = d->Hq; a->Hk = d->Hk;
    a->rot = d->rot; a->interleaved = d->interleaved; a->norm = d->norm;
    a->eps = d->eps; a->share = d->norm == kRms ? 1.f / d->d : 1.f;
    a->q_scale = d->q_scale; a->rot_scale = d->rot_scale;
    return DPLR_OK;
}

// Single tokens of many rows are the tokens of one.
void flatten(Args* a) {
    if (a->T != 1 || !a->pos) return;      // without positions every row has the same one, not one after the other
    for (Rows* r : {&a->q, &a->k, &a->oq, &a->ok, &a->gq, &a->gk}) r->st = r->sb;
    a->pst = a->psb;
    a->T = a->B;
    a->B = 1;
}

}  // namespace
}  // namespace nr
}  // namespace dplr

using namespace dplr;
using namespace dplr::nr;

#define NR_TRY(x) do { const dplr_status st_ = (x); if (st_ != DPLR_OK) return st_; } while (0)

extern "C" {

dplr_status dplr_nr_check(const dplr_nr_desc* desc) { return check_desc(desc); }

dplr_status dplr_nr_turns(const double* radians, int32_t n, uint64_t* turns) {
    if (n < 0 || (n > 0 && (!radians || !turns))) return DPLR_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i)
        if (!std::isfinite(radians[i]) || radians[i] < 0) return DPLR_ERR_INVALID_ARG;
    // 1 / (2 pi) in two parts, so that a fraction of a turn keeps all of its 64 bits
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kRest = -0x1.6b01ec5417056p-57;
    for (int32_t i = 0; i < n; ++i) {
        // rounded here, whatever compilers for Arm make of a product and a difference
        const double t = std::fma(radians[i], kTurn, 0.0), rest = std::fma(radians[i], kTurn, -t) + radians[i] * kRest;
        // the fraction's bits below 2^-64 and the rest are rounded together
        const double units = std::ldexp(t - std::floor(t), 64), whole = std::floor(units);
        const double below = std::ldexp(rest - std::floor(rest + 0.5), 64) + (units - whole);
        turns[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint(below));
    }
    return DPLR_OK;
}

dplr_status dplr_nr_forward(const dplr_nr_desc* desc, const dplr_hd_tensor* q, const dplr_hd_tensor* k,
                            const int32_t* positions, int64_t pos_sb, int64_t pos_st, int32_t first_position,
                            const uint64_t* turns, const float* q_weight, const float* k_weight,
                            const dplr_hd_tensor* q_out, const dplr_hd_tensor* k_out, void* stream) {
    NR_TRY(check_desc(desc));
    Args a{};
    NR_TRY(common(desc, positions, pos_sb, pos_st, first_position, turns, q_weight, k_weight, &a));
    NR_TRY(rows_of(desc, q, desc->Hq, desc->in_dtype, false, &a.q));
    NR_TRY(rows_of(desc, k, desc->Hk, desc->in_dtype, false, &a.k));
    NR_TRY(rows_of(desc, q_out, desc->Hq, desc->in_dtype, true, &a.oq));
    NR_TRY(rows_of(desc, k_out, desc->Hk, desc->in_dtype, true, &a.ok));
    if (hd::taken({a.oq.p, a.ok.p}, {a.q.p, a.k.p, positions, turns, q_weight, k_weight})) return DPLR_ERR_INVALID_ARG;
    if (desc->T == 0) return DPLR_OK;
    flatten(&a);
    return launch_forward(a, desc->in_dtype == DPLR_BF16, desc->d, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DPLR_OK : DPLR_ERR_CUDA;
}

size_t dplr_nr_backward_workspace_size(const dplr_nr_desc* desc) {
    return check_desc(desc) == DPLR_OK ? kHeader + sizeof(float) * 2 * (size_t)(kGradCtas + kGradGroups) * desc->d : 0;
}

dplr_status dplr_nr_backward(const dplr_nr_desc* desc, const dplr_hd_tensor* dq_out, const dplr_hd_tensor* dk_out,
                             const dplr_hd_tensor* q, const dplr_hd_tensor* k, const int32_t* positions, int64_t pos_sb,
                             int64_t pos_st, int32_t first_position, const uint64_t* turns, const float* q_weight,
                             const float* k_weight, const dplr_hd_tensor* dq, const dplr_hd_tensor* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t ws_bytes, void* stream) {
    NR_TRY(check_desc(desc));
    Args a{};
    NR_TRY(common(desc, positions, pos_sb, pos_st, first_position, turns, q_weight, k_weight, &a));
    if (desc->norm != kNone) {
        NR_TRY(rows_of(desc, q, desc->Hq, desc->in_dtype, false, &a.q));
        NR_TRY(rows_of(desc, k, desc->Hk, desc->in_dtype, false, &a.k));
    }
    NR_TRY(rows_of(desc, dq_out, desc->Hq, desc->grad_dtype, false, &a.gq));
    NR_TRY(rows_of(desc, dk_out, desc->Hk, desc->grad_dtype, false, &a.gk));
    NR_TRY(rows_of(desc, dq, desc->Hq, desc->in_dtype, true, &a.oq));
    NR_TRY(rows_of(desc, dk, desc->Hk, desc->in_dtype, true, &a.ok));
    if (!aligned(dq_weight, 4, false) || !aligned(dk_weight, 4, false) || (dq_weight && !q_weight) || (dk_weight && !k_weight))
        return DPLR_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < dplr_nr_backward_workspace_size(desc) || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
        return DPLR_ERR_WORKSPACE;
    if (hd::taken({a.oq.p, a.ok.p, dq_weight, dk_weight},
                  {a.q.p, a.k.p, a.gq.p, a.gk.p, positions, turns, q_weight, k_weight, workspace}))
        return DPLR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (float* w : {desc->T == 0 ? dq_weight : nullptr, desc->T == 0 || desc->Hk == 0 ? dk_weight : nullptr})
        if (w && cudaMemsetAsync(w, 0, sizeof(float) * desc->d, s) != cudaSuccess) return DPLR_ERR_CUDA;
    if (desc->T == 0) return DPLR_OK;
    flatten(&a);
    a.dwq = dq_weight;
    a.dwk = desc->Hk ? dk_weight : nullptr;
    a.done = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + 64);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader);
    return launch_backward(a, desc->in_dtype == DPLR_BF16, desc->grad_dtype == DPLR_BF16, desc->d, s) == cudaSuccess
               ? DPLR_OK : DPLR_ERR_CUDA;
}

}  // extern "C"
