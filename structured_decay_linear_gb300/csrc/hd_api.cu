// Host side of the per-head-decay operator's C ABI: checks, segment and workspace plans, and the launches of the forward,
// the backward, the ragged forward and the one-token step (hd_internal.h has the operator and its passes).
#include "hd_internal.h"

namespace dplr {
namespace hd {
namespace {

constexpr size_t kAlign = 256;
constexpr int kSMs = 152;   // a constant, so that a workspace size holds on whichever device is current
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool valid_dim(int d) { return d == 32 || d == 64 || d == 128; }

dplr_status check_desc(const dplr_hd_desc* d) {
    if (!d) return DPLR_ERR_INVALID_ARG;
    if (d->in_dtype != DPLR_F32 && d->in_dtype != DPLR_BF16) return DPLR_ERR_INVALID_ARG;
    if (d->B < 1 || d->H < 1 || d->Hq < 1 || d->T < 0 || d->dk < 1 || d->dv < 1) return DPLR_ERR_INVALID_ARG;
    if (d->H % d->Hq != 0 || (d->per_head != 0 && d->per_head != 1)) return DPLR_ERR_INVALID_ARG;
    if (!valid_dim(d->dk) || !valid_dim(d->dv)) return DPLR_ERR_UNSUPPORTED;
    const long long bh = (long long)d->B * d->H;
    if (bh >= (1LL << 24) || bh * d->T >= (1LL << 31)) return DPLR_ERR_UNSUPPORTED;
    return DPLR_OK;
}

int esize(const dplr_hd_desc* d) { return d->in_dtype == DPLR_BF16 ? 2 : 4; }

// A row sequence of `heads` heads and D features; `out`: its rows must not overlap either.
dplr_status view_of(const dplr_hd_desc* d, const dplr_hd_tensor* t, int heads, int D, bool out, View* v) {
    v->div = d->H / heads;
    if (d->T == 0) {
        v->p = nullptr; v->sb = v->sh = v->st = D;
        return DPLR_OK;
    }
    if (!t || !t->data || (reinterpret_cast<uintptr_t>(t->data) & 15u)) return DPLR_ERR_INVALID_ARG;
    const int es = esize(d);
    const long long n[3] = {d->B, heads, d->T};
    long long st[3] = {t->sb, t->sh, t->st};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) { st[i] = D; continue; }
        if (st[i] <= 0 || (st[i] * es) % 16 != 0) return DPLR_ERR_INVALID_ARG;
        if (st[i] >= (1LL << 40) / es) return DPLR_ERR_UNSUPPORTED;
    }
    if (out) {     // ascending strides, each past what lies inside it
        int o[3] = {0, 1, 2};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (st[o[j]] > st[o[j + 1]]) { const int x = o[j]; o[j] = o[j + 1]; o[j + 1] = x; }
        long long span = D;
        for (int i = 0; i < 3; ++i) {
            if (n[o[i]] == 1) continue;
            if (st[o[i]] < span) return DPLR_ERR_INVALID_ARG;
            span += (n[o[i]] - 1) * st[o[i]];
        }
    }
    v->p = t->data; v->sb = st[0]; v->sh = st[1]; v->st = st[2];
    return DPLR_OK;
}

struct Gates { const float* p; long long sb, sh, st; };

dplr_status gates_of(const dplr_hd_desc* d, const dplr_hd_tensor* t, Gates* g) {
    *g = Gates{nullptr, 0, 0, 0};
    if (d->T == 0) return DPLR_OK;
    if (!t || !t->data || (reinterpret_cast<uintptr_t>(t->data) & 3u)) return DPLR_ERR_INVALID_ARG;
    g->p = static_cast<const float*>(t->data);
    if (d->per_head) { g->sh = 1; return DPLR_OK; }
    if ((d->B > 1 && t->sb < 0) || (d->H > 1 && t->sh < 0) || (d->T > 1 && t->st < 0)) return DPLR_ERR_INVALID_ARG;
    g->sb = d->B > 1 ? t->sb : 0;
    g->sh = d->H > 1 ? t->sh : 0;
    g->st = d->T > 1 ? t->st : 0;
    return DPLR_OK;
}

bool state_ok(const void* p, bool needed) {
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) == 0 : !needed;
}

dplr_status check_workspace(size_t need, const void* ws, size_t bytes) {
    if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0) return DPLR_ERR_WORKSPACE;
    return DPLR_OK;
}

// ---- segments of a dense batch
struct Cut { int nseg, L; };

Cut cut(int T, int want, int unit, int least, int most) {
    // `want` segments of at least `least` and (if most > 0) at most `most` tokens, a multiple of `unit`
    if (T <= 0) return Cut{1, unit};
    long long L = (T + (long long)want - 1) / want;
    if (L < least) L = least;
    if (most > 0 && L > most) L = most;
    L = (L + unit - 1) / unit * unit;
    const int n = (int)((T + L - 1) / L);
    return Cut{n, (int)L};
}

// CTAs that one segment per sequence gives a pass over a state of DZ columns.
long long base_ctas(const dplr_hd_desc* d, int DZ) { return (long long)d->B * d->H * (DZ / fp32_zblock(DZ)); }

bool on_tensor_cores(const dplr_hd_desc* d) { return tc_supported(d->in_dtype == DPLR_BF16, d->dk, d->dv); }

Cut forward_cut(const dplr_hd_desc* d) {
    if (on_tensor_cores(d)) {
        const long long want = kSMs / ((long long)d->B * d->H);
        // Up to 512 tokens stay whole (B1 H16 T512: 19 us, in two segments 23 us: a scan and a pass more); longer sequences are
        // cut into segments of 256 and more (T1024: 23 us, of 512 31 us; T2048: 27 and 31 us).
        return cut(d->T, want < 1 ? 1 : (int)want, kChunk, d->T <= 512 ? 512 : 256, 0);
    }
    // Segments of 128 tokens, or of 64 where those would leave SMs without one (fp32 64 x 64, 16 heads: T777 48 -> 35 us; at
    // T2001, with 256 of 128 tokens, 64 would take 64 us instead of 58: more states to scan).
    const long long target = 2LL * kSMs, base = base_ctas(d, d->dv), want = target / base;
    return cut(d->T, want < 1 ? 1 : (int)want, 32, base * ((d->T + 127) / 128) < kSMs ? 64 : 128, 0);
}

Cut backward_cut(const dplr_hd_desc* d) {
    if (on_tensor_cores(d)) {
        const long long want = kSMs / ((long long)d->B * d->H);
        return cut(d->T, want < 1 ? 1 : (int)want, kChunk, 256, 512);
    }
    const long long target = 2LL * kSMs;
    const long long want = target / base_ctas(d, d->dv);
    return cut(d->T, want < 1 ? 1 : (int)want, 32, 128, 512);
}

size_t state_bytes(const dplr_hd_desc* d) { return sizeof(float) * (size_t)d->dk * d->dv; }

struct ForwardPlan { Cut c; size_t bound, gsum, total; };

ForwardPlan forward_plan(const dplr_hd_desc* d) {
    ForwardPlan p{};
    p.c = forward_cut(d);
    size_t off = kAlign;
    const size_t n = (size_t)d->B * d->H * (p.c.nseg + 1);
    p.bound = off;
    if (p.c.nseg > 1) off = up(off + n * state_bytes(d));
    p.gsum = off;
    if (p.c.nseg > 1) off = up(off + n * sizeof(float));
    p.total = off;
    return p;
}

struct BackwardPlan { Cut c; int nzq; size_t fwd, bwd, gsum, dotq, dotk, seg, part_q, part_k, total; };

BackwardPlan backward_plan(const dplr_hd_desc* d) {
    BackwardPlan p{};
    p.c = backward_cut(d);
    p.nzq = on_tensor_cores(d) ? 1 : d->dk / fp32_zblock(d->dk);
    const size_t bh = (size_t)d->B * d->H, tok = bh * d->T;
    size_t off = kAlign;
    auto take = [&](size_t bytes) { const size_t at = off; off = up(off + bytes); return at; };
    const size_t n = bh * (p.c.nseg + 1);
    p.fwd = take(p.c.nseg > 1 ? n * state_bytes(d) : bh * state_bytes(d));     // one segment: S_T alone
    p.bwd = take(p.c.nseg > 1 ? n * state_bytes(d) : 0);
    p.gsum = take(p.c.nseg > 1 ? n * sizeof(float) : 0);
    p.dotq = take(p.nzq * tok * sizeof(float));
    p.dotk = take(p.nzq * tok * sizeof(float));
    p.seg = take(bh * p.c.nseg * sizeof(double));
    const size_t part = d->H != d->Hq ? tok * d->dk * sizeof(float) : 0;
    p.part_q = take(part);
    p.part_k = take(part);
    p.total = off;
    return p;
}

Geometry dense(const dplr_hd_desc* d, const Cut& c) {
    Geometry g{};
    g.H = d->H; g.T = d->T; g.nseg = c.nseg; g.L = c.L;
    return g;
}

Pass base_pass(const Gates& g, int DX, int DZ, bool ext_turned, bool bound_turned) {
    Pass p{};
    p.g = g.p; p.gb = g.sb; p.gh = g.sh; p.gt = g.st;
    p.DX = DX; p.DZ = DZ;
    p.ext_turned = ext_turned;
    p.bound_turned = bound_turned;
    return p;
}

void output(Pass& p, const View& o) { p.o = const_cast<void*>(o.p); p.ob = o.sb; p.oh = o.sh; p.ot = o.st; }

cudaError_t launch(const Launch& a, bool tensor_cores, cudaStream_t s) {
    return tensor_cores ? launch_tc(a, s) : launch_fp32(a, s);
}

cudaError_t copy_state(float* dst, const float* src, size_t bytes, cudaStream_t s) {
    if (!dst || dst == src) return cudaSuccess;
    return src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, bytes, s);
}

}  // namespace
}  // namespace hd
}  // namespace dplr

using namespace dplr;
using namespace dplr::hd;

#define HD_TRY(x) do { const dplr_status st_ = (x); if (st_ != DPLR_OK) return st_; } while (0)
#define HD_CUDA(x) do { if ((x) != cudaSuccess) return DPLR_ERR_CUDA; } while (0)

extern "C" {

dplr_status dplr_hd_check(const dplr_hd_desc* desc) { return check_desc(desc); }

const char* dplr_hd_path(const dplr_hd_desc* desc) {
    if (check_desc(desc) != DPLR_OK) return "";
    return on_tensor_cores(desc) ? "hd_tcgen05" : "hd_fp32";
}

size_t dplr_hd_workspace_size(const dplr_hd_desc* desc) {
    return check_desc(desc) == DPLR_OK ? forward_plan(desc).total : 0;
}

dplr_status dplr_hd_forward(const dplr_hd_desc* desc, const dplr_hd_tensor* q, const dplr_hd_tensor* k,
                            const dplr_hd_tensor* v, const dplr_hd_tensor* decay, const float* S0,
                            const dplr_hd_tensor* o, float* S_T, void* workspace, size_t ws_bytes, void* stream) {
    HD_TRY(check_desc(desc));
    View vq, vk, vv, vo;
    Gates g;
    HD_TRY(view_of(desc, q, desc->Hq, desc->dk, false, &vq));
    HD_TRY(view_of(desc, k, desc->Hq, desc->dk, false, &vk));
    HD_TRY(view_of(desc, v, desc->H, desc->dv, false, &vv));
    HD_TRY(view_of(desc, o, desc->H, desc->dv, true, &vo));
    HD_TRY(gates_of(desc, decay, &g));
    if (!state_ok(S0, false) || !state_ok(S_T, false)) return DPLR_ERR_INVALID_ARG;
    const ForwardPlan pl = forward_plan(desc);
    HD_TRY(check_workspace(pl.total, workspace, ws_bytes));
    if (taken({vo.p, S_T}, {vq.p, vk.p, vv.p, g.p, S_T == S0 ? nullptr : S0, workspace}) || (vo.p && vo.p == S0))
        return DPLR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) {
        HD_CUDA(copy_state(S_T, S0, (size_t)desc->B * desc->H * state_bytes(desc), s));
        return DPLR_OK;
    }
    char* ws = static_cast<char*>(workspace);
    Launch a{};
    a.geo = dense(desc, pl.c);
    a.B = desc->B; a.bf16 = desc->in_dtype == DPLR_BF16; a.npass = 1;
    a.status = static_cast<int*>(workspace);
    a.wait_cycles = wait_limit();
    Pass& p = a.pass[0];
    p = base_pass(g, desc->dk, desc->dv, false, false);
    p.x = vq; p.y = vk; p.z = vv;
    if (pl.c.nseg > 1) {
        p.bound = reinterpret_cast<float*>(ws + pl.bound);
        p.gsum = reinterpret_cast<float*>(ws + pl.gsum);
        p.states_only = 1;
        HD_CUDA(launch(a, on_tensor_cores(desc), s));
        Scan sc{};
        sc.geo = a.geo; sc.B = desc->B; sc.dk = desc->dk; sc.dv = desc->dv;
        sc.fwd = p.bound; sc.fwd_ext = S0; sc.gsum = p.gsum;
        HD_CUDA(launch_scan(sc, s));
        p.states_only = 0;
        a.follows = 1;
    }
    p.ext_in = S0; p.ext_out = S_T;
    output(p, vo);
    HD_CUDA(launch(a, on_tensor_cores(desc), s));
    return DPLR_OK;
}

size_t dplr_hd_backward_workspace_size(const dplr_hd_desc* desc) {
    return check_desc(desc) == DPLR_OK ? backward_plan(desc).total : 0;
}

dplr_status dplr_hd_backward(const dplr_hd_desc* desc, const dplr_hd_tensor* q, const dplr_hd_tensor* k,
                             const dplr_hd_tensor* v, const dplr_hd_tensor* decay, const float* S0,
                             const dplr_hd_tensor* dO, const float* dST, const dplr_hd_tensor* dq,
                             const dplr_hd_tensor* dk, const dplr_hd_tensor* dv, float* ddecay, float* dS0,
                             void* workspace, size_t ws_bytes, void* stream) {
    HD_TRY(check_desc(desc));
    View vq, vk, vv, vdo, vdq, vdk, vdv;
    Gates g;
    HD_TRY(view_of(desc, q, desc->Hq, desc->dk, false, &vq));
    HD_TRY(view_of(desc, k, desc->Hq, desc->dk, false, &vk));
    HD_TRY(view_of(desc, v, desc->H, desc->dv, false, &vv));
    HD_TRY(view_of(desc, dO, desc->H, desc->dv, false, &vdo));
    HD_TRY(view_of(desc, dq, desc->Hq, desc->dk, true, &vdq));
    HD_TRY(view_of(desc, dk, desc->Hq, desc->dk, true, &vdk));
    HD_TRY(view_of(desc, dv, desc->H, desc->dv, true, &vdv));
    HD_TRY(gates_of(desc, decay, &g));
    if (!state_ok(S0, false) || !state_ok(dST, false) || !state_ok(dS0, false)) return DPLR_ERR_INVALID_ARG;
    if (ddecay && (reinterpret_cast<uintptr_t>(ddecay) & 3u)) return DPLR_ERR_INVALID_ARG;
    const BackwardPlan pl = backward_plan(desc);
    HD_TRY(check_workspace(pl.total, workspace, ws_bytes));
    if (taken({vdq.p, vdk.p, vdv.p, ddecay, dS0}, {vq.p, vk.p, vv.p, g.p, S0, vdo.p, dST, workspace}))
        return DPLR_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long bh = (long long)desc->B * desc->H;
    if (desc->T == 0) {
        HD_CUDA(copy_state(dS0, dST, (size_t)bh * state_bytes(desc), s));
        if (ddecay && desc->per_head) HD_CUDA(cudaMemsetAsync(ddecay, 0, sizeof(float) * desc->H, s));
        return DPLR_OK;
    }
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    const bool many = pl.c.nseg > 1;
    Launch a{};
    a.geo = dense(desc, pl.c);
    a.B = desc->B; a.bf16 = desc->in_dtype == DPLR_BF16;
    a.status = static_cast<int*>(workspace);
    a.wait_cycles = wait_limit();
    const int K = desc->dk, V = desc->dv;
    if (many) {
        a.npass = 2;
        // boundary states as S^T and dS^T [dv][dk], the way dq and dk start from them (dv turns them)
        Pass& f = a.pass[0];
        f = base_pass(g, V, K, false, false);
        f.y = vv; f.z = vk; f.bound = at(pl.fwd); f.gsum = at(pl.gsum);
        f.states_only = 2;          // the last segment's too: its gates, and S_T
        Pass& b = a.pass[1];
        b = base_pass(g, V, K, false, false);
        b.y = vdo; b.z = vq; b.reverse = 1; b.bound = at(pl.bwd);
        b.states_only = 1;
        HD_CUDA(launch(a, on_tensor_cores(desc), s));
        Scan sc{};
        sc.geo = a.geo; sc.B = desc->B; sc.dk = K; sc.dv = V;
        sc.fwd = at(pl.fwd); sc.fwd_ext = S0; sc.upto_end = 1;
        sc.bwd = at(pl.bwd); sc.bwd_ext = dST; sc.gsum = at(pl.gsum); sc.turned = 1;
        HD_CUDA(launch_scan(sc, s));
        a.follows = 1;
    }
    const bool shared = desc->H != desc->Hq;
    auto partial = [&](Pass& p, size_t off) {      // shared heads: fp32 [B,H,T,dk], summed afterwards
        p.o = at(off); p.o_f32 = 1;
        p.ob = (long long)desc->H * desc->T * K; p.oh = (long long)desc->T * K; p.ot = K;
    };
    a.npass = 3;
    Pass& pq = a.pass[0];
    pq = base_pass(g, V, K, true, false);
    pq.x = vdo; pq.y = vv; pq.z = vk;
    pq.ext_in = S0; pq.bound = many ? at(pl.fwd) : nullptr;
    if (!many && ddecay && dST) pq.ext_out = at(pl.fwd);
    Pass& pk = a.pass[1];
    pk = base_pass(g, V, K, true, false);
    pk.x = vv; pk.y = vdo; pk.z = vq; pk.reverse = 1;
    pk.ext_in = dST; pk.bound = many ? at(pl.bwd) : nullptr;
    Pass& pv = a.pass[2];
    pv = base_pass(g, K, V, false, true);
    pv.x = vk; pv.y = vq; pv.z = vdo; pv.reverse = 1;
    pv.ext_in = dST; pv.bound = pk.bound; pv.ext_out = dS0;
    output(pq, vdq);
    output(pk, vdk);
    output(pv, vdv);
    if (shared) {
        partial(pq, pl.part_q);
        partial(pk, pl.part_k);
    }
    if (ddecay) {
        pq.w = vq; pq.dots = at(pl.dotq);
        pk.w = vk; pk.dots = at(pl.dotk);
    }
    HD_CUDA(launch(a, on_tensor_cores(desc), s));
    if (ddecay) {
        GateGrad gg{};
        gg.B = desc->B; gg.H = desc->H; gg.T = desc->T; gg.nseg = pl.c.nseg; gg.L = pl.c.L; gg.dk = K; gg.dv = V;
        gg.dq_dots = pq.dots; gg.nq = pl.nzq; gg.dk_dots = pk.dots; gg.nk = pl.nzq;
        if (many) { gg.fwd = at(pl.fwd); gg.bwd = at(pl.bwd); }
        gg.last_end = dST != nullptr;
        gg.S_T = at(pl.fwd); gg.dST = dST;
        if (desc->per_head) { gg.seg_sum = reinterpret_cast<double*>(ws + pl.seg); gg.dg_head = ddecay; }
        else gg.dg_token = ddecay;
        HD_CUDA(launch_gate_grad(gg, s));
    }
    if (shared) {
        GroupSum gs{};
        gs.B = desc->B; gs.H = desc->H; gs.Hq = desc->Hq; gs.T = desc->T; gs.D = K; gs.bf16 = a.bf16;
        gs.one[0] = {at(pl.part_q), const_cast<void*>(vdq.p), vdq.sb, vdq.sh, vdq.st};
        gs.one[1] = {at(pl.part_k), const_cast<void*>(vdk.p), vdk.sb, vdk.sh, vdk.st};
        HD_CUDA(launch_group_sum(gs, s));
    }
    return DPLR_OK;
}

// Whether a ragged batch's blocks are put in order of their lengths: not where every CTA has one at most, and not where each
// has so many that the last one's length does not matter and one CTA would take long to sort them.
static bool ordered(const dplr_hd_desc* desc, long long max_blocks) {
    return on_tensor_cores(desc) && max_blocks * desc->H > kSMs && max_blocks <= 16384;
}

size_t dplr_hd_packed_workspace_size(const dplr_hd_desc* desc, int32_t R, int32_t block) {
    if (check_desc(desc) != DPLR_OK || desc->B != 1 || R < 1 || block < 32 || block % 32 != 0) return 0;
    const long long most = (long long)desc->T / block + R;
    size_t off = kAlign;
    if (desc->T > block) {
        const size_t n = (size_t)most * desc->H;
        off = up(off + n * state_bytes(desc));
        off = up(off + n * sizeof(float));
    }
    if (ordered(desc, most)) off = up(off + (size_t)most * sizeof(int));
    return off;
}

dplr_status dplr_hd_forward_packed(const dplr_hd_desc* desc, int32_t R, int32_t block, int32_t n_slots,
                                   const int32_t* blocks, const int32_t* block_starts, const int32_t* slots,
                                   const int32_t* context, const dplr_hd_tensor* q, const dplr_hd_tensor* k,
                                   const dplr_hd_tensor* v, const dplr_hd_tensor* decay, float* S,
                                   const dplr_hd_tensor* o, void* workspace, size_t ws_bytes, void* stream) {
    HD_TRY(check_desc(desc));
    if (desc->B != 1 || R < 1 || n_slots < 1 || block < 32 || block % 32 != 0) return DPLR_ERR_INVALID_ARG;
    auto al = [](const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (!al(blocks, 16) || !al(block_starts, 4) || !al(slots, 4) || !al(context, 4) || !state_ok(S, true))
        return DPLR_ERR_INVALID_ARG;
    View vq, vk, vv, vo;
    Gates g;
    HD_TRY(view_of(desc, q, desc->Hq, desc->dk, false, &vq));
    HD_TRY(view_of(desc, k, desc->Hq, desc->dk, false, &vk));
    HD_TRY(view_of(desc, v, desc->H, desc->dv, false, &vv));
    HD_TRY(view_of(desc, o, desc->H, desc->dv, true, &vo));
    HD_TRY(gates_of(desc, decay, &g));
    HD_TRY(check_workspace(dplr_hd_packed_workspace_size(desc, R, block), workspace, ws_bytes));
    if (taken({vo.p, S}, {vq.p, vk.p, vv.p, g.p, blocks, block_starts, slots, context, workspace})) return DPLR_ERR_INVALID_ARG;
    if (desc->T == 0) return DPLR_OK;
    const long long max_blocks = (long long)desc->T / block + R;
    if (max_blocks * desc->H >= (1LL << 24) || (long long)R * desc->H >= (1LL << 24)) return DPLR_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    Launch a{};
    a.geo.H = desc->H; a.geo.T = desc->T;
    a.geo.blocks = blocks; a.geo.block_starts = block_starts; a.geo.slots = slots; a.geo.context = context;
    a.geo.n_slots = n_slots; a.geo.R = R;
    a.B = 1; a.bf16 = desc->in_dtype == DPLR_BF16; a.max_blocks = (int)max_blocks; a.npass = 1;
    a.status = static_cast<int*>(workspace);
    a.wait_cycles = wait_limit();
    int* order = nullptr;
    if (ordered(desc, max_blocks)) {
        order = reinterpret_cast<int*>(ws + dplr_hd_packed_workspace_size(desc, R, block) - up((size_t)max_blocks * sizeof(int)));
        HD_CUDA(launch_order(a.geo, (int)max_blocks, order, a.status + 16, s));
        a.follows = 1;
    } else if (on_tensor_cores(desc)) {
        HD_CUDA(cudaMemsetAsync(a.status + 16, 0, sizeof(int), s));     // the unit counter
    }
    Pass& p = a.pass[0];
    p = base_pass(g, desc->dk, desc->dv, false, false);
    p.x = vq; p.y = vk; p.z = vv;
    if (desc->T > block) {
        const size_t n = (size_t)max_blocks * desc->H;
        p.bound = reinterpret_cast<float*>(ws + kAlign);
        p.gsum = reinterpret_cast<float*>(ws + up(kAlign + n * state_bytes(desc)));
        p.states_only = 1;
        HD_CUDA(launch(a, on_tensor_cores(desc), s));
        Scan sc{};
        sc.geo = a.geo; sc.B = 1; sc.R = R; sc.dk = desc->dk; sc.dv = desc->dv;
        sc.fwd = p.bound; sc.fwd_ext = S; sc.gsum = p.gsum;
        HD_CUDA(launch_scan(sc, s));
        p.states_only = 0;
        a.follows = 1;
    }
    a.order = order;
    p.ext_in = S; p.ext_out = S;
    output(p, vo);
    HD_CUDA(launch(a, on_tensor_cores(desc), s));
    return DPLR_OK;
}

dplr_status dplr_hd_decode_step(const dplr_hd_desc* desc, int32_t n_slots, const int32_t* slots,
                                const dplr_hd_tensor* q, const dplr_hd_tensor* k, const dplr_hd_tensor* v,
                                const dplr_hd_tensor* decay, float* S, const dplr_hd_tensor* o, int32_t* status,
                                void* stream) {
    HD_TRY(check_desc(desc));
    if (desc->T != 1 || n_slots < 1) return DPLR_ERR_INVALID_ARG;
    View vq, vk, vv, vo;
    Gates g;
    HD_TRY(view_of(desc, q, desc->Hq, desc->dk, false, &vq));
    HD_TRY(view_of(desc, k, desc->Hq, desc->dk, false, &vk));
    HD_TRY(view_of(desc, v, desc->H, desc->dv, false, &vv));
    HD_TRY(view_of(desc, o, desc->H, desc->dv, true, &vo));
    HD_TRY(gates_of(desc, decay, &g));
    if (!slots || (reinterpret_cast<uintptr_t>(slots) & 3u) || !state_ok(S, true)) return DPLR_ERR_INVALID_ARG;
    if (status && (reinterpret_cast<uintptr_t>(status) & 3u)) return DPLR_ERR_INVALID_ARG;
    if (taken({vo.p, S, status}, {vq.p, vk.p, vv.p, g.p, slots})) return DPLR_ERR_INVALID_ARG;
    HD_CUDA(launch_decode(vq, vk, vv, g.p, g.sb, g.sh, S, slots, n_slots, desc->B, desc->H, desc->dk, desc->dv,
                          desc->in_dtype == DPLR_BF16, const_cast<void*>(vo.p), vo.sb, vo.sh, status,
                          static_cast<cudaStream_t>(stream)));
    return DPLR_OK;
}

}  // extern "C"
