// One token of linear attention with one decay per head for every row of a serving batch, on a pool of states:
//   S <- e^g S + k v^T in place,  o = S^T q = e^g (S_old^T q) + (q . k) v
//
// The state is read and written once (8 dk dv bytes a row and head) and nothing else comes near that: the step is bound
// by HBM. A CTA takes NC columns of one state; a thread holds 4 columns of dk NC / 1024 rows, all loaded before the
// first use, so that a CTA has its whole block in flight. The sum over rows goes through shuffles and one exchange of
// the warps' partial sums. Measured (bf16, H 16, 128 x 128, 32 columns a CTA): 249 states 82 us, 6.4 TB/s; 8 states 6 us;
// whole calls of 256, 1024 and 4096 rows 90, 342 and 1380 us, 6.0, 6.3 and 6.2 TB/s. Each CTA looks through the slots in front
// of its row for its own, 4 bytes a row from L2: with small states and many rows (not measured) that would grow past them.
#include <cuda_bf16.h>

#include "hd_internal.h"

namespace dplr {
namespace hd {
namespace {

constexpr int TH = 256;

struct StepArgs {
    View q, k, v;
    const float* g; long long gb, gh;
    float* S; const int* slots; int nslots, H;
    void* o; long long ob, oh;
    int* status;
};

template <class IT> __device__ __forceinline__ float val(const void* p, long long i) {
    return static_cast<float>(static_cast<const IT*>(p)[i]);
}

template <class IT, int DK, int DV, int NC>
__global__ void __launch_bounds__(TH) hd_decode_kernel(const __grid_constant__ StepArgs a) {
    constexpr int CG = NC / 4, RG = TH / CG, PER = DK / RG;   // column groups, row groups, rows per thread
    constexpr int NB = DV / NC;
    static_assert(PER >= 1, "every row group has a row");
    __shared__ float sq[DK], sk[DK], sv[NC];
    __shared__ float4 red[TH / 32][CG < 32 ? CG : 32];
    __shared__ float qk_part[TH / 32];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, lane = tid & 31, warp = tid >> 5;
    const int nb = blockIdx.x % NB;
    const int h = (blockIdx.x / NB) % a.H;
    const int row = blockIdx.x / NB / a.H;
    const int c0 = nb * NC;
    const int slot = a.slots[row];
    const bool here = slot >= 0 && slot < a.nslots;
    // the state's block: rows rg, rg + RG, ..
    float4 s[PER];
    float* Sp = a.S + ((long long)(here ? slot : 0) * a.H + h) * (DK * DV) + c0 + 4 * cg;
    if (here) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = *reinterpret_cast<const float4*>(Sp + (rg + RG * i) * DV);
    }
    // a slot that an earlier row has belongs to that row
    bool taken = false;
    if (here)
        for (int j = tid; j < row; j += TH) taken |= a.slots[j] == slot;
    float qk = 0.f;
    for (int i = tid; i < DK; i += TH) {
        const float x = val<IT>(a.q.p, row * a.q.sb + (h / a.q.div) * a.q.sh + i);
        const float y = val<IT>(a.k.p, row * a.k.sb + (h / a.k.div) * a.k.sh + i);
        sq[i] = x; sk[i] = y;
        qk = x * y;
    }
    if (tid < NC) sv[tid] = val<IT>(a.v.p, row * a.v.sb + h * a.v.sh + c0 + tid);
    float g = a.g[row * a.gb + h * a.gh];
    g = g < kMinGate ? kMinGate : g;
    const float e = __expf(g);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, off);
    if (lane == 0) qk_part[warp] = qk;
    taken = __syncthreads_or(taken);
    const long long oat = row * a.ob + h * a.oh + c0;
    if (!here || taken) {
        if (tid < NC) {
            if (sizeof(IT) == 4) static_cast<float*>(a.o)[oat + tid] = 0.f;
            else static_cast<__nv_bfloat16*>(a.o)[oat + tid] = __float2bfloat16_rn(0.f);
        }
        if (tid == 0 && a.status && slot != -1) *a.status = (int)DPLR_ERR_INVALID_ARG;
        return;
    }
    const float4 v = make_float4(sv[4 * cg], sv[4 * cg + 1], sv[4 * cg + 2], sv[4 * cg + 3]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = rg + RG * i;
        const float q = sq[r], k = sk[r];
        s[i].x *= e; s[i].y *= e; s[i].z *= e; s[i].w *= e;
        acc.x = fmaf(q, s[i].x, acc.x); acc.y = fmaf(q, s[i].y, acc.y);
        acc.z = fmaf(q, s[i].z, acc.z); acc.w = fmaf(q, s[i].w, acc.w);
        s[i].x = fmaf(k, v.x, s[i].x); s[i].y = fmaf(k, v.y, s[i].y);
        s[i].z = fmaf(k, v.z, s[i].z); s[i].w = fmaf(k, v.w, s[i].w);
        *reinterpret_cast<float4*>(Sp + r * DV) = s[i];
    }
    // lanes of a warp with the same columns, then the warps
#pragma unroll
    for (int off = CG; off < 32; off <<= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
    }
    if (lane < CG) red[warp][lane] = acc;
    __syncthreads();
    if (tid < NC) {
        float o = 0.f, all = 0.f;
#pragma unroll
        for (int w = 0; w < TH / 32; ++w) {
            o += reinterpret_cast<const float*>(red[w])[tid];
            all += qk_part[w];
        }
        o = fmaf(all, sv[tid], o);
        if (sizeof(IT) == 4) static_cast<float*>(a.o)[oat + tid] = o;
        else static_cast<__nv_bfloat16*>(a.o)[oat + tid] = __float2bfloat16_rn(o);
    }
}

template <class IT, int DK, int DV>
cudaError_t launch_step(const StepArgs& a, int B, cudaStream_t s) {
    constexpr int NC = DV < 32 ? DV : 32;
    hd_decode_kernel<IT, DK, DV, NC><<<(unsigned)((long long)B * a.H * (DV / NC)), TH, 0, s>>>(a);
    return cudaGetLastError();
}

template <class IT>
cudaError_t step_by_size(const StepArgs& a, int B, int dk, int dv, cudaStream_t s) {
    switch (dk * 1000 + dv) {
        case 32032: return launch_step<IT, 32, 32>(a, B, s);
        case 32064: return launch_step<IT, 32, 64>(a, B, s);
        case 32128: return launch_step<IT, 32, 128>(a, B, s);
        case 64032: return launch_step<IT, 64, 32>(a, B, s);
        case 64064: return launch_step<IT, 64, 64>(a, B, s);
        case 64128: return launch_step<IT, 64, 128>(a, B, s);
        case 128032: return launch_step<IT, 128, 32>(a, B, s);
        case 128064: return launch_step<IT, 128, 64>(a, B, s);
        case 128128: return launch_step<IT, 128, 128>(a, B, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode(const View& q, const View& k, const View& v, const float* g, long long gb, long long gh,
                          float* S, const int* slots, int nslots, int B, int H, int dk, int dv, bool bf16, void* o,
                          long long ob, long long oh, int* status, cudaStream_t s) {
    const StepArgs a{q, k, v, g, gb, gh, S, slots, nslots, H, o, ob, oh, status};
    return bf16 ? step_by_size<__nv_bfloat16>(a, B, dk, dv, s) : step_by_size<float>(a, B, dk, dv, s);
}

}  // namespace hd
}  // namespace dplr
