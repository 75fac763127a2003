// Attention, plain: one CTA per (query row, query head), its warps stride over
// the keys with a running maximum and sum each, and are joined at the end.
#include "lora_internal.cuh"
#include "lora_kv.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4;

template <class H>
__device__ __forceinline__ float to_f(H x) { return (float)x; }

template <int DIM, class H>
struct DenseKv {
    const H *kp, *vp;
    long long kts, vts;
    __device__ __forceinline__ bool at(int j, float (&k)[DIM / 32], float (&v)[DIM / 32]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < DIM / 32; ++i) {
            k[i] = (float)kp[j * kts + lane * (DIM / 32) + i];
            v[i] = (float)vp[j * vts + lane * (DIM / 32) + i];
        }
        return true;
    }
};

template <int DIM, class H, class Kv>
__device__ __forceinline__ void attend_row(const Kv &kv, int n, const H *q, H *o, float *lse, float scale) {
    constexpr int E = DIM / 32;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][DIM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float qv[E], acc[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) qv[i] = to_f(q[lane * E + i]) * scale;
    for (int j = warp; j < n; j += kWarps) {
        float k[E], v[E], s = 0.f;
        if (!kv.at(j, k, v)) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(qv[i], k[i], s);
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn, f = __expf(m - ref), p = __expf(s - ref);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + (p > 0.f || p != p ? p * v[i] : 0.f);
        m = mn;
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][lane * E + i] = acc[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
    const float ref = mm == -INFINITY ? 0.f : mm;   // scores may all be NaN
    for (int w = 0; w < kWarps; ++w) ll += sm_l[w] * __expf(sm_m[w] - ref);
    for (int d = threadIdx.x; d < DIM; d += kWarps * 32) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += sm_o[w][d] * __expf(sm_m[w] - ref);
        o[d] = (H)(ll == 0.f ? 0.f : s / ll);
    }
    if (lse && threadIdx.x == 0) *lse = ref + logf(ll);
}

template <int DIM, class H>
__global__ void __launch_bounds__(kWarps * 32) attend_prompt_kernel(PromptArgs a) {
    const int t = blockIdx.x, hq = blockIdx.y, h = hq / (a.hq / a.hkv);
    for (int r = 0; r < a.R; ++r) {
        const int q0 = a.cu_q[r], q1 = a.cu_q[r + 1], k0 = a.cu_k[r], k1 = a.cu_k[r + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) {
            if (a.err && threadIdx.x == 0 && t == 0 && hq == 0) atomicOr(a.err, LORA_DEV_ERR_BAD_LENGTH);
            continue;
        }
        if (t < q0 || t >= q1) continue;
        __syncthreads();
        const DenseKv<DIM, H> kv{reinterpret_cast<const H *>(a.k.p) + k0 * a.k.ts + h * a.k.hs,
                                 reinterpret_cast<const H *>(a.v.p) + k0 * a.v.ts + h * a.v.hs, a.k.ts, a.v.ts};
        attend_row<DIM, H>(kv, (k1 - k0) - (q1 - q0) + (t - q0) + 1,
                           reinterpret_cast<const H *>(a.q.p) + t * a.q.ts + hq * a.q.hs,
                           reinterpret_cast<H *>(a.o.p) + t * a.o.ts + hq * a.o.hs,
                           a.lse ? a.lse + (size_t)t * a.hq + hq : nullptr, a.scale);
    }
}

}  // namespace

int launch_prompt(const PromptArgs &a, cudaStream_t st) {
    const dim3 grid(a.Tq, a.hq);
    if (a.dim == 64 && a.dtype == LORA_BF16) attend_prompt_kernel<64, __nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.dim == 64) attend_prompt_kernel<64, __half><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.dtype == LORA_BF16) attend_prompt_kernel<128, __nv_bfloat16><<<grid, kWarps * 32, 0, st>>>(a);
    else attend_prompt_kernel<128, __half><<<grid, kWarps * 32, 0, st>>>(a);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace lora
