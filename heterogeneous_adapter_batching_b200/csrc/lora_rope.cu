// Rotary positions, and the 4-bit KV cache's write and read-back.
//
// Rotation of a pair by angle = pos * freq: (a, b) -> m (a cos - b sin, b cos +
// a sin).  The angle, its sine and cosine are formed in 64 bits: at position
// 10^6 a 32-bit product is off by hundredths of a radian.  A token's angles are
// the same for all its heads, so a CTA forms them once per token in shared
// memory.  Keys that go into the cache are also rotated in 64 bits, so that the
// value that is rounded to the row type, and then to a 4-bit code, does not
// depend on the order of operations: a 32-bit error would move one code in a
// million across a border.  Queries, and keys that are not cached, use 32 bits
// (rounded once at the end).
//
// Quantisation of 64 dimensions x of one head: low = fp16(min x), step =
// fp16((max x - min x) / 15), code = clamp(round_even((x - low) / step), 0, 15).
// The quotient is formed in 32 bits; where it lies within 2^-10 of a border
// between two codes (its error is below 15.5 * 2^-21) the side is decided by the
// sign of (x - low) - step * (border) in 64 bits, which is exact.
//
// Layout of the work: a head is dim / 16 chunks of 16 elements, one thread per
// chunk: elements [8 c, 8 c + 8) and [rot / 2 + 8 c, + 8) in the half layout,
// [16 c, 16 c + 16) interleaved or past rot.  So a thread owns both elements of
// its pairs (an output may be its input), every access is 16 bytes or wider, and
// the dim / 16 neighbouring lanes that share a head reduce min and max by
// shuffles.  The kernel moves each row once and is bound by memory.
#include "lora_internal.cuh"
#include "lora_kv.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;       // most tokens of one CTA

template <class T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <class H, class H2>
struct Elem16 {
    static __device__ __forceinline__ void load8(const H *p, float (&x)[8]) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const H *h = reinterpret_cast<const H *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)h[i];
    }
    static __device__ __forceinline__ void store8(H *p, const float (&x)[8]) {
        uint4 u;
        H *h = reinterpret_cast<H *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (H)x[i];
        *reinterpret_cast<uint4 *>(p) = u;
    }
};
template <> struct Elem<__nv_bfloat16> : Elem16<__nv_bfloat16, __nv_bfloat162> {};
template <> struct Elem<__half> : Elem16<__half, __half2> {};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Code of x for (step, low), inv = 1 / step (see the head of the file).
__device__ __forceinline__ uint32_t code_of(float x, float low, float step, float inv) {
    const float t = (x - low) * inv;
    const float k = floorf(t);
    float n = rintf(t);
    if (fabsf(t - k - 0.5f) < 0x1p-10f) {
        const double side = fma(-(double)step, (double)k + 0.5, (double)x - (double)low);
        n = k + (side > 0.0 || (side == 0.0 && ((int)k & 1)) ? 1.f : 0.f);
    }
    return (uint32_t)fminf(fmaxf(n, 0.f), 15.f);   // a NaN becomes 0
}

__device__ __forceinline__ uint32_t pack8(const float (&x)[8], float low, float step, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= code_of(x[i], low, step, inv) << (4 * i);
    return w;
}

// Address of token `off` of head h in a block: the K half (which = 0) or V half of its granule.
__device__ __forceinline__ unsigned char *half_of(const KvCache &c, int dim, int page, int off, int h, int which) {
    return c.pages + page * c.page_bytes +
           (long long)(h * c.granules + off / LORA_KV_GRANULE) * kv_granule_bytes(dim) + which * kv_half_bytes(dim);
}

// Rotate 8 pairs in precision F; cs holds (cosine, sine) of each.
template <class F, class F2>
__device__ __forceinline__ void turn_pair(float &u, float &v, F2 cs) {
    const F p = u, q = v;
    u = (float)(p * cs.x - q * cs.y);
    v = (float)(q * cs.x + p * cs.y);
}
template <class F, class F2>
__device__ __forceinline__ void turn_half(float (&x)[8], float (&y)[8], const F2 *cs) {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair<F>(x[j], y[j], cs[j]);
}
template <class F, class F2>
__device__ __forceinline__ void turn_interleaved(float (&x)[8], float (&y)[8], const F2 *cs) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        turn_pair<F>(x[2 * j], x[2 * j + 1], cs[j]);
        turn_pair<F>(y[2 * j], y[2 * j + 1], cs[4 + j]);
    }
}

template <class S, class D, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int tok_per_cta) {
    // sine and cosine of the CTA's tokens, [token][pair], both precisions
    extern __shared__ double2 cs64[];
    float2 *cs32 = reinterpret_cast<float2 *>(cs64 + (CACHE ? tok_per_cta * (a.rot / 2) : 0));
    const int half = a.rot / 2, t0 = blockIdx.x * tok_per_cta, nt = min(tok_per_cta, a.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int pos = a.positions[t0 + i / half];
        double s, c;
        sincos((double)pos * (double)a.freq[i % half], &s, &c);
        s *= a.mscale;
        c *= a.mscale;
        if (CACHE) cs64[i] = make_double2(c, s);
        cs32[i] = make_float2((float)c, (float)s);
    }
    __syncthreads();

    const int chunks = a.dim / 16, per_tok = (a.hq + a.hk + a.hv) * chunks;
    for (int i = threadIdx.x; i < nt * per_tok; i += kThreads) {
        const int tl = i / per_tok, t = t0 + tl, w = i - tl * per_tok;
        const int head = w / chunks, c = w - head * chunks;
        if (a.positions[t] < 0) continue;
        const int kind = head < a.hq ? 0 : head < a.hq + a.hk ? 1 : 2;
        const int h = kind == 0 ? head : kind == 1 ? head - a.hq : head - a.hq - a.hk;
        const Rows &src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const bool turned = kind < 2 && 16 * c < a.rot;
        const bool split = turned && !a.interleaved;
        const int d0 = split ? 8 * c : 16 * c, d1 = split ? half + 8 * c : 16 * c + 8;
        const S *in = reinterpret_cast<const S *>(src.p) + t * src.ts + h * src.hs;
        float x[8], y[8];
        Elem<S>::load8(in + d0, x);
        Elem<S>::load8(in + d1, y);
        if (turned) {
            if (CACHE && kind == 1)
                a.interleaved ? turn_interleaved<double>(x, y, cs64 + tl * half + 8 * c)
                              : turn_half<double>(x, y, cs64 + tl * half + 8 * c);
            else
                a.interleaved ? turn_interleaved<float>(x, y, cs32 + tl * half + 8 * c)
                              : turn_half<float>(x, y, cs32 + tl * half + 8 * c);
        }
        if (kind == 0 || (kind == 1 ? a.has_ko : a.has_vo)) {
            const Rows &dst = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
            D *out = reinterpret_cast<D *>(dst.p) + t * dst.ts + h * dst.hs;
            Elem<D>::store8(out + d0, x);
            Elem<D>::store8(out + d1, y);
        }
        if (!CACHE || kind == 0) continue;
        const int slot = a.slots[t];
        if (slot < 0) continue;
        const int page = slot / a.c.block, off = slot - page * a.c.block;
        if (page >= a.c.num_pages) {
            if (c == 0 && h == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_PAGE);
            continue;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // what the row type holds is what is cached
            x[j] = (float)(D)x[j];
            y[j] = (float)(D)y[j];
        }
        float lo[2] = {x[0], y[0]}, hi[2] = {x[0], y[0]};
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            lo[0] = min_nan(lo[0], x[j]);
            hi[0] = max_nan(hi[0], x[j]);
            lo[1] = min_nan(lo[1], y[j]);
            hi[1] = max_nan(hi[1], y[j]);
        }
        // the lanes of this head: chunks is 4 or 8 and heads start at multiples of it
        const int lane = threadIdx.x & 31;
        const uint32_t mask = (chunks == 8 ? 0xffu : 0xfu) << (lane & ~(chunks - 1));
        const int g0 = d0 / LORA_KV_GROUP, g1 = d1 / LORA_KV_GROUP;
        float step0 = 0.f, low0 = 0.f, step1 = 0.f, low1 = 0.f;
        unsigned char *base = half_of(a.c, a.dim, page, off, h, kind - 1);
        for (int g = 0; g < a.dim / LORA_KV_GROUP; ++g) {
            float l = INFINITY, u = -INFINITY;
            if (g0 == g) {
                l = lo[0];
                u = hi[0];
            }
            if (g1 == g) {
                l = min_nan(l, lo[1]);
                u = max_nan(u, hi[1]);
            }
            for (int d = 1; d < chunks; d <<= 1) {
                l = min_nan(l, __shfl_xor_sync(mask, l, d));
                u = max_nan(u, __shfl_xor_sync(mask, u, d));
            }
            const __half hl = __float2half_rn(l), hs = __float2half_rn((float)(((double)u - (double)l) / 15.0));
            if (c == 0)
                reinterpret_cast<__half2 *>(base + kv_code_bytes(a.dim))[(off % LORA_KV_GRANULE) * (a.dim / LORA_KV_GROUP) + g] =
                    __halves2half2(hs, hl);
            if (g0 == g) {
                step0 = __half2float(hs);
                low0 = __half2float(hl);
            }
            if (g1 == g) {
                step1 = __half2float(hs);
                low1 = __half2float(hl);
            }
        }
        unsigned char *row = base + (off % LORA_KV_GRANULE) * (a.dim / 2);
        const uint32_t w0 = pack8(x, low0, step0, step0 > 0.f ? 1.f / step0 : 0.f);
        const uint32_t w1 = pack8(y, low1, step1, step1 > 0.f ? 1.f / step1 : 0.f);
        *reinterpret_cast<uint32_t *>(row + d0 / 2) = w0;
        *reinterpret_cast<uint32_t *>(row + d1 / 2) = w1;
    }
}

template <class D>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(GatherKvArgs a) {
    const int chunks = a.dim / 16, per_tok = 2 * a.c.heads * chunks;
    const long long n = (long long)a.T * per_tok;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
        const int t = (int)(i / per_tok), w = (int)(i - (long long)t * per_tok);
        const int which = w / (a.c.heads * chunks), h = w / chunks - which * a.c.heads, c = w % chunks;
        if (!(which ? a.has_v : a.has_k)) continue;
        const int slot = a.slots[t];
        if (slot < 0) continue;
        const int page = slot / a.c.block, off = slot - page * a.c.block;
        if (page >= a.c.num_pages) {
            if (c == 0 && h == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_PAGE);
            continue;
        }
        const unsigned char *base = half_of(a.c, a.dim, page, off, h, which);
        const uint2 codes = *reinterpret_cast<const uint2 *>(base + (off % LORA_KV_GRANULE) * (a.dim / 2) + 8 * c);
        const float2 p = __half22float2(reinterpret_cast<const __half2 *>(
            base + kv_code_bytes(a.dim))[(off % LORA_KV_GRANULE) * (a.dim / LORA_KV_GROUP) + 16 * c / LORA_KV_GROUP]);
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = fmaf((float)((codes.x >> (4 * j)) & 15u), p.x, p.y);
            y[j] = fmaf((float)((codes.y >> (4 * j)) & 15u), p.x, p.y);
        }
        const Rows &dst = which ? a.vo : a.ko;
        D *out = reinterpret_cast<D *>(dst.p) + t * dst.ts + h * dst.hs + 16 * c;
        Elem<D>::store8(out, x);
        Elem<D>::store8(out + 8, y);
    }
}

template <class S, class D>
int rope_types(const RopeArgs &a, cudaStream_t st) {
    // few tokens: a CTA each, for latency; many: four share a CTA's angles
    const int per = a.T >= 2368 ? kMaxTok : 1;
    const int grid = (a.T + per - 1) / per;
    const size_t pairs = (size_t)per * (a.rot / 2);
    if (a.slots)
        rope_kernel<S, D, true><<<grid, kThreads, pairs * (sizeof(double2) + sizeof(float2)), st>>>(a, per);
    else
        rope_kernel<S, D, false><<<grid, kThreads, pairs * sizeof(float2), st>>>(a, per);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace

int launch_rope(const RopeArgs &a, int src, int dst, cudaStream_t st) {
    if (dst == LORA_BF16)
        return src == LORA_FP32 ? rope_types<float, __nv_bfloat16>(a, st) : rope_types<__nv_bfloat16, __nv_bfloat16>(a, st);
    return src == LORA_FP32 ? rope_types<float, __half>(a, st) : rope_types<__half, __half>(a, st);
}

int launch_kv_gather(const GatherKvArgs &a, int dst, cudaStream_t st) {
    const long long n = (long long)a.T * 2 * a.c.heads * (a.dim / 16);
    const int grid = (int)min((n + kThreads - 1) / kThreads, 148LL * 32);
    if (dst == LORA_BF16) kv_gather_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else if (dst == LORA_FP16) kv_gather_kernel<__half><<<grid, kThreads, 0, st>>>(a);
    else kv_gather_kernel<float><<<grid, kThreads, 0, st>>>(a);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace lora
