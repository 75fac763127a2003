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
// A low that is infinite comes with a NaN as step: n * step + low would be that
// infinity, which attention drops as a key of weight zero.
// The quotient is formed in 32 bits; where it lies within 2^-17 of a border
// between two codes (its error is below 15.5 * 3 * 2^-24) the side is decided by
// the sign of (x - low) - step * (border) in 64 bits; a difference of which 64
// bits hold only a part comes with the rest.  That happens to one warp in a
// hundred.  The span, its fifteenth and the rounding to fp16 go through 64 bits:
// a quotient that 64 bits do not hold is rounded to odd there (its last bit says
// that more follows), which makes the rounding to fp16 the only one.
//
// Layout of the work: a head is dim / 16 chunks of 16 elements, one thread per
// chunk: elements [8 c, 8 c + 8) and [rot / 2 + 8 c, + 8) in the half layout,
// [16 c, 16 c + 16) interleaved or past rot.  So a thread owns both elements of
// its pairs (an output may be its input), every access is 16 bytes or wider, and
// the dim / 16 neighbouring lanes that share a head reduce min and max by
// shuffles.  The kernel moves each row once and is bound by memory: 8191 tokens of
// 32 + 32 heads of 128 with 64 rotated, bf16, take 46 us (5.8 TB/s, 89 % of a copy's rate); 8101
// tokens of 32 + 8 + 8 heads from fp32 to bf16 and to the cache, with the read-back, 74 us
// (4.7 TB/s, 72 %), where the quantisation's instructions compete with the loads.
// Small batches are a chain of latencies: a launch, the positions, 64-bit sines
// (16 tokens: 3.4 us, 256 with the cache: 8.5 us).
#include "lora_internal.cuh"
#include "lora_kv.cuh"

namespace lora {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxTok = 2;       // most tokens of one CTA

// Eight elements of a row as they lie in memory, and as numbers.
template <class T> struct Elem;
template <> struct Elem<float> {
    struct Raw { float4 a, b; };
    static __device__ __forceinline__ Raw load(const float *p) {
        return Raw{*reinterpret_cast<const float4 *>(p), *reinterpret_cast<const float4 *>(p + 4)};
    }
    static __device__ __forceinline__ void get(const Raw &r, float (&x)[8]) {
        x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
        x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
    }
    static __device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <class H>
struct Elem16 {
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw load(const H *p) { return *reinterpret_cast<const uint4 *>(p); }
    static __device__ __forceinline__ void get(const Raw &u, float (&x)[8]) {
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
template <> struct Elem<__nv_bfloat16> : Elem16<__nv_bfloat16> {};
template <> struct Elem<__half> : Elem16<__half> {};

// Pairs of the row type: packing, unpacking, and the smaller of each (a NaN wins).
template <class D> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    static __device__ __forceinline__ float2 get(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
        uint32_t y;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    static constexpr uint32_t kInf = 0x7f807f80u;
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 p = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    static __device__ __forceinline__ float2 get(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
        uint32_t y;
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    static constexpr uint32_t kInf = 0x7c007c00u;
};
// (least, minus the greatest) of eight packed elements.
template <class D>
__device__ __forceinline__ uint32_t range_of(const uint32_t (&u)[4]) {
    uint32_t l = Pair<D>::less(Pair<D>::less(u[0], u[1]), Pair<D>::less(u[2], u[3]));
    uint32_t g = Pair<D>::less(Pair<D>::less(u[0] ^ 0x80008000u, u[1] ^ 0x80008000u),
                               Pair<D>::less(u[2] ^ 0x80008000u, u[3] ^ 0x80008000u));
    return Pair<D>::less(__byte_perm(l, g, 0x5410), __byte_perm(l, g, 0x7632));
}

// x - y rounded, and what the rounding left out (Knuth's two-sum).
__device__ __forceinline__ double minus(double x, double y, double &rest) {
    const double d = x - y, b = d - x;
    rest = (x - (d - b)) - (y + b);
    return d;
}
// (x - y) / 15 rounded once to fp16: through a quotient rounded to odd (Boldo and Melquiond's method against double rounding).
__device__ __forceinline__ __half fifteenth(double x, double y) {
    double rest;
    const double diff = minus(x, y, rest);
    // a neighbour of the quotient: a first value, and its remainder times the reciprocal
    const double first = diff * (1.0 / 15.0), quot = fma(fma(-15.0, first, diff), 1.0 / 15.0, first);
    const double more = fma(-15.0, quot, diff) + rest;   // 15 (exact - quot)
    const long long bits = __double_as_longlong(quot);
    return __double2half(__longlong_as_double(more > 0.0 ? bits | 1 : more < 0.0 ? (bits - 1) | 1 : bits));
}

// Codes of eight elements for (step, low), inv = 1 / step or 0 (see the head of the file).
template <class D>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&u)[4], float low, float step, float inv) {
    uint32_t w = 0;
    bool close = false;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 v = Pair<D>::get(u[i]);
#pragma unroll
        for (int k = 1; k >= 0; --k) {
            const float t = fminf(fmaxf(((k ? v.y : v.x) - low) * inv, 0.f), 15.f);   // a NaN becomes 0
            const float r = t + 12582912.f;                                           // 1.5 * 2^23: the nearest integer in the low bits
            close |= fabsf(t - (r - 12582912.f)) > 0.5f - 0x1p-17f;
            w = (w << 4) | (__float_as_uint(r) & 15u);
        }
    }
    if (close) {   // some element lies at a border between codes: decide it exactly
        w = 0;
        for (int i = 7; i >= 0; --i) {
            const float2 v = Pair<D>::get(u[0] * (i < 2) | u[1] * (i / 2 == 1) | u[2] * (i / 2 == 2) | u[3] * (i / 2 == 3));
            const float x = i & 1 ? v.y : v.x, t = fminf(fmaxf((x - low) * inv, 0.f), 15.f), k = floorf(t);
            float n = rintf(t);
            if (fabsf(t - k - 0.5f) < 0x1p-16f) {
                double rest;
                const double diff = minus((double)x, (double)low, rest);
                double side = fma(-(double)step, (double)k + 0.5, diff);   // zero, or far above the rest
                if (side == 0.0) side = rest;
                n = k + (side > 0.0 || (side == 0.0 && ((int)k & 1)) ? 1.f : 0.f);
            }
            w = (w << 4) | (uint32_t)n;
        }
    }
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

// A walk over (token of the CTA, head) pairs, `step` heads at a time.
struct HeadWalk {
    int tl, head;
    __device__ __forceinline__ void wrap(int heads) {
        while (head >= heads) {
            head -= heads;
            ++tl;
        }
    }
};

template <class S, class D, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a, int tok_per_cta) {
    // sine and cosine of the CTA's tokens, [token][pair], both precisions
    extern __shared__ double2 cs64[];
    __shared__ int sm_pos[kMaxTok], sm_slot[kMaxTok];
    float2 *cs32 = reinterpret_cast<float2 *>(cs64 + (CACHE ? tok_per_cta * (a.rot / 2) : 0));
    const int half = a.rot / 2, t0 = blockIdx.x * tok_per_cta, nt = min(tok_per_cta, a.T - t0);
    const int chunks = a.dim / 16, step = kThreads / chunks, heads = a.hq + a.hk + a.hv, c = threadIdx.x % chunks;
    const bool split = 16 * c < a.rot && !a.interleaved;   // of a rotated head: the thread's elements are half a rotation apart
    const int ds0 = split ? 8 * c : 16 * c, ds1 = split ? half + 8 * c : 16 * c + 8;

    HeadWalk w{0, (int)threadIdx.x / chunks};
    if (w.head >= step) w.tl = nt;                          // threads beyond the last whole head
    w.wrap(heads);
    typename Elem<S>::Raw r0, r1;
    const auto load = [&]() {   // the walk's rows, one step ahead of their use
        if (w.tl >= nt) return;
        const bool q = w.head < a.hq, k = !q && w.head < a.hq + a.hk;
        const Rows &src = q ? a.q : k ? a.k : a.v;
        const int h = w.head - (q ? 0 : k ? a.hq : a.hq + a.hk);
        const S *in = reinterpret_cast<const S *>(src.p) + (t0 + w.tl) * src.ts + h * src.hs;
        r0 = Elem<S>::load(in + (q || k ? ds0 : 16 * c));
        r1 = Elem<S>::load(in + (q || k ? ds1 : 16 * c + 8));
    };
    load();
    if (threadIdx.x < nt) {
        sm_pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
        if (CACHE) sm_slot[threadIdx.x] = a.slots[t0 + threadIdx.x];
    }
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int tl = i / half, pos = a.positions[t0 + tl];
        double s, co;
        sincos((double)pos * (double)a.freq[i - tl * half], &s, &co);
        s *= a.mscale;
        co *= a.mscale;
        if (CACHE) cs64[i] = make_double2(co, s);
        cs32[i] = make_float2((float)co, (float)s);
    }
    __syncthreads();

    while (w.tl < nt) {
        const int tl = w.tl, t = t0 + tl, head = w.head;
        float x[8], y[8];
        Elem<S>::get(r0, x);
        Elem<S>::get(r1, y);
        w.head += step;
        w.wrap(heads);
        load();
        if (sm_pos[tl] < 0) continue;
        const int kind = head < a.hq ? 0 : head < a.hq + a.hk ? 1 : 2;
        const int h = kind == 0 ? head : kind == 1 ? head - a.hq : head - a.hq - a.hk;
        const int d0 = kind < 2 ? ds0 : 16 * c, d1 = kind < 2 ? ds1 : 16 * c + 8;
        if (kind < 2 && 16 * c < a.rot) {
            if (CACHE && kind == 1)
                a.interleaved ? turn_interleaved<double>(x, y, cs64 + tl * half + 8 * c)
                              : turn_half<double>(x, y, cs64 + tl * half + 8 * c);
            else
                a.interleaved ? turn_interleaved<float>(x, y, cs32 + tl * half + 8 * c)
                              : turn_half<float>(x, y, cs32 + tl * half + 8 * c);
        }
        uint32_t ux[4], uy[4];   // what the row type holds is what is written, and what is cached
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ux[j] = Pair<D>::pack(x[2 * j], x[2 * j + 1]);
            uy[j] = Pair<D>::pack(y[2 * j], y[2 * j + 1]);
        }
        if (kind == 0 || (kind == 1 ? a.has_ko : a.has_vo)) {
            const Rows &dst = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
            D *out = reinterpret_cast<D *>(dst.p) + t * dst.ts + h * dst.hs;
            *reinterpret_cast<uint4 *>(out + d0) = make_uint4(ux[0], ux[1], ux[2], ux[3]);
            *reinterpret_cast<uint4 *>(out + d1) = make_uint4(uy[0], uy[1], uy[2], uy[3]);
        }
        if (!CACHE || kind == 0) continue;
        const int slot = sm_slot[tl];
        if (slot < 0) continue;
        const int page = slot / a.c.block, off = slot - page * a.c.block;
        if (page >= a.c.num_pages) {
            if (c == 0 && h == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_PAGE);
            continue;
        }
        const uint32_t rx = range_of<D>(ux), ry = range_of<D>(uy);
        // the lanes of this head: chunks is 4 or 8 and heads start at multiples of it
        const int lane = threadIdx.x & 31;
        const uint32_t mask = (chunks == 8 ? 0xffu : 0xfu) << (lane & ~(chunks - 1));
        const int g0 = d0 / LORA_KV_GROUP, g1 = d1 / LORA_KV_GROUP;
        float step0 = 0.f, low0 = 0.f, step1 = 0.f, low1 = 0.f;
        unsigned char *base = half_of(a.c, a.dim, page, off, h, kind - 1);
        for (int g = 0; g < a.dim / LORA_KV_GROUP; ++g) {
            uint32_t r = Pair<D>::less(g0 == g ? rx : Pair<D>::kInf, g1 == g ? ry : Pair<D>::kInf);
            for (int d = 1; d < chunks; d <<= 1) r = Pair<D>::less(r, __shfl_xor_sync(mask, r, d));
            const float2 e = Pair<D>::get(r);   // least, minus the greatest
            const __half hl = __float2half_rn(e.x);
            __half hs = fifteenth(-(double)e.y, (double)e.x);
            if (__hisinf(hl)) hs = __ushort_as_half(0x7fff);   // no sum with an infinite low is a value: NaN
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
        *reinterpret_cast<uint32_t *>(row + d0 / 2) = codes_of<D>(ux, low0, step0, step0 > 0.f ? 1.f / step0 : 0.f);
        *reinterpret_cast<uint32_t *>(row + d1 / 2) = codes_of<D>(uy, low1, step1, step1 > 0.f ? 1.f / step1 : 0.f);
    }
}

template <class D>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(GatherKvArgs a, int tok_per_cta) {
    const int chunks = a.dim / 16, step = kThreads / chunks, c = threadIdx.x % chunks, heads = 2 * a.c.heads;   // K heads, then V heads
    const int t0 = blockIdx.x * tok_per_cta, nt = min(tok_per_cta, a.T - t0);
    HeadWalk w{0, (int)threadIdx.x / chunks};
    for (w.wrap(heads); w.tl < nt; w.head += step, w.wrap(heads)) {
        const int t = t0 + w.tl, which = w.head >= a.c.heads, h = w.head - (which ? a.c.heads : 0);
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
    // A CTA per token for latency; from eight tokens per SM on two share one, whose threads then have twice the work behind one
    // wait for the angles (with the cache, 32 + 8 + 8 heads of 128: 8.5 against 10.5 us at 256 tokens, 78 against 74 us at
    // 8101; CTAs of 256 threads with four tokens take 81 us).
    const int per = a.T >= 1184 ? kMaxTok : 1;
    const int grid = (a.T - 1) / per + 1;   // T is at least 1
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
    const int per = a.T >= 1184 ? kMaxTok : 1, grid = (a.T - 1) / per + 1;
    if (dst == LORA_BF16) kv_gather_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, per);
    else if (dst == LORA_FP16) kv_gather_kernel<__half><<<grid, kThreads, 0, st>>>(a, per);
    else kv_gather_kernel<float><<<grid, kThreads, 0, st>>>(a, per);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace lora
