// Attention of each request's newest tokens over the paged 4-bit cache.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q . k_j), one pass over the
// cache with a running reference for the exponent.  Every cached byte is read
// once per 8 (16) query columns, so with few new tokens the cache's bytes bound
// it; per byte there are two values to unpack, so the unpacking must stay near
// one instruction per value to keep up with memory.
//
// Columns: the new rows of a request times the q heads of one kv head, row
// major; a tile of NC = 8 NT of them shares one reading of the cache.  Per
// granule (16 tokens) a warp forms S^T = K Q^T and O^T += V^T P^T with
// m16n8k16 products whose A operand is the unpacked cache (tokens x dims, then
// dims x tokens) and whose N = 8 dimension is the columns, so that even 4 heads
// per kv head waste only half a column tile.  The order of dimensions inside an
// operand is free as long as both sides use it, and so is the order of tokens:
// a thread reads whole words of codes from shared memory and a mask-and-or
// turns bit fields into numbers.
//   field | 0x6400 is the fp16 number 1024 + n, or 1024 + 16 n for the odd fields.
//   K: queries meet odd fields divided by 16, and the accumulators start at minus
//   (1032 sum of even + 72 sum of odd) query elements, so that they end at
//   q . (n - 8).  The queries go in as fp16 numbers times a power of two of their
//   own (exact down to 2^-24 of the row's largest element).
//   V: one fused multiply-add makes it n - 8.
// So the products take exact integers; steps and lows enter in fp32: a score is
// step * (q . n) + low * sum q per group of 64 dimensions, the weight of a value
// is p * step per group, and sum p * (low + 8 step) is kept apart.  p * step is
// rounded to fp16 (2^-11 relative: an eighth of a bf16 step) after scaling by
// 32 / sref, sref the largest step so far rounded up to a power of two, so that
// neither small steps nor small weights leave fp16's range.  Everything else is
// fp32; the scores' accumulators carry the offsets of 1032 and 72, so that fp32's
// last places of a score go with them (lse off by up to 4e-5 for normal queries,
// 2e-4 where their elements sum to 128).
//
// The exponent's reference m is only moved when a score exceeds it by 10 (in
// powers of two): weights then reach at most 2^10 * 32 in fp16, and the usual
// granule needs no reduction over the warp for its maximum.
//
// Work split: a unit is 8 granules (128 tokens) of one (request, kv head, column
// tile), two for each of 4 warps; the units of the batch are numbered and every CTA takes an equal
// contiguous range, whatever the lengths.  Inside a CTA, 4 warps take granules
// in turn, each with its own ring of cp.async stages that runs ahead across
// (request, head) borders, and are joined in shared memory at the end of a
// piece.  A piece that is not a whole (request, head, tile) leaves its sums in
// the workspace (at most two per CTA: its first and its last), and a second
// launch joins those in order.  (Joining by whichever CTA counts itself last
// saved nothing: 25.4 against 23.1 us for one request, 54.5 against 47.9 us for
// 48 requests of up to 4 tokens at that time, as the main loop spills more registers.)
//
// Measured, 32 / 8 heads of 128, bf16: 32 requests of 8192 tokens 77 us, 3.9 TB/s
// or 60 % of a copy's rate; 128 requests of 1 to 16384 tokens 62 us (49 %); one of
// 32749 tokens 23 us.  Latency bounds it: at 12 warps an SM, which the registers
// allow, warps wait for their own chains (scores, exponentials, transposition,
// values) and instructions are issued in 57 to 60 % of the cycles; 356
// instructions a granule, 16 of them products.  Memory would allow 46 us.  Two
// granules a warp and step at 3 CTAs an SM: one granule at 4 CTAs takes
// 86 to 90 us, four at 2 CTAs 75 us but 1.5 times as long for short requests.
// Short requests cost their pieces' beginning and end, about 4 us each and CTA
// (1024 requests of 64 tokens: 79 us).
#include <type_traits>

#include "lora_internal.cuh"
#include "lora_kv.cuh"
#include "lora_ptx.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kMaxCtas = 444;                      // one column tile: 3 CTAs on each of 148 SMs; two: 2
constexpr int kStages = 3;
constexpr int kFixed = 2;                          // units that starting and joining a segment costs beside its rounds (1: 67, 3: 66, 2: 62 us, ragged)
constexpr float kJump = 10.f;                      // log2 by which a score may exceed the reference
constexpr int kShift = 5;                          // weights are scaled by 2^kShift in fp16
constexpr int kJoinThreads = 512;

// What a CTA leaves for the joining kernel about the segment that begins in it and ends in CTA `last`.
struct alignas(16) Split {
    int last, h, gc0, cols;   // last = 0: none; gc0: its first column, cols: its columns
    int q0, pad[3];           // the request's first query
};

template <int DIM, int NT, int U>
struct Smem {
    alignas(128) unsigned char ring[kWarps][kStages][U * kv_granule_bytes(DIM)];
    float o[kWarps][8 * NT][DIM + 4];
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    long long scan[kWarps];
    long long base;
    int first;
};

constexpr size_t partial_floats(int dim, int nc) { return (size_t)nc * (dim + 2); }   // O, then m, then l

struct Req {
    int q0, nq, len, rounds, tiles;
};

// ROUND: granules the CTA's warps take at a time.
template <int NC, int ROUND>
__device__ __forceinline__ Req load_req(const AttendArgs &a, int r, int G, bool &bad) {
    Req q;
    q.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    q.len = a.kv_len[r];
    q.nq = q1 - q.q0;
    bad = q1 != q.q0 && (q.q0 < 0 || q1 < q.q0 || q1 > a.T || q.nq > a.max_q || q.len < 0 ||
                         (long long)q.len > (long long)a.max_blocks * a.c.block);
    if (bad || q1 == q.q0) q.nq = 0;
    q.tiles = (q.nq * G + NC - 1) / NC;
    constexpr int tokens = ROUND * LORA_KV_GRANULE;
    q.rounds = q.len <= 0 ? 1 : (q.len - 1) / tokens + 1;   // lengths reach 2^31 - 17
    return q;
}

// Units of a request: every (head, tile) is kFixed units and its rounds.
__device__ __forceinline__ long long units_of(const Req &q, int heads) {
    return (long long)q.tiles * heads * (q.rounds + kFixed);
}

// A walk over this CTA's pieces in order.
template <int NC, int ROUND>
struct Walk {
    Req q;
    int r, h, ct, round, n;   // current piece: rounds [round, round + n) of (r, h, ct); n = 0 only right after start()
    long long left;           // units after this piece
    __device__ __forceinline__ void start(const AttendArgs &a, int G, int r0, long long off, long long units) {
        r = r0;
        bool bad;
        q = load_req<NC, ROUND>(a, r, G, bad);
        const int all = q.rounds + kFixed;
        const long long seg = off <= UINT32_MAX ? (long long)((uint32_t)off / (uint32_t)all) : off / all;
        const int from = (int)(off - seg * all), to = (int)min((long long)all, from + units);
        h = q.tiles == 1 ? (int)seg : (int)(seg / q.tiles);
        ct = (int)(seg - (long long)h * q.tiles);
        round = max(0, from - kFixed);
        n = max(0, to - kFixed) - round;
        left = units - (to - from);
    }
    __device__ __forceinline__ bool next(const AttendArgs &a, int G) {
        if (left <= kFixed) return false;   // none, or not one round of the next segment
        round = 0;
        if (++ct == q.tiles) {
            ct = 0;
            if (++h == a.c.heads) {
                h = 0;
                bool bad;
                do q = load_req<NC, ROUND>(a, ++r, G, bad);
                while (q.nq == 0);
            }
        }
        n = (int)min((long long)q.rounds, left - kFixed);
        left -= n + kFixed;
        return true;
    }
    // granules of the piece: [g0, g1)
    __device__ __forceinline__ int g0() const { return round * ROUND; }
    __device__ __forceinline__ int g1() const {
        const int all = q.len <= 0 ? 0 : (q.len - 1) / LORA_KV_GRANULE + 1;
        return min(all, (round + n) * ROUND);
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t mov_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t y;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
    return y;
}
// d += a b, fp16 operands, fp32 accumulators; mma_from: d = a b + (c0, c1, c0, c1).
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};" : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         float c0, float c1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %11, %10, %11};" : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// The masks and exponents of the unpacking, in registers: a mask-and-or with
// two literals would take two instructions.
struct Consts {
    uint32_t lo, hi, h1024, sixteenth;
    __device__ __forceinline__ Consts() {
        asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(lo));
        asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(hi));
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(h1024));
        asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(sixteenth));
    }
};
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(w), "r"(mask), "r"(bits));   // (w & mask) | bits
    return y;
}
__device__ __forceinline__ uint32_t add_h2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// Four fp16 pairs n - 8 from the fields of w: pair j holds fields j and j + 4.
__device__ __forceinline__ void unpack_h(uint32_t w, uint32_t (&x)[4], const Consts &k) {
    const uint32_t sub = 0xe408e408u /* -1032 */, sub72 = 0xd480d480u /* -72 */, v = w >> 8;
    x[0] = add_h2(and_or(w, k.lo, k.h1024), sub);
    x[1] = fma_h2(and_or(w, k.hi, k.h1024), k.sixteenth, sub72);
    x[2] = add_h2(and_or(v, k.lo, k.h1024), sub);
    x[3] = fma_h2(and_or(v, k.hi, k.h1024), k.sixteenth, sub72);
}
// Four fp16 pairs 1024 + n (even fields) and 1024 + 16 n (odd fields).
__device__ __forceinline__ void unpack_raw(uint32_t w, uint32_t (&x)[4], const Consts &k) {
    const uint32_t v = w >> 8;
    x[0] = and_or(w, k.lo, k.h1024);
    x[1] = and_or(w, k.hi, k.h1024);
    x[2] = and_or(v, k.lo, k.h1024);
    x[3] = and_or(v, k.hi, k.h1024);
}
// (step, low) of a token's groups.
template <int NG>
__device__ __forceinline__ void load_params(const unsigned char *p, float2 (&x)[NG]) {
    if (NG == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        x[0] = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        x[NG - 1] = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    } else {
        x[0] = __half22float2(*reinterpret_cast<const __half2 *>(p));
    }
}

template <int DIM, int NT, int U, bool BF>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv_attend_kernel(AttendArgs a, Split *split, float *part) {
    using H = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int NC = 8 * NT, NG = DIM / LORA_KV_GROUP, GB = kv_granule_bytes(DIM), HB = kv_half_bytes(DIM), CB = kv_code_bytes(DIM);
    constexpr int ROUND = kWarps * U;
    extern __shared__ unsigned char smem_raw[];
    Smem<DIM, NT, U> &sm = *reinterpret_cast<Smem<DIM, NT, U> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int G = a.group;

    // Units of the batch and this CTA's range of them.
    const int per = (a.R + kThreads - 1) / kThreads, ra = min(a.R, tid * per), rb = min(a.R, ra + per);
    long long mine = 0;
    bool any_bad = false;
    for (int r = ra; r < rb; ++r) {
        bool bad;
        mine += units_of(load_req<NC, ROUND>(a, r, G, bad), a.c.heads);
        any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_LENGTH);
    long long run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run += x;
    }
    if (lane == 31) sm.scan[warp] = run;
    __syncthreads();
    long long total = 0;
    run -= mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) run += sm.scan[w];
        total += sm.scan[w];
    }
    const long long ctas = min((long long)gridDim.x, total);
    const auto begin_of = [&](long long cta) {   // 32-bit division where it fits: it is on the way to the first load
        const long long x = total * cta;
        return x <= UINT32_MAX ? (long long)((uint32_t)x / (uint32_t)ctas) : x / ctas;
    };
    const long long u0 = blockIdx.x < ctas ? begin_of(blockIdx.x) : total;
    const long long u1 = blockIdx.x < ctas ? begin_of(blockIdx.x + 1) : total;
    if (tid == 0) split[blockIdx.x].last = 0;
    if (u0 >= u1) return;
    if (run <= u0 && u0 < run + mine) {
        long long base = run;
        int r = ra;
        for (;; ++r) {
            bool bad;
            const long long n = units_of(load_req<NC, ROUND>(a, r, G, bad), a.c.heads);
            if (u0 < base + n) break;
            base += n;
        }
        sm.first = r;
        sm.base = base;
    }
    __syncthreads();
    Walk<NC, ROUND> load, comp;
    comp.start(a, G, sm.first, u0 - sm.base, u1 - u0);
    if (comp.n == 0 && !comp.next(a, G)) return;
    load = comp;
    // Columns of a tile as (row, head): the tile's first row and the columns of that row before it, once per piece; then a product
    // in place of each division by G (exact: x < LORA_KV_MAX_GROUP + NC).
    const auto by_g = [&](int x) { return (int)((uint32_t)x * a.inv_group >> 16); };
    const auto first_row = [&](int ct, int &rest) {
        const int row = ct == 0 ? 0 : ct * NC / G;
        rest = ct * NC - row * G;
        return row;
    };
    // Queries of a piece, asked for before they are needed: behind the prologue's table and cache loads, or the join.
    uint4 raw[NT][NG][2];
    const auto load_queries = [&]() {
        int rest;
        const int row0 = first_row(comp.ct, rest);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int x = rest + nt * 8 + g, over = by_g(x), qi = row0 + over, head = comp.h * G + x - over * G;
            const H *row = reinterpret_cast<const H *>(a.q.p) + (long long)(comp.q.q0 + qi) * a.q.ts + (long long)head * a.q.hs;
#pragma unroll
            for (int ng = 0; ng < NG; ++ng)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    raw[nt][ng][i] = make_uint4(0, 0, 0, 0);
                    if (qi < comp.q.nq) raw[nt][ng][i] = *reinterpret_cast<const uint4 *>(row + 64 * ng + 16 * t4 + 8 * i);
                }
        }
    };
    load_queries();

    // The warp's granules, U at a time, into its ring.
    const Consts kc;
    const uint32_t ring = ptx::smem_u32(sm.ring[warp]) + lane * 16;
    const unsigned char *pages = a.c.pages + lane * 16;
    int lg = load.g0() + U * warp, lend = load.g1(), in_ids = 0;
    int page_of = -1, at_of = 0;   // lane i: page and byte offset in it of the i-th granule the warp loads from the last fetch on
    bool more = true;
    uint32_t valid = 0;     // bits s U .. s U + U - 1: the granules that stage s holds
    int in_slot = 0;
    const auto fetch_ids = [&]() {   // the warp's next 32 granules of the piece
        in_ids = 0;
        const int gi = lg + ROUND * (lane / U) + lane % U, blk = gi / a.c.granules;
        at_of = -1;   // none
        if (gi < lend) {
            at_of = (load.h * a.c.granules + gi - blk * a.c.granules) * GB;
            page_of = a.table[(size_t)load.r * a.max_blocks + blk];   // looked at when the granule is asked for: nothing waits here
        }
    };
    const auto advance = [&]() {
        while (more && lg >= lend) {
            more = load.next(a, G);
            if (more) {
                lg = load.g0() + U * warp;
                lend = load.g1();
                if (lg < lend) fetch_ids();
            }
        }
    };
    const auto issue = [&]() {
        if (more) {
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int page = __shfl_sync(~0u, page_of, in_ids + u), at = __shfl_sync(~0u, at_of, in_ids + u);
                if (at < 0) continue;
                if (page >= 0 && page < a.c.num_pages) {
                    const unsigned char *src = pages + page * a.c.page_bytes + at;
                    const uint32_t dst = ring + (in_slot * U + u) * GB;
#pragma unroll
                    for (int i = 0; i < GB / 512; ++i) cp16(dst + 512 * i, src + 512 * i);
                    if (lane < GB % 512 / 16) cp16(dst + GB / 512 * 512, src + GB / 512 * 512);
                    bits |= 1u << u;
                } else if (lane == 0 && a.err) {
                    atomicOr(a.err, LORA_DEV_ERR_BAD_PAGE);
                }
            }
            valid = (valid & ~(((1u << U) - 1) << (in_slot * U))) | bits << (in_slot * U);
            lg += ROUND;
            in_ids += U;
            if (lg >= lend) advance();
            else if (in_ids == 32) fetch_ids();
        }
        cp_commit();
        in_slot = in_slot + 1 == kStages ? 0 : in_slot + 1;
    };
    if (lg < lend) fetch_ids();
    advance();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // Scores stay as step * (q . (n - 8)) + ... until the exponential, which takes them times cq = c 2^qx (c >= 0: a negative
    // scale turns the queries' signs).
    const float c = fabsf(a.scale) * 1.4426950408889634f;
    const int tok = g ^ ((g >> 1) & 1);   // token (of 8) in the operands' row g: both tokens of a pair on different banks
    int out_slot = 0;
    bool first_piece = true;
    for (;;) {
        // Queries of this piece as fp16 numbers times 2^-qx: fragments, per group their sums and the accumulators' start.
        uint32_t qf[NT][NG][4][2];
        float qs[NT][NG][2], start[NT][NG][2], cq[NT][2], jump[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float scale = 1.f, back = 1.f;   // 2^-qx, 2^qx
            {
                float top = 0.f;
#pragma unroll
                for (int ng = 0; ng < NG; ++ng)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf((float)reinterpret_cast<const H *>(&raw[nt][ng][i])[j]));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                // the largest element goes to [2^13, 2^14): odd ones are divided by 16, sums of products stay far from fp32's ends
                const uint32_t e = __float_as_uint(top) >> 23;
                if (e != 0 && e != 255) {
                    const uint32_t to = min(267u - e, 253u);
                    scale = __uint_as_float(to << 23);
                    back = __uint_as_float((254u - to) << 23);
                }
                if (a.scale < 0.f) scale = -scale;
            }
#pragma unroll
            for (int ng = 0; ng < NG; ++ng) {
                float even = 0.f, odd = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const H *e = reinterpret_cast<const H *>(&raw[nt][ng][i]);
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] = (float)e[j] * scale;
                        if (j & 1) {
                            odd += x[j];
                            x[j] *= 0.0625f;
                        } else {
                            even += x[j];
                        }
                    }
                    // pairs (j, j + 4) of the eight dimensions, as the codes unpack
                    qf[nt][ng][2 * i][0] = pack_h2(x[0], x[4]);
                    qf[nt][ng][2 * i][1] = pack_h2(x[1], x[5]);
                    qf[nt][ng][2 * i + 1][0] = pack_h2(x[2], x[6]);
                    qf[nt][ng][2 * i + 1][1] = pack_h2(x[3], x[7]);
                }
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    even += __shfl_xor_sync(~0u, even, d);
                    odd += __shfl_xor_sync(~0u, odd, d);
                }
                const float from = fmaf(-1032.f, even, -72.f * odd);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qs[nt][ng][e] = __shfl_sync(~0u, even + odd, 8 * t4 + 4 * e);
                    start[nt][ng][e] = __shfl_sync(~0u, from, 8 * t4 + 4 * e);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                cq[nt][e] = c * __shfl_sync(~0u, back, 8 * t4 + 4 * e);
                jump[nt][e] = __fdividef(kJump, cq[nt][e]);   // where it lies exactly does not matter
            }
        }
        // Last key each of the thread's columns sees, and the least of the tile.
        int lim[NT][2];
        int rest;
        const int row0 = first_row(comp.ct, rest), back = comp.q.len - comp.q.nq, least = back + row0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) lim[nt][e] = back + min(comp.q.nq - 1, row0 + by_g(rest + nt * 8 + 2 * t4 + e));

        float o[NT][NG][4][4] = {}, om[NT][NG][2] = {}, l[NT][2] = {};
        float m[NT][2], mc[NT][2], thr[NT][2];   // reference score (-inf: none yet); it times c (0); the score that moves it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = thr[nt][e] = -INFINITY;
                mc[nt][e] = 0.f;
            }
        bool begun = false;
        float sref = 0.f, rs = 0.f;   // largest step so far as a power of two; 2^kShift over it

        // U granules at `st`, the first of them granule gi of the request. EDGE: some are missing (`bits`) or hold masked tokens.
        const auto step = [&](auto edge, const unsigned char *st, int gi, uint32_t bits) {
            constexpr bool EDGE = decltype(edge)::value;
            float s[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned char *k = st + u * GB;
                // S^T = K Q^T: rows g and g + 8 of the operand are tokens tok and tok + 8.
                float acc[NT][NG][4];
#pragma unroll
                for (int ng = 0; ng < NG; ++ng) {
                    const uint2 w0 = *reinterpret_cast<const uint2 *>(k + tok * (DIM / 2) + 32 * ng + 8 * t4);
                    const uint2 w1 = *reinterpret_cast<const uint2 *>(k + (tok + 8) * (DIM / 2) + 32 * ng + 8 * t4);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t x[4], y[4];
                        unpack_raw(i ? w0.y : w0.x, x, kc);
                        unpack_raw(i ? w1.y : w1.x, y, kc);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // fields (0, 4) and (1, 5) against dimensions 0, 4 and 1, 5; then (2, 6) and (3, 7)
                            if (i == 0)
                                mma_from(acc[nt][ng], x[0], y[0], x[1], y[1], qf[nt][ng][0][0], qf[nt][ng][0][1], start[nt][ng][0], start[nt][ng][1]);
                            else
                                mma(acc[nt][ng], x[0], y[0], x[1], y[1], qf[nt][ng][2][0], qf[nt][ng][2][1]);
                            mma(acc[nt][ng], x[2], y[2], x[3], y[3], qf[nt][ng][2 * i + 1][0], qf[nt][ng][2 * i + 1][1]);
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float2 p[NG];
                    load_params<NG>(k + CB + (tok + 8 * w) * 4 * NG, p);
#pragma unroll
                    for (int ng = 0; ng < NG; ++ng) {
                        const float low = fmaf(8.f, p[ng].x, p[ng].y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = ng == 0 ? low * qs[nt][0][e] : fmaf(low, qs[nt][ng][e], s[u][nt][2 * w + e]);
                                s[u][nt][2 * w + e] = fmaf(p[ng].x, acc[nt][ng][2 * w + e], x);
                            }
                    }
                    if (EDGE) {
                        const int j = (gi + u) * LORA_KV_GRANULE + tok + 8 * w;
                        const bool here = (bits >> u) & 1;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!here || j > lim[nt][e]) s[u][nt][2 * w + e] = -INFINITY;
                    }
                }
            }
            // Steps and lows of the values.
            float vs[U][NG][2], vl[U][NG][2], most = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float2 p[NG];
                    load_params<NG>(st + u * GB + HB + CB + (tok + 8 * w) * 4 * NG, p);
#pragma unroll
                    for (int ng = 0; ng < NG; ++ng) {
                        vs[u][ng][w] = p[ng].x;
                        vl[u][ng][w] = fmaf(8.f, p[ng].x, p[ng].y);
                        if (EDGE && (!((bits >> u) & 1) || (gi + u) * LORA_KV_GRANULE + tok + 8 * w >= comp.q.len))
                            vs[u][ng][w] = vl[u][ng][w] = 0.f;   // not the request's: whatever is there
                        most = fmaxf(most, vs[u][ng][w]);
                    }
                }
            bool up = most > sref;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                    for (int u = 1; u < U; ++u) t = fmaxf(t, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
                    up |= t > thr[nt][e];
                }
            if (__any_sync(~0u, up)) {
                // Move the references: rare after a request's first granules.
                float top = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
                        for (int w = 0; w < 2; ++w) top = fmaxf(top, vs[u][ng][w] < INFINITY ? vs[u][ng][w] : 0.f);
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                float ratio = 1.f;   // old sref over new
                if (top > sref) {
                    // the next power of two above (steps that are not finite only reach the columns that see them)
                    const float n = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + 0x00800000u);
                    const float inv = __uint_as_float(0x7f000000u - __float_as_uint(n));   // 1 / n: n lies within 2^-23 and 2^16
                    ratio = sref * inv;
                    sref = n;
                    rs = (float)(1 << kShift) * inv;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = -INFINITY;
#pragma unroll
                        for (int u = 0; u < U; ++u) t = fmaxf(t, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
                        t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
                        const float n = fmaxf(m[nt][e], t);
                        const float f = m[nt][e] == n ? 1.f : m[nt][e] == -INFINITY ? 0.f : ex2((m[nt][e] - n) * cq[nt][e]);
                        m[nt][e] = n;
                        mc[nt][e] = n == -INFINITY ? 0.f : n * cq[nt][e];
                        thr[nt][e] = n + jump[nt][e];
                        if (!begun) continue;   // nothing to scale yet
                        l[nt][e] *= f;
#pragma unroll
                        for (int ng = 0; ng < NG; ++ng) {
                            om[nt][ng][e] *= f;
#pragma unroll
                            for (int mt = 0; mt < 4; ++mt) {
                                o[nt][ng][mt][e] *= f * ratio;
                                o[nt][ng][mt][2 + e] *= f * ratio;
                            }
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // Weights, their sums, and the B operands p * step of the second product.
                uint32_t pb[NT][NG][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2(fmaf(s[u][nt][e], cq[nt][e & 1], -mc[nt][e & 1]));
                        if (EDGE && s[u][nt][e] == -INFINITY) p[e] = 0.f;   // with scale 0 too
                        l[nt][e & 1] += p[e];
                    }
#pragma unroll
                    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const float vr = vs[u][ng][w] * rs;
                            float x0 = p[2 * w] * vr, x1 = p[2 * w + 1] * vr;
                            float y0 = p[2 * w] * vl[u][ng][w], y1 = p[2 * w + 1] * vl[u][ng][w];
                            if (EDGE) {   // a masked token does not count, even one that is not finite
                                if (s[u][nt][2 * w] == -INFINITY) x0 = y0 = 0.f;
                                if (s[u][nt][2 * w + 1] == -INFINITY) x1 = y1 = 0.f;
                            }
                            om[nt][ng][0] += y0;
                            om[nt][ng][1] += y1;
                            pb[nt][ng][w] = mov_trans(pack_h2(x0, x1));
                        }
                }
                // O^T += V^T P^T: a thread's tokens are those of operand columns 2 t4, 2 t4 + 1 and 8 above.
                const int ta = 2 * t4 + (t4 & 1), tb = 2 * t4 + 1 - (t4 & 1);
#pragma unroll
                for (int ng = 0; ng < NG; ++ng) {
                    const unsigned char *v = st + u * GB + HB + 32 * ng + 4 * g;
                    uint32_t lo[2][4], hi[2][4];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t x = *reinterpret_cast<const uint32_t *>(v + (ta + 8 * w) * (DIM / 2));
                        const uint32_t y = *reinterpret_cast<const uint32_t *>(v + (tb + 8 * w) * (DIM / 2));
                        unpack_h(__byte_perm(x, y, 0x5410), lo[w], kc);   // dimensions 8 g + 0 .. 3 of both tokens
                        unpack_h(__byte_perm(x, y, 0x7632), hi[w], kc);   // 8 g + 4 .. 7
                    }
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        const uint32_t(&z)[2][4] = mt < 2 ? lo : hi;
                        const int i = 2 * (mt & 1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma(o[nt][ng][mt], z[0][i], z[0][i + 1], z[1][i], z[1][i + 1], pb[nt][ng][0], pb[nt][ng][1]);
                    }
                }
            }
            begun = true;
        };

        const int gend = comp.g1();
        for (int gi = comp.g0() + U * warp; gi < gend; gi += ROUND) {
            cp_wait<kStages - 2>();
            __syncwarp();
            issue();
            const uint32_t bits = (valid >> (out_slot * U)) & ((1u << U) - 1);
            const unsigned char *st = sm.ring[warp][out_slot];
            out_slot = out_slot + 1 == kStages ? 0 : out_slot + 1;
            if (bits == (1u << U) - 1 && (gi + U) * LORA_KV_GRANULE - 1 <= least) step(std::false_type{}, st, gi, bits);
            else if (bits) step(std::true_type{}, st, gi, bits);
        }

        const Walk<NC, ROUND> cur = comp;
        const bool again = comp.next(a, G);
        if (again) load_queries();
        // Join the warps.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
#pragma unroll
                    for (int ng = 0; ng < NG; ++ng) om[nt][ng][e] += __shfl_xor_sync(~0u, om[nt][ng][e], d);
                }
            }
        __syncthreads();   // the buffers' last readers are done
        const float unit = sref * (1.f / (1 << kShift));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * t4 + e;
                if (g == 0) {
                    sm.m[warp][col] = m[nt][e] == -INFINITY ? -INFINITY : mc[nt][e];
                    sm.l[warp][col] = l[nt][e];
                }
#pragma unroll
                for (int ng = 0; ng < NG; ++ng) {
                    float x[8];
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {   // rows g and g + 8 are dimensions 8 g + 2 mt and one above
                        x[2 * mt] = fmaf(o[nt][ng][mt][e], unit, om[nt][ng][e]);
                        x[2 * mt + 1] = fmaf(o[nt][ng][mt][2 + e], unit, om[nt][ng][e]);
                    }
                    float4 *d = reinterpret_cast<float4 *>(&sm.o[warp][col][64 * ng + 8 * g]);
                    d[0] = make_float4(x[0], x[1], x[2], x[3]);
                    d[1] = make_float4(x[4], x[5], x[6], x[7]);
                }
            }
        __syncthreads();
        const bool whole = cur.round == 0 && cur.n == cur.q.rounds;
        const int slot = 2 * blockIdx.x + (first_piece && cur.round > 0 ? 0 : 1);
        float *dst = part + (size_t)slot * partial_floats(DIM, NC);
        constexpr int kChunks = DIM / 8;
        for (int i = tid; i < NC * kChunks; i += kThreads) {
            const int col = i / kChunks, d0 = (i % kChunks) * 8;
            float mm = sm.m[0][col], ll = 0.f, x[8] = {};
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm.m[w][col]);
            const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sm.m[w][col] - ref);
                ll = fmaf(f, sm.l[w][col], ll);
                const float4 u = *reinterpret_cast<const float4 *>(&sm.o[w][col][d0]);
                const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][col][d0 + 4]);
                x[0] = fmaf(f, u.x, x[0]); x[1] = fmaf(f, u.y, x[1]); x[2] = fmaf(f, u.z, x[2]); x[3] = fmaf(f, u.w, x[3]);
                x[4] = fmaf(f, v.x, x[4]); x[5] = fmaf(f, v.y, x[5]); x[6] = fmaf(f, v.z, x[6]); x[7] = fmaf(f, v.w, x[7]);
            }
            if (!whole) {
                float4 *p = reinterpret_cast<float4 *>(dst + col * DIM + d0);
                p[0] = make_float4(x[0], x[1], x[2], x[3]);
                p[1] = make_float4(x[4], x[5], x[6], x[7]);
                if (d0 == 0) {
                    dst[NC * DIM + col] = mm;
                    dst[NC * DIM + NC + col] = ll;
                }
                continue;
            }
            const int x0 = rest + col, over = by_g(x0), qi = row0 + over, head = cur.h * G + x0 - over * G;
            if (qi >= cur.q.nq) continue;
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            uint4 u;
            H *e = reinterpret_cast<H *>(&u);
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = (H)(x[k] * inv);
            *reinterpret_cast<uint4 *>(reinterpret_cast<H *>(a.o.p) + (long long)(cur.q.q0 + qi) * a.o.ts +
                                       (long long)head * a.o.hs + d0) = u;
            if (a.lse && d0 == 0)
                a.lse[(size_t)(cur.q.q0 + qi) * a.hq + head] = ll == 0.f ? -INFINITY : 0.6931471805599453f * (ref + log2f(ll));
        }
        if (tid == 0 && !whole && cur.round + cur.n < cur.q.rounds && !(first_piece && cur.round > 0)) {
            // the segment begins here and goes on: its last unit is u1 - 1 + (rounds not done)
            const long long end = u1 - 1 + (cur.q.rounds - cur.round - cur.n);
            long long last = ((end + 1) * ctas + total - 1) / total - 1;   // the CTA whose range holds `end`
            while (total * (last + 1) / ctas <= end) ++last;
            while (total * last / ctas > end) --last;
            split[blockIdx.x] = Split{(int)last, cur.h, cur.ct * NC, min(NC, cur.q.nq * G - cur.ct * NC), cur.q.q0, {}};
        }
        first_piece = false;
        if (!again) break;
    }
    cp_wait<0>();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // here, not at the start: waiting CTAs take slots (14.5 against 13.8 us)
}

// Joins the pieces of the segment that begins in CTA blockIdx.x, in order: the warps are dealt out to the columns that
// there are (4 query heads of one token: 4 warps each), a lane has DIM / 32 dimensions.  What it costs is a chain of
// latencies - its launch, Split, the maxima, the sums - about 6 of the 23 us of one request of 32749 tokens.
template <int DIM, int NT, bool BF>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttendArgs a, const Split *split, const float *part) {
    using H = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int NC = 8 * NT, E = DIM / 32, kJoinWarps = kJoinThreads / 32;
    __shared__ float sm_o[kJoinWarps][DIM], sm_l[kJoinWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Split s = split[blockIdx.x];
    if (s.last == 0) return;
    const int G = a.group, first = blockIdx.x, n = s.last - first + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cols = s.cols, W = kJoinWarps / cols;   // W: warps of a column
    const int col = warp % cols, w = warp / cols;
    if (W == 1 && w > 0) return;
    // piece i: the second slot of the first CTA, the first slot of the others
    const auto at = [&](int i) { return part + (size_t)(2 * (first + i) + (i == 0)) * partial_floats(DIM, NC); };
    float mm = -INFINITY;
    for (int i = lane; i < n; i += 32) mm = fmaxf(mm, at(i)[NC * DIM + col]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, d));
    const float ref = mm == -INFINITY ? 0.f : mm;
    float x[E] = {}, ll = 0.f;
#pragma unroll 8
    for (int i = w < W ? w : n; i < n; i += W) {
        const float *p = at(i);
        const float f = ex2(p[NC * DIM + col] - ref);
        ll = fmaf(f, p[NC * DIM + NC + col], ll);
        if (E == 4) {
            const float4 u = *reinterpret_cast<const float4 *>(p + col * DIM + lane * 4);
            x[0] = fmaf(f, u.x, x[0]);
            x[1] = fmaf(f, u.y, x[1]);
            x[E - 2] = fmaf(f, u.z, x[E - 2]);
            x[E - 1] = fmaf(f, u.w, x[E - 1]);
        } else {
            const float2 u = *reinterpret_cast<const float2 *>(p + col * DIM + lane * 2);
            x[0] = fmaf(f, u.x, x[0]);
            x[1] = fmaf(f, u.y, x[1]);
        }
    }
    if (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = x[e];
        if (lane == 0) sm_l[warp] = ll;
        __syncthreads();
        if (w != 0) return;
        for (int k = 1; k < W; ++k) {
            ll += sm_l[k * cols + col];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] += sm_o[k * cols + col][lane * E + e];
        }
    }
    const int gc = s.gc0 + col, qi = gc / G, head = s.h * G + gc - qi * G;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    H *out = reinterpret_cast<H *>(a.o.p) + (long long)(s.q0 + qi) * a.o.ts + (long long)head * a.o.hs + lane * E;
    alignas(8) H y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = (H)(x[e] * inv);
    if (E == 4) *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(y);
    else *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(y);
    if (a.lse && lane == 0) a.lse[(size_t)(s.q0 + qi) * a.hq + head] = ll == 0.f ? -INFINITY : 0.6931471805599453f * (ref + log2f(ll));
}

// Two column tiles that share one reading of the cache, or one at a time: up to 8 columns there is only one.  Above, two take 26.6
// against 27.9 us (32 requests of 8192, 16 heads on one kv head), 62 against 78 (128 of those), 110 against 116 and 168 against
// 180 (32 of 8192, 4 and 8 tokens of 32 / 8 heads), but 43.9 against 42.0 us (48 of up to 4096 with 1 to 4 tokens), 42.5 against
// 37.0 (64 of up to 8192 with 1 to 3) and 65 against 55 (256 of 256 with 4): drafts that do not fill their columns, and short
// contexts, where 8 warps an SM hide less.  Lengths and rows lie on the device; by the sizes the host has, reading a long cache
// once is the safer side.
int tiles_of(int hq, int hkv, int max_q) { return (long long)max_q * (hq / hkv) <= 8 ? 1 : 2; }
template <int NT>
constexpr int ctas_per_sm() { return NT == 1 ? 3 : 2; }   // what the registers allow

constexpr size_t kSplitBytes = (kMaxCtas * sizeof(Split) + 255) / 256 * 256;

template <int DIM, int NT, bool BF>
int launch(const AttendArgs &a, cudaStream_t st) {
    Split *split = static_cast<Split *>(a.ws);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kSplitBytes);
    constexpr int U = 2;
    const size_t smem = sizeof(Smem<DIM, NT, U>);
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (int rc = cuda_check(cudaGetDevice(&dev))) return rc;
    if (int rc = allow_smem(kv_attend_kernel<DIM, NT, U, BF>, smem, done, dev)) return rc;
    const int grid = 148 * ctas_per_sm<NT>();
    kv_attend_kernel<DIM, NT, U, BF><<<grid, kThreads, smem, st>>>(a, split, part);
    count_launch();
    if (int rc = cuda_check(cudaGetLastError())) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    return cuda_check(cudaLaunchKernelEx(&cfg, kv_join_kernel<DIM, NT, BF>, a, (const Split *)split, (const float *)part));
}

template <int DIM, int NT>
int launch_type(const AttendArgs &a, cudaStream_t st) {
    return a.dtype == LORA_BF16 ? launch<DIM, NT, true>(a, st) : launch<DIM, NT, false>(a, st);
}

}  // namespace

size_t attend_workspace(int hq, int hkv, int dim, int max_q) {
    const size_t n = partial_floats(dim, 8 * tiles_of(hq, hkv, max_q)) * 2 * kMaxCtas * sizeof(float);
    return kSplitBytes + (n + 255) / 256 * 256;
}

int launch_kv_attend(const AttendArgs &a, cudaStream_t st) {
    const bool one = tiles_of(a.hq, a.c.heads, a.max_q) == 1;
    if (a.dim == 64) return one ? launch_type<64, 1>(a, st) : launch_type<64, 2>(a, st);
    return one ? launch_type<128, 1>(a, st) : launch_type<128, 2>(a, st);
}

}  // namespace lora
