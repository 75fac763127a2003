// Causal attention over packed prompts on the 5th-generation tensor cores.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q . k_j), j <= m - n + i for
// query i of a request with n query and m key rows.  A CTA owns two tiles of
// 128 query rows of one kv head and walks the keys in tiles of 128 with a
// running reference for the exponent, the scores and the output accumulators in
// tensor memory:
//   S_t = Q_t K^T     tcgen05.mma, both operands in shared memory (TMA, SW128)
//   P_t = exp2(S_t)   one thread per row reads S_t from tensor memory and writes
//                     P_t, rounded to the row type, over it
//   O_t += P_t V      tcgen05.mma, A = P_t in tensor memory, B = V as TMA lays it
//                     (keys x dims, read MN-major)
// While one tile's scores go through the exponential the tensor cores work on the
// other.  Per 128 x 128 tile at head_dim 128 the two products take 1024 cycles and
// the 16384 exponentials 1024 cycles of the 16-wide unit, so the two are balanced
// and everything else has to hide behind them.
//
// Rows of a tile are tokens x PK query heads of the kv head (PK: the largest
// power of two that divides the group), token major: a short prompt fills
// more of a tile, and a group shares its keys' and values' way through shared
// memory.
//
// The reference of a row moves only when a score exceeds it by 8 powers of two;
// O_t is then rescaled in tensor memory by the row's own thread.  S_t of the next
// keys is issued behind the product that reads P_t, so its arrival also says that
// O_t is at rest.
//
// One CTA per SM works through a list of items (request, tile pair, head block)
// without draining its pipelines between them: the next item's queries are loaded
// when the current one's last scores are done, its keys follow the current one's
// values through the same ring, and its first scores are issued while the row
// owners still write the current outputs.  Items are taken in the order of 16
// classes of work, most keys first, so that the last ones are small.
//
// Roles: warp 0 loads, warp 1 issues the products (one lane) and clears the values
// behind a request's last key in its last tile, warp 3 lists the items, warps 4-7
// and 8-11 own tile 0 and 1.  Waits are bounded (LORA_DEV_ERR_TIMEOUT).  No
// cluster multicast.
//
// Measured, bf16, 32 / 8 heads of 128, among calls of the same kind, which bring the
// card to its power limit: one prompt of 8192 tokens 525 to 555 us, 0.99 to 1.05
// PFLOP/s (a large library product: 1.64 in bursts, 1.38 sustained; alone, under a
// profiler, 498 us); 16 of 128 to 2048 tokens 182 to 209 us; 64 of 128 tokens
// 46 us; 24 of up to 97 tokens, fp16, heads of 64, 12 us; one of 16 tokens 8 us.
// What bounds long prompts is the tensor pipe's start: a product whose 16 instructions should take 1024
// cycles takes about 1450 when it is issued by itself, as the two products of a
// tile are (one waits for the exponentials, which keep pace).  Products issued by
// two warps, weights handed over in halves, a quarter of the exponentials as
// polynomials, or two threads a row all came out equal or slower (484 to 1020 us
// at 8192), and so did scores that do not wait for the product before them (P_t
// in columns of its own, which leaves room for tiles of 80 keys: 774 us, as twice
// the starts cost more than the waits).  Ragged batches lose to diagonal tiles and to rows of short prompts
// that a tile of 128 does not fill.
#include <cuda.h>

#include <type_traits>

#include "lora_internal.cuh"
#include "lora_kv.cuh"
#include "lora_ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 384;
constexpr int kM = 128, kN = 128;    // rows of a tile, keys of a tile
constexpr float kJump = 8.f;         // log2 by which a score may exceed the reference
constexpr long long kWaitLimit = 2000000000LL;

template <int DIM>
constexpr int stages() { return DIM == 128 ? 5 : 8; }

constexpr int kClasses = 16;

struct Item {
    int q0, nq, k0, nk, tok0, head;   // nq < 0: no more items
};

template <int DIM>
struct Smem {
    unsigned char q[2][kM * DIM * 2];              // [dim half][row][64] SW128
    unsigned char kv[stages<DIM>()][kN * DIM * 2]; // the same
    uint64_t q_full[2], q_empty[2], full[stages<DIM>()], empty[stages<DIM>()], s_full[2], p_ready[2], o_full[2], drain;
    uint64_t item_full[2], item_empty[2];
    Item item[2];
    uint32_t tmem;
    int abort;
    int most, hist[kClasses];                      // most key tiles of an item; tile pairs of each class
};

struct Maps {
    CUtensorMap q, k, v;
};

struct KArgs {
    void *o;
    long long ots, ohs;
    float *lse;
    const int32_t *cu_q, *cu_k;
    int Tq, Tk, R, hq, G, pk, groups;   // pk: heads in a tile; groups: tiles' head blocks, hq / pk
    uint32_t items;   // most items of row ranges that do not overlap
    float scale;
    int32_t *err;
    const int32_t *kv_len;   // null, or what each request has with its past: no more than its rows, else it is refused
};

template <class Sm>
__device__ __forceinline__ bool wait(uint64_t *b, uint32_t parity, Sm &sm, int32_t *err) {
    const uint32_t a = ptx::smem_u32(b);
    if (ptx::mbar_try(a, parity)) return true;
    const long long t0 = clock64();
    while (!ptx::mbar_try(a, parity)) {
        if (*(volatile int *)&sm.abort) return false;
        if (clock64() - t0 > kWaitLimit) {
            *(volatile int *)&sm.abort = 1;
            if (err) atomicOr(err, LORA_DEV_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// For this thread's own asynchronous work before the CTA exits: bounded, not cut short by the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t *b, uint32_t parity) {
    const long long t0 = clock64();
    while (!ptx::mbar_try(ptx::smem_u32(b), parity) && clock64() - t0 < kWaitLimit / 8) {
    }
}

// Shared memory descriptors (SW128, 8 rows of 128 bytes apart by 1024): the upper half is a constant, so that the steps through
// a tile are 32-bit additions.
constexpr uint32_t kDescHi = 1024u >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t sdesc(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | (lbo >> 4) << 16; }
// kind::f16 with fp32 accumulators; type 0 = fp16, 1 = bf16.
constexpr uint32_t idesc(int type, int N, int b_mn) {
    return 1u << 4 | (uint32_t)type << 7 | (uint32_t)type << 10 | (uint32_t)b_mn << 16 | (uint32_t)(N >> 3) << 17 | (uint32_t)(kM >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(id), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(id), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define R8(r, i) "=f"(r[i]), "=f"(r[i + 1]), "=f"(r[i + 2]), "=f"(r[i + 3]), "=f"(r[i + 4]), "=f"(r[i + 5]), "=f"(r[i + 6]), "=f"(r[i + 7])
#define W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void ld32(float (&r)[32], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
                 "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];" : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24) : "r"(addr));
}
__device__ __forceinline__ void ld16(float (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : R8(r, 0), R8(r, 8) : "r"(addr));
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(addr), W8(r, 0), W8(r, 8) : "memory");
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
                 "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr), W8(r, 0), W8(r, 8), W8(r, 16), W8(r, 24) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations an instruction (the same rate of operations, half the issue slots).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t y;
    if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// A request's rows and keys; nq = -1 if its ranges are none.
struct Req {
    int q0, nq, k0, nk;
};
__device__ __forceinline__ Req request(const KArgs &a, int r) {
    const int q0 = a.cu_q[r], q1 = a.cu_q[r + 1], k0 = a.cu_k[r], k1 = a.cu_k[r + 1];
    const bool past = a.kv_len && a.kv_len[r] > (long long)q1 - q0;
    const bool bad = past || q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk;
    return bad ? Req{0, -1, 0, 0} : Req{q0, q1 - q0, k0, k1 - k0};
}
// Key tiles that rows up to token `last` see.
__device__ __forceinline__ int tiles_to(const Req &q, int last) {
    const int key = q.nk - q.nq + last;
    return key < 0 ? 0 : key / kN + 1;
}
// First tile pair (of 1 << sh tokens) of a request with at least x key tiles; its number of pairs if none.
__device__ __forceinline__ int first_pair(const Req &q, int x, int sh) {
    if (q.nq <= 0) return 0;
    const int n = (q.nq - 1 >> sh) + 1;
    if (x <= 0) return 0;
    const long long last = (long long)(x - 1) * kN - (q.nk - q.nq);   // the first token that sees that many
    return last <= 0 ? 0 : last > q.nq - 1 ? n : (int)(last >> sh);
}

template <int DIM, bool BF>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Maps maps, KArgs a) {
    using H = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int ST = stages<DIM>(), HALVES = DIM / 64;
    constexpr uint32_t TILE = kN * DIM * 2, HALF = kN * 128;   // bytes of a tile and of its 64-column block
    constexpr float kShift = BF ? 0.f : 7.f;                   // fp16 weights are scaled by 2^7: room below for small ones
    extern __shared__ unsigned char raw[];
    Smem<DIM> &sm = *reinterpret_cast<Smem<DIM> *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int toks = kM / a.pk, sh = __ffs(toks), lpk = __ffs(a.pk) - 1;   // tokens of a tile; log2 of a pair's, of the heads'

    Req q{0, 0, 0, 0};   // warp 3: the lane's request
    if (warp == 3 && a.R <= 32 && lane < a.R) q = request(a, lane);
    if (warp == 2 && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(&sm.full[s], 1);
            ptx::mbar_init(&sm.empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(&sm.q_full[t], 1);
            ptx::mbar_init(&sm.q_empty[t], 1);
            ptx::mbar_init(&sm.s_full[t], 1);
            ptx::mbar_init(&sm.p_ready[t], 4);
            ptx::mbar_init(&sm.o_full[t], 1);
            ptx::mbar_init(&sm.item_full[t], 1);
            ptx::mbar_init(&sm.item_empty[t], 10);
        }
        ptx::mbar_init(&sm.drain, 1);
        sm.abort = 0;
        sm.most = 0;
        for (int b = 0; b < kClasses; ++b) sm.hist[b] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sm.tmem;
    // The classes of work: items of x key tiles are class x / width.  Up to 32 requests are one warp's affair (warp 3: 24 short
    // prompts take 13.3 us, 15.7 with the count); with more, where a warp would walk the list once per class, the CTA counts
    // the tile pairs of each class first.
    const bool few = a.R <= 32;
    if (!few) {
        int most = 0;
        for (int r = tid; r < a.R; r += kThreads) {
            const Req q = request(a, r);
            if (q.nq < 0 && blockIdx.x == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_LENGTH);
            if (q.nq > 0) most = max(most, tiles_to(q, q.nq - 1));
        }
        if (most > 0) atomicMax(&sm.most, most);
        __syncthreads();
        const int width = sm.most / kClasses + 1;
        for (int r = tid; r < a.R; r += kThreads) {
            const Req q = request(a, r);
            if (q.nq <= 0) continue;
            int from = 0;
            for (int b = 0; b < kClasses; ++b) {
                const int to = b + 1 == kClasses ? (q.nq - 1 >> sh) + 1 : first_pair(q, (b + 1) * width, sh);
                if (to > from) atomicAdd(&sm.hist[b], to - from);
                from = to;
            }
        }
        __syncthreads();
    }

    // Every role reads the items in order.
    uint32_t items = 0;
    const auto next_item = [&](Item &it) {
        const int s = items & 1;
        bool ok = wait(&sm.item_full[s], (items >> 1) & 1, sm, a.err);
        ok = __all_sync(~0u, ok);
        if (ok) it = sm.item[s];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.item_empty[s]);
        ++items;
        return ok && it.nq >= 0;
    };
    // Key tiles of each query tile: up to the last key its last token sees.
    const auto key_tiles = [&](const Item &it, int t) {
        const int first = it.tok0 + t * toks, last = min(it.nq, first + toks) - 1, key = it.nk - it.nq + last;
        return last < first || key < 0 ? 0 : key / kN + 1;
    };

    // Registers go to the row owners: 128 x (88 + 2 x 208) is what the block was launched with, 384 x 168 (checked by the host).
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 3) {
            int r0 = 0;                           // where the list is: class, block of 32 requests,
            long long before = 0;                 // pairs listed before this block
            int cnt = 0, run = 0, lo = 0;         // this lane's request: pairs in the class, their inclusive sum, the first of them
            bool fresh = true;
            int cls = kClasses - 1, width;
            if (few) {
                if (q.nq < 0 && blockIdx.x == 0 && a.err) atomicOr(a.err, LORA_DEV_ERR_BAD_LENGTH);
                int most = q.nq > 0 ? tiles_to(q, q.nq - 1) : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) most = max(most, __shfl_xor_sync(~0u, most, d));
                // the pairs of one request are in order already
                width = a.R == 1 ? most + 1 : most / kClasses + 1;
                cls = most / width;               // the classes above are empty
            } else {
                width = sm.most / kClasses + 1;
            }
            for (uint32_t n = 0;; ++n) {
                // every other round of items backwards: a CTA's largest item of one round goes with its smallest of the next
                const uint32_t k = n * gridDim.x + ((n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x), want = k / a.groups;
                Item it{0, -1, 0, 0, 0, 0};
                while (cls >= 0 && k < a.items) {
                    if (!few && r0 == 0 && fresh && before + sm.hist[cls] <= want) {   // the class as a whole is behind
                        before += sm.hist[cls];
                        --cls;
                        continue;
                    }
                    if (fresh) {
                        if (!few) q = r0 + lane < a.R ? request(a, r0 + lane) : Req{0, 0, 0, 0};
                        cnt = 0;
                        if (q.nq > 0) {
                            lo = first_pair(q, cls * width, sh);
                            cnt = (cls + 1 == kClasses ? (q.nq - 1 >> sh) + 1 : first_pair(q, (cls + 1) * width, sh)) - lo;
                        }
                        run = cnt;
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) {
                            const int x = __shfl_up_sync(~0u, run, d);
                            if (lane >= d) run += x;
                        }
                        fresh = false;
                    }
                    const uint32_t hit = __ballot_sync(~0u, before + run > want);
                    if (hit) {
                        const int l = __ffs(hit) - 1;
                        const int pair = lo + (int)(before + run - 1 - want);   // the longest rows of a request first
                        it.q0 = __shfl_sync(~0u, q.q0, l);
                        it.nq = __shfl_sync(~0u, q.nq, l);
                        it.k0 = __shfl_sync(~0u, q.k0, l);
                        it.nk = __shfl_sync(~0u, q.nk, l);
                        it.tok0 = __shfl_sync(~0u, pair, l) << sh;
                        it.head = (int)(k - want * a.groups) * a.pk;
                        break;
                    }
                    before += __shfl_sync(~0u, run, 31);
                    r0 += 32;
                    fresh = true;
                    if (r0 >= a.R) {
                        r0 = 0;
                        --cls;
                    }
                }
                const int s = n & 1;
                bool ok = n < 2 || wait(&sm.item_empty[s], (n / 2 - 1) & 1, sm, a.err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                if (lane == 0) {
                    sm.item[s] = it;
                    ptx::mbar_arrive(&sm.item_full[s]);
                }
                if (it.nq < 0) break;
            }
        } else if (warp == 0) {
            Item it;
            int i = 0, qn[2] = {0, 0};
            bool ok = true;
            while (ok && next_item(it)) {
                const int nt0 = key_tiles(it, 0), nt1 = key_tiles(it, 1), total = max(nt0, nt1), kvh = it.head / a.G;
                if (lane == 0) {
                    for (int j = 0; ok && j < 2 * total; ++j) {
                        const int s = i % ST;
                        ok = i < ST || wait(&sm.empty[s], (i / ST - 1) & 1, sm, a.err);
                        if (!ok) break;
                        ptx::mbar_expect_tx(&sm.full[s], TILE);
                        for (int h = 0; h < HALVES; ++h)
                            ptx::tma_load_3d(sm.kv[s] + h * HALF, (j & 1) ? &maps.v : &maps.k, h * 64, kvh, it.k0 + (j >> 1) * kN, &sm.full[s]);
                        ++i;
                        if (j > 0) continue;
                        for (int t = 0; ok && t < 2; ++t) {   // behind the first keys: these do not wait for the last item's scores
                            if ((t ? nt1 : nt0) == 0) continue;
                            ok = qn[t] == 0 || wait(&sm.q_empty[t], (qn[t] - 1) & 1, sm, a.err);
                            if (!ok) break;
                            ++qn[t];
                            ptx::mbar_expect_tx(&sm.q_full[t], TILE);
                            for (int h = 0; h < HALVES; ++h)
                                ptx::tma_load_3d(sm.q[t] + h * HALF, &maps.q, h * 64, it.head, it.q0 + it.tok0 + t * toks, &sm.q_full[t]);
                        }
                    }
                }
                ok = __shfl_sync(~0u, (int)ok, 0);
            }
            if (lane == 0 && *(volatile int *)&sm.abort) {   // loads in flight land before the CTA goes
                for (int t = 0; t < 2; ++t)
                    if (qn[t] > 0) drain_wait(&sm.q_full[t], (qn[t] - 1) & 1);
                for (int j = max(0, i - ST); j < i; ++j) drain_wait(&sm.full[j % ST], (j / ST) & 1);
            }
            __syncwarp();
        } else if (warp == 1) {
            constexpr uint32_t id_s = idesc(BF ? 1 : 0, kN, 0), id_o = idesc(BF ? 1 : 0, DIM, 1);
            const auto scores = [&](int t, int s) {   // one lane
                const uint32_t dq = sdesc(ptx::smem_u32(sm.q[t]), 16), dk = sdesc(ptx::smem_u32(sm.kv[s]), 16);
#pragma unroll
                for (int k = 0; k < DIM / 16; ++k) {
                    const uint32_t off = (k / 4) * (HALF >> 4) + (k % 4) * 2;
                    mma_ss(tmem + t * kN, dq + off, dk + off, id_s, k != 0);
                }
                commit(&sm.s_full[t]);
            };
            // The tensor pipe takes few instructions ahead, so what runs between two products is time that it stands still: no vote
            // on the outcome of a wait (3 to 7 % of a prompt of 1024 or more).  Lanes that differ about it (a wait that ran out) take the same
            // steps up to the next item all the same.
            const auto await = [&](uint64_t *b, uint32_t parity) {
                const bool r = wait(b, parity, sm, a.err);
                __syncwarp();
                return r;
            };
            Item it;
            int i = 0;                        // ring position of the item's first keys
            uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
            bool ok = true;
            while (__all_sync(~0u, ok) && next_item(it)) {
                const int nt[2] = {key_tiles(it, 0), key_tiles(it, 1)}, total = max(nt[0], nt[1]);
                if (total == 0) continue;
                const int tail_rows = it.nk - (total - 1) * kN;   // rows of the last key tile that are the request's (maybe more than kN)
                ok &= await(&sm.full[i % ST], (i / ST) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (nt[t] == 0) continue;
                    ok &= await(&sm.q_full[t], qn[t] & 1);
                    ++qn[t];
                    if (ok && lane == 0) {
                        fence_after();
                        scores(t, i % ST);
                        if (nt[t] == 1) commit(&sm.q_empty[t]);
                    }
                }
                if (ok && lane == 0) commit(&sm.empty[i % ST]);
                for (int j = 0; j < total; ++j) {
                    const int vi = i + 2 * j + 1, ki = vi + 1, vs = vi % ST, ks = ki % ST;
                    ok &= await(&sm.full[vs], (vi / ST) & 1);
                    if (j == total - 1 && tail_rows < kN) {
                        // values behind the request's last key: other rows, whatever they hold; 0 x NaN would reach this request
                        for (int x = tail_rows * 8 + lane; ok && x < kN * 8; x += 32)
                            for (int h = 0; h < HALVES; ++h)
                                *reinterpret_cast<uint4 *>(sm.kv[vs] + h * HALF + x * 16) = make_uint4(0, 0, 0, 0);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    if (j + 1 < total) ok &= await(&sm.full[ks], (ki / ST) & 1);
                    const uint32_t dv = sdesc(ptx::smem_u32(sm.kv[vs]), HALF);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j >= nt[t]) continue;
                        ok &= await(&sm.p_ready[t], pn[t] & 1);
                        ++pn[t];
                        if (ok && lane == 0) {
                            fence_after();
#pragma unroll
                            for (int k = 0; k < kN / 16; ++k)
                                mma_ts(tmem + 2 * kN + t * 128, tmem + t * kN + k * 8, dv + k * (2048 >> 4), id_o, j != 0 || k != 0);
                            if (j + 1 < nt[t]) {
                                scores(t, ks);
                                if (j + 2 == nt[t]) commit(&sm.q_empty[t]);
                            } else {
                                commit(&sm.o_full[t]);
                            }
                        }
                    }
                    if (ok && lane == 0) {
                        commit(&sm.empty[vs]);
                        if (j + 1 < total) commit(&sm.empty[ks]);
                    }
                }
                i += 2 * total;
            }
            if (lane == 0) {
                commit(&sm.drain);
                drain_wait(&sm.drain, 0);   // no product runs when the CTA goes
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;            // the warp's 32 lanes of tensor memory
        const uint32_t ts = tmem + t * kN + lanes, to = tmem + 2 * kN + t * 128 + lanes;
        const float c = fmaxf(a.scale * 1.4426950408889634f, 1e-37f), jump = kJump / c;
        Item it;
        uint32_t sn = 0, on = 0;
        const bool wide = (((uintptr_t)a.o | (uintptr_t)(a.ots * 2) | (uintptr_t)(a.ohs * 2)) & 31) == 0;
        bool ok = true;
        while (ok && next_item(it)) {
            const int nt = key_tiles(it, t), back = it.nk - it.nq;
            const int tok = it.tok0 + t * toks + (row >> lpk), hq = it.head + (row & (a.pk - 1));
            const bool mine = tok < it.nq;
            const int lim = min(back + tok, it.nk - 1);                      // last key this row sees
            const int least = min(back + it.tok0 + t * toks, it.nk - 1);     // of the tile's first row
            float m = -INFINITY, mc = -kShift, thr = -INFINITY, l = 0.f;
            for (int j = 0; j < nt; ++j, ++sn) {
                ok = wait(&sm.s_full[t], sn & 1, sm, a.err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                fence_after();
                // Scores of keys that some row does not see are masked where they are: the code of the other tiles stays small.
                if (j * kN + kN - 1 > least) {
                    const int from = lim - j * kN;
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        float s[32];
                        ld32(s, ts + ch * 32);
                        wait_ld();
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = ch * 32 + e > from ? 0xff800000u : __float_as_uint(s[e]);
                        st32(ts + ch * 32, w);
                    }
                    wait_st();
                }
                float x[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) ld32(x[ch], ts + ch * 32);
                wait_ld();
                float u[4];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    u[ch] = x[ch][0];
#pragma unroll
                    for (int e = 1; e < 31; e += 2) u[ch] = fmaxf(u[ch], fmaxf(x[ch][e], x[ch][e + 1]));
                    u[ch] = fmaxf(u[ch], x[ch][31]);
                }
                const float top = fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3]));
                const bool up = top > thr;
                if (__any_sync(~0u, up)) {
                    const float n = up ? top : m;
                    const float f = !up ? 1.f : m == -INFINITY ? 0.f : ex2((m - n) * c);
                    m = n;
                    mc = (n == -INFINITY ? 0.f : n * c) - kShift;
                    thr = n + jump;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int ch = 0; ch < DIM / 16; ++ch) {
                            float o[16];
                            ld16(o, to + ch * 16);
                            wait_ld();
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
                            st16(to + ch * 16, w);
                        }
                    }
                }
                // Weights, as a pipeline over the 64 pairs of the row: exponents two pairs ahead of the exponentials, sums and
                // packing four pairs behind them.
                const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
                float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
                float2 y[kN / 2];
                uint32_t p[16];
                constexpr int kAhead = 2, kLag = 4;
#pragma unroll
                for (int i = -kAhead; i < kN / 2 + kLag; ++i) {
                    const int n = i + kAhead, k = i - kLag;
                    if (n < kN / 2) y[n] = fma2(make_float2(x[n / 16][n % 16 * 2], x[n / 16][n % 16 * 2 + 1]), c2, mc2);
                    if (i >= 0 && i < kN / 2) y[i] = make_float2(ex2(y[i].x), ex2(y[i].y));
                    if (k >= 0) {
                        sum[k & 1] = add2(sum[k & 1], y[k]);
                        p[k % 16] = pack<BF>(y[k].x, y[k].y);
                        if (k % 16 == 15) st16(ts + k / 16 * 16, p);
                    }
                }
                l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sm.p_ready[t]);
            }
            if (ok && nt > 0) {
                ok = wait(&sm.o_full[t], on & 1, sm, a.err);
                ok = __all_sync(~0u, ok);
                ++on;
                fence_after();
            }
            if (!ok) break;
            const bool none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            H *out = reinterpret_cast<H *>(a.o) + (long long)(it.q0 + tok) * a.ots + (long long)hq * a.ohs;
#pragma unroll 1
            for (int ch = 0; ch < DIM / 32; ++ch) {
                float o[32];
                if (nt > 0) {
                    ld32(o, to + ch * 32);
                    wait_ld();
                }
                if (mine) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {   // a whole 32-byte sector at a time where rows lie so
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = none ? 0u : pack<BF>(o[16 * i + 2 * e] * inv, o[16 * i + 2 * e + 1] * inv);
                        H *at = out + ch * 32 + 16 * i;
                        if (wide) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), W8(w, 0) : "memory");
                        } else {
                            reinterpret_cast<uint4 *>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4 *>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            fence_before();   // the next item's products may write over these outputs
            if (a.lse && mine) a.lse[(size_t)(it.q0 + tok) * a.hq + hq] = none ? -INFINITY : 0.6931471805599453f * (mc + log2f(l));
        }
    }

    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// [tokens][heads][dim] rows as a 3D map with boxes of 64 dims x `heads` x `toks`, 128-byte swizzle.
int rows_map(CUtensorMap *m, const Rows &r, int dim, int heads, int T, int dtype, int box_heads, int box_toks) {
    // the stride of a dimension with one element is free
    const uint64_t ts = T > 1 ? (uint64_t)r.ts * 2 : 16, hs = heads > 1 ? (uint64_t)r.hs * 2 : 16;
    return make_tensor_map_3d(m, dtype == LORA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, r.p,
                              (uint64_t)dim, (uint64_t)heads, (uint64_t)(T > 0 ? T : 1), hs, ts, 64, box_heads, box_toks);
}

template <int DIM, bool BF>
int launch(const PromptArgs &a, cudaStream_t st) {
    KArgs k{};
    k.o = a.o.p; k.ots = a.o.ts; k.ohs = a.o.hs; k.lse = a.lse;
    k.cu_q = a.cu_q; k.cu_k = a.cu_k; k.Tq = a.Tq; k.Tk = a.Tk; k.R = a.R;
    k.hq = a.hq; k.G = a.hq / a.hkv; k.scale = a.scale; k.err = a.err; k.kv_len = a.kv_len;
    k.pk = k.G & -k.G;
    k.groups = a.hq / k.pk;
    const int pair = 2 * kM / k.pk;                                     // tokens of a CTA
    const long long items = ((long long)a.Tq / pair + a.R) * k.groups;  // at least the tile pairs of any row ranges
    if (items > INT32_MAX / 2) return LORA_ERR_TOO_LARGE;
    k.items = (uint32_t)items;
    Maps maps;
    // without keys nothing is loaded: any valid address serves
    const Rows kr = a.Tk > 0 ? a.k : a.q, vr = a.Tk > 0 ? a.v : a.q;
    if (int rc = rows_map(&maps.q, a.q, DIM, a.hq, a.Tq, a.dtype, k.pk, kM / k.pk)) return rc;
    if (int rc = rows_map(&maps.k, kr, DIM, a.hkv, a.Tk, a.dtype, 1, kN)) return rc;
    if (int rc = rows_map(&maps.v, vr, DIM, a.hkv, a.Tk, a.dtype, 1, kN)) return rc;
    const size_t smem = sizeof(Smem<DIM>) + 1024;
    static_assert(sizeof(Smem<DIM>) + 1024 <= 227 * 1024, "prompt kernel: shared memory beyond the per-block limit");
    static std::atomic<uint64_t> done{0};
    static_assert(kThreads * 168 == 128 * (88 + 2 * 208), "register split");
    int dev = 0, sms = 0;
    if (int rc = cuda_check(cudaGetDevice(&dev))) return rc;
    if (dev >= 64 || !(done.load() >> dev & 1)) {
        cudaFuncAttributes fa;
        if (int rc = cuda_check(cudaFuncGetAttributes(&fa, prompt_kernel<DIM, BF>))) return rc;
        // the row owners would wait for registers that the block does not have; build.py refuses such a build
        if (fa.numRegs != 168) return LORA_ERR_CUDA;
    }
    if (int rc = allow_smem(prompt_kernel<DIM, BF>, smem, done, dev)) return rc;
    if (int rc = cuda_check(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev))) return rc;
    prompt_kernel<DIM, BF><<<(int)(items < sms ? items : sms), kThreads, smem, st>>>(maps, k);
    count_launch();
    return cuda_check(cudaGetLastError());
}

}  // namespace

int launch_prompt(const PromptArgs &a, cudaStream_t st) {
    if (!tma_supported()) return LORA_ERR_CUDA;
    if (a.dim == 64) return a.dtype == LORA_BF16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
    return a.dtype == LORA_BF16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace lora
