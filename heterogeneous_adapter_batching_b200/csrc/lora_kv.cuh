// Internal declarations of the KV-cache and attention calls: the cache format,
// row tensors and the launchers behind the entry points in lora_kv_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "lora_internal.cuh"

namespace lora {

// Bytes of the K half (equally the V half) of a granule: codes, then (step, low) pairs.
constexpr int kv_code_bytes(int dim) { return LORA_KV_GRANULE * dim / 2; }
constexpr int kv_half_bytes(int dim) { return kv_code_bytes(dim) + LORA_KV_GRANULE * 4 * (dim / LORA_KV_GROUP); }
constexpr int kv_granule_bytes(int dim) { return 2 * kv_half_bytes(dim); }
static_assert(kv_granule_bytes(128) == 2304 && kv_granule_bytes(64) == 1152, "granule size");

// A cache as kernels see it.
struct KvCache {
    unsigned char *pages;
    long long page_bytes;
    int num_pages, heads, block, granules;   // granules = block / LORA_KV_GRANULE
};

struct Rows {
    void *p;
    long long ts, hs;   // strides in elements
};

// Dynamic shared memory of a kernel, asked for once per device (bit d of `done`: device d has it).
template <class K>
inline int allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done, int dev) {
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return LORA_OK;
    if (int rc = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes))) return rc;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return LORA_OK;
}

struct LayoutArgs {
    const int32_t *past, *fresh_len, *req_ids;
    int R, T, block;
    int32_t *table;
    int max_blocks;
    const int32_t *free_pages;
    int num_free;
    const int32_t *free_head;
    int32_t *cu, *kv_len, *positions, *slots, *ids, *head_out, *err;
    const int32_t *held;   // null: a row holds the blocks of its past
    int32_t *held_out;
};
int launch_kv_layout(const LayoutArgs &a, cudaStream_t st);

struct RopeArgs {
    Rows q, k, v, qo, ko, vo;
    int hq, hk, hv;          // heads of each; hv > 0 only with a cache
    bool has_ko, has_vo;
    int T, dim, rot, interleaved;
    double mscale;
    const int32_t *positions;
    const float *freq;
    const int32_t *slots;    // null: no cache
    KvCache c;
    int32_t *err;
};
int launch_rope(const RopeArgs &a, int src, int dst, cudaStream_t st);

struct GatherKvArgs {
    KvCache c;
    int dim, T;
    const int32_t *slots;
    Rows ko, vo;
    bool has_k, has_v;
    int32_t *err;
};
int launch_kv_gather(const GatherKvArgs &a, int dst, cudaStream_t st);

struct AttendArgs {
    Rows q, o;
    int T, hq, dim, dtype;
    KvCache c;
    const int32_t *table;
    int max_blocks;
    const int32_t *cu_q, *kv_len;
    int R, max_q;
    float scale;
    float *lse;
    void *ws;
    int32_t *err;
    int group;              // q heads of a kv head
    uint32_t inv_group;     // 65536 / group + 1
};
size_t attend_workspace(int hq, int hkv, int dim, int max_q);
int launch_kv_attend(const AttendArgs &a, cudaStream_t st);

struct PromptArgs {
    Rows q, k, v, o;
    int Tq, Tk, hq, hkv, dim, dtype;
    const int32_t *cu_q, *cu_k;
    int R;
    float scale;
    float *lse;
    int32_t *err;
    const int32_t *kv_len;   // may be null
};
int launch_prompt(const PromptArgs &a, cudaStream_t st);

}  // namespace lora
