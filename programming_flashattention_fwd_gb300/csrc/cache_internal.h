// cache_internal.h -- declarations shared by the host API of the cache operators (cache_api.cpp)
// and their kernels.  Not part of the public ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache_schedule.h"

struct fa_cache;   // include/fa.h

namespace fa {
namespace cache {

// CTAs that a workspace has room for; a launch uses at most one per SM and at most this many.
constexpr int kMaxCtas = 160;
constexpr int kRowTile = 128;

// Launches a kernel that may be scheduled while the kernel before it on the stream drains; it waits on the
// device (grid_wait) before it touches memory.  Back to back this hides the launch and the kernel's start.
template <typename Kernel, typename... Args>
cudaError_t launch_overlapped(Kernel kern, dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Checks of a cache's own fields, and of the pointers of a non-empty one, shared by the entry points: FA_OK or the status code.
int check_cache(const fa_cache *c);
int check_cache_pointers(const fa_cache *c);

// Where the slots of a sequence are: slot s on row s % page of page table[b * max_pages + s / page]
// (page b * max_pages + s / page without a table).
struct Pages {
    const int32_t *table;
    int page, max_pages, num_pages;
};

// A cut unit, left by the CTA whose share starts with its first cut for whoever joins its parts.
struct Cut {
    int b, kvh, tile;   // which unit
    int parts;          // 0: nothing to join here
    int n;              // slots (weights) or drafted tokens (attention) of the sequence
    int pad[3];
};

struct TreeParams {
    TreeShape s;
    Pages pages;
    const int32_t *parent;   // [B, T] or null: token t follows t - 1
    const void *v_new;       // [B, Hkv, T, D], also read by the maps
    void *o;                 // [B, Hq, T, D]
    float *lse;              // [B, Hq, T]
    float *part_o;           // [2 * kMaxCtas][part_rows][D]
    float *part_lse;         // [2 * kMaxCtas][part_rows], log2 units
    Cut *cuts;               // [kMaxCtas]
    int part_rows;           // min(rows, tile)
    int q_panel, q_box;      // bytes of a 64-column panel of a query tile in shared memory, and of one copy into it
    int q_bufs;              // query tiles in flight
    int box_rows;            // rows of one copy: gcd(page, 128), at most BN
    float sl2;               // scale * log2 e
    uint64_t timeout_ns;     // limit of a wait (0: the default)
    uint32_t inject;         // fault injection: the first V tile is never loaded (bit 0: in every CTA, bit 1: in CTA 0); bit 2: no room
};

struct TreeMaps {
    CUtensorMap q, k, v, k_new, v_new;
};

int tree_log_keys(int D);                // log2 of the keys per step
int tree_tile(int D, long long rows);    // rows of a unit: 128, or 256 (two row tiles share K and V)
cudaError_t launch_tree(int D, bool bf16, const TreeMaps &m, const TreeParams &p, cudaStream_t st);
cudaError_t read_and_clear_tree_status(uint32_t *word);

// ---------------------------------------------------------------- accumulated attention weight
struct WeighParams {
    WeighShape s;
    Pages pages;
    const void *q;            // [B, Hq, T, D], read directly in kPath mode
    const float *lse;         // [B, Hq, T]
    const int32_t *path;      // [B, T] (kPath)
    const float *weight;      // [B, Hkv, capacity] or null: zero
    float *out;               // [B, Hkv, capacity]
    float *part;              // [2 * kMaxCtas][256]
    Cut *cuts;                // [kMaxCtas]
    int box_rows;
    float sl2;
    uint64_t timeout_ns;      // limit of a wait (0: the default)
    uint32_t inject;          // fault injection: the first K tile is never loaded (bit 0: in every CTA, bit 1: in CTA 0)
};

struct WeighMaps {
    CUtensorMap k, q;         // q: (D, rows of a plane, planes), not used in kPath mode
};

int weigh_rows(int D);        // query rows of a step
cudaError_t launch_weigh(int D, bool bf16, const WeighMaps &m, const WeighParams &p, cudaStream_t st);
cudaError_t read_and_clear_weigh_status(uint32_t *word);

// ---------------------------------------------------------------- writing the cache
struct AppendParams {
    Pages pages;
    uint4 *k, *v;                  // [num_pages, Hkv, page, D]
    const uint4 *k_new, *v_new;    // [B, Hkv, T, D]
    const int32_t *seq_len;        // [B]
    const int32_t *path, *count;   // [B, T], [B]; null: every token in order
    const int32_t *start;          // [B]: position of the first token written
    float *weight;                 // [B, Hkv, capacity] or null
    int32_t *pos;                  // [B, Hkv, capacity] or null
    int B, Hkv, T, capacity;
    int chunks;                    // 16-byte chunks of a row: D / 8
    int blocks_per_head;           // blocks over the T tokens of one (sequence, KV head)
};
cudaError_t launch_append(const AppendParams &p, int blocks, cudaStream_t st);
int append_tokens(int D);          // tokens of one block

// ---------------------------------------------------------------- eviction
struct EvictParams {
    Pages pages;
    uint4 *k, *v;                    // [num_pages, Hkv, page, D]
    const int32_t *seq_len;          // [B]
    const float *weight;             // [B, Hkv, capacity]
    const int32_t *pos;              // [B, Hkv, capacity]
    const int32_t *next_pos;         // [B] or null when last == 0
    float *weight_out;               // may be weight
    int32_t *pos_out;                // may be pos
    int32_t *new_len;                // [B]
    uint2 *from, *to;                // [B * Hkv][longest] (row, slot): slots that move, freed slots they move to
    int longest;                     // min(keep, capacity - keep)
    int B, Hkv, capacity, chunks;    // chunks: 16-byte chunks of a row
    int keep, first, last;
    int held, paged;                 // keys and page numbers of a CTA's slots held in shared memory
};
cudaError_t launch_evict(const EvictParams &p, cudaStream_t st);

} // namespace cache

} // namespace fa
