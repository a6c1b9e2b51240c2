// rotary_internal.h -- declarations shared by the host API of the rotary operators (rotary_api.cpp) and their
// kernel.  Not part of the public ABI.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_internal.h"
#include "fa_internal.h"

namespace fa {
namespace rotary {

// Heads that are read from one view and written to another: element e of head h of token t of sequence b is at
// b * *b + h * *h + t * *t + e.  y null: only written to the cache.
struct Segment {
    const void *x;
    void *y;
    long long xb, xh, xt, yb, yh, yt;
    int end;        // heads of this and the earlier segments
    int turned;     // rotated, or laid out anew as they are
    int pool;       // 0: none, 1: keys, 2: values go to the cache
};

struct Params {
    Segment seg[3];
    const uint64_t *freq;     // [rot / 2] 2^64 turns a position
    const int32_t *start;     // [B] or null
    const int32_t *position;  // [B, T] or null
    float amplitude, sign;    // sign -1: the inverse rotation
    int B, T, D, rot, interleaved;
    int heads, per;           // all heads; heads of a thread
    FastDiv f_T;
    // the cache (fa_rotary_append)
    cache::Pages pages;
    void *k, *v;
    const int32_t *seq_len, *count;
    float *weight;
    int32_t *pos;
    int Hkv, capacity;
};

cudaError_t launch_rotary(const Params &p, bool bf16, bool append, cudaStream_t st);

} // namespace rotary
} // namespace fa
