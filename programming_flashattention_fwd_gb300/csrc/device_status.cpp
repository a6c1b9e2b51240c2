// device_status.cpp -- fa_device_status of include/fa.h: the watchdog words of every kernel.
#include <cstdint>

#include <cuda_runtime.h>

#include "bwd_internal.h"
#include "cache_internal.h"
#include "fa.h"
#include "fa_internal.h"

extern "C" {

int fa_device_status(fa_stream_t stream, uint32_t *detail)
{
    // every kernel's word is read and cleared; of those that are set the first in this order is reported
    uint32_t word[7] = {};
    if (fa::read_and_clear_status(reinterpret_cast<cudaStream_t>(stream), &word[0]) != cudaSuccess ||
        fa::read_and_clear_fa1_status(&word[1]) != cudaSuccess || fa::read_and_clear_gemm_status(&word[2]) != cudaSuccess ||
        fa::read_and_clear_softmax_status(&word[3]) != cudaSuccess || fa::cache::read_and_clear_tree_status(&word[4]) != cudaSuccess ||
        fa::cache::read_and_clear_weigh_status(&word[5]) != cudaSuccess || fa::bwd::read_and_clear_bwd_status(&word[6]) != cudaSuccess)
        return FA_ERR_NO_DEVICE;
    uint32_t w = word[0];
    for (uint32_t x : word)
        if (!(w & 1u)) w = x;
    if (detail) *detail = w;
    return (w & 1u) ? FA_ERR_DEVICE_TIMEOUT : FA_OK;
}

} // extern "C"
