// spx_error.cpp -- the device-side errors of every kernel, read as one status.
// A source of its own: a new kernel's error word then changes no other
// kernel's source, whose hash the recorded DRAM traffic is kept by.
#include <cuda_runtime.h>

#include "spx_internal.h"

extern "C" spx_status spx_last_device_error(spx_stream_t stream) {
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SPX_ERR_CUDA;
    const int timed[] = {spx_bsr_error_take(), spx_wcsr_error_take(), spx_experts_error_take()};
    const int coo = spx_coo_error_take();
    // the checked build's index errors (always 0 in the product build, which reads no word for them)
    const int checked[] = {spx_bsr_check_take(), spx_spmv_check_take(), spx_spmm_check_take(), spx_sell_check_take(),
                           spx_wcsr_check_take(), spx_bsrg_check_take(), spx_route_check_take(), spx_experts_check_take(),
                           spx_experts_simt_check_take(), spx_int8_check_take()};
    for (int c : timed)
        if (c == SPX_ERR_TIMEOUT) return SPX_ERR_TIMEOUT;
    for (int c : timed)
        if (c) return SPX_ERR_CUDA;
    for (int c : checked)
        if (c == SPX_ERR_CUDA) return SPX_ERR_CUDA;
    if (coo) return static_cast<spx_status>(coo);
    for (int c : checked)
        if (c) return static_cast<spx_status>(c);
    return SPX_OK;
}
