// Host entry points of decode attention over 4-bit caches (decode4.cu), for decode.cu.
#pragma once

#include "common.cuh"

namespace sk {

// Arguments of one call; the layer is contiguous (ring / global) or paged.
struct Kv4DecodeArgs {
    const sk_kv_layer* layer;        // or null
    const sk_paged_layer* paged;     // or null
    const void* q;
    const float* sink_logits;
    void* out;
    void* ws;
    int nrep, io_dtype;
};

// Workspace bytes; 0: an unsupported head_dim or number of q heads per kv head.
size_t kv4_decode_workspace(int batch, int n_kv_heads, int head_dim, int nrep);

// False: unsupported.  *e is the launch's result.
bool kv4_decode_run(const Kv4DecodeArgs& a, cudaStream_t st, cudaError_t* e);

}  // namespace sk
