// The values that 4-bit cache rows stand for, in bf16 or fp32.
#include <algorithm>

#include "kv4.cuh"

namespace sk {
namespace {

template <typename T> struct Out8;  // 8 values of a row

template <> struct Out8<__nv_bfloat16> {
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = ElemIO<__nv_bfloat16>::pack(f);
    }
};

template <> struct Out8<float> {
    __device__ __forceinline__ static void store(float* p, const float* f) {
        reinterpret_cast<uint4*>(p)[0] = ElemIO<float>::pack(f);
        reinterpret_cast<uint4*>(p)[1] = ElemIO<float>::pack(f + 4);
    }
};

// A thread has one word of 8 codes of a row (D / 8 words of K, then D / 8 of V, in the order
// of the dims, so that stores are contiguous) and goes from row to row: kUnroll rows with
// their loads in flight together, and no index arithmetic but two pointer steps.
constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_unpack_kernel(const uint8_t* __restrict__ rows, int64_t n_rows,
                                                              T* __restrict__ k, T* __restrict__ v) {
    constexpr int WPH = D / 8;                       // words per half
    constexpr int RPB = kThreads / (2 * WPH);        // rows a block handles at once
    const int c = threadIdx.x % WPH;
    const bool is_v = (threadIdx.x / WPH) & 1;
    const int word_at = (is_v ? kv4_half_bytes(D) : 0) + kv4_word_offset(D, c % 4, c / 4);
    const int par_at = (is_v ? kv4_half_bytes(D) : 0) + kv4_param_offset(D, c / 4);
    int64_t row = int64_t(blockIdx.x) * (RPB * kUnroll) + threadIdx.x / (2 * WPH);
    const int64_t step = int64_t(gridDim.x) * (RPB * kUnroll);
    const uint8_t* src = rows + row * kv4_row_bytes(D);
    T* dst = (is_v ? v : k) + row * D + c * 8;
    for (; row < n_rows; row += step, src += step * kv4_row_bytes(D), dst += step * D) {
        uint32_t word[kUnroll], par[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (row + u * RPB >= n_rows) break;
            word[u] = __ldcs(reinterpret_cast<const uint32_t*>(src + u * RPB * kv4_row_bytes(D) + word_at));
            par[u] = __ldcs(reinterpret_cast<const uint32_t*>(src + u * RPB * kv4_row_bytes(D) + par_at));
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (row + u * RPB >= n_rows) break;
            float f[8];
            kv4_decode_word(word[u], par[u], f);
            Out8<T>::store(dst + u * RPB * D, f);
        }
    }
}

template <typename T, int D>
cudaError_t launch_unpack(const void* rows, int64_t n_rows, void* k, void* v, cudaStream_t st) {
    constexpr int rows_per_block = kThreads / (D / 4) * kUnroll;
    const int64_t blocks = std::min<int64_t>((n_rows + rows_per_block - 1) / rows_per_block,
                                             int64_t(device_sm_count()) * 16);
    kv4_unpack_kernel<T, D><<<unsigned(blocks), kThreads, 0, st>>>(static_cast<const uint8_t*>(rows), n_rows,
                                                                   static_cast<T*>(k), static_cast<T*>(v));
    return cudaGetLastError();
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" sk_status sk_kv4_unpack(const void* rows, int64_t n_rows, int32_t head_dim, void* k, void* v,
                                   int32_t out_dtype, void* stream) {
    SK_RET_IF(n_rows < 0 || n_rows > (int64_t(1) << 48), SK_ERR_ARG);
    SK_RET_IF(head_dim != 64 && head_dim != 128, SK_ERR_UNSUPPORTED);
    SK_RET_IF(out_dtype != SK_BF16 && out_dtype != SK_F32, SK_ERR_UNSUPPORTED);
    if (n_rows == 0) return SK_OK;
    SK_RET_IF(rows == nullptr || k == nullptr || v == nullptr, SK_ERR_ARG);
    SK_RET_IF((reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) &
                  15u,
              SK_ERR_ARG);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (out_dtype == SK_BF16)
        e = head_dim == 64 ? launch_unpack<__nv_bfloat16, 64>(rows, n_rows, k, v, st)
                           : launch_unpack<__nv_bfloat16, 128>(rows, n_rows, k, v, st);
    else
        e = head_dim == 64 ? launch_unpack<float, 64>(rows, n_rows, k, v, st)
                           : launch_unpack<float, 128>(rows, n_rows, k, v, st);
    return e == cudaSuccess ? SK_OK : SK_ERR_CUDA;
}
