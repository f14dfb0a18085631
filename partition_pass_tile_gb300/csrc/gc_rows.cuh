// gc_rows.cuh -- device building blocks of the row operators (experts.cu,
// embedding.cu, sample.cu): element types, pieces of 2 to 16 bytes of a row
// with their float32 values, and ids of either width.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace gcd {

__device__ __forceinline__ float row_to_float(float x) { return x; }
__device__ __forceinline__ float row_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float row_to_float(__half x) { return __half2float(x); }

// One rounding, to nearest even.
template <class T>
__device__ __forceinline__ T row_from_float(float x);
template <>
__device__ __forceinline__ float row_from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 row_from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half row_from_float<__half>(float x) { return __float2half_rn(x); }

// Pieces of a row that a thread has under way at a time where they are narrow:
// rows of odd width move in pieces of 2 or 4 bytes.  One at a time, combine of
// 8192 x 8 pairs of 2047 bf16 takes 125 us, four at a time 96 (rows of 2048: 61).
template <class T, int N>
constexpr int kNarrow = sizeof(T) * N >= 16 ? 1 : sizeof(T) * N == 8 ? 2 : 4;

// N consecutive elements of a row, loaded and stored as one access of
// sizeof(Piece) bytes; the address is a multiple of that.
template <class T, int N>
struct alignas(sizeof(T) * N) Piece {
    T v[N];
};

template <class T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T *p)
{
    return *reinterpret_cast<const Piece<T, N> *>(p);
}

template <class T, int N>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, N> &x)
{
    *reinterpret_cast<Piece<T, N> *>(p) = x;
}

// A store of a row that is not read again soon: the lines leave L2 first.
template <class T, int N>
__device__ __forceinline__ void stream_piece(T *p, const Piece<T, N> &x)
{
    if constexpr (sizeof(Piece<T, N>) == 16) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&x));
    else store_piece<T, N>(p, x);
}

template <class T, int N>
__device__ __forceinline__ Piece<T, N> zero_piece()
{
    Piece<T, N> z;
#pragma unroll
    for (int i = 0; i < N; ++i) z.v[i] = row_from_float<T>(0.0f);
    return z;
}

// Id i of an int32 or int64 array; any value outside [0, limit) becomes limit
// (limit <= 2^31 - 1).
__device__ __forceinline__ uint32_t load_id(const void *ids, bool wide, uint64_t i, uint32_t limit)
{
    const int64_t v = wide ? static_cast<const int64_t *>(ids)[i]
                           : int64_t(static_cast<const int32_t *>(ids)[i]);
    return v >= 0 && v < int64_t(limit) ? uint32_t(v) : limit;
}

// Zeros over `bytes` of a row by one warp, whatever its alignment: 16 bytes at
// a time between the boundaries, two outside them.
__device__ __forceinline__ void zero_row(void *row, size_t bytes)
{
    uint8_t *p = static_cast<uint8_t *>(row);
    const uint32_t lane = threadIdx.x & 31;
    const size_t lead = size_t(-reinterpret_cast<intptr_t>(p)) & 15u, head = lead < bytes ? lead : bytes;
    const size_t body = (bytes - head) / 16, tail = head + body * 16;
    if (lane < head / 2) reinterpret_cast<uint16_t *>(p)[lane] = 0;
    for (size_t i = lane; i < body; i += 32) reinterpret_cast<uint4 *>(p + head)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lane < (bytes - tail) / 2) reinterpret_cast<uint16_t *>(p + tail)[lane] = 0;
}

// Programmatic launches: a kernel launched by launch_next may start while the
// one before it in the stream still runs.  Each kernel of such a chain lets
// its successor start at once and touches nothing that its predecessor writes
// (or reads, if it writes it) before chain_wait, which returns when the
// predecessor has finished.
__device__ __forceinline__ void chain_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace gcd

namespace gch {

template <class... P, class... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Elements per access for rows of `elem`-byte elements: the largest piece of
// at most 16 bytes that divides every address and length in `bits` (the
// bitwise or of pointers, stride bytes and width bytes).
inline int piece_elems(uint64_t bits, int elem)
{
    int bytes = 16;
    while (bytes > elem && (bits & uint64_t(bytes - 1)) != 0) bytes >>= 1;
    return bytes / elem;
}

}  // namespace gch
