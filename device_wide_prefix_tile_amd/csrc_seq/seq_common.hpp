// Shared pieces of the sequence operators: element types, 16-byte vectors of
// them, activations, and host-side checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "dwpt_seq.h"
#include "seq_plan.hpp"

namespace dwpt_seq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

using bf16 = __bf16;
using f16 = _Float16;

// V consecutive elements of T, moved with the widest access that V * sizeof(T) allows.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float (&f)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)p.v[i];
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V])
{
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = (T)f[i];  // round to nearest even
    return p;
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p)
{
    return *reinterpret_cast<const Pack<T, V>*>(p);
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack()
{
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = (T)0.0f;
    return p;
}

// Hides from the compiler that p is what it was, so that values made of it earlier are made again
// instead of being kept in registers.
template <typename P>
__device__ __forceinline__ void opaque(P& p)
{
    u32x4 v = __builtin_bit_cast(u32x4, p);
    asm volatile("" : "+v"(v));
    p = __builtin_bit_cast(P, v);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 2^x and 1/x by the hardware instructions (1 ulp; results below 2^-126 flush to zero).
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-u): e^-u overflows to infinity for u < -88, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid(float u) { return rcp_fast(1.0f + exp2_fast(-kLog2e * u)); }
// u * sigmoid(u) is 0 * -inf at u = -inf, as in the definition.
__device__ __forceinline__ float silu(float u) { return u * sigmoid(u); }

// softplus(v) = ln(1 + e^v).  With e = e^v rounded into w = 1 + e, ln(w) * e / (w - 1) undoes the
// rounding of the sum (w - 1 is exact): the result keeps its relative accuracy where e is far
// below 1, which is where the steps of a state-space scan lie.  Above 20, ln(1 + e^v) - v < 2.1e-9,
// less than half a unit in the last place of v.
__device__ __forceinline__ float softplus(float v)
{
    const float e = exp2_fast(kLog2e * v);
    const float w = 1.0f + e;
    const float d = w - 1.0f;
    const float l = __builtin_amdgcn_logf(w) * kLn2;  // log2
    const float r = d == 0.0f ? e : l * (e * rcp_fast(d));
    return v > 20.0f ? v : r;
}

// Value of another lane of the quad (4 consecutive lanes): CTRL 0xB1 exchanges lanes 0-1 and 2-3,
// 0x4E lanes 0-2 and 1-3.
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowRor4 = 0x124, kRowRor8 = 0x128;

__device__ __forceinline__ float quad_sum(float v)
{
    v += dpp<kQuadXor1>(v);
    return v + dpp<kQuadXor2>(v);
}

// Orders one wavefront's LDS accesses: a lane's reads after this see every lane's writes before
// it (the wavefront's LDS instructions execute in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Exclusive prefix of v over the WAVES wavefronts of a workgroup, and the sum, in an order that depends on the threads
// alone.  part: WAVES values in LDS that nothing else reads or writes until the next barrier behind.
template <int WAVES, typename N>
__device__ __forceinline__ N block_prefix(N v, N* part, N& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    N incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const N t = __shfl_up(incl, o, 64);
        if (lane >= o) incl += t;
    }
    const N excl = __shfl_up(incl, 1, 64);
    if (lane == 63) part[w] = incl;
    __syncthreads();
    N before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
        before = q < w ? before + part[q] : before;
        all += part[q];
    }
    total = all;
    return lane ? before + excl : before;
}

// A launch's workgroups are numbered over two dimensions of the grid, kGridWidth in a row: HIP takes
// less than 2^32 work items along one.  The last row may hold numbers behind the last workgroup.
constexpr uint32_t kGridWidth = 1u << 22;
__device__ __forceinline__ uint32_t workgroup() { return blockIdx.y * kGridWidth + blockIdx.x; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ------------------------------------------------------------ host side
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t dtype_size(int dt) { return dt == SEQ_F32 ? 4 : 2; }
inline bool valid_dtype(int dt) { return dt == SEQ_F32 || dt == SEQ_F16 || dt == SEQ_BF16; }
inline size_t round_up(size_t n, size_t a) { return (n + a - 1) / a * a; }

// The memory of `rows` rows of `width` elements, `stride` elements apart.
struct Range {
    const void* p;
    size_t rows, stride, width;  // the last two in bytes
};
inline Range range(const void* p, uint64_t rows, int64_t stride, uint64_t width, size_t es)
{
    return Range{p, (size_t)rows, (size_t)stride * es, (size_t)width * es};
}
inline Range range(const void* p, uint64_t bytes) { return Range{p, 1, (size_t)bytes, (size_t)bytes}; }

// Whether two ranges share a byte.  Rows of one stride may lie beside one another, as the halves
// of one array do; of other rows that interleave, it is assumed that they do.
inline bool overlap(const Range& a, const Range& b)
{
    if (!a.p || !b.p || !a.rows || !b.rows || !a.width || !b.width) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + (a.rows - 1) * a.stride + a.width, b1 = b0 + (b.rows - 1) * b.stride + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.stride == b.stride && a.rows > 1 && b.rows > 1) {
        const size_t apart = b0 >= a0 ? (b0 - a0) % a.stride : (a.stride - (a0 - b0) % a.stride) % a.stride;
        return apart < a.width || apart + b.width > a.stride;
    }
    return true;
}
// Whether one of the outputs overlaps an input or another output.
template <size_t NO, size_t NI>
bool any_overlap(const Range (&out)[NO], const Range (&in)[NI])
{
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

// Rows at p, `stride` elements apart.
struct Array {
    const void* p;
    int64_t stride;
};
inline bool valid_rows(int dtype, uint64_t rows, uint32_t width, const Array& a)
{
    if (rows == 0) return true;
    return a.p && aligned(a.p, dtype_size(dtype)) && a.stride >= (int64_t)width && a.stride <= ((int64_t)1 << 31);
}

// The grid of `workgroups` (of 256 lanes or fewer) for workgroup(); more of them than kMostInGrid
// would need arrays larger than a card's memory.
constexpr uint64_t kMostInGrid = 0x7FFFFFFF;
inline dim3 grid_of(uint64_t workgroups)
{
    return dim3((unsigned)std::min<uint64_t>(workgroups, kGridWidth), (unsigned)((workgroups + kGridWidth - 1) / kGridWidth));
}

inline scan_status_t launched() { return hipGetLastError() == hipSuccess ? SCAN_OK : SCAN_ERR_HIP; }

// Calls f with a value of the element type of dt.
template <class F>
scan_status_t with_dtype(int dt, F f)
{
    switch (dt) {
        case SEQ_F32: return f((float)0);
        case SEQ_F16: return f((f16)0);
        case SEQ_BF16: return f((bf16)0);
    }
    return SCAN_ERR_UNSUPPORTED;
}

}  // namespace dwpt_seq
