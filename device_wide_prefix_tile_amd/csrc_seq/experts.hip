// Tokens sorted by expert and back, with weights applied, and the gradients.
//
// Split: the choices (token by token, `choices` experts each) are grouped by expert, in ascending order
// within an expert: a stable split, as radix_split's, by the whole expert number.  A wavefront ranks 64
// choices at a time: the lanes that hold one expert are found by a ballot for each bit of the number, and
// a count per (wavefront, expert) in LDS carries on from round to round.  Up to kChunk choices that is one
// launch of one workgroup; above, a first launch ranks every chunk's choices within the chunk and leaves its
// counts in memory, a second adds what comes before (with many chunks, prefixes of the counts
// are made in between).
//
// Moves: dispatch reads a token's row once and writes it to its choices' places; combine reads the rows at a
// token's places and adds them up in the order of the choices; combine's gradient does both at once, with
// the product sums that are the weights' gradients.  All three are HBM-bound.
#include <initializer_list>
#include <utility>

#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr uint32_t kMaxChannels = 1u << 20;
constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxChoices = 256;

// ------------------------------------------------------------ split
constexpr int kBlock = 1024;
constexpr int kWaves = kBlock / 64;
constexpr int kRounds = 4;
constexpr uint32_t kChunk = kBlock * kRounds;
// More chunks than this: prefixes of the counts by a launch of its own, else every workgroup of the second launch adds up all
// counts.  With / without that launch, us: 16 chunks of 128 experts 11.8 / 10.0, 64 of 128 13.9 / 12.9, 128 of 256 17.2 /
// 18.5, 256 of 256 22.3 / 26.9.
constexpr uint32_t kFewChunks = 64;

struct SplitPlan {
    uint32_t n, experts, bits, chunks;
};

SplitPlan make_plan(size_t n, uint32_t experts)
{
    SplitPlan p{(uint32_t)n, experts, 0, (uint32_t)std::max<size_t>(1, (n + kChunk - 1) / kChunk)};
    while ((1u << p.bits) < experts) ++p.bits;
    return p;
}

// Chunk blockIdx.x.  ONE: the only chunk, everything.  Otherwise places receives every choice's rank among its
// chunk's choices of the same expert, counts[chunk] how many choices each expert has there.
template <bool ONE>
__global__ __launch_bounds__(kBlock) void rank_kernel(const int32_t* __restrict__ experts, SplitPlan p, int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ places, int32_t* __restrict__ source,
                                                      uint32_t* __restrict__ counts)
{
    extern __shared__ uint32_t s_cnt[];  // [wavefront][experts]
    __shared__ uint32_t s_part[kWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (uint32_t i = threadIdx.x; i < kWaves * p.experts; i += kBlock) s_cnt[i] = 0;
    // wavefront w owns choices [first, first + 64 kRounds) of the chunk
    const uint32_t first = blockIdx.x * kChunk + (uint32_t)(w * 64 * kRounds) + lane;
    uint32_t e[kRounds], rank[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = first + u * 64;
        e[u] = i < p.n ? (uint32_t)experts[i] : 0xFFFFFFFFu;
    }
    __syncthreads();
    uint32_t* my = s_cnt + (uint32_t)w * p.experts;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const bool in = e[u] < p.experts;
        uint64_t same = __builtin_amdgcn_ballot_w64(in);
        for (uint32_t b = 0; b < p.bits; ++b) {
            const bool one = e[u] >> b & 1;
            const uint64_t ones = __builtin_amdgcn_ballot_w64(one);
            same &= one ? ones : ~ones;
        }
        rank[u] = 0;
        if (in) rank[u] = my[e[u]] + (uint32_t)__builtin_popcountll(same & below);
        wave_sync();  // every lane has read the count
        if (in && (same >> lane) == 1) my[e[u]] = rank[u] + 1;  // the last of them
        wave_sync();
    }
    __syncthreads();

    // thread t < experts (1024 at most): the wavefronts' counts of expert t become their first ranks
    uint32_t sum = 0;
    if (threadIdx.x < p.experts) {
        for (int q = 0; q < kWaves; ++q) {
            const uint32_t c = s_cnt[q * p.experts + threadIdx.x];
            s_cnt[q * p.experts + threadIdx.x] = sum;
            sum += c;
        }
    }
    if (ONE) {
        uint32_t total;
        const uint32_t begin = block_prefix<kWaves>(sum, s_part, total);
        if (threadIdx.x < p.experts) {
            for (int q = 0; q < kWaves; ++q) s_cnt[q * p.experts + threadIdx.x] += begin;
            offsets[threadIdx.x] = (int32_t)begin;
        }
        if (threadIdx.x == 0) offsets[p.experts] = (int32_t)total;
        for (uint32_t i = total + threadIdx.x; i < p.n; i += kBlock) source[i] = -1;
    } else if (threadIdx.x < p.experts) {
        counts[(size_t)blockIdx.x * p.experts + threadIdx.x] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = first + u * 64;
        if (i >= p.n) continue;
        const bool in = e[u] < p.experts;
        const uint32_t at = in ? my[e[u]] + rank[u] : 0xFFFFFFFFu;
        places[i] = (int32_t)at;
        if (ONE && in) source[at] = (int32_t)i;
    }
}

// counts[chunk][expert] becomes the sum over the chunks before; totals[expert] the sum over all.  Workgroup x
// has the experts from 64 x on, each wavefront a run of the chunks.
__global__ __launch_bounds__(kBlock) void prefix_kernel(SplitPlan p, uint32_t* __restrict__ counts, uint32_t* __restrict__ totals)
{
    __shared__ uint32_t s_sum[kWaves][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint32_t e = blockIdx.x * 64 + lane, run = (p.chunks + kWaves - 1) / kWaves;
    const uint32_t lo = min((uint32_t)w * run, p.chunks), hi = min(lo + run, p.chunks);
    uint32_t sum = 0;
    if (e < p.experts)
        for (uint32_t c = lo; c < hi; ++c) sum += counts[(size_t)c * p.experts + e];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (e >= p.experts) return;
    uint32_t at = 0;
    for (int q = 0; q < w; ++q) at += s_sum[q][lane];
    for (uint32_t c = lo; c < hi; ++c) {
        uint32_t* q = counts + (size_t)c * p.experts + e;
        const uint32_t had = *q;
        *q = at;
        at += had;
    }
    if (w == kWaves - 1) totals[e] = at;
}

// Ranks within chunk blockIdx.x become places.  FEW: counts as rank_kernel left them, else prefixes and totals.
template <bool FEW>
__global__ __launch_bounds__(kBlock) void place_kernel(const int32_t* __restrict__ experts, SplitPlan p,
                                                       const uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals,
                                                       int32_t* __restrict__ offsets, int32_t* places, int32_t* __restrict__ source)
{
    __shared__ uint32_t s_base[kMaxExperts], s_part[kWaves];
    const uint32_t t = threadIdx.x;
    uint32_t e[kRounds], rank[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = min(blockIdx.x * kChunk + u * kBlock + t, p.n - 1);
        e[u] = (uint32_t)experts[i];
        rank[u] = (uint32_t)places[i];
    }
    uint32_t before = 0, sum = 0;  // of expert t: in the chunks before this one, in all
    if (t < p.experts) {
        if (FEW) {
            // eight loads in flight together
            for (uint32_t c0 = 0; c0 < p.chunks; c0 += 8) {
                uint32_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = counts[(size_t)min(c0 + u, p.chunks - 1) * p.experts + t];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t n = c0 + u < p.chunks ? v[u] : 0u;
                    before += c0 + u < blockIdx.x ? n : 0u;
                    sum += n;
                }
            }
        } else {
            before = counts[(size_t)blockIdx.x * p.experts + t];
            sum = totals[t];
        }
    }
    uint32_t total;
    const uint32_t begin = block_prefix<kWaves>(sum, s_part, total);
    if (t < p.experts) {
        s_base[t] = begin + before;
        if (blockIdx.x == 0) offsets[t] = (int32_t)begin;
    }
    if (blockIdx.x == 0 && t == 0) offsets[p.experts] = (int32_t)total;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const uint32_t i = blockIdx.x * kChunk + u * kBlock + t;
        if (i >= p.n) break;
        if (e[u] < p.experts) {
            const uint32_t at = s_base[e[u]] + rank[u];
            places[i] = (int32_t)at;
            source[at] = (int32_t)i;
        }
        if (i >= total) source[i] = -1;
    }
}

// ------------------------------------------------------------ moves
// What a pass works on: `tokens` rows outside, `rows` rows in the experts' order, places between them.
struct Moves {
    const int32_t* places;
    uint32_t tokens, rows, choices, channels;
};

// The place of choice j of token t; -1 if there is none in the array.
__device__ __forceinline__ int place_of(const Moves& m, uint32_t t, uint32_t j)
{
    const int at = uniform(m.places[(uint64_t)t * m.choices + j]);
    return at >= 0 && (uint32_t)at < m.rows ? at : -1;
}

template <typename T, int V>
__device__ __forceinline__ void store_stream(T* out, const Pack<T, V>& p)
{
    if constexpr (sizeof(p) == 16)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, p), reinterpret_cast<u32x4*>(out));
    else
        *reinterpret_cast<Pack<T, V>*>(out) = p;
}

// A row of the experts' order is read once.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_stream(const T* p)
{
    if constexpr (sizeof(Pack<T, V>) == 16)
        return __builtin_bit_cast(Pack<T, V>, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
    else
        return load_pack<T, V>(p);
}

// Which rows are cleared before a move fills those that a place leads to: from *used on, or all (used NULL).  Rows that
// `source` shows to be led to are left out: the move writes them.
struct Clear {
    const int32_t *used, *source;
    uint32_t source_rows;
};

// A workgroup looks at kClearRows rows and sets 64 V kClearParts channels of them to zero, a wavefront every fourth row.
// It runs in front of the move, so a row that is cleared although a place leads to it (a source of another origin) is
// written afterwards.  A map of the rows that are led to would need memory; this needs the launch (2.4 us for 512 rows,
// 5.3 for 65536), and writes no more than the rows without a choice where source is the split's.
constexpr int kClearRows = 16;
constexpr int kClearParts = 8;
template <typename T, int V>
__global__ __launch_bounds__(256) void clear_kernel(Moves m, Clear c, uint32_t chunks, T* __restrict__ out, int64_t stride)
{
    const uint32_t wg = workgroup();
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint64_t r0 = (uint64_t)(wg / chunks) * kClearRows, r = r0 + (uint32_t)lane;
    if (r0 >= m.rows) return;
    bool empty = lane < kClearRows && r < m.rows;
    if (empty && c.used) empty = (int64_t)r >= (int64_t)*c.used;
    if (empty && r < c.source_rows) {
        const int i = c.source[r];
        empty = i < 0 || (uint32_t)i >= m.tokens * m.choices || m.places[i] != (int)r;
    }
    const uint32_t c0 = (wg % chunks * (64 * kClearParts) + (uint32_t)lane) * V;
    int n = w;
    for (uint64_t rows = __builtin_amdgcn_ballot_w64(empty); rows; rows &= rows - 1) {
        if (n++ % 4) continue;
        T* row = out + (int64_t)(r0 + (uint32_t)__builtin_ctzll(rows)) * stride;
#pragma unroll
        for (int u = 0; u < kClearParts; ++u) {
            const uint32_t at = c0 + u * 64 * V;
            if (at < m.channels) *reinterpret_cast<Pack<T, V>*>(row + at) = zero_pack<T, V>();
        }
    }
}

// A wavefront copies 64 V kCopies channels of a token to the token's places.  8192 tokens to 8 places of 2048 bfloat16
// channels 52 us (5.8 TB/s), to 4 of 4096, the same ones
// every time, with 2 / 4 / 8 copies 51 / 55 / 60 us.
constexpr int kCopies = 2;
template <typename T, int V>
__global__ __launch_bounds__(256) void dispatch_kernel(Moves m, uint32_t chunks, const T* __restrict__ x, int64_t x_stride,
                                                       T* __restrict__ out, int64_t out_stride)
{
    const uint64_t unit = (uint64_t)workgroup() * 4 + (uint32_t)uniform((int)(threadIdx.x >> 6));
    const uint64_t t = unit / chunks;
    if (t >= m.tokens) return;
    const uint32_t c0 = (uint32_t)(unit % chunks * 64 * kCopies + (threadIdx.x & 63)) * V;
    Pack<T, V> p[kCopies];
#pragma unroll
    for (int u = 0; u < kCopies; ++u) {
        const uint32_t c = c0 + u * 64 * V;
        p[u] = c < m.channels ? load_pack<T, V>(x + (int64_t)t * x_stride + c) : zero_pack<T, V>();
    }
    for (uint32_t j = 0; j < m.choices; ++j) {
        const int at = place_of(m, (uint32_t)t, j);
        if (at < 0) continue;
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
            const uint32_t c = c0 + u * 64 * V;
            if (c < m.channels) store_stream<T, V>(out + (int64_t)at * out_stride + c, p[u]);
        }
    }
}

// A wavefront adds up 64 V channels of a token's rows; the loads of kAhead of them are in flight together.  HBM-bound: 8192
// x 8 x 2048 bfloat16 50 us (6.0 TB/s) with 4 or 8 ahead; 16000 x 4 x 590, two channels per access, 29 and 33 us, its
// gradient 46 and 65 (places that are not there are still looked at).
constexpr int kAhead = 4;
template <typename T, typename W, int V>
__global__ __launch_bounds__(256) void combine_kernel(Moves m, uint32_t chunks, const W* __restrict__ weights, const T* __restrict__ y,
                                                      int64_t y_stride, T* __restrict__ out, int64_t out_stride)
{
    const uint64_t unit = (uint64_t)workgroup() * 4 + (uint32_t)uniform((int)(threadIdx.x >> 6));
    const uint64_t t = unit / chunks;
    const uint32_t c = (uint32_t)(unit % chunks * 64 + (threadIdx.x & 63)) * V;
    if (t >= m.tokens || c >= m.channels) return;
    float acc[V] = {};
    for (uint32_t j0 = 0; j0 < m.choices; j0 += kAhead) {
        Pack<T, V> p[kAhead];
        int at[kAhead];
        float w[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            at[u] = j0 + u < m.choices ? place_of(m, (uint32_t)t, j0 + u) : -1;
            w[u] = weights && at[u] >= 0 ? (float)weights[t * m.choices + j0 + u] : 1.0f;
            if (at[u] >= 0) p[u] = load_stream<T, V>(y + (int64_t)at[u] * y_stride + c);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (at[u] < 0) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = fmaf(w[u], (float)p[u].v[k], acc[k]);
        }
    }
    store_stream<T, V>(out + (int64_t)t * out_stride + c, pack<T, V>(acc));
}

// One workgroup per token: dy at the token's places is its weight times dout, the weight's gradient the product
// sum of dout and y.  8192 x 4 x 4096 bfloat16: 107 us, 5.6 TB/s.
template <typename T, typename W, int V>
__global__ __launch_bounds__(256) void combine_grad_kernel(Moves m, const W* __restrict__ weights, const T* __restrict__ dout,
                                                           int64_t dout_stride, const T* __restrict__ y, int64_t y_stride,
                                                           T* __restrict__ dy, int64_t dy_stride, float* __restrict__ dweights)
{
    __shared__ float s_sum[4][kAhead];
    const uint32_t t = workgroup();
    if (t >= m.tokens) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (uint32_t j0 = 0; j0 < m.choices; j0 += kAhead) {
        int at[kAhead];
        float weight[kAhead], sum[kAhead] = {};
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            at[u] = j0 + u < m.choices ? place_of(m, t, j0 + u) : -1;
            weight[u] = weights && at[u] >= 0 ? (float)weights[(uint64_t)t * m.choices + j0 + u] : 1.0f;
        }
        for (uint32_t c = threadIdx.x * V; c < m.channels; c += 256 * V) {
            Pack<T, V> p[kAhead];
            float g[V];
            const Pack<T, V> d = load_pack<T, V>(dout + (int64_t)t * dout_stride + c);
            if (dweights) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (at[u] >= 0) p[u] = load_stream<T, V>(y + (int64_t)at[u] * y_stride + c);
            }
            unpack(d, g);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (at[u] < 0) continue;
                float out[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    out[k] = weight[u] * g[k];
                    asm("" : "+v"(out[k]));  // rounded to 32 bits first in every type: float16 has a fused product and rounding
                    if (dweights) sum[u] = fmaf(g[k], (float)p[u].v[k], sum[u]);
                }
                store_stream<T, V>(dy + (int64_t)at[u] * dy_stride + c, pack<T, V>(out));
            }
        }
        if (!dweights) continue;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) sum[u] += __shfl_xor(sum[u], o, 64);
        }
        __syncthreads();
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) s_sum[w][u] = sum[u];
        }
        __syncthreads();
        if (threadIdx.x < kAhead && j0 + threadIdx.x < m.choices) {
            float all = s_sum[0][threadIdx.x];
            for (int q = 1; q < 4; ++q) all += s_sum[q][threadIdx.x];
            dweights[(uint64_t)t * m.choices + j0 + threadIdx.x] = all;
        }
    }
}

// ------------------------------------------------------------ host side
// Calls f with the elements per access as an integral constant: the most of 16 bytes, two elements and one element
// that every row can be cut into.  Two / one: combine of 1999 x 2 rows of 1002 float32 7.5 / 11.8 us, of 16000 x 4 of 590
// bfloat16 33 / 55 (with eight rows ahead).
template <typename T, typename F>
void with_pack(uint32_t channels, std::initializer_list<Array> arrays, F f)
{
    const auto fits = [&](int v) {
        bool ok = channels % v == 0;
        for (const Array& a : arrays) ok = ok && (!a.p || (a.stride % v == 0 && aligned(a.p, v * sizeof(T))));
        return ok;
    };
    constexpr int V = 16 / sizeof(T);
    if (fits(V))
        f(std::integral_constant<int, V>());
    else if (fits(2))
        f(std::integral_constant<int, 2>());
    else
        f(std::integral_constant<int, 1>());
}

scan_status_t check_moves(int dtype, uint64_t tokens, uint64_t rows, uint32_t choices, uint32_t channels, const int32_t* places)
{
    if (!valid_dtype(dtype)) return SCAN_ERR_UNSUPPORTED;
    if (choices < 1 || choices > kMaxChoices || channels < 1 || channels > kMaxChannels) return SCAN_ERR_INVALID;
    constexpr uint64_t most = (uint64_t)1 << 31;
    if (tokens >= most || tokens * choices >= most || rows >= most) return SCAN_ERR_INVALID;
    return (tokens == 0 || places) && aligned(places, 4) ? SCAN_OK : SCAN_ERR_INVALID;
}

// Clears rows of `out`, rows of V elements per access, in front of a move; false if they are too many for a grid.
template <typename T, int V>
bool clear_rows(const Moves& m, const Clear& c, T* out, int64_t stride, hipStream_t s)
{
    const uint32_t chunks = (m.channels + 64 * kClearParts * V - 1) / (64 * kClearParts * V);
    const uint64_t wgs = ((uint64_t)m.rows + kClearRows - 1) / kClearRows * chunks;
    if (wgs > kMostInGrid) return false;
    if (wgs) hipLaunchKernelGGL((clear_kernel<T, V>), grid_of(wgs), dim3(256), 0, s, m, c, chunks, out, stride);
    return true;
}

bool valid_clear(const int32_t* used, const int32_t* source, uint64_t source_rows)
{
    return aligned(used, 4) && aligned(source, 4) && source_rows < ((uint64_t)1 << 31) && (source || source_rows == 0);
}

// Calls f with a value of the weights' type.
template <typename T, class F>
void with_weights(int weight_dtype, F f)
{
    if (weight_dtype == SEQ_F32)
        f((float)0);
    else
        f(T());
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

size_t expert_split_workspace(size_t n, uint32_t n_experts)
{
    if (n >= ((size_t)1 << 31) || n_experts < 1 || n_experts > kMaxExperts) return 0;
    const SplitPlan p = make_plan(n, n_experts);
    return p.chunks == 1 ? 0 : round_up(((size_t)p.chunks + 1) * n_experts * 4, 256);
}

scan_status_t expert_split(const int32_t* experts, size_t n, uint32_t n_experts, int32_t* offsets, int32_t* places, int32_t* source,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    if (n >= ((size_t)1 << 31) || n_experts < 1 || n_experts > kMaxExperts) return SCAN_ERR_INVALID;
    const size_t need = expert_split_workspace(n, n_experts);
    if (!offsets || (n && (!experts || !places || !source))) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)experts, (const void*)offsets, (const void*)places, (const void*)source})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(offsets, ((uint64_t)n_experts + 1) * 4), range(places, n * 4), range(source, n * 4), range(need ? workspace : nullptr, need)};
    const Range ins[] = {range(experts, n * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const SplitPlan p = make_plan(n, n_experts);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const size_t lds = (size_t)kWaves * n_experts * 4;
    uint32_t *counts = static_cast<uint32_t*>(workspace), *totals = counts + (size_t)p.chunks * n_experts;
    if (p.chunks == 1) {
        hipLaunchKernelGGL((rank_kernel<true>), dim3(1), dim3(kBlock), lds, s, experts, p, offsets, places, source, counts);
        return launched();
    }
    hipLaunchKernelGGL((rank_kernel<false>), dim3(p.chunks), dim3(kBlock), lds, s, experts, p, offsets, places, source, counts);
    if (p.chunks > kFewChunks) hipLaunchKernelGGL(prefix_kernel, dim3((n_experts + 63) / 64), dim3(kBlock), 0, s, p, counts, totals);
    hipLaunchKernelGGL((p.chunks > kFewChunks ? place_kernel<false> : place_kernel<true>), dim3(p.chunks), dim3(kBlock), 0, s, experts, p,
                       (const uint32_t*)counts, (const uint32_t*)totals, offsets, places, source);
    return launched();
}

scan_status_t expert_dispatch(const expert_dispatch_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const expert_dispatch_args_t& a = *args;
    const scan_status_t st = check_moves(a.dtype, a.tokens, a.rows, a.choices, a.channels, a.places);
    if (st != SCAN_OK) return st;
    if (!valid_rows(a.dtype, a.tokens, a.channels, {a.x, a.x_stride}) || !valid_rows(a.dtype, a.rows, a.channels, {a.out, a.out_stride}))
        return SCAN_ERR_INVALID;
    if (!valid_clear(a.used, a.source, a.source_rows)) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype);
    const Range outs[] = {range(a.out, a.rows, a.out_stride, a.channels, es)};
    const Range ins[] = {range(a.x, a.tokens, a.x_stride, a.channels, es), range(a.places, a.tokens * a.choices * 4), range(a.used, 4),
                         range(a.source, a.source_rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    if (a.rows == 0) return SCAN_OK;
    const Moves m{a.places, (uint32_t)a.tokens, (uint32_t)a.rows, a.choices, a.channels};
    const Clear c{a.clear ? nullptr : a.used, a.source, (uint32_t)a.source_rows};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t launch = SCAN_OK;
        with_pack<T>(a.channels, {{a.x, a.x_stride}, {a.out, a.out_stride}}, [&](auto n) {
            constexpr int V = decltype(n)::value;
            const uint32_t chunks = (a.channels + 64 * V * kCopies - 1) / (64 * V * kCopies);
            const uint64_t wgs = (a.tokens * chunks + 3) / 4;
            T* out = static_cast<T*>(a.out);
            if (wgs > kMostInGrid || ((a.clear || a.used) && !clear_rows<T, V>(m, c, out, a.out_stride, s)))
                launch = SCAN_ERR_INVALID;
            else if (wgs)
                hipLaunchKernelGGL((dispatch_kernel<T, V>), grid_of(wgs), dim3(256), 0, s, m, chunks, static_cast<const T*>(a.x), a.x_stride,
                                   out, a.out_stride);
        });
        return launch == SCAN_OK ? launched() : launch;
    });
}

scan_status_t expert_combine(const expert_combine_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const expert_combine_args_t& a = *args;
    const scan_status_t st = check_moves(a.dtype, a.tokens, a.rows, a.choices, a.channels, a.places);
    if (st != SCAN_OK) return st;
    if (a.weights && a.weight_dtype != a.dtype && a.weight_dtype != SEQ_F32) return SCAN_ERR_UNSUPPORTED;
    if (!valid_rows(a.dtype, a.rows, a.channels, {a.y, a.y_stride}) || !valid_rows(a.dtype, a.tokens, a.channels, {a.out, a.out_stride}))
        return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype);
    if (!aligned(a.weights, ws)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(a.out, a.tokens, a.out_stride, a.channels, es)};
    const Range ins[] = {range(a.y, a.rows, a.y_stride, a.channels, es), range(a.places, a.tokens * a.choices * 4),
                         range(a.weights, a.tokens * a.choices * ws)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    if (a.tokens == 0) return SCAN_OK;
    const Moves m{a.places, (uint32_t)a.tokens, (uint32_t)a.rows, a.choices, a.channels};
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t launch = SCAN_OK;
        with_pack<T>(a.channels, {{a.y, a.y_stride}, {a.out, a.out_stride}}, [&](auto n) {
            constexpr int V = decltype(n)::value;
            const uint32_t chunks = (a.channels + 64 * V - 1) / (64 * V);
            const uint64_t wgs = (a.tokens * chunks + 3) / 4;
            if (wgs > kMostInGrid) {
                launch = SCAN_ERR_INVALID;
                return;
            }
            with_weights<T>(a.weight_dtype, [&](auto we) {
                using W = decltype(we);
                hipLaunchKernelGGL((combine_kernel<T, W, V>), grid_of(wgs), dim3(256), 0, static_cast<hipStream_t>(stream), m, chunks,
                                   static_cast<const W*>(a.weights), static_cast<const T*>(a.y), a.y_stride, static_cast<T*>(a.out),
                                   a.out_stride);
            });
        });
        return launch == SCAN_OK ? launched() : launch;
    });
}

scan_status_t expert_combine_grad(const expert_combine_grad_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const expert_combine_grad_args_t& a = *args;
    const scan_status_t st = check_moves(a.dtype, a.tokens, a.rows, a.choices, a.channels, a.places);
    if (st != SCAN_OK) return st;
    if (a.weights && a.weight_dtype != a.dtype && a.weight_dtype != SEQ_F32) return SCAN_ERR_UNSUPPORTED;
    if (!valid_rows(a.dtype, a.tokens, a.channels, {a.dout, a.dout_stride}) || !valid_rows(a.dtype, a.rows, a.channels, {a.dy, a.dy_stride}))
        return SCAN_ERR_INVALID;
    if (a.dweights && !valid_rows(a.dtype, a.rows, a.channels, {a.y, a.y_stride})) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype);
    if (!aligned(a.weights, ws) || !valid_clear(a.used, a.source, a.source_rows) || !aligned(a.dweights, 4)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(a.dy, a.rows, a.dy_stride, a.channels, es), range(a.dweights, a.tokens * a.choices * 4)};
    const Range ins[] = {range(a.dout, a.tokens, a.dout_stride, a.channels, es), range(a.dweights ? a.y : nullptr, a.rows, a.y_stride, a.channels, es),
                         range(a.places, a.tokens * a.choices * 4), range(a.weights, a.tokens * a.choices * ws), range(a.used, 4),
                         range(a.source, a.source_rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const bool clears = (a.clear || a.used) && a.rows;
    if (a.tokens == 0 && !clears) return SCAN_OK;
    const Moves m{a.places, (uint32_t)a.tokens, (uint32_t)a.rows, a.choices, a.channels};
    const Clear clear{a.clear ? nullptr : a.used, a.source, (uint32_t)a.source_rows};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t launch = SCAN_OK;
        const Array y{a.dweights ? a.y : nullptr, a.y_stride};
        with_pack<T>(a.channels, {{a.dout, a.dout_stride}, y, {a.dy, a.dy_stride}}, [&](auto n) {
            constexpr int V = decltype(n)::value;
            T* dy = static_cast<T*>(a.dy);
            if (clears && !clear_rows<T, V>(m, clear, dy, a.dy_stride, s)) {
                launch = SCAN_ERR_INVALID;
                return;
            }
            if (a.tokens == 0) return;
            with_weights<T>(a.weight_dtype, [&](auto we) {
                using W = decltype(we);
                hipLaunchKernelGGL((combine_grad_kernel<T, W, V>), grid_of(a.tokens), dim3(256), 0, s, m, static_cast<const W*>(a.weights),
                                   static_cast<const T*>(a.dout), a.dout_stride, static_cast<const T*>(a.y), a.y_stride, dy, a.dy_stride,
                                   a.dweights);
            });
        });
        return launch == SCAN_OK ? launched() : launch;
    });
}

}  // extern "C"
