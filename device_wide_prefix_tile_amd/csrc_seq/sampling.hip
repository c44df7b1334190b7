// Sampling of tokens with temperature, top-k, top-p and min-p from given random numbers.
//
// One workgroup per row.  With w[i] = exp((logit[i] - max) / temperature), the tokens by falling logit (equal
// ones by ascending index) have a first part that top-k, top-p and min-p leave; the sampled token
// is the first kept one in the order of the indices up to which the kept weights exceed uniform times
// their sum: a scan of the row, of which only the path to one element is needed.
//
// The border of the first part is found without a sort.  Counts or weights go into bins by the logit's
// distance from the largest (kPerOctave bins for every halving of the weight), a prefix over the bins gives
// the bin in which the limit is met, and the few logits in that bin are told apart by eight bits of
// their value at a time.  Weights are integers there (multiples of 2^-44), so that the order in which
// LDS atomics add them up does not matter: 2^19 of them fit 64 bits.  The final sums are of fixed order,
// in 32 bits over the elements of a 16-byte piece and in 64 bits beyond.
#include <cfloat>
#include <cmath>

#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr uint32_t kMaxTokens = 1u << 19;
constexpr int kBlock = 1024;
constexpr int kWaves = kBlock / 64;
constexpr int kBins = 2 * kBlock;
constexpr float kPerOctave = 32.0f;  // the last bin holds weights below 2^-64, which are 0 as multiples of 2^-44
constexpr uint32_t kList = 4096;     // logits of the bin with the border that are kept in LDS; more are looked up in the row
constexpr int kMostSums = (kMaxTokens / 4 + 1 + kBlock - 1) / kBlock * kWaves;

struct Settings {
    const float *uniform, *temperatures, *top_ps, *min_ps;
    const int32_t* top_ks;
    double temperature, top_p, min_p;
    int64_t top_k;
};

struct Shared {
    uint64_t bins[kBins];
    float list_logit[kList];
    uint32_t list_index[kList];
    double sums[kMostSums];
    uint64_t part[kWaves];
    float fpart[kWaves];
    uint32_t upart[kWaves];
    uint64_t base;
    uint32_t at, count;
};

// ------------------------------------------------------------ the row
// A row as 16-byte pieces from the aligned address at or before its start; places outside the row read as
// minus infinity.  Wavefront w takes pieces [64 w, 64 w + 64) of every kBlock: indices ascend
// with (round, wavefront, lane, element).
template <typename T>
struct Row {
    static constexpr int V = 16 / sizeof(T);
    const T* p;
    uint32_t n, off, pieces;

    __device__ Row(const T* q, uint32_t len) : p(q), n(len)
    {
        off = (uint32_t)((uintptr_t)q % 16 / sizeof(T));
        pieces = (len + off + V - 1) / V;
    }
    // Index of element e of piece q; wraps around to a large number in front of the row.
    __device__ uint32_t index(uint32_t q, int e) const { return q * V + (uint32_t)e - off; }
    __device__ void load(uint32_t q, float (&f)[V]) const
    {
        const uint32_t i = index(q, 0);
        if (i < n && n - i >= (uint32_t)V) {
            unpack(load_pack<T, V>(p + i), f);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const uint32_t k = index(q, e);
                f[e] = k < n ? (float)p[k] : -INFINITY;
            }
        }
    }
};

// ------------------------------------------------------------ sums over the workgroup
__device__ __forceinline__ float block_max(float v, Shared& s)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.fpart[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.fpart[0];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v = fmaxf(v, s.fpart[q]);
    return v;
}

__device__ __forceinline__ uint32_t block_min(uint32_t v, Shared& s)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = min(v, (uint32_t)__shfl_xor(v, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.upart[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.upart[0];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v = min(v, s.upart[q]);
    return v;
}

// Exclusive prefix over the threads, and the sum.
__device__ __forceinline__ uint64_t block_prefix(uint64_t v, Shared& s, uint64_t& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t t = __shfl_up((unsigned long long)incl, o, 64);
        if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 63) s.part[w] = incl;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) {
        before += q < w ? s.part[q] : 0;
        all += s.part[q];
    }
    total = all;
    return before + incl - v;
}

// ------------------------------------------------------------ weights
// t = log2 of the weight: (logit - max) log2(e) / temperature, the factor in two parts (both above 0, so that minus
// infinity stays what it is).  `usual`: the largest logit is finite, the temperature below 2^60.
struct Scale {
    float max, hi, lo;
    bool usual;

    __device__ float log2_weight(float logit) const
    {
        float d = logit - max;
        if (!usual) {
            if (max == INFINITY)
                d = logit == max ? 0.0f : -INFINITY;  // next to a plus infinity nothing else weighs
            else
                d = logit * 0x1p-100f - max * 0x1p-100f;  // the factor holds 2^100
        }
        return fmaf(d, lo, d * hi);
    }
    __device__ static float weight(float t) { return fmaxf(exp2_fast(t), 0.0f); }  // NaN: 0
};

__device__ __forceinline__ Scale make_scale(float max, double temperature)
{
    double c = 1.4426950408889634 / temperature;
    const bool high = c < 0x1p-60;
    if (high) c *= 0x1p100;
    // an infinite temperature: 2^-160 makes all weights of finite logits 1; above 2^100 only ties with the largest are left
    c = fmin(fmax(c, 0x1p-60), 0x1p100);
    float hi = (float)c;
    if ((double)hi >= c) hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, hi) - 1);
    return Scale{max, hi, (float)(c - (double)hi), !high && max < INFINITY};
}

__device__ __forceinline__ uint32_t bin_of(float t) { return (uint32_t)fminf(-t * kPerOctave, (float)(kBins - 1)); }

// floor(w 2^44), w <= 1
__device__ __forceinline__ uint64_t mass(float w)
{
    const float s = w * 0x1p44f;
    const uint32_t hi = (uint32_t)(s * 0x1p-32f);
    const uint32_t lo = (uint32_t)fmaf((float)hi, -0x1p32f, s);
    return (uint64_t)hi << 32 | lo;
}

// Unsigned numbers in the order of the floats; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __builtin_bit_cast(float, key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The kept part: logits above `logit`, and those equal to it with indices up to `index`.
struct Cut {
    float logit;
    uint32_t index;

    __device__ bool keeps(float l, uint32_t i) const { return l > logit || (l == logit && i <= index); }
};

// What an element counts: 1 (COUNT), or its weight as an integer, if `all` keeps it; 0 elsewhere.
template <bool COUNT>
__device__ __forceinline__ uint64_t value_of(float l, uint32_t i, float t, const Cut& all)
{
    if (!all.keeps(l, i)) return 0;
    return COUNT ? (l > -INFINITY ? 1u : 0u) : mass(Scale::weight(t));
}

// The first part of what `all` keeps, up to the element at which the values add up to the limit: `limit` itself
// (COUNT), or share times the sum of the values.
template <bool COUNT, typename T>
__device__ Cut find_cut(const Row<T>& row, const Scale& scale, const Cut& all, uint64_t limit, double share, Shared& s)
{
    constexpr int V = Row<T>::V;
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    s.bins[2 * tid] = s.bins[2 * tid + 1] = 0;
    if (tid == 0) s.at = 0xFFFFFFFFu, s.count = 0;
    __syncthreads();
    for (uint32_t q = tid; q < row.pieces; q += kBlock) {
        float l[V];
        row.load(q, l);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float t = scale.log2_weight(l[e]);
            const uint64_t v = value_of<COUNT>(l[e], row.index(q, e), t, all);
            if (v) atomicAdd((unsigned long long*)&s.bins[bin_of(t)], (unsigned long long)v);
        }
    }
    __syncthreads();
    uint64_t total;
    const uint64_t b0 = s.bins[2 * tid], b1 = s.bins[2 * tid + 1];
    const uint64_t before = block_prefix(b0 + b1, s, total);
    if (!COUNT) limit = max((uint64_t)1, (uint64_t)ceil(share * (double)total));
    if (before < limit && limit <= before + b0 + b1) {
        const bool second = before + b0 < limit;
        s.at = 2 * tid + (second ? 1 : 0);
        s.base = second ? before + b0 : before;
    }
    __syncthreads();
    const uint32_t bin = s.at;
    if (bin == 0xFFFFFFFFu) return all;  // less than the limit in all
    uint64_t base = s.base;

    // the bin's elements
    for (uint32_t q = tid; q < row.pieces; q += kBlock) {
        float l[V];
        row.load(q, l);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float t = scale.log2_weight(l[e]);
            if (bin_of(t) == bin && value_of<COUNT>(l[e], row.index(q, e), t, all)) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kList) {
                    s.list_logit[at] = l[e];
                    s.list_index[at] = row.index(q, e);
                }
            }
        }
    }
    __syncthreads();
    const uint32_t listed = s.count;
    // f(logit, index, value) for each of them
    const auto each = [&](auto f) {
        if (listed <= kList) {
            for (uint32_t k = tid; k < listed; k += kBlock) {
                const float l = s.list_logit[k];
                f(l, s.list_index[k], COUNT ? (uint64_t)1 : mass(Scale::weight(scale.log2_weight(l))));
            }
        } else {
            for (uint32_t q = tid; q < row.pieces; q += kBlock) {
                float l[V];
                row.load(q, l);
                for (int e = 0; e < V; ++e) {
                    const float t = scale.log2_weight(l[e]);
                    if (bin_of(t) != bin) continue;
                    const uint64_t v = value_of<COUNT>(l[e], row.index(q, e), t, all);
                    if (v) f(l[e], row.index(q, e), v);
                }
            }
        }
    };

    // their values, eight bits at a time from the top
    uint32_t key = 0, mask = 0;
    uint64_t equal = 0;  // the values of the elements with the key so far
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (tid < 256) s.bins[tid] = 0;
        __syncthreads();
        each([&](float l, uint32_t, uint64_t v) {
            const uint32_t k = key_of(l);
            if ((k & mask) == key) atomicAdd((unsigned long long*)&s.bins[255 - (k >> shift & 255)], (unsigned long long)v);
        });
        __syncthreads();
        const uint64_t b = tid < 256 ? s.bins[tid] : 0;
        uint64_t sum;
        const uint64_t above = base + block_prefix(b, s, sum);
        if (above < limit && limit <= above + b) {
            s.at = 255 - tid;
            s.base = above;
            s.bins[0] = b;  // every thread has its own
        }
        __syncthreads();
        key |= s.at << shift;
        mask |= 255u << shift;
        base = s.base;
        equal = s.bins[0];
    }
    const float logit = logit_of(key);
    const uint64_t each_value = COUNT ? 1 : mass(Scale::weight(scale.log2_weight(logit)));
    const uint64_t wanted = (limit - base + each_value - 1) / each_value, there = equal / each_value;
    if (wanted >= there) return Cut{logit, all.logit == logit ? all.index : 0xFFFFFFFFu};

    // of equal logits the first `wanted` by index, ten bits of it at a time
    uint32_t index = 0, imask = 0;
    uint64_t found = 0;
    for (int shift = 10; shift >= 0; shift -= 10) {
        __syncthreads();
        s.bins[tid] = 0;
        __syncthreads();
        each([&](float l, uint32_t i, uint64_t) {
            if (l == logit && (i & imask) == index) atomicAdd((unsigned long long*)&s.bins[i >> shift & 1023], 1ull);
        });
        __syncthreads();
        const uint64_t b = s.bins[tid];
        uint64_t sum;
        const uint64_t below = found + block_prefix(b, s, sum);
        if (below < wanted && wanted <= below + b) {
            s.at = tid;
            s.base = below;
        }
        __syncthreads();
        index |= s.at << shift;
        imask |= 1023u << shift;
        found = s.base;
    }
    return Cut{logit, index};
}

// ------------------------------------------------------------ the kernel
template <typename T, typename I>
__global__ __launch_bounds__(kBlock) void sample_kernel(Settings set, uint32_t rows, uint32_t n, const T* __restrict__ logits,
                                                        int64_t stride, I* __restrict__ tokens)
{
    constexpr int V = Row<T>::V;
    __shared__ Shared s;
    const uint32_t r = workgroup(), tid = threadIdx.x;
    if (r >= rows) return;
    const int lane = tid & 63, w = uniform((int)(tid >> 6));
    const Row<T> row(logits + (int64_t)r * stride, n);
    const double temperature = set.temperatures ? (double)set.temperatures[r] : set.temperature;
    const int64_t top_k = set.top_ks ? (int64_t)set.top_ks[r] : set.top_k;
    const double top_p = set.top_ps ? (double)set.top_ps[r] : set.top_p;
    const double min_p = set.min_ps ? (double)set.min_ps[r] : set.min_p;

    float most = -INFINITY;
    for (uint32_t q = tid; q < row.pieces; q += kBlock) {
        float l[V];
        row.load(q, l);
#pragma unroll
        for (int e = 0; e < V; ++e) most = fmaxf(most, l[e]);
    }
    most = block_max(most, s);
    if (most == -INFINITY) {
        if (tid == 0) tokens[r] = (I)-1;
        return;
    }
    if (!(temperature > 0.0)) {
        uint32_t first = 0xFFFFFFFFu;
        for (uint32_t q = tid; q < row.pieces; q += kBlock) {
            float l[V];
            row.load(q, l);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (l[e] == most) first = min(first, row.index(q, e));
        }
        first = block_min(first, s);
        if (tid == 0) tokens[r] = (I)first;
        return;
    }
    const Scale scale = make_scale(most, temperature);
    Cut cut{-INFINITY, 0xFFFFFFFFu};
    if (top_k > 0 && top_k < (int64_t)n) cut = find_cut<true>(row, scale, cut, (uint64_t)top_k, 0.0, s);
    if (top_p < 1.0) cut = find_cut<false>(row, scale, cut, 0, fmax(top_p, 0.0), s);
    float least = 0.0f;  // the smallest float that is not below min_p
    if (min_p > 0.0) {
        least = (float)fmin(min_p, 1.0);
        if ((double)least < fmin(min_p, 1.0)) least = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, least) + 1);
    }
    // the kept weights of piece q, and their sum
    const auto kept = [&](uint32_t q, float (&f)[V]) {
        row.load(q, f);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float v = Scale::weight(scale.log2_weight(f[e]));
            f[e] = cut.keeps(f[e], row.index(q, e)) && v >= least ? v : 0.0f;
            sum += f[e];
        }
        return sum;
    };
    const uint32_t entries = (row.pieces + kBlock - 1) / kBlock * kWaves;
    for (uint32_t q0 = 0; q0 < row.pieces; q0 += kBlock) {
        const uint32_t q = q0 + tid;
        float f[V];
        double sum = q < row.pieces ? (double)kept(q, f) : 0.0;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
        if (lane == 0) s.sums[q0 / kBlock * kWaves + w] = sum;
    }
    __syncthreads();
    if (w != 0) return;

    // the first lane whose inclusive prefix exceeds the target, else the last with a sum of its own
    const auto pick = [&](double incl, double mine, double target) {
        const uint64_t over = __builtin_amdgcn_ballot_w64(incl > target && mine > 0.0), some = __builtin_amdgcn_ballot_w64(mine > 0.0);
        return over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
    };
    const auto prefix = [&](double v) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double t = __shfl_up(v, o, 64);
            if (lane >= o) v += t;
        }
        return v;
    };
    const uint32_t run = (entries + 63) / 64, lo = min(lane * run, entries), hi = min(lo + run, entries);
    double mine = 0.0;
    for (uint32_t k = lo; k < hi; ++k) mine += s.sums[k];
    double incl = prefix(mine);
    const float u = set.uniform[r];
    const double target = (double)(u > 0.0f ? fminf(u, 1.0f) : 0.0f) * __shfl(incl, 63, 64);
    int leader = pick(incl, mine, target);
    // that lane's entries one after another; every lane walks along
    const uint32_t from = (uint32_t)__builtin_amdgcn_readlane((int)lo, leader), to = (uint32_t)__builtin_amdgcn_readlane((int)hi, leader);
    double base = __shfl(incl - mine, leader, 64), at = base;
    uint32_t entry = from;
    for (uint32_t k = from; k < to; ++k) {
        const double v = s.sums[k];
        if (v > 0.0) {
            entry = k;
            base = at;
            if (at + v > target) break;
        }
        at += v;
    }
    const uint32_t q = entry / kWaves * kBlock + entry % kWaves * 64 + lane;
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 0.0f;
    mine = q < row.pieces ? (double)kept(q, f) : 0.0;
    incl = base + prefix(mine);
    leader = pick(incl, mine, target);
    if (lane != leader) return;
    at = incl - mine;
    uint32_t token = 0;
    for (int e = 0; e < V; ++e) {
        if (f[e] > 0.0f) {
            token = row.index(q, e);
            at += (double)f[e];
            if (at > target) break;
        }
    }
    tokens[r] = (I)token;
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

scan_status_t sample_tokens(const sample_tokens_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const sample_tokens_args_t& a = *args;
    if (!valid_dtype(a.dtype)) return SCAN_ERR_UNSUPPORTED;
    if (a.token_bytes != 4 && a.token_bytes != 8) return SCAN_ERR_INVALID;
    if (a.rows >= ((uint64_t)1 << 31) || a.n < 1 || a.n > kMaxTokens) return SCAN_ERR_INVALID;
    if (a.rows == 0) return SCAN_OK;
    const size_t es = dtype_size(a.dtype);
    if (!a.logits || !aligned(a.logits, es) || a.logits_stride < (int64_t)a.n || a.logits_stride > ((int64_t)1 << 31)) return SCAN_ERR_INVALID;
    if (!a.uniform || !a.tokens || !aligned(a.tokens, (size_t)a.token_bytes)) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)a.uniform, (const void*)a.temperatures, (const void*)a.top_ks, (const void*)a.top_ps, (const void*)a.min_ps})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(a.tokens, a.rows * (uint64_t)a.token_bytes)};
    const Range ins[] = {range(a.logits, a.rows, a.logits_stride, a.n, es), range(a.uniform, a.rows * 4), range(a.temperatures, a.rows * 4),
                         range(a.top_ks, a.rows * 4), range(a.top_ps, a.rows * 4), range(a.min_ps, a.rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const Settings set{a.uniform, a.temperatures, a.top_ps, a.min_ps, a.top_ks, a.temperature, a.top_p, a.min_p, a.top_k};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        const T* logits = static_cast<const T*>(a.logits);
        if (a.token_bytes == 4)
            hipLaunchKernelGGL((sample_kernel<T, int32_t>), grid_of(a.rows), dim3(kBlock), 0, s, set, (uint32_t)a.rows, a.n, logits,
                               a.logits_stride, static_cast<int32_t*>(a.tokens));
        else
            hipLaunchKernelGGL((sample_kernel<T, int64_t>), grid_of(a.rows), dim3(kBlock), 0, s, set, (uint32_t)a.rows, a.n, logits,
                               a.logits_stride, static_cast<int64_t*>(a.tokens));
        return launched();
    });
}

}  // extern "C"
