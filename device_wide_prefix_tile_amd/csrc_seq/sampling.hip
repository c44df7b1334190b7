// Sampling of tokens with temperature, top-k, top-p and min-p from given random numbers.
//
// One workgroup per row, which it reads once for every pass over it: from the caches but for the first.  (Held in
// registers, 64 of them for 128000 logits of 16 bits, every pass is unrolled over all pieces, and the instructions
// come from memory instead: 256 x 128000 top-k 56 us against 36 in an earlier version.)  With w[i] = exp((logit[i] - max) / temperature), the
// tokens by falling logit (equal ones by ascending index) have a first part that top-k, top-p and min-p leave; the
// sampled token is the first kept one in the order of the indices up to which the kept weights exceed uniform
// times their sum: a scan of the row, of which only the path to one element is needed.
//
// top-k up to kMostSorted: the k-th largest of the threads' largest logits bounds the k-th largest of the row
// from below, and hardly more than k logits reach it.  They go to LDS, are sorted, cut by top-k, top-p and
// min-p, sorted by index and scanned.
//
// Otherwise the border of the first part is found without a sort.  Counts or weights go into bins by the logit's
// distance from the largest (kPerOctave bins for every halving of the weight), a prefix over the bins gives
// the bin in which the limit is met, and the few logits in that bin are ranked against one another (many: told apart by
// eight bits of their value at a time).  Weights so small that all of the row's tokens with such weights could not hold the share that
// top-p leaves out are only added up.
//
// Weights and their sums are held in 64 bits: of 2^17 kept tokens each has some 2^-17 of the sum, and an error of e in
// the running sum moves a row's token with a probability of some 2^17 e.  (With 32 bits in the weights and a wavefront's
// sums, 1 of 700 to 800 rows of 131072 had another token than the definition; with the weights in 64 bits and the sums in
// 32, emulated on the host, 2 of 4096.)  Where LDS atomics add weights up, they are integers, so that the order does not
// matter: rounded multiples of 2^-63 n, of which n fit 64 bits.  All other sums are of fixed order.
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
// Of them, every one is compared with every other one, up to this many.  0 / 64 / 512: 300 rows of 1000 float32 logits 37 / 30 /
// 31 us, 64 of 50001 80 / 72 / 83, 256 of 128000 bfloat16 with top-p 137 / 138 / 169.
constexpr uint32_t kRanked = 64;
constexpr int kMostSums = (kMaxTokens / 4 + 1 + kBlock - 1) / kBlock * kWaves;

struct Settings {
    const float *uniform, *temperatures, *top_ps, *min_ps;
    const int32_t* top_ks;
    double temperature, top_p, min_p;
    int64_t top_k;
};

constexpr uint32_t kSorted = 2 * kBlock;  // logits that are sorted in LDS
// Largest top-k that is sorted: the bound from 1024 threads' largest logits leaves 0.6% of a row for 512 of them, 3% for
// 1000.  256 rows of 128000 bfloat16 logits, sorted / by counts: top-k 50 38 / 112 us, 400 52 / 142, 700 64 / 154, 1000
// (more than can be sorted, then counted) 184 / 162.
constexpr int64_t kMostSorted = kBlock / 4 * 3;

struct Shared {
    uint64_t bins[kBins];  // also the logits that are sorted
    float list_logit[kList];
    uint32_t list_index[kList];
    double sums[kMostSums];
    uint64_t part[kWaves];
    double dpart[kWaves];
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
    __device__ Pack<T, V> load(uint32_t q) const
    {
        const uint32_t i = index(q, 0);
        if (i < n && n - i >= (uint32_t)V) return load_pack<T, V>(p + i);
        Pack<T, V> f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const uint32_t k = index(q, e);
            f.v[e] = k < n ? p[k] : (T)-INFINITY;
        }
        return f;
    }
};

// Logits in 32 bits; NaN becomes minus infinity.  By a comparison: the hardware's maximum of a number and a signalling NaN
// is a NaN.
template <typename T, int V>
__device__ __forceinline__ void unpack_clean(const Pack<T, V>& p, float (&l)[V])
{
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float v = (float)p.v[e];
        l[e] = v == v ? v : -INFINITY;
    }
}

// The pieces of a thread.  (1, 2 or 4 of them in flight take the same time: 16 wavefronts ask at once.)
template <typename T>
struct Pieces {
    static constexpr int V = Row<T>::V;
    // low bits that are 0 in every logit of the type, 8 of them together
    static constexpr int kZeros = std::is_same<T, bf16>::value ? 16 : std::is_same<T, f16>::value ? 8 : 0;
    static constexpr int kFlight = 4;  // pieces whose loads are in flight together
    Row<T> row;

    __device__ Pieces(const T* q, uint32_t len) : row(q, len) {}
    // f(piece's number, its logits) for every one of the thread's pieces
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
        const uint32_t lane = threadIdx.x & 63;
        // whole wavefronts: lanes behind the last piece see minus infinity
        for (uint32_t q = threadIdx.x; q - lane < row.pieces; q += kFlight * kBlock) {
            Pack<T, V> a[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) a[i] = row.load(min(q + i * kBlock, row.pieces - 1));
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (q - lane + i * kBlock >= row.pieces) break;
                float l[V];
                unpack_clean(a[i], l);
                if (q + i * kBlock >= row.pieces) {
#pragma unroll
                    for (int e = 0; e < V; ++e) l[e] = -INFINITY;
                }
                f(q + i * kBlock, l);
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

// The sum over the wavefront, in lane 63, in an order that depends on the lanes alone: within rows of 16, then over
// the rows.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double v)
{
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    const u32x2 o = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.x, CTRL, ROWS, 0xF, false),
                     (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.y, CTRL, ROWS, 0xF, false)};
    return v + __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double wave_sum(double v)
{
    v = add_from<0x111, 0xF>(v);  // row_shr:1
    v = add_from<0x112, 0xF>(v);
    v = add_from<0x114, 0xF>(v);
    v = add_from<0x118, 0xF>(v);
    v = add_from<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    return add_from<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}

// Exclusive prefix over the threads, and the sum, in a fixed order.
__device__ __forceinline__ uint64_t block_prefix(uint64_t v, Shared& s, uint64_t& total)
{
    __syncthreads();
    return dwpt_seq::block_prefix<kWaves>(v, s.part, total);
}
__device__ __forceinline__ double block_prefix(double v, Shared& s, double& total)
{
    __syncthreads();
    return dwpt_seq::block_prefix<kWaves>(v, s.dpart, total);
}

// ------------------------------------------------------------ weights
// 2^t for t <= 0 in 64 bits.  With n the integer next to t and f = t - n (exact), 2^f = 1 + f q(f): q of degree 8 takes the
// values of (2^f - 1) / f at nine Chebyshev nodes of [-1/2, 1/2] (computed in 70 digits), the error is 2^-44.6 at most, and
// 2^0 is 1.  Below 2^-1074 the weight is 0.
__device__ __forceinline__ double exp2_wide(double t)
{
    t = fmax(t, -1100.0);
    const double n = __builtin_rint(t), f = t - n;
    double q = 0x1.b63880a30e9ffp-24;
    q = fma(q, f, 0x1.63d136366db24p-20);
    q = fma(q, f, 0x1.ffcb9515a8016p-17);
    q = fma(q, f, 0x1.4308ac85aa947p-13);
    q = fma(q, f, 0x1.5d87fe86fe88ep-10);
    q = fma(q, f, 0x1.3b2ab7181b755p-7);
    q = fma(q, f, 0x1.c6b08d7047e52p-5);
    q = fma(q, f, 0x1.ebfbdff823cedp-3);
    q = fma(q, f, 0x1.62e42fefa39efp-1);
    return __builtin_amdgcn_ldexp(fma(f, q, 1.0), (int)n);
}

// Weights, and where they lie.  t = log2 of the weight, (logit - max) log2(e) / temperature.
// For the bins 32 bits of t are enough, as long as t falls with the logit: the factor in two parts (both above 0, so that
// minus infinity stays what it is); pre is 1, or 2^-100 for temperatures from 2^60 on, whose factor holds the 2^100.  Next to a
// plus infinity everything else is at minus infinity; its own difference is NaN, of which the minimum with 0 makes 0.
// The weight itself in 64 bits: the difference is exact but for its last bit, top is 2^1000 next to a plus infinity.
struct Scale {
    float pre, max, hi, lo;  // max: times pre
    double top, factor, unit;  // unit: of weights as integers

    __device__ float log2_weight(float logit) const
    {
        const float d = fminf(fmaf(logit, pre, -max), 0.0f);
        return fmaf(d, lo, d * hi);
    }
    __device__ double weight(float logit) const { return exp2_wide(fmin(((double)logit - top) * factor, 0.0)); }
    // The weight as a multiple of 1 / unit
    __device__ uint64_t mass(double w) const { return (uint64_t)fma(w, unit, 0.5); }
    // The logit whose weight is 2^t, but for roundings; minus infinity where that is not to be had.
    __device__ bool usual() const { return pre == 1.0f && max < INFINITY; }
    __device__ float logit_at(float t) const { return usual() ? max + t / (hi + lo) : -INFINITY; }
};

// n: logits of a row
__device__ __forceinline__ Scale make_scale(float max, double temperature, uint32_t n)
{
    double c = 1.4426950408889634 / temperature;
    // an infinite temperature: 2^-200 makes all weights of finite logits 1; above 2^900 only ties with the largest are left
    const double factor = fmin(fmax(c, 0x1p-200), 0x1p900);
    const bool high = c < 0x1p-60;
    if (high) c *= 0x1p100;
    // an infinite temperature: 2^-160 makes all weights of finite logits 1; above 2^100 only ties with the largest are left
    c = fmin(fmax(c, 0x1p-60), 0x1p100);
    float hi = (float)c;
    if ((double)hi >= c) hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, hi) - 1);
    const float pre = high ? 0x1p-100f : 1.0f;
    const int bits = n > 1 ? 32 - __builtin_clz(n - 1) : 0;  // n <= 2^bits
    return Scale{pre, max == INFINITY ? max : max * pre, hi, (float)(c - (double)hi), max == INFINITY ? 0x1p1000 : (double)max, factor,
                 __builtin_amdgcn_ldexp(1.0, 63 - bits)};
}

__device__ __forceinline__ uint32_t bin_of(float t) { return (uint32_t)fminf(-t * kPerOctave, (float)(kBins - 1)); }

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

// What an element counts: 1 (COUNT), or its weight as an integer, if `all` keeps it (ALL: it keeps everything); 0 elsewhere.
template <bool COUNT, bool ALL>
__device__ __forceinline__ uint64_t value_of(float l, uint32_t i, const Scale& scale, const Cut& all)
{
    if (!ALL && !all.keeps(l, i)) return 0;
    return COUNT ? 1u : scale.mass(scale.weight(l));
}

// A logit that at least k of the row's reach: the least of the threads' largest logits up to the bin in which the k-th of
// those lies.  mine: the thread's largest.  Minus infinity if fewer threads have one.
__device__ __forceinline__ float bound_of(const Scale& scale, float mine, uint32_t k, Shared& s)
{
    const uint32_t tid = threadIdx.x;
    const bool any = mine > -INFINITY;
    const uint32_t bin = any ? bin_of(scale.log2_weight(mine)) : 0;
    __syncthreads();
    s.bins[2 * tid] = s.bins[2 * tid + 1] = 0;
    if (tid == 0) s.at = 0xFFFFFFFFu;
    __syncthreads();
    if (any) atomicAdd((unsigned long long*)&s.bins[bin], 1ull);
    __syncthreads();
    uint64_t total;
    const uint64_t b0 = s.bins[2 * tid], b1 = s.bins[2 * tid + 1], before = block_prefix(b0 + b1, s, total);
    if (before < k && k <= before + b0 + b1) s.at = 2 * tid + (before + b0 < k ? 1 : 0);
    __syncthreads();
    if (s.at == 0xFFFFFFFFu) return -INFINITY;
    return -block_max(any && bin <= s.at ? -mine : -INFINITY, s);
}

// The first part of what `all` keeps, up to the element at which the values add up to the limit: `limit` itself
// (COUNT), or share times the sum of the values.  bound: a logit that the element reaches (COUNT).
template <bool COUNT, bool ALL, typename P>
__device__ __forceinline__ Cut find_cut(const P& pieces, const Scale& scale, const Cut& all, uint64_t limit, double share, float bound, Shared& s)
{
    constexpr int V = P::V;
    const auto& row = pieces.row;
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    s.bins[2 * tid] = s.bins[2 * tid + 1] = 0;
    if (tid == 0) s.at = 0xFFFFFFFFu, s.count = 0;
    __syncthreads();
    // the row's weights below this logit add up to less than half of what the share leaves out of a sum of at least 1
    const float small = COUNT ? bound : scale.logit_at(__builtin_amdgcn_logf((float)((1.0 - share) / row.n)) - 1.0f);
    double rest = 0.0;
    pieces.each([&](uint32_t q, const float(&l)[V]) __attribute__((always_inline)) {
        double w[V];
        if (!COUNT) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                w[e] = ALL || all.keeps(l[e], row.index(q, e)) ? scale.weight(l[e]) : 0.0;
                rest += l[e] < small ? w[e] : 0.0;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (l[e] < small) continue;
            // one more minus infinity among the counts is one more in the last bin, behind every other
            const uint64_t v = COUNT ? (uint64_t)(ALL || all.keeps(l[e], row.index(q, e))) : scale.mass(w[e]);
            if (ALL || v) atomicAdd((unsigned long long*)&s.bins[bin_of(scale.log2_weight(l[e]))], (unsigned long long)v);
        }
    });
    __syncthreads();
    uint64_t total;
    const uint64_t b0 = s.bins[2 * tid], b1 = s.bins[2 * tid + 1];
    const uint64_t before = block_prefix(b0 + b1, s, total);
    if (!COUNT) {
        uint64_t more;
        block_prefix(scale.mass(rest), s, more);
        limit = max((uint64_t)1, (uint64_t)ceil(share * (double)(total + more)));
    }
    if (before < limit && limit <= before + b0 + b1) {
        const bool second = before + b0 < limit;
        s.at = 2 * tid + (second ? 1 : 0);
        s.base = second ? before + b0 : before;
    }
    __syncthreads();
    const uint32_t bin = s.at;
    if (bin == 0xFFFFFFFFu) return all;  // less than the limit in all
    uint64_t base = s.base;

    // the bin's elements: an interval of logits, with room for roundings, and in it the bin itself
    float from = -INFINITY, to = INFINITY;
    if (scale.usual() && bin + 1 < (uint32_t)kBins) {
        from = scale.logit_at(-(float)(bin + 1) / kPerOctave);
        to = scale.logit_at(-(float)bin / kPerOctave);
        const float room = (fabsf(from) + fabsf(scale.max)) * 0x1p-20f;
        from -= room, to += room;
    }
    pieces.each([&](uint32_t q, const float(&l)[V]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (!(l[e] >= from && l[e] <= to)) continue;
            if (bin_of(scale.log2_weight(l[e])) == bin && value_of<COUNT, ALL>(l[e], row.index(q, e), scale, all)) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kList) {
                    s.list_logit[at] = l[e];
                    s.list_index[at] = row.index(q, e);
                }
            }
        }
    });
    __syncthreads();
    const uint32_t listed = s.count;
    if (listed <= kRanked) {
        // the one up to which those before it, by logit and index, and itself reach the limit
        const bool in = tid < listed;
        const float l = in ? s.list_logit[tid] : 0.0f;
        const uint32_t index = in ? s.list_index[tid] : 0;
        const uint64_t v = !in ? 0 : COUNT ? 1 : scale.mass(scale.weight(l));
        if (in) s.bins[tid] = v;
        if (tid == 0) s.at = 0;
        __syncthreads();
        if (in) {
            uint64_t before = base;
            bool later = false;  // one that equals it follows
            for (uint32_t k = 0; k < listed; ++k) {
                const float o = s.list_logit[k];
                const uint32_t i = s.list_index[k];
                if (o > l || (o == l && i < index)) before += s.bins[k];
                later |= o == l && i > index;
            }
            if (before < limit && limit <= before + v) s.at = tid, s.count = later ? 1u : 0u;
        }
        __syncthreads();
        const uint32_t k = s.at;
        const float logit = s.list_logit[k];
        return Cut{logit, s.count ? s.list_index[k] : all.logit == logit ? all.index : 0xFFFFFFFFu};
    }
    // f(logit, index, value) for each of them
    const auto each = [&](auto f) {
        if (listed <= kList) {
            for (uint32_t k = tid; k < listed; k += kBlock) {
                const float l = s.list_logit[k];
                f(l, s.list_index[k], COUNT ? (uint64_t)1 : scale.mass(scale.weight(l)));
            }
        } else {
            for (uint32_t q = tid; q < row.pieces; q += kBlock) {
                float l[V];
                unpack_clean(row.load(q), l);
                for (int e = 0; e < V; ++e) {
                    if (bin_of(scale.log2_weight(l[e])) != bin) continue;
                    const uint64_t v = value_of<COUNT, ALL>(l[e], row.index(q, e), scale, all);
                    if (v) f(l[e], row.index(q, e), v);
                }
            }
        }
    };

    // their values, eight bits at a time from the top
    uint32_t key = 0, mask = 0;
    uint64_t equal = 0;  // the values of the elements with the key so far
    for (int shift = 24; shift >= P::kZeros; shift -= 8) {
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
    if (!(key & 0x80000000u)) key |= (1u << P::kZeros) - 1;  // the bits of negative numbers are turned over
    const float logit = logit_of(key);
    const uint64_t each_value = COUNT ? 1 : scale.mass(scale.weight(logit));
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

// What the sums are compared with; with a random number of 1 no sum exceeds it, however it was rounded.
__device__ __forceinline__ double share_of(float uniform, double total) { return uniform < 1.0f ? (double)uniform * total : INFINITY; }

// ------------------------------------------------------------ top-k by sorting
// Sorts a[0 .. size) ascending (size: a power of two, at most 2 kBlock).
__device__ void sort(uint64_t* a, uint32_t size)
{
    for (uint32_t run = 2; run <= size; run *= 2) {
        for (uint32_t step = run / 2; step > 0; step /= 2) {
            __syncthreads();
            const uint32_t i = threadIdx.x;
            if (i < size / 2) {
                const uint32_t lo = (i / step) * 2 * step + i % step, hi = lo + step;
                const uint64_t x = a[lo], y = a[hi];
                if ((x > y) != ((lo & run) != 0)) a[lo] = y, a[hi] = x;
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t power_of_two(uint32_t n)
{
    uint32_t p = 2;
    while (p < n) p *= 2;
    return p;
}

// The token, if no more than kSorted of the row's logits reach `bound`, which the first k do; false elsewhere.
template <typename P>
__device__ __forceinline__ bool sample_sorted(const P& pieces, const Scale& scale, float bound, uint32_t k, double top_p, double least, float uniform,
                                              Shared& s, uint32_t& token)
{
    constexpr int V = P::V;
    const auto& row = pieces.row;
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) s.count = 0;
    __syncthreads();
    pieces.each([&](uint32_t q, const float(&l)[V]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (l[e] >= bound && l[e] > -INFINITY) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                // by falling logit, then by index
                if (at < kSorted) s.bins[at] = (uint64_t)~key_of(l[e]) << 32 | row.index(q, e);
            }
        }
    });
    __syncthreads();
    const uint32_t count = s.count;
    if (count > kSorted) return false;
    uint32_t size = power_of_two(count);
    for (uint32_t i = count + tid; i < size; i += kBlock) s.bins[i] = ~0ull;
    sort(s.bins, size);
    const uint32_t first = min(k, count);
    // thread t has ranks 2 t and 2 t + 1
    double w[2], total;
    uint64_t entry[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t r = 2 * tid + j;
        const uint64_t v = r < first ? s.bins[r] : 0;
        const float l = logit_of(~(uint32_t)(v >> 32));
        entry[j] = v << 32 | __builtin_bit_cast(uint32_t, l);
        w[j] = r < first ? scale.weight(l) : 0.0;
    }
    const double before = block_prefix(w[0] + w[1], s, total);
    const double limit = top_p < 1.0 ? fmax(top_p, 0.0) * total : INFINITY;
    if (tid == 0) s.count = 0;
    __syncthreads();
    // what is kept, by index
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (w[j] > 0.0 && ((j ? before + w[0] : before) < limit || 2 * tid + j == 0) && w[j] >= least)
            s.bins[atomicAdd(&s.count, 1u)] = entry[j];
    }
    __syncthreads();
    const uint32_t kept = s.count;
    size = power_of_two(kept);
    for (uint32_t i = kept + tid; i < size; i += kBlock) s.bins[i] = ~0ull;
    sort(s.bins, size);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t r = 2 * tid + j;
        entry[j] = r < kept ? s.bins[r] : 0;
        w[j] = r < kept ? scale.weight(__builtin_bit_cast(float, (uint32_t)entry[j])) : 0.0;
    }
    const double start = block_prefix(w[0] + w[1], s, total);
    const double target = share_of(uniform, total);
    // the first whose sum exceeds the target, else the last
    uint32_t over = kept - 1;
    if (start + (w[0] + w[1]) > target) over = min(over, 2 * tid + (start + w[0] > target ? 0u : 1u));
    over = block_min(over, s);
    if (tid == 0) s.at = (uint32_t)(s.bins[over] >> 32);
    __syncthreads();
    token = s.at;
    return true;
}

// ------------------------------------------------------------ the kernel
// 512 rows of 131072 bfloat16 logits without a cut 95 us (68 with weights and partial sums in 32 bits, which gave wrong
// tokens): HBM is read once (134 MB, 20 us), the second pass comes from the caches; vector units busy 75%, 35 vector
// instructions per logit, of which a weight in 64 bits and its sum take some 20.  256 x 128000 with settings of their own 154 us:
// the longest row's, which takes five passes (counts, their border, weights, their border, sums).
template <typename T>
__global__ __launch_bounds__(kBlock) void sample_kernel(Settings set, uint32_t rows, uint32_t n, const T* __restrict__ logits,
                                                        int64_t stride, void* __restrict__ tokens, int token_bytes)
{
    constexpr int V = Row<T>::V;
    __shared__ Shared s;
    const uint32_t r = workgroup(), tid = threadIdx.x;
    if (r >= rows) return;
    const int lane = tid & 63, w = uniform((int)(tid >> 6));
    const Pieces<T> pieces(logits + (int64_t)r * stride, n);
    const Row<T>& row = pieces.row;
    const double temperature = set.temperatures ? (double)set.temperatures[r] : set.temperature;
    const int64_t top_k = set.top_ks ? (int64_t)set.top_ks[r] : set.top_k;
    const double top_p = set.top_ps ? (double)set.top_ps[r] : set.top_p;
    const double min_p = set.min_ps ? (double)set.min_ps[r] : set.min_p;
    const float u = set.uniform[r], uniform01 = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
    const auto result = [&](int64_t token) {
        if (token_bytes == 4)
            static_cast<int32_t*>(tokens)[r] = (int32_t)token;
        else
            static_cast<int64_t*>(tokens)[r] = token;
    };

    float mine = -INFINITY;
    pieces.each([&](uint32_t, const float(&l)[V]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e) mine = fmaxf(mine, l[e]);
    });
    const float most = block_max(mine, s);
    if (most == -INFINITY) {
        if (tid == 0) result(-1);
        return;
    }
    if (!(temperature > 0.0)) {
        uint32_t first = 0xFFFFFFFFu;
        if (mine == most) {
            pieces.each([&](uint32_t q, const float(&l)[V]) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (l[e] == most) first = min(first, row.index(q, e));
            });
        }
        first = block_min(first, s);
        if (tid == 0) result(first);
        return;
    }
    const Scale scale = make_scale(most, temperature, n);
    const double least = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;
    Cut cut{-INFINITY, 0xFFFFFFFFu};
    if (top_k > 0 && top_k < (int64_t)n) {
        uint32_t token;
        const float bound = top_k <= kBlock && n > kSorted ? bound_of(scale, mine, (uint32_t)top_k, s) : -INFINITY;
        if ((n <= kSorted || (bound > -INFINITY && top_k <= kMostSorted)) &&
            sample_sorted(pieces, scale, bound, (uint32_t)min(top_k, (int64_t)n), top_p, least, uniform01, s, token)) {
            if (tid == 0) result(token);
            return;
        }
        cut = find_cut<true, true>(pieces, scale, cut, (uint64_t)top_k, 0.0, bound, s);
        if (top_p < 1.0) cut = find_cut<false, false>(pieces, scale, cut, 0, fmax(top_p, 0.0), 0.0f, s);
    } else if (top_p < 1.0) {
        cut = find_cut<false, true>(pieces, scale, cut, 0, fmax(top_p, 0.0), 0.0f, s);
    }
    // The kept weights of a piece, and their sum.  CHECK 0: everything is kept, 1: logits from the cut's on with the least
    // weight, 2: some of those that equal the cut's are not.
    const auto kept = [&](auto check, uint32_t q, const float(&l)[V], double(&f)[V]) __attribute__((always_inline)) {
        constexpr int CHECK = decltype(check)::value;
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const double v = scale.weight(l[e]);
            const bool keep = CHECK == 0 || (v >= least && (CHECK == 1 ? l[e] >= cut.logit : cut.keeps(l[e], row.index(q, e))));
            f[e] = keep ? v : 0.0;
            sum += f[e];
        }
        return sum;
    };
    const auto sums = [&](auto check) __attribute__((always_inline)) {
        pieces.each([&](uint32_t q, const float(&l)[V]) __attribute__((always_inline)) {
            if (decltype(check)::value > 0) {
                // where little is kept, most wavefronts have nothing to keep
                float largest = l[0];
#pragma unroll
                for (int e = 1; e < V; ++e) largest = fmaxf(largest, l[e]);
                if (!__builtin_amdgcn_ballot_w64(largest >= cut.logit)) return;
            }
            double f[V];
            const double sum = wave_sum(kept(check, q, l, f));
            if (lane == 63) s.sums[q / kBlock * kWaves + w] = sum;
        });
    };
    const uint32_t entries = (row.pieces + kBlock - 1) / kBlock * kWaves;
    for (uint32_t k = tid; k < entries; k += kBlock) s.sums[k] = 0.0;
    __syncthreads();
    if (cut.index != 0xFFFFFFFFu)
        sums(std::integral_constant<int, 2>());
    else if (cut.logit > -INFINITY || least > 0.0)
        sums(std::integral_constant<int, 1>());
    else
        sums(std::integral_constant<int, 0>());
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
    double own = 0.0;
    for (uint32_t k = lo; k < hi; ++k) own += s.sums[k];
    double incl = prefix(own);
    const double target = share_of(uniform01, __shfl(incl, 63, 64));
    int leader = pick(incl, own, target);
    // that lane's entries one after another; every lane walks along
    const uint32_t from = (uint32_t)__builtin_amdgcn_readlane((int)lo, leader), to = (uint32_t)__builtin_amdgcn_readlane((int)hi, leader);
    double base = __shfl(incl - own, leader, 64), at = base;
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
    float l[V];
    double f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 0.0;
    own = 0.0;
    if (q < row.pieces) {
        unpack_clean(row.load(q), l);
        own = kept(std::integral_constant<int, 2>(), q, l, f);
    }
    incl = base + prefix(own);
    leader = pick(incl, own, target);
    if (lane != leader) return;
    at = incl - own;
    uint32_t token = 0;
    for (int e = 0; e < V; ++e) {
        if (f[e] > 0.0) {
            token = row.index(q, e);
            at += f[e];
            if (at > target) break;
        }
    }
    result(token);
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
        hipLaunchKernelGGL((sample_kernel<T>), grid_of(a.rows), dim3(kBlock), 0, s, set, (uint32_t)a.rows, a.n, static_cast<const T*>(a.logits),
                           a.logits_stride, a.tokens, a.token_bytes);
        return launched();
    });
}

}  // extern "C"
