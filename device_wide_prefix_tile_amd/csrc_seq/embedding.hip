// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[i] = scale * table[tokens[i]], a gather of rows; HBM-bound (one
// row read and one written per token).
//
// Gradient: dtable[v] = scale * sum over {i : tokens[i] = v} of dout[i].  The
// positions are first grouped by token, in ascending order within a token (a
// stable split, as radix_split's, but by the whole token at once), then each
// row of the table is the sum of one run of that order.  No atomics add
// floating-point values, so the sums' order is fixed.
//
//   group:  tokens are dealt to `buckets` workgroups by their low bits, so
//           that neighbouring tokens (byte-level text in a large vocabulary)
//           spread out.  Every workgroup reads all tokens (of its segment of
//           65536) and keeps those of its bucket: counts per (wavefront,
//           token) in LDS, a scan of them that gives every wavefront the first
//           place of each token, and a second walk that writes the positions.
//           Up to 65536 tokens that is one launch; above, the counts of every
//           segment go through memory (three launches).
//   sums:   rows with more than kPiece positions are cut along the windows of
//           kPiece sorted positions, and each window's part of such a row is
//           summed by a workgroup of its own (32 bits, to the workspace);
//           every other row is summed whole, or zero.  One launch.
//   join:   the rows of pieces.
#include <initializer_list>
#include <utility>

#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr int kGroupBlock = 1024;
constexpr int kGroupWaves = kGroupBlock / 64;
// Tokens that one pass of the grouping kernels reads.  Every workgroup reads a segment whole, which
// short ones make cheaper, but every segment's counts of the whole table go through memory.  Gradient
// with 65536 / 32768 / 16384 / 8192 / 4096, us: 65536 x 2048 bfloat16 into 50000 rows 139 / 143 / 132 /
// 137 / 149; 262144 x 1024 into 50000 228 / 223 / 229 / 257 / 308; 65536 x 64 into 2^20 163 / 193 / 221 /
// 321 / 510; 65536 x 8 into 2^24 2714 / 3204 / 4220 / 5812 / 9087.
constexpr uint32_t kSegment = 65536;
// Table rows per bucket: 16 wavefronts' counters take 128 KB of LDS.  Fewer make more workgroups that
// read every token: 65536 tokens into 2^20 rows 163 / 176 / 214 us with 2048 / 1024 / 512, 262144 into
// 2^20 346 / 382 / 552; into 2^24 rows 2714 / 2307 / 2884.
constexpr uint32_t kMaxPerBucket = 2048;
constexpr int kPiece = 64;                // sorted positions per window of the long rows
constexpr size_t kMaxRows = (size_t)1 << 24;

struct GroupPlan {
    uint32_t n, v, segments, buckets, log_buckets, per;  // per: table rows per bucket
    // place of table row r in start and count, and the row of a place
    __host__ __device__ uint32_t slot(uint32_t r) const { return (r & (buckets - 1)) * per + (r >> log_buckets); }
    __host__ __device__ uint32_t row(uint32_t slot) const { return slot % per << log_buckets | slot / per; }
};

GroupPlan make_plan(size_t n, size_t v)
{
    GroupPlan p{};
    p.n = (uint32_t)n;
    p.v = (uint32_t)v;
    p.segments = (uint32_t)((n + kSegment - 1) / kSegment);
    if (p.segments == 0) p.segments = 1;
    // one workgroup per compute unit (16384 x 1024 bfloat16 into 50000 rows: 128 / 256 / 512 buckets
    // 40.8 / 40.4 / 43.8 us, 65536 x 2048 142 / 139 / 151); with several segments 64 buckets each fill the
    // chip and read every token a quarter as often (262144 x 1024: 32 / 64 / 256 buckets 235 / 228 / 265
    // us, 2^20 x 256 390 / 411 / 554)
    p.log_buckets = p.segments == 1 ? 8 : 6;
    while (((v + ((size_t)1 << p.log_buckets) - 1) >> p.log_buckets) > kMaxPerBucket) ++p.log_buckets;
    p.buckets = 1u << p.log_buckets;
    p.per = (uint32_t)((v + p.buckets - 1) / p.buckets);
    return p;
}

// Workspace: order[n], start[buckets * per], count[buckets * per] (uint32, a bucket's rows side by
// side: scattered over the table's order, their 4-byte writes took as long as the rest of the
// grouping); with several segments the counts [segment][bucket][per] and the buckets' totals
// [segment][bucket]; the pieces' sums [window][2][channels] (float).
struct GroupSpace {
    uint32_t *order, *start, *count, *grouped, *seg_counts, *totals;  // grouped: number of positions in order
    float* pieces;
    size_t bytes;
};

GroupSpace lay_out(const GroupPlan& p, uint32_t channels, void* base)
{
    GroupSpace s{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char* q = static_cast<char*>(base) + at;
        at += round_up(bytes, 256);
        return q;
    };
    s.order = reinterpret_cast<uint32_t*>(take((size_t)p.n * 4));
    s.start = reinterpret_cast<uint32_t*>(take((size_t)p.buckets * p.per * 4));
    s.count = reinterpret_cast<uint32_t*>(take((size_t)p.buckets * p.per * 4));
    s.grouped = reinterpret_cast<uint32_t*>(take(4));
    if (p.segments > 1) {
        s.seg_counts = reinterpret_cast<uint32_t*>(take((size_t)p.segments * p.buckets * p.per * 4));
        s.totals = reinterpret_cast<uint32_t*>(take((size_t)p.segments * p.buckets * 4));
    }
    s.pieces = reinterpret_cast<float*>(take(((size_t)p.n + kPiece - 1) / kPiece * 2 * channels * 4));
    s.bytes = at;
    return s;
}

// Token i as a table row, or v (no row) if it lies outside the table.
template <typename I>
__device__ __forceinline__ uint32_t table_row(const I* __restrict__ tokens, uint32_t i, uint32_t v)
{
    const I t = tokens[i];
    return t >= 0 && t < (I)v ? (uint32_t)t : v;
}

// Rounds of 64 tokens whose loads are in flight together.  Every workgroup looks at every token, so
// what that costs bounds the grouping: per round four vector instructions in the first walk, three
// in the second, the rest on the scalar unit (with branches per lane instead, and one round's loads
// at a time, 65536 tokens took 54 us).
constexpr int kRounds = 16;

// Token as an unsigned number that is at least 2^31 for every token outside a table.
__device__ __forceinline__ uint32_t as_row(int32_t t) { return (uint32_t)t; }
__device__ __forceinline__ uint32_t as_row(int64_t t) { return (uint64_t)t >> 31 ? 0xFFFFFFFFu : (uint32_t)t; }

template <typename I>
__device__ __forceinline__ void load_rounds(const I* __restrict__ tokens, uint32_t base, uint32_t hi, int lane,
                                            uint32_t (&r)[kRounds])
{
    if (base + 64 * kRounds <= hi) {
        I t[kRounds];
#pragma unroll
        for (int u = 0; u < kRounds; ++u) t[u] = tokens[base + lane + u * 64];
#pragma unroll
        for (int u = 0; u < kRounds; ++u) r[u] = as_row(t[u]);
    } else {
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            const uint32_t i = base + lane + u * 64;
            r[u] = i < hi ? as_row(tokens[i]) : 0xFFFFFFFFu;
        }
    }
}

// ------------------------------------------------------------ grouping
// MODE 0: one segment, everything.  MODE 1: counts of (bucket x, segment y) to memory.  MODE 2:
// the positions of (bucket x, segment y), whose first places seg_counts now holds.
template <int MODE, typename I>
__global__ __launch_bounds__(kGroupBlock) void group_kernel(const I* __restrict__ tokens, GroupPlan p,
                                                            uint32_t* __restrict__ order, uint32_t* __restrict__ start,
                                                            uint32_t* __restrict__ count,
                                                            uint32_t* __restrict__ grouped,
                                                            uint32_t* __restrict__ seg_counts,
                                                            uint32_t* __restrict__ totals)
{
    extern __shared__ uint32_t s_cnt[];  // [wavefront][per]
    __shared__ uint32_t s_part[kGroupWaves], s_low[kGroupWaves];
    const uint32_t b = blockIdx.x, seg = blockIdx.y;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint32_t mask = p.buckets - 1;
    for (uint32_t i = threadIdx.x; i < kGroupWaves * p.per; i += kGroupBlock) s_cnt[i] = 0;
    __syncthreads();

    // wavefront w owns tokens [lo, hi) of the segment
    const uint32_t first = seg * kSegment;
    const uint32_t cnt = p.n - first < kSegment ? p.n - first : kSegment;
    const uint32_t m = (((cnt + kGroupWaves - 1) / kGroupWaves) + 63u) & ~63u;
    const uint32_t lo = (uint32_t)uniform((int)(min((uint32_t)w * m, cnt) + first));
    const uint32_t hi = (uint32_t)uniform((int)(min((uint32_t)(w + 1) * m, cnt) + first));
    uint32_t* my = s_cnt + (uint32_t)w * p.per;
    uint32_t lower = 0;  // the wavefront's tokens of smaller buckets
    for (uint32_t base = lo; base < hi; base += 64 * kRounds) {
        uint32_t r[kRounds];
        load_rounds(tokens, base, hi, lane, r);
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            const uint32_t bk = r[u] & mask;
            const uint64_t inside = __builtin_amdgcn_ballot_w64(r[u] < p.v);
            const uint64_t mine = __builtin_amdgcn_ballot_w64(bk == b) & inside;
            if (MODE == 0) lower += __builtin_popcountll(__builtin_amdgcn_ballot_w64(bk < b) & inside);
            if (mine) {
                // LDS adds of many lanes to one word are slow: a round whose lanes hold one token adds once
                const int leader = __builtin_ctzll(mine);
                const uint32_t token = (uint32_t)__builtin_amdgcn_readlane((int)r[u], leader);
                const bool one = (__builtin_amdgcn_ballot_w64(r[u] == token) & mine) == mine;
                if (one ? lane == leader : (bool)(mine >> lane & 1))
                    atomicAdd(my + (r[u] >> p.log_buckets), one ? (uint32_t)__builtin_popcountll(mine) : 1u);
            }
        }
    }
    if (MODE == 0 && lane == 0) s_low[w] = lower;
    __syncthreads();

    // the tokens' totals in this segment and their exclusive scan, each thread a run of them
    const uint32_t run = (p.per + kGroupBlock - 1) / kGroupBlock;
    const uint32_t l0 = min(threadIdx.x * run, p.per), l1 = min(l0 + run, p.per);
    if (MODE == 1) {
        uint32_t sum = 0;
        uint32_t* out = seg_counts + ((size_t)seg * p.buckets + b) * p.per;
        for (uint32_t l = l0; l < l1; ++l) {
            uint32_t c = 0;
            for (int q = 0; q < kGroupWaves; ++q) c += s_cnt[q * p.per + l];
            out[l] = c;
            sum += c;
        }
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
        if (lane == 0) s_part[w] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t t = 0;
            for (int q = 0; q < kGroupWaves; ++q) t += s_part[q];
            totals[(size_t)seg * p.buckets + b] = t;
        }
        return;
    }
    if (MODE == 0) {
        uint32_t sum = 0;
        for (uint32_t l = l0; l < l1; ++l)
            for (int q = 0; q < kGroupWaves; ++q) sum += s_cnt[q * p.per + l];
        uint32_t incl = sum;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t t = __shfl_up(incl, o, 64);
            if (lane >= o) incl += t;
        }
        if (lane == 63) s_part[w] = incl;
        __syncthreads();
        uint32_t at = incl - sum;
        for (int q = 0; q < kGroupWaves; ++q) at += s_low[q] + (q < w ? s_part[q] : 0u);
        for (uint32_t l = l0; l < l1; ++l) {
            const uint32_t begin = at;
            for (int q = 0; q < kGroupWaves; ++q) {
                const uint32_t c = s_cnt[q * p.per + l];
                s_cnt[q * p.per + l] = at;
                at += c;
            }
            start[b * p.per + l] = begin;
            count[b * p.per + l] = at - begin;
        }
        if (b == p.buckets - 1 && threadIdx.x == kGroupBlock - 1) *grouped = at;  // the end of the last token's run
    } else {
        const uint32_t* from = seg_counts + ((size_t)seg * p.buckets + b) * p.per;
        for (uint32_t l = l0; l < l1; ++l) {
            uint32_t at = from[l];
            for (int q = 0; q < kGroupWaves; ++q) {
                const uint32_t c = s_cnt[q * p.per + l];
                s_cnt[q * p.per + l] = at;
                at += c;
            }
        }
    }
    __syncthreads();

    // second walk: the lanes of a round that hold one token take consecutive places
    for (uint32_t base = lo; base < hi; base += 64 * kRounds) {
        uint32_t r[kRounds];
        load_rounds(tokens, base, hi, lane, r);
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            const bool mine = r[u] < p.v && (r[u] & mask) == b;
            uint64_t left = __builtin_amdgcn_ballot_w64(mine);
            while (left) {
                const int leader = __builtin_ctzll(left);
                const uint32_t token = (uint32_t)__builtin_amdgcn_readlane((int)r[u], leader);
                const bool same = mine && r[u] == token;
                const uint64_t eq = __builtin_amdgcn_ballot_w64(same);
                uint32_t at = 0;
                if (lane == leader) at = atomicAdd(my + (token >> p.log_buckets), (uint32_t)__builtin_popcountll(eq));
                at = (uint32_t)__builtin_amdgcn_readlane((int)at, leader);
                if (same) order[at + __builtin_popcountll(eq & ((1ull << lane) - 1))] = base + u * 64 + lane;
                left &= ~eq;
            }
        }
    }
}

// Several segments: bucket x's tokens in all segments.  seg_counts becomes the first place of
// every (segment, token).
__global__ __launch_bounds__(kGroupBlock) void group_places_kernel(GroupPlan p, uint32_t* __restrict__ start,
                                                                   uint32_t* __restrict__ count,
                                                                   uint32_t* __restrict__ grouped,
                                                                   uint32_t* __restrict__ seg_counts,
                                                                   const uint32_t* __restrict__ totals)
{
    __shared__ uint32_t s_part[kGroupWaves], s_low[kGroupWaves];
    const uint32_t b = blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint32_t lower = 0;
    for (uint32_t i = threadIdx.x; i < p.segments * p.buckets; i += kGroupBlock)
        if ((i & (p.buckets - 1)) < b) lower += totals[i];
    for (int o = 32; o > 0; o >>= 1) lower += __shfl_xor(lower, o, 64);
    if (lane == 0) s_low[w] = lower;
    const uint32_t run = (p.per + kGroupBlock - 1) / kGroupBlock;
    const uint32_t l0 = min(threadIdx.x * run, p.per), l1 = min(l0 + run, p.per);
    const size_t step = (size_t)p.buckets * p.per;
    uint32_t* mine = seg_counts + (size_t)b * p.per;
    uint32_t sum = 0;
    for (uint32_t l = l0; l < l1; ++l)
        for (uint32_t s = 0; s < p.segments; ++s) sum += mine[s * step + l];
    uint32_t incl = sum;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t t = __shfl_up(incl, o, 64);
        if (lane >= o) incl += t;
    }
    if (lane == 63) s_part[w] = incl;
    __syncthreads();
    uint32_t at = incl - sum;
    for (int q = 0; q < kGroupWaves; ++q) at += s_low[q] + (q < w ? s_part[q] : 0u);
    for (uint32_t l = l0; l < l1; ++l) {
        const uint32_t begin = at;
        for (uint32_t s = 0; s < p.segments; ++s) {
            const uint32_t c = mine[s * step + l];
            mine[s * step + l] = at;
            at += c;
        }
        start[b * p.per + l] = begin;
        count[b * p.per + l] = at - begin;
    }
    if (b == p.buckets - 1 && threadIdx.x == kGroupBlock - 1) *grouped = at;
}

// ------------------------------------------------------------ sums
// Adds rows order[from .. to) of dout, columns [c, c + V), to acc, one after another; the loads of
// eight rows are in flight together.
template <typename T, int V>
__device__ __forceinline__ void sum_rows(const T* __restrict__ dout, int64_t stride, const uint32_t* __restrict__ order,
                                         uint32_t from, uint32_t to, uint32_t c, float (&acc)[V])
{
    constexpr int U = 8;
    uint32_t i = from;
    for (; i + U <= to; i += U) {
        Pack<T, V> p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = load_pack<T, V>(dout + (int64_t)order[i + u] * stride + c);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += (float)p[u].v[k];
    }
    for (; i < to; ++i) {
        const Pack<T, V> p = load_pack<T, V>(dout + (int64_t)order[i] * stride + c);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += (float)p.v[k];
    }
}

// One launch sums everything but the pieces themselves.  Workgroups below `windows * columns`: window
// x (sorted positions [x * kPiece, ..)), the sums of its parts of rows with more than kPiece
// positions.  At most two such rows touch a window: one that began before it or at its start (slot
// 0), one that begins inside it (slot 1) and reaches its end.  The others: kRows rows of the table per
// wavefront, 64 * V columns; the first position of each is in flight together, as most rows have one
// or none.  Rows of pieces are left to join_kernel.
// Measured (gradient of 4096 x 1024 float32 tokens into 32000 rows / of 65536 x 2048 bfloat16 into
// 50000): kRows 4 36.1 / 139 us, 8 38.0 / 143, 16 37.8 / 165; windows of 32 positions 37.7 / 148 and of
// 128 39.1 / 144 (kRows 8); with ordinary instead of streaming stores 43.2 / 153.
constexpr int kRows = 4;

// A row that nothing reads soon goes past the caches.
template <typename O, int V>
__device__ __forceinline__ void store_stream(O* out, const Pack<O, V>& p)
{
    if constexpr (sizeof(p) % 16 == 0) {
#pragma unroll
        for (size_t i = 0; i < sizeof(p) / 16; ++i)
            __builtin_nontemporal_store(reinterpret_cast<const u32x4*>(&p)[i], reinterpret_cast<u32x4*>(out) + i);
    } else {
        *reinterpret_cast<Pack<O, V>*>(out) = p;
    }
}

template <typename T, typename O, int V>
__device__ __forceinline__ void store_row(O* __restrict__ dtable, uint32_t channels, uint32_t r, uint32_t c, float scale,
                                          int accumulate, float (&acc)[V])
{
    O* out = dtable + (size_t)r * channels + c;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= scale;
    if (accumulate) {
        float had[V];
        unpack(load_pack<O, V>(out), had);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += had[k];
    }
    store_stream(out, pack<O, V>(acc));
}

struct Sums {
    GroupPlan plan;
    uint32_t channels, columns, windows;  // columns: workgroups (of 256 * V columns) per window
    uint32_t workgroups;                  // of sums_kernel
    int64_t stride;
    const uint32_t *order, *start, *count, *grouped;
    float* pieces;
    float scale;
    int accumulate;
};

template <typename T, typename O, typename I, int V>
__global__ __launch_bounds__(256) void sums_kernel(Sums a, const I* __restrict__ tokens, const T* __restrict__ dout,
                                                   O* __restrict__ dtable)
{
    const uint32_t wg = workgroup();
    if (wg >= a.workgroups) return;
    if (wg < a.windows * a.columns) {
        const uint32_t x = wg / a.columns;
        const uint32_t c = (wg % a.columns * 256 + threadIdx.x) * V;
        // places behind the last grouped position (tokens outside the table have none) hold nothing
        const uint32_t lo = x * kPiece;
        const uint32_t grouped = *a.grouped;
        if (lo >= grouped) return;
        const uint32_t hi = min(lo + (uint32_t)kPiece, grouped);
        const uint32_t r0 = table_row(tokens, a.order[lo], a.plan.v), r1 = table_row(tokens, a.order[hi - 1], a.plan.v);
        if (c >= a.channels) return;
#pragma unroll
        for (int slot = 0; slot < 2; ++slot) {
            const uint32_t at = a.plan.slot(slot ? r1 : r0);
            const uint32_t s = a.start[at], n = a.count[at];
            if (n <= (uint32_t)kPiece || (slot == 1) != (s > lo)) continue;
            float acc[V] = {};
            sum_rows<T, V>(dout, a.stride, a.order, max(s, lo), min(s + n, hi), c, acc);
            *reinterpret_cast<Pack<float, V>*>(a.pieces + ((size_t)x * 2 + slot) * a.channels + c) = pack<float, V>(acc);
        }
        return;
    }
    const uint32_t chunks = (a.channels + 64 * V - 1) / (64 * V);
    const uint32_t unit = (wg - a.windows * a.columns) * 4 + (uint32_t)uniform((int)(threadIdx.x >> 6));
    const uint32_t first = unit / chunks * kRows;
    const uint32_t c = (unit % chunks * 64 + (threadIdx.x & 63)) * V;
    const uint32_t slots = a.plan.buckets * a.plan.per;  // rows in the order of start and count
    if (first >= slots || c >= a.channels) return;
    uint32_t s[kRows], n[kRows];
    Pack<T, V> p[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const bool in = first + i < slots;
        n[i] = in ? a.count[first + i] : 0u;
        s[i] = in ? a.start[first + i] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        p[i] = n[i] && n[i] <= (uint32_t)kPiece ? load_pack<T, V>(dout + (int64_t)a.order[s[i]] * a.stride + c) : zero_pack<T, V>();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint32_t r = a.plan.row(first + i);
        if (first + i >= slots || r >= a.plan.v || n[i] > (uint32_t)kPiece || (a.accumulate && n[i] == 0)) continue;
        float acc[V];
        unpack(p[i], acc);
        if (n[i] > 1) sum_rows<T, V>(dout, a.stride, a.order, s[i] + 1, s[i] + n[i], c, acc);
        store_row<T, O, V>(dtable, a.channels, r, c, a.scale, a.accumulate, acc);
    }
}

// Window x: the row of pieces that begins in it, if there is one, from its windows' sums in order.
template <typename T, typename O, typename I, int V>
__global__ __launch_bounds__(256) void join_kernel(Sums a, const I* __restrict__ tokens, O* __restrict__ dtable)
{
    const uint32_t wg = workgroup();
    if (wg >= a.windows * a.columns) return;
    const uint32_t x = wg / a.columns;
    const uint32_t c = (wg % a.columns * 256 + threadIdx.x) * V;
    const uint32_t lo = x * kPiece, grouped = *a.grouped;
    if (lo >= grouped || c >= a.channels) return;
    // it reaches the end of the window, for it is longer than one
    const uint32_t r = table_row(tokens, a.order[min(lo + (uint32_t)kPiece, grouped) - 1], a.plan.v);
    const uint32_t s = a.start[a.plan.slot(r)], n = a.count[a.plan.slot(r)];
    if (n <= (uint32_t)kPiece || s < lo) return;
    const uint32_t last = (s + n - 1) / kPiece;
    // it began before the later windows: slot 0 there
    const auto piece = [&](uint32_t w) { return load_pack<float, V>(a.pieces + (size_t)w * 2 * a.channels + c); };
    float acc[V];
    unpack(load_pack<float, V>(a.pieces + ((size_t)x * 2 + (s > lo ? 1 : 0)) * a.channels + c), acc);
    uint32_t w = x + 1;
    for (; w + 8 <= last + 1; w += 8) {
        Pack<float, V> p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) p[u] = piece(w + u);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += p[u].v[k];
    }
    for (; w <= last; ++w) {
        const Pack<float, V> p = piece(w);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += p.v[k];
    }
    store_row<T, O, V>(dtable, a.channels, r, c, a.scale, a.accumulate, acc);
}

// ------------------------------------------------------------ lookup
// One wavefront per row and block of 4 * 64 * V columns.
template <typename T, typename I, int V>
__global__ __launch_bounds__(256) void lookup_kernel(const I* __restrict__ tokens, uint32_t n,
                                                     const T* __restrict__ table, int64_t stride, uint32_t v,
                                                     uint32_t channels, float scale, T* __restrict__ out)
{
    const uint32_t i = (blockIdx.z * kGridWidth + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (i >= n) return;
    const uint32_t r = (uint32_t)uniform((int)table_row(tokens, i, v));
    const uint32_t c0 = (blockIdx.y * 256 + (threadIdx.x & 63)) * V;
    Pack<T, V> p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t c = c0 + k * 64 * V;
        p[k] = r < v && c < channels ? load_pack<T, V>(table + (int64_t)r * stride + c) : zero_pack<T, V>();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t c = c0 + k * 64 * V;
        if (c >= channels) break;
        float f[V];
        unpack(p[k], f);
        if (r < v) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                f[j] *= scale;
                asm("" : "+v"(f[j]));  // rounded to 32 bits first in every type: float16 has a fused product and rounding
            }
        }
        *reinterpret_cast<Pack<T, V>*>(out + (size_t)i * channels + c) = pack<T, V>(f);
    }
}

// Calls f with the elements per access as an integral constant: 16 bytes, else 4 bytes of a 16-bit
// type, else one element, as channels, strides and pointers allow.  16-bit rows of 590 by one element
// and by two: gradient of 2 tokens into 39746 rows 43.7 and 26.9 us, of 4096 tokens 51.0 and 34.4,
// lookup of 16000 tokens 10.1 and 8.5; an odd 591 stays at 43.3.
template <typename T, typename F>
void with_pack(uint32_t channels, int64_t stride, std::initializer_list<std::pair<const void*, size_t>> arrays, F f)
{
    const auto fits = [&](int v) {
        bool ok = channels % v == 0 && stride % v == 0;
        for (const auto& a : arrays) ok = ok && aligned(a.first, std::min<size_t>(16, v * a.second));
        return ok;
    };
    constexpr int V = 16 / sizeof(T);
    if (fits(V))
        f(std::integral_constant<int, V>());
    else if (sizeof(T) == 2 && fits(2))
        f(std::integral_constant<int, sizeof(T) == 2 ? 2 : 1>());
    else
        f(std::integral_constant<int, 1>());
}

template <typename T, typename I>
scan_status_t run_lookup(const I* tokens, size_t n, const T* table, int64_t stride, size_t v, uint32_t channels,
                         float scale, T* out, hipStream_t s)
{
    with_pack<T>(channels, stride, {{table, sizeof(T)}, {out, sizeof(T)}}, [&](auto pack) {
        constexpr int V = decltype(pack)::value;
        const dim3 rows = grid_of((n + 3) / 4), grid(rows.x, (channels + 256 * V - 1) / (256 * V), rows.y);
        hipLaunchKernelGGL((lookup_kernel<T, I, V>), grid, dim3(256), 0, s, tokens, (uint32_t)n, table, stride, (uint32_t)v,
                           channels, scale, out);
    });
    return launched();
}

template <typename I>
void run_group(const I* tokens, const GroupPlan& p, const GroupSpace& w, hipStream_t s)
{
    const size_t lds = (size_t)kGroupWaves * p.per * 4;
    if (p.segments == 1) {
        hipLaunchKernelGGL((group_kernel<0, I>), dim3(p.buckets), dim3(kGroupBlock), lds, s, tokens, p, w.order, w.start,
                           w.count, w.grouped, w.seg_counts, w.totals);
        return;
    }
    hipLaunchKernelGGL((group_kernel<1, I>), dim3(p.buckets, p.segments), dim3(kGroupBlock), lds, s, tokens, p, w.order,
                       w.start, w.count, w.grouped, w.seg_counts, w.totals);
    hipLaunchKernelGGL(group_places_kernel, dim3(p.buckets), dim3(kGroupBlock), 0, s, p, w.start, w.count, w.grouped, w.seg_counts,
                       w.totals);
    hipLaunchKernelGGL((group_kernel<2, I>), dim3(p.buckets, p.segments), dim3(kGroupBlock), lds, s, tokens, p, w.order,
                       w.start, w.count, w.grouped, w.seg_counts, w.totals);
}

// The grouping, the sums and the join.
template <typename T, typename O, int V, typename I>
scan_status_t run_sums(const I* tokens, const GroupPlan& p, const GroupSpace& w, const T* dout, int64_t stride,
                       uint32_t channels, float scale, int accumulate, O* dtable, hipStream_t s)
{
    const uint32_t columns = (channels + 256 * V - 1) / (256 * V), chunks = (channels + 64 * V - 1) / (64 * V);
    const uint32_t windows = p.n > kPiece ? (p.n + kPiece - 1) / kPiece : 0;  // else no row is that long
    const uint64_t units = ((uint64_t)p.buckets * p.per + kRows - 1) / kRows * chunks;
    const uint64_t workgroups = (uint64_t)windows * columns + (units + 3) / 4;
    if (workgroups > kMostInGrid / 4) return SCAN_ERR_INVALID;  // the kernel counts wavefronts
    run_group(tokens, p, w, s);
    const Sums a{p,       channels, columns, windows,   (uint32_t)workgroups, stride, w.order,
                 w.start, w.count,  w.grouped, w.pieces, scale,                accumulate};
    hipLaunchKernelGGL((sums_kernel<T, O, I, V>), grid_of(workgroups), dim3(256), 0, s, a, tokens, dout, dtable);
    if (windows)
        hipLaunchKernelGGL((join_kernel<T, O, I, V>), grid_of((uint64_t)windows * columns), dim3(256), 0, s, a, tokens, dtable);
    return launched();
}

template <typename T, typename O, typename I>
scan_status_t run_grad(const I* tokens, size_t n, const T* dout, int64_t stride, size_t v, uint32_t channels, float scale,
                       int accumulate, O* dtable, void* workspace, hipStream_t s)
{
    const GroupPlan p = make_plan(n, v);
    const GroupSpace w = lay_out(p, channels, workspace);
    scan_status_t st = SCAN_OK;
    with_pack<T>(channels, stride, {{dout, sizeof(T)}, {dtable, sizeof(O)}}, [&](auto pack) {
        st = run_sums<T, O, decltype(pack)::value>(tokens, p, w, dout, stride, channels, scale, accumulate, dtable, s);
    });
    return st;
}

bool valid_tokens(const void* tokens, int token_bytes, size_t n)
{
    return (token_bytes == 4 || token_bytes == 8) && n < ((size_t)1 << 31) &&
           (n == 0 || (tokens && aligned(tokens, (size_t)token_bytes)));
}

constexpr uint32_t kMaxChannels = 1u << 20;

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

scan_status_t embedding_lookup(seq_dtype_t dtype, const void* tokens, int token_bytes, size_t n, const void* table,
                               int64_t table_stride, size_t n_rows, uint32_t channels, float scale, void* out,
                               void* stream)
{
    if (!valid_dtype(dtype)) return SCAN_ERR_UNSUPPORTED;
    if (!valid_tokens(tokens, token_bytes, n)) return SCAN_ERR_INVALID;
    if (n_rows < 1 || n_rows > kMaxRows || channels < 1 || channels > kMaxChannels) return SCAN_ERR_INVALID;
    if (n == 0) return SCAN_OK;
    const size_t es = dtype_size(dtype);
    if (!table || !out || !aligned(table, es) || !aligned(out, es)) return SCAN_ERR_INVALID;
    if (table_stride < (int64_t)channels || table_stride > ((int64_t)1 << 31)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(out, n, channels, channels, es)};
    const Range ins[] = {range(tokens, n * token_bytes), range(table, n_rows, table_stride, channels, es)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        const T* t = static_cast<const T*>(table);
        const hipStream_t s = static_cast<hipStream_t>(stream);
        return token_bytes == 4
                   ? run_lookup(static_cast<const int32_t*>(tokens), n, t, table_stride, n_rows, channels, scale,
                                static_cast<T*>(out), s)
                   : run_lookup(static_cast<const int64_t*>(tokens), n, t, table_stride, n_rows, channels, scale,
                                static_cast<T*>(out), s);
    });
}

size_t embedding_grad_workspace(size_t n, size_t n_rows, uint32_t channels)
{
    if (n >= ((size_t)1 << 31) || n_rows < 1 || n_rows > kMaxRows || channels > kMaxChannels) return 0;
    return lay_out(make_plan(n, n_rows), channels, nullptr).bytes;
}

scan_status_t embedding_grad(seq_dtype_t dtype, seq_dtype_t grad_dtype, const void* tokens, int token_bytes, size_t n,
                             const void* dout, int64_t dout_stride, size_t n_rows, uint32_t channels, float scale,
                             int accumulate, void* dtable, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_dtype(dtype) || (grad_dtype != dtype && grad_dtype != SEQ_F32)) return SCAN_ERR_UNSUPPORTED;
    if (!valid_tokens(tokens, token_bytes, n)) return SCAN_ERR_INVALID;
    if (n_rows < 1 || n_rows > kMaxRows || channels < 1 || channels > kMaxChannels) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(dtype), gs = dtype_size(grad_dtype), need = embedding_grad_workspace(n, n_rows, channels);
    if (!dtable || !aligned(dtable, gs)) return SCAN_ERR_INVALID;
    if (n > 0 && (!dout || !aligned(dout, es) || dout_stride < (int64_t)channels || dout_stride > ((int64_t)1 << 31)))
        return SCAN_ERR_INVALID;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return SCAN_ERR_INVALID;
    const Range outs[] = {range(dtable, n_rows, channels, channels, gs), range(workspace, need)};
    const Range ins[] = {range(tokens, n * token_bytes), range(dout, n, dout_stride, channels, es)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        const T* d = static_cast<const T*>(dout);
        const hipStream_t s = static_cast<hipStream_t>(stream);
        const auto go = [&](auto* tok) {
            return grad_dtype == dtype ? run_grad(tok, n, d, dout_stride, n_rows, channels, scale, accumulate,
                                                  static_cast<T*>(dtable), workspace, s)
                                       : run_grad(tok, n, d, dout_stride, n_rows, channels, scale, accumulate,
                                                  static_cast<float*>(dtable), workspace, s);
        };
        return token_bytes == 4 ? go(static_cast<const int32_t*>(tokens)) : go(static_cast<const int64_t*>(tokens));
    });
}

}  // extern "C"
