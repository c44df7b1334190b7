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
//   pieces: rows with more than kPiece positions are cut along the windows of
//           kPiece sorted positions; each window's part of such a row is
//           summed by a wavefront of its own (32 bits, to the workspace).
//   rows:   every row of the table: the sum of its positions, or of its
//           pieces, or zero.
#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr int kGroupBlock = 1024;
constexpr int kGroupWaves = kGroupBlock / 64;
constexpr uint32_t kSegment = 65536;      // tokens that one pass of the grouping kernels reads
constexpr uint32_t kMaxPerBucket = 2048;  // table rows per bucket: 16 wavefronts' counters take 128 KB of LDS
constexpr int kPiece = 64;                // sorted positions per window of the long rows
constexpr size_t kMaxRows = (size_t)1 << 24;

struct GroupPlan {
    uint32_t n, v, segments, buckets, log_buckets, per;  // per: table rows per bucket
};

GroupPlan make_plan(size_t n, size_t v)
{
    GroupPlan p{};
    p.n = (uint32_t)n;
    p.v = (uint32_t)v;
    p.segments = (uint32_t)((n + kSegment - 1) / kSegment);
    if (p.segments == 0) p.segments = 1;
    // one workgroup per compute unit; with several segments 64 buckets each fill the chip and
    // read every token a quarter as often
    p.log_buckets = p.segments == 1 ? 8 : 6;
    while (((v + ((size_t)1 << p.log_buckets) - 1) >> p.log_buckets) > kMaxPerBucket) ++p.log_buckets;
    p.buckets = 1u << p.log_buckets;
    p.per = (uint32_t)((v + p.buckets - 1) / p.buckets);
    return p;
}

// Workspace: order[n], start[v], count[v] (uint32); with several segments the counts
// [segment][bucket][per] and the buckets' totals [segment][bucket]; the pieces' sums
// [window][2][channels] (float).
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
    s.start = reinterpret_cast<uint32_t*>(take((size_t)p.v * 4));
    s.count = reinterpret_cast<uint32_t*>(take((size_t)p.v * 4));
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
    const uint32_t lo = min((uint32_t)w * m, cnt) + first, hi = min((uint32_t)(w + 1) * m, cnt) + first;
    uint32_t* my = s_cnt + (uint32_t)w * p.per;
    uint32_t lower = 0;  // tokens of smaller buckets, in this lane
#pragma unroll 4
    for (uint32_t i = lo + lane; i < hi; i += 64) {
        const uint32_t r = table_row(tokens, i, p.v);
        if (r < p.v) {
            const uint32_t bk = r & mask;
            if (bk == b) atomicAdd(my + (r >> p.log_buckets), 1u);
            lower += bk < b;
        }
    }
    if (MODE == 0) {
        for (int o = 32; o > 0; o >>= 1) lower += __shfl_xor(lower, o, 64);
        if (lane == 0) s_low[w] = lower;
    }
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
            const uint32_t row = (l << p.log_buckets) | b;
            const uint32_t begin = at;
            for (int q = 0; q < kGroupWaves; ++q) {
                const uint32_t c = s_cnt[q * p.per + l];
                s_cnt[q * p.per + l] = at;
                at += c;
            }
            if (row < p.v) {
                start[row] = begin;
                count[row] = at - begin;
            }
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
    for (uint32_t base = lo; base < hi; base += 64) {
        const uint32_t i = base + lane;
        const uint32_t r = i < hi ? table_row(tokens, i, p.v) : p.v;
        const bool mine = r < p.v && (r & mask) == b;
        uint64_t left = __builtin_amdgcn_ballot_w64(mine);
        while (left) {
            const int leader = __builtin_ctzll(left);
            const uint32_t token = (uint32_t)__builtin_amdgcn_readlane((int)r, leader);
            const bool same = mine && r == token;
            const uint64_t eq = __builtin_amdgcn_ballot_w64(same);
            uint32_t* place = my + (token >> p.log_buckets);
            const uint32_t at = *place;
            if (same) order[at + __builtin_popcountll(eq & ((1ull << lane) - 1))] = i;
            wave_sync();
            if (lane == leader) *place = at + (uint32_t)__builtin_popcountll(eq);
            wave_sync();
            left &= ~eq;
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
        const uint32_t row = (l << p.log_buckets) | b;
        const uint32_t begin = at;
        for (uint32_t s = 0; s < p.segments; ++s) {
            const uint32_t c = mine[s * step + l];
            mine[s * step + l] = at;
            at += c;
        }
        if (row < p.v) {
            start[row] = begin;
            count[row] = at - begin;
        }
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

// Window x (sorted positions [x * kPiece, ..)): the sums of its parts of rows with more than
// kPiece positions.  At most two such rows touch a window: one that began before it or at its
// start (slot 0), one that begins inside it (slot 1) and reaches its end.
template <typename T, typename I, int V>
__global__ __launch_bounds__(256) void piece_kernel(const I* __restrict__ tokens, const T* __restrict__ dout,
                                                    int64_t stride, uint32_t v, uint32_t channels,
                                                    const uint32_t* __restrict__ order,
                                                    const uint32_t* __restrict__ start,
                                                    const uint32_t* __restrict__ count, const uint32_t* __restrict__ grouped_at,
                                                    float* __restrict__ pieces)
{
    const uint32_t x = blockIdx.x;
    const uint32_t c = (blockIdx.y * 256 + threadIdx.x) * V;
    // places behind the last grouped position (tokens outside the table have none) hold nothing
    const uint32_t lo = x * kPiece;
    const uint32_t grouped = *grouped_at;
    if (lo >= grouped) return;
    const uint32_t hi = min(lo + (uint32_t)kPiece, grouped);
    const uint32_t r0 = table_row(tokens, order[lo], v), r1 = table_row(tokens, order[hi - 1], v);
    if (c >= channels) return;
#pragma unroll
    for (int slot = 0; slot < 2; ++slot) {
        const uint32_t r = slot ? r1 : r0;
        const uint32_t s = start[r], n = count[r];
        if (n <= (uint32_t)kPiece || (slot == 1) != (s > lo)) continue;
        float acc[V] = {};
        sum_rows<T, V>(dout, stride, order, max(s, lo), min(s + n, hi), c, acc);
        float* out = pieces + ((size_t)x * 2 + slot) * channels + c;
#pragma unroll
        for (int k = 0; k < V; ++k) out[k] = acc[k];
    }
}

// Four rows of the table, one per wavefront: columns [c, c + V) per lane.
template <typename T, typename O, int V>
__global__ __launch_bounds__(256) void rows_kernel(const T* __restrict__ dout, int64_t stride, uint32_t v,
                                                  uint32_t channels, const uint32_t* __restrict__ order,
                                                  const uint32_t* __restrict__ start, const uint32_t* __restrict__ count,
                                                  const float* __restrict__ pieces, float scale, int accumulate,
                                                  O* __restrict__ dtable)
{
    const uint32_t r = blockIdx.x * 4 + (threadIdx.x >> 6);
    const uint32_t c = (blockIdx.y * 64 + (threadIdx.x & 63)) * V;
    if (r >= v || c >= channels) return;
    const uint32_t n = (uint32_t)uniform((int)count[r]), s = (uint32_t)uniform((int)start[r]);
    if (accumulate && n == 0) return;
    float acc[V] = {};
    if (n <= (uint32_t)kPiece) {
        sum_rows<T, V>(dout, stride, order, s, s + n, c, acc);
    } else {
        const uint32_t last = (s + n - 1) / kPiece;
        for (uint32_t x = s / kPiece; x <= last; ++x) {
            const float* p = pieces + ((size_t)x * 2 + (s > x * kPiece ? 1 : 0)) * channels + c;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += p[k];
        }
    }
    O* out = dtable + (size_t)r * channels + c;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= scale;
    if (accumulate) {
        float had[V];
        unpack(load_pack<O, V>(out), had);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += had[k];
    }
    *reinterpret_cast<Pack<O, V>*>(out) = pack<O, V>(acc);
}

// ------------------------------------------------------------ lookup
// One wavefront per row and block of 4 * 64 * V columns.
template <typename T, typename I, int V>
__global__ __launch_bounds__(256) void lookup_kernel(const I* __restrict__ tokens, uint32_t n,
                                                     const T* __restrict__ table, int64_t stride, uint32_t v,
                                                     uint32_t channels, float scale, T* __restrict__ out)
{
    const uint32_t i = blockIdx.x * 4 + (threadIdx.x >> 6);
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

template <typename T, typename I>
scan_status_t run_lookup(const I* tokens, size_t n, const T* table, int64_t stride, size_t v, uint32_t channels,
                         float scale, T* out, hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const bool vec = channels % V == 0 && stride % V == 0 && aligned(table, 16) && aligned(out, 16);
    const dim3 grid((unsigned)((n + 3) / 4), (channels + 256 * (vec ? V : 1) - 1) / (256 * (vec ? V : 1)));
    if (vec)
        hipLaunchKernelGGL((lookup_kernel<T, I, V>), grid, dim3(256), 0, s, tokens, (uint32_t)n, table, stride,
                           (uint32_t)v, channels, scale, out);
    else
        hipLaunchKernelGGL((lookup_kernel<T, I, 1>), grid, dim3(256), 0, s, tokens, (uint32_t)n, table, stride,
                           (uint32_t)v, channels, scale, out);
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

template <typename T, typename O, int V, typename I>
void run_sums(const I* tokens, const GroupPlan& p, const GroupSpace& w, const T* dout, int64_t stride,
              uint32_t channels, float scale, int accumulate, O* dtable, hipStream_t s)
{
    if (p.n > kPiece)  // otherwise no row is that long
        hipLaunchKernelGGL((piece_kernel<T, I, V>), dim3((p.n + kPiece - 1) / kPiece, (channels + 256 * V - 1) / (256 * V)),
                           dim3(256), 0, s, tokens, dout, stride, p.v, channels, w.order, w.start, w.count, w.grouped,
                           w.pieces);
    hipLaunchKernelGGL((rows_kernel<T, O, V>), dim3((p.v + 3) / 4, (channels + 64 * V - 1) / (64 * V)), dim3(256), 0, s,
                       dout, stride, p.v, channels, w.order, w.start, w.count, w.pieces, scale, accumulate, dtable);
}

template <typename T, typename O, typename I>
scan_status_t run_grad(const I* tokens, size_t n, const T* dout, int64_t stride, size_t v, uint32_t channels, float scale,
                       int accumulate, O* dtable, void* workspace, hipStream_t s)
{
    const GroupPlan p = make_plan(n, v);
    const GroupSpace w = lay_out(p, channels, workspace);
    run_group(tokens, p, w, s);
    constexpr int V = 16 / sizeof(T);
    if (channels % V == 0 && stride % V == 0 && aligned(dout, 16) && aligned(dtable, 16))
        run_sums<T, O, V>(tokens, p, w, dout, stride, channels, scale, accumulate, dtable, s);
    else
        run_sums<T, O, 1>(tokens, p, w, dout, stride, channels, scale, accumulate, dtable, s);
    return launched();
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
