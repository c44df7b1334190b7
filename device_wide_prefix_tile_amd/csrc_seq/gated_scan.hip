// Gated linear recurrence: for every channel
//   f = sigmoid(decay_gate), g = sigmoid(input_gate), a = exp(rate f), w = sqrt(1 - a^2)
//   h[t] = a h[t-1] + w g x[t],  y[t] = h[t]
// its gradient, and its form for single tokens.
//
// A scan of real affine maps h -> a h + b, one per row and channel, that is read once and written once: 8
// bytes per element forwards in 16 bits, 14 backwards (the states are made again), against some 35 vector
// instructions, six of them transcendental, forwards and twice as many backwards.
//
// Layout.  A workgroup takes a tile of kTileRows rows by 64 V channels; each of its wavefronts some consecutive
// rows of it, each lane V channels.  A wavefront makes its rows' maps in registers and composes them;
// the wavefronts' maps go through LDS, the tiles' through memory; then every wavefront walks its rows
// from the state that reaches them, as a sequential scan would, and stores them.
//
// Single pass.  Tiles are taken in order (a counter), every tile publishes the composed map of its rows
// and waits for those of the tiles before it in its run: a sequence, or all packed rows.  Floating-point results must
// not depend on which of them are there first, so the order of compositions is fixed: a run's tiles form groups of
// kGroup, the state at a group's start is published by the last tile of the group before it, and a tile applies the
// maps of the earlier tiles of its own group to that state one after another.  A published value is its own flag:
// the words hold a pattern beforehand (written by a small launch in front) that no published value has.  A tile only
// waits for tiles with smaller numbers, whose workgroups already run, so every wait ends.
//
// Packed sequences are segments: a row that begins one starts from the initial state; a tile looks back
// no further than to the tile in which its first row's sequence begins.  The gradient is the same
// scan from the other end.
#include <atomic>

#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr uint32_t kMaxChannels = 1u << 20;
// Rows of a wavefront (the forward pass saves the state before every such rows for the gradient) and wavefronts of a
// workgroup.  4 / 8 wavefronts: forward of 8 x 2048 x 4096 bfloat16 135 / 125 us, its gradient 266 / 215, forward of
// 16384 x 2048 float16 116 / 80.
constexpr int kRows = 8;
constexpr int kWaves = 8;
constexpr uint32_t kTileRows = kRows * kWaves;
// Tiles of a group.  Few make the chain of groups long, many make more maps to read and to wait for: 4 / 8 / 12 / 16 forward of
// 16384 x 2048 float16 96 / 80 / 91 / 91 us, of 8 x 2048 x 4096 bfloat16 124 / 125 / 164 / 170.
constexpr uint32_t kGroup = 8;
constexpr uint32_t kChannelPad = 256;  // channels of a tile in the workspace and the saved states: a multiple of this
constexpr uint32_t kEmptyStep = 32;    // workgroups that look for empty sequences, in all
// Looks of a wait before it gives up, some seconds, yields NaN and sets the device's word.
std::atomic<uint32_t> g_spin_limit{1u << 22};
__device__ uint32_t g_gave_up;

// The rows cut into tiles.  Sequences of one length are runs of `run` tiles each, the last of which may have
// fewer rows; packed sequences are one run.  Tiles are numbered over all runs' first tiles, then all second ones, so
// that few tiles of a run are in work at the same time and most find what they wait for.
struct Cut {
    Sequences seqs;
    uint32_t channels, padded, runs, run, run_rows, tiles, groups;  // tiles: in all; groups: per run
};

Cut make_cut(uint32_t channels, uint64_t rows, uint64_t seqs, const int32_t* offsets)
{
    Cut c{};
    c.seqs = Sequences{offsets, (uint32_t)rows, (uint32_t)seqs, seqs ? (uint32_t)(rows / seqs) : 0u};
    c.channels = channels;
    c.padded = (uint32_t)round_up(channels, kChannelPad);
    // sequences that would leave more than half of a tile empty share tiles, as packed ones do
    const bool own = !offsets && c.seqs.len >= kTileRows / 2;
    c.runs = own ? (uint32_t)seqs : 1;
    c.run_rows = own ? c.seqs.len : (uint32_t)rows;
    c.run = (c.run_rows + kTileRows - 1) / kTileRows;
    c.tiles = c.runs * c.run;
    c.groups = (c.run + kGroup - 1) / kGroup;
    return c;
}

// Workspace: the tile counter; with several tiles to a run their maps [tile][padded] and the states at the groups' starts
// [run][group][padded]; the gradient's sums for the rates [tile][padded].  Tile: run by run.
struct Space {
    uint32_t* counter;
    uint64_t* maps;
    uint32_t* starts;
    float* rates;
    size_t bytes;
};

Space lay_out(const Cut& c, bool grad, void* base)
{
    Space s{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        char* q = static_cast<char*>(base) + at;
        at += round_up(bytes, 256);
        return q;
    };
    s.counter = reinterpret_cast<uint32_t*>(take(256));
    if (c.run > 1) {
        s.maps = reinterpret_cast<uint64_t*>(take((size_t)c.tiles * c.padded * 8));
        s.starts = reinterpret_cast<uint32_t*>(take((size_t)c.runs * c.groups * c.padded * 4));
    }
    if (grad) s.rates = reinterpret_cast<float*>(take((size_t)c.tiles * c.padded * 4));
    s.bytes = at;
    return s;
}

// ------------------------------------------------------------ published values
constexpr uint32_t kUnset = 0xFFFFFFFFu;  // a NaN that publish() does not write

__device__ __forceinline__ uint32_t publishable(float v)
{
    return v == v ? __builtin_bit_cast(uint32_t, v) : 0x7FC00000u;
}
__device__ __forceinline__ void publish_map(uint64_t* p, float a, float h)
{
    const uint64_t word = (uint64_t)publishable(h) << 32 | publishable(a);
    __hip_atomic_store(p, word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(uint32_t* p, float h)
{
    __hip_atomic_store(p, publishable(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t peek(const uint32_t* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// V floats at an address of any alignment that floats have.
template <int V>
__device__ __forceinline__ Pack<float, V> load_pack_floats(const float* p)
{
    Pack<float, V> f;
#pragma unroll
    for (int j = 0; j < V; ++j) f.v[j] = p[j];
    return f;
}

// What the words hold before the scan, and the counter.
__global__ __launch_bounds__(256) void unset_kernel(uint32_t* counter, uint64_t* maps, uint64_t n_maps, uint32_t* starts,
                                                    uint64_t n_starts)
{
    // two values per access; both counts are multiples of kChannelPad
    const uint64_t i = ((uint64_t)workgroup() * 256 + threadIdx.x) * 2;
    if (i == 0) *counter = 0;
    const u32x4 unset = {kUnset, kUnset, kUnset, kUnset};
    if (i < n_maps) *reinterpret_cast<u32x4*>(maps + i) = unset;
    if (i < n_starts) *reinterpret_cast<uint64_t*>(starts + i) = ~0ull;
}

// The state (STEP 1; -1: the gradient, from behind) that reaches tile k of the lane's channel.  `first` is the tile in
// which the sequence begins (ends), whose map needs no state.  maps, starts: the run's of that channel, `pitch` words apart.
template <int STEP>
__device__ __forceinline__ float carry(const uint64_t* maps, const uint32_t* starts, uint32_t pitch, uint32_t k, uint32_t first,
                                       uint32_t spin_limit)
{
    constexpr int N = kGroup - 1;
    // the tiles of k's group on the way to k: n of them, from `from` on
    const uint32_t g = k / kGroup;
    const bool inside = first / kGroup == g;
    const uint32_t from = inside ? first : STEP > 0 ? g * kGroup : g * kGroup + kGroup - 1;
    const int n = (int)(STEP > 0 ? k - from : from - k);
    // starts[g]: the state before group g's first tile; backwards, the gradient behind its last one
    const uint32_t* start = starts + (uint64_t)g * pitch;
    const auto map = [&](int i) { return maps + (uint64_t)(from + (uint32_t)(i * STEP)) * pitch; };
    uint64_t v[N] = {};
    uint32_t h0 = 0;
    bool all = false;
    for (uint32_t polls = 0; !all && polls < spin_limit; ++polls) {
        if (polls) {
            // One load asks for all: lane i for the i-th map of the wavefront's first channel, one more for the start.
            const int lane = threadIdx.x & 63;
            uint32_t seen = 0;
            if (lane < n) seen = (uint32_t)peek(map(lane) - lane);
            if (lane == n && !inside) seen = peek(start - lane);
            if (__builtin_amdgcn_ballot_w64(seen == kUnset)) {
                __builtin_amdgcn_s_sleep(1);
                continue;
            }
        }
        // without branches, which would wait for one load before the next; places beyond n read the last again
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = peek(n ? map(min(i, n - 1)) : maps + (uint64_t)k * pitch);
        if (!inside) h0 = peek(start);
        bool set = h0 != kUnset;
#pragma unroll
        for (int i = 0; i < N; ++i) set = set && ((uint32_t)v[i] != kUnset || n == 0);
        all = __builtin_amdgcn_ballot_w64(!set) == 0;
    }
    float h = __builtin_bit_cast(float, h0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i < n) {
            const float a = __builtin_bit_cast(float, (uint32_t)v[i]), b = __builtin_bit_cast(float, (uint32_t)(v[i] >> 32));
            h = inside && i == 0 ? b : fmaf(a, h, b);
        }
    }
    if (all) return h;
    __hip_atomic_store(&g_gave_up, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_nanf("");
}

// ------------------------------------------------------------ the gates
// 1 - a^2 of a = 2^y.  Near 1 the difference has lost what the series of -2 a sinh(z), z = y ln 2, keeps (its next
// term is below 2^-26 of the sum for |z| <= 1/2).  Above that the rate is positive and the result negative.
__device__ __forceinline__ float one_minus_square(float a, float y)
{
    const float q = y * y;
    constexpr float k0 = -2.0f * kLn2, q1 = kLn2 * kLn2;
    const float s = fmaf(q, fmaf(q, fmaf(q, k0 * q1 * q1 * q1 / 5040, k0 * q1 * q1 / 120), k0 * q1 / 6), k0);
    return y >= -0.5f * kLog2e ? a * y * s : fmaf(-a, a, 1.0f);
}

// The hardware's roots take values below 2^-126 as 0 (the inverse one is infinite then): 1 - a^2 of a nearly closed gate
// is that small, so the roots are taken of 2^24 times as much.  (Forward and gradient of 8 x 2048 x 4096 bfloat16 339 us
// with, 337 without.)
constexpr float kRootScale = 0x1p24f, kRootBack = 0x1p-12f;

// A row's map h -> a h + b; log2_rate: the rate times log2 e.
__device__ __forceinline__ void make_map(float decay, float input, float x, float log2_rate, float& a, float& b)
{
    const float y = log2_rate * sigmoid(decay);
    a = exp2_fast(y);
    b = __builtin_amdgcn_sqrtf(one_minus_square(a, y) * kRootScale) * kRootBack * sigmoid(input) * x;
}

// ------------------------------------------------------------ a wavefront's rows
// kRows rows from one on, below an end: which belong to a sequence, begin one, end one (bits of the row), and in lane i < kRows
// the sequence of row i and its first row and end.
struct Rows {
    uint32_t live, head, tail;
    int seq;
    uint32_t st, en;

    // Row i's sequence's part of a state (sequences x channels).
    __device__ uint64_t state(int i, uint32_t channels) const { return (uint64_t)(uint32_t)__builtin_amdgcn_readlane(seq, i) * channels; }
};

__device__ __forceinline__ Rows rows_at(const Sequences& s, uint32_t r0, uint32_t end, int lane)
{
    Rows q{};
    const uint32_t r = r0 + (uint32_t)lane;
    bool live = false, head = false, tail = false;
    if (lane < kRows && r < end) {
        const int seq = s.find(r);
        if (seq >= 0 && seq < (int)s.count) {
            q.seq = seq;
            q.st = s.start((uint32_t)seq);
            q.en = s.end((uint32_t)seq);
            live = r >= q.st && r < q.en;
            head = live && q.st == r;
            tail = live && q.en == r + 1;
        }
    }
    q.live = (uint32_t)__builtin_amdgcn_ballot_w64(live);
    q.head = (uint32_t)__builtin_amdgcn_ballot_w64(head);
    q.tail = (uint32_t)__builtin_amdgcn_ballot_w64(tail);
    return q;
}

// Unsigned integers of SIZE bytes, one or several side by side.
template <int SIZE>
struct Raw;
template <>
struct Raw<2> {
    using type = uint16_t;
};
template <>
struct Raw<4> {
    using type = uint32_t;
};
template <>
struct Raw<8> {
    using type = uint32_t __attribute__((ext_vector_type(2)));
};
template <>
struct Raw<16> {
    using type = u32x4;
};
#define DWPT_GLOBAL __attribute__((address_space(1)))

// Rows one after another: the address of the present one, the same for all lanes.  Hidden from the compiler it stays
// in scalar registers and is stepped by an addition (else rows' addresses are products, and sums with the lane's offset in
// vector registers: 6 of 50 vector instructions per element forwards).
template <typename T, int V>
struct Walk {
    using R = typename Raw<V * sizeof(T)>::type;
    DWPT_GLOBAL char* row;
    int64_t step;

    __device__ Walk(const void* base, int64_t stride, uint32_t r) : step(stride * (int64_t)sizeof(T))
    {
        row = (DWPT_GLOBAL char*)const_cast<void*>(base) + (int64_t)r * step;
        asm("" : "+s"(row));
    }
    __device__ void next()
    {
        row += step;
        asm("" : "+s"(row));
    }
    __device__ void back()
    {
        row -= step;
        asm("" : "+s"(row));
    }
    // V columns from `at` bytes behind the row's start on.  Every value is used once, past the caches: forward of 8 x
    // 2048 x 4096 bfloat16 130 -> 125 us, its gradient 220 -> 215, gradient of 8 x 2048 x 1024 float32 139 -> 122.
    __device__ Pack<T, V> load(uint32_t at) const
    {
        return __builtin_bit_cast(Pack<T, V>, __builtin_nontemporal_load((const DWPT_GLOBAL R*)(row + at)));
    }
    __device__ void store(uint32_t at, const float (&f)[V]) const
    {
        __builtin_nontemporal_store(__builtin_bit_cast(R, (pack<T, V>(f))), (DWPT_GLOBAL R*)(row + at));
    }
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_at(const void* base, int64_t stride, uint32_t r, uint32_t at)
{
    return Walk<T, V>(base, stride, r).load(at);
}

// The rows' V columns; in place of a row of no sequence the first one of a sequence is read.
template <bool PLAIN, typename T, int V>
__device__ __forceinline__ void load_rows(Pack<T, V> (&out)[kRows], const void* base, int64_t stride, uint32_t r0, const Rows& q,
                                          uint32_t at)
{
    if (PLAIN) {
        Walk<T, V> row(base, stride, r0);
#pragma unroll
        for (int i = 0; i < kRows; ++i, row.next()) out[i] = row.load(at);
        return;
    }
    const int first = __builtin_ctz(q.live);
#pragma unroll
    for (int i = 0; i < kRows; ++i) out[i] = load_at<T, V>(base, stride, r0 + (uint32_t)((q.live >> i & 1) ? i : first), at);
}

// A tile: the k-th one of run r, rows [r0, end).  plain: all kTileRows of them lie in the middle of one sequence
// (nothing is looked at row by row).  first, last: the tiles of the run in which the sequence of its first row began, that
// of its last row ends, if those are other ones, else -1.
struct Tile {
    uint32_t r, k, r0, end;
    bool plain;
    int first, last;

    __device__ Tile(const Cut& c, uint32_t number, bool backwards) : plain(false), first(-1), last(-1)
    {
        r = number % c.runs;
        k = backwards ? c.run - 1 - number / c.runs : number / c.runs;
        const Sequences& s = c.seqs;
        const uint32_t row0 = r * c.run_rows;
        r0 = row0 + k * kTileRows;
        end = min(r0 + kTileRows, row0 + c.run_rows);
        const int q = s.find(r0);
        if (q >= 0 && q < (int)s.count) {
            const uint32_t st = s.start((uint32_t)q), en = s.end((uint32_t)q);
            if (st >= row0 && st < r0 && r0 < en) {
                first = (int)((st - row0) / kTileRows);
                plain = en > r0 + kTileRows;
            }
        }
        const uint32_t z = end - 1;
        const int e = plain ? q : s.find(z);
        if (e < 0 || e >= (int)s.count || s.start((uint32_t)e) > z) return;
        const uint32_t en = s.end((uint32_t)e);
        if (en > end && k + 1 < c.run) last = (int)((en - 1 - row0) / kTileRows);
    }
    // Place of the tile's values in arrays [tile][..].
    __device__ uint64_t at(const Cut& c) const { return (uint64_t)r * c.run + k; }
};

// The rows from r0 on of a run that ends before `end`; in place of rows behind it the last one is read.
template <typename T, int V>
__device__ __forceinline__ void load_run(Pack<T, V> (&out)[kRows], const void* base, int64_t stride, uint32_t r0, uint32_t end, bool whole,
                                         uint32_t at)
{
    if (whole) {
        Walk<T, V> row(base, stride, r0);
#pragma unroll
        for (int i = 0; i < kRows; ++i, row.next()) out[i] = row.load(at);
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) out[i] = load_at<T, V>(base, stride, min(r0 + i, end - 1), at);
    }
}

struct Inputs {
    const void *x, *decay, *input;
    int64_t x_stride, decay_stride, input_stride;
    const float *rate, *initial;
};

// A sequence without rows ends in its initial state (backwards: the initial state's gradient is the final one's).
__device__ __forceinline__ void empty_sequences(const Sequences& s, uint32_t channels, uint32_t wg, const float* from, float* to)
{
    for (uint32_t q = wg; q < s.count; q += kEmptyStep) {
        if (s.end(q) > s.start(q)) continue;
        for (uint32_t c = threadIdx.x; c < channels; c += blockDim.x)
            to[(uint64_t)q * channels + c] = from ? from[(uint64_t)q * channels + c] : 0.0f;
    }
}

// ------------------------------------------------------------ forwards
struct Forward {
    Cut cut;
    Inputs in;
    void* y;
    int64_t y_stride;
    float *final_state, *saved;
    Space ws;
    uint32_t spin_limit, blocks;  // blocks: of 64 V channels
};

template <int V>
struct ForwardShared {
    float a[kWaves][64 * V], h[kWaves][64 * V], in[64 * V];
    uint32_t head[kWaves], tile;
};

// 8 x 2048 x 4096 bfloat16: 125 us, 4.3 TB/s (float32 187 us, 5.7 TB/s); vector units busy 69%, 36 vector instructions per
// element, 6 of them transcendental.  What is left is waiting: a round trip through memory takes some 5 us while the
// card streams, and a tile makes two between its loads and its results (an earlier version
// of 129 us took 101 without them, and without their results).  One prompt of 16384 x 2048: 80 us, of which the chain of 32 groups sets most.
template <typename T, int V, bool CHAIN, bool PLAIN>
__device__ __forceinline__ void forward_tile(const Forward& p, ForwardShared<V>& s, const Tile& t, uint32_t c0)
{
    constexpr int C = 64 * V;
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint32_t pitch = p.cut.padded, r0 = t.r0 + (uint32_t)(w * kRows);
    Rows rows{};
    if (!PLAIN) rows = rows_at(p.cut.seqs, r0, t.end, lane);
    const uint32_t mine = c0 + (uint32_t)(lane * V);
    const bool inside = mine < p.cut.channels;
    const uint32_t c = inside ? mine : 0, at = c * (uint32_t)sizeof(T);

    float a[kRows][V], b[kRows][V], am[V], hm[V];
#pragma unroll
    for (int j = 0; j < V; ++j) am[j] = 1.0f, hm[j] = 0.0f;
    if (PLAIN || rows.live) {
        Pack<T, V> x[kRows], dec[kRows], inp[kRows];
        load_rows<PLAIN>(dec, p.in.decay, p.in.decay_stride, r0, rows, at);
        load_rows<PLAIN>(inp, p.in.input, p.in.input_stride, r0, rows, at);
        load_rows<PLAIN>(x, p.in.x, p.in.x_stride, r0, rows, at);
        Pack<float, V> rate = load_pack_floats<V>(p.in.rate + c);
#pragma unroll
        for (int j = 0; j < V; ++j) rate.v[j] *= kLog2e;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                make_map((float)dec[i].v[j], (float)inp[i].v[j], (float)x[i].v[j], rate.v[j], a[i][j], b[i][j]);
            if (!PLAIN && (rows.head >> i & 1)) {
                // from the sequence's initial state: what came before ends here
                if (p.in.initial) {
                    const Pack<float, V> first = load_pack_floats<V>(p.in.initial + rows.state(i, p.cut.channels) + c);
#pragma unroll
                    for (int j = 0; j < V; ++j) b[i][j] = fmaf(a[i][j], first.v[j], b[i][j]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) hm[j] = b[i][j];
            } else if (PLAIN || (rows.live >> i & 1)) {
#pragma unroll
                for (int j = 0; j < V; ++j) am[j] *= a[i][j], hm[j] = fmaf(a[i][j], hm[j], b[i][j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s.a[w][lane * V + j] = am[j], s.h[w][lane * V + j] = hm[j];
    if (!PLAIN && lane == 0) s.head[w] = rows.head;
    __syncthreads();

    if (CHAIN) {
        // one thread per channel: the tile's map, and the state that reaches it
        const uint32_t ch = threadIdx.x;
        if (ch < (uint32_t)C) {
            float am = 1.0f, hm = 0.0f;
            bool any = false;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) {
                const bool cut = !PLAIN && s.head[q] != 0;
                any = any || cut;
                hm = cut ? s.h[q][ch] : fmaf(s.a[q][ch], hm, s.h[q][ch]);
                am *= s.a[q][ch];
            }
            uint64_t* maps = p.ws.maps + (uint64_t)t.r * p.cut.run * pitch + c0 + ch;
            uint32_t* starts = p.ws.starts + (uint64_t)t.r * p.cut.groups * pitch + c0 + ch;
            publish_map(maps + (uint64_t)t.k * pitch, am, hm);
            const float h = PLAIN || t.first >= 0 ? carry<1>(maps, starts, pitch, t.k, (uint32_t)t.first, p.spin_limit) : 0.0f;
            if ((t.k + 1) % kGroup == 0 && t.k + 1 < p.cut.run)
                publish_state(starts + (uint64_t)((t.k + 1) / kGroup) * pitch, any ? hm : fmaf(am, h, hm));
            s.in[ch] = h;
        }
        __syncthreads();
    }
    if (!(PLAIN || rows.live) || !inside) return;

    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = CHAIN ? s.in[lane * V + j] : 0.0f;
    for (int q = 0; q < w; ++q) {
        const bool cut = !PLAIN && s.head[q] != 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = s.h[q][lane * V + j];
            h[j] = cut ? t : fmaf(s.a[q][lane * V + j], h[j], t);
        }
    }
    if (p.saved) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.saved[(t.at(p.cut) * kWaves + w) * pitch + c + j] = h[j];
    }
    Walk<T, V> row(p.y, p.y_stride, r0);
#pragma unroll
    for (int i = 0; i < kRows; ++i, row.next()) {
        if (!PLAIN && !(rows.live >> i & 1)) continue;
        const bool head = !PLAIN && (rows.head >> i & 1);
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = head ? b[i][j] : fmaf(a[i][j], h[j], b[i][j]);
        if (p.y) row.store(at, h);
        if (!PLAIN && p.final_state && (rows.tail >> i & 1)) {
            float* last = p.final_state + rows.state(i, p.cut.channels) + c;
#pragma unroll
            for (int j = 0; j < V; ++j) last[j] = h[j];
        }
    }
}

template <typename T, int V, bool CHAIN>
__global__ __launch_bounds__(kWaves * 64) void forward_kernel(Forward p)
{
    __shared__ ForwardShared<V> s;
    const uint32_t total = p.cut.tiles * p.blocks;
    uint32_t id = workgroup();
    if (id >= total) {
        if (id - total < kEmptyStep && p.final_state)
            empty_sequences(p.cut.seqs, p.cut.channels, id - total, p.in.initial, p.final_state);
        return;
    }
    if (CHAIN) {
        if (threadIdx.x == 0) s.tile = __hip_atomic_fetch_add(p.ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = (uint32_t)uniform((int)s.tile);
    }
    const Tile t(p.cut, id / p.blocks, false);
    if (t.plain)
        forward_tile<T, V, CHAIN, true>(p, s, t, id % p.blocks * (64 * V));
    else
        forward_tile<T, V, CHAIN, false>(p, s, t, id % p.blocks * (64 * V));
}

// ------------------------------------------------------------ backwards
// With dh[t] the gradient of h[t] and e[t] = a[t+1] dh[t+1] what reaches row t from behind:
//   dh = dy + e,  dx = dh w g,  dinput = dh w x g (1 - g)
//   dlog a = dh (a h[t-1] - g x a^2 / w),  drate = sum of dlog a f,  ddecay = dlog a rate f (1 - f)
// What stands beside dh is made on a walk forwards, from the states that the forward pass saved; what reaches
// the wavefront from behind is then known (as forwards, from the other end), and the walk back is one
// product for every result.  Where w is 0 in 32 bits (no decay), its derivative is taken as 0.
// 1 - f of f = 1 / (1 + e), without a difference: e f.  Where e is cut off, f is 0 and so is what this multiplies.
__device__ __forceinline__ float rest(float e, float f) { return fminf(e, 0x1p126f) * f; }

// A sum with what its additions lost: the error of n terms does not grow with n (of 4096 equal ones a plain sum is off by
// some 450 units of 2^-24).  Infinities stay what they are.
struct Sum {
    float s = 0.0f, lost = 0.0f;

    __device__ __forceinline__ void add(float v)
    {
        const float t = s + v, u = t - s;
        lost += (s - (t - u)) + (v - u);
        s = t;
    }
    __device__ __forceinline__ float value() const { return __builtin_fabsf(s) < INFINITY ? s + lost : s; }
};

struct Backward {
    Cut cut;
    Inputs in;
    const void* dy;
    int64_t dy_stride;
    const float *dfinal, *saved;
    void *dx, *ddecay, *dinput;
    int64_t dx_stride, ddecay_stride, dinput_stride;
    float* dinitial;
    Space ws;
    uint32_t spin_limit, blocks;
};

// One row: from the state before it the factors of dh, and the state behind it.
__device__ __forceinline__ void make_factors(float decay, float input, float x, float rate, float& h, float& a, float& fx, float& fi,
                                             float& fr, float& fd)
{
    const float eu = exp2_fast(-kLog2e * decay), es = exp2_fast(-kLog2e * input);
    const float f = rcp_fast(1.0f + eu), g = rcp_fast(1.0f + es), gx = g * x;
    const float y = rate * kLog2e * f;
    a = exp2_fast(y);
    const float w2 = one_minus_square(a, y) * kRootScale, w = __builtin_amdgcn_sqrtf(w2) * kRootBack;
    const float back = w2 == 0.0f ? 0.0f : __builtin_amdgcn_rsqf(w2) * (1.0f / kRootBack);  // 1 / w
    const float b = w * gx;
    fx = w * g;
    fi = b * rest(es, g);
    fr = a * fmaf(-(gx * a), f * back, f * h);
    fd = fr * (rate * rest(eu, f));
    h = fmaf(a, h, b);
}

template <int V>
struct BackwardShared {
    float a[kWaves][64 * V], e[kWaves][64 * V], rate[kWaves][64 * V], in[64 * V];
    uint32_t tail[kWaves], tile;
};

template <typename T, int V, bool CHAIN, bool PLAIN>
__device__ __forceinline__ void backward_tile(const Backward& p, BackwardShared<V>& s, const Tile& t, uint32_t c0)
{
    constexpr int C = 64 * V;
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint32_t pitch = p.cut.padded, r0 = t.r0 + (uint32_t)(w * kRows);
    Rows rows{};
    if (!PLAIN) rows = rows_at(p.cut.seqs, r0, t.end, lane);
    const uint32_t mine = c0 + (uint32_t)(lane * V);
    const bool inside = mine < p.cut.channels;
    const uint32_t c = inside ? mine : 0, at = c * (uint32_t)sizeof(T);
    const auto last_of = [&](int i) {
        return p.dfinal ? load_pack_floats<V>(p.dfinal + rows.state(i, p.cut.channels) + c) : zero_pack<float, V>();
    };

    // factors of dh in its row's results: dx, dinput, the rate's sum, ddecay
    float a[kRows][V], fx[kRows][V], fi[kRows][V], fr[kRows][V], fd[kRows][V];
    Pack<T, V> dy[kRows];
    float am[V], em[V];
#pragma unroll
    for (int j = 0; j < V; ++j) am[j] = 1.0f, em[j] = 0.0f;
    if (PLAIN || rows.live) {
        Pack<T, V> x[kRows], dec[kRows], inp[kRows];
        load_rows<PLAIN>(dec, p.in.decay, p.in.decay_stride, r0, rows, at);
        load_rows<PLAIN>(inp, p.in.input, p.in.input_stride, r0, rows, at);
        load_rows<PLAIN>(x, p.in.x, p.in.x_stride, r0, rows, at);
        load_rows<PLAIN>(dy, p.dy, p.dy_stride, r0, rows, at);
        const Pack<float, V> rate = load_pack_floats<V>(p.in.rate + c);
        Pack<float, V> h = load_pack_floats<V>(p.saved + (t.at(p.cut) * kWaves + w) * pitch + c);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (!PLAIN && (rows.head >> i & 1)) {
                if (p.in.initial)
                    h = load_pack_floats<V>(p.in.initial + rows.state(i, p.cut.channels) + c);
                else
                    h = zero_pack<float, V>();
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                make_factors((float)dec[i].v[j], (float)inp[i].v[j], (float)x[i].v[j], rate.v[j], h.v[j], a[i][j], fx[i][j], fi[i][j],
                             fr[i][j], fd[i][j]);
        }
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            if (!PLAIN && !(rows.live >> i & 1)) continue;
            if (!PLAIN && (rows.tail >> i & 1)) {
                const Pack<float, V> last = last_of(i);
#pragma unroll
                for (int j = 0; j < V; ++j) em[j] = last.v[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) am[j] *= a[i][j], em[j] = a[i][j] * ((float)dy[i].v[j] + em[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s.a[w][lane * V + j] = am[j], s.e[w][lane * V + j] = em[j];
    if (!PLAIN && lane == 0) s.tail[w] = rows.tail;
    __syncthreads();

    if (CHAIN) {
        const uint32_t ch = threadIdx.x;
        if (ch < (uint32_t)C) {
            float am = 1.0f, em = 0.0f;
            bool any = false;
#pragma unroll
            for (int q = kWaves - 1; q >= 0; --q) {
                const bool cut = !PLAIN && s.tail[q] != 0;
                any = any || cut;
                em = cut ? s.e[q][ch] : fmaf(s.a[q][ch], em, s.e[q][ch]);
                am *= s.a[q][ch];
            }
            uint64_t* maps = p.ws.maps + (uint64_t)t.r * p.cut.run * pitch + c0 + ch;
            uint32_t* starts = p.ws.starts + (uint64_t)t.r * p.cut.groups * pitch + c0 + ch;
            publish_map(maps + (uint64_t)t.k * pitch, am, em);
            const float e = PLAIN || t.last >= 0 ? carry<-1>(maps, starts, pitch, t.k, (uint32_t)t.last, p.spin_limit) : 0.0f;
            if (t.k % kGroup == 0 && t.k > 0)
                publish_state(starts + (uint64_t)(t.k / kGroup - 1) * pitch, any ? em : fmaf(am, e, em));
            s.in[ch] = e;
        }
        __syncthreads();
    }

    float acc[V] = {};
    if (PLAIN || rows.live) {
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = CHAIN ? s.in[lane * V + j] : 0.0f;
        for (int q = kWaves - 1; q > w; --q) {
            const bool cut = !PLAIN && s.tail[q] != 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float t = s.e[q][lane * V + j];
                e[j] = cut ? t : fmaf(s.a[q][lane * V + j], e[j], t);
            }
        }
        Walk<T, V> wx(p.dx, p.dx_stride, r0 + kRows - 1), wi(p.dinput, p.dinput_stride, r0 + kRows - 1),
            wd(p.ddecay, p.ddecay_stride, r0 + kRows - 1);
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i, wx.back(), wi.back(), wd.back()) {
            if (!PLAIN && !(rows.live >> i & 1)) continue;
            if (!PLAIN && (rows.tail >> i & 1)) {
                const Pack<float, V> last = last_of(i);
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = last.v[j];
            }
            float ox[V], oi[V], od[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dh = (float)dy[i].v[j] + e[j];
                ox[j] = dh * fx[i][j];
                oi[j] = dh * fi[i][j];
                od[j] = dh * fd[i][j];
                acc[j] = fmaf(dh, fr[i][j], acc[j]);
                e[j] = a[i][j] * dh;
            }
            if (inside) {
                wx.store(at, ox);
                wi.store(at, oi);
                wd.store(at, od);
                if (!PLAIN && p.dinitial && (rows.head >> i & 1)) {
                    float* first = p.dinitial + rows.state(i, p.cut.channels) + c;
#pragma unroll
                    for (int j = 0; j < V; ++j) first[j] = e[j];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s.rate[w][lane * V + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < (uint32_t)C) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) sum += s.rate[q][threadIdx.x];
        p.ws.rates[t.at(p.cut) * pitch + c0 + threadIdx.x] = sum;
    }
}

template <typename T, int V, bool CHAIN>
__global__ __launch_bounds__(kWaves * 64) void backward_kernel(Backward p)
{
    __shared__ BackwardShared<V> s;
    const uint32_t total = p.cut.tiles * p.blocks;
    uint32_t id = workgroup();
    if (id >= total) {
        if (id - total < kEmptyStep && p.dinitial) empty_sequences(p.cut.seqs, p.cut.channels, id - total, p.dfinal, p.dinitial);
        return;
    }
    if (CHAIN) {
        if (threadIdx.x == 0) s.tile = __hip_atomic_fetch_add(p.ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = (uint32_t)uniform((int)s.tile);
    }
    const Tile t(p.cut, id / p.blocks, true);
    if (t.plain)
        backward_tile<T, V, CHAIN, true>(p, s, t, id % p.blocks * (64 * V));
    else
        backward_tile<T, V, CHAIN, false>(p, s, t, id % p.blocks * (64 * V));
}

// With enough runs and channels to fill the chip a workgroup walks through its run's tiles one after another, from the
// last to the first, and nothing passes through memory between tiles: every wavefront composes all wavefronts' maps of
// a tile from LDS, which takes turns between two halves so that one barrier per tile is enough.  The next tile's rows
// are on their way while this one's are finished.  (8 x 2048 x 4096 bfloat16: 215 us, 270 with tiles that wait for one another.
// Forwards the same gained nothing, 125 against 122: its tiles wait less, two workgroups to a compute unit.)
template <typename T, int V>
__global__ __launch_bounds__(kWaves * 64) void backward_run_kernel(Backward p)
{
    constexpr int C = 64 * V;
    __shared__ float s_a[2][kWaves][C], s_e[2][kWaves][C];
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint32_t id = workgroup();
    if (id >= p.cut.runs * p.blocks) return;
    const uint32_t run = id / p.blocks, mine = id % p.blocks * C + (uint32_t)(lane * V), pitch = p.cut.padded;
    const bool inside = mine < p.cut.channels;
    const uint32_t c = inside ? mine : 0, at = c * (uint32_t)sizeof(T);
    const uint32_t row0 = run * p.cut.run_rows, end = row0 + p.cut.run_rows;
    const Pack<float, V> rate = load_pack_floats<V>(p.in.rate + c);
    Pack<float, V> behind = p.dfinal ? load_pack_floats<V>(p.dfinal + (uint64_t)run * p.cut.channels + c) : zero_pack<float, V>();
    Sum acc[V];  // of the tiles' sums
    Pack<T, V> x[kRows], dec[kRows], inp[kRows], dy[kRows];
    Pack<float, V> h;
    const uint32_t whole = p.cut.run_rows / kTileRows;
    const auto load = [&](uint32_t k) {
        const uint32_t r0 = row0 + k * kTileRows + (uint32_t)(w * kRows);
        load_run(dec, p.in.decay, p.in.decay_stride, r0, end, k < whole, at);
        load_run(inp, p.in.input, p.in.input_stride, r0, end, k < whole, at);
        load_run(x, p.in.x, p.in.x_stride, r0, end, k < whole, at);
        load_run(dy, p.dy, p.dy_stride, r0, end, k < whole, at);
        // states that the forward pass did not save (no row behind them) are not used; the first row's is the initial one
        if (r0 != row0)
            h = load_pack_floats<V>(p.saved + (((uint64_t)run * p.cut.run + k) * kWaves + w) * pitch + c);
        else if (p.in.initial)
            h = load_pack_floats<V>(p.in.initial + (uint64_t)run * p.cut.channels + c);
        else
            h = zero_pack<float, V>();
    };
    const auto tile = [&](auto full, uint32_t k) {
        constexpr bool FULL = decltype(full)::value;
        const uint32_t r0 = row0 + k * kTileRows + (uint32_t)(w * kRows);
        const int n = FULL ? kRows : r0 >= end ? 0 : (int)min((uint32_t)kRows, end - r0);
        float a[kRows][V], fx[kRows][V], fi[kRows][V], fr[kRows][V], fd[kRows][V], g[kRows][V], am[V], em[V];
#pragma unroll
        for (int j = 0; j < V; ++j) am[j] = 1.0f, em[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (!FULL && i >= n) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                make_factors((float)dec[i].v[j], (float)inp[i].v[j], (float)x[i].v[j], rate.v[j], h.v[j], a[i][j], fx[i][j], fi[i][j], fr[i][j],
                             fd[i][j]);
                g[i][j] = (float)dy[i].v[j];
            }
        }
        if (k) load(k - 1);
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            if (!FULL && i >= n) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) am[j] *= a[i][j], em[j] = a[i][j] * (g[i][j] + em[j]);
        }
        float(&sa)[kWaves][C] = s_a[k & 1], (&se)[kWaves][C] = s_e[k & 1];
#pragma unroll
        for (int j = 0; j < V; ++j) sa[w][lane * V + j] = am[j], se[w][lane * V + j] = em[j];
        __syncthreads();
        float e[V];
#pragma unroll
        for (int q = kWaves - 1; q >= 0; --q) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                e[j] = q == w ? behind.v[j] : e[j];
                behind.v[j] = fmaf(sa[q][lane * V + j], behind.v[j], se[q][lane * V + j]);
            }
        }
        float part[V] = {};
        Walk<T, V> wx(p.dx, p.dx_stride, r0 + kRows - 1), wi(p.dinput, p.dinput_stride, r0 + kRows - 1),
            wd(p.ddecay, p.ddecay_stride, r0 + kRows - 1);
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i, wx.back(), wi.back(), wd.back()) {
            if (!FULL && i >= n) continue;
            float ox[V], oi[V], od[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dh = g[i][j] + e[j];
                ox[j] = dh * fx[i][j];
                oi[j] = dh * fi[i][j];
                od[j] = dh * fd[i][j];
                part[j] = fmaf(dh, fr[i][j], part[j]);
                e[j] = a[i][j] * dh;
            }
            if (inside) {
                wx.store(at, ox);
                wi.store(at, oi);
                wd.store(at, od);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j].add(part[j]);
        if (p.dinitial && r0 == row0 && inside) {
            float* first = p.dinitial + (uint64_t)run * p.cut.channels + c;
#pragma unroll
            for (int j = 0; j < V; ++j) first[j] = e[j];
        }
    };
    uint32_t k = p.cut.run;
    load(k - 1);
    if (p.cut.run_rows % kTileRows) tile(std::false_type(), --k);
    while (k) tile(std::true_type(), --k);
    // the run's sum for the rates, in the place of its first tile (rates_kernel: one place per run)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) s_a[0][w][lane * V + j] = acc[j].value();
    __syncthreads();
    if (threadIdx.x < (uint32_t)C) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) sum += s_a[0][q][threadIdx.x];
        p.ws.rates[(uint64_t)run * pitch + id % p.blocks * C + threadIdx.x] = sum;
    }
}

// drate: the tiles' (or runs') sums, each of 16 wavefronts every sixteenth.
__global__ __launch_bounds__(1024) void rates_kernel(const float* __restrict__ sums, uint32_t tiles, uint32_t pitch, uint32_t channels,
                                                     float* __restrict__ drate)
{
    __shared__ float s_sum[16][64];
    const uint32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    Sum mine;
    for (uint32_t t = w; t < tiles; t += 16) mine.add(sums[(uint64_t)t * pitch + c]);  // c < pitch, a multiple of 64
    float sum = s_sum[w][lane] = mine.value();
    __syncthreads();
    if (w == 0 && c < channels) {
#pragma unroll
        for (int q = 1; q < 16; ++q) sum += s_sum[q][lane];
        drate[c] = sum;
    }
}

// ------------------------------------------------------------ single tokens
// A wavefront takes 64 V channels of one row.
template <typename T, int V>
__global__ __launch_bounds__(256) void step_kernel(Inputs in, uint32_t rows, uint32_t channels, uint32_t chunks,
                                                   const int32_t* __restrict__ slots, uint32_t n_slots, float* state,
                                                   T* __restrict__ y, int64_t y_stride)
{
    const uint64_t unit = (uint64_t)workgroup() * 4 + (uint32_t)uniform((int)(threadIdx.x >> 6));
    const uint64_t row = unit / chunks;
    if (row >= rows) return;
    const uint32_t c = (uint32_t)(unit % chunks * 64 + (threadIdx.x & 63)) * V;
    const int slot = slots ? slots[row] : (int)row;
    if (slot < 0 || (uint32_t)slot >= n_slots || c >= channels) return;
    const Pack<T, V> x = load_pack<T, V>(static_cast<const T*>(in.x) + (int64_t)row * in.x_stride + c);
    const Pack<T, V> dec = load_pack<T, V>(static_cast<const T*>(in.decay) + (int64_t)row * in.decay_stride + c);
    const Pack<T, V> inp = load_pack<T, V>(static_cast<const T*>(in.input) + (int64_t)row * in.input_stride + c);
    const Pack<float, V> rate = load_pack_floats<V>(in.rate + c);
    float* h = state + (uint64_t)slot * channels + c;
    const Pack<float, V> had = load_pack_floats<V>(h);
    float out[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float a, b;
        make_map((float)dec.v[j], (float)inp.v[j], (float)x.v[j], rate.v[j] * kLog2e, a, b);
        out[j] = fmaf(a, had.v[j], b);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = out[j];
    *reinterpret_cast<Pack<T, V>*>(y + (int64_t)row * y_stride + c) = pack<T, V>(out);
}

// ------------------------------------------------------------ host side
// The most channels per lane, of 4, 2 and 1, that every row can be cut into.  Forward with 4 / 2 / 1: 8 x 2048 x 4096 bfloat16
// 125 / 133 / 215 us, 2048 x 2048 19 / 20 / 25, 16384 x 2048 float16 80 / 79 / 113; float32 rows fill 8 bytes a lane with 2, which
// are the most there: 8 x 2048 x 4096 187 / 237, 8 x 2048 x 1024 61 / 70, 16 x 1024 x 2048 105 / 125 (4, in an earlier version: 2 to
// 5% slower than 2).  The gradient takes 2 at most: 4 do not fit the registers.
template <size_t N>
int channels_per_lane(int dtype, uint32_t channels, const Array (&arrays)[N])
{
    for (int v = 4; v > 1; v /= 2) {
        bool fits = channels % v == 0;
        for (const Array& a : arrays) fits = fits && (!a.p || (a.stride % v == 0 && aligned(a.p, v * dtype_size(dtype))));
        if (fits) return v;
    }
    return 1;
}

scan_status_t check_gated(const gated_scan_args_t& a)
{
    if (!valid_dtype(a.dtype)) return SCAN_ERR_UNSUPPORTED;
    if (a.rows >= ((uint64_t)1 << 31) || a.seqs >= ((uint64_t)1 << 31)) return SCAN_ERR_INVALID;
    if (a.channels < 1 || a.channels > kMaxChannels) return SCAN_ERR_INVALID;
    if (!a.seq_offsets && (a.seqs == 0 ? a.rows != 0 : a.rows % a.seqs != 0)) return SCAN_ERR_INVALID;
    for (const Array& r : {Array{a.x, a.x_stride}, Array{a.decay_gate, a.decay_stride}, Array{a.input_gate, a.input_stride}})
        if (!valid_rows(a.dtype, a.rows, a.channels, r)) return SCAN_ERR_INVALID;
    if (!a.rate) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)a.seq_offsets, (const void*)a.rate, (const void*)a.initial_state, (const void*)a.final_state,
                          (const void*)a.saved})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    return SCAN_OK;
}

Cut cut_of(const gated_scan_args_t& a) { return make_cut(a.channels, a.rows, a.seqs, a.seq_offsets); }

Inputs inputs_of(const gated_scan_args_t& a)
{
    return Inputs{a.x, a.decay_gate, a.input_gate, a.x_stride, a.decay_stride, a.input_stride, a.rate, a.initial_state};
}

// What is waited for, set to unset values.
void unset(const Cut& c, const Space& w, hipStream_t s)
{
    const uint64_t maps = (uint64_t)c.tiles * c.padded, starts = (uint64_t)c.runs * c.groups * c.padded;
    hipLaunchKernelGGL(unset_kernel, grid_of((maps + 511) / 512), dim3(256), 0, s, w.counter, w.maps, maps, w.starts, starts);
}

// Whether the gradient's workgroups walk through whole runs with this many channels per lane: from one workgroup per
// compute unit on.  Tiles / runs: 512 workgroups, float32, 16 x 1024 x 2048 228 / 188 to 202 us, 8 x 2048 x 4096 402 / 394 to 406; 256
// (8 x 2048 x 4096 bfloat16, 2 channels) 270 / 215; 128 (8 x 2048 x 1024 float32) 121 / 134; 16 (one run of 16384 x 2048 float16)
// 146 / 1410.
constexpr uint64_t kRunWorkgroups = 256;
bool by_runs(const Cut& c, uint32_t channels, int per_lane)
{
    const uint32_t blocks = (channels + 64 * per_lane - 1) / (64 * per_lane);
    return !c.seqs.offsets && c.run > 1 && c.run_rows == c.seqs.len && (uint64_t)c.runs * blocks >= kRunWorkgroups;
}

// Calls f(V) with an integral constant.
template <int MOST, class F>
void with_channels(int v, F f)
{
    if (MOST >= 4 && v >= 4)
        f(std::integral_constant<int, MOST >= 4 ? 4 : 2>());
    else if (v >= 2)
        f(std::integral_constant<int, 2>());
    else
        f(std::integral_constant<int, 1>());
}

scan_status_t forward(const gated_scan_args_t& a, hipStream_t s)
{
    Forward p{cut_of(a), inputs_of(a), a.y, a.y_stride, a.final_state, a.saved, {}, g_spin_limit, 0};
    p.ws = lay_out(p.cut, false, a.workspace);
    const Array arrays[] = {{a.x, a.x_stride}, {a.decay_gate, a.decay_stride}, {a.input_gate, a.input_stride}, {a.y, a.y_stride}};
    const int v = channels_per_lane(a.dtype, a.channels, arrays);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t st = SCAN_OK;
        with_channels<std::is_same<T, float>::value ? 2 : 4>(v, [&](auto n) {
            constexpr int V = decltype(n)::value;
            p.blocks = (a.channels + 64 * V - 1) / (64 * V);
            const bool chain = p.cut.run > 1;
            const uint64_t wgs = (uint64_t)p.cut.tiles * p.blocks, extra = a.final_state && a.seqs ? kEmptyStep : 0;
            if (wgs + extra > kMostInGrid) {
                st = SCAN_ERR_INVALID;
                return;
            }
            if (wgs + extra == 0) return;
            if (chain) unset(p.cut, p.ws, s);
            hipLaunchKernelGGL((chain ? forward_kernel<T, V, true> : forward_kernel<T, V, false>), grid_of(wgs + extra),
                               dim3(kWaves * 64), 0, s, p);
        });
        return st == SCAN_OK ? launched() : st;
    });
}

scan_status_t gradient(const gated_scan_grad_args_t& g, hipStream_t s)
{
    const gated_scan_args_t& a = g.args;
    Backward p{cut_of(a), inputs_of(a), g.dy, g.dy_stride, g.dfinal_state, a.saved, g.dx, g.ddecay_gate, g.dinput_gate, g.dx_stride,
               g.ddecay_stride, g.dinput_stride, g.dinitial_state, {}, g_spin_limit, 0};
    p.ws = lay_out(p.cut, true, a.workspace);
    const Array arrays[] = {{a.x, a.x_stride}, {a.decay_gate, a.decay_stride}, {a.input_gate, a.input_stride}, {g.dy, g.dy_stride},
                            {g.dx, g.dx_stride}, {g.ddecay_gate, g.ddecay_stride}, {g.dinput_gate, g.dinput_stride}};
    const int v = channels_per_lane(a.dtype, a.channels, arrays);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t st = SCAN_OK;
        with_channels<2>(v, [&](auto n) {
            constexpr int V = decltype(n)::value;
            // Whole runs: two channels of float32 rows per lane would spill registers; rows of 16 bits take one where two leave too few
            // workgroups: 4 x 2048 x 4096 bfloat16 tiles / runs 143 / 123 us, 8 x 2048 x 2048 149 / 121 to 126.
            constexpr int RV = std::is_same<T, float>::value ? 1 : V;
            const int run_channels = by_runs(p.cut, a.channels, RV) ? RV : 1;
            const bool chain = p.cut.run > 1, runs = by_runs(p.cut, a.channels, run_channels);
            const uint32_t width = 64 * (runs ? run_channels : V);
            p.blocks = (a.channels + width - 1) / width;
            const uint64_t wgs = (uint64_t)p.cut.tiles * p.blocks, extra = g.dinitial_state && a.seqs ? kEmptyStep : 0;
            if (wgs + extra > kMostInGrid) {
                st = SCAN_ERR_INVALID;
                return;
            }
            if (chain && !runs) unset(p.cut, p.ws, s);
            if (runs)
                hipLaunchKernelGGL((run_channels == RV ? backward_run_kernel<T, RV> : backward_run_kernel<T, 1>),
                                   grid_of((uint64_t)p.cut.runs * p.blocks), dim3(kWaves * 64), 0, s, p);
            else if (wgs + extra)
                hipLaunchKernelGGL((chain ? backward_kernel<T, V, true> : backward_kernel<T, V, false>), grid_of(wgs + extra),
                                   dim3(kWaves * 64), 0, s, p);
            hipLaunchKernelGGL(rates_kernel, dim3((a.channels + 63) / 64), dim3(1024), 0, s, p.ws.rates, runs ? p.cut.runs : p.cut.tiles, p.cut.padded,
                               a.channels, g.drate);
        });
        return st == SCAN_OK ? launched() : st;
    });
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

uint32_t seq_set_spin_limit(uint32_t polls) { return g_spin_limit.exchange(polls); }

scan_status_t seq_get_device_error(void* stream)
{
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint32_t gave_up = 0;
    const uint32_t zero = 0;
    if (hipStreamSynchronize(s) != hipSuccess) return SCAN_ERR_HIP;
    if (hipMemcpyFromSymbol(&gave_up, HIP_SYMBOL(g_gave_up), 4) != hipSuccess) return SCAN_ERR_HIP;
    if (!gave_up) return SCAN_OK;
    return hipMemcpyToSymbol(HIP_SYMBOL(g_gave_up), &zero, 4) == hipSuccess ? SCAN_ERR_TIMEOUT : SCAN_ERR_HIP;
}

size_t gated_scan_workspace(const gated_scan_args_t* args)
{
    if (!args || check_gated(*args) != SCAN_OK) return 0;
    return lay_out(cut_of(*args), false, nullptr).bytes;
}

size_t gated_scan_saved(const gated_scan_args_t* args)
{
    if (!args || check_gated(*args) != SCAN_OK) return 0;
    const Cut c = cut_of(*args);
    return (size_t)c.tiles * kWaves * c.padded;
}

scan_status_t gated_scan(const gated_scan_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const gated_scan_args_t& a = *args;
    const scan_status_t st = check_gated(a);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(a.dtype), need = gated_scan_workspace(&a);
    if (a.y && !valid_rows(a.dtype, a.rows, a.channels, {a.y, a.y_stride})) return SCAN_ERR_INVALID;
    if (!a.workspace || !aligned(a.workspace, 256) || a.workspace_bytes < need) return SCAN_ERR_INVALID;
    const uint64_t state = a.seqs * a.channels * 4;
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es), range(a.final_state, state),
                          range(a.saved, gated_scan_saved(&a) * 4), range(a.workspace, need)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.decay_gate, a.rows, a.decay_stride, a.channels, es),
                         range(a.input_gate, a.rows, a.input_stride, a.channels, es),
                         range(a.rate, (uint64_t)a.channels * 4),
                         range(a.initial_state, state),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return forward(a, static_cast<hipStream_t>(stream));
}

size_t gated_scan_grad_workspace(const gated_scan_args_t* args)
{
    if (!args || check_gated(*args) != SCAN_OK) return 0;
    return lay_out(cut_of(*args), true, nullptr).bytes;
}

scan_status_t gated_scan_grad(const gated_scan_grad_args_t* grad, void* stream)
{
    if (!grad) return SCAN_ERR_INVALID;
    const gated_scan_grad_args_t& g = *grad;
    const gated_scan_args_t& a = g.args;
    const scan_status_t st = check_gated(a);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(a.dtype), need = gated_scan_grad_workspace(&a);
    for (const Array& r : {Array{g.dy, g.dy_stride}, Array{g.dx, g.dx_stride}, Array{g.ddecay_gate, g.ddecay_stride},
                           Array{g.dinput_gate, g.dinput_stride}})
        if (!valid_rows(a.dtype, a.rows, a.channels, r)) return SCAN_ERR_INVALID;
    if (!g.drate || (a.rows && !a.saved)) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)g.dfinal_state, (const void*)g.drate, (const void*)g.dinitial_state})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    if (!a.workspace || !aligned(a.workspace, 256) || a.workspace_bytes < need) return SCAN_ERR_INVALID;
    const uint64_t state = a.seqs * a.channels * 4;
    const Range outs[] = {range(g.dx, a.rows, g.dx_stride, a.channels, es),
                          range(g.ddecay_gate, a.rows, g.ddecay_stride, a.channels, es),
                          range(g.dinput_gate, a.rows, g.dinput_stride, a.channels, es),
                          range(g.drate, (uint64_t)a.channels * 4),
                          range(g.dinitial_state, state),
                          range(a.workspace, need)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.decay_gate, a.rows, a.decay_stride, a.channels, es),
                         range(a.input_gate, a.rows, a.input_stride, a.channels, es),
                         range(g.dy, a.rows, g.dy_stride, a.channels, es),
                         range(a.rate, (uint64_t)a.channels * 4),
                         range(a.initial_state, state),
                         range(g.dfinal_state, state),
                         range(a.saved, gated_scan_saved(&a) * 4),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return gradient(g, static_cast<hipStream_t>(stream));
}

scan_status_t gated_scan_step(const gated_scan_step_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const gated_scan_step_args_t& a = *args;
    if (!valid_dtype(a.dtype)) return SCAN_ERR_UNSUPPORTED;
    if (a.rows >= ((uint64_t)1 << 31) || a.n_slots >= ((uint64_t)1 << 31)) return SCAN_ERR_INVALID;
    if (a.channels < 1 || a.channels > kMaxChannels) return SCAN_ERR_INVALID;
    if (a.rows == 0) return SCAN_OK;
    const Array arrays[] = {{a.x, a.x_stride}, {a.decay_gate, a.decay_stride}, {a.input_gate, a.input_stride}, {a.y, a.y_stride}};
    for (const Array& r : arrays)
        if (!valid_rows(a.dtype, a.rows, a.channels, r)) return SCAN_ERR_INVALID;
    if (!a.rate || !a.state || !aligned(a.rate, 4) || !aligned(a.state, 4) || !aligned(a.slots, 4)) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype);
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es), range(a.state, a.n_slots * a.channels * 4)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.decay_gate, a.rows, a.decay_stride, a.channels, es),
                         range(a.input_gate, a.rows, a.input_stride, a.channels, es),
                         range(a.rate, (uint64_t)a.channels * 4),
                         range(a.slots, a.rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const Inputs in{a.x, a.decay_gate, a.input_gate, a.x_stride, a.decay_stride, a.input_stride, a.rate, nullptr};
    const int v = channels_per_lane(a.dtype, a.channels, arrays);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t st = SCAN_OK;
        with_channels<4>(v, [&](auto n) {
            constexpr int V = decltype(n)::value;
            const uint32_t chunks = (a.channels + 64 * V - 1) / (64 * V);
            const uint64_t wgs = (a.rows * chunks + 3) / 4;
            if (wgs > kMostInGrid) {
                st = SCAN_ERR_INVALID;
                return;
            }
            hipLaunchKernelGGL((step_kernel<T, V>), grid_of(wgs), dim3(256), 0, static_cast<hipStream_t>(stream), in, (uint32_t)a.rows,
                               a.channels, chunks, a.slots, (uint32_t)a.n_slots, a.state, static_cast<T*>(a.y), a.y_stride);
        });
        return st == SCAN_OK ? launched() : st;
    });
}

}  // extern "C"
