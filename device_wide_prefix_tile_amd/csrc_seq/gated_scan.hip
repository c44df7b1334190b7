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
// and waits for those of the tiles before it.  Floating-point results must not depend on which of them
// are there first, so the order of compositions is fixed: tiles form groups of kGroup, the state at a
// group's start is published by the last tile of the group before it, and a tile applies the maps of the
// earlier tiles of its own group to that state one after another.  A published value is its own flag: the
// words hold a pattern beforehand (written by a small launch in front) that no published value has.
// A tile only waits for tiles with smaller numbers, whose workgroups already run, so every wait ends.
//
// Packed sequences are segments: a row that begins one starts from the initial state; a tile looks back
// no further than to the tile in which its first row's sequence begins.  The gradient is the same
// scan from the other end.
#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr uint32_t kMaxChannels = 1u << 20;
constexpr int kRows = 8;          // rows of a wavefront; the forward pass saves the state before every such rows for the gradient
constexpr int kWaves = 8;         // wavefronts of a workgroup
constexpr uint32_t kTileRows = kRows * kWaves;
constexpr uint32_t kGroup = 16;
constexpr uint32_t kChannelPad = 256;  // channels of a tile in the workspace and the saved states: a multiple of this
constexpr uint32_t kEmptyStep = 32;    // workgroups per channel block that look for empty sequences
constexpr uint32_t kMaxPolls = 1u << 22;  // some seconds; a wait that gives up yields NaN

struct Cut {
    Sequences seqs;
    uint32_t channels, padded, tiles, groups;
};

Cut make_cut(uint32_t channels, uint64_t rows, uint64_t seqs, const int32_t* offsets)
{
    Cut c{};
    c.seqs = Sequences{offsets, (uint32_t)rows, (uint32_t)seqs, seqs ? (uint32_t)(rows / seqs) : 0u};
    c.channels = channels;
    c.padded = (uint32_t)round_up(channels, kChannelPad);
    c.tiles = (uint32_t)((rows + kTileRows - 1) / kTileRows);
    c.groups = (c.tiles + kGroup - 1) / kGroup;
    return c;
}

// Workspace: the tile counter; with several tiles their maps [tile][padded] and the states at the
// groups' starts [group][padded]; the gradient's sums for the rates [tile][padded].
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
    if (c.tiles > 1) {
        s.maps = reinterpret_cast<uint64_t*>(take((size_t)c.tiles * c.padded * 8));
        s.starts = reinterpret_cast<uint32_t*>(take((size_t)c.groups * c.padded * 4));
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

// Waits until `seen`, read from p, is a published value.
template <typename W>
__device__ __forceinline__ W await(const W* p, W seen, uint32_t& polls)
{
    while ((uint32_t)seen == kUnset && polls < kMaxPolls) {
        __builtin_amdgcn_s_sleep(1);
        seen = peek(p);
        ++polls;
    }
    return seen;
}

// What the groups' words and the tiles' maps hold before the scan, and the counter.
__global__ __launch_bounds__(256) void unset_kernel(uint32_t* counter, uint64_t* maps, uint64_t n_maps, uint32_t* starts,
                                                    uint64_t n_starts)
{
    // two values per access; both counts are even (multiples of kChannelPad)
    const uint64_t i = ((uint64_t)workgroup() * 256 + threadIdx.x) * 2;
    if (i == 0) *counter = 0;
    const u32x4 unset = {kUnset, kUnset, kUnset, kUnset};
    if (i < n_maps) *reinterpret_cast<u32x4*>(maps + i) = unset;
    if (i < n_starts) *reinterpret_cast<uint64_t*>(starts + i) = ~0ull;
}

// The state (forwards) or gradient (backwards) that reaches tile k of one channel: the maps of tiles from
// `first` on, towards k, one after another; first is the tile in which the sequence begins (ends), whose map needs
// no state.  STEP 1: tiles before k, -1: behind it.  maps, starts: the channel's, `pitch` words apart.
template <int STEP>
__device__ __forceinline__ float carry(const uint64_t* maps, const uint32_t* starts, uint32_t pitch, uint32_t k, uint32_t first)
{
    constexpr int N = kGroup - 1;
    // the tiles of k's group on the way to k: n of them, the i-th is from + i STEP
    const uint32_t g = k / kGroup;
    const bool inside = first / kGroup == g;
    const uint32_t edge = STEP > 0 ? g * kGroup : g * kGroup + kGroup - 1;
    const uint32_t from = inside ? first : edge;
    const int n = (int)(STEP > 0 ? k - from : from - k);
    uint64_t v[N];
    uint32_t polls = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) v[i] = peek(maps + (uint64_t)(from + (uint32_t)(i * STEP)) * pitch);
    float h = 0.0f;
    if (!inside) {
        // starts[g]: the state before group g's first tile; backwards, the gradient behind its last one
        const uint32_t* p = starts + (uint64_t)g * pitch;
        h = __builtin_bit_cast(float, await(p, peek(p), polls));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i < n) {
            v[i] = await(maps + (uint64_t)(from + (uint32_t)(i * STEP)) * pitch, v[i], polls);
            const float a = __builtin_bit_cast(float, (uint32_t)v[i]), b = __builtin_bit_cast(float, (uint32_t)(v[i] >> 32));
            h = inside && i == 0 ? b : fmaf(a, h, b);
        }
    }
    return polls < kMaxPolls ? h : __builtin_nanf("");
}

// ------------------------------------------------------------ the gates
// 1 - a^2 = -2 a sinh(z) with z = ln a: near 1 the difference has lost what the series keeps (the next term
// of it is below 2^-26 for |z| <= 1/2).
__device__ __forceinline__ float one_minus_square(float a, float z)
{
    const float q = z * z;
    const float s = fmaf(q * (1.0f / 6), fmaf(q * (1.0f / 20), fmaf(q, 1.0f / 42, 1.0f), 1.0f), 1.0f);
    return z >= -0.5f && z <= 0.5f ? -2.0f * a * z * s : fmaf(-a, a, 1.0f);
}

// A row's map h -> a h + b.
__device__ __forceinline__ void make_map(float decay, float input, float x, float rate, float& a, float& b)
{
    const float z = rate * sigmoid(decay);
    a = exp2_fast(kLog2e * z);
    b = __builtin_amdgcn_sqrtf(one_minus_square(a, z)) * sigmoid(input) * x;
}

// ------------------------------------------------------------ a wavefront's rows
// kRows rows from one on: which belong to a sequence, begin one, end one (bits of the row), and in lane i < kRows
// the sequence of row i and its first row and end.
struct Rows {
    uint32_t live, head, tail;
    int seq;
    uint32_t st, en;

    // Row i's sequence's part of a state (sequences x channels).
    __device__ uint64_t state(int i, uint32_t channels) const { return (uint64_t)(uint32_t)__builtin_amdgcn_readlane(seq, i) * channels; }
};

__device__ __forceinline__ Rows rows_at(const Sequences& s, uint32_t r0, int lane)
{
    Rows q{};
    const uint32_t r = r0 + (uint32_t)lane;
    bool live = false, head = false, tail = false;
    if (lane < kRows && r < s.rows) {
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

// Columns c .. c + V of the rows; in place of a row of no sequence the first one of a sequence is read.
template <typename T, int V>
__device__ __forceinline__ void load_rows(Pack<T, V> (&out)[kRows], const void* base, int64_t stride, uint32_t r0, const Rows& q,
                                          uint32_t c)
{
    const int first = __builtin_ctz(q.live);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint32_t r = r0 + (uint32_t)((q.live >> i & 1) ? i : first);
        out[i] = load_pack<T, V>(static_cast<const T*>(base) + (int64_t)r * stride + c);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(void* base, int64_t stride, uint32_t r, uint32_t c, const float (&f)[V])
{
    *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(base) + (int64_t)r * stride + c) = pack<T, V>(f);
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
    uint32_t blocks;  // of 64 V channels
};

template <typename T, int V, bool CHAIN>
__global__ __launch_bounds__(kWaves * 64) void forward_kernel(Forward p)
{
    constexpr int C = 64 * V;
    __shared__ float s_a[kWaves][C], s_h[kWaves][C], s_in[C];
    __shared__ uint32_t s_head[kWaves], s_tile;
    __shared__ int s_first;
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint32_t total = p.cut.tiles * p.blocks;
    uint32_t id = workgroup();
    if (id >= total) {
        if (id - total < kEmptyStep && p.final_state)
            empty_sequences(p.cut.seqs, p.cut.channels, id - total, p.in.initial, p.final_state);
        return;
    }
    if (CHAIN) {
        if (threadIdx.x == 0) s_tile = __hip_atomic_fetch_add(p.ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = (uint32_t)uniform((int)s_tile);
    }
    const uint32_t tile = id / p.blocks, c0 = id % p.blocks * C, pitch = p.cut.padded;
    const uint32_t r0 = tile * kTileRows + (uint32_t)(w * kRows);
    const Rows rows = rows_at(p.cut.seqs, r0, lane);
    const uint32_t mine = c0 + (uint32_t)(lane * V);
    const bool inside = mine < p.cut.channels;
    const uint32_t c = inside ? mine : 0;
    // the tile in which the first row's sequence begins, if that is an earlier row
    if (w == 0 && lane == 0) s_first = (rows.live & 1) && !(rows.head & 1) ? (int)(rows.st / kTileRows) : -1;

    float a[kRows][V], b[kRows][V], am[V], hm[V];
#pragma unroll
    for (int j = 0; j < V; ++j) am[j] = 1.0f, hm[j] = 0.0f;
    if (rows.live) {
        Pack<T, V> x[kRows], dec[kRows], inp[kRows];
        load_rows(dec, p.in.decay, p.in.decay_stride, r0, rows, c);
        load_rows(inp, p.in.input, p.in.input_stride, r0, rows, c);
        load_rows(x, p.in.x, p.in.x_stride, r0, rows, c);
        const Pack<float, V> rate = load_pack_floats<V>(p.in.rate + c);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                make_map((float)dec[i].v[j], (float)inp[i].v[j], (float)x[i].v[j], rate.v[j], a[i][j], b[i][j]);
            if (rows.head >> i & 1) {
                // from the sequence's initial state: what came before ends here
                if (p.in.initial) {
                    const Pack<float, V> first = load_pack_floats<V>(p.in.initial + rows.state(i, p.cut.channels) + c);
#pragma unroll
                    for (int j = 0; j < V; ++j) b[i][j] = fmaf(a[i][j], first.v[j], b[i][j]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) hm[j] = b[i][j];
            } else if (rows.live >> i & 1) {
#pragma unroll
                for (int j = 0; j < V; ++j) am[j] *= a[i][j], hm[j] = fmaf(a[i][j], hm[j], b[i][j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_a[w][lane * V + j] = am[j], s_h[w][lane * V + j] = hm[j];
    if (lane == 0) s_head[w] = rows.head;
    __syncthreads();

    if (CHAIN) {
        // one thread per channel: the tile's map, and the state that reaches it
        const uint32_t ch = threadIdx.x;
        if (ch < (uint32_t)C) {
            float at = 1.0f, ht = 0.0f;
            bool any = false;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) {
                const bool cut = s_head[q] != 0;
                any = any || cut;
                ht = cut ? s_h[q][ch] : fmaf(s_a[q][ch], ht, s_h[q][ch]);
                at *= s_a[q][ch];
            }
            uint64_t* maps = p.ws.maps + c0 + ch;
            uint32_t* starts = p.ws.starts + c0 + ch;
            publish_map(maps + (uint64_t)tile * pitch, at, ht);
            const float h = s_first >= 0 ? carry<1>(maps, starts, pitch, tile, (uint32_t)s_first) : 0.0f;
            if ((tile + 1) % kGroup == 0 && tile + 1 < p.cut.tiles)
                publish_state(starts + (uint64_t)((tile + 1) / kGroup) * pitch, any ? ht : fmaf(at, h, ht));
            s_in[ch] = h;
        }
        __syncthreads();
    }
    if (!rows.live || !inside) return;

    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = CHAIN ? s_in[lane * V + j] : 0.0f;
    for (int q = 0; q < w; ++q) {
        const bool cut = s_head[q] != 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = s_h[q][lane * V + j];
            h[j] = cut ? t : fmaf(s_a[q][lane * V + j], h[j], t);
        }
    }
    if (p.saved) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.saved[((uint64_t)tile * kWaves + w) * pitch + c + j] = h[j];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (!(rows.live >> i & 1)) continue;
        const bool head = rows.head >> i & 1;
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = head ? b[i][j] : fmaf(a[i][j], h[j], b[i][j]);
        if (p.y) store_row<T, V>(p.y, p.y_stride, r0 + i, c, h);
        if (p.final_state && (rows.tail >> i & 1)) {
            float* last = p.final_state + rows.state(i, p.cut.channels) + c;
#pragma unroll
            for (int j = 0; j < V; ++j) last[j] = h[j];
        }
    }
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
    uint32_t blocks;
};

template <typename T, int V, bool CHAIN>
__global__ __launch_bounds__(kWaves * 64) void backward_kernel(Backward p)
{
    constexpr int C = 64 * V;
    __shared__ float s_a[kWaves][C], s_e[kWaves][C], s_rate[kWaves][C], s_in[C];
    __shared__ uint32_t s_tail[kWaves], s_tile;
    __shared__ int s_last;
    const int lane = threadIdx.x & 63, w = uniform((int)(threadIdx.x >> 6));
    const uint32_t total = p.cut.tiles * p.blocks;
    uint32_t id = workgroup();
    if (id >= total) {
        if (id - total < kEmptyStep && p.dinitial) empty_sequences(p.cut.seqs, p.cut.channels, id - total, p.dfinal, p.dinitial);
        return;
    }
    if (CHAIN) {
        if (threadIdx.x == 0) s_tile = __hip_atomic_fetch_add(p.ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = (uint32_t)uniform((int)s_tile);
    }
    const uint32_t tile = p.cut.tiles - 1 - id / p.blocks, c0 = id % p.blocks * C, pitch = p.cut.padded;
    const uint32_t r0 = tile * kTileRows + (uint32_t)(w * kRows);
    const Rows rows = rows_at(p.cut.seqs, r0, lane);
    const uint32_t mine = c0 + (uint32_t)(lane * V);
    const bool inside = mine < p.cut.channels;
    const uint32_t c = inside ? mine : 0;
    // the tile in which the last row's sequence ends, if that is a later row
    if (w == kWaves - 1 && lane == kRows - 1)
        s_last = (rows.live >> lane & 1) && !(rows.tail >> lane & 1) ? (int)((rows.en - 1) / kTileRows) : -1;

    // factors of dh in its row's results: dx, dinput, the rate's sum, ddecay
    float a[kRows][V], fx[kRows][V], fi[kRows][V], fr[kRows][V], fd[kRows][V];
    Pack<T, V> dy[kRows];
    float am[V], em[V];
#pragma unroll
    for (int j = 0; j < V; ++j) am[j] = 1.0f, em[j] = 0.0f;
    if (rows.live) {
        Pack<T, V> x[kRows], dec[kRows], inp[kRows];
        load_rows(dec, p.in.decay, p.in.decay_stride, r0, rows, c);
        load_rows(inp, p.in.input, p.in.input_stride, r0, rows, c);
        load_rows(x, p.in.x, p.in.x_stride, r0, rows, c);
        load_rows(dy, p.dy, p.dy_stride, r0, rows, c);
        const Pack<float, V> rate = load_pack_floats<V>(p.in.rate + c);
        Pack<float, V> h = load_pack_floats<V>(p.saved + ((uint64_t)tile * kWaves + w) * pitch + c);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (rows.head >> i & 1) {
                if (p.in.initial)
                    h = load_pack_floats<V>(p.in.initial + rows.state(i, p.cut.channels) + c);
                else
                    h = zero_pack<float, V>();
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float eu = exp2_fast(-kLog2e * (float)dec[i].v[j]), es = exp2_fast(-kLog2e * (float)inp[i].v[j]);
                const float f = rcp_fast(1.0f + eu), g = rcp_fast(1.0f + es), xv = (float)x[i].v[j];
                const float z = rate.v[j] * f, av = exp2_fast(kLog2e * z);
                const float w2 = one_minus_square(av, z), wv = __builtin_amdgcn_sqrtf(w2);
                const float slope = w2 == 0.0f ? 0.0f : f * __builtin_amdgcn_rsqf(w2);  // f / w
                a[i][j] = av;
                fx[i][j] = wv * g;
                fi[i][j] = wv * g * xv * rest(es, g);
                fr[i][j] = av * (f * h.v[j] - g * xv * av * slope);
                fd[i][j] = fr[i][j] * rate.v[j] * rest(eu, f);
                h.v[j] = fmaf(av, h.v[j], wv * g * xv);
            }
        }
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            if (!(rows.live >> i & 1)) continue;
            if (rows.tail >> i & 1) {
                const Pack<float, V> last =
                    p.dfinal ? load_pack_floats<V>(p.dfinal + rows.state(i, p.cut.channels) + c) : zero_pack<float, V>();
#pragma unroll
                for (int j = 0; j < V; ++j) em[j] = last.v[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) am[j] *= a[i][j], em[j] = a[i][j] * ((float)dy[i].v[j] + em[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_a[w][lane * V + j] = am[j], s_e[w][lane * V + j] = em[j];
    if (lane == 0) s_tail[w] = rows.tail;
    __syncthreads();

    if (CHAIN) {
        const uint32_t ch = threadIdx.x;
        if (ch < (uint32_t)C) {
            float at = 1.0f, et = 0.0f;
            bool any = false;
#pragma unroll
            for (int q = kWaves - 1; q >= 0; --q) {
                const bool cut = s_tail[q] != 0;
                any = any || cut;
                et = cut ? s_e[q][ch] : fmaf(s_a[q][ch], et, s_e[q][ch]);
                at *= s_a[q][ch];
            }
            uint64_t* maps = p.ws.maps + c0 + ch;
            uint32_t* starts = p.ws.starts + c0 + ch;
            publish_map(maps + (uint64_t)tile * pitch, at, et);
            const float e = s_last >= 0 ? carry<-1>(maps, starts, pitch, tile, (uint32_t)s_last) : 0.0f;
            if (tile % kGroup == 0 && tile > 0)
                publish_state(starts + (uint64_t)(tile / kGroup - 1) * pitch, any ? et : fmaf(at, e, et));
            s_in[ch] = e;
        }
        __syncthreads();
    }

    float acc[V] = {};
    if (rows.live) {
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = CHAIN ? s_in[lane * V + j] : 0.0f;
        for (int q = kWaves - 1; q > w; --q) {
            const bool cut = s_tail[q] != 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float t = s_e[q][lane * V + j];
                e[j] = cut ? t : fmaf(s_a[q][lane * V + j], e[j], t);
            }
        }
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            if (!(rows.live >> i & 1)) continue;
            if (rows.tail >> i & 1) {
                const Pack<float, V> last =
                    p.dfinal ? load_pack_floats<V>(p.dfinal + rows.state(i, p.cut.channels) + c) : zero_pack<float, V>();
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
                store_row<T, V>(p.dx, p.dx_stride, r0 + i, c, ox);
                store_row<T, V>(p.dinput, p.dinput_stride, r0 + i, c, oi);
                store_row<T, V>(p.ddecay, p.ddecay_stride, r0 + i, c, od);
                if (p.dinitial && (rows.head >> i & 1)) {
                    float* first = p.dinitial + rows.state(i, p.cut.channels) + c;
#pragma unroll
                    for (int j = 0; j < V; ++j) first[j] = e[j];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_rate[w][lane * V + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < (uint32_t)C) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) sum += s_rate[q][threadIdx.x];
        p.ws.rates[(uint64_t)tile * pitch + c0 + threadIdx.x] = sum;
    }
}

// drate: the tiles' sums, each of 16 wavefronts every sixteenth.
__global__ __launch_bounds__(1024) void rates_kernel(const float* __restrict__ sums, uint32_t tiles, uint32_t pitch, uint32_t channels,
                                                     float* __restrict__ drate)
{
    __shared__ float s_sum[16][64];
    const uint32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float sum = 0.0f;
    for (uint32_t t = w; t < tiles; t += 16) sum += sums[(uint64_t)t * pitch + c];  // c < pitch, a multiple of 64
    s_sum[w][lane] = sum;
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
        make_map((float)dec.v[j], (float)inp.v[j], (float)x.v[j], rate.v[j], a, b);
        out[j] = fmaf(a, had.v[j], b);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = out[j];
    *reinterpret_cast<Pack<T, V>*>(y + (int64_t)row * y_stride + c) = pack<T, V>(out);
}

// ------------------------------------------------------------ host side
struct Array {
    const void* p;
    int64_t stride;
};

bool valid_rows(int dtype, uint64_t rows, uint32_t width, const Array& a)
{
    if (rows == 0) return true;
    return a.p && aligned(a.p, dtype_size(dtype)) && a.stride >= (int64_t)width && a.stride <= ((int64_t)1 << 31);
}

// The most channels per lane, of 4, 2 and 1, that every row can be cut into.
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

// What the tiles wait for, set to unset values.
void unset(const Cut& c, const Space& w, hipStream_t s)
{
    const uint64_t maps = (uint64_t)c.tiles * c.padded, starts = (uint64_t)c.groups * c.padded;
    hipLaunchKernelGGL(unset_kernel, grid_of((maps + 511) / 512), dim3(256), 0, s, w.counter, w.maps, maps, w.starts, starts);
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
    Forward p{cut_of(a), inputs_of(a), a.y, a.y_stride, a.final_state, a.saved, {}, 0};
    p.ws = lay_out(p.cut, false, a.workspace);
    const Array arrays[] = {{a.x, a.x_stride}, {a.decay_gate, a.decay_stride}, {a.input_gate, a.input_stride}, {a.y, a.y_stride}};
    const int v = channels_per_lane(a.dtype, a.channels, arrays);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t st = SCAN_OK;
        with_channels<4>(v, [&](auto n) {
            constexpr int V = decltype(n)::value;
            p.blocks = (a.channels + 64 * V - 1) / (64 * V);
            const uint64_t wgs = (uint64_t)p.cut.tiles * p.blocks, extra = a.final_state && a.seqs ? kEmptyStep : 0;
            if (wgs + extra > kMostInGrid) {
                st = SCAN_ERR_INVALID;
                return;
            }
            if (wgs + extra == 0) return;
            const bool chain = p.cut.tiles > 1;
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
               g.ddecay_stride, g.dinput_stride, g.dinitial_state, {}, 0};
    p.ws = lay_out(p.cut, true, a.workspace);
    const Array arrays[] = {{a.x, a.x_stride}, {a.decay_gate, a.decay_stride}, {a.input_gate, a.input_stride}, {g.dy, g.dy_stride},
                            {g.dx, g.dx_stride}, {g.ddecay_gate, g.ddecay_stride}, {g.dinput_gate, g.dinput_stride}};
    const int v = channels_per_lane(a.dtype, a.channels, arrays);
    return with_dtype(a.dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        scan_status_t st = SCAN_OK;
        with_channels<2>(v, [&](auto n) {
            constexpr int V = decltype(n)::value;
            p.blocks = (a.channels + 64 * V - 1) / (64 * V);
            const uint64_t wgs = (uint64_t)p.cut.tiles * p.blocks, extra = g.dinitial_state && a.seqs ? kEmptyStep : 0;
            if (wgs + extra > kMostInGrid) {
                st = SCAN_ERR_INVALID;
                return;
            }
            const bool chain = p.cut.tiles > 1;
            if (chain) unset(p.cut, p.ws, s);
            if (wgs + extra)
                hipLaunchKernelGGL((chain ? backward_kernel<T, V, true> : backward_kernel<T, V, false>), grid_of(wgs + extra),
                                   dim3(kWaves * 64), 0, s, p);
            hipLaunchKernelGGL(rates_kernel, dim3((a.channels + 63) / 64), dim3(1024), 0, s, p.ws.rates, p.cut.tiles, p.cut.padded,
                               a.channels, g.drate);
        });
        return st == SCAN_OK ? launched() : st;
    });
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

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
