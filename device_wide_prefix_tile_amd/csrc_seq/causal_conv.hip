// Depthwise causal convolution of 2 to 4 taps along every sequence, its
// gradient and its form for single tokens.
//
//   u[t] = bias + sum_k w[k] x[t - K + 1 + k],  y = act(u)
//   g[t] = dy[t] act'(u[t]);  dx[t] = sum_k w[k] g[t + K - 1 - k];
//   dw[k] = sum_t g[t] x[t - K + 1 + k];  dbias = sum_t g[t]
//
// A few operations per element: forwards HBM-bound (read x, write y; 5.7 TB/s
// with the vector units busy 71% of the time); the gradient (read x and dy,
// write dx) is bound by the issue of its vector instructions (82%) as much as
// by memory (3.8 TB/s).  A lane owns V neighbouring channels and walks a block
// of rows with the last K - 1 inputs in registers, so every input is read once
// but for the K - 1 rows before each block.  The gradient recomputes u rather
// than keep it, walks K - 1 rows past its block for the g that reach back into
// it, and adds up dw in registers; a workgroup joins its lanes' sums in LDS,
// a second launch the workgroups'.
#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr int kBlock = 256;
// Channels per lane on the vector path (8 bytes of a 16-bit type).  With 8 the gradient needs 240
// registers and two wavefronts per SIMD do not hide the loads.  2 / 4 / 8 channels, bfloat16, us: forward
// of 8 x 2048 x 4096 52 / 49 / 54, its gradient 96 / 98 / 121; forward of ragged 8191 x 4096 27 / 26 / 28.
// The single-token kernel, which keeps little, takes 16 bytes.
constexpr int kPack = 4;
constexpr uint32_t kMaxChannels = 1u << 20;

// Channel vectors per row of a workgroup (a power of two up to 64); the other lanes take other row blocks.
uint32_t channel_lanes(uint32_t nvec)
{
    uint32_t cl = 8;
    while (cl < 64 && cl < nvec) cl *= 2;
    return cl;
}

struct Shape {
    Sequences seqs;
    uint32_t channels, nvec, cl, row_blocks, rows_per_block, groups;  // groups: row blocks per workgroup
    uint32_t nx, ny;      // workgroups along the channels (neighbours in the launch) and along the rows
    uint32_t workgroups;  // of the launch, those of the states included
};

template <typename T>
struct Conv {
    const T* x;
    int64_t x_stride;
    const T* initial;
    T* y;
    int64_t y_stride;
    T* final_state;
};

// w[k][j] = weight[c + j][k], b[j] = bias[c + j]
template <typename W, int K, int V>
__device__ __forceinline__ void load_weights(const W* __restrict__ weight, const W* __restrict__ bias, uint32_t c,
                                             float (&w)[K][V], float (&b)[V])
{
    // V rows of K weights are V * K consecutive ones: K packs of V
    float f[K][V];
#pragma unroll
    for (int q = 0; q < K; ++q) unpack(load_pack<W, V>(weight + (size_t)c * K + q * V), f[q]);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) w[k][j] = f[(j * K + k) / V][(j * K + k) % V];
    if (bias) {
        unpack(load_pack<W, V>(bias + c), b);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = 0.0f;
    }
}

// Input at position p (p >= st - (K - 1)) of sequence s that starts at row st: before st from the
// initial state.
template <typename T, int K, int V>
__device__ __forceinline__ Pack<T, V> input(const T* __restrict__ x, int64_t stride, const T* __restrict__ initial,
                                            uint32_t s, uint32_t st, int64_t p, uint32_t c, uint32_t channels)
{
    if (p >= (int64_t)st) return load_pack<T, V>(x + p * stride + c);
    if (!initial) return zero_pack<T, V>();
    return load_pack<T, V>(initial + ((size_t)s * (K - 1) + (size_t)(p - (int64_t)st + (K - 1))) * channels + c);
}

template <int ACT>
__device__ __forceinline__ float act(float u)
{
    return ACT == SEQ_ACT_SILU ? silu(u) : u;
}
template <int ACT>
__device__ __forceinline__ float act_grad(float u)
{
    if (ACT != SEQ_ACT_SILU) return 1.0f;
    const float s = sigmoid(u);
    return s * (1.0f + u * (1.0f - s));
}

template <int K, int V>
__device__ __forceinline__ void taps(const float (&win)[K][V], const float (&w)[K][V], const float (&b)[V],
                                     float (&u)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        u[j] = b[j];
#pragma unroll
        for (int k = 0; k < K; ++k) u[j] = fmaf(w[k][j], win[k][j], u[j]);
    }
}

template <typename T, typename W, int K, int V, int ACT>
__global__ __launch_bounds__(kBlock) void conv_kernel(Shape sh, Conv<T> a, const W* __restrict__ weight,
                                                      const W* __restrict__ bias)
{
    const uint32_t wg = workgroup();
    if (wg >= sh.workgroups) return;
    const uint32_t bx = wg % sh.nx, by = wg / sh.nx;
    const uint32_t cv = bx * sh.cl + threadIdx.x % sh.cl;
    const uint32_t rb = by * sh.groups + threadIdx.x / sh.cl;
    if (cv >= sh.nvec) return;
    const uint32_t c = cv * V;
    if (by >= sh.ny) {
        // behind the row blocks: the sequences' final states
        const uint32_t s = rb - sh.ny * sh.groups;
        if (s >= sh.seqs.count) return;
        const uint32_t st = sh.seqs.start(s);
        uint32_t en = sh.seqs.end(s);
        if (en < st) en = st;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const Pack<T, V> p = input<T, K, V>(a.x, a.x_stride, a.initial, s, st, (int64_t)en - (K - 1) + j, c, sh.channels);
            *reinterpret_cast<Pack<T, V>*>(a.final_state + ((size_t)s * (K - 1) + j) * sh.channels + c) = p;
        }
        return;
    }
    if (rb >= sh.row_blocks) return;
    float w[K][V], b[V];
    load_weights<W, K, V>(weight, bias, c, w, b);
    uint32_t pos = rb * sh.rows_per_block;
    const uint32_t limit = min(pos + sh.rows_per_block, sh.seqs.rows);
    int s = sh.seqs.find(pos);
    uint32_t st, en;
    while (sh.seqs.seek(s, pos, limit, st, en)) {
        const uint32_t e = min(en, limit);
        float win[K][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
            unpack(input<T, K, V>(a.x, a.x_stride, a.initial, (uint32_t)s, st, (int64_t)pos - (K - 1) + k, c, sh.channels),
                   win[k + 1]);
        T* yp = a.y + (int64_t)pos * a.y_stride + c;
        const auto step = [&](const Pack<T, V>& p) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
            unpack(p, win[K - 1]);
            float u[V];
            taps<K, V>(win, w, b, u);
#pragma unroll
            for (int j = 0; j < V; ++j) u[j] = act<ACT>(u[j]);
            *reinterpret_cast<Pack<T, V>*>(yp) = pack<T, V>(u);
            yp += a.y_stride;
        };
        const T* xp = a.x + (int64_t)pos * a.x_stride + c;
        for (; pos + 4 <= e; pos += 4) {
            Pack<T, V> p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = load_pack<T, V>(xp + i * a.x_stride);
#pragma unroll
            for (int i = 0; i < 4; ++i) step(p[i]);
            xp += 4 * a.x_stride;
        }
        for (; pos < e; ++pos, xp += a.x_stride) step(load_pack<T, V>(xp));
    }
}

// ------------------------------------------------------------ gradient
template <typename T>
struct ConvGrad {
    const T* dy;
    int64_t dy_stride;
    const T* dfinal;
    T* dx;
    int64_t dx_stride;
    T* dinitial;
    float* partial;  // [workgroup row][K + 1][nvec * V]
};

template <typename T, typename W, int K, int V, int ACT>
__global__ __launch_bounds__(kBlock) void conv_grad_kernel(Shape sh, Conv<T> a, ConvGrad<T> g,
                                                           const W* __restrict__ weight, const W* __restrict__ bias)
{
    extern __shared__ float s_sum[];  // [groups][K + 1][cl * V]
    const uint32_t wg = workgroup();
    if (wg >= sh.workgroups) return;
    const uint32_t lane_c = threadIdx.x % sh.cl, group = threadIdx.x / sh.cl;
    const uint32_t bx = wg % sh.nx, by = wg / sh.nx;
    const uint32_t cv = bx * sh.cl + lane_c;
    const uint32_t c = cv * V;
    const bool active = cv < sh.nvec;
    float w[K][V], b[V];
    if (active) load_weights<W, K, V>(weight, bias, c, w, b);

    if (by >= sh.ny) {
        // behind the row blocks: the gradients of the initial states,
        // dinitial[j] = sum_{k <= j} w[k] g[start + j - k], and what final states shorter
        // sequences pass on
        const uint32_t s = (by - sh.ny) * sh.groups + group;
        if (!active || s >= sh.seqs.count) return;
        const uint32_t st = sh.seqs.start(s);
        uint32_t en = sh.seqs.end(s);
        if (en < st) en = st;
        const uint32_t len = en - st;
        float d[K - 1][V] = {};
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            if ((uint32_t)i >= len) continue;
            float win[K][V], u[V], dy[V];
#pragma unroll
            for (int k = 0; k < K; ++k)
                unpack(input<T, K, V>(a.x, a.x_stride, a.initial, s, st, (int64_t)st + i - (K - 1) + k, c, sh.channels), win[k]);
            taps<K, V>(win, w, b, u);
            unpack(load_pack<T, V>(g.dy + (int64_t)(st + i) * g.dy_stride + c), dy);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                const int k = j - i;
                if (k < 0) continue;
#pragma unroll
                for (int q = 0; q < V; ++q) d[j][q] = fmaf(w[k][q], dy[q] * act_grad<ACT>(u[q]), d[j][q]);
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            if (g.dfinal && (uint32_t)j >= len) {
                float f[V];
                unpack(load_pack<T, V>(g.dfinal + ((size_t)s * (K - 1) + (j - len)) * sh.channels + c), f);
#pragma unroll
                for (int q = 0; q < V; ++q) d[j][q] += f[q];
            }
            *reinterpret_cast<Pack<T, V>*>(g.dinitial + ((size_t)s * (K - 1) + j) * sh.channels + c) = pack<T, V>(d[j]);
        }
        return;
    }

    float dw[K + 1][V] = {};  // the last one: dbias
    const uint32_t rb = by * sh.groups + group;
    if (active && rb < sh.row_blocks) {
        uint32_t pos = rb * sh.rows_per_block;
        const uint32_t limit = min(pos + sh.rows_per_block, sh.seqs.rows);
        int s = sh.seqs.find(pos);
        uint32_t st, en;
        while (sh.seqs.seek(s, pos, limit, st, en)) {
            const uint32_t e = min(en, limit);
            float win[K][V], gw[K][V] = {};
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
                unpack(input<T, K, V>(a.x, a.x_stride, a.initial, (uint32_t)s, st, (int64_t)pos - (K - 1) + k, c, sh.channels),
                       win[k + 1]);
            // g of rows t - (K - 1) .. t in gw; row t completes dx[t - (K - 1)]
            const auto step = [&](uint32_t t, const Pack<T, V>& px, const Pack<T, V>& pdy) {
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        win[k][q] = win[k + 1][q];
                        gw[k][q] = gw[k + 1][q];
                    }
                if (t < en) {
                    float u[V], dy[V];
                    unpack(px, win[K - 1]);
                    unpack(pdy, dy);
                    taps<K, V>(win, w, b, u);
#pragma unroll
                    for (int q = 0; q < V; ++q) gw[K - 1][q] = dy[q] * act_grad<ACT>(u[q]);
                    if (t < e) {
#pragma unroll
                        for (int q = 0; q < V; ++q) {
#pragma unroll
                            for (int k = 0; k < K; ++k) dw[k][q] = fmaf(gw[K - 1][q], win[k][q], dw[k][q]);
                            dw[K][q] += gw[K - 1][q];
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < V; ++q) gw[K - 1][q] = 0.0f;
                }
                if (t >= pos + (K - 1)) {
                    const uint32_t r = t - (K - 1);
                    float d[V];
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        d[q] = 0.0f;
#pragma unroll
                        for (int k = 0; k < K; ++k) d[q] = fmaf(w[k][q], gw[K - 1 - k][q], d[q]);
                    }
                    if (g.dfinal && r + (K - 1) >= en) {
                        float f[V];
                        unpack(load_pack<T, V>(g.dfinal + ((size_t)s * (K - 1) + (r + (K - 1) - en)) * sh.channels + c), f);
#pragma unroll
                        for (int q = 0; q < V; ++q) d[q] += f[q];
                    }
                    *reinterpret_cast<Pack<T, V>*>(g.dx + (int64_t)r * g.dx_stride + c) = pack<T, V>(d);
                }
            };
            // rows up to e + K - 2, four at a time, the next four on their way
            const uint32_t stop = e + K - 1, in = min(stop, en);
            struct Four {
                Pack<T, V> x[4], dy[4];
            };
            const auto fetch = [&](Four& f, uint32_t at) {
                const T *xs = a.x + (int64_t)at * a.x_stride + c, *ds = g.dy + (int64_t)at * g.dy_stride + c;
                if (at + 4 <= in) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f.x[i] = load_pack<T, V>(xs + i * a.x_stride);
                        f.dy[i] = load_pack<T, V>(ds + i * g.dy_stride);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (at + i < in) {
                            f.x[i] = load_pack<T, V>(xs + i * a.x_stride);
                            f.dy[i] = load_pack<T, V>(ds + i * g.dy_stride);
                        }
                }
            };
            Four f, next;
            fetch(f, pos);
            for (uint32_t t = pos; t < stop; t += 4) {
                if (t + 4 < in) fetch(next, t + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t + i < stop) step(t + i, f.x[i], f.dy[i]);
                f = next;
            }
            pos = e;
        }
    }
    // the workgroup's row blocks added up in order
    const uint32_t width = sh.cl * V;
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int q = 0; q < V; ++q) s_sum[(group * (K + 1) + k) * width + q * sh.cl + lane_c] = dw[k][q];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < (K + 1) * width; i += kBlock) {
        const uint32_t k = i / width, at = i % width;
        const uint32_t ch = (bx * sh.cl + at % sh.cl) * V + at / sh.cl;
        if (ch >= sh.channels) continue;
        float sum = 0.0f;
        for (uint32_t q = 0; q < sh.groups; ++q) sum += s_sum[(q * (K + 1) + k) * width + at];
        g.partial[((size_t)by * (K + 1) + k) * sh.channels + ch] = sum;
    }
}

// dweight[c][k] and dbias[c]: the workgroups' sums, four runs of them side by side.
__global__ __launch_bounds__(kBlock) void conv_join_kernel(const float* __restrict__ partial, uint32_t count,
                                                           uint32_t channels, int width, float* __restrict__ dweight,
                                                           float* __restrict__ dbias)
{
    __shared__ float s_part[4][64];
    const uint32_t total = (uint32_t)(width + 1) * channels;
    const uint32_t at = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const uint32_t i = blockIdx.x * 64 + at;
    const uint32_t per = (count + 3) / 4, lo = min(slice * per, count), hi = min(lo + per, count);
    float sum = 0.0f;
    if (i < total) {
#pragma unroll 8
        for (uint32_t q = lo; q < hi; ++q) sum += partial[(size_t)q * total + i];
    }
    s_part[slice][at] = sum;
    __syncthreads();
    if (slice || i >= total) return;
    sum = ((s_part[0][at] + s_part[1][at]) + s_part[2][at]) + s_part[3][at];
    const uint32_t k = i / channels, ch = i % channels;
    if (k < (uint32_t)width)
        dweight[(size_t)ch * width + k] = sum;
    else if (dbias)
        dbias[ch] = sum;
}

// ------------------------------------------------------------ single tokens
template <typename T, typename W, int K, int V, int ACT>
__global__ __launch_bounds__(kBlock) void conv_step_kernel(uint32_t rows, uint32_t n_slots, uint32_t nvec,
                                                           uint32_t channels, const int32_t* __restrict__ slots,
                                                           const T* __restrict__ x, int64_t x_stride,
                                                           const W* __restrict__ weight, const W* __restrict__ bias,
                                                           T* __restrict__ state, T* __restrict__ y, int64_t y_stride)
{
    const uint32_t cv = blockIdx.x * kBlock + threadIdx.x, r = blockIdx.y;
    if (cv >= nvec) return;
    const uint32_t c = cv * V;
    const int32_t slot = slots ? slots[r] : (int32_t)r;
    if (slot < 0 || (uint32_t)slot >= n_slots) return;
    T* sp = state + (size_t)slot * (K - 1) * channels + c;
    Pack<T, V> p[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) p[k] = load_pack<T, V>(sp + (size_t)k * channels);
    p[K - 1] = load_pack<T, V>(x + (int64_t)r * x_stride + c);
    float w[K][V], b[V], win[K][V], u[V];
    load_weights<W, K, V>(weight, bias, c, w, b);
#pragma unroll
    for (int k = 0; k < K; ++k) unpack(p[k], win[k]);
    taps<K, V>(win, w, b, u);
#pragma unroll
    for (int j = 0; j < V; ++j) u[j] = act<ACT>(u[j]);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) *reinterpret_cast<Pack<T, V>*>(sp + (size_t)k * channels) = p[k + 1];
    *reinterpret_cast<Pack<T, V>*>(y + (int64_t)r * y_stride + c) = pack<T, V>(u);
}

// ------------------------------------------------------------ host side
// Rows per lane.  Long blocks re-read fewer rows (K - 1 in front of each) and leave fewer sums to
// join, short ones fill the chip: blocks are halved while there are fewer lanes than the numbers
// below.  Forward 16 rows 29.9 us, 32 rows 30.7 (8191 x 4096); gradient 32 / 64 / 128 rows 158 / 157 /
// 152 us (8 x 2048 x 4096, with the forward pass).
uint32_t forward_rows(uint64_t rows, uint32_t nvec)
{
    uint32_t r = 16;
    while (r > 2 && rows / r * nvec < 256 * 4 * 64 * 2) r /= 2;
    return r;
}
uint32_t grad_rows(uint64_t rows, uint32_t nvec)
{
    uint32_t r = 128;
    while (r > 4 && rows / r * nvec < 65536) r /= 2;
    return r;
}

Shape make_shape(const causal_conv1d_args_t& a, int v, bool grad)
{
    Shape sh{};
    sh.seqs = Sequences{a.seq_offsets, (uint32_t)a.rows, (uint32_t)a.seqs, a.seqs ? (uint32_t)(a.rows / a.seqs) : 0u};
    sh.channels = a.channels;
    sh.nvec = (a.channels + v - 1) / v;
    sh.cl = channel_lanes(sh.nvec);
    sh.groups = kBlock / sh.cl;
    sh.rows_per_block = grad ? grad_rows(a.rows, sh.nvec) : forward_rows(a.rows, sh.nvec);
    sh.row_blocks = (uint32_t)((a.rows + sh.rows_per_block - 1) / sh.rows_per_block);
    sh.nx = (sh.nvec + sh.cl - 1) / sh.cl;
    sh.ny = (sh.row_blocks + sh.groups - 1) / sh.groups;
    return sh;
}

// Calls f(T, W, K) for the types and the width.
template <class F>
scan_status_t dispatch(int dtype, int weight_dtype, int width, F f)
{
    return with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        const auto width_of = [&](auto we) -> scan_status_t {
            using W = decltype(we);
            switch (width) {
                case 2: return f(T(), W(), std::integral_constant<int, 2>());
                case 3: return f(T(), W(), std::integral_constant<int, 3>());
                case 4: return f(T(), W(), std::integral_constant<int, 4>());
            }
            return SCAN_ERR_UNSUPPORTED;
        };
        return weight_dtype == dtype ? width_of(T()) : width_of((float)0);
    });
}

scan_status_t check_common(const causal_conv1d_args_t& a)
{
    if (!valid_dtype(a.dtype) || (a.weight_dtype != a.dtype && a.weight_dtype != SEQ_F32)) return SCAN_ERR_UNSUPPORTED;
    if (a.width < 2 || a.width > 4 || (a.activation != SEQ_ACT_NONE && a.activation != SEQ_ACT_SILU))
        return SCAN_ERR_UNSUPPORTED;
    if (a.channels < 1 || a.channels > kMaxChannels || a.rows >= ((uint64_t)1 << 31) || a.seqs >= ((uint64_t)1 << 31))
        return SCAN_ERR_INVALID;
    if (!a.seq_offsets && (a.seqs == 0 ? a.rows != 0 : a.rows % a.seqs != 0)) return SCAN_ERR_INVALID;
    if (a.seq_offsets && !aligned(a.seq_offsets, 4)) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype);
    if (!a.weight || !aligned(a.weight, ws) || !aligned(a.bias, ws) || !aligned(a.initial_state, es)) return SCAN_ERR_INVALID;
    if (a.rows && (!a.x || !aligned(a.x, es) || a.x_stride < (int64_t)a.channels || a.x_stride > ((int64_t)1 << 31)))
        return SCAN_ERR_INVALID;
    return SCAN_OK;
}

bool valid_rows_out(const void* p, int64_t stride, const causal_conv1d_args_t& a)
{
    return a.rows == 0 || (p && aligned(p, dtype_size(a.dtype)) && stride >= (int64_t)a.channels && stride <= ((int64_t)1 << 31));
}

// Whether the vector path can be taken.  One rule for every form: whole 16-byte pieces of dtype, which the
// single-token kernel moves; the other two move kPack elements and would do with those.
bool vector_ok(const causal_conv1d_args_t& a, const void* extra0, int64_t s0, const void* extra1, int64_t s1,
               const void* extra2, const void* extra3)
{
    const int v = 16 / (int)dtype_size(a.dtype);
    return a.channels % v == 0 && a.x_stride % v == 0 && s0 % v == 0 && s1 % v == 0 && aligned(a.x, 16) &&
           aligned(a.weight, 16) && aligned(a.bias, 16) && aligned(a.initial_state, 16) && aligned(extra0, 16) &&
           aligned(extra1, 16) && aligned(extra2, 16) && aligned(extra3, 16);
}

scan_status_t forward(const causal_conv1d_args_t& a, hipStream_t s)
{
    const bool vec = vector_ok(a, a.y, a.y_stride, nullptr, 0, a.final_state, nullptr);
    return dispatch(a.dtype, a.weight_dtype, a.width, [&](auto te, auto we, auto ke) {
        using T = decltype(te);
        using W = decltype(we);
        constexpr int K = decltype(ke)::value, V = kPack;
        Shape sh = make_shape(a, vec ? V : 1, false);
        const Conv<T> p{static_cast<const T*>(a.x), a.x_stride, static_cast<const T*>(a.initial_state), static_cast<T*>(a.y),
                        a.y_stride, static_cast<T*>(a.final_state)};
        const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
        const uint64_t wgs = sh.nx * ((uint64_t)sh.ny + (a.final_state ? (sh.seqs.count + sh.groups - 1) / sh.groups : 0u));
        if (wgs == 0) return SCAN_OK;
        if (wgs > kMostInGrid) return SCAN_ERR_INVALID;
        sh.workgroups = (uint32_t)wgs;
        const dim3 grid = grid_of(wgs);
        const bool act = a.activation == SEQ_ACT_SILU;
        auto k = vec ? (act ? conv_kernel<T, W, K, V, SEQ_ACT_SILU> : conv_kernel<T, W, K, V, SEQ_ACT_NONE>)
                     : (act ? conv_kernel<T, W, K, 1, SEQ_ACT_SILU> : conv_kernel<T, W, K, 1, SEQ_ACT_NONE>);
        hipLaunchKernelGGL(k, grid, dim3(kBlock), 0, s, sh, p, w, b);
        return launched();
    });
}

scan_status_t gradient(const causal_conv1d_grad_args_t& g, hipStream_t s)
{
    const causal_conv1d_args_t& a = g.args;
    const bool vec = vector_ok(a, g.dy, g.dy_stride, g.dx, g.dx_stride, g.dfinal_state, g.dinitial_state);
    return dispatch(a.dtype, a.weight_dtype, a.width, [&](auto te, auto we, auto ke) {
        using T = decltype(te);
        using W = decltype(we);
        constexpr int K = decltype(ke)::value, V = kPack;
        const int v = vec ? V : 1;
        Shape sh = make_shape(a, v, true);
        const Conv<T> p{static_cast<const T*>(a.x), a.x_stride, static_cast<const T*>(a.initial_state), nullptr, 0, nullptr};
        const ConvGrad<T> q{static_cast<const T*>(g.dy), g.dy_stride,   static_cast<const T*>(g.dfinal_state),
                            static_cast<T*>(g.dx),       g.dx_stride,   static_cast<T*>(g.dinitial_state),
                            static_cast<float*>(g.workspace)};
        const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
        const uint64_t wgs = sh.nx * ((uint64_t)sh.ny + (g.dinitial_state ? (sh.seqs.count + sh.groups - 1) / sh.groups : 0u));
        if (wgs > kMostInGrid) return SCAN_ERR_INVALID;
        if (wgs) {
            sh.workgroups = (uint32_t)wgs;
            const dim3 grid = grid_of(wgs);
            const bool act = a.activation == SEQ_ACT_SILU;
            auto k = vec ? (act ? conv_grad_kernel<T, W, K, V, SEQ_ACT_SILU> : conv_grad_kernel<T, W, K, V, SEQ_ACT_NONE>)
                         : (act ? conv_grad_kernel<T, W, K, 1, SEQ_ACT_SILU> : conv_grad_kernel<T, W, K, 1, SEQ_ACT_NONE>);
            const size_t lds = (size_t)kBlock * v * (K + 1) * 4;
            hipLaunchKernelGGL(k, grid, dim3(kBlock), lds, s, sh, p, q, w, b);
        }
        const uint32_t outs = (K + 1) * a.channels;
        hipLaunchKernelGGL(conv_join_kernel, dim3((outs + 63) / 64), dim3(kBlock), 0, s, q.partial, sh.ny, a.channels, K,
                           g.dweight, g.dbias);
        return launched();
    });
}

Range state_range(const void* p, uint64_t seqs, const causal_conv1d_args_t& a)
{
    return range(p, seqs * (uint64_t)(a.width - 1) * a.channels * dtype_size(a.dtype));
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

scan_status_t causal_conv1d(const causal_conv1d_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const causal_conv1d_args_t& a = *args;
    const scan_status_t st = check_common(a);
    if (st != SCAN_OK) return st;
    if (!valid_rows_out(a.y, a.y_stride, a) || !aligned(a.final_state, dtype_size(a.dtype))) return SCAN_ERR_INVALID;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype);
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es), state_range(a.final_state, a.seqs, a)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es), state_range(a.initial_state, a.seqs, a),
                         range(a.weight, (uint64_t)a.channels * a.width * ws), range(a.bias, (uint64_t)a.channels * ws),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return forward(a, static_cast<hipStream_t>(stream));
}

size_t causal_conv1d_grad_workspace(const causal_conv1d_args_t* args)
{
    if (!args || check_common(*args) != SCAN_OK) return 0;
    // the element-wise path has the most row blocks
    size_t most = 0;
    for (int v : {1, kPack}) {
        const Shape sh = make_shape(*args, v, true);
        most = std::max(most, (size_t)sh.ny);
    }
    return std::max<size_t>(256, round_up(most * (args->width + 1) * args->channels * 4, 256));
}

scan_status_t causal_conv1d_grad(const causal_conv1d_grad_args_t* grad, void* stream)
{
    if (!grad) return SCAN_ERR_INVALID;
    const causal_conv1d_grad_args_t& g = *grad;
    const causal_conv1d_args_t& a = g.args;
    const scan_status_t st = check_common(a);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype), need = causal_conv1d_grad_workspace(&a);
    if (!valid_rows_out(g.dy, g.dy_stride, a) || !valid_rows_out(g.dx, g.dx_stride, a)) return SCAN_ERR_INVALID;
    if (!g.dweight || !aligned(g.dweight, 4) || !aligned(g.dbias, 4) || !aligned(g.dfinal_state, es) ||
        !aligned(g.dinitial_state, es))
        return SCAN_ERR_INVALID;
    if (!g.workspace || !aligned(g.workspace, 256) || g.workspace_bytes < need) return SCAN_ERR_INVALID;
    const Range outs[] = {range(g.dx, a.rows, g.dx_stride, a.channels, es), range(g.dweight, (uint64_t)a.channels * a.width * 4),
                          range(g.dbias, (uint64_t)a.channels * 4), state_range(g.dinitial_state, a.seqs, a),
                          range(g.workspace, need)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es), range(g.dy, a.rows, g.dy_stride, a.channels, es),
                         state_range(a.initial_state, a.seqs, a), state_range(g.dfinal_state, a.seqs, a),
                         range(a.weight, (uint64_t)a.channels * a.width * ws), range(a.bias, (uint64_t)a.channels * ws),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return gradient(g, static_cast<hipStream_t>(stream));
}

scan_status_t causal_conv1d_step(const causal_conv1d_step_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const causal_conv1d_step_args_t& a = *args;
    if (!valid_dtype(a.dtype) || (a.weight_dtype != a.dtype && a.weight_dtype != SEQ_F32)) return SCAN_ERR_UNSUPPORTED;
    if (a.width < 2 || a.width > 4 || (a.activation != SEQ_ACT_NONE && a.activation != SEQ_ACT_SILU))
        return SCAN_ERR_UNSUPPORTED;
    if (a.channels < 1 || a.channels > kMaxChannels || a.rows > 65535 || a.n_slots >= ((uint64_t)1 << 31))
        return SCAN_ERR_INVALID;
    if (a.rows == 0) return SCAN_OK;
    const size_t es = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype);
    const auto rows_ok = [&](const void* p, int64_t stride) {
        return p && aligned(p, es) && stride >= (int64_t)a.channels && stride <= ((int64_t)1 << 31);
    };
    if (!rows_ok(a.x, a.x_stride) || !rows_ok(a.y, a.y_stride) || !a.weight || !aligned(a.weight, ws) ||
        !aligned(a.bias, ws) || !a.state || !aligned(a.state, es) || !aligned(a.slots, 4))
        return SCAN_ERR_INVALID;
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es),
                          range(a.state, a.n_slots * (a.width - 1) * a.channels * es)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es), range(a.weight, (uint64_t)a.channels * a.width * ws),
                         range(a.bias, (uint64_t)a.channels * ws), range(a.slots, a.rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const int v = 16 / (int)es;
    const bool vec = a.channels % v == 0 && a.x_stride % v == 0 && a.y_stride % v == 0 && aligned(a.x, 16) &&
                     aligned(a.y, 16) && aligned(a.state, 16) && aligned(a.weight, 16) && aligned(a.bias, 16);
    return dispatch(a.dtype, a.weight_dtype, a.width, [&](auto te, auto we, auto ke) {
        using T = decltype(te);
        using W = decltype(we);
        constexpr int K = decltype(ke)::value, V = 16 / sizeof(T);
        const uint32_t nvec = (a.channels + (vec ? V : 1) - 1) / (vec ? V : 1);
        const bool act = a.activation == SEQ_ACT_SILU;
        auto k = vec ? (act ? conv_step_kernel<T, W, K, V, SEQ_ACT_SILU> : conv_step_kernel<T, W, K, V, SEQ_ACT_NONE>)
                     : (act ? conv_step_kernel<T, W, K, 1, SEQ_ACT_SILU> : conv_step_kernel<T, W, K, 1, SEQ_ACT_NONE>);
        hipLaunchKernelGGL(k, dim3((nvec + kBlock - 1) / kBlock, (unsigned)a.rows), dim3(kBlock), 0,
                           static_cast<hipStream_t>(stream), (uint32_t)a.rows, (uint32_t)a.n_slots, nvec, a.channels, a.slots,
                           static_cast<const T*>(a.x), a.x_stride, static_cast<const W*>(a.weight),
                           static_cast<const W*>(a.bias), static_cast<T*>(a.state), static_cast<T*>(a.y), a.y_stride);
        return launched();
    });
}

}  // extern "C"
