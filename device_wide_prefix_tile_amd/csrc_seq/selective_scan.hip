// Selective state-space scan: for every channel d and state n
//   dt = softplus(delta + bias);  a = exp(dt A);  h = a h' + dt x B;
//   y = (sum_n C h + D x) silu(z)
// its gradient, and its form for single tokens.
//
// The recurrence is a scan of real affine maps h -> a h + b, as many as
// rows x channels x states, that are made from far fewer inputs and are not
// stored.  Per map: one exponential and three or four multiplies or fused
// multiply-adds, against 1/16 of the bytes of a row: the kernels are bound by
// the issue of vector instructions, not by memory.  One wavefront's
// instruction takes 1.73 ns of its SIMD, an exponential or reciprocal 3.48
// (measured on chains of them at full occupancy).
//
// Layout.  A wavefront owns 16 channels (32 in the gradient); four lanes share a channel's states, S =
// states / 4 rounded up to 4, 8 or 16 each (Place).  The sum over a channel's states is then S - 1 adds
// in the lane and a sum over four lanes, four rows at a time.  Rows are taken in tiles: the lanes load
// 16-byte pieces of the tile's rows (the next tile's while this one is worked on), turn them into dt
// and dt x in LDS, B and C into 32-bit rows, and walk the rows; results go back through LDS to the
// lanes that loaded the inputs, which finish and store them as 16-byte pieces.  Forwards no wavefront
// waits for another; in the gradient a workgroup's wavefronts share B and C and add up dB and dC.
//
// Spans.  Where sequences and channels are too few to fill the chip, the rows
// are cut into spans that are scanned at the same time: a first launch takes
// every span from a zero state to its end (no C, no output) and keeps that
// state E and the sum of dt, whose exponential is the product of the span's
// factors; the second takes the states of the spans before it in the same
// sequence, h = exp(A sum dt) h + E one after another, and scans its rows from
// there.  This is the library's reduce-then-scan with its middle step folded
// into the last one.
//
// Packed sequences are segments: a wavefront walks them one after another,
// starting each from its initial state.
#include <cfloat>

#include "seq_common.hpp"

namespace dwpt_seq {
namespace {

constexpr uint32_t kMaxChannels = 1u << 20;
constexpr uint32_t kEmptyStep = 32;  // workgroups per channel block that look for empty sequences

constexpr int kSub = 4;               // rows whose factors and states the gradient keeps in registers

// S states per lane: TT rows per tile of the forward kernels.
template <int S>
struct Cfg {
    static constexpr int NP = 4 * S;  // states, padded
    static constexpr int TT = S == 16 ? 16 : 32;
};

int states_per_lane(uint32_t states) { return states <= 16 ? 4 : states <= 32 ? 8 : 16; }

struct Inputs {
    const void *x, *delta, *B, *C, *z;
    int64_t x_stride, delta_stride, b_stride, c_stride, z_stride;
    const float *A, *D, *delta_bias, *initial;
    int softplus, vec;  // vec: every row of the inputs and outputs consists of whole 16-byte pieces
};

// ------------------------------------------------------------ tiles
// How the lanes share a tile of TT rows by CW channels: PIECES 16-byte pieces each.
template <typename T, int TT, int CW, bool VEC>
struct Tile {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int LPR = CW / V;    // lanes per row
    static constexpr int RPL = 64 / LPR;  // rows per piece
    static constexpr int PIECES = TT > RPL ? TT / RPL : 1;
    using P = Pack<T, V>;

    __device__ static __forceinline__ int row(int i, int lane) { return i * RPL + lane / LPR; }
    __device__ static __forceinline__ int col(int lane) { return (lane % LPR) * V; }

    // Rows [r0, r0 + len), channels [c0, c0 + nch) of p; zeros elsewhere.
    __device__ static __forceinline__ void load(P (&out)[PIECES], const void* base, int64_t stride, uint32_t r0, int len,
                                                uint32_t c0, int nch, int lane)
    {
        const T* p = static_cast<const T*>(base);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int r = row(i, lane), c = col(lane);
            out[i] = zero_pack<T, V>();
            if (r < len && c < nch) {
                const T* q = p + (int64_t)(r0 + r) * stride + c0 + c;
                if (VEC) {
                    out[i] = load_pack<T, V>(q);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (c + j < nch) out[i].v[j] = q[j];
                }
            }
        }
    }
    __device__ static __forceinline__ void store(void* base, int64_t stride, uint32_t r0, int len, uint32_t c0, int nch,
                                                 int lane, int i, const float (&f)[V])
    {
        const int r = row(i, lane), c = col(lane);
        if (r >= len || c >= nch) return;
        T* q = static_cast<T*>(base) + (int64_t)(r0 + r) * stride + c0 + c;
        const P p = pack<T, V>(f);
        if (VEC) {
            *reinterpret_cast<P*>(q) = p;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < nch) q[j] = p.v[j];
        }
    }
};

// A tile of TT rows by NP states of B or C, shared by LANES lanes.
template <typename T, int TT, int NP, int LANES, bool VEC>
struct StateTile {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int LPR = NP / V;
    static constexpr int TOTAL = TT * LPR;  // pieces of the tile
    static constexpr int PIECES = (TOTAL + LANES - 1) / LANES;
    using P = Pack<T, V>;

    __device__ static __forceinline__ void load(P (&out)[PIECES], const void* base, int64_t stride, uint32_t r0, int len,
                                                uint32_t at, int states, int lane)
    {
        const T* p = static_cast<const T*>(base);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int k = i * LANES + lane, r = k / LPR, n = (k % LPR) * V;
            out[i] = zero_pack<T, V>();
            if (k < TOTAL && r < len && n < states) {
                const T* q = p + (int64_t)(r0 + r) * stride + at + n;
                if (VEC) {
                    out[i] = load_pack<T, V>(q);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (n + j < states) out[i].v[j] = q[j];
                }
            }
        }
    }
    __device__ static __forceinline__ void put(float* lds, const P (&in)[PIECES], int lane)
    {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int k = i * LANES + lane;
            if (TOTAL % LANES && k >= TOTAL) continue;
            float f[V];
            unpack(in[i], f);
#pragma unroll
            for (int j = 0; j < V; j += 4) *reinterpret_cast<f32x4*>(lds + k * V + j) = f32x4{f[j], f[j + 1], f[j + 2], f[j + 3]};
        }
    }
};

// S consecutive floats, 16-byte aligned.
template <int S>
__device__ __forceinline__ void read_floats(const float* p, float (&f)[S])
{
#pragma unroll
    for (int s = 0; s < S; s += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + s);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[s + j] = v[j];
    }
}

// The four lanes of a quad hold four values each; lane q receives the sum over the quad of value q.
__device__ __forceinline__ float quad_transpose_sum(const float (&v)[4], int q)
{
    const bool odd = q & 1, high = q & 2;
    float a = odd ? v[1] : v[0], b = odd ? v[3] : v[2];
    a += dpp<kQuadXor1>(odd ? v[0] : v[1]);
    b += dpp<kQuadXor1>(odd ? v[2] : v[3]);
    const float keep = high ? b : a, give = high ? a : b;
    return keep + dpp<kQuadXor2>(give);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Exchanges the upper half of a with the lower half of b (32 lanes), or the odd 16-lane rows of a
// with the even ones of b.
__device__ __forceinline__ float swap32_sum(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];  // a bit cast of a vector's element would take the first one both times
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float swap16_sum(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];  // a bit cast of a vector's element would take the first one both times
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
// Row q of the lanes receives the sum of v[q] over the four rows.
__device__ __forceinline__ float row_transpose_sum(const float (&v)[4])
{
    return swap16_sum(swap32_sum(v[0], v[2]), swap32_sum(v[1], v[3]));
}

// Where a wavefront stands: its CW channels, and its lane's part of them: channel d (and d + 16 ...),
// quarter q of its states.  QUADS: lane = 4 d + q, and the lane's states are S q .. S q + S - 1; else
// lane = 16 q + d, and they are 4 q .. 4 q + 3 of every 16.
template <int CW, bool QUADS>
struct Place {
    static constexpr int CH = CW / 16;  // channels per lane
    template <int S>
    __device__ __forceinline__ uint32_t state(int i) const
    {
        return QUADS ? q * S + i : (i / 4) * 16 + 4 * q + i % 4;
    }
    // Whether the lane's state i exists.  A state of the padding has A = B = C = 0, but 0 times an
    // infinite dt x is NaN: sums over the states leave it out.
    template <int S>
    __device__ __forceinline__ bool real(int i, uint32_t states) const
    {
        return state<S>(i) < states;
    }
    int lane, w, d, q;                  // channel and quarter of the lane
    uint32_t group, c0;                 // first channel of the wavefront
    int nch;                            // channels of the wavefront (0: none)
    __device__ __forceinline__ Place(const Plan& p, uint32_t block)
    {
        lane = threadIdx.x & 63;
        w = uniform(threadIdx.x >> 6);
        d = QUADS ? lane >> 2 : lane & 15;
        q = QUADS ? lane & 3 : lane >> 4;
        group = block / p.blocks_per_group;
        const uint32_t first = (block % p.blocks_per_group) * kWgChannels + w * CW;
        c0 = group * p.group_channels + first;
        nch = first < p.group_channels ? (int)min(p.group_channels - first, (uint32_t)CW) : 0;
    }
};

// The lane's S states of each of its channels.
template <int S, int CH, bool QUADS>
struct LaneStates {
    using Me = Place<16 * CH, QUADS>;
    float v[CH][S];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < S; ++i) v[c][i] = 0.0f;
    }
    // from and to an array (channels x states); zeros where padded
    __device__ __forceinline__ void load(const float* __restrict__ p, const Plan& pl, const Me& me)
    {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const uint32_t n = me.template state<S>(i);
                const int ch = me.d + 16 * c;
                v[c][i] = ch < me.nch && n < pl.states ? p[(size_t)(me.c0 + ch) * pl.states + n] : 0.0f;
            }
    }
    // A / ln 2, whose product with dt is the power of two.  A rate of minus infinity forgets at once, as
    // the lowest finite one does, which times the zero step of a row behind a tile is zero and not NaN.
    __device__ __forceinline__ void load_rates(const float* __restrict__ A, const Plan& pl, const Me& me)
    {
        load(A, pl, me);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const float r = v[c][i] * kLog2e;
                v[c][i] = r < -FLT_MAX ? -FLT_MAX : r > FLT_MAX ? FLT_MAX : r;
            }
    }
    __device__ __forceinline__ void store(float* __restrict__ p, const Plan& pl, const Me& me) const
    {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const uint32_t n = me.template state<S>(i);
                const int ch = me.d + 16 * c;
                if (ch < me.nch && n < pl.states) p[(size_t)(me.c0 + ch) * pl.states + n] = v[c][i];
            }
    }
    // the state of sequence s in an array of them, or zero without one
    __device__ __forceinline__ void start(const float* __restrict__ p, const Plan& pl, const Me& me, uint32_t s)
    {
        if (p)
            load(p + (size_t)s * pl.channels * pl.states, pl, me);
        else
            zero();
    }
    // from and to the workspace, padded to 4 S states per channel: [index][channels][4 S]
    __device__ __forceinline__ void load_padded(const float* __restrict__ p, const Plan& pl, const Me& me, size_t index)
    {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = me.d + 16 * c;
            if (ch < me.nch) {
                const float* o = p + (index * pl.channels + me.c0 + ch) * (4 * S);
#pragma unroll
                for (int i = 0; i < S; i += 4) {
                    const f32x4 f = *reinterpret_cast<const f32x4*>(o + me.template state<S>(i));
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[c][i + j] = f[j];
                }
            } else {
#pragma unroll
                for (int i = 0; i < S; ++i) v[c][i] = 0.0f;
            }
        }
    }
    __device__ __forceinline__ void store_padded(float* __restrict__ p, const Plan& pl, const Me& me, size_t index) const
    {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = me.d + 16 * c;
            if (ch >= me.nch) continue;
            float* o = p + (index * pl.channels + me.c0 + ch) * (4 * S);
#pragma unroll
            for (int i = 0; i < S; i += 4)
                *reinterpret_cast<f32x4*>(o + me.template state<S>(i)) = f32x4{v[c][i], v[c][i + 1], v[c][i + 2], v[c][i + 3]};
        }
    }
};

// What later spans need of a span: its state from a zero start (or its gradient, backwards) and
// the sum of dt over the rows.
struct SpanTotals {
    float* states;  // [span][channels][NP]
    float* dt_sum;  // [span][channels]
};
// h = the state behind spans first .. last, joined in that order, up or down.
template <int S, int CH, bool QUADS>
__device__ __forceinline__ void join_spans(const SpanTotals& t, const Plan& pl, const Place<16 * CH, QUADS>& me,
                                           uint32_t first, uint32_t last, const LaneStates<S, CH, QUADS>& A2,
                                           LaneStates<S, CH, QUADS>& h)
{
    h.load_padded(t.states, pl, me, first);
    const uint32_t step = first <= last ? 1u : ~0u;
#pragma unroll 4
    for (uint32_t left = first <= last ? last - first : first - last; left; --left) {
        first += step;
        LaneStates<S, CH, QUADS> e;
        e.load_padded(t.states, pl, me, first);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = me.d + 16 * c;
            const float sum = ch < me.nch ? t.dt_sum[(size_t)first * pl.channels + me.c0 + ch] : 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) h.v[c][i] = fmaf(exp2_fast(A2.v[c][i] * sum), h.v[c][i], e.v[c][i]);
        }
    }
}

// dt of one element: raw = delta + bias
__device__ __forceinline__ float step_size(float raw, int sp) { return sp ? softplus(raw) : raw; }

// dt of V elements of a row; of a row behind the tile, dt = 0 (softplus(-inf)).
template <int V>
__device__ __forceinline__ void step_sizes(const float (&delta)[V], const float (&bias)[V], int sp, bool in_tile,
                                           float (&dt)[V])
{
    const float none = sp ? -INFINITY : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) dt[j] = in_tile ? delta[j] + bias[j] : none;
    if (sp) {
#pragma unroll
        for (int j = 0; j < V; ++j) dt[j] = softplus(dt[j]);
    }
}

// ------------------------------------------------------------ forward
// Bound by the issue of vector instructions, so what can be done elsewhere is: the products dt x B of
// four rows, 16 channels and 16 states come from one v_mfma_f32_16x16x1_4b_f32, which multiplies four
// columns of 16 by four rows of 16 (a fused product of 32-bit values, exact but for its one rounding)
// and leaves state 4 q + i of channel d in lane 16 q + d, where the recurrence wants it.  Left per row,
// channel and state: a product and an exponential for the factor, a fused multiply-add for the state,
// one for the output.  Counted on 16384 rows of 2048 channels, per row and 16 channels (64 lanes x 4
// states): 29 vector instructions in the output's pass, 160 us, and 19 in the totals', 98; the vector
// units are busy 86% of the time.
//
// CH channels per lane: two would share what a lane reads of C, but need 248 registers (two wavefronts
// per SIMD); one, held to 168 for three, measured 190 against 207 us on ragged prompts (6001 x 4096)
// and the same on one prompt (16384 x 2048).  At 168 registers float32 inputs and rows without whole
// 16-byte pieces spill 14 to 17 of them (60 to 72 bytes of scratch per lane).
constexpr int kFwdWaveChannels = 16;
constexpr int kFwdWaves = kWgChannels / kFwdWaveChannels;

// TOTALS: the span's totals only.
template <typename T, int S, bool VEC, bool TOTALS>
__global__ __launch_bounds__(kFwdWaves * 64) __attribute__((amdgpu_waves_per_eu(S == 16 ? 1 : S == 8 ? 2 : 3))) void scan_kernel(Plan pl, Inputs in, SpanTotals totals, void* y,
                                                                  int64_t y_stride, float* final_state, float* saved)
{
    using C = Cfg<S>;
    constexpr int TT = C::TT, NP = C::NP, CW = kFwdWaveChannels, CH = CW / 16, WAVES = kFwdWaves, BLK = S / 4;
    using X = Tile<T, TT, CW, VEC>;
    using BC = StateTile<T, TT, NP, 64, VEC>;
    constexpr int V = X::V;
    // four rows more than a tile: the walk over the rows reads that far ahead
    __shared__ __align__(16) float s_dt[WAVES][(TT + 4) * CW];  // dt, as [row / 4][channel][row % 4]
    __shared__ __align__(16) float s_dx[WAVES][(TT + 4) * CW];  // dt x, as [row][channel]
    __shared__ __align__(16) float s_b[WAVES][(TT + 4) * NP];
    __shared__ __align__(16) float s_c[TOTALS ? 1 : WAVES][TOTALS ? 4 : (TT + 4) * NP];
    __shared__ __align__(16) float s_y[TOTALS ? 1 : WAVES][TOTALS ? 4 : TT * CW];
    __shared__ __align__(16) float s_par[WAVES][2 * CW];  // delta_bias and D of the wavefront's channels

    const uint32_t wg = workgroup(), block = wg % pl.blocks, span = wg / pl.blocks;
    const Place<CW, false> me(pl, block);
    if (me.nch == 0) return;
    if (span >= pl.spans) {
        // behind the spans: the final states of empty sequences
        if (TOTALS || !final_state || span - pl.spans >= kEmptyStep) return;
        for (uint32_t s = span - pl.spans; s < pl.seqs.count; s += kEmptyStep) {
            if (pl.seqs.end(s) > pl.seqs.start(s)) continue;
            LaneStates<S, CH, false> h;
            h.start(in.initial, pl, me, s);
            h.store(final_state + (size_t)s * pl.channels * pl.states, pl, me);
        }
        return;
    }
    uint32_t r0, r1;
    pl.rows_of(span, r0, r1);
    float* const dt = s_dt[me.w];
    float* const dx = s_dx[me.w];
    float* const lb = s_b[me.w];
    float* const lc = s_c[TOTALS ? 0 : me.w];
    float* const ly = s_y[TOTALS ? 0 : me.w];
    float* const bias = s_par[me.w] + X::col(me.lane);
    float* const skip = bias + CW;
    if (me.lane < 2 * CW) {  // 64 lanes or fewer
        const int c = me.lane % CW;
        const float* p = me.lane < CW ? in.delta_bias : in.D;
        s_par[me.w][me.lane] = p && c < me.nch ? p[me.c0 + c] : 0.0f;
    }
    LaneStates<S, CH, false> A2, h;
    A2.load_rates(in.A, pl, me);
    const uint32_t bc_at = me.group * pl.states;

    uint32_t pos = r0, st, en;
    int s = pl.seqs.find(pos);
    while (pl.seqs.seek(s, pos, r1, st, en)) {
        pos = (uint32_t)uniform((int)pos);
        const uint32_t e = min(en, r1);
        if (TOTALS && en <= r1) {  // ends here: no later span continues it
            pos = e;
            continue;
        }
        uint32_t from, to;
        if (!pl.spans_before(span, r0, pos, st, from, to))
            h.start(in.initial, pl, me, (uint32_t)s);
        else if (TOTALS)
            h.zero();
        else
            join_spans<S, CH, false>(totals, pl, me, from, to, A2, h);
        float sum[CH] = {};
        typename X::P px[X::PIECES], pd[X::PIECES], pz[X::PIECES];
        typename BC::P pb[BC::PIECES], pc[BC::PIECES];
        const auto fetch = [&](uint32_t at, int len) {
            X::load(px, in.x, in.x_stride, at, len, me.c0, me.nch, me.lane);
            X::load(pd, in.delta, in.delta_stride, at, len, me.c0, me.nch, me.lane);
            BC::load(pb, in.B, in.b_stride, at, len, bc_at, pl.states, me.lane);
            if (!TOTALS) {
                BC::load(pc, in.C, in.c_stride, at, len, bc_at, pl.states, me.lane);
                if (in.z) X::load(pz, in.z, in.z_stride, at, len, me.c0, me.nch, me.lane);
            }
        };
        // whole tiles where a state is saved, up to there elsewhere
        const auto tile_len = [&](uint32_t at) {
            const uint32_t off = (at - r0) % kSaveRows;
            return (int)(min(at + (off ? kSaveRows - off : (uint32_t)TT), e) - at);
        };
        int len = tile_len(pos);
        fetch(pos, len);
        while (true) {
            const bool save = !TOTALS && saved && (pos - r0) % kSaveRows == 0;
            const size_t slot = (size_t)span * pl.tiles_per_span + (pos - r0) / kSaveRows;
            // (dt, dt x) of the tile; rows behind len keep the state: dt = 0
            typename X::P cx[X::PIECES], cz[X::PIECES];
            wave_sync();
#pragma unroll
            for (int i = 0; i < X::PIECES; ++i) {
                float xf[V], df[V], bf[V];
                cx[i] = px[i];
                if (!TOTALS) cz[i] = pz[i];
                unpack(cx[i], xf);
                unpack(pd[i], df);
                const int r = X::row(i, me.lane);
                if (TT % X::RPL && r >= TT) continue;
                read_floats<V>(bias, bf);
                step_sizes<V>(df, bf, in.softplus, r < len, df);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dt[((r >> 2) * CW + X::col(me.lane) + j) * 4 + (r & 3)] = df[j];
                    xf[j] *= df[j];
                }
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    *reinterpret_cast<f32x4*>(dx + r * CW + X::col(me.lane) + j) = f32x4{xf[j], xf[j + 1], xf[j + 2], xf[j + 3]};
            }
            BC::put(lb, pb, me.lane);
            if (!TOTALS) BC::put(lc, pc, me.lane);
            wave_sync();
            const uint32_t next = pos + len;
            int next_len = 0;
            if (next < e) {
                next_len = tile_len(next);
                fetch(next, next_len);
            }
            // four rows at a time, their LDS reads and products made while the four before are walked
            struct Four {
                f32x4 dt[CH];
                f32x4 c[4][BLK];
                float left[BLK], right[CH];
            };
            const auto read = [&](Four& w, int t) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    w.dt[c] = *reinterpret_cast<const f32x4*>(dt + t * CW + (me.d + 16 * c) * 4);
                    w.right[c] = dx[(t + me.q) * CW + me.d + 16 * c];
                }
#pragma unroll
                for (int k = 0; k < BLK; ++k) {
                    w.left[k] = lb[(t + me.q) * NP + 16 * k + me.d];
                    if (!TOTALS) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) w.c[u][k] = *reinterpret_cast<const f32x4*>(lc + (t + u) * NP + 16 * k + 4 * me.q);
                    }
                }
            };
            const auto products = [&](const Four& w, f32x16 (*p)[BLK]) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int k = 0; k < BLK; ++k)
                        p[c][k] = __builtin_amdgcn_mfma_f32_16x16x1f32(w.left[k], w.right[c], f32x16{}, 0, 0, 0);
            };
            const auto walk = [&](const Four& w, const f32x16 (*p)[BLK], int t) {
                float part[CH][4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const float v = w.dt[c][u];
                        if (TOTALS) sum[c] += v;
                        float y_ = 0.0f;
#pragma unroll
                        for (int i = 0; i < S; ++i) {
                            float& hi = h.v[c][i];
                            hi = fmaf(exp2_fast(v * A2.v[c][i]), hi, p[c][i / 4][4 * u + i % 4]);
                            const float ht = VEC || me.template real<S>(i, pl.states) ? hi : 0.0f;
                            if (!TOTALS) y_ = i ? fmaf(w.c[u][i / 4][i % 4], ht, y_) : w.c[u][0][0] * ht;
                        }
                        part[c][u] = y_;
                    }
                if (!TOTALS) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) ly[(t + me.q) * CW + me.d + 16 * c] = row_transpose_sum(part[c]);
                }
            };
            Four w0, w1;
            f32x16 p0[CH][BLK], p1[CH][BLK];
            read(w0, 0);
            products(w0, p0);
            for (int t = 0; t < len; t += 8) {
                if (save && t % kSaveRows == 0) h.store_padded(saved, pl, me, slot + t / kSaveRows);
                read(w1, t + 4);
                __builtin_amdgcn_sched_barrier(0);
                walk(w0, p0, t);
                products(w1, p1);
                read(w0, t + 8);
                __builtin_amdgcn_sched_barrier(0);
                walk(w1, p1, t + 4);
                products(w0, p0);
            }
            if (!TOTALS && y) {
                wave_sync();
#pragma unroll
                for (int i = 0; i < X::PIECES; ++i) {
                    const int r = X::row(i, me.lane);
                    if (r >= len) continue;
                    float f[V], xf[V], zf[V], df[V];
                    opaque(cx[i]);
                    unpack(cx[i], xf);
                    unpack(cz[i], zf);
                    read_floats<V>(skip, df);
                    read_floats<V>(ly + r * CW + X::col(me.lane), f);
                    if (in.D) {  // without it no term: 0 * x is not 0 for every x
#pragma unroll
                        for (int j = 0; j < V; ++j) f[j] = fmaf(df[j], xf[j], f[j]);
                    }
                    if (in.z) {
#pragma unroll
                        for (int j = 0; j < V; ++j) f[j] *= silu(zf[j]);
                    }
                    X::store(y, y_stride, pos, len, me.c0, me.nch, me.lane, i, f);
                }
            }
            pos = next;
            if (pos >= e) break;
            len = next_len;
        }
        if (TOTALS) {
            h.store_padded(totals.states, pl, me, span);
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (me.q == 0 && me.d + 16 * c < me.nch)
                    totals.dt_sum[(size_t)span * pl.channels + me.c0 + me.d + 16 * c] = sum[c];
        } else if (final_state && en <= r1) {
            h.store(final_state + (size_t)s * pl.channels * pl.states, pl, me);
        }
    }
}

// ------------------------------------------------------------ single tokens
// HBM-bound: the states are read and written once.  A wavefront takes 16 channels of R rows, whose
// loads are in flight together: four rows where there are enough of them to fill the chip (256 rows
// x 4096 channels: 41 us with one row per wavefront), else one.
constexpr int kGradWaves = kWgChannels / 16;

template <typename T, int S, bool VEC, int R>
__global__ __launch_bounds__(kGradWaves * 64) void scan_step_kernel(Plan pl, Inputs in, const int32_t* __restrict__ slots,
                                                                    uint32_t n_slots, float* __restrict__ state,
                                                                    T* __restrict__ y, int64_t y_stride)
{
    const uint32_t wg = workgroup(), block = wg % pl.blocks, r0 = wg / pl.blocks * R;
    const Place<16, true> me(pl, block);
    if (me.d >= me.nch) return;
    const uint32_t c = me.c0 + me.d, first = me.q * S;
    const size_t bc_at = me.group * pl.states + first;
    const float* ap = in.A + (size_t)c * pl.states + first;
    float h[R][S], a[S], x[R], raw[R], z[R];
    Pack<T, S> b[R], cc[R];
    float* sp[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const uint32_t r = r0 + u;
        const int32_t slot = r < pl.seqs.rows ? (slots ? slots[r] : (int32_t)r) : -1;
        sp[u] = slot >= 0 && (uint32_t)slot < n_slots ? state + ((size_t)slot * pl.channels + c) * pl.states + first : nullptr;
        if (!sp[u]) continue;
        const T* bp = static_cast<const T*>(in.B) + (int64_t)r * in.b_stride + bc_at;
        const T* cp = static_cast<const T*>(in.C) + (int64_t)r * in.c_stride + bc_at;
        if (VEC) {
            read_floats<S>(sp[u], h[u]);
#pragma unroll
            for (int i = 0; i < S; i += 4) {
                const Pack<T, 4> p = load_pack<T, 4>(bp + i), q = load_pack<T, 4>(cp + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[u].v[i + j] = p.v[j];
                    cc[u].v[i + j] = q.v[j];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const bool ok = first + i < pl.states;
                h[u][i] = ok ? sp[u][i] : 0.0f;
                b[u].v[i] = ok ? bp[i] : (T)0.0f;
                cc[u].v[i] = ok ? cp[i] : (T)0.0f;
            }
        }
        x[u] = (float)static_cast<const T*>(in.x)[(int64_t)r * in.x_stride + c];
        raw[u] = (float)static_cast<const T*>(in.delta)[(int64_t)r * in.delta_stride + c];
        z[u] = in.z ? (float)static_cast<const T*>(in.z)[(int64_t)r * in.z_stride + c] : 0.0f;
    }
    if (VEC) {
        read_floats<S>(ap, a);
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) a[i] = first + i < pl.states ? ap[i] : 0.0f;
    }
    const float bias = in.delta_bias ? in.delta_bias[c] : 0.0f, skip = in.D ? in.D[c] : 0.0f;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        if (!sp[u]) continue;
        const float dt = step_size(raw[u] + bias, in.softplus), dx = dt * x[u];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            h[u][i] = fmaf(exp2_fast(dt * (a[i] * kLog2e)), h[u][i], dx * (float)b[u].v[i]);
            if (VEC || first + i < pl.states) sum = fmaf((float)cc[u].v[i], h[u][i], sum);
        }
        if (VEC) {
#pragma unroll
            for (int i = 0; i < S; i += 4)
                *reinterpret_cast<f32x4*>(sp[u] + i) = f32x4{h[u][i], h[u][i + 1], h[u][i + 2], h[u][i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (first + i < pl.states) sp[u][i] = h[u][i];
        }
        sum = quad_sum(sum);
        if (me.q == 0) {
            if (in.D) sum = fmaf(skip, x[u], sum);
            if (in.z) sum *= silu(z[u]);
            y[(int64_t)(r0 + u) * y_stride + c] = (T)sum;
        }
    }
}

// ------------------------------------------------------------ gradient
struct Grads {
    const void* dy;
    int64_t dy_stride;
    const float* dfinal;
    void *dx, *ddelta, *dz;
    int64_t dx_stride, ddelta_stride, dz_stride;
    float* dinitial;
    const float* saved;
    float* bc;    // [channel block][rows][2 NP]: the block's sums for dB and dC
    float* dA;    // [span][channels][NP]
    float* dch;   // [span][2][channels]: dD, ddelta_bias
};

// Backwards, g = a[t+1] dh[t+1] is what the later rows pass on to row t's state:
//   dh = dv C + g;  g' = a dh         (dv = dy silu(z))
// Totals of a span for the spans before it: g at its first row from g = 0 behind its last (or from
// dfinal where the sequence ends in it), and the sum of dt.  110 us for 8192 x 4096 channels, the vector
// units busy all the while.
template <typename T, int S, bool VEC>
__global__ __launch_bounds__(kGradWaves * 64) void grad_totals_kernel(Plan pl, Inputs in, Grads gr, SpanTotals totals)
{
    using C = Cfg<S>;
    constexpr int TT = C::TT, NP = C::NP;
    using X = Tile<T, TT, 16, VEC>;
    using BC = StateTile<T, TT, NP, 64, VEC>;
    constexpr int V = X::V;
    __shared__ __align__(16) f32x2 s_dt[kGradWaves][TT * 16];
    __shared__ __align__(16) float s_c[kGradWaves][TT * NP];

    const uint32_t wg = workgroup(), block = wg % pl.blocks, span = wg / pl.blocks;
    const Place<16, true> me(pl, block);
    if (me.nch == 0 || span >= pl.spans) return;
    uint32_t r0, r1, st, en;
    pl.rows_of(span, r0, r1);
    uint32_t pos = r0;
    int s = pl.seqs.find(pos);
    // only a sequence that began in an earlier span needs this span's totals
    if (!pl.seqs.seek(s, pos, r1, st, en) || pos != r0 || st == r0) return;
    f32x2* const dt = s_dt[me.w];
    float* const lc = s_c[me.w];
    LaneStates<S, 1, true> A2, g;
    A2.load_rates(in.A, pl, me);
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = X::col(me.lane) + j;
        bias[j] = in.delta_bias && c < me.nch ? in.delta_bias[me.c0 + c] : 0.0f;
    }
    if (en <= r1)
        g.start(gr.dfinal, pl, me, (uint32_t)s);
    else
        g.zero();
    uint32_t hi = (uint32_t)uniform((int)min(en, r1));
    float sum = 0.0f;
    typename X::P pd[X::PIECES], pz[X::PIECES], py[X::PIECES];
    typename BC::P pc[BC::PIECES];
    const auto fetch = [&](uint32_t at, int len) {
        X::load(pd, in.delta, in.delta_stride, at, len, me.c0, me.nch, me.lane);
        X::load(py, gr.dy, gr.dy_stride, at, len, me.c0, me.nch, me.lane);
        if (in.z) X::load(pz, in.z, in.z_stride, at, len, me.c0, me.nch, me.lane);
        BC::load(pc, in.C, in.c_stride, at, len, me.group * pl.states, pl.states, me.lane);
    };
    uint32_t lo = r0 + (hi - 1 - r0) / TT * TT;
    fetch(lo, (int)(hi - lo));
    while (true) {
        const int len = (int)(hi - lo);
#pragma unroll
        for (int i = 0; i < X::PIECES; ++i) {
            float df[V], yf[V], zf[V];
            unpack(pd[i], df);
            unpack(py[i], yf);
            if (in.z) unpack(pz[i], zf);
            const int r = X::row(i, me.lane);
            if (TT % X::RPL && r >= TT) continue;
            step_sizes<V>(df, bias, in.softplus, r < len, df);
            if (in.z) {
#pragma unroll
                for (int j = 0; j < V; ++j) yf[j] *= silu(zf[j]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) dt[r * 16 + X::col(me.lane) + j] = f32x2{df[j], yf[j]};
        }
        BC::put(lc, pc, me.lane);
        wave_sync();
        const bool more = lo > r0;
        if (more) fetch(lo - TT, TT);
        for (int t = (len - 1) | 3; t >= 0; t -= 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const f32x2 v = dt[(t - u) * 16 + me.d];
                float c[S];
                read_floats<S>(lc + (t - u) * NP + me.q * S, c);
                sum += v[0];
#pragma unroll
                for (int i = 0; i < S; ++i) g.v[0][i] = exp2_fast(v[0] * A2.v[0][i]) * fmaf(v[1], c[i], g.v[0][i]);
            }
        }
        wave_sync();
        if (!more) break;
        hi = lo;
        lo -= TT;
    }
    g.store_padded(totals.states, pl, me, span);
    if (me.q == 0 && me.d < me.nch) totals.dt_sum[(size_t)span * pl.channels + me.c0 + me.d] = sum;
}

// Every gradient of a span's rows.  Measured: 697 of the 1069 us of a training step (4 x 2048 x 4096
// channels, 16 states, bfloat16); 113 vector instructions per row and 16 channels for 4 states per
// lane keep the vector units busy 64% of the time, the matrix unit is busy 17% of it; two wavefronts
// per SIMD at 256 registers, 31 more of which are spilled (128 bytes of scratch per lane; 17 to 32
// states 76 and 276, above that one wavefront per SIMD with 256 accumulation registers, 23 and 96).
// With one channel per lane, eight rows' factors in registers and twice the matrix instructions it
// took 870.
//
// Tiles are taken from the last to the first.  A tile's states
// are recomputed from its saved one: once forwards, keeping the state in front of every kSub rows,
// then kSub rows at a time with their factors a and states h in registers, which the walk back over
// those rows uses:
//   dh = dv C + g;  g' = a dh;  dA += dt g' h[t-1];  ddt = sum A g' h[t-1] + x sum dh B
//
// dB and dC are sums over channels, which lie across the lanes: the matrix unit adds them up.
// v_mfma_f32_16x16x4_f32 multiplies a 16 x 4 matrix by a 4 x 16 one whose element (k, j) is in
// lane 16 k + j; with a first matrix of ones it leaves the sum of any register's four 16-lane rows in
// every row of the result, and the lane row that keeps tile row t takes it.  That is one matrix
// instruction and one selection per row and state (a lane's channels are added up before); what is
// left is a sum over the 4 channels of a lane row, once a tile.  (A first matrix that is 1 in one row
// and 0 elsewhere would need no selection, but 0 times a value that is not finite would reach the
// tile's other rows; the training step takes 1% less with it.)  The wavefronts of a workgroup add
// theirs in LDS, the workgroups theirs in a second launch, always in the same order.
template <int S>
struct Bwd {
    static constexpr int CW = S == 4 ? 32 : 16, WAVES = kWgChannels / CW;
};

template <typename T, int S, bool VEC>
__global__ __launch_bounds__(Bwd<S>::WAVES * 64) __attribute__((amdgpu_waves_per_eu(S == 16 ? 1 : 2))) void grad_kernel(
    Plan pl, Inputs in, Grads gr, SpanTotals totals)
{
    constexpr int TT = kSaveRows, NP = 4 * S, CW = Bwd<S>::CW, CH = CW / 16, WAVES = Bwd<S>::WAVES, BLOCKS = TT / kSub;
    using X = Tile<T, TT, CW, VEC>;
    using BC = StateTile<T, TT, NP, WAVES * 64, VEC>;
    constexpr int V = X::V;
    __shared__ __align__(16) f32x2 s_dt[WAVES][TT * CW];  // (dt, dt x), then the row's sums (dt part, x part)
    __shared__ __align__(16) float s_dv[WAVES][TT * CW];  // dv, then sum_n C h
    __shared__ __align__(16) float s_h[WAVES][BLOCKS * 64 * S * CH];  // state in front of every kSub rows
    __shared__ __align__(16) float s_b[TT * NP], s_c[TT * NP];
    __shared__ __align__(16) float s_par[WAVES][2 * CW];  // delta_bias and D of the wavefront's channels
    // the wavefront's sums for dB and dC take the place of the states, which are used up by then
    static_assert(BLOCKS * 64 * S * CH >= TT * 2 * NP, "the sums fit");

    const uint32_t wg = workgroup(), block = wg % pl.blocks, span = wg / pl.blocks;
    const Place<CW, true> me(pl, block);
    if (span >= pl.spans) return;
    uint32_t r0, r1;
    pl.rows_of(span, r0, r1);
    f32x2* const dt = s_dt[me.w];
    float* const ldv = s_dv[me.w];
    float* const lh = s_h[me.w];
    const float* const bias = s_par[me.w] + X::col(me.lane);
    const float* const skip = bias + CW;
    if (me.lane < 2 * CW) {  // 64 lanes or fewer
        const int c = me.lane % CW;
        const float* p = me.lane < CW ? in.delta_bias : in.D;
        s_par[me.w][me.lane] = p && c < me.nch ? p[me.c0 + c] : 0.0f;
    }
    LaneStates<S, CH, true> A2, g, h, dA;
    A2.load_rates(in.A, pl, me);
    dA.zero();
    float dskip[V] = {}, dbias[V] = {};
    const uint32_t bc_at = me.group * pl.states;
    float* const bc_out = gr.bc + (size_t)block * pl.seqs.rows * (2 * NP);

    uint32_t hi = r1;
    while (hi > r0) {
        // the sequence that row hi - 1 lies in
        int s = pl.seqs.find(hi - 1);
        if (s < 0) break;
        if (s >= (int)pl.seqs.count) {  // behind the last one
            hi = (uint32_t)uniform((int)min(hi - 1, pl.seqs.start(pl.seqs.count)));
            continue;
        }
        s = uniform(s);
        const uint32_t st = pl.seqs.start((uint32_t)s), en = max(pl.seqs.end((uint32_t)s), hi);
        const uint32_t first = (uint32_t)uniform((int)max(st, r0));
        uint32_t from, to;
        if (pl.spans_behind(span, r1, hi, en, from, to))
            join_spans<S, CH, true>(totals, pl, me, from, to, A2, g);
        else
            g.start(gr.dfinal, pl, me, (uint32_t)s);
        typename X::P px[X::PIECES], pd[X::PIECES], pz[X::PIECES], py[X::PIECES];
        typename BC::P pb[BC::PIECES], pc[BC::PIECES];
        const auto fetch = [&](uint32_t at, int len) {
            X::load(px, in.x, in.x_stride, at, len, me.c0, me.nch, me.lane);
            X::load(pd, in.delta, in.delta_stride, at, len, me.c0, me.nch, me.lane);
            X::load(py, gr.dy, gr.dy_stride, at, len, me.c0, me.nch, me.lane);
            if (in.z) X::load(pz, in.z, in.z_stride, at, len, me.c0, me.nch, me.lane);
            BC::load(pb, in.B, in.b_stride, at, len, bc_at, pl.states, threadIdx.x);
            BC::load(pc, in.C, in.c_stride, at, len, bc_at, pl.states, threadIdx.x);
            // the state in front of the tile
            if (at == st)
                h.start(in.initial, pl, me, (uint32_t)s);
            else
                h.load_padded(gr.saved, pl, me, (size_t)span * pl.tiles_per_span + (at - r0) / TT);
        };
        uint32_t lo = max(r0 + (hi - 1 - r0) / TT * TT, first);
        fetch(lo, (int)(hi - lo));
        while (true) {
            const int len = (int)(hi - lo);
            typename X::P cx[X::PIECES], cd[X::PIECES], cz[X::PIECES], cy[X::PIECES];
            wave_sync();
#pragma unroll
            for (int i = 0; i < X::PIECES; ++i) {
                cx[i] = px[i];
                cd[i] = pd[i];
                cy[i] = py[i];
                cz[i] = pz[i];
                float xf[V], df[V], yf[V], zf[V], bf[V];
                unpack(cx[i], xf);
                unpack(cd[i], df);
                unpack(cy[i], yf);
                unpack(cz[i], zf);
                const int r = X::row(i, me.lane);
                if (TT % X::RPL && r >= TT) continue;
                read_floats<V>(bias, bf);
                step_sizes<V>(df, bf, in.softplus, r < len, df);
                if (in.z) {
#pragma unroll
                    for (int j = 0; j < V; ++j) yf[j] *= silu(zf[j]);
                }
                const int at = r * CW + X::col(me.lane);
#pragma unroll
                for (int j = 0; j < V; ++j) dt[at + j] = f32x2{df[j], df[j] * xf[j]};
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    *reinterpret_cast<f32x4*>(ldv + at + j) = f32x4{yf[j], yf[j + 1], yf[j + 2], yf[j + 3]};
            }
            BC::put(s_b, pb, threadIdx.x);
            BC::put(s_c, pc, threadIdx.x);
            __syncthreads();
            // forwards: the states in front of every kSub rows
            const int blocks = (len + kSub - 1) / kSub;
            for (int k = 0;; ++k) {
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < S; i += 4)
                        *reinterpret_cast<f32x4*>(lh + ((k * CH + c) * 64 + me.lane) * S + i) =
                            f32x4{h.v[c][i], h.v[c][i + 1], h.v[c][i + 2], h.v[c][i + 3]};
                if (k + 1 >= blocks) break;
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const int t = k * kSub + u;
                    float b[S];
                    read_floats<S>(s_b + t * NP + me.q * S, b);
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const f32x2 v = dt[t * CW + me.d + 16 * c];
#pragma unroll
                        for (int i = 0; i < S; ++i) h.v[c][i] = fmaf(exp2_fast(v[0] * A2.v[c][i]), h.v[c][i], v[1] * b[i]);
                    }
                }
            }
            // backwards, kSub rows at a time
            f32x4 accB[S], accC[S];
#pragma unroll
            for (int i = 0; i < S; ++i) accB[i] = accC[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = blocks - 1; k >= 0; --k) {
                float a[kSub][CH][S], hs[kSub + 1][CH][S];  // the factors; the states before each row and behind the last
#pragma unroll
                for (int c = 0; c < CH; ++c) read_floats<S>(lh + ((k * CH + c) * 64 + me.lane) * S, hs[0][c]);
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const int t = k * kSub + u;
                    float b[S];
                    read_floats<S>(s_b + t * NP + me.q * S, b);
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const f32x2 v = dt[t * CW + me.d + 16 * c];
#pragma unroll
                        for (int i = 0; i < S; ++i) {
                            a[u][c][i] = exp2_fast(v[0] * A2.v[c][i]);
                            hs[u + 1][c][i] = fmaf(a[u][c][i], hs[u][c][i], v[1] * b[i]);
                        }
                    }
                }
                float ch[CH][kSub], sd[CH][kSub], sx[CH][kSub];  // the lane's sums of C h, A g h, dh B
                const bool mine = (me.lane >> 4) == k;           // the lane row that keeps these kSub rows' dB and dC
#pragma unroll
                for (int u = kSub - 1; u >= 0; --u) {
                    const int t = k * kSub + u;
#pragma unroll
                    for (int c = 0; c < CH; ++c) ch[c][u] = sd[c][u] = sx[c][u] = 0.0f;
                    if (u && t >= len) continue;  // a row behind the tile: 0 times an infinite state is no zero
                    float b[S], cc[S], pb_[S], pc_[S];
                    read_floats<S>(s_b + t * NP + me.q * S, b);
                    read_floats<S>(s_c + t * NP + me.q * S, cc);
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const f32x2 v = dt[t * CW + me.d + 16 * c];
                        const float dv = ldv[t * CW + me.d + 16 * c];
#pragma unroll
                        for (int i = 0; i < S; ++i) {
                            const float ht = hs[u + 1][c][i];
                            const float dh = fmaf(dv, cc[i], g.v[c][i]);
                            pc_[i] = c ? fmaf(dv, ht, pc_[i]) : dv * ht;
                            pb_[i] = c ? fmaf(dh, v[1], pb_[i]) : dh * v[1];
                            g.v[c][i] = a[u][c][i] * dh;
                            const float through = g.v[c][i] * hs[u][c][i];
                            dA.v[c][i] = fmaf(v[0], through, dA.v[c][i]);
                            const bool real = VEC || me.template real<S>(i, pl.states);
                            const float hr = real ? ht : 0.0f, dr = real ? dh : 0.0f, tr = real ? through : 0.0f;
                            ch[c][u] = i ? fmaf(cc[i], hr, ch[c][u]) : cc[i] * hr;
                            sx[c][u] = i ? fmaf(dr, b[i], sx[c][u]) : dr * b[i];
                            sd[c][u] = i ? fmaf(A2.v[c][i], tr, sd[c][u]) : A2.v[c][i] * tr;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < S; ++i) {
                        const f32x4 c4 = __builtin_amdgcn_mfma_f32_16x16x4f32(1.0f, pc_[i], f32x4{}, 0, 0, 0);
                        const f32x4 b4 = __builtin_amdgcn_mfma_f32_16x16x4f32(1.0f, pb_[i], f32x4{}, 0, 0, 0);
                        accC[i][u] = mine ? c4[0] : accC[i][u];
                        accB[i][u] = mine ? b4[0] : accB[i][u];
                    }
                }
                // every lane of the quad has read the rows' values: lane q writes row q's sums over them
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int at = (k * kSub + me.q) * CW + me.d + 16 * c;
                    const float d = quad_transpose_sum(sd[c], me.q), x = quad_transpose_sum(sx[c], me.q);
                    const float y = quad_transpose_sum(ch[c], me.q);
                    dt[at] = f32x2{d * kLn2, x};
                    ldv[at] = y;
                }
            }
            // the next tile's inputs, now that the registers of the walk are free
            const bool more = lo > first;
            const uint32_t next = more ? max(r0 + (lo - 1 - r0) / TT * TT, first) : lo;
            if (more) fetch(next, (int)(lo - next));
            {
                // lane 16 k + j of the accumulators has rows 4 k .. 4 k + 3, column j = 4 (channel mod 4) +
                // quarter; each of the four lanes of a quarter keeps one row
                const int pick = (me.lane >> 2) & 3, row = 4 * (me.lane >> 4) + pick;
                float fb[S], fc[S];
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    float vb[4], vc[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        vb[j] = accB[i][j];
                        vc[j] = accC[i][j];
                        vb[j] += dpp<kRowRor4>(vb[j]);
                        vc[j] += dpp<kRowRor4>(vc[j]);
                        vb[j] += dpp<kRowRor8>(vb[j]);
                        vc[j] += dpp<kRowRor8>(vc[j]);
                    }
                    fb[i] = pick == 0 ? vb[0] : pick == 1 ? vb[1] : pick == 2 ? vb[2] : vb[3];
                    fc[i] = pick == 0 ? vc[0] : pick == 1 ? vc[1] : pick == 2 ? vc[2] : vc[3];
                }
                wave_sync();
#pragma unroll
                for (int i = 0; i < S; i += 4) {
                    *reinterpret_cast<f32x4*>(lh + row * 2 * NP + me.q * S + i) = f32x4{fb[i], fb[i + 1], fb[i + 2], fb[i + 3]};
                    *reinterpret_cast<f32x4*>(lh + row * 2 * NP + NP + me.q * S + i) =
                        f32x4{fc[i], fc[i + 1], fc[i + 2], fc[i + 3]};
                }
            }
            __syncthreads();
            // the workgroup's sums for dB and dC
            for (int i = threadIdx.x; i < len * 2 * NP / 4; i += WAVES * 64) {
                f32x4 v = *reinterpret_cast<const f32x4*>(&s_h[0][i * 4]);
#pragma unroll
                for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const f32x4*>(&s_h[w][i * 4]);
                *reinterpret_cast<f32x4*>(bc_out + (size_t)lo * (2 * NP) + (size_t)i * 4) = v;
            }
            // the rows' own gradients
#pragma unroll
            for (int i = 0; i < X::PIECES; ++i) {
                const int r = X::row(i, me.lane);
                if (r >= len) continue;
                float ox[V], od[V], oz[V], xf[V], df[V], yf[V], zf[V], bf[V], sf[V], vf[V];
                opaque(cx[i]);
                opaque(cd[i]);
                opaque(cy[i]);
                opaque(cz[i]);
                unpack(cx[i], xf);
                unpack(cd[i], df);
                unpack(cy[i], yf);
                unpack(cz[i], zf);
                const int at = r * CW + X::col(me.lane);
                read_floats<V>(bias, bf);
                read_floats<V>(skip, sf);
                step_sizes<V>(df, bf, in.softplus, true, vf);
                if (in.z) {
                    float full[V];
                    read_floats<V>(ldv + at, full);
                    if (in.D) {
#pragma unroll
                        for (int j = 0; j < V; ++j) full[j] = fmaf(sf[j], xf[j], full[j]);
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float z = zf[j], sg = sigmoid(z);
                        oz[j] = yf[j] * full[j] * sg * (1.0f + z * (1.0f - sg));
                        yf[j] *= z * sg;  // dv
                    }
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const f32x2 q = dt[at + j];
                    ox[j] = vf[j] * q[1];
                    if (in.D) ox[j] = fmaf(yf[j], sf[j], ox[j]);  // as in the forward pass: without D no term
                    od[j] = fmaf(xf[j], q[1], q[0]);
                    dskip[j] = fmaf(yf[j], xf[j], dskip[j]);
                }
                if (in.softplus) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float raw = df[j] + bf[j];
                        od[j] *= raw > 20.0f ? 1.0f : sigmoid(raw);
                    }
                }
#pragma unroll
                for (int j = 0; j < V; ++j) dbias[j] += od[j];
                X::store(gr.dx, gr.dx_stride, lo, len, me.c0, me.nch, me.lane, i, ox);
                X::store(gr.ddelta, gr.ddelta_stride, lo, len, me.c0, me.nch, me.lane, i, od);
                if (in.z) X::store(gr.dz, gr.dz_stride, lo, len, me.c0, me.nch, me.lane, i, oz);
            }
            __syncthreads();
            hi = lo;
            if (!more) break;
            lo = next;
        }
        if (first == st && gr.dinitial) g.store(gr.dinitial + (size_t)s * pl.channels * pl.states, pl, me);
    }
    dA.store_padded(gr.dA, pl, me, span);
    // lanes that loaded the same channels
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int o = X::LPR; o < 64; o <<= 1) {
            dskip[j] += __shfl_xor(dskip[j], o, 64);
            dbias[j] += __shfl_xor(dbias[j], o, 64);
        }
        const int c = X::col(me.lane) + j;
        if (me.lane < X::LPR && c < me.nch) {
            float* out = gr.dch + (size_t)span * 2 * pl.channels + me.c0 + c;
            out[0] = dskip[j];
            out[pl.channels] = dbias[j];
        }
    }
}

// dB and dC: the workgroups' sums of a group's channels.  A lane takes 4 columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void join_bc_kernel(Plan pl, const float* __restrict__ bc, uint32_t np, T* __restrict__ dB,
                                                      int64_t db_stride, T* __restrict__ dC, int64_t dc_stride)
{
    const uint32_t quads = np / 2;  // 2 np columns
    const uint64_t i = workgroup() * (uint64_t)256 + threadIdx.x;
    const uint32_t col = (uint32_t)(i % quads) * 4;
    const uint64_t rg = i / quads;
    const uint32_t group = (uint32_t)(rg % pl.groups);
    const uint64_t row = rg / pl.groups;
    if (row >= pl.seqs.rows || row < pl.seqs.start(0) || row >= pl.seqs.start(pl.seqs.count)) return;
    const size_t step = (size_t)pl.seqs.rows * 2 * np;
    const float* p = bc + (size_t)group * pl.blocks_per_group * step + row * 2 * np + col;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (uint32_t b = 0; b < pl.blocks_per_group; ++b) v += *reinterpret_cast<const f32x4*>(p + b * step);
    const uint32_t n = col % np;
    T* out = (col < np ? dB + (int64_t)row * db_stride : dC + (int64_t)row * dc_stride) + group * pl.states + n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < pl.states) out[j] = (T)v[j];
}

// dA, dD and ddelta_bias: the spans' sums.
__global__ __launch_bounds__(256) void join_spans_kernel(Plan pl, const float* __restrict__ dA_part,
                                                         const float* __restrict__ dch, uint32_t np, float* __restrict__ dA,
                                                         float* __restrict__ dD, float* __restrict__ dbias)
{
    const uint64_t i = workgroup() * (uint64_t)256 + threadIdx.x, na = (uint64_t)pl.channels * np;
    float sum = 0.0f;
    if (i < na) {
#pragma unroll 8
        for (uint32_t s = 0; s < pl.spans; ++s) sum += dA_part[s * na + i];
        const uint32_t n = (uint32_t)(i % np);
        if (n < pl.states) dA[i / np * pl.states + n] = sum;
    } else if (i < na + 2 * (uint64_t)pl.channels) {
        const uint64_t c = i - na;
#pragma unroll 8
        for (uint32_t s = 0; s < pl.spans; ++s) sum += dch[s * 2 * (uint64_t)pl.channels + c];
        if (c < pl.channels) {
            if (dD) dD[c] = sum;
        } else if (dbias) {
            dbias[c - pl.channels] = sum;
        }
    }
}

// dinitial of empty sequences is dfinal.
template <int S>
__global__ __launch_bounds__(kGradWaves * 64) void grad_empty_kernel(Plan pl, const float* __restrict__ dfinal,
                                                                 float* __restrict__ dinitial)
{
    const uint32_t wg = workgroup(), block = wg % pl.blocks;
    const Place<16, true> me(pl, block);
    if (wg / pl.blocks >= kEmptyStep) return;
    for (uint32_t s = wg / pl.blocks; s < pl.seqs.count; s += kEmptyStep) {
        if (pl.seqs.end(s) > pl.seqs.start(s)) continue;
        LaneStates<S, 1, true> g;
        g.start(dfinal, pl, me, s);
        g.store(dinitial + (size_t)s * pl.channels * pl.states, pl, me);
    }
}

// ------------------------------------------------------------ host side
Plan make_plan(const selective_scan_args_t& a)
{
    return make_scan_plan(a.channels, a.states, a.groups, a.rows, a.seqs, a.seq_offsets);
}

size_t padded_states(uint32_t states) { return 4 * (size_t)states_per_lane(states); }

struct Space {
    SpanTotals totals;
    float *bc, *dA, *dch;
    size_t bytes;
};
Space lay_out(const Plan& p, bool grad, void* base)
{
    Space s{};
    size_t at = 0;
    const auto take = [&](size_t floats) {
        float* q = reinterpret_cast<float*>(static_cast<char*>(base) + at);
        at += round_up(floats * 4, 256);
        return q;
    };
    const size_t np = padded_states(p.states);
    if (p.per_seq > 1) {
        s.totals.states = take((size_t)p.spans * p.channels * np);
        s.totals.dt_sum = take((size_t)p.spans * p.channels);
    }
    if (grad) {
        s.bc = take((size_t)p.blocks * p.seqs.rows * 2 * np);
        s.dA = take((size_t)p.spans * p.channels * np);
        s.dch = take((size_t)p.spans * 2 * p.channels);
    }
    s.bytes = std::max<size_t>(at, 256);
    return s;
}

scan_status_t check_sizes(int dtype, uint64_t rows, uint32_t channels, uint32_t states, uint32_t groups)
{
    if (!valid_dtype(dtype)) return SCAN_ERR_UNSUPPORTED;
    if (states < 1 || states > 64) return SCAN_ERR_UNSUPPORTED;
    if (channels < 1 || channels > kMaxChannels || groups < 1 || channels % groups) return SCAN_ERR_INVALID;
    if (rows >= ((uint64_t)1 << 31)) return SCAN_ERR_INVALID;
    return SCAN_OK;
}

struct Rows {
    int dtype;
    uint64_t rows;
    bool ok(const void* p, int64_t stride, uint32_t width) const
    {
        return rows == 0 ||
               (p && aligned(p, dtype_size(dtype)) && stride >= (int64_t)width && stride <= ((int64_t)1 << 31));
    }
    bool vec(const void* p, int64_t stride) const
    {
        return aligned(p, 16) && stride % (16 / (int64_t)dtype_size(dtype)) == 0;
    }
};

scan_status_t check_scan(const selective_scan_args_t& a)
{
    const scan_status_t st = check_sizes(a.dtype, a.rows, a.channels, a.states, a.groups);
    if (st != SCAN_OK) return st;
    if (a.seqs >= ((uint64_t)1 << 31)) return SCAN_ERR_INVALID;
    if (!a.seq_offsets && (a.seqs == 0 ? a.rows != 0 : a.rows % a.seqs != 0)) return SCAN_ERR_INVALID;
    if (!aligned(a.seq_offsets, 4)) return SCAN_ERR_INVALID;
    const Rows r{a.dtype, a.rows};
    const uint32_t gn = a.groups * a.states;
    if (!r.ok(a.x, a.x_stride, a.channels) || !r.ok(a.delta, a.delta_stride, a.channels) || !r.ok(a.B, a.b_stride, gn) ||
        !r.ok(a.C, a.c_stride, gn) || (a.z && !r.ok(a.z, a.z_stride, a.channels)))
        return SCAN_ERR_INVALID;
    if (!a.A) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)a.A, (const void*)a.D, (const void*)a.delta_bias, (const void*)a.initial_state,
                          (const void*)a.final_state})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    return aligned(a.saved, 16) ? SCAN_OK : SCAN_ERR_INVALID;
}

template <class A>
Inputs make_inputs(const A& a, const Rows& r)
{
    Inputs in{};
    in.x = a.x;
    in.delta = a.delta;
    in.B = a.B;
    in.C = a.C;
    in.z = a.z;
    in.x_stride = a.x_stride;
    in.delta_stride = a.delta_stride;
    in.b_stride = a.b_stride;
    in.c_stride = a.c_stride;
    in.z_stride = a.z_stride;
    in.A = a.A;
    in.D = a.D;
    in.delta_bias = a.delta_bias;
    in.softplus = a.delta_softplus != 0;
    const uint32_t v = 16 / (uint32_t)dtype_size(a.dtype);
    in.vec = a.channels / a.groups % v == 0 && r.vec(a.x, a.x_stride) && r.vec(a.delta, a.delta_stride) &&
             (!a.z || r.vec(a.z, a.z_stride)) && a.states == padded_states(a.states) && r.vec(a.B, a.b_stride) &&
             r.vec(a.C, a.c_stride);
    return in;
}

// Calls f(T, S).
template <class F>
scan_status_t dispatch(int dtype, uint32_t states, F f)
{
    return with_dtype(dtype, [&](auto e) -> scan_status_t {
        using T = decltype(e);
        switch (states_per_lane(states)) {
            case 4: return f(T(), std::integral_constant<int, 4>());
            case 8: return f(T(), std::integral_constant<int, 8>());
            default: return f(T(), std::integral_constant<int, 16>());
        }
    });
}

scan_status_t forward(const selective_scan_args_t& a, hipStream_t stream)
{
    const Plan p = make_plan(a);
    const Space w = lay_out(p, false, a.workspace);
    const Rows r{a.dtype, a.rows};
    Inputs in = make_inputs(a, r);
    in.initial = a.initial_state;
    if (a.y) in.vec = in.vec && r.vec(a.y, a.y_stride);
    return dispatch(a.dtype, a.states, [&](auto te, auto se) -> scan_status_t {
        using T = decltype(te);
        constexpr int S = decltype(se)::value;
        const uint64_t wgs = (uint64_t)p.spans * p.blocks;
        const uint64_t extra = a.final_state ? (uint64_t)std::min<uint64_t>(p.seqs.count, kEmptyStep) * p.blocks : 0;
        if (wgs + extra > kMostInGrid) return SCAN_ERR_INVALID;
        if (p.per_seq > 1)
            hipLaunchKernelGGL((in.vec ? scan_kernel<T, S, true, true> : scan_kernel<T, S, false, true>), grid_of(wgs),
                               dim3(kFwdWaves * 64), 0, stream, p, in, w.totals, (void*)nullptr, (int64_t)0, (float*)nullptr,
                               (float*)nullptr);
        if (wgs + extra)
            hipLaunchKernelGGL((in.vec ? scan_kernel<T, S, true, false> : scan_kernel<T, S, false, false>),
                               grid_of(wgs + extra), dim3(kFwdWaves * 64), 0, stream, p, in, w.totals, a.y, a.y_stride,
                               a.final_state, a.saved);
        return launched();
    });
}

scan_status_t gradient(const selective_scan_grad_args_t& g, hipStream_t stream)
{
    const selective_scan_args_t& a = g.args;
    const Plan p = make_plan(a);
    const Space w = lay_out(p, true, a.workspace);
    const Rows r{a.dtype, a.rows};
    Inputs in = make_inputs(a, r);
    in.initial = a.initial_state;
    in.vec = in.vec && r.vec(g.dy, g.dy_stride) && r.vec(g.dx, g.dx_stride) && r.vec(g.ddelta, g.ddelta_stride) &&
             (!a.z || r.vec(g.dz, g.dz_stride));
    const Grads gr{g.dy, g.dy_stride, g.dfinal_state, g.dx,        g.ddelta, g.dz, g.dx_stride, g.ddelta_stride,
                   g.dz_stride, g.dinitial_state, a.saved, w.bc, w.dA, w.dch};
    return dispatch(a.dtype, a.states, [&](auto te, auto se) -> scan_status_t {
        using T = decltype(te);
        constexpr int S = decltype(se)::value;
        const uint32_t np = 4 * S;
        const uint64_t wgs = (uint64_t)p.spans * p.blocks;
        const uint64_t bc = ((uint64_t)a.rows * a.groups * (np / 2) + 255) / 256;
        if (wgs > kMostInGrid || bc > kMostInGrid) return SCAN_ERR_INVALID;
        const dim3 block(kGradWaves * 64);
        if (p.per_seq > 1)
            hipLaunchKernelGGL((in.vec ? grad_totals_kernel<T, S, true> : grad_totals_kernel<T, S, false>), grid_of(wgs), block, 0, stream, p, in, gr, w.totals);
        if (wgs) {
            hipLaunchKernelGGL((in.vec ? grad_kernel<T, S, true> : grad_kernel<T, S, false>), grid_of(wgs),
                               dim3(Bwd<S>::WAVES * 64), 0, stream, p, in, gr, w.totals);
            hipLaunchKernelGGL((join_bc_kernel<T>), grid_of(bc), dim3(256), 0, stream, p, (const float*)w.bc, np,
                               static_cast<T*>(g.dB), g.db_stride, static_cast<T*>(g.dC), g.dc_stride);
        }
        const uint64_t sums = (uint64_t)a.channels * (np + 2);
        hipLaunchKernelGGL(join_spans_kernel, grid_of((sums + 255) / 256), dim3(256), 0, stream, p,
                           (const float*)w.dA, (const float*)w.dch, np, g.dA, g.dD, g.ddelta_bias);
        if (g.dinitial_state && p.seqs.count && (a.seq_offsets || a.rows == 0))
            hipLaunchKernelGGL((grad_empty_kernel<S>), grid_of((uint64_t)std::min(p.seqs.count, kEmptyStep) * p.blocks), block,
                               0, stream, p, g.dfinal_state, g.dinitial_state);
        return launched();
    });
}

}  // namespace
}  // namespace dwpt_seq

using namespace dwpt_seq;

extern "C" {

size_t selective_scan_workspace(const selective_scan_args_t* args)
{
    if (!args || check_scan(*args) != SCAN_OK) return 0;
    return lay_out(make_plan(*args), false, nullptr).bytes;
}

size_t selective_scan_saved(const selective_scan_args_t* args)
{
    if (!args || check_scan(*args) != SCAN_OK) return 0;
    const Plan p = make_plan(*args);
    return (size_t)p.spans * p.tiles_per_span * p.channels * padded_states(p.states);
}

scan_status_t selective_scan(const selective_scan_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const selective_scan_args_t& a = *args;
    const scan_status_t st = check_scan(a);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(a.dtype), need = selective_scan_workspace(&a);
    if (a.y && !Rows{a.dtype, a.rows}.ok(a.y, a.y_stride, a.channels)) return SCAN_ERR_INVALID;
    if (!a.workspace || !aligned(a.workspace, 256) || a.workspace_bytes < need) return SCAN_ERR_INVALID;
    const uint64_t state = (uint64_t)a.seqs * a.channels * a.states * 4;
    const uint32_t gn = a.groups * a.states;
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es), range(a.final_state, state),
                          range(a.saved, selective_scan_saved(&a) * 4), range(a.workspace, need)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.delta, a.rows, a.delta_stride, a.channels, es),
                         range(a.z, a.rows, a.z_stride, a.channels, es),
                         range(a.B, a.rows, a.b_stride, gn, es),
                         range(a.C, a.rows, a.c_stride, gn, es),
                         range(a.A, (uint64_t)a.channels * a.states * 4),
                         range(a.D, (uint64_t)a.channels * 4),
                         range(a.delta_bias, (uint64_t)a.channels * 4),
                         range(a.initial_state, state),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return forward(a, static_cast<hipStream_t>(stream));
}

size_t selective_scan_grad_workspace(const selective_scan_grad_args_t* args)
{
    if (!args || check_scan(args->args) != SCAN_OK) return 0;
    return lay_out(make_plan(args->args), true, nullptr).bytes;
}

scan_status_t selective_scan_grad(const selective_scan_grad_args_t* grad, void* stream)
{
    if (!grad) return SCAN_ERR_INVALID;
    const selective_scan_grad_args_t& g = *grad;
    const selective_scan_args_t& a = g.args;
    const scan_status_t st = check_scan(a);
    if (st != SCAN_OK) return st;
    const size_t es = dtype_size(a.dtype), need = selective_scan_grad_workspace(&g);
    const Rows r{a.dtype, a.rows};
    const uint32_t gn = a.groups * a.states;
    if (!r.ok(g.dy, g.dy_stride, a.channels) || !r.ok(g.dx, g.dx_stride, a.channels) ||
        !r.ok(g.ddelta, g.ddelta_stride, a.channels) || !r.ok(g.dB, g.db_stride, gn) || !r.ok(g.dC, g.dc_stride, gn) ||
        (a.z && !r.ok(g.dz, g.dz_stride, a.channels)))
        return SCAN_ERR_INVALID;
    if (!g.dA || (a.D != nullptr) != (g.dD != nullptr) || (a.delta_bias != nullptr) != (g.ddelta_bias != nullptr) ||
        (!a.z && g.dz) || (a.rows && !a.saved))
        return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)g.dfinal_state, (const void*)g.dA, (const void*)g.dD, (const void*)g.ddelta_bias,
                          (const void*)g.dinitial_state})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    if (!a.workspace || !aligned(a.workspace, 256) || a.workspace_bytes < need) return SCAN_ERR_INVALID;
    const uint64_t state = (uint64_t)a.seqs * a.channels * a.states * 4;
    const Range outs[] = {range(g.dx, a.rows, g.dx_stride, a.channels, es),
                          range(g.ddelta, a.rows, g.ddelta_stride, a.channels, es),
                          range(g.dz, a.rows, g.dz_stride, a.channels, es),
                          range(g.dB, a.rows, g.db_stride, gn, es),
                          range(g.dC, a.rows, g.dc_stride, gn, es),
                          range(g.dA, (uint64_t)a.channels * a.states * 4),
                          range(g.dD, (uint64_t)a.channels * 4),
                          range(g.ddelta_bias, (uint64_t)a.channels * 4),
                          range(g.dinitial_state, state),
                          range(a.workspace, need)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.delta, a.rows, a.delta_stride, a.channels, es),
                         range(a.z, a.rows, a.z_stride, a.channels, es),
                         range(a.B, a.rows, a.b_stride, gn, es),
                         range(a.C, a.rows, a.c_stride, gn, es),
                         range(g.dy, a.rows, g.dy_stride, a.channels, es),
                         range(a.A, (uint64_t)a.channels * a.states * 4),
                         range(a.D, (uint64_t)a.channels * 4),
                         range(a.delta_bias, (uint64_t)a.channels * 4),
                         range(a.initial_state, state),
                         range(g.dfinal_state, state),
                         range(a.saved, selective_scan_saved(&a) * 4),
                         range(a.seq_offsets, (a.seqs + 1) * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    return gradient(g, static_cast<hipStream_t>(stream));
}

scan_status_t selective_scan_step(const selective_scan_step_args_t* args, void* stream)
{
    if (!args) return SCAN_ERR_INVALID;
    const selective_scan_step_args_t& a = *args;
    const scan_status_t st = check_sizes(a.dtype, a.rows, a.channels, a.states, a.groups);
    if (st != SCAN_OK) return st;
    if (a.n_slots >= ((uint64_t)1 << 31)) return SCAN_ERR_INVALID;
    if (a.rows == 0) return SCAN_OK;
    const Rows r{a.dtype, a.rows};
    const uint32_t gn = a.groups * a.states;
    const size_t es = dtype_size(a.dtype);
    if (!r.ok(a.x, a.x_stride, a.channels) || !r.ok(a.delta, a.delta_stride, a.channels) || !r.ok(a.B, a.b_stride, gn) ||
        !r.ok(a.C, a.c_stride, gn) || (a.z && !r.ok(a.z, a.z_stride, a.channels)) || !r.ok(a.y, a.y_stride, a.channels))
        return SCAN_ERR_INVALID;
    if (!a.A || !a.state) return SCAN_ERR_INVALID;
    for (const void* p : {(const void*)a.A, (const void*)a.D, (const void*)a.delta_bias, (const void*)a.state,
                          (const void*)a.slots})
        if (!aligned(p, 4)) return SCAN_ERR_INVALID;
    const Range outs[] = {range(a.y, a.rows, a.y_stride, a.channels, es),
                          range(a.state, a.n_slots * (uint64_t)a.channels * a.states * 4)};
    const Range ins[] = {range(a.x, a.rows, a.x_stride, a.channels, es),
                         range(a.delta, a.rows, a.delta_stride, a.channels, es),
                         range(a.z, a.rows, a.z_stride, a.channels, es),
                         range(a.B, a.rows, a.b_stride, gn, es),
                         range(a.C, a.rows, a.c_stride, gn, es),
                         range(a.A, (uint64_t)a.channels * a.states * 4),
                         range(a.D, (uint64_t)a.channels * 4),
                         range(a.delta_bias, (uint64_t)a.channels * 4),
                         range(a.slots, a.rows * 4)};
    if (any_overlap(outs, ins)) return SCAN_ERR_INVALID;
    const Plan p = make_scan_plan(a.channels, a.states, a.groups, a.rows, 1, nullptr);
    const uint64_t all = a.rows * (uint64_t)p.blocks;
    const bool four = all >= 4 * (uint64_t)kTargetWorkgroups;
    const uint64_t wgs = four ? (a.rows + 3) / 4 * p.blocks : all;
    if (wgs > kMostInGrid) return SCAN_ERR_INVALID;
    Inputs in = make_inputs(a, r);
    in.vec = a.states == padded_states(a.states) && aligned(a.state, 16) && aligned(a.A, 16) && r.vec(a.B, a.b_stride) &&
             r.vec(a.C, a.c_stride);
    return dispatch(a.dtype, a.states, [&](auto te, auto se) -> scan_status_t {
        using T = decltype(te);
        constexpr int S = decltype(se)::value;
        const auto k = four ? (in.vec ? scan_step_kernel<T, S, true, 4> : scan_step_kernel<T, S, false, 4>)
                            : (in.vec ? scan_step_kernel<T, S, true, 1> : scan_step_kernel<T, S, false, 1>);
        hipLaunchKernelGGL(k, grid_of(wgs), dim3(kGradWaves * 64), 0, static_cast<hipStream_t>(stream), p, in, a.slots,
                           (uint32_t)a.n_slots, a.state, static_cast<T*>(a.y), a.y_stride);
        return launched();
    });
}

}  // extern "C"
