// Rows and who walks them: the sequences' row ranges, and the selective scan's
// cut of the rows into spans.  Plain integer code, for the device and the host.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#ifdef __HIPCC__
#define SEQ_HD __host__ __device__ __forceinline__
#else
#define SEQ_HD inline
#endif

namespace dwpt_seq {

// The sequences of a call: `len` rows each (offsets == nullptr), or the ranges between consecutive
// offsets.  Offsets are clamped to 0 .. rows, so that no value of them leads outside the arrays.
struct Sequences {
    const int32_t* offsets;
    uint32_t rows, count, len;

    SEQ_HD uint32_t start(uint32_t s) const
    {
        if (!offsets) return s * len;
        const int32_t o = offsets[s];
        return o < 0 ? 0u : (uint32_t)o > rows ? rows : (uint32_t)o;
    }
    SEQ_HD uint32_t end(uint32_t s) const { return start(s + 1); }

    // The sequence that row r belongs to: the last s with start(s) <= r; -1 if r lies before the
    // first, count if behind the last.  (Of sequences that start at one row, all but the last are
    // empty.)
    SEQ_HD int find(uint32_t r) const
    {
        if (!offsets) return (int)(r / len);
        uint32_t lo = 0, hi = count + 1;  // offsets [0, lo) are <= r, [hi, ..) are > r
        while (lo < hi) {
            const uint32_t mid = (lo + hi) >> 1;
            if (start(mid) <= r)
                lo = mid + 1;
            else
                hi = mid;
        }
        return (int)lo - 1;
    }

    // Moves (s, pos) to the first row at or behind pos that belongs to a sequence, whose range is
    // then [st, en); false if there is none below `limit`.  s: find(pos), or an earlier sequence.
    SEQ_HD bool seek(int& s, uint32_t& pos, uint32_t limit, uint32_t& st, uint32_t& en) const
    {
        if (s < 0) s = 0;
        while (pos < limit && s < (int)count) {
            st = start((uint32_t)s);
            en = end((uint32_t)s);
            if (en <= pos || en <= st) {
                ++s;
            } else {
                if (pos < st) pos = st;
                return pos < limit;
            }
        }
        return false;
    }
};

// ------------------------------------------------------------ the selective scan's spans
constexpr int kWgChannels = 64;  // channels per workgroup
constexpr int kSaveRows = 16;    // rows between the states that the gradient starts from; rows of its tiles

// Rows cut into spans.  Sequences of one length: `per_seq` spans of `span_rows` rows for each (the
// last one shorter); packed sequences: every span_rows rows, wherever sequences begin.
struct Plan {
    Sequences seqs;
    uint32_t channels, states, groups, group_channels;
    uint32_t blocks_per_group, blocks;  // workgroups along a group's channels, along all
    uint32_t span_rows, per_seq, spans, tiles_per_span;

    SEQ_HD void rows_of(uint32_t span, uint32_t& r0, uint32_t& r1) const
    {
        if (seqs.offsets) {
            r0 = span * span_rows;
            r1 = r0 + span_rows < seqs.rows ? r0 + span_rows : seqs.rows;
        } else {
            const uint32_t s = span / per_seq, first = (span % per_seq) * span_rows;
            r0 = s * seqs.len + first;
            r1 = s * seqs.len + (first + span_rows < seqs.len ? first + span_rows : seqs.len);
        }
    }
    // The span that row r of the sequence that `span` meets lies in (r in a sequence of `span`).
    SEQ_HD uint32_t span_of(uint32_t span, uint32_t r) const
    {
        if (seqs.offsets) return r / span_rows;
        const uint32_t s = span / per_seq;
        return s * per_seq + (r - s * seqs.len) / span_rows;
    }

    // Whether a walk that begins at row pos of `span` = rows [r0, ..), in a sequence that began at row
    // st, goes on where spans first .. last (first <= last < span) ended.  Elsewhere it starts from the
    // initial state: at the sequence's own first row, and where offsets that do not ascend make a
    // sequence begin before the end of the one walked last.
    SEQ_HD bool spans_before(uint32_t span, uint32_t r0, uint32_t pos, uint32_t st, uint32_t& first, uint32_t& last) const
    {
        if (pos != r0 || st >= r0) return false;
        first = span_of(span, st);
        last = span - 1;
        return true;
    }
    // The same backwards: a walk down from row hi (exclusive) of `span` = rows [.., r1), in a sequence
    // that ends at row en, goes on where spans first .. last (first >= last > span) ended.
    SEQ_HD bool spans_behind(uint32_t span, uint32_t r1, uint32_t hi, uint32_t en, uint32_t& first, uint32_t& last) const
    {
        if (hi != r1 || en <= r1) return false;
        first = span_of(span, en - 1);
        last = span + 1;
        return true;
    }
};

// Workgroups that the rows are cut for.  Measured (one prompt of 16384 x 2048 channels / ragged 6001 x
// 4096 / training 4 x 2048 x 4096, us): 512 workgroups 266 / 206 / 1680, 768 257 / 193 / 1212, 1024 247 /
// 180 / 1069, 2048 251 / 188 / 1094.
constexpr uint32_t kTargetWorkgroups = 1024;
// Shortest span, and the most workgroups for the sake of many short sequences (which bounds the
// workspace).  A span's rows are walked twice and its start joins the spans before it one by one, so
// a sequence of L rows is cut into about sqrt(L) spans at most.  Spans of at least 128 / 64 / 32 rows:
// forward 512 rows x 2048 channels 30 / 23 / 23 us, 2048 x 1024 32 / 30 / 30 (at 64 spans, without the
// square root, 40: the joins); forward and gradients 1 x 256 x 2048 245 / 94 / 69, 1 x 1024 x 2048 169 /
// 134 / 108; 128 rows x 2048 forward 20 (one launch) / 20 / 23.
constexpr uint32_t kMinSpanRows = 32;
constexpr uint32_t kMostWorkgroups = 8192;

inline Plan make_scan_plan(uint32_t channels, uint32_t states, uint32_t groups, uint64_t rows, uint64_t seqs, const int32_t* offsets)
{
    Plan p{};
    p.seqs = Sequences{offsets, (uint32_t)rows, (uint32_t)seqs, seqs ? (uint32_t)(rows / seqs) : 0u};
    p.channels = channels;
    p.states = states;
    p.groups = groups;
    p.group_channels = channels / groups;
    p.blocks_per_group = (p.group_channels + kWgChannels - 1) / kWgChannels;
    p.blocks = groups * p.blocks_per_group;
    constexpr uint32_t tt = 32;  // spans are whole tiles
    // rows of one sequence, or of all packed ones; and how many spans they may be cut into
    const uint64_t run = offsets ? rows : p.seqs.len, runs = offsets ? 1 : seqs;
    uint64_t cuts = 1;
    if (run) {
        cuts = (kTargetWorkgroups + runs * p.blocks - 1) / (runs * p.blocks);
        uint64_t most = run / kMinSpanRows;
        if (offsets) {
            // a wavefront walks its span's sequences one after another: a few for each
            cuts = std::max<uint64_t>(cuts, std::min<uint64_t>(seqs / 4, kMostWorkgroups / p.blocks));
            most = std::min<uint64_t>(most, (uint64_t)std::sqrt((double)rows * (double)seqs));
        } else {
            most = std::min<uint64_t>(most, (uint64_t)std::sqrt((double)run));
        }
        if (run <= 2 * kMinSpanRows) most = 1;
        cuts = std::max<uint64_t>(1, std::min<uint64_t>(cuts, most));
    }
    p.span_rows = (uint32_t)std::max<uint64_t>(tt, ((run + cuts - 1) / cuts + tt - 1) / tt * tt);
    p.per_seq = (uint32_t)((run + p.span_rows - 1) / p.span_rows);
    p.spans = offsets ? p.per_seq : (uint32_t)(p.per_seq * seqs);
    p.tiles_per_span = p.span_rows / kSaveRows;
    return p;
}

}  // namespace dwpt_seq
