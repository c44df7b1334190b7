// The selective scan's walks over rows, spans and sequences on the CPU, with the kernels' own
// integer code (csrc_seq/seq_plan.hpp): which rows, states and span totals a forward and a
// backward call touch, for random sizes and for offsets that ascend, that do not, and that lie
// outside the rows.  Every index is checked against its array.  With ascending offsets also:
// every row of a sequence is walked exactly once, and no total or saved state is read that was
// not written.
//   scan_walk_model seed=N cases=N
// Prints "result ok=1 cases=N joins=N" and returns 0, or the first case that is wrong.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../device_wide_prefix_tile_amd/csrc_seq/seq_plan.hpp"

using namespace dwpt_seq;

static uint64_t g_joins = 0;
static const char* g_wrong = nullptr;
#define NEED(c)                      \
    do {                             \
        if (!(c)) {                  \
            if (!g_wrong) g_wrong = #c; \
            return;                  \
        }                            \
    } while (0)

struct Seen {
    std::vector<int> totals, saved, rows, back;  // writes so far
};

// scan_kernel: the totals' pass or the output's.
static void forward(const Plan& p, Seen& seen, bool totals, bool ordered)
{
    for (uint32_t span = 0; span < p.spans; ++span) {
        uint32_t r0, r1;
        p.rows_of(span, r0, r1);
        NEED(r0 < r1 && r1 <= p.seqs.rows);
        uint32_t pos = r0, st, en, from, to, before = r0;
        int s = p.seqs.find(pos);
        NEED(s >= -1 && s <= (int)p.seqs.count);
        while (p.seqs.seek(s, pos, r1, st, en)) {
            NEED(s >= 0 && s < (int)p.seqs.count && st <= pos && pos >= before && pos < en && en <= p.seqs.rows);
            const uint32_t e = en < r1 ? en : r1;
            before = e;
            if (totals && en <= r1) {
                pos = e;
                continue;
            }
            if (p.spans_before(span, r0, pos, st, from, to)) {
                NEED(p.per_seq > 1 && from <= to && to < span);
                if (!totals)
                    for (uint32_t k = from; k <= to; ++k) {
                        NEED(!ordered || seen.totals[k] == 1);
                        ++g_joins;
                    }
            } else {
                NEED(!ordered || pos == st);
            }
            for (uint32_t r = pos; r < e; ++r) {
                const size_t slot = (size_t)span * p.tiles_per_span + (r - r0) / kSaveRows;
                NEED(slot < seen.saved.size());
                if (!totals) ++seen.rows[r];
                if (!totals && (r - r0) % kSaveRows == 0) ++seen.saved[slot];
            }
            pos = e;
            if (totals) ++seen.totals[span];
        }
    }
}

// grad_totals_kernel
static void backward_totals(const Plan& p, Seen& seen)
{
    for (uint32_t span = 0; span < p.spans; ++span) {
        uint32_t r0, r1, st, en;
        p.rows_of(span, r0, r1);
        uint32_t pos = r0;
        int s = p.seqs.find(pos);
        if (!p.seqs.seek(s, pos, r1, st, en) || pos != r0 || st == r0) continue;
        const uint32_t hi = en < r1 ? en : r1;
        NEED(hi > r0 && hi <= p.seqs.rows && s >= 0 && s < (int)p.seqs.count);
        ++seen.totals[span];
    }
}

// grad_kernel
static void backward(const Plan& p, Seen& seen, bool ordered)
{
    for (uint32_t span = 0; span < p.spans; ++span) {
        uint32_t r0, r1, from, to;
        p.rows_of(span, r0, r1);
        uint32_t hi = r1;
        while (hi > r0) {
            const int s = p.seqs.find(hi - 1);
            NEED(s >= -1 && s <= (int)p.seqs.count);
            if (s < 0) break;
            if (s >= (int)p.seqs.count) {
                const uint32_t last = p.seqs.start(p.seqs.count);
                hi = hi - 1 < last ? hi - 1 : last;
                continue;
            }
            const uint32_t st = p.seqs.start((uint32_t)s), end = p.seqs.end((uint32_t)s), en = end > hi ? end : hi;
            const uint32_t first = st > r0 ? st : r0;
            NEED(first < hi && en <= p.seqs.rows);
            if (p.spans_behind(span, r1, hi, en, from, to)) {
                NEED(p.per_seq > 1 && from >= to && to > span && from < p.spans);
                for (uint32_t k = to; k <= from; ++k) {
                    NEED(!ordered || seen.totals[k] == 1);
                    ++g_joins;
                }
            } else {
                NEED(!ordered || hi == en);
            }
            uint32_t lo = r0 + (hi - 1 - r0) / kSaveRows * kSaveRows;
            if (lo < first) lo = first;
            while (true) {
                NEED(lo < hi && lo >= first && hi - lo <= (uint32_t)kSaveRows);
                if (lo != st) {
                    const size_t slot = (size_t)span * p.tiles_per_span + (lo - r0) / kSaveRows;
                    NEED(slot < seen.saved.size() && (!ordered || seen.saved[slot] == 1));
                }
                for (uint32_t r = lo; r < hi; ++r) ++seen.back[r];
                hi = lo;
                if (lo <= first) break;
                lo = r0 + (lo - 1 - r0) / kSaveRows * kSaveRows;
                if (lo < first) lo = first;
            }
        }
    }
}

int main(int argc, char** argv)
{
    uint64_t seed = 1, cases = 2000;
    for (int i = 1; i < argc; ++i) {
        if (!std::strncmp(argv[i], "seed=", 5)) seed = std::strtoull(argv[i] + 5, nullptr, 10);
        if (!std::strncmp(argv[i], "cases=", 6)) cases = std::strtoull(argv[i] + 6, nullptr, 10);
    }
    std::mt19937_64 rng(seed);
    const auto upto = [&](uint64_t n) { return rng() % (n + 1); };
    for (uint64_t c = 0; c < cases; ++c) {
        const int kind = (int)(c % 4);  // one length; ascending; any order; any order and outside the rows
        const uint32_t seqs = (uint32_t)upto(upto(3) ? 10 : 300) + (kind == 0), channels = 1u << upto(13);
        uint32_t rows = (uint32_t)upto(upto(3) ? 300 : 4000);
        if (kind == 0) rows = rows / seqs * seqs;
        std::vector<int32_t> off(seqs + 1);
        for (int32_t& o : off) o = kind == 3 ? (int32_t)upto(3 * rows + 8) - (int32_t)rows - 4 : (int32_t)upto(rows);
        if (kind == 3 && upto(1)) off[upto(seqs)] = upto(1) ? INT32_MAX : INT32_MIN;
        if (kind == 1) std::sort(off.begin(), off.end());
        const Plan p = make_scan_plan(channels, 16, 1, rows, seqs, kind ? off.data() : nullptr);
        Seen seen;
        const auto clear = [&](std::vector<int>& v, size_t n) { v.assign(n, 0); };
        clear(seen.totals, p.spans);
        clear(seen.saved, (size_t)p.spans * p.tiles_per_span);
        clear(seen.rows, rows);
        clear(seen.back, rows);
        const bool ordered = kind < 2;
        if (p.per_seq > 1) forward(p, seen, true, ordered);
        forward(p, seen, false, ordered);
        clear(seen.totals, p.spans);
        if (p.per_seq > 1) backward_totals(p, seen);
        backward(p, seen, ordered);
        if (ordered && !g_wrong) {
            const uint32_t lo = kind ? (uint32_t)off.front() : 0, hi = kind ? (uint32_t)off.back() : rows;
            for (uint32_t r = 0; r < rows; ++r) {
                const int want = r >= lo && r < hi;
                if (seen.rows[r] != want || seen.back[r] != want) g_wrong = "every row of a sequence once";
            }
        }
        if (g_wrong) {
            std::printf("result ok=0 case=%llu kind=%d rows=%u seqs=%u channels=%u span_rows=%u\n%s\noffsets", (unsigned long long)c,
                        kind, rows, seqs, channels, p.span_rows, g_wrong);
            for (int32_t o : off) std::printf(" %d", o);
            std::printf("\n");
            return 1;
        }
    }
    std::printf("result ok=1 cases=%llu joins=%llu\n", (unsigned long long)cases, (unsigned long long)g_joins);
    return 0;
}
