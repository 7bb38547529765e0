// hl_reorder_plan.h -- what headloss_reorder decides on the host: whether its states share memory, and how many
// units of work a line is.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <new>

#include "headloss_beam.h"

namespace hl_reorder {

// The bytes base + i0 step0 + i1 step1 + i2 step2 + [0, run), each i below its n.
struct Box {
    int64_t base, n[3], step[3], run;
    int64_t end() const {  // one behind the last; past 2^63 it counts as there
        __int128 e = __int128(base) + run;
        for (int k = 0; k < 3; ++k) e += __int128(n[k] - 1) * step[k];
        return e > INT64_MAX ? INT64_MAX : int64_t(e);
    }
};

inline Box box_of(const headloss_state& s, const void* at, int64_t rows) {
    return {int64_t(reinterpret_cast<uintptr_t>(at)), {rows, s.outer, s.positions},
            {rows > 1 ? s.row_stride : 0, s.outer > 1 ? s.outer_stride : 0, s.positions > 1 ? s.position_stride : 0}, s.run_bytes};
}

// Whether two boxes share a byte: whether indices exist with -b.run < (b's byte - a's byte) < a.run. The steps from the
// longest to the shortest, each index only where the shorter steps can still reach; of layouts whose steps nest that
// leaves two or three a step. `budget` bounds the search; used up, the answer is yes.
inline bool share(const Box& a, const Box& b, int64_t& budget) {
    struct Term {
        int64_t step, lo, hi;
    } t[6];
    int n = 0;
    auto add = [&](int64_t step, int64_t lo, int64_t hi) {
        if (step == 0 || lo == hi) return;
        for (int k = 0; k < n; ++k)
            if (t[k].step == step) {
                t[k].lo += lo, t[k].hi += hi;
                return;
            }
        t[n++] = {step, lo, hi};
    };
    for (int k = 0; k < 3; ++k) {
        add(a.step[k], 1 - a.n[k], 0);
        add(b.step[k], 0, b.n[k] - 1);
    }
    std::sort(t, t + n, [](const Term& x, const Term& y) { return x.step > y.step; });
    __int128 low[7], high[7];  // what the steps from k on can add
    low[n] = high[n] = 0;
    for (int k = n - 1; k >= 0; --k) {
        low[k] = low[k + 1] + __int128(t[k].lo) * t[k].step;
        high[k] = high[k + 1] + __int128(t[k].hi) * t[k].step;
    }
    auto floor_div = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };  // y > 0
    auto search = [&](auto&& self, int k, __int128 d) -> bool {
        if (--budget < 0) return true;
        if (k == n) return -b.run < d && d < a.run;
        const __int128 from = -floor_div(-(1 - b.run - high[k + 1] - d), t[k].step);  // rounded up
        const __int128 to = floor_div(a.run - 1 - low[k + 1] - d, t[k].step);
        const __int128 last = to < t[k].hi ? to : t[k].hi;
        for (__int128 v = from > t[k].lo ? from : t[k].lo; v <= last; ++v)
            if (self(self, k + 1, d + v * t[k].step)) return true;
        return false;
    };
    return search(search, 0, __int128(b.base) - a.base);
}

constexpr int64_t SEARCH = 1 << 26;  // steps of one check: tenths of a second

// Whether memory that one state's `rows` rows write is read or written for another, or read in another place for the
// same: such rows would depend on the order of the threads. True, too, where there is no memory for the check.
inline bool conflict(const headloss_state* states, int n, int64_t rows) {
    struct Use {
        Box box;
        int64_t end;
        bool writes;
    };
    Use* uses = new (std::nothrow) Use[2 * size_t(n)];
    int* open[2] = {new (std::nothrow) int[2 * size_t(n)], new (std::nothrow) int[2 * size_t(n)]};  // reads, writes
    bool found = !uses || !open[0] || !open[1];
    int m = 0, opened[2] = {0, 0};
    for (int i = 0; i < n && !found; ++i) {
        const headloss_state& s = states[i];
        uses[m].box = box_of(s, s.out, rows);
        uses[m].writes = true;
        ++m;
        if (s.state != s.out) {
            uses[m].box = box_of(s, s.state, rows);
            uses[m].writes = false;
            ++m;
        }
    }
    for (int i = 0; i < m; ++i) uses[i].end = uses[i].box.end();
    if (!found) std::sort(uses, uses + m, [](const Use& x, const Use& y) { return x.box.base < y.box.base; });
    int64_t budget = SEARCH;
    for (int i = 0; i < m && !found; ++i) {
        const Use& u = uses[i];
        for (int w = u.writes ? 0 : 1; w < 2 && !found; ++w) {
            int kept = 0;
            for (int k = 0; k < opened[w] && !found; ++k) {
                const Use& v = uses[open[w][k]];
                if (v.end <= u.box.base) continue;
                open[w][kept++] = open[w][k];
                found = share(v.box, u.box, budget);
            }
            if (!found) opened[w] = kept;
        }
        open[u.writes][opened[u.writes]++] = i;
    }
    delete[] uses;
    delete[] open[0];
    delete[] open[1];
    return found;
}

// The states without those that are the same as one before them (which is moved once for all); their number.
inline int without_repeats(const headloss_state* from, int n, headloss_state* to) {
    auto less = [](const headloss_state& x, const headloss_state& y, bool& equal) {
        const int64_t a[8] = {int64_t(uintptr_t(x.state)), int64_t(uintptr_t(x.out)), x.outer, x.positions, x.run_bytes,
                              x.row_stride, x.outer > 1 ? x.outer_stride : 0, x.positions > 1 ? x.position_stride : 0};
        const int64_t b[8] = {int64_t(uintptr_t(y.state)), int64_t(uintptr_t(y.out)), y.outer, y.positions, y.run_bytes,
                              y.row_stride, y.outer > 1 ? y.outer_stride : 0, y.positions > 1 ? y.position_stride : 0};
        equal = std::equal(a, a + 8, b);
        return std::lexicographical_compare(a, a + 8, b, b + 8);
    };
    int* order = new (std::nothrow) int[n];
    bool* again = new (std::nothrow) bool[n]();
    int m = -1;
    if (order && again) {
        for (int i = 0; i < n; ++i) order[i] = i;
        bool equal;
        std::sort(order, order + n, [&](int i, int j) {
            const bool before = less(from[i], from[j], equal);
            return equal ? i < j : before;
        });
        for (int i = 1; i < n; ++i) {
            (void)less(from[order[i - 1]], from[order[i]], equal);
            again[order[i]] = equal;
        }
        m = 0;
        for (int i = 0; i < n; ++i)
            if (!again[i]) to[m++] = from[i];
    }
    delete[] order;
    delete[] again;
    return m;
}

// The shares of a line, of lines (below 2^31) whose longest has `most` words in `chunks` of a CTA's: enough for four
// units a CTA, so that lines of different lengths even out, and for eight where a unit still has 4096 words (16 caches of
// 16 x 4 beams 66 and 64 us; 32 caches of one request, 8192 words a line, 8.5 and 11). The units, and a step of the
// grid past the last of them, are counted in 32 bits.
inline int64_t shares_of(int64_t lines, int64_t most, int64_t chunks, int64_t grid) {
    int64_t shares = (4 * grid + lines - 1) / lines;
    if (most / (2 * shares) >= 4096 && 2 * shares * lines <= INT32_MAX) shares *= 2;
    return shares < chunks ? shares : chunks;
}

}  // namespace hl_reorder
