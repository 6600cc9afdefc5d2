// Host driver of the arithmetic by which the attention kernels cut their line
// of steps (tests/test_attention_sanitizers.py), built with the address and
// undefined-behaviour sanitizers. Random sequence starts, in order and not:
// no piece leaves a partial result past the places that the host makes room
// for, and starts in order are counted and cut exactly.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "attn_line.h"

using namespace ck4;

static int g_failures = 0, g_cut = 0, g_refused = 0;

static void expect(bool ok, const char *what, int64_t a, int64_t b) {
    if (ok) return;
    if (++g_failures < 20) std::printf("FAIL %s: %lld %lld\n", what, (long long)a, (long long)b);
}

// Steps of a tile by their definition.
template <bool KEYS>
static int64_t steps_of(const Span &s, bool causal, int group, int tile) {
    if (!KEYS) {
        const int last = std::min(tile * 256 + 255, s.nq - 1);
        return std::max((limit(s, causal, last) + 63) / 64, 1);
    }
    const int shift = s.nk - s.nq, first = causal ? std::max(tile * 256 - shift, 0) : 0;  // the first row that sees a key
    return (int64_t)std::max((s.nq + 63) / 64 - first / 64, 1) * group;
}

template <bool KEYS>
static void check(const std::vector<int> &cu_q, const std::vector<int> &cu_k, int tq, int tk, int heads, int group,
                  bool causal, bool ordered) {
    const int seqs = (int)cu_q.size() - 1;
    const int most = most_steps<256, KEYS>(seqs, tq, tk, heads, group);
    expect(partial_floats(most, 10) == 20 * (int64_t)most_pieces(most) && (most > 0) == (partial_floats(most, 10) > 0),
           "room", most, most_pieces(most));
    if (most == 0) return;
    LineSum lanes[64];
    int64_t exact = 0, longest = 0;
    for (int i = 0; i < seqs; ++i) {
        const Span s = span_between(tq, tk, cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]);
        expect(s.q0 >= 0 && s.nq >= 0 && s.q0 + s.nq <= tq && s.k0 >= 0 && s.nk >= 0 && s.k0 + s.nk <= tk, "rows", i, seqs);
        const auto r = ramp_of<256, KEYS>(s, causal, group);
        int64_t sum = 0;
        for (int t = 0; t < r.tiles; ++t) {  // keys in falling order
            expect(r.before(t) == sum, "steps before a tile", r.before(t), sum);
            const int64_t n = steps_of<KEYS>(s, causal, group, KEYS ? r.tiles - 1 - t : t);
            expect(r.steps(t) == n, "steps of a tile", r.steps(t), n);
            sum += n;
            longest = std::max(longest, n);
        }
        expect(r.before(r.tiles) == sum && sum * heads <= most, "steps of a sequence", sum * heads, most);
        exact += sum * heads;
        lanes[i % 64].add(r, heads, most);
    }
    // over the lanes as a wavefront adds them
    for (int step = 32; step > 0; step /= 2) {
        LineSum next[64];
        for (int l = 0; l < 64; ++l) {
            next[l].total = add_steps(lanes[l].total, lanes[l ^ step].total, most);
            next[l].longest = std::max(lanes[l].longest, lanes[l ^ step].longest);
        }
        std::copy(next, next + 64, lanes);
    }
    const LineSum sum = lanes[0];
    expect(sum.total == std::min(exact, (int64_t)most + 1), "total", sum.total, exact);
    expect(sum.longest == longest, "longest", sum.longest, longest);
    if (ordered) expect(exact <= most, "starts in order fit", exact, most);
    const Cut c(sum, most);
    if (exact > most) {
        expect(c.count == 0, "a line past its bound is not cut", c.count, exact);
        ++g_refused;
    }
    if (c.count == 0) return;
    ++g_cut;
    const int64_t room = 2 * (int64_t)most_pieces(most);
    for (int w = 0; w < c.count; ++w) {
        expect(Cut::place(w, true) < room && Cut::place(w, false) < room, "place of a partial result", w, room);
        expect(c.piece_of(c.start(w)) == w && c.piece_of(c.start(w + 1) - 1) == w, "piece", w, c.start(w));
    }
    expect(c.start(0) == 0 && c.start(c.count) == exact, "the pieces cover the line", c.start(c.count), exact);
}

static void both(const std::vector<int> &cu_q, const std::vector<int> &cu_k, int tq, int tk, int hq, int hk, bool ordered) {
    for (bool causal : {false, true}) {
        check<false>(cu_q, cu_k, tq, tk, hq, 1, causal, ordered);
        check<true>(cu_q, cu_k, tq, tk, hk, hq / hk, causal, ordered);
    }
}

int main() {
    std::mt19937 g(1);
    const auto upto = [&](int n) { return (int)(g() % (unsigned)(n + 1)); };
    for (int i = 0; i < 20000; ++i) {
        const auto rows = [&]() { return 1 + upto((1 << (4 + upto(i % 10 ? 10 : 26))) - 1); };  // up to 2^30
        const int tq = rows(), tk = rows();
        const int seqs = 1 + upto(i % 3 ? 9 : 130), hk = 1 + upto(4), hq = hk * (1 + upto(4));
        std::vector<int> cu_q(seqs + 1), cu_k(seqs + 1);
        for (int &v : cu_q) v = upto(tq);
        for (int &v : cu_k) v = upto(tk);
        if (i % 4 == 0)  // all rows in every other sequence
            for (int n = 0; n <= seqs; ++n) cu_q[n] = n % 2 ? tq : 0, cu_k[n] = n % 2 ? tk : 0;
        if (i % 4 == 1)  // outside the tensors
            for (int n = 0; n <= seqs; ++n) cu_q[n] = n % 2 ? INT_MAX : INT_MIN, cu_k[n] = n % 3 ? INT_MAX - n : -n;
        both(cu_q, cu_k, tq, tk, hq, hk, false);
        std::sort(cu_q.begin(), cu_q.end());
        std::sort(cu_k.begin(), cu_k.end());
        cu_q[0] = cu_k[0] = 0;
        cu_q[seqs] = tq;
        cu_k[seqs] = tk;
        both(cu_q, cu_k, tq, tk, hq, hk, true);
    }
    std::printf("%d lines cut, %d past their bound, %d failures\n", g_cut, g_refused, g_failures);
    return g_failures != 0 || g_cut < 1000 || g_refused < 1000;
}
