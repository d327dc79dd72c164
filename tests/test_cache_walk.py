"""How the cache attention's work is cut (no GPU): the host side of the functions in
csrc/cache_walk.cuh, compiled into a small program that checks them against counting."""
import subprocess

from compressed_attention_adaptive_gb300 import build as mita_build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "cache_walk.cuh"
using namespace mita;

static int failed = 0;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); ++failed; } } while (0)

static Line make_line(const CacheArgs& a, int rtile, int extra, int max_pieces) {
    Line l{};
    l.extra = extra;
    for (int b = 0; b < a.B; ++b) {
        const SeqWork s = seq_work(a, b, rtile);
        l.total += s.items * (s.chunks + extra);
    }
    l.pieces = l.total < max_pieces ? l.total : max_pieces;
    l.q = l.pieces ? l.total / l.pieces : 0;
    l.r = l.total - l.q * l.pieces;
    return l;
}

static void counted(int seed) {
    srand(seed);
    CacheArgs a{};
    a.B = 1 + rand() % 40;
    a.Hkv = 1 + rand() % 3;
    a.G = 1 + rand() % 9;
    a.T = 1 + rand() % 5;
    a.page = 16;
    a.cols = 64;
    std::vector<int> len(a.B), count(a.B);
    for (int b = 0; b < a.B; ++b) {
        len[b] = rand() % 3 ? rand() % 1024 : 0;
        count[b] = rand() % (a.T + 1);
    }
    a.len = len.data();
    a.count = count.data();
    const int rtile = 8, extra = rand() % 3;
    const Line l = make_line(a, rtile, extra, 1 + rand() % 200);
    // every unit by counting: its sequence, its piece, and the pieces that an item goes over
    int w = 0;
    std::vector<int> piece_at;
    for (int p = 0; p < l.pieces; ++p)
        for (int x = l.at(p); x < l.at(p + 1); ++x) piece_at.push_back(p);
    CHECK((int)piece_at.size() == l.total);
    for (int b = 0; b < a.B; ++b) {
        const SeqWork s = seq_work(a, b, rtile);
        for (int j = 0; j < s.items; ++j) {
            for (int u = 0; u < s.chunks + extra; ++u, ++w) {
                int before = 0;
                SeqWork sw = seq_work(a, 0, rtile);
                CHECK(find_unit(a, l, rtile, w, 0, a.B, &before, &sw) == b);
                CHECK(w >= before && (w - before) / (s.chunks + extra) == j);
                CHECK(l.piece_of(w) == piece_at[w]);
                int piece = -1;
                const int first = before + j * (s.chunks + extra) + extra;
                CHECK(item_pieces(l, s, before, j, &piece) == piece_at[first + s.chunks - 1] - piece_at[first] + 1);
                CHECK(piece == piece_at[first]);
            }
        }
    }
}

// Lengths that change between the reading of the line and the search: nothing behind the
// sequences is read, and no part lies past the pieces.
static void changed() {
    CacheArgs a{};
    a.B = 6;
    a.Hkv = a.G = a.T = 1;
    a.page = 16;
    a.cols = 64;
    // what lies behind the six lengths would be found if it were read
    std::vector<int> len = {1000, 1000, 1000, 1000, 1000, 1000, 1000, 1000, 1000, 1000};
    a.len = len.data();
    const Line l = make_line(a, 8, 0, 20);
    for (int b = 0; b < a.B; ++b) len[b] = 10;
    for (int w = 0; w < l.total; ++w) {
        int before = 0;
        SeqWork sw = seq_work(a, 0, 8);
        CHECK(find_unit(a, l, 8, w, 0, a.B, &before, &sw) == (w < 6 ? w : -1));
        before = 3;
        sw = seq_work(a, 3, 8);
        CHECK(find_unit(a, l, 8, w, 3, 5, &before, &sw) == (w < 4 ? 3 : w < 5 ? 4 : -1));
    }
    for (int b = 0; b < a.B; ++b) len[b] = 1024;
    int piece = -1;
    for (int before = 0; before < 2 * l.total; ++before) {
        const int parts = item_pieces(l, seq_work(a, 0, 8), before, 0, &piece);
        CHECK(parts == 0 || (piece >= 0 && piece + parts <= l.pieces));
        CHECK((parts > 0) == (before + 8 <= l.total));
    }
    Line none{};  // a call without rows
    CHECK(item_pieces(none, seq_work(a, 0, 8), 0, 0, &piece) == 0);
}

// Whatever the arrays hold: lengths and counts end in range, and a group is one of the pool's or none.
static void any_numbers() {
    const int odd[] = {0, 1, -1, 4, 5, 63, 64, 65, 1 << 30, 2147483647, -2147483647 - 1, 127, 128, 200};
    const int k = sizeof odd / sizeof odd[0];
    for (int page = 16; page <= 48; page += 16) {
        CacheArgs a{};
        a.B = k;
        a.Hkv = 3;
        a.T = 5;
        a.page = page;
        a.pgroups = page / 16;
        a.n_pages = 5;
        a.cols = 4;
        std::vector<int> table;
        for (int i = 0; i < k * a.cols; ++i) table.push_back(odd[i * 5 % k]);
        a.table = table.data();
        a.len = a.count = odd;
        for (int b = 0; b < k; ++b) {
            const int n = cache_len(a, b), c = cache_count(a, b);
            CHECK(n >= 0 && n <= a.cols * page && (n == odd[b]) == (odd[b] >= 0 && odd[b] <= a.cols * page));
            CHECK(c >= 0 && c <= a.T && (c == odd[b]) == (odd[b] >= 0 && odd[b] <= a.T));
            for (int gi = 0; gi * 16 < a.cols * page; ++gi)
                for (int h = 0; h < a.Hkv; ++h) {
                    const int pg = table[b * a.cols + gi / a.pgroups], g = cache_group(a, b, h, gi);
                    if (pg < 0 || pg >= a.n_pages)
                        CHECK(g == -1);
                    else
                        CHECK(g == (pg * a.Hkv + h) * a.pgroups + gi % a.pgroups);
                }
        }
    }
}

int main() {
    any_numbers();
    for (int i = 0; i < 300; ++i) counted(i);
    changed();
    if (!failed) printf("ok\n");
    return failed != 0;
}
"""


def test_line_of_pieces(tmp_path):
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(PROGRAM)
    cmd = [mita_build._nvcc()] + mita_build.ARCH + ["-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", mita_build.CSRC,
                                                    str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:]
