// Host walk over the units of the windowed kernels: every (row, key) pair that the
// definition shows is covered exactly once, and no other one.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "cp_common.cuh"

using namespace cp;

static bool seen(const Window &w, int p, int j) { return j <= p && (j > p - w.window || j < w.sinks); }

template <int TILE>
static void rows_walk(const Window &w, int Sq, int Sk, int qt)
{
    for (int q0 = 0; q0 < Sq; q0 += qt) {
        const int p0 = q0 + w.off, p1 = (q0 + qt < Sq ? q0 + qt : Sq) - 1 + w.off;
        std::vector<int> hit((size_t)(p1 - p0 + 1) * Sk, 0);
        WinIter<TILE> it;
        int tiles = 0;
        for (it.begin(w, p0, p1); it.valid(); it.next(), ++tiles) {
            const int kl = it.len(), ks = it.start();
            if (kl < 1 || kl > TILE) exit((printf("len %d\n", kl), 1));
            for (int p = p0; p <= p1; ++p) {
                const int hi = p - ks + 1 < kl ? p - ks + 1 : kl;
                for (int c0 = 0; c0 < TILE; c0 += 32) {
                    const uint32_t bits = visible_bits(c0, hi, it.window_col(w, p), it.sink_cols());
                    for (int c = c0; c < c0 + 32; ++c) {
                        const bool on = it.full(w, p0, p1) || (bits >> (c - c0) & 1u);
                        if (!on) continue;
                        const int key = it.packed() && c < it.pk ? c : ks + c;
                        if (key < 0 || key >= Sk || !seen(w, p, key)) exit((printf("p %d key %d\n", p, key), 1));
                        ++hit[(size_t)(p - p0) * Sk + key];
                    }
                }
            }
        }
        if (tiles != WinIter<TILE>::count(w, p0, p1)) exit((printf("count\n"), 1));
        for (int p = p0; p <= p1; ++p)
            for (int j = 0; j < Sk; ++j)
                if (hit[(size_t)(p - p0) * Sk + j] != (seen(w, p, j) ? 1 : 0))
                    exit((printf("Sq %d Sk %d W %d K %d pack %d p %d j %d: %d\n", Sq, Sk, w.window, w.sinks, w.pack, p, j,
                                 hit[(size_t)(p - p0) * Sk + j]),
                          1));
    }
}

template <int KEYS, int TILE>
static void keys_walk(const Window &w, int Sq, int Sk, int grp)
{
    const SinkPlan sp = sink_plan<KEYS, TILE>(w, Sq, Sk, grp);
    std::vector<int> hit((size_t)grp * Sq * Sk, 0);
    auto add = [&](WinQIter<TILE> it, int ks, int kl, bool sinks) {
        for (; it.count() > 0; it.next())
            for (int c = 0; c < it.len(); ++c)
                for (int j = ks; j < ks + kl; ++j) {
                    const int row = it.start() + c, back = row + w.off - j;
                    if (row < 0 || row >= Sq || it.head() < 5 || it.head() >= 5 + grp) exit((printf("row %d\n", row), 1));
                    if (sinks ? j < w.sinks && back >= w.window : back >= 0 && back < w.window)
                        ++hit[((size_t)(it.head() - 5) * Sq + row) * Sk + j];
                }
    };
    for (int ks = 0; ks < Sk; ks += KEYS) {
        const int kl = Sk - ks < KEYS ? Sk - ks : KEYS;
        WinQIter<TILE> it;
        it.window(w, Sq, ks, kl, 5, grp);
        add(it, ks, kl, false);
        if (ks / KEYS < sp.tiles)
            for (int p = 0; p < sp.pieces; ++p) {
                it.sinks(w, Sq, ks, 5, grp, p, sp.each);
                add(it, ks, kl, true);
            }
    }
    for (int h = 0; h < grp; ++h)
        for (int i = 0; i < Sq; ++i)
            for (int j = 0; j < Sk; ++j)
                if (hit[((size_t)h * Sq + i) * Sk + j] != (seen(w, i + w.off, j) ? 1 : 0))
                    exit((printf("keys: Sq %d Sk %d W %d K %d row %d key %d: %d\n", Sq, Sk, w.window, w.sinks, i, j,
                                 hit[((size_t)h * Sq + i) * Sk + j]),
                          1));
}

int main()
{
    const int sizes[][2] = {{1, 1}, {1, 400}, {130, 130}, {257, 257}, {300, 513}, {600, 600}, {64, 700}};
    const int windows[] = {1, 2, 16, 63, 64, 65, 100, 127, 128, 129, 255, 256, 300, 700};
    const int sinks[] = {0, 1, 4, 16, 17, 48, 64, 65, 130, 300, 700};
    for (const auto &s : sizes)
        for (int W : windows)
            for (int K : sinks)
                for (int packed = 0; packed < 2; ++packed) {
                    Window w{s[1] - s[0], W < s[1] ? W : s[1], K < s[1] ? K : s[1], 0};
                    if (packed) w.pack = w.sinks <= 64 ? (w.sinks + 15) / 16 * 16 : 0;
                    rows_walk<256>(w, s[0], s[1], 128);
                    rows_walk<128>(w, s[0], s[1], 128);
                    if (packed) w.pack = w.sinks <= 32 ? w.sinks : 0;
                    rows_walk<64>(w, s[0], s[1], 32);
                    if (packed) continue;
                    keys_walk<128, 128>(w, s[0], s[1], 1);
                    keys_walk<32, 64>(w, s[0], s[1], 3);
                }
    // the launches' divisions
    const uint32_t ds[] = {1, 2, 3, 5, 7, 8, 12, 31, 32, 33, 96, 127, 1000, 4095, 65537, 16777215, 1073741825, 2147483647};
    for (uint32_t d : ds) {
        const FastDiv f = fast_div(d);
        const uint32_t us[] = {0, 1, d - 1, d, d + 1, 2 * d - 1, 2147483647, 2147483646, 2147483647 / d * d, 2147483647 / d * d - 1};
        for (uint32_t u : us)
            if (u < 2147483648u && f.div(u) != u / d) return printf("%u / %u\n", u, d), 1;
        for (uint32_t i = 0; i < 200000; ++i) {
            const uint32_t u = (i * 2654435761u) >> 1;
            if (f.div(u) != u / d) return printf("%u / %u\n", u, d), 1;
        }
    }
    // positions near the largest
    Window w{0x7ffffbff - 200, 0x7ffffbff, 4, 16};
    WinIter<256> it;
    it.begin(w, w.off, w.off + 199);
    if (it.lo != 0 || it.nt <= 0) return printf("large\n"), 1;
    w.window = 100;
    it.begin(w, w.off, w.off + 199);
    if (it.nt != 2 || it.pk != 16) return printf("large, window\n"), 1;
    printf("ok\n");
    return 0;
}
