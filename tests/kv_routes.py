"""Which kernels and layouts the cache, attention and adapter calls choose, from the
library's own host code: a small program built from csrc/mnb_api.cpp and the
host-only stand-ins for the HIP side prints the choice for each batch or shape."""
import os
import random
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_wise_int4_matmulnbits_amd", "csrc")

MAIN = r"""
#include <stdio.h>
#include <string.h>
#include <algorithm>
#include "mnb_internal.h"
// Sequences follow as pairs of new tokens and lengths.
int main()
{
    char op[16];
    long a, b, c, d, e, f;
    while (scanf("%15s %ld %ld %ld %ld %ld %ld", op, &a, &b, &c, &d, &e, &f) == 7) {
        if (!strcmp(op, "append")) {           // page size, tokens, sequences, heads, head dim
            printf("%d\n", (int)mnb::append_one_wave(a, b, c, d, e));
        } else if (!strcmp(op, "many")) {      // tokens, query heads, head dim
            printf("%d\n", mnb::attention_many_rows(a, b, c));
        } else if (!strcmp(op, "shares")) {
            printf("%d %d %d\n", mnb::kAttentionBegin, mnb::kAttentionWorkgroups, mnb::kLoraDownWorkgroups);
        } else if (!strcmp(op, "cut")) {       // sequences, query heads, heads, head dim, tokens
            const mnb::AttentionLayout lay = mnb::attention_layout(e, a, b, c, d);
            const int64_t BR = mnb::tile_rows(d), G = b / c;
            int64_t all = 0, tiles = 0, longest = 0;
            for (long s = 0; s < a; ++s) {
                long n, length;
                if (scanf("%ld %ld", &n, &length) != 2) return 1;
                const int64_t t = n * G > lay.many ? (n * G + BR - 1) / BR : 0;
                const int64_t first = G * (std::max(length - n, 0l) + 64 * mnb::kTileBegin);
                tiles += t;
                if (t) longest = std::max(longest, first + t * BR);
                all += (t * first + BR * (t * (t + 1) / 2)) * c;
            }
            auto divide = [](int64_t x, int64_t y) { return x / y; };
            const int64_t S = lay.shares;
            printf("%d\n", S ? (int)mnb::tiles_cut(all, tiles * c, longest, G, S, mnb::tile_share((all + S - 1) / S, G), divide) : 0);
        } else {                               // lora m K N R adapters
            const mnb::LoraLayout l = mnb::lora_layout(a, b, c, d, e);
            printf("%d %d %d\n", (int)l.wide, l.up_tiles, l.down_tiles);
        }
    }
}
"""


def ragged(S, most, longest):
    """(new tokens, lengths with them) of a batch of differing sequences."""
    r = random.Random(S * longest)
    new = [r.randint(1, most) for _ in range(S)]
    total = [n + int(longest ** r.random()) for n in new]
    total[0] = new[0] + longest
    return new, total


def batch(shape):
    """(new tokens, lengths, page size, query heads, heads, head dim) of a data entry."""
    if shape[0] == "ragged":
        return ragged(*shape[1:4]) + tuple(shape[4:])
    S, n, L = shape[:3]
    return ([n] * S, [L] * S) + tuple(shape[3:])


class Routes:
    def __init__(self, folder):
        main = os.path.join(str(folder), "kv_routes.cpp")
        self.program = os.path.join(str(folder), "kv_routes")
        with open(main, "w") as f:
            f.write(MAIN)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", self.program,
                        main, os.path.join(CSRC, "mnb_api.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "mnb_hip_stub.cpp")], check=True)

    def _ask(self, lines):
        p = subprocess.run([self.program], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        out = [tuple(map(int, line.split())) for line in p.stdout.splitlines()]
        assert len(out) == len(lines), p.stdout
        return out

    def append_threads(self, shapes):
        """Waves of a workgroup."""
        return ["1" if one else "4" for one, in
                self._ask(["append %d %d %d %d %d 0" % (P, S * n, S, h, D) for S, n, _, P, h, D, _ in shapes])]

    def attention_many_rows(self, shapes):
        """Whether a batch of equal sequences goes to the tiles."""
        found = self._ask(["many %d %d %d 0 0 0" % (s[0] * s[1], s[4], s[6]) for s in shapes])
        return ["tiles" if s[1] * (s[4] // s[5]) > many else "rows" for s, (many,) in zip(shapes, found)]

    def attention_cut(self, shapes):
        """Whether tiles are cut into shares."""
        lines = []
        for new, total, _, hq, h, D in map(batch, shapes):
            lines.append("cut %d %d %d %d %d 0 " % (len(new), hq, h, D, sum(new)) +
                         " ".join("%d %d" % pair for pair in zip(new, total)))
        return ["cut" if cut else "whole" for cut, in self._ask(lines)]

    def attention_shares(self, shapes):
        """What a row tile's begin counts as (with the workgroups that stand for the default)."""
        (begin, groups, _), = self._ask(["shares 0 0 0 0 0 0"])
        return ["begin%d" % begin if groups == 512 else "wg%d" % groups] * len(shapes)

    def _lora(self, shapes):
        return self._ask(["lora %d %d %d %d %d 0" % tuple(s[:5]) for s in shapes])

    def lora_up(self, shapes):
        """The second launch: 64 columns a wave, or 16 with tiles of 32 or 64 rows."""
        return ["wide" if wide else "narrow4" if up == 4 else "narrow2" for wide, up, _ in self._lora(shapes)]

    def lora_down(self, shapes):
        """Row tiles of 16 of the first launch."""
        return ["down%d" % down for _, _, down in self._lora(shapes)]

    def lora_splits(self, shapes):
        """Workgroups that the first launch's slices are made for."""
        (_, _, groups), = self._ask(["shares 0 0 0 0 0 0"])
        return ["split%d" % groups] * len(shapes)
