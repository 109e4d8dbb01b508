"""Which kernels the 8-bit operators and the expert layer run, from the
library's own host code: a small program built from csrc/mnb_api.cpp and the
host-only stand-ins for the HIP side prints the choice for each shape, as on a
device of 256 compute units."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_wise_int4_matmulnbits_amd", "csrc")
CUS = 256

# The tiles in the order of their numbers: bytes of K of a stage, stages in LDS.
TILES = {"256x256": (64, 4), "256x128": (128, 3), "128x128": (128, 4), "128x64": (256, 3), "64x64": (256, 3),
         "64x32": (512, 3), "32x32": (512, 4)}

MAIN = r"""
#include <stdio.h>
#include <string.h>
#include "mnb_internal.h"
int main()
{
    char op[16];
    long a, m, K, N, k;
    while (scanf("%15s %ld %ld %ld %ld %ld", op, &a, &m, &K, &N, &k) == 6) {
        if (!strcmp(op, "int8")) {
            const mnb::Int8Route r = mnb::int8_route((int)a, m, K, N, CUS);
            printf("%d %d %d %d\n", r.tile, r.waves, r.nu, (int)r.fused);
        } else if (!strcmp(op, "quantize")) {
            printf("%d\n", mnb::quantize_variant(m, K));
        } else {                       // moe T H I E k; arrays on 256 bytes
            const mnb::MoeLayout l = mnb::moe_layout(a, m, K, N, (int)k);
            mnb::MoeArgs args{};
            args.w.hidden = m;
            args.w.inter = K;
            args.w.experts = N;
            args.T = (int32_t)a;
            args.top_k = (int32_t)k;
            const mnb::MoeRoute r = mnb::moe_route(args, l, CUS);
            printf("%d %d %d %d %d %d\n", l.wide, l.rq, r.up_vec, r.down_vec, r.stage_blocks, r.down_quads);
        }
    }
}
"""


class Routes:
    def __init__(self, folder):
        main = os.path.join(str(folder), "routes.cpp")
        self.program = os.path.join(str(folder), "routes")
        with open(main, "w") as f:
            f.write(MAIN)
        subprocess.run(["g++", "-std=c++17", "-O1", "-DCUS=%d" % CUS, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                        "-o", self.program, main, os.path.join(CSRC, "mnb_api.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "mnb_hip_stub.cpp")], check=True)

    def _ask(self, lines):
        p = subprocess.run([self.program], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        out = [tuple(map(int, line.split())) for line in p.stdout.splitlines()]
        assert len(out) == len(lines), p.stdout
        return out

    def int8(self, shapes):
        """(tile name or None, waves, units of each wave, fused) for (a_dtype, m, K, N)."""
        names = list(TILES)
        return [(names[t] if t >= 0 else None, w, nu, bool(f))
                for t, w, nu, f in self._ask(["int8 %d %d %d %d 0" % s for s in shapes])]

    def quantize(self, shapes):
        """Threads of a row x pieces of each for (m, K)."""
        names = ("64x1", "256x1", "256x8", "1024x1", "1024x4")
        return [names[v] for v, in self._ask(["quantize 0 %d %d 0 0" % s for s in shapes])]

    def moe_choice(self, shapes):
        """(kernels, column quads of the second narrow launch) of (T, H, I, E, k)."""
        return [("wide%d" % (16 * wide) if wide else "narrow%d" % (4 * rq), str(quads))
                for wide, rq, _, _, _, quads in self._ask(["moe %d %d %d %d %d" % s for s in shapes])]

    def moe(self, shapes):
        """The kernel instances of (T, H, I, E, k) with fp16 and with bf16 rows."""
        found = []
        for (T, H, _, _, _), (wide, rq, uv, dv, stage, quads) in zip(shapes, self._ask(["moe %d %d %d %d %d" % s for s in shapes])):
            if wide:
                found.append({"wide up %d vec %d" % (16 * wide, uv), "wide down %d vec %d" % (16 * wide, dv)})
                continue
            mode = "spans" if stage < H // 32 else "tokens" if T <= 4 * rq else "batch"
            found.append({"up %d vec %d %s %s" % (4 * rq, uv, t, mode) for t in ("f16", "bf16")} |
                         {"down %d quads %d vec %d" % (4 * rq, quads, dv)})
        return found
