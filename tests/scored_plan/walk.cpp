// Replays on the host the walk of the score-shaped attention's tile kernel, with
// the planner and the geometry functions that the kernel itself uses. Reads
// problems from standard input, one a line:
//   B T H W NH HD KT KH KW options mode   (options: 1 documents, 2 a cap, 3 both;
//                                          mode 0 forward, 1 dQ, 2 dK and dV)
// and checks for every brick, warp and chunk that what is read lies inside the
// grid and what is staged inside its buffer. Prints one line for each problem:
// "ok <chunks>", "unplanned", or the first thing that is wrong.
#include <cstdio>

#include "na3d_scored_plan.cuh"

using namespace na3d;
using namespace na3d::scored;

#define WANT(cond)                                                                             \
    do {                                                                                       \
        if (!(cond)) {                                                                         \
            std::printf("wrong: %s (brick %d %d %d, warp %d, frame %d, chunk %d %d)\n", #cond, \
                        x.o.t0, x.o.h0, x.o.w0, warp, t, ih, iw);                              \
            return;                                                                            \
        }                                                                                      \
    } while (0)

template <bool DKV>
void walk(const ScoredParams& p, const TileGeom& g) {
    long long chunks = 0;
    Unit x = unit_of<DKV>(p, g, g.units - g.bricks / p.B);   // the bricks of the last entry's last head
    for (int u = g.units - g.bricks / p.B; u < g.units; ++u, next_unit<DKV>(p, g, x)) {
        int warp = -1, t = -1, ih = -1, iw = -1;
        const Unit again = unit_of<DKV>(p, g, u);
        WANT(again.head == p.NH - 1 && again.o.b == p.B - 1);
        WANT(again.o.t0 == x.o.t0 && again.o.h0 == x.o.h0 && again.o.w0 == x.o.w0 && again.o.b == x.o.b);
        // the chunks cover the box
        WANT(x.bt.x >= 0 && x.bt.y <= p.T && x.bh.x >= 0 && x.bh.y <= p.H && x.bw.x >= 0 && x.bw.y <= p.W);
        WANT(x.bt.y - x.bt.x <= g.nt && x.bh.y - x.bh.x <= g.nhc * g.cr && x.bw.y - x.bw.x <= g.nwc * g.cc);
        for (warp = 0; warp < g.nw; ++warp) {
            const int2 mine = warp_rows<DKV>(p, g, x, warp);
            for (int it = 0; it < g.nt; ++it) {
                t = x.bt.x + it;
                int steps = 0;
                for (ih = 0; ih < g.nhc; ++ih)
                    for (iw = 0; iw < g.nwc; ++iw, ++chunks) {
                        const Part o = part_of(g, x, mine, ih, iw);
                        const int n = o.n > 0 ? (o.n + 15) / 16 : 0;
                        steps += n;
                        WANT(n <= g.chunk_steps && 16 * n <= g.cr * g.cc + 15);
                        WANT(steps <= g.frame_steps);
                        if (n == 0 || !has_frame(x, t)) continue;
                        // columns of the part: documents and statistics are read at (t, hf + row, w + column)
                        // where the column is inside W
                        const int rows = (o.n + g.cc - 1) / g.cc;
                        WANT(t >= 0 && t < p.T);
                        WANT(o.hf >= 0 && o.hf + rows <= p.H && o.w >= 0);
                        // ... and its rows in a stage, with the last step's past the part
                        const int first = (o.hf - x.bh.x - ih * g.cr) * g.cc;
                        WANT(first >= 0 && first + 16 * n <= g.cr * g.cc + 16);
                    }
                ih = iw = -1;
            }
            t = -1;
        }
    }
    std::printf("ok %lld\n", chunks);
}

int main() {
    int hd, docs, mode;
    ScoredParams p{};
    int32_t one = 0;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &p.B, &p.T, &p.H, &p.W, &p.NH, &hd, &p.KT, &p.KH, &p.KW,
                      &docs, &mode) == 11) {
        p.doc = docs & 1 ? &one : nullptr;
        p.softcap = docs & 2 ? 1.f : 0.f;
        TileGeom g;
        if (!plan_tiles(&g, p, hd, mode, 152)) std::printf("unplanned\n");
        else if (g.smem > kSmemMax / blocks_per_sm(hd, mode) || g.cc > 256 || g.cr > 256 || g.bh > 256 ||
                 g.off_x < 0 || g.off_stat < g.off_x || g.off_doc < g.off_stat || g.off_lut < g.off_doc ||
                 g.off_hw < g.off_lut || g.off_bar < g.off_hw || g.smem < g.off_bar)
            std::printf("wrong: shared memory of %d bytes, box %d x %d\n", g.smem, g.cr, g.cc);
        else if (mode == kDkv) walk<true>(p, g);
        else walk<false>(p, g);
    }
    return 0;
}
