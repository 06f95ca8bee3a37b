// Host-side check of the scale rows that a warp of the int4 products asks for
// (csrc/int4_mv.cuh part_rows, slice_row, ScaleRows), over sizes of K with odd
// tails, groups, slices and warps: the warps' rows cover K once; every scale
// row asked for exists and belongs to rows that the warp has; and every block
// of rows finds its own group's scales.  Prints "OK <rows asked for>" or the
// first violation.
#include <cstdio>
#include <initializer_list>
#include <random>

#include "int4_mv.cuh"

using namespace l4moe::mv;

static long long asked = 0;

static bool walk(int K, int group, int lg, int parts) {
    const int groups = (int)(((long long)K + group - 1) / group);
    int covered = 0;
    for (int slice = 0; slice < 1 << lg; ++slice) {
        for (int part = 0; part < parts; ++part) {
            int r0, r1;
            const int blocks = part_rows(slice_row(K, slice, lg), slice_row(K, slice + 1, lg), part, parts, r0, r1);
            auto bad = [&](const char* what, int row, int grp) {
                printf("%s: K %d group %d slices %d slice %d warp %d of %d: row %d of [%d, %d), scale row %d of %d\n", what,
                       K, group, 1 << lg, slice, part, parts, row, r0, r1, grp, groups);
                return false;
            };
            if (blocks < 0 || r0 != covered || r1 < r0 || r1 > K) return bad("rows", r0, 0);
            covered = r1;
            ScaleRows scales(r0, group);
            int held = -1;  // the group whose scales the warp holds
            for (int s = 0; s < (blocks + 1) / 2; ++s) {
                const int row = r0 + s * kRows;
                bool due[2];
                scales.stage(row, r1, due[0], due[1]);
                for (int h = 0; h < 2; ++h) {
                    const int grp = h ? scales.grp : scales.first(due[1]);
                    if (due[h]) {
                        ++asked;
                        if (grp < 0 || grp >= groups) return bad("past the scales", row + h * kBlock, grp);
                        if (row + h * kBlock >= r1) return bad("scales of rows past the warp's", row + h * kBlock, grp);
                        held = grp;
                    }
                    if (row + h * kBlock < r1 && held != (row + h * kBlock) / group)
                        return bad("another group's scales", row + h * kBlock, held);
                }
            }
        }
    }
    if (covered != K) printf("K %d: %d rows covered\n", K, covered);
    return covered == K;
}

int main() {
    std::mt19937 rng(1);
    for (int group : {32, 64, 96, 128, 256, 1024, 4128, 1 << 20, 0x7fffffe0}) {
        for (int lg = 0; lg <= 3; ++lg) {
            for (int parts : {2, 4}) {
                for (int K = 1; K <= 2200; K += K < 400 ? 1 : 7)
                    if (!walk(K, group, lg, parts)) return 1;
                for (int i = 0; i < 40; ++i)
                    if (!walk(1 + (int)(rng() % 20000), group, lg, parts)) return 1;
            }
        }
    }
    if (!walk(1 << 30, 1 << 24, 3, 4) || !walk((1 << 30) - 1, 0x7fffffe0, 0, 4)) return 1;
    printf("OK %lld\n", asked);
    return 0;
}
