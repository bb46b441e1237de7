// experts_cut.cu -- how an expert product is cut into tiles (experts.cuh).
#include "experts.h"

namespace moe {

// The cut with the least time for tiles in whole waves over the SMs.  The
// constants are cycles, measured: a stage of 64 (e4m3: 128) of k is bound by
// its bytes, 16 KB of A and 128 per row of B in a block at about 61 a cycle,
// or, for a pair with 256 columns, by the matrix instructions (545); after
// the last stage the accumulator takes about 1000 per 32 columns and group,
// and a joint sum about 2500.  Narrower tiles pay where they fill the last
// wave: 5000 rows, 4096 -> 2048 (160 tiles of 256, 2.1 waves of 76 pairs)
// take 63.6 us 256 wide and 55.6 us 192 wide.
// `live` experts have `n` of the ragged axis together (`each`: wgrad, whose n
// is the same for every expert); their sizes are not known on the host, half
// a tile each is taken for lost.
static Cut pick(int m, long long n, int live, bool each, long long k_stages, bool narrow)
{
    static const Cut cuts[] = {{2, 256, 1}, {2, 224, 1}, {2, 192, 1}, {2, 160, 1}, {2, 128, 1}, {1, 128, 8},
                               {1, 96, 1},  {1, 64, 1},  {1, 32, 8}};
    Cut best = cuts[0];
    double least = 0.0;
    const int sms = device_sm_count();
    for (const Cut &c : cuts) {
        if (!narrow && c.bn != 256 && c.bn != 128) continue;  // wgrad loads B by 64 columns
        const long long tm = (m + 128 * c.cg - 1) / (128 * c.cg);
        long long tn = live == 1 || each ? (n + c.bn - 1) / c.bn * (each ? live : 1) : n / c.bn + (live + 1) / 2;
        if (tn < live) tn = live;
        const double bytes = 270.0 + 2.1 * c.bn / c.cg, mma = 2.13 * c.bn;
        const double stage = c.cg == 2 && mma > bytes ? mma : bytes;
        for (int split = 1; split <= c.split; split *= 2) {
            if (split > 1 && k_stages < 4 * split) break;
            // clusters of 4 and 8 leave some SMs of a GPC over
            const long long slots = split < 4 ? sms / (c.cg * split) : sms * 7 / 8 / split;
            // unknown sizes: 15 % more tiles, or a full last wave turns into two
            const long long tiles = live == 1 || each ? tm * tn : tm * tn * 23 / 20;
            const long long waves = (tiles + slots - 1) / slots;
            const double cycles = (double)waves * k_stages / split * stage + 1000.0 * ((c.bn / split + 63) / 64) +
                                  (split > 1 ? 2500.0 * waves : 0.0);
            if (least == 0.0 || cycles < least) {
                least = cycles;
                best = {c.cg, c.bn, split};
            }
        }
    }
    return best;
}

Cut rows_cut(int m, int rows, int E, long long k_stages)
{
    return pick(m, rows, rows < E ? rows : E, false, k_stages, true);
}

Cut wgrad_cut(int N, int K, int rows, int E) { return pick(N, K, E, true, (rows / E + 63) / 64, false); }

}  // namespace moe
