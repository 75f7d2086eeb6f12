// Host-side walk of gemm_pair_kernel's rings, built and run by test_pair_rings.py.
//
// For every CTA of a plan it goes through the share's segments as the dequantizing groups do and
// checks what their waits rest on.  A barrier's wait returns at once when the phase before the
// awaited one has not completed either (one parity bit), so for each wait the phase before has
// to be known complete from what the same group has waited for already.
//   argv[1] = 1: the groups start every segment anew (group k with its k-th block), which
//   must be found at fault.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "../weight_only_quantization_rtn_b200/csrc/pair_plan.cuh"

using namespace w4a16;

static bool g_restart = false;
static long g_plans = 0, g_waits = 0, g_faults = 0;

static void fault(const char* what, int64_t M, int64_t rows, int64_t blocks, int sms, int j) {
    if (g_faults++ < 5)
        std::printf("%s: M=%ld rows=%ld blocks=%ld sms=%d block %d\n", what, (long)M, (long)rows, (long)blocks, sms, j);
}

template <bool PAIR, int BITS, bool DGRAD>
static void check(int64_t M, int64_t rows, int64_t blocks, int sms) {
    using Cfg = PairConfig<PAIR, BITS, DGRAD>;
    constexpr int UB = Cfg::kUnitBlocks, NG = Cfg::kGroups;
    const PairPlan p = pair_plan(M, rows, DGRAD ? 2 * kPairRows : kPairRows, blocks, UB, sms);
    if ((p.ctas == 2) != PAIR) std::abort();
    ++g_plans;
    PairArgs a{};
    pair_plan_args(p, &a);
    a.products = 1;
    const PairRings r = pair_rings<Cfg>(a.bt, a.acc_cols, a.blocks);
    // steps that the kernel takes without a modulus, ring sizes, shared memory, tensor memory
    if (NG > r.na || NG > r.sx || (UB - 1 + NG) / UB > r.sp || r.na > kPairMaxA || r.sp > kPairMaxX || r.sx > kPairMaxX ||
        r.sp * Cfg::kUnitBytes + r.sx * a.bt * kPairBlock * 2 > Cfg::kLoads ||
        (Cfg::kTmemA ? 2 * a.acc_cols + 64 * r.na > 512 : 2 * a.acc_cols > 512))
        fault("ring sizes", M, rows, blocks, sms, 0);
    int64_t covered = 0;
    for (int slot = 0; slot < p.grid; ++slot) {
        PairWalk<UB> w;
        w.init(a, slot, p.grid);
        int cnt = 0, units = 0;
        int last[NG];                                  // each group's last block, -1: none
        int unit_of[4096], first_of[4096];             // unit of a block; first block of a unit (of the last ones)
        for (int& l : last) l = -1;
        std::set<int> own[NG];                         // blocks that a group dequantized
        while (w.next(a, p.grid)) {
            const int nb = w.count(a);
            covered += w.units;
            for (int i = 0; i < nb; ++i) unit_of[(cnt + i) % 4096] = units + i / UB;
            for (int u = 0; u < w.units; ++u) first_of[(units + u) % 4096] = cnt + u * UB;
            for (int i = 0; i < nb; ++i) {
                const int j = cnt + i, u = unit_of[j % 4096];
                const int grp = g_restart ? i % NG : j % NG;
                if (!g_restart && pair_first(cnt, grp, NG) % NG != i % NG) std::abort();
                g_waits += 3;
                const int done = j - r.na;             // its MMAs are complete once the A slot is free
                // A slot: the MMAs of block j - 2·NA
                if (j >= 2 * r.na && last[grp] - r.na < j - 2 * r.na) fault("A slot", M, rows, blocks, sms, j);
                // code unit: a block of the unit that held the slot before was dequantized
                if (u >= r.sp) {
                    const int f = first_of[(u - r.sp) % 4096];
                    bool known = f <= done;
                    for (int b : own[grp]) known = known || (b >= f && unit_of[b % 4096] == u - r.sp);
                    if (!known) fault("code unit", M, rows, blocks, sms, j);
                }
                // tokens: block j - SX was multiplied
                if (j >= r.sx && j - r.sx > done) fault("tokens", M, rows, blocks, sms, j);
                last[grp] = j;
                own[grp].insert(j);
                if (own[grp].size() > 16) own[grp].erase(own[grp].begin());
            }
            cnt += nb;
            units += w.units;
            if (cnt > 3000) break;                     // (the tables above; steady by then)
        }
        if (cnt > 3000) covered = -1;
        if (covered < 0) break;
    }
    if (covered >= 0 && covered != p.tiles * PairWalk<UB>::upt(a)) fault("coverage", M, rows, blocks, sms, 0);
}

int main(int argc, char** argv) {
    g_restart = argc > 1 && std::atoi(argv[1]) != 0;
    const int64_t singles[] = {1, 16, 17, 32, 33, 48, 61, 64, 65, 80, 81, 96};
    const int64_t pairs[] = {97, 128, 129, 200, 256, 257, 333, 700};
    const int64_t rows[] = {1, 128, 257, 1000, 4096, 11008, 19200, 40000};
    for (int sms : {148, 132, 20, 2})
        for (int64_t b = 1; b < 200; b = b < 24 ? b + 1 : b + 37)
            for (int64_t n : rows) {
                for (int64_t M : singles) {
                    check<false, 4, false>(M, n, b, sms);
                    check<false, 8, false>(M, n, b, sms);
                    check<false, 4, true>(M, n, b, sms);
                    check<false, 8, true>(M, n, b, sms);
                }
                for (int64_t M : pairs) {
                    check<true, 4, false>(M, n, b, sms);
                    check<true, 8, false>(M, n, b, sms);
                    check<true, 4, true>(M, n, b, sms);
                    check<true, 8, true>(M, n, b, sms);
                }
            }
    std::printf("%ld plans, %ld waits, %ld faults\n", g_plans, g_waits, g_faults);
    return g_faults != 0;
}
