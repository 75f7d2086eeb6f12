// Host-side check of the decode kernel's split, built and run by test_pair_rings.py: every row
// block's first owner waits only for blocks of the grid with a lower index than its own.
// And that no two launches have one value for the ready flags of their workspaces.
#include <cstdio>
#include <set>

#include "../weight_only_quantization_rtn_b200/csrc/host.cuh"

using namespace w4a16;

int main() {
    long waits = 0;
    for (int64_t C : {1, 2, 7, 20, 132, 148})
        for (int64_t rb : {1, 2, 5, 43, 86, 112, 224})
            for (int64_t kbn : {1, 2, 3, 16, 32, 86}) {
                const int64_t U = rb * kbn;
                if (C > U) continue;
                int64_t block_of[148], seen = 0;
                for (int64_t b = 0; b < C; ++b) {
                    const int64_t c = decode_share(b, C);
                    if (c < 0 || c >= C) return std::printf("share out of range\n"), 1;
                    block_of[c] = b;
                    seen += (c + 1) * U / C - c * U / C;
                }
                if (seen != U) return std::printf("units lost\n"), 1;
                for (int64_t r = 0; r < rb; ++r) {
                    const int64_t first = owner_of(r * kbn, U, C), last = owner_of(r * kbn + kbn - 1, U, C);
                    for (int64_t p = first + 1; p <= last; ++p, ++waits)
                        if (block_of[p] >= block_of[first])
                            return std::printf("block %ld waits for block %ld\n", (long)block_of[first], (long)block_of[p]), 1;
                }
            }
    std::set<uint64_t> flags;
    for (int i = 0; i < 200000; ++i) flags.insert(launch_flag());
    if (flags.size() != 200000 || flags.count(0)) return std::printf("ready flags repeat\n"), 1;
    std::printf("%ld waits\n", waits);
    return waits == 0;
}
