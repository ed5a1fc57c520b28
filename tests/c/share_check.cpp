// Host check of how two products in one grid share its blocks
// (train_internal.h): no block without a tile, no block left over while a
// tile waits, and both products under way.  Prints one line per failure and
// "all checks passed".
#include <cstdio>

#include "train_internal.h"

using namespace zero;

static int failures = 0;

static void check(int64_t a, int64_t b, double work_a, double work_b, int64_t most) {
    int64_t first = -1, second = -1;
    share_blocks(a, b, work_a, work_b, most, &first, &second);
    const int64_t blocks = a + b < most ? a + b : most;
    const bool right = first >= (a > 0) && first <= a && second >= (b > 0) && second <= b && first + second == blocks;
    // by the work, but for what the other cannot use
    const double wa = static_cast<double>(a) * work_a, wb = static_cast<double>(b) * work_b;
    const double ideal = a + b <= most || a == 0 ? static_cast<double>(a) : static_cast<double>(most) * wa / (wa + wb);
    const bool fair = first == a || second == b || (first - ideal <= 1 && ideal - first <= 1);
    if (!right || !fair) {
        std::printf("FAIL %lld and %lld tiles of %g and %g on %lld blocks: %lld and %lld\n", (long long)a, (long long)b,
                    work_a, work_b, (long long)most, (long long)first, (long long)second);
        ++failures;
    }
}

int main() {
    const double works[] = {64, 128, 576, 2112, 10064, 1048640};
    for (int64_t a = 0; a <= 1400; a += a < 40 ? 1 : 7)
        for (int64_t b = 0; b <= 1400; b += b < 40 ? 1 : 7)
            for (double x : works)
                for (double y : works) check(a, b, x, y, 512);
    check(8, 67108864, 64, 1048640, 512);
    check(67108864, 8, 64, 1048640, 512);
    // 100 tokens x 1000 x 10000: dx's tiles in slices, dw's
    check(152, 632, 576, 192, 512);
    if (failures == 0) std::printf("all checks passed\n");
    return failures != 0;
}
