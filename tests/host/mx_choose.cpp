// The few-row kernels' launches over the sizes that the C ABI takes.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <random>

#include "mxchoose.h"

using namespace moe;

static bool taken(int64_t M, int64_t G, int64_t N, int64_t K) {          // by the C ABI
    return (N + 256) * (K / 2) <= 0xFFFF0000ll && ((M + 127) / 128 + G) * ((N + 255) / 256) < (1ll << 31) &&
           M <= (1ll << 31) - 65536;
}

static long long checked = 0, few = 0;

static void check(int64_t M, int G, int N, int K, int cus) {
    if (!taken(M, G, N, K)) return;
    ++checked;
    const MxKernel k = mx_choose(M, G, N, K, cus);
    if (k == TILES) return;
    ++few;
    const MxGrid g = mx_rows_grid(mx_rows(k), M, G, N);
    if (g.x < 1 || g.y < 1 || g.y > 65535 || g.x * g.y > 0xFFFFFFFFll / 256) {
        printf("M=%lld G=%d N=%d K=%d: kernel %d, %lld x %lld blocks\n", (long long)M, G, N, K, (int)k, (long long)g.x,
               (long long)g.y);
        exit(1);
    }
}

int main() {
    std::mt19937_64 rng(1);
    auto up_to = [&](double most) {                      // 1 .. most, even over the logarithm
        return (int64_t)exp2(std::uniform_real_distribution<double>(0, log2(most))(rng));
    };
    for (int cus : {64, 256}) {
        for (int K : {32, 64, 128}) {
            check(1024, 1024, 1 << 20, K, cus);          // many columns to few rows
            check(64, 8, 1 << 27, K, cus);
            check(1, 1, 1 << 27, K, cus);
        }
        for (int i = 0; i < 2000000; ++i)
            check(up_to(2147418112.0), (int)up_to(1024), (int)up_to(268435456.0), 32 * (int)up_to(2048), cus);
    }
    printf("%lld calls, %lld of them few rows\n", checked, few);
    return few > 100000 ? 0 : 1;
}
