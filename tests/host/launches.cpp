// The launches of the balance loss's gradient over the sizes that the C ABI takes.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <random>

#include "launch.h"

using namespace moe;

static long long checked = 0, more = 0;

static void check(int64_t T, int E) {
    const int64_t each = balance_block_tokens(E);
    ++checked;
    int launches = 0;
    for (int64_t from = 0, next; from < T; from = next, ++launches) {
        next = from + balance_backward_tokens(E);
        const int64_t blocks = balance_backward_blocks(T - from, E), end = from + blocks * each;
        // under 2^32 threads, no block without a token, every token before the next launch's
        if (blocks < 1 || blocks * 256 > 0xFFFFFFFFll || end - each >= T || end < (next < T ? next : T) || end > next) {
            printf("T=%lld E=%d: %lld blocks from %lld\n", (long long)T, E, (long long)blocks, (long long)from);
            exit(1);
        }
    }
    more += launches > 1;
}

int main() {
    std::mt19937_64 rng(1);
    for (int E = 1; E <= 256; ++E) {
        for (int bit = 0; bit <= 30; ++bit)
            for (int64_t off : {-65, -64, -17, -16, -1, 0, 1, 16, 64}) {
                const int64_t T = ((int64_t)1 << bit) + off;
                if (T >= 1 && T <= (int64_t)1 << 30) check(T, E);
            }
        for (int i = 0; i < 1000; ++i) check(1 + (int64_t)(rng() % ((uint64_t)1 << 30)), E);
    }
    printf("%lld calls, %lld of them in several launches\n", checked, more);
    return more > 1000 ? 0 : 1;
}
