// The sizes of launches, as plain arithmetic for the host.
#pragma once

#include <stdint.h>

namespace moe {

// Blocks of a launch that has work for `want` blocks: a launch is held under 2^32
// threads, and kernels whose work may pass that go on in steps of the grid.
inline unsigned launch_blocks(int64_t want, int threads) {
    const int64_t most = 0xFFFFFFFFll / threads;
    return (unsigned)(want < most ? want : most);
}

// The balance loss's gradient: 64 lanes a token (16 for up to 64 experts), each group of
// which goes through so many tokens, in blocks of 256 threads.
constexpr int BALANCE_EACH = 4;
constexpr int balance_block_tokens(int E) { return BALANCE_EACH * 256 / (E > 64 ? 64 : 16); }
// Blocks of the launch that starts where T tokens are left, and tokens that a launch goes
// through at most.
inline unsigned balance_backward_blocks(int64_t T, int E) {
    return launch_blocks((T + balance_block_tokens(E) - 1) / balance_block_tokens(E), 256);
}
inline int64_t balance_backward_tokens(int E) { return (int64_t)launch_blocks(INT64_MAX, 256) * balance_block_tokens(E); }

}  // namespace moe
