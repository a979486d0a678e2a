// Offsets of the MXFP4 product's buffer accesses: a vector offset for each lane and
// a scalar one for the wave.
//
// The descriptors' bounds alone keep the accesses inside the tensors, and do so
// whether the range check leaves the scalar offset out (vector offset against
// num_records) or counts it (against num_records - scalar offset, which wraps where
// that is negative): what may be read has its scalar offset inside its row, what
// may not has its vector offset past every descriptor, and no scalar offset passes
// the descriptor's size.
#pragma once

#include <stdint.h>

namespace moe {

// Past the end of every descriptor (the C ABI keeps their sizes at or under it),
// with room for the offsets inside a row and a 16-byte access under 2^32: reads
// there return 0 and touch no memory.
constexpr uint32_t OUT = 0xFFFF0000u;

struct BufferOffset { uint32_t vector, scalar; };

// Bytes of a descriptor of rows of codes of row_bytes each.  Of a tensor without
// rows, whose every access is at OUT, it has those of one.
__host__ __device__ inline uint32_t code_records(int64_t rows, uint32_t row_bytes) {
    return (uint32_t)(rows > 0 ? rows : 1) * row_bytes;
}

// Bytes of a descriptor of rows of nblk scales each (one where there is none, as
// above) that starts `off` bytes before them, at a word: it ends on a word.
__host__ __device__ inline uint32_t scale_records(int64_t rows, int nblk, uint32_t off) {
    return ((uint32_t)(rows > 0 ? rows : 1) * (uint32_t)nblk + off + 3u) & ~3u;
}

// Block 16 c + 4 j + kb of a row of codes: chunk c of 512 values, `row` the offset
// of the row's block kb, or OUT.
__host__ __device__ inline BufferOffset code_of_chunk(bool in_row, uint32_t row, int c, int j) {
    return {in_row ? row + (uint32_t)j * 64u : OUT, (uint32_t)c * 256u};
}

// Block 4 s + b of a row of codes: stage s of 128 values, which may lie past the end
// of K altogether; `row` the offset of the row's block b, or OUT.
__host__ __device__ inline BufferOffset code_of_stage(uint32_t row, int s, int b, int nblk) {
    return {s * 4 + b < nblk ? row : OUT, s * 4 < nblk ? (uint32_t)s * 64u : 0u};
}

// The 16 scales of chunk c; `row` the offset of the row's first, or OUT.  in_row: all
// that is accessed lies in the row.  Otherwise an access may begin past the row's end
// or go on past it, and past the tensor's: the scalar offset is left alone.  (In the
// few-row kernel an addition for each row's access costs 1.5 %: 256 rows in 32
// groups, N = 4096, K = 7168, 91.2 us against 90.)
__host__ __device__ inline BufferOffset scales_of_chunk(bool in_row, uint32_t row, int c) {
    return in_row ? BufferOffset{row, (uint32_t)c * 16u} : BufferOffset{row + (uint32_t)c * 16u, 0u};
}

}  // namespace moe
