// The MXFP4 product's buffer offsets under both readings of the range check: every
// dword that a reading lets through lies in the tensor, and those that the product
// needs are let through.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#define __host__
#define __device__
#include "mxoffsets.h"

using namespace moe;

static long long checked = 0;

// A 4-byte read at the offsets.  needed: at this address, and by both readings.
static void dword(BufferOffset at, uint32_t records, uint32_t tensor, bool needed, uint32_t address, const char* what) {
    const bool alone = (uint64_t)at.vector + 4 <= records;
    const bool counted = (uint64_t)at.vector + 4 <= (uint32_t)(records - at.scalar);
    const uint64_t reads = (uint64_t)at.vector + at.scalar;
    const bool inside = reads + 4 <= tensor;
    ++checked;
    if ((alone || counted) && !inside) {
        printf("%s: vector %u scalar %u records %u: reads %llu of %u bytes\n", what, at.vector, at.scalar, records,
               (unsigned long long)reads, tensor);
        exit(1);
    }
    if (needed && !(alone && counted && reads == address)) {
        printf("%s: vector %u scalar %u records %u: a value of the tensor is not read\n", what, at.vector, at.scalar, records);
        exit(1);
    }
}

// Where a tensor's last byte is not a word's, the rest of the word is taken to be there.
static uint32_t words(uint32_t bytes) { return (bytes + 3) & ~3u; }

static void tensor(int rows, int nblk) {
    const uint32_t rb = (uint32_t)nblk * 16;
    const int nchunk = (nblk + 15) / 16;
    const uint32_t codes = code_records(rows, rb), bytes = (uint32_t)rows * rb;
    for (int r = -1; r < rows; ++r) {                    // -1: a row that is not there
        for (int kb = 0; kb < 4; ++kb) {
            const uint32_t at = r < 0 ? OUT : (uint32_t)r * rb + (uint32_t)kb * 16;
            for (int c = 0; c < nchunk; ++c)
                for (int j = 0; j < 4; ++j)
                    for (int whole = 0; whole <= (c < nblk / 16); ++whole) {
                        const int block = c * 16 + j * 4 + kb;
                        BufferOffset o = code_of_chunk(whole || block < nblk, at, c, j);
                        for (int w = 0; w < 4; ++w, o.vector += 4)
                            dword(o, codes, bytes, r >= 0 && block < nblk, (uint32_t)r * rb + block * 16 + w * 4, "codes of a chunk");
                    }
            for (int s = 0; s < nchunk * 4 + 4; ++s) {   // sent for ahead, past the end of K
                const int block = s * 4 + kb;
                BufferOffset o = code_of_stage(at, s, kb, nblk);
                for (int w = 0; w < 4; ++w, o.vector += 4)
                    dword(o, codes, bytes, r >= 0 && block < nblk, (uint32_t)r * rb + block * 16 + w * 4, "codes of a stage");
            }
        }
        for (uint32_t off = 0; off < 4; ++off) {
            const uint32_t first = (uint32_t)r * nblk + off, at = r < 0 ? OUT : first & ~3u;
            const uint32_t scales = scale_records(rows, nblk, off), there = words((uint32_t)rows * nblk + off);
            for (int c = 0; c <= nchunk; ++c)            // a chunk ahead
                for (int w = 0; w < 5; ++w) {            // five words where rows do not start on one
                    const uint32_t a = at + c * 16 + w * 4;
                    const bool needed = r >= 0 && a < first + nblk && a + 4 > first;
                    BufferOffset o = scales_of_chunk(false, at, c);
                    o.vector += w * 4;
                    dword(o, scales, there, needed, a, "scales");
                    if (w == 4 || c >= nblk / 16 || nblk % 4 || off) continue;
                    o = scales_of_chunk(true, at, c);
                    o.vector += w * 4;
                    dword(o, scales, there, needed, a, "scales in the row");
                }
        }
    }
}

int main() {
    for (int rows = 0; rows <= 5; ++rows)
        for (int nblk = 1; nblk <= 70; ++nblk) tensor(rows, nblk);
    for (int rows : {0, 1, 3})
        for (int nblk : {511, 512, 2047, 2048}) tensor(rows, nblk);      // up to the largest K
    printf("%lld reads checked\n", checked);
}
