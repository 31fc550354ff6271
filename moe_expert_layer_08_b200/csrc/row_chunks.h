// row_chunks.h -- how an expert's rows are cut into the row chunks of work items:
// plain C++, so that a host program can check it at any size.
#pragma once

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

struct RowChunks {
    int count, size;  // chunk c has rows c * size .. min((c + 1) * size, rows) - 1
};

// As few chunks of at most `most` rows (a multiple of 16) as hold `rows` > 0, of equal
// size up to the MMA's 16.  Every chunk has a row: (count - 1) * size <= (count - 1) *
// most < rows.  No sum passes `rows` by more than 15, so any int will do.
MOE_HOST_DEVICE RowChunks row_chunks(int rows, int most) {
    const int count = rows / most + (rows % most != 0);
    const int each = rows / count + (rows % count != 0);
    return {count, (each + 15) / 16 * 16};
}

}  // namespace moe
