// schedule.h - rules of the kernels' schedules that hold by arithmetic alone, in plain C++ so that tests run them on the
// host.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define C2D_HD __host__ __device__ __forceinline__
#else
#define C2D_HD inline
#endif

namespace c2d {

// Where the block-scaled products keep scales in tensor memory. A group of up to four neighbouring k-blocks shares a copy
// of its scales, made with the first of them and read by the MMAs of all; nothing documented orders a copy behind the MMAs
// issued before it, so a place is only written again once its readers are known to be done. The issuing thread knows that
// of k-block i - S when stage i mod S of the ring is full again, which it waits for before it handles k-block i. So there
// are S places, given to the groups in turn: the S - 1 groups between two uses of a place have a k-block each at least,
// which puts the first use's last reader at i - S or before. (A place for each stage would not do: its last reader may come
// three k-blocks after the one that the stage was filled for.)
struct ScalePlaces {
  uint32_t places, at;
  C2D_HD uint32_t next() {
    const uint32_t p = at;
    at = at + 1 == places ? 0 : at + 1;
    return p;
  }
};
// Whether k-block kb begins a group, for a loop that starts with kb0.
C2D_HD bool scales_begin(int kb, int kb0) { return kb == kb0 || (kb & 3) == 0; }

// Blocks (or clusters) that walk `rows` rows, block i those of i, i + blocks, ..., where all rows of a block must begin
// alike: a block for each row, or a multiple of eight of them. Never more than `most`; 0 where neither is possible.
C2D_HD long blocks_alike(long most, long rows) { return most >= rows ? rows : most / 8 * 8; }

}  // namespace c2d
