// groups.h -- what is asked of a group's two ends before anything is read by them.
#pragma once

#ifdef __CUDACC__
#define FA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FA_HOST_DEVICE inline
#endif

namespace fa {

// Whether s0 .. s1 - 1 are two or more of B sequences, for any two 32-bit numbers: their
// difference is formed only where it lies in [1, B].
FA_HOST_DEVICE bool group_of_several(int s0, int s1, int B) {
  return s0 >= 0 && s1 <= B && s0 < s1 && s1 - s0 >= 2;
}

}  // namespace fa
