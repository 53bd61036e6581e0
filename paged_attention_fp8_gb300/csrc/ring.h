// ring.h -- which loads of a ring of slots are the last ones.  Plain C++: the
// tree kernel's producers and a host test use the same code.
#pragma once

#ifdef __CUDACC__
#define PAFP8_HD __host__ __device__
#else
#define PAFP8_HD
#endif

namespace pafp8 {

// Tile n goes to slot n % stages and is loaded by warp n % warps, which has
// loaded its tiles below next[n % warps].  The last tile loaded into `slot`, or
// -1.  Slots are filled in turn, so that tile completes the newest phase of the
// slot's barrier: a wait for its parity ends when it has landed, where a wait
// for an earlier tile of the slot would wait for a phase that has passed.
PAFP8_HD constexpr int ring_last_load(const int* next, int warps, int stages, int slot) {
    int n = -1;
    for (int w = 0; w < warps; ++w) n = next[w] - 1 > n ? next[w] - 1 : n;
    for (; n >= 0; --n)
        if (n % stages == slot && n < next[n % warps]) return n;
    return -1;
}

}  // namespace pafp8
