// Which copies of a warp's ring are in flight. Plain C++ (no CUDA types), so that the host can
// run the same rules.
#pragma once

#ifdef __CUDACC__
#define W4A8_RING_FN __device__ __forceinline__
#else
#define W4A8_RING_FN inline
#endif

namespace w4a8 {
namespace moe {

constexpr int kStages = 2;

// Boxes are numbered in the order they are requested; box i uses stage i % kStages, whose barrier
// is then in its phase i / kStages. A box is requested only when the one before it on its stage
// has arrived, so at most the last kStages requested are in flight.
struct RingCount {
    int issued, used;  // boxes requested, boxes taken (after a wait that ran out: only counted)
    bool dead;         // a wait ran out: nothing more is requested or waited for

    W4A8_RING_FN void reset() {
        issued = used = 0;
        dead = false;
    }
    W4A8_RING_FN static int stage(int box) { return box % kStages; }
    W4A8_RING_FN static int parity(int box) { return (box / kStages) & 1; }
    // The first box that the warp waits for before its shared memory is given back, up to `issued`.
    // Not `used`, which runs past the boxes in flight once a wait has run out.
    W4A8_RING_FN int first_pending() const { return issued < kStages ? 0 : issued - kStages; }
};

}  // namespace moe
}  // namespace w4a8
