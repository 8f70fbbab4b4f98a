// window.cuh -- how the windowed attention kernels see a sequence.
//
// A token at position p attends to positions j <= p with j > p - window or j < sinks: the
// first `sinks` tokens, a gap, and a window.  Blocks that lie in the gap as a whole are left
// out: the kernels run over the blocks that hold the sinks followed by those from the one that
// holds the oldest window token on, as if they were one sequence, and mask the rest of the gap
// (fewer than two blocks' rows: what shares a block with the last sink or the first window
// token).  Position j is then place j in the sinks' blocks and place j - shift * block_size
// from there on; table entry i of a place's block is i, or i + shift past the sinks' blocks.
#pragma once

#include <stdint.h>

namespace pkv {

struct WindowView {
  int shift;  // blocks left out
  int gap;    // places sinks .. sinks + gap - 1 are masked
};

// `oldest`: the oldest position in the window (0 if the window reaches the start).
__host__ __device__ inline WindowView window_view(int oldest, int sinks, int sink_blocks, int block_size) {
  WindowView v;
  const int out = oldest / block_size - sink_blocks;
  v.shift = out > 0 ? out : 0;
  const int gap = oldest - v.shift * block_size - sinks;
  v.gap = gap > 0 ? gap : 0;
  return v;
}

}  // namespace pkv
