// decode_window.cu -- decode attention over a sliding window and the first
// tokens: the split kernel of decode_split.cuh over the stages that hold a
// visible token only (kWindowed), merged by the q8 combine.
//
// A token t of a sequence of L tokens is visible when t < sinks or t >= L -
// windows[b].  The unit's list of 64-token stages is then the stages of the
// first tokens followed by those of the window (one run where they meet), cut
// into equal shares like a whole context's; a stage's tokens outside both are
// masked in the scores, where their weight and V scale become 0.  Stages
// outside are neither copied nor is their block id looked at, so the blocks
// between may have been given back.
#include "decode_split.cuh"

namespace kvq8 {

cudaError_t launch_decode_window_split(const DecodeParams &p, int group, cudaStream_t s) {
    switch (group) {
        case 1: return launch_split_gm<1, false, 1, kWindowed>(p, s);
        case 2: return launch_split_two<kWindowed>(p, s);
        case 4: return launch_split_gm<4, false, 1, kWindowed>(p, s);
        case 8: return launch_split_gm<8, false, 1, kWindowed>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvq8
