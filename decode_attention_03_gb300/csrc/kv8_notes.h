// What a worker of gqa_decode_kv8 notes for the merge kernel about a (sequence, head) that more than one worker streams.
// Plain C++: the arithmetic is tested on the host.
#pragma once
#ifdef __CUDACC__
#define KV8_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KV8_HOST_DEVICE inline
#endif

namespace gqa {

// `pieces` neighbouring workers have the keys of head g of sequence b (fewer than 2: nothing to fold); the first one's partial
// is in slot `first` (worker w has the slots 2w and 2w + 1), the others' in the first slots of the workers after it.
struct Kv8Note {
  int pieces, first, b, g;
};

KV8_HOST_DEVICE int kv8_slot(const Kv8Note& n, int piece) { return piece == 0 ? n.first : (n.first & ~1) + 2 * piece; }

// Notes lie in the workspace, and a worker that gave up has left some unwritten: what is there then may be anything, so that
// only a note whose sequence, head and slots exist is followed.
KV8_HOST_DEVICE bool kv8_note_ok(const Kv8Note& n, int workers, int sequences, int heads) {
  return n.pieces >= 2 && n.b >= 0 && n.b < sequences && n.g >= 0 && n.g < heads && n.first >= 0 &&
         n.first / 2 < workers && n.pieces <= workers - n.first / 2;
}

}  // namespace gqa
