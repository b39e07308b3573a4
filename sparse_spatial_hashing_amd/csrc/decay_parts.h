// Segments of a document: plain arithmetic in 32 bits, on the device and on the host.
#ifndef SSH_DECAY_PARTS_H
#define SSH_DECAY_PARTS_H

// Where the segment that begins at token `from` of a document of n ends, 0 <= from <= n. The last
// one's sum with its length may pass 2^31.
constexpr int part_end(int from, int n, int segment) { return n - from > segment ? from + segment : n; }

#endif  // SSH_DECAY_PARTS_H
