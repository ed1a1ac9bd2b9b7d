// How the attention kernels share work out to their blocks.  Whole-number arithmetic of the host and the device
// alike, so that it can be walked through without a GPU.
#pragma once

#ifdef __CUDACC__
#define LQ_HD __host__ __device__ __forceinline__
#else
#define LQ_HD inline
#endif

namespace lq {

// n things shared out to c parties in order, the first n % c of them one more.  (n up to 2^31 - 1: nothing passes n + c.)
struct Shares {
    int q, rem;
    LQ_HD Shares(int n, int c) : q((int)((unsigned)n / (unsigned)c)), rem(n - q * c) {}
    LQ_HD int first(int k) const { return q * k + (k < rem ? k : rem); }   // of party k
    LQ_HD int of(int i) const {                                            // the party of thing i
        const int more = rem * (q + 1);
        return i < more ? i / (q + 1) : rem + (i - more) / q;
    }
};

constexpr int kPreUnitCost = 6;  // what a unit costs a block of the prefix kernel, in its key blocks

// The prefix kernel's work: units of `each` key blocks.  In the sequence that the blocks share, a unit is its cost in
// places and then its key blocks.  A block leaves every unit's sums in a slot of its own, numbered from the first unit
// of its share.
LQ_HD int prefix_block_at(int each, int place) {   // first key block (of all units) at or after a place
    const int u = place / (each + kPreUnitCost), in = place - u * (each + kPreUnitCost);
    return u * each + (in > kPreUnitCost ? in - kPreUnitCost : 0);
}
LQ_HD int prefix_unit_place(int each, int unit) { return unit * (each + kPreUnitCost) + kPreUnitCost; }   // its first key block's
LQ_HD int prefix_slot(const Shares& s, int each, int block, int unit) { return unit - s.first(block) / (each + kPreUnitCost); }
LQ_HD int prefix_slots(int each, int total, int blocks) {   // units that the longest share reaches at most
    const long long period = each + kPreUnitCost, longest = ((long long)total + blocks - 1) / blocks;
    return (int)((longest + period - 2) / period) + 1;
}

}  // namespace lq
