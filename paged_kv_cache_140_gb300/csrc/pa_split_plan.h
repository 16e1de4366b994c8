// How long the partitions of the split decode kernels are: host code without CUDA
// in it, so that a host test can go over the rule by itself.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace pa {

// SMs the cuts are planned for (a constant: the workspace's size does not depend
// on the device).
constexpr int64_t kSmsTarget = 152;

// Partition length, in tokens, for `lists` lists (entries x boxes of heads, `boxes`
// of them per entry) of about `len` tokens at most; 0 when the request is invalid.
// Partitions are as long as they may be while an SM's equal share of the slots is
// no shorter (shares are cut exactly then, and fewer partials joined; lists are
// taken to be 2/5 of `len` on average), and at least 4 slots.  Entries of several
// boxes are cut at 512 tokens: their boxes' rows and scales lie next to one another
// in memory and are best read at about the same time.  Lists of up to 6 slots are
// not cut: reading a slot takes an SM about a microsecond, joining partials a
// launch of its own.
inline int split_partition(int64_t lists, int64_t boxes, int64_t len, int block_size, int slot_tokens, int requested) {
    const int64_t cap = 32 * block_size;
    // A partition's block ids sit in the 32 lanes of a warp.  One that starts inside a
    // block (at a multiple of 16 tokens, so at most block_size - 16 into it) reaches into
    // one block more than its length has: up to this length 32 hold it even so.
    const int64_t anywhere = cap - block_size + 16;
    if (requested != 0) {
        if (requested < 16 || requested % 16 != 0 || requested > cap) return 0;
        return requested % block_size != 0 && requested > anywhere ? 0 : requested;
    }
    const double share = static_cast<double>(lists) * len * 0.4 / (static_cast<double>(slot_tokens) * kSmsTarget);
    int64_t P = static_cast<int64_t>(std::min(share, 1e6)) * slot_tokens;
    if (boxes > 1) P = std::min<int64_t>(P, 512);
    P = std::max<int64_t>(P, 4 * slot_tokens);
    if (len <= std::min<int64_t>(cap, std::max<int64_t>(P, 6 * slot_tokens))) {
        P = std::max<int64_t>(16, (len + 15) / 16 * 16);   // one partition (`len` may be an estimate, see plan_split)
        return static_cast<int>(P % block_size != 0 && P > anywhere ? cap : P);
    }
    P = std::min<int64_t>(P, cap);
    if (P > slot_tokens) P -= P % slot_tokens;   // whole ring slots
    if (P % block_size != 0 && P > anywhere) P = anywhere - anywhere % slot_tokens;
    return static_cast<int>(P);
}

}  // namespace pa
