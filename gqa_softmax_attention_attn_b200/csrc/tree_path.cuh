// tree_path.cuh -- which of a sequence's drafted tokens a token descends from.
#pragma once

#include "kernels.h"

namespace attn_sink {

constexpr int kPathWords = kTreeMaxTokens / 32;

// The depth of tokens [i0, i0 + n) of sequence q and the tokens they see (bit
// a of a row's kPathWords words: token a is the row's token or an ancestor of
// it fewer than `window` levels up).  Every thread of the group calls it, with
// sync() a barrier of the group; par is scratch of kTreeMaxTokens entries.
// A parent counts only when it lies in front of its child (an entry outside
// [0, i) makes token i a root), so every walk ends.  The parents are walked in
// shared memory: one round trip to L2 for all of them instead of one a level.
template <typename Sync>
__device__ __forceinline__ void tree_paths(const TreeShape &s, const TreeSeq &q, int i0, int n, int tid, int nthreads,
                                           int16_t *par, uint32_t (*bits)[kPathWords], int16_t *depth, Sync sync)
{
    for (int i = tid; i < i0 + n; i += nthreads) {
        const int a = s.parents[q.row0 + i];
        par[i] = (int16_t)(a >= 0 && a < i ? a : -1);
    }
    sync();
    for (int k = tid; k < n; k += nthreads) {
        for (int w = 0; w < kPathWords; ++w) bits[k][w] = 0u;
        // the walk meets the words of the row from the last to the first: each is gathered in a register
        int d = 0, w = (i0 + k) >> 5;
        uint32_t word = 0u;
        for (int a = i0 + k; a >= 0; a = par[a], ++d) {
            if (a >> 5 != w) {
                bits[k][w] = word;
                word = 0u;
                w = a >> 5;
            }
            if (s.window <= 0 || d < s.window) word |= 1u << (a & 31);
        }
        bits[k][w] = word;
        depth[k] = (int16_t)(d - 1);
    }
    sync();
}

}  // namespace attn_sink
