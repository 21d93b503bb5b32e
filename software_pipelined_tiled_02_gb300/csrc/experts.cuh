// experts.cuh -- what the files of the experts' feed-forward blocks share: how
// pairs of a token and an expert are ordered, and the work around the products.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ffn.cuh"

namespace tg {

// Pairs are worked on in expert order: by expert, then by pair index.  There are
// two numberings of these rows.  In the plain one expert e's rows begin at the
// number of all pairs of experts below e; g, u and h are kept so.  In the padded
// one every expert begins at a multiple of 32 and its rows are filled up to one
// with zeros; the workspaces are kept so, so that boxes of 32 rows never reach
// into another expert's and sums over an expert's rows run over whole steps.
constexpr int kPadRows = 32;
constexpr int kRowTile = 256;        // rows of a tile: one CTA pair
constexpr int kChunkPairs = 1024;    // pairs that one CTA counts and places
constexpr int64_t kCountedInPlace = 4096;  // up to so many pairs every CTA counts them all
constexpr int64_t kScannedCounts = 4096;   // beyond so many counts (chunks x experts) a kernel of its own sums them first
constexpr int kMostExperts = 1024;
constexpr int kMostTop = 32;

// One tile's rows.
struct RowTile {
    int expert, row, padded, rows;  // first row in either numbering, and how many there are (1 .. kRowTile)
};

// What the placing kernel leaves in the workspace.
struct Placed {
    int *counts;      // [chunks + 1][experts] pairs of each expert in each chunk (more than kCountedInPlace pairs)
    int *offsets;     // [experts + 1] first plain rows
    int *padded;      // [experts + 1] first padded rows
    int *tiles;       // number of row tiles
    RowTile *table;   // the row tiles, by expert
    int *row_of;      // [pairs] padded row, -1 for an expert that does not exist
    int *pair_of;     // [padded rows] pair, -1 for filling
};

struct ExpertSizes {
    int64_t tokens, experts, pairs, padded_rows, row_tiles;  // the last two: at most
    int top;
};

inline ExpertSizes expert_sizes(int64_t tokens, int64_t experts, int top)
{
    ExpertSizes z{};
    z.tokens = tokens;
    z.experts = experts;
    z.top = top;
    z.pairs = tokens * top;
    const int64_t used = experts < z.pairs ? experts : z.pairs;
    z.padded_rows = z.pairs + used * (kPadRows - 1);
    z.row_tiles = z.pairs / kRowTile + used;
    return z;
}

inline int64_t chunks_of(const ExpertSizes &z) { return (z.pairs + kChunkPairs - 1) / kChunkPairs; }

int experts_place(const ExpertSizes &z, const int *chosen, const Placed &p, cudaStream_t s);

// Rows of one or two matrices [tokens, width] in padded expert order, filling as zeros.
struct Gather {
    const void *from[2];
    int64_t ld[2];
    void *to[2];  // [padded rows, width]
};
int experts_gather(const ExpertSizes &z, int64_t width, const Gather &g, const Placed &p, cudaStream_t s);

// out[t] = sum over t's pairs of (weights) rows[row_of[pair]], rounded once.  With
// `parts`: also dweights[pair] = the sum of its row's `nparts` partial sums.
struct Combine {
    const float *rows;     // [padded rows, width]
    const float *weights;  // NULL: 1
    void *out;             // NULL: not wanted
    int64_t ld;
    const float *parts;    // [nparts][padded rows]
    int64_t part_stride;
    int nparts;
    float *dweights;       // NULL: not wanted
    const int *chosen;     // not NULL: a pair's row is the pair, if its expert is one of `experts`
    int experts;
};
int experts_combine(const ExpertSizes &z, int64_t width, bool bf16, const Combine &c, const Placed &p, cudaStream_t s);

// The forward pass of a few tokens without g, u and h for a backward pass
// (experts_few.cu).  `combine` has the results' place and the fp32 rows', one a pair.
struct ExpertsFewCall {
    const void *x;
    int64_t ldx, width, hidden;
    const int *chosen;
    const void *w[3];  // gate, up, down
    int64_t ld[3], es[3];
    void *h;           // [pairs, hidden]
    int act;
};
int experts_few(const ExpertsFewCall &call, const Combine &combine, const ExpertSizes &z, int sms, bool bf16, cudaStream_t s);

// Whether it takes so many: up to kFewPairs, where hardly an expert has more than 8 of
// them, because it reads an expert's weights again for every 8.
bool experts_are_few(const ExpertSizes &z);
constexpr int64_t kFewPairs = 384;

}  // namespace tg
