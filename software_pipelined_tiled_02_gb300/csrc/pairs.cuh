// pairs.cuh -- what the kernels for a few rows share: the pairs of a token and an
// expert that take one expert's matrix, and the tensor-core step on registers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tg {

// `pairs` indices of experts; one outside 0 .. num_experts - 1 names none.
struct Pairs {
    const int *experts;
    int pairs, num_experts;
};

__device__ __forceinline__ int expert_of(const Pairs &p, int i)
{
    const int e = p.experts[i];
    return e < 0 || e >= p.num_experts ? -1 : e;
}

// A grid has a slot for each pair, or with more pairs than experts for each expert
// and one for the pairs without.
inline int slots_of(const Pairs &p) { return p.pairs <= p.num_experts ? p.pairs : p.num_experts + 1; }

// The expert of slot y, -1 for none: pair y's, or y itself.  False where another
// slot has it: a pair before names the same.  The whole CTA calls it.
__device__ __forceinline__ bool slot_expert(const Pairs &p, int y, int &expert)
{
    if (p.pairs > p.num_experts) {
        expert = y == p.num_experts ? -1 : y;
        return true;
    }
    expert = expert_of(p, y);
    bool before = false;
    for (int i = int(threadIdx.x); i < y; i += int(blockDim.x)) before |= expert_of(p, i) == expert;
    return !__syncthreads_or(before);
}

// The pairs that take `expert`, from pair `from` on, in order, at most `most`; the
// place to go on from.  One warp.
__device__ __forceinline__ int list_pairs(const Pairs &p, int expert, int from, int most, int *list, int &count)
{
    const int lane = int(threadIdx.x) % 32;
    count = 0;
    while (from < p.pairs && count < most) {
        const bool mine = from + lane < p.pairs && expert_of(p, from + lane) == expert;
        const unsigned found = __ballot_sync(0xffffffffu, mine);
        const int place = count + __popc(found & ((1u << lane) - 1u));
        if (mine && place < most) list[place] = from + lane;
        if (count + __popc(found) > most) {  // go on behind the last one taken
            from += __ffs(int(__ballot_sync(0xffffffffu, mine && place == most - 1)));
            count = most;
        } else {
            from += 32;
            count += __popc(found);
        }
    }
    return min(from, p.pairs);
}

// C += A . B^T for 16 rows, 8 columns and 16 k: a0, a2 of row g, a1, a3 of row
// g + 8, b0, b1 of column g (g = lane / 4).
template <bool BF16>
__device__ __forceinline__ void mma_few(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with C = A . B^T.
template <bool BF16>
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%10,%10,%10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%10,%10,%10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

}  // namespace tg
