// Attention of chunks of new tokens over the paged cache, on the tensor cores (tcgen05).
// [LM4] = "Build a language model in C# from scratch (4): running GPT-2 weights", "Generation with
// a KV cache" (the new tokens' queries against every cached position, no mask but the order).
//
// A block takes two tiles of 128 query rows of one key / value head (the H / Hkv heads that share it
// side by side: row i is query i / G, head i % G, so its keys are read once for all of them) and
// walks the keys in tiles of 128:
//   S = Q K^T   (M = 128 rows, N = 128 keys, K = head size) into tensor memory;
//   softmax     a thread per row: P = 2^(s - m) with s in powers of two, as bf16 over S in tensor
//               memory (an operand of the product has 16 bits; 2^-8 of a weight at most, as y's own
//               rounding, where a second part would double the products; sums of weights stay float32);
//               the reference m moves (and O is rescaled there) only when the row's maximum passes it
//               by more than 8;
//   O += P V    (N = head size, K = 128 keys), accumulated in tensor memory.
// Head sizes up to 64 leave room there for P beside S: the next S is computed as soon as the scores of
// this one have been read, under the softmax. With 128 P lies over S, and the next S waits for P V.
// The two tiles take turns: while one group of four warps turns its S into P, the tensor core
// computes the other's products. Warp 8 sends for the keys by TMA, a box per page (pages lie anywhere).
// 8-bit codes become bf16 (exactly) first: in one pass into the workspace, if it has room (for all heads or a few
// at a time) and heads are wide or rows many; else on the way, by warps 8-11. Codes carry no scale into the products: the key's scale multiplies the score and
// the value's scale the weight, both from shared memory. Warp 12 issues the MMAs.
// K and V have rings of their own (a K tile is free once both S are there, a V tile after both
// products), of three tiles each for head sizes up to 64 and two for 128.
// Registers: 512 threads at 128; the softmax warpgroups take 184 each, the copying one 96, the MMA warp's
// 48 (where the copying one unpacks codes: 176, 104, 48).
// All mbarrier waits are bounded (timeout -> GK_ERR_TIMEOUT in the error word).
// Measured: two chunks of up to 2048 tokens behind 16384 keys, 32 heads over 8 of 128: bf16 pages 498 us, 1.06
// PFLOP/s (0.55 of a dense product); 8-bit ones 670 us with the pass that expands them (1980 unpacked on the way):
// the softmax warps bound both, by a thread's 128 exponentials, maxima and packing a tile, for 8 bits by two more
// products a score. Three chunks of up to 1000 over 8100 keys, 12 heads of 64: 86 us (half the products a tile for
// the same softmax). Key tiles that two groups of blocks read side by side come from L2.
#include "paged_attn_tiles.cuh"

namespace gk {

gk_status launch_attn_tiles(gk_ctx* ctx, const AttnArgs& a) { return launch_tiles<WHOLE>(ctx, a); }

}  // namespace gk
