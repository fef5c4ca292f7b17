// kernels_router.h -- argument blocks and host launchers of the router's
// training kernels.  Internal to the library; the public interface is
// include/moe_lora.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe_lora {

// Which tokens take part: those of sequences [offsets[s], offsets[s + 1])
// (offsets null: one sequence of all tokens) whose mask byte is not 0 (mask
// null: all).  Offsets are clamped to [0, T]; offsets that decrease give
// meaningless sums but no access outside the arrays.
struct TokenSet {
    const uint8_t *mask;
    const int32_t *offsets;  // [S + 1] or null
    int T, S;
};

struct BalanceArgs {
    TokenSet tok;
    const float *logits;       // [T, E]
    const int32_t *ids;        // [T, k]
    int E, k;
    int chunk, n_chunks;       // tokens per block of the first kernel
    float *part_p;             // [n_chunks + S, E]: row c + s holds chunk c's share of sequence s
    int32_t *part_n;           // [n_chunks + S, E]
    int32_t *part_t;           // [n_chunks + S]
    float *part_loss;          // [S, ceil(E / 64)]
    uint32_t *ticket;          // blocks of the second kernel that are done
    float *loss;               // [1]
    int32_t *counts;           // [S, E]
    float *probs;              // [S, E]
    int32_t *tokens;           // [S]
};

struct RouteBackwardArgs {
    TokenSet tok;
    const float *logits;       // [T, E], or null when no softmax is needed
    const int32_t *ids;        // [T, k]
    const float *weights;      // [T, k], or null with d_weights
    const float *d_weights;    // [T, k] or null
    const int32_t *counts;     // [S, E] or null: the balance loss's gradient
    const int32_t *tokens;     // [S]
    const float *d_loss;       // [1]
    float *d_logits;           // [T, E]
    int E, k, method;
};

struct FinalizeBackwardArgs {
    const uint16_t *d_out;     // [T, H]
    const uint16_t *Y;         // [n, H], or null without d_weights
    const int32_t *exp2perm;   // [n]
    const float *weights;      // [n], or null without d_Y
    uint16_t *d_Y;             // [n, H] or null
    float *d_weights;          // [n] or null
    int n, H, k;
    float scale;
};

// Chunking of the balance loss's first kernel, and its workspace (0 when the
// whole batch is one block's work).
int balance_chunk(int T);
size_t balance_workspace(int T, int E, int S);
void balance_layout(BalanceArgs *a, void *workspace);
hipError_t launch_balance(const BalanceArgs &a, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs &a, hipStream_t s);
hipError_t launch_finalize_backward(const FinalizeBackwardArgs &a, hipStream_t s);

} // namespace moe_lora
