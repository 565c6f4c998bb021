// What the adapters' kernels and calls share.
#pragma once
#include <algorithm>

#include "internal.cuh"

namespace qe {

constexpr int kAdapterTile = 128;       // tokens of a tile
constexpr int kAdapterCols = 128;       // columns of a block
constexpr int kAdapterStep = 64;        // values of a 128-byte row: the step of a contraction
constexpr int kAdapterMaxRank = 128, kAdapterMaxCount = 1024;

// Ranks as the products take them; those behind the last are 0.
__host__ __device__ constexpr int rank_pad(int r)
{
    return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
}

struct AdapterPlan {
    int *off;           // [L + 2] first token of an adapter in perm; then those without one
    int *perm;          // [n] tokens in the order of their adapters
    int4 *tiles;        // (adapter, first place in perm, tokens, cost of the tiles before);
                        // adapter L: none
    int *n_tiles;       // tiles, and the cost of all
    unsigned *tickets;  // parts that have arrived: of tiles, then of outer blocks
    unsigned *most;     // [L] largest |u| of an adapter's tokens, the bits of an fp32 value
};

struct AdapterWorkspace {
    AdapterPlan p;
    int slices, splits;         // parts of a contraction: of a tile, of an adapter's tokens
    int tickets;
    unsigned *outer_tickets;
    float *mid;                 // h or u in perm's order: [n][rank_pad] values, then (or in their
                                // place) [n][parts][rank_pad] of the activations' type
    float *part, *outer_part;
    size_t bytes;
};

// What 128 columns of a tile cost when they are expanded (128 tokens 1.9 us, 35 tokens 1.46
// us; 128 tokens that are only copied 1.95 us).
__host__ __device__ constexpr int tile_cost(bool none, int tokens)
{
    return none ? 8 + 3 * tokens : 280 + tokens;
}

// Most tiles of n tokens: an adapter's tokens end with one that is not full.
inline int adapter_tiles(int n, int L) { return n / kAdapterTile + std::min(n, L + 1); }

struct AdapterCall {
    const void *x;
    long long ldx;
    const void *A, *B, *base;
    long long ldb;
    void *out;
    long long ldo;
    void *h;
    const float *scale;
    int n, L, r, K, N, sms;
    AdapterWorkspace w;
};
struct AdapterGradCall {
    const void *dy, *x;
    long long lddy, ldx;
    const void *h;
    const void *A, *B, *base;
    long long ldb;
    void *dx;
    long long lddx;
    void *dA, *dB;
    const float *scale;
    int n, L, r, K, N, sms;
    AdapterWorkspace w;
};

// Behind the plan's kernel.
cudaError_t adapter_fp16(const AdapterCall &c, cudaStream_t st);
cudaError_t adapter_bf16(const AdapterCall &c, cudaStream_t st);
cudaError_t adapter_grad_fp16(const AdapterGradCall &c, cudaStream_t st);
cudaError_t adapter_grad_bf16(const AdapterGradCall &c, cudaStream_t st);

}  // namespace qe
