// How a call of the gated linear recurrence is cut into tiles, and what its
// workspace holds: host arithmetic of sizes only.
#pragma once

#include "api_checks.h"
#include "glr_launch.h"

namespace glr {

constexpr int kLanes = 64;

// The scan: a tile is 128 tokens, eight waves of 16.
constexpr int kScanWaves = 8, kScanTokens = 16, kScanTile = kScanWaves * kScanTokens;

// The gradients: waves of eight tokens, eight to a tile, but four where each
// lane forms the gates of two channels and a workgroup of eight would leave
// room for no second one beside it (20011 tokens of 4096 channels: 364 us with
// eight, 272 with four; plain, 191 with eight and 211 with four).
constexpr int kGradTokens = 8;
constexpr int grad_waves(bool gated, int V) { return gated && V == 2 ? 4 : 8; }
constexpr int grad_tile(bool gated, int V) { return grad_waves(gated, V) * kGradTokens; }
static_assert(grad_tile(true, 2) % kKept == 0 && grad_tile(true, 1) % kKept == 0, "a tile starts from a kept state");
static_assert(kScanTile % kKept == 0 && kKept % kScanTokens == 0, "kept states lie at the waves' borders");

inline int64_t tiles_of(int64_t n_tokens, int tile) { return (n_tokens + tile - 1) / tile; }
inline int blocks_of(int32_t D, int V) { return (D + kLanes * V - 1) / (kLanes * V); }

// Workspace of a chain: a ticket for each block of channels, then one word for
// each tile and channel (a block's by the lanes' first channels, then their
// second ones, so that a wave's words are whole lines).  A block's workgroups
// take its tiles in order, by its ticket, and store a map before they wait, so a
// tile waits only for tiles that workgroups which run already have taken, and
// the lowest of those waits for nothing: every wait ends.  Tickets lie 256 bytes
// apart (in one line they are as slow as one ticket for all: 1517 tokens of 1001
// channels in fp32, the gradients 14.8 us, apart 12.4; 20011 of 4096, gated, 286
// and 277).
// (Workgroups that stay and ask for their next tile ahead were slower, 20011
// tokens of 4096 channels by 44% and their gradients by 19%: the tile they hold
// waits for the one they are at.  Without asking ahead the gradients took as
// long as now, and the scan, short of registers, 26% longer.)
struct Chain {
    uint32_t *tickets;                   // nullptr: one tile, which needs no chain
    uint64_t *words;
    int tiles, blocks;                   // of tokens, of channels
    int pitch;                           // words a tile
    int items;                           // workgroups: of the tiles, then of groups of sequences
};
constexpr size_t kTicket = 256;
inline size_t tickets_bytes(int32_t D) { return blocks_of(D, 1) * kTicket; }
inline size_t chain_bytes(int64_t tiles, int32_t D)
{
    return tiles > 1 ? tickets_bytes(D) + (size_t)tiles * blocks_of(D, 2) * (2 * kLanes * 8) : 0;
}
inline Chain make_chain(void *ws, int32_t D, int V, int tiles, int64_t groups)
{
    const int blocks = blocks_of(D, V), pitch = blocks * kLanes * V;
    const int items = (int)((int64_t)tiles * blocks + groups);
    if (tiles < 2) return Chain{nullptr, nullptr, tiles, blocks, pitch, items};
    return Chain{static_cast<uint32_t *>(ws),
                 reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + tickets_bytes(D)), tiles, blocks, pitch, items};
}

// workgroups that look for empty sequences, 64 each
inline int64_t empty_groups(const Args &a, bool wanted)
{
    return wanted && (a.cu_seqlens || !a.n_tokens) ? ((int64_t)a.n_seqs + kLanes - 1) / kLanes : 0;
}

// Pairs of channels a lane can be taken where every row of every tensor starts
// on a pair (D even, addresses to two elements); but not for the gates of fp32
// inputs, whose pairs would not fit the registers beside a second workgroup
// (and fill whole lines of memory without them).
inline bool pairs_fit(const Args &a)
{
    const size_t es = a.bf16 ? 2 : 4;
    uintptr_t in = 0, st = 0;
    for (const void *p : {a.x, a.r, a.i, (const void *)a.h, a.dh, (const void *)a.dx, (const void *)a.dr, (const void *)a.di})
        in |= reinterpret_cast<uintptr_t>(p);
    for (const float *p : {a.g, a.rate, a.h0, (const float *)a.h_T, (const float *)a.kept, a.dh_T, (const float *)a.dg,
                           (const float *)a.drate, (const float *)a.dh0})
        st |= reinterpret_cast<uintptr_t>(p);
    return (a.bf16 || !a.gated) && a.D % 2 == 0 && in % (2 * es) == 0 && st % 8 == 0;
}

struct Plan {
    int V;                               // channels a lane
    Chain chain;
};

inline Plan plan_scan(const Args &a)
{
    // pairs of channels where the workgroups of single ones would be more than
    // two for each of 256 compute units, half the work one after another before
    // that (bf16, gated, 4096 channels: 77 tokens 9.9 us with pairs and 7.8
    // without, 1024 tokens 14.1 and 12.5, 2048 tokens 20.9 and 26.5)
    const int64_t tiles = tiles_of(a.n_tokens, kScanTile);
    const int V = pairs_fit(a) && tiles * blocks_of(a.D, 2) > 256 ? 2 : 1;
    return Plan{V, make_chain(a.ws, a.D, V, (int)tiles, empty_groups(a, a.h_T))};
}

// workspace of the backward: kept states (where they are formed again), the
// tiles' shares of drate, the chain (the forward's first, which is never longer)
struct GradParts {
    float *kept, *part;
    void *chain;
    // one fp32 row for each kept state, and no fewer than tiles
    static size_t rows(int64_t n_tokens, int32_t D) { return api::round256((size_t)tiles_of(n_tokens, kKept) * D * 4); }
    static size_t bytes(int64_t n_tokens, int32_t D)
    {
        return 2 * rows(n_tokens, D) + chain_bytes(tiles_of(n_tokens, grad_tile(true, 2)), D);
    }
    explicit GradParts(const Args &a)
    {
        char *w = static_cast<char *>(a.ws);
        const size_t r = rows(a.n_tokens, a.D);
        kept = reinterpret_cast<float *>(w);
        part = reinterpret_cast<float *>(w + r);
        chain = w + 2 * r;
    }
};

inline Plan plan_grad(const Args &a, void *chain)
{
    // gated, pairs of channels (and their smaller tiles) once there are 16
    // workgroups of them for each compute unit (4096 channels: 2048 tokens 38.9
    // us with pairs and 37.2 without, 4096 tokens 61.9 and 69.0); plain, always
    // (bf16: 256 tokens 9.2 and 8.7, 512 tokens 10.3 and 10.6, 1024 tokens 15.4 and
    // 17.6; fp32 was measured where there is work for all compute units only)
    const int least = a.gated ? 4096 : 0;
    const int V = pairs_fit(a) && tiles_of(a.n_tokens, grad_tile(a.gated, 2)) * blocks_of(a.D, 2) >= least ? 2 : 1;
    const int tiles = (int)tiles_of(a.n_tokens, grad_tile(a.gated, V));
    return Plan{V, make_chain(chain, a.D, V, tiles, empty_groups(a, a.dh0))};
}

}  // namespace glr
