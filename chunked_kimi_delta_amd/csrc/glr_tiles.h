// glr_tiles.h -- the scan of the gated linear recurrence in tiles that hand states to each other: what the
// tiles' kernels share (glr_tiles.hip, glr_tiles_back.hip).
//
// A workgroup takes one tile: some tokens of one strip of channels, each input read once into registers. It
// publishes what the tile does to a state, (c, s) and E. TILES tiles make a window, whose last tile publishes
// what the window does; WINDOWS windows make a span, whose last tile publishes the state behind it. A tile's own
// start is the state at its span's start, behind the span's windows and the window's tiles ahead of it: at most
// 1 + WINDOWS - 1 + TILES - 1 words a channel to read, and a chain of one word a span (with windows alone, of 16
// tiles, the chain was the bound where channels are few: 32768 tokens of 64 channels 47 us for 22). Everything is
// combined in one order, so results do not depend on who came first.
//
// Waits end: a strip's tiles are numbered by a counter in the order in which its workgroups begin, and a tile waits
// only for tiles of its strip with lower numbers, which some running workgroup has begun. (One counter for all strips:
// 185 -> 282 us for 21412 packed tokens of 4096 channels, raw.) A word holds its value
// and its own flag (a sign bit that no value has), so nothing has to be ordered around it: stores and loads of 8
// bytes at device scope, zeros before the launch. A wait gives up after SPINS polls (a tenth of a second) all the same, so
// that a workspace that two calls share at once, against the rules, does not hang: what has not come is taken as NaN,
// and so are all states behind it.
#pragma once

#include "glr_scan.h"

namespace glr {

constexpr int TILES = 8, WINDOWS = 8, SPAN = TILES * WINDOWS;
constexpr int TICKET = 64;
constexpr int SPINS = 1 << 17;

struct Tiles {
    uint32_t *ticket;                   // a strip's counter, TICKET words apart
    uint64_t *tile, *window, *span;     // [places][strips * CH] what tiles and windows do, and states behind spans
};

// What a tile does, as a word: E's 32 bits, the flag, and c without its sign (s == 1: not above zero, else not below),
// whose last bit is s. c is rounded to 23 bits: up to 2^-23 of it a tile, either way, and as much of a state over the
// 1 / |c| tiles that it remembers. A slight growth in the form e^g - 1 > 0 has a sign that the word has no place for: e^g.
__host__ __device__ __forceinline__ uint64_t word_of(float c, float s, float E) {
    if (s != 0.f && c > 0.f) {
        c += 1.f;
        s = 0.f;
    }
    uint32_t b = __builtin_bit_cast(uint32_t, c) & 0x7fffffffu;
    b += b >> 1 & 1;                                        // to even; below a sign bit that a NaN would carry into
    b = ((b < 0x7fffffffu ? b : 0x7fffffffu) & 0x7ffffffeu) | (s != 0.f ? 1u : 0u);
    return (uint64_t)(b | 0x80000000u) << 32 | __builtin_bit_cast(uint32_t, E);
}
__host__ __device__ __forceinline__ void from_word(uint64_t w, float &c, float &s, float &E) {
    const uint32_t b = (uint32_t)(w >> 32);
    const float x = __builtin_bit_cast(float, b & 0x7ffffffeu);
    c = b & 1 ? -x : x;
    s = b & 1 ? 1.f : 0.f;
    E = __builtin_bit_cast(float, (uint32_t)w);
}
__device__ __forceinline__ void publish(uint64_t *p, uint64_t w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A word as it is, or NaN for one that was not published.
__host__ __device__ __forceinline__ uint64_t met(uint64_t w) { return w >> 63 ? w : ~0ull; }
// N maps of VEC channels for every lane that takes part: waits until all are published.
template <int N, int VEC>
__device__ __forceinline__ void await(const uint64_t *const (&p)[N], const bool (&on)[N], uint64_t (&w)[N][VEC]) {
    for (int n = 0; n < SPINS; ++n) {
        bool missing = false;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                w[i][v] = on[i] ? __hip_atomic_load(p[i] + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 1ull << 63;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) missing = missing || !(w[i][v] >> 63);
        if (__builtin_amdgcn_ballot_w64(missing) == 0) return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[i][v] = met(w[i][v]);
}

// Slot -> (sequence, tile of it). Sequence s's tile t lies in slot floor(bos_s / tile) + s + t; the last
// sequence whose first slot is not behind `slot` is the one. False: a slot with no tile. A sequence of no tokens
// has one slot with tile 0 and n = 0. Every lane of a wave calls; the last 64 candidates are looked at at once, one a
// lane (one after the other their loads took 20 us of 215 for 21412 packed tokens of 4096 channels).
__device__ __forceinline__ bool tile_of(const kda::SeqGeom &sg, int tile, int64_t slot, int &seq, int64_t &t,
                                        int64_t &bos, int64_t &n) {
    int lo = 0, hi = sg.N - 1;
    while (hi - lo >= 64) {
        const int mid = (lo + hi + 1) >> 1;
        if (kda::seq_bos(sg, mid) / tile + mid <= slot) lo = mid; else hi = mid - 1;
    }
    const int mine = lo + (int)(threadIdx.x & 63);
    const int64_t first = mine <= hi ? kda::seq_bos(sg, mine) : 0, end = mine <= hi ? kda::seq_eos(sg, mine, first) : 0;
    // (lo's own first slot is not behind: sequence 0's is 0)
    const uint64_t ahead = __builtin_amdgcn_ballot_w64(mine <= hi && first / tile + mine <= slot) | 1;
    const int at = 63 - __builtin_clzll(ahead);
    seq = lo + at;
    bos = (int64_t)__builtin_amdgcn_readlane((int)(first >> 32), at) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)first, at);
    n = ((int64_t)__builtin_amdgcn_readlane((int)(end >> 32), at) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)end, at)) - bos;
    t = slot - (bos / tile + seq);
    return t >= 0 && (t * tile < n || (t == 0 && n == 0));
}
// The place of a sequence's group of `size` tiles that tile t is in: injective over all sequences, below
// slots / size + N.
__device__ __forceinline__ int64_t place_of(int64_t first_slot, int seq, int64_t t, int size) {
    return first_slot / size + seq + t / size;
}

// What a workgroup's waves do to a state, and the windows and tiles ahead of it in order.
constexpr int AHEAD = WINDOWS - 1 + TILES - 1;
template <int CH, int W>
struct Shared {
    float c[W][CH], s[W][CH], E[W][CH], G[W][CH];
    float pc[AHEAD][CH], ps[AHEAD][CH], pE[AHEAD][CH], start[CH];
    uint32_t number;
};

// One map after another, for the map of all: decays as a product, and as distances from 1, which are exact
// enough where the product is near it and no factor is above 1 (e^32 e^-32 - 1 by way of e^32 has no digit left).
struct Chain {
    float A = 1.f, D = 0.f, E = 0.f, most = 0.f;
    __device__ __forceinline__ void then(float c, float s, float e) {
        E = fmaf(c, E, fmaf(s, E, e));
        const float d = s != 0.f ? c : c - 1.f;
        D = fmaf(D, d, D + d);
        most = fmaxf(most, d);
        A *= s != 0.f ? 1.f + c : c;
    }
    __device__ __forceinline__ uint64_t word() const {
        const bool slow = A >= 0.625f && most <= 0.f;       // then every factor was (c, 1), c <= 0
        return word_of(slow ? D : A, slow ? 1.f : 0.f, E);
    }
};

// From each lane's tokens to the state `in` that they start from, and the state `out` behind the tile (every
// wave has it). t: the tile in its sequence, slot0: the sequence's first slot; start: the sequence's first
// state (read in its first span); row, at: words of a place, and this lane's among them.
template <typename T, int LPR, int VEC, int W>
__device__ __forceinline__ void hand_over(const Tiles &x, const float (&G)[VEC], const float (&E)[VEC],
                                          const float (&start)[VEC], float (&in)[VEC], float (&out)[VEC],
                                          Shared<LPR * VEC, W> &sh, int64_t slot0, int seq, int64_t t, bool last,
                                          int64_t row, int at, int wave, int lane) {
    Part p[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        p[v] = Part{exp_<T>(G[v]), E[v], G[v], 1.f, 0.f};
        if constexpr (LPR <= 8) level<8>(p[v], lane);
        if constexpr (LPR <= 16) level<16>(p[v], lane);
        if constexpr (LPR <= 32) level<32>(p[v], lane);
    }
    const int ch = lane % LPR * VEC;
    const bool takes = lane < LPR;
    if (takes) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float c, s;
            decay<T>(p[v].G, c, s);
            sh.c[wave][ch + v] = c;
            sh.s[wave][ch + v] = s;
            sh.E[wave][ch + v] = p[v].E;
            sh.G[wave][ch + v] = p[v].G;
        }
    }
    // every wave has `start` before a word goes out: the sequence's last tile may write where it was read
#pragma unroll
    for (int v = 0; v < VEC; ++v) asm volatile("" : : "v"(start[v]));
    __syncthreads();
    const int tile = (int)(t % TILES), window = (int)(t % SPAN) / TILES;   // in the window, in the span
    if (wave == 0 && !last && tile < TILES - 1) {           // (no tile reads a window's last one)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float g = 0.f, e = 0.f, c, s;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                e = fmaf(sh.c[w][ch + v], e, fmaf(sh.s[w][ch + v], e, sh.E[w][ch + v]));
                g += sh.G[w][ch + v];
            }
            decay<T>(g, c, s);
            if (takes) publish(x.tile + (slot0 + t) * row + at + v, word_of(c, s, e));
        }
    }
    const int ahead = window + tile;
    // maps lo .. hi - 1 of the windows and tiles ahead, into LDS
    auto take = [&](int lo, int hi) {
        constexpr int N = (AHEAD + W - 1) / W;
        const uint64_t *from[N];
        bool on[N];
        uint64_t w[N][VEC];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = lo + wave + i * W;
            on[i] = takes && j < hi;
            from[i] = j >= hi      ? x.tile + at
                      : j < window ? x.window + place_of(slot0, seq, t - t % SPAN + j * TILES, TILES) * row + at
                                   : x.tile + (slot0 + t - ahead + j) * row + at;
        }
        await<N, VEC>(from, on, w);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (on[i]) {
                    const int j = lo + wave + i * W;
                    from_word(w[i][v], sh.pc[j][ch + v], sh.ps[j][ch + v], sh.pE[j][ch + v]);
                }
    };
    if (t > 0) {
        // a window's last tile publishes what the window does before it waits for other windows
        const bool closes = tile == TILES - 1 && window < WINDOWS - 1 && !last;
        if (closes) {
            take(window, ahead);
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    Chain m;
                    for (int j = window; j < ahead; ++j) m.then(sh.pc[j][ch + v], sh.ps[j][ch + v], sh.pE[j][ch + v]);
                    for (int w = 0; w < W; ++w) m.then(sh.c[w][ch + v], sh.s[w][ch + v], sh.E[w][ch + v]);
                    if (takes) publish(x.window + place_of(slot0, seq, t, TILES) * row + at + v, m.word());
                }
            }
        }
        take(0, closes ? window : ahead);
        if (wave == W - 1 && t >= SPAN) {
            const uint64_t *from[1] = {x.span + place_of(slot0, seq, t - SPAN, SPAN) * row + at};
            const bool on[1] = {takes};
            uint64_t w[1][VEC];
            await<1, VEC>(from, on, w);
            if (takes) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) sh.start[ch + v] = __builtin_bit_cast(float, (uint32_t)w[0][v]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float h = t >= SPAN ? sh.start[ch + v] : start[v], mine = 0.f;
        for (int j0 = 0; j0 < ahead; j0 += 4) {
            float c[4], s[4], e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + i < AHEAD ? j0 + i : AHEAD - 1;
                c[i] = sh.pc[j][ch + v];
                s[i] = sh.ps[j][ch + v];
                e[i] = sh.pE[j][ch + v];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j0 + i < ahead) h = fmaf(c[i], h, fmaf(s[i], h, e[i]));
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wave) mine = h;
            h = fmaf(sh.c[w][ch + v], h, fmaf(sh.s[w][ch + v], h, sh.E[w][ch + v]));
        }
        out[v] = h;
        in[v] = fmaf(p[v].A0, mine, p[v].E0);
        if (wave == 0 && takes && !last && t % SPAN == SPAN - 1)
            publish(x.span + place_of(slot0, seq, t, SPAN) * row + at + v, (uint64_t)1 << 63 | __builtin_bit_cast(uint32_t, h));
    }
}

// ----------------------------------------------------------------------------- host side

struct TilePlan {
    Tiles x;
    int64_t slots, bytes;
};
inline TilePlan plan_tiles(const Params &p, int tile, int ch, void *ws)
{
    TilePlan r = {};
    r.slots = p.seq.T_total / tile + p.seq.N;
    const int64_t row = (int64_t)p.strips * ch, windows = r.slots / TILES + p.seq.N, spans = r.slots / SPAN + p.seq.N;
    uint8_t *const at = (uint8_t *)ws;
    r.x.ticket = (uint32_t *)at;
    r.x.tile = (uint64_t *)(at + p.strips * TICKET * 4);
    r.x.window = r.x.tile + r.slots * row;
    r.x.span = r.x.window + windows * row;
    r.bytes = p.strips * TICKET * 4 + (r.slots + windows + spans) * row * 8;
    return r;
}
hipError_t clear_tiles(const TilePlan &r, hipStream_t st);

}  // namespace glr
