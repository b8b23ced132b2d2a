// gdn_step_maps.cuh -- a step's index arrays from its requests' lengths
// (gdn_step_maps in include/gdn_spec.h).
//
// Two running sums over the requests (tokens, new blocks) and one row of output
// per token.  One launch: every CTA sums all N requests for itself (a few KB
// from L2) instead of waiting for another, marks where the requests that cross
// its packed rows begin, and a running maximum over the marks tells each row its
// request.  Where there are many, a thread takes four requests or rows at a
// time, the rows' 16 bytes then as whole words.  Bound by latency: two global
// loads one behind the other (the request, its block) and the scans between:
// 128 requests and 640 rows in 2.7 us, 1024 requests and 34,000 rows in 4.6,
// 96 requests and 205,000 rows in 3.9 (5.4 with four requests a thread).
#pragma once

#include "gdn_spec_common.cuh"

namespace gdn {
namespace spec {

// Division by a number known on the host (Granlund and Montgomery, "Division by
// invariant integers using multiplication"): exact for every 32-bit dividend.
struct Divisor {
    uint32_t by, factor, shift1, shift2;
    static Divisor of(uint32_t d)
    {
        uint32_t l = 0;
        while (l < 32 && (1ull << l) < d)
            ++l;
        return {d, static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1), l < 1 ? l : 1, l > 1 ? l - 1 : 0};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const
    {
        const uint32_t t = __umulhi(factor, n);
        return (t + ((n - t) >> shift1)) >> shift2;
    }
};

struct MapsParams {
    const int32_t *lengths, *context, *slots;
    int32_t *cu_seqlens, *state_indices, *row_seq, *positions;
    int32_t *tables;                       // from here to slot_map: with a blocked cache only
    const int32_t *held, *free_blocks, *free_head;
    int32_t *held_out, *free_head_out;
    int64_t *slot_map;
    uint32_t *status;
    int64_t b_row;
    int32_t N, C, B, F, blocked;
    Divisor block_size;
};

constexpr int MAPS_THREADS = 256;
constexpr int MAPS_WARPS = MAPS_THREADS / 32;

// Running sums of (tokens, new blocks).
struct Sums {
    long long tok, blk;
    __device__ __forceinline__ void add(const Sums &x)
    {
        tok += x.tok;
        blk += x.blk;
    }
};

// The sums over the threads before this one, and over all of them in `all`.
__device__ __forceinline__ Sums cta_before(const Sums &own, Sums *warp_sums, Sums *all)
{
    const int lane = threadIdx.x & 31, warp = warp_index();
    Sums x = own;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums b = {__shfl_up_sync(~0u, x.tok, o), __shfl_up_sync(~0u, x.blk, o)};
        if (lane >= o)
            x.add(b);
    }
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    Sums before = {x.tok - own.tok, x.blk - own.blk};
    *all = {0, 0};
#pragma unroll
    for (int w = 0; w < MAPS_WARPS; ++w) {
        if (w < warp)
            before.add(warp_sums[w]);
        all->add(warp_sums[w]);
    }
    return before;
}

// What the rows of a request need of it.
struct MapsRequest {
    int32_t seq, begin, context, held, fresh;      // fresh: where its new blocks begin in free_blocks
};

// REQS, ROWS: requests of a scan step, and rows, per thread.
template <int REQS, int ROWS>
__global__ void __launch_bounds__(MAPS_THREADS) gdn_step_maps_kernel(const MapsParams a)
{
    constexpr int TILE = MAPS_THREADS * ROWS, STEP = MAPS_THREADS * REQS;
    __shared__ Sums warp_sums[2][MAPS_WARPS];
    __shared__ MapsRequest mark[TILE];                // request that begins, or goes on, at this row; seq -1: none
    __shared__ int32_t warp_max[MAPS_WARPS];
    __shared__ Sums cut;                                   // sums before the first request that does not fit; tok -1: all fit
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const long long row0 = static_cast<long long>(blockIdx.x) * TILE;

    pdl_wait();
    const bool blocks = a.blocked != 0;
    int32_t head = 0;
    long long room = 0;                                    // free blocks left
    uint32_t bad = 0;
    if (blocks)
        head = *a.free_head;
#pragma unroll
    for (int e = 0; e < ROWS; ++e)
        mark[e * MAPS_THREADS + tid].seq = -1;
    if (tid == 0)
        cut = {-1, 0};

    Sums base = {0, 0};
    const int steps = (a.N + STEP - 1) / STEP;
    for (int k = 0; k < steps; ++k) {
        const int32_t i0 = k * STEP + tid * REQS;
        int32_t slot[REQS], len[REQS], have[REQS], held[REQS];
#pragma unroll
        for (int e = 0; e < REQS; ++e) {
            const bool in = i0 + e < a.N;
            slot[e] = in ? a.slots[i0 + e] : -1;
            len[e] = in ? a.lengths[i0 + e] : 0;
            have[e] = in ? a.context[i0 + e] : 0;
            held[e] = in && blocks ? a.held[i0 + e] : 0;
        }
        if (k == 0 && blocks) {
            const bool usable = head >= 0 && head <= a.F;
            room = usable ? a.F - head : -1;               // -1: nothing fits
            bad |= usable ? 0u : GDN_DEV_BAD_BLOCKS;
        }
        Sums mine[REQS], own = {0, 0};
#pragma unroll
        for (int e = 0; e < REQS; ++e) {
            mine[e] = {0, 0};
            uint32_t wrong = slot[e] < -1 ? GDN_DEV_BAD_SLOT : 0u;
            if (len[e] < 0 || have[e] < 0 || static_cast<long long>(len[e]) + have[e] > INT32_MAX)
                wrong |= GDN_DEV_BAD_LENGTH;
            if (slot[e] != -1 && !wrong && len[e] > 0) {
                mine[e].tok = len[e];
                if (blocks) {
                    const uint32_t need = a.block_size.quotient(static_cast<uint32_t>(have[e]) + len[e] + a.block_size.by - 1);
                    if (held[e] < 0 || held[e] > a.B || static_cast<long long>(held[e]) * a.block_size.by < have[e] ||
                        need > static_cast<uint32_t>(a.B)) {
                        wrong |= GDN_DEV_BAD_BLOCKS;
                        mine[e].tok = 0;
                    } else if (need > static_cast<uint32_t>(held[e])) {
                        mine[e].blk = need - held[e];
                    }
                }
            }
            if (slot[e] != -1)
                bad |= wrong;
            own.add(mine[e]);
        }
        Sums all, from = cta_before(own, warp_sums[k & 1], &all);
        from.add(base);
        // both sums only grow, so what fits is a run of requests from the first
        auto fits = [&](const Sums &s) { return s.tok <= a.C && (!blocks || s.blk <= room); };
        Sums to[REQS];
        Sums at = from;
#pragma unroll
        for (int e = 0; e < REQS; ++e) {
            const Sums prior = at;
            at.add(mine[e]);
            to[e] = at;
            if (i0 + e < a.N && !fits(at) && (i0 + e == 0 || fits(prior)))
                cut = prior;
        }
        base.add(all);
        const bool whole = fits(base);                     // then no request up to here was cut
        if (!whole)
            __syncthreads();
#pragma unroll
        for (int e = 0; e < REQS; ++e) {
            const int32_t i = i0 + e;
            const bool in = whole || fits(to[e]), runs = mine[e].tok > 0 && in;
            const Sums prior = {to[e].tok - mine[e].tok, to[e].blk - mine[e].blk};
            if (mine[e].tok > 0 && !in)
                bad |= GDN_DEV_NO_ROOM;
            if (i < a.N && k % gridDim.x == blockIdx.x) {
                a.cu_seqlens[i + 1] = static_cast<int32_t>(in ? to[e].tok : cut.tok);
                a.state_indices[i] = runs ? slot[e] : -1;
                if (blocks)
                    a.held_out[i] = runs ? held[e] + static_cast<int32_t>(mine[e].blk) : held[e];
            }
            if (runs && to[e].tok > row0 && prior.tok < row0 + TILE)
                mark[prior.tok > row0 ? prior.tok - row0 : 0] = {i, static_cast<int32_t>(prior.tok), have[e], held[e],
                                                                 head + static_cast<int32_t>(prior.blk)};
        }
    }
    if (steps == 0 && blocks && (head < 0 || head > a.F))
        bad |= GDN_DEV_BAD_BLOCKS;
    __syncthreads();                                       // marks and the cut
    const Sums end = cut.tok >= 0 ? cut : base;
    if (blockIdx.x == 0) {
        if (tid == 0) {
            a.cu_seqlens[0] = 0;
            if (blocks)
                *a.free_head_out = head + static_cast<int32_t>(end.blk);
        }
        if (bad)
            report(a.status, bad);
    }

    // ---- each row's request: the last mark at or before it
    const int r0 = tid * ROWS;
    int32_t h = -1;
#pragma unroll
    for (int e = 0; e < ROWS; ++e)
        if (mark[r0 + e].seq >= 0)
            h = r0 + e;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t b = __shfl_up_sync(~0u, h, o);
        if (lane >= o)
            h = max(h, b);
    }
    if (lane == 31)
        warp_max[warp] = h;
    h = __shfl_up_sync(~0u, h, 1);
    h = lane ? h : -1;                                     // before this thread's rows, in its warp
    __syncthreads();
#pragma unroll
    for (int w = 0; w < MAPS_WARPS; ++w)
        if (w < warp)
            h = max(h, warp_max[w]);
    const long long t0 = row0 + r0;
    if (t0 >= a.C)
        return;
    int32_t seq[ROWS], pos[ROWS], block[ROWS], in[ROWS];
    int32_t *fresh[ROWS];                                  // where a new block's first token enters it, else NULL
#pragma unroll
    for (int e = 0; e < ROWS; ++e) {
        if (mark[r0 + e].seq >= 0)
            h = r0 + e;
        seq[e] = pos[e] = block[e] = -1;
        in[e] = 0;
        fresh[e] = nullptr;
        if (t0 + e < end.tok && h >= 0) {
            const MapsRequest q = mark[h];
            seq[e] = q.seq;
            pos[e] = q.context + static_cast<int32_t>(t0 + e - q.begin);
            if (blocks) {
                const int32_t lb = static_cast<int32_t>(a.block_size.quotient(pos[e]));
                int32_t *const entry = a.tables + q.seq * a.b_row + lb;
                in[e] = pos[e] - lb * static_cast<int32_t>(a.block_size.by);
                block[e] = lb < q.held ? *entry : a.free_blocks[q.fresh + lb - q.held];
                fresh[e] = lb >= q.held && in[e] == 0 ? entry : nullptr;
            }
        }
    }
    // (stores behind all loads: they might alias for all the compiler knows)
    long long place[ROWS];
#pragma unroll
    for (int e = 0; e < ROWS; ++e) {
        place[e] = seq[e] >= 0 ? static_cast<long long>(block[e]) * a.block_size.by + in[e] : -1;
        if (fresh[e])
            *fresh[e] = block[e];
    }
    const uintptr_t lie = reinterpret_cast<uintptr_t>(a.row_seq) | reinterpret_cast<uintptr_t>(a.positions) |
                          reinterpret_cast<uintptr_t>(a.slot_map);
    if (ROWS == 4 && t0 + ROWS <= a.C && (lie & 15u) == 0) {
        *reinterpret_cast<int4 *>(a.row_seq + t0) = make_int4(seq[0], seq[1 % ROWS], seq[2 % ROWS], seq[3 % ROWS]);
        *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1 % ROWS], pos[2 % ROWS], pos[3 % ROWS]);
        if (blocks) {
            *reinterpret_cast<longlong2 *>(a.slot_map + t0) = make_longlong2(place[0], place[1 % ROWS]);
            *reinterpret_cast<longlong2 *>(a.slot_map + t0 + 2) = make_longlong2(place[2 % ROWS], place[3 % ROWS]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < ROWS; ++e)
            if (t0 + e < a.C) {
                a.row_seq[t0 + e] = seq[e];
                a.positions[t0 + e] = pos[e];
                if (blocks)
                    a.slot_map[t0 + e] = place[e];
            }
    }
}

}  // namespace spec
}  // namespace gdn
