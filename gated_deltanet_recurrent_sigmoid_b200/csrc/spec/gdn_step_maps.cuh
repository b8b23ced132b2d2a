// gdn_step_maps.cuh -- a step's index arrays from its requests' lengths
// (gdn_step_maps in include/gdn_spec.h).
//
// Two exclusive sums over the requests (tokens, new blocks) and one row of
// output per token.  One launch: every CTA sums all N requests for itself (a
// few KB from L2) instead of waiting for another, marks where the requests
// that cross its 1024 packed rows begin, and a running maximum over the marks
// tells each row its request.  Bound by latency, then by the 16 bytes written
// per row.
#pragma once

#include "gdn_spec_common.cuh"

namespace gdn {
namespace spec {

struct MapsParams {
    const int32_t *lengths, *context, *slots;
    int32_t *cu_seqlens, *state_indices, *row_seq, *positions;
    int32_t *tables;                       // from here to slot_map: with a blocked cache only
    const int32_t *held, *free_blocks, *free_head;
    int32_t *held_out, *free_head_out;
    int64_t *slot_map;
    uint32_t *status;
    int64_t b_row;
    int32_t N, C, B, F, block_size, blocked;
};

constexpr int MAPS_THREADS = 1024;         // = packed rows a CTA = requests a scan step

// Inclusive sums over the CTA of (tokens, blocks) per thread.
struct Sums {
    long long tok, blk;
};
__device__ __forceinline__ Sums cta_scan(Sums x, Sums *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = warp_index();
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, x.tok, o), b = __shfl_up_sync(~0u, x.blk, o);
        if (lane >= o) {
            x.tok += t;
            x.blk += b;
        }
    }
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        Sums w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(~0u, w.tok, o), b = __shfl_up_sync(~0u, w.blk, o);
            if (lane >= o) {
                w.tok += t;
                w.blk += b;
            }
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        x.tok += warp_sums[warp - 1].tok;
        x.blk += warp_sums[warp - 1].blk;
    }
    return x;
}

__global__ void __launch_bounds__(MAPS_THREADS) gdn_step_maps_kernel(const MapsParams a)
{
    __shared__ Sums warp_sums[32];
    __shared__ int32_t mark[MAPS_THREADS];                 // request that begins (or goes on) at this row, or -1
    __shared__ int32_t begin[MAPS_THREADS], fresh_at[MAPS_THREADS];
    __shared__ int32_t warp_max[32];
    __shared__ long long cut_tok, cut_blk;                 // sums before the first request that does not fit
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
    const long long row0 = static_cast<long long>(blockIdx.x) * MAPS_THREADS;

    pdl_wait();
    mark[tid] = -1;
    if (tid == 0)
        cut_tok = -1;
    const bool blocks = a.blocked != 0;
    int32_t head = 0;
    long long room = 0;                                    // free blocks left
    uint32_t bad = 0;
    if (blocks) {
        head = *a.free_head;
        if (head < 0 || head > a.F) {
            bad |= GDN_DEV_BAD_BLOCKS;
            room = -1;                                     // nothing fits
        } else {
            room = a.F - head;
        }
    }
    __syncthreads();

    Sums base = {0, 0};
    const int steps = (a.N + MAPS_THREADS - 1) / MAPS_THREADS;
    for (int k = 0; k < steps; ++k) {
        const int32_t i = k * MAPS_THREADS + tid;
        int32_t slot = -1, len = 0, held = 0;
        Sums mine = {0, 0};
        if (i < a.N) {
            slot = a.slots[i];
            len = a.lengths[i];
            const int32_t have = a.context[i];
            uint32_t wrong = 0;
            if (slot < -1)
                wrong |= GDN_DEV_BAD_SLOT;
            if (len < 0 || have < 0 || static_cast<long long>(len) + have > INT32_MAX)
                wrong |= GDN_DEV_BAD_LENGTH;
            if (blocks)
                held = a.held[i];
            if (slot != -1 && !wrong && len > 0) {
                mine.tok = len;
                if (blocks) {
                    const uint32_t need = (static_cast<uint32_t>(have) + len + a.block_size - 1) / static_cast<uint32_t>(a.block_size);
                    if (held < 0 || held > a.B || static_cast<long long>(held) * a.block_size < have ||
                        need > static_cast<uint32_t>(a.B)) {
                        wrong |= GDN_DEV_BAD_BLOCKS;
                        mine.tok = 0;
                    } else if (need > static_cast<uint32_t>(held)) {
                        mine.blk = need - held;
                    }
                }
            }
            if (slot != -1)
                bad |= wrong;
        }
        const Sums own = mine;
        Sums to = cta_scan(mine, warp_sums);
        to.tok += base.tok;
        to.blk += base.blk;
        const Sums from = {to.tok - own.tok, to.blk - own.blk};
        // both sums only grow, so what fits is a run of requests from the first
        const bool fits = to.tok <= a.C && (!blocks || to.blk <= room);
        const bool fitted = from.tok <= a.C && (!blocks || from.blk <= room);
        if (i < a.N && !fits && (fitted || (i == 0))) {
            cut_tok = from.tok;
            cut_blk = from.blk;
        }
        __syncthreads();
        const bool runs = own.tok > 0 && fits;
        if (own.tok > 0 && !fits)
            bad |= GDN_DEV_NO_ROOM;
        if (i < a.N && k % gridDim.x == blockIdx.x) {
            a.cu_seqlens[i + 1] = static_cast<int32_t>(fits ? to.tok : cut_tok);
            a.state_indices[i] = runs ? slot : -1;
            if (blocks)
                a.held_out[i] = runs ? held + static_cast<int32_t>(own.blk) : held;
        }
        if (runs && to.tok > row0 && from.tok < row0 + MAPS_THREADS) {
            const int at = from.tok > row0 ? static_cast<int>(from.tok - row0) : 0;
            mark[at] = i;
            begin[at] = static_cast<int32_t>(from.tok);
            fresh_at[at] = head + static_cast<int32_t>(from.blk);
        }
        base.tok += warp_sums[31].tok;
        base.blk += warp_sums[31].blk;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        if (tid == 0) {
            a.cu_seqlens[0] = 0;
            if (blocks)
                *a.free_head_out = head + static_cast<int32_t>(cut_tok >= 0 ? cut_blk : base.blk);
        }
        if (bad)
            report(a.status, bad);
    }
    pdl_trigger();

    // ---- each row's request: the last mark at or before it
    int32_t h = mark[tid] >= 0 ? tid : -1;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t b = __shfl_up_sync(~0u, h, o);
        if (lane >= o)
            h = max(h, b);
    }
    if (lane == 31)
        warp_max[warp] = h;
    __syncthreads();
    for (int w = 0; w < warp; ++w)
        h = max(h, warp_max[w]);
    const long long total = cut_tok >= 0 ? cut_tok : base.tok;
    const long long t = row0 + tid;
    if (t >= a.C)
        return;
    int32_t seq = -1, pos = -1;
    long long place = -1;
    if (t < total && h >= 0) {
        seq = mark[h];
        pos = a.context[seq] + static_cast<int32_t>(t - begin[h]);
        if (blocks) {
            const int32_t held = a.held[seq], lb = pos / a.block_size, in = pos - lb * a.block_size;
            int32_t block;
            if (lb < held) {
                block = a.tables[seq * a.b_row + lb];
            } else {
                block = a.free_blocks[fresh_at[h] + lb - held];
                if (in == 0)                               // a new block's first token
                    a.tables[seq * a.b_row + lb] = block;
            }
            place = static_cast<long long>(block) * a.block_size + in;
        }
    }
    a.row_seq[t] = seq;
    a.positions[t] = pos;
    if (blocks)
        a.slot_map[t] = place;
}

}  // namespace spec
}  // namespace gdn
