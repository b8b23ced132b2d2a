// gdn_verify_drafts.cuh -- drafted tokens judged and the next token drawn
// (gdn_verify_drafts in include/gdn_spec.h).
//
// Only the row that the token is drawn from is read whole: the judging takes
// two gathered values a draft.  One cluster per sequence; its warps sum
// w = max(p - q, 0) over contiguous segments of the row.  The segment sums
// cross the cluster through distributed shared memory; every CTA then knows W
// and which segment holds the first v with w_0 + ... + w_v > u W, and the CTA
// that owns it goes through that one segment again (from L2).  The order of all
// sums is fixed by the sizes alone.
//
// The token must not depend on that order, so a sum keeps what its additions
// round off: it is a pair (s, c) of fp32 values, s the rounded sum and c the
// exact errors of its additions (and of p - q) added up, good to about 2^-48.
// An addition is 7 fp32 operations at 128 a clock and SM; one in fp64 would
// need 2 conversions (4 with q) at 16 a clock beside it.
// Bound by HBM: one row of p, one of q at a rejection.
#pragma once

#include "gdn_spec_common.cuh"

namespace gdn {
namespace spec {

struct VerifyParams {
    const void *target, *draft;
    const int32_t *tokens;
    const float *uniforms;
    const int32_t *cu_seqlens, *indices;
    int32_t *out, *num;
    uint32_t *status;
    int64_t t_row;                   // element strides
    int64_t x_seq, x_pos;
    int64_t d_seq, d_pos;
    int64_t u_seq, u_pos;
    int64_t o_seq, o_pos, n_seq;
    int32_t N, D, T_fixed, T_tot, vocab;
    int32_t seg;                     // elements per warp, a multiple of a warp's 16-byte words
};

constexpr int VERIFY_MAX_THREADS = 1024;
constexpr int VERIFY_MAX_WARPS = VERIFY_MAX_THREADS / 32;
constexpr int VERIFY_MAX_CLUSTER = 8;
constexpr int VERIFY_MAX_SEGS = VERIFY_MAX_WARPS * VERIFY_MAX_CLUSTER;

// What the drafted distribution takes off p.
enum class Less { none, row, token };

// A positive finite number (or +0).
__device__ __forceinline__ bool counts(float x) { return __float_as_uint(x) < 0x7f800000u; }

// A sum that keeps its rounding errors: s + c.
struct PairSum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = s + x, b = t - s;
        c += (s - (t - b)) + (x - b);                // s + x = t + this, exactly
        s = t;
    }
    __device__ __forceinline__ void add(const PairSum &x)
    {
        add(x.s);
        c += x.c;
    }
    // The weight of a token: p, or p - q.
    template <bool ROW>
    __device__ __forceinline__ void weight(float p, float q, bool in)
    {
        if (ROW) {
            const float d = p - q, e = (p - d) - q;  // p - q = d + e, exactly (0 <= q < p)
            in = in && counts(d);
            add(in ? d : 0.f);
            c += in ? e : 0.f;
        } else {
            add(in && counts(p) ? p : 0.f);
        }
    }
    __device__ __forceinline__ bool positive() const { return s + c > 0.f; }
    // Whether this + x > goal.
    __device__ __forceinline__ bool passes(const PairSum &x, const PairSum &goal) const
    {
        PairSum d = *this;
        d.add(x);
        d.add(PairSum{-goal.s, -goal.c});
        return d.s + d.c > 0.f;
    }
    __device__ __forceinline__ PairSum times(float u) const
    {
        const float x = u * s;
        return PairSum{x, fmaf(u, s, -x) + u * c};
    }
};

__device__ __forceinline__ PairSum shfl(const PairSum &x, int from)
{
    return PairSum{__shfl_sync(~0u, x.s, from), __shfl_sync(~0u, x.c, from)};
}
__device__ __forceinline__ PairSum shfl_up(const PairSum &x, int by)
{
    return PairSum{__shfl_up_sync(~0u, x.s, by), __shfl_up_sync(~0u, x.c, by)};
}
// Sums over the lanes up to this one.
__device__ __forceinline__ PairSum warp_upto(PairSum x)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const PairSum b = shfl_up(x, o);
        x.add(lane >= o ? b : PairSum{});
    }
    return x;
}

// Whether u q < p, exactly: the fused multiply-add's one rounding keeps the
// sign, and values near the smallest numbers are scaled away from them first.
__device__ __forceinline__ bool accepts(float u, float q, float p)
{
    const float by = p < 0x1p-40f && q < 0x1p40f ? 0x1p80f : 1.f;
    return fmaf(u, q * by, -(p * by)) < 0.f;
}

// A row's weights: p, less the row q or less the token `out`.
template <typename T>
struct Weights {
    const T *p, *q;
    int32_t out;
    template <bool ROW>
    __device__ __forceinline__ void add_to(PairSum &s, int64_t v) const
    {
        s.weight<ROW>(Elem<T>::get(p[v]), ROW ? Elem<T>::get(q[v]) : 0.f, ROW || v != out);
    }
    __device__ __forceinline__ PairSum at(int64_t v) const
    {
        PairSum s;
        if (q)
            add_to<true>(s, v);
        else
            add_to<false>(s, v);
        return s;
    }
};

// This lane's share of the sum over a segment of the row.  The segment is
// counted from the 16-byte boundary at or before the row, `skew` elements
// before it: x0 <= v + skew < x1, x0 a multiple of a warp's 16-byte words, so
// that all but the row's first and last word are loaded whole.  Where q lies
// differently in its words both rows are loaded element by element.
template <bool ROW, typename T>
__device__ __forceinline__ PairSum lane_sum(const Weights<T> &w, int32_t x0, int32_t x1, int32_t skew, int32_t vocab)
{
    constexpr int E = Elem<T>::PER16, U = 4;         // elements a word, words in flight a lane
    const int lane = threadIdx.x & 31;
    PairSum s[2];
    if (ROW && ((reinterpret_cast<uintptr_t>(w.p) ^ reinterpret_cast<uintptr_t>(w.q)) & 15u) != 0) {
        const int32_t v1 = min(x1 - skew, vocab);
#pragma unroll 8
        for (int32_t v = max(x0 - skew, 0) + lane; v < v1; v += 32)
            w.template add_to<ROW>(s[0], v);
        return s[0];
    }
    for (int32_t x = x0 + lane * E; x < x1; x += 32 * E * U) {
        uint4 p[U], q[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int32_t v = x - skew + 32 * E * k;
            const bool whole = x + 32 * E * k < x1 && v >= 0 && v + E <= vocab;
            p[k] = whole ? __ldg(reinterpret_cast<const uint4 *>(w.p + v)) : make_uint4(0, 0, 0, 0);
            if (ROW)
                q[k] = whole ? __ldg(reinterpret_cast<const uint4 *>(w.q + v)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float pf[E], qf[E];
            unpack16(p[k], pf, static_cast<const T *>(nullptr));
            if (ROW)
                unpack16(q[k], qf, static_cast<const T *>(nullptr));
#pragma unroll
            for (int j = 0; j < E; ++j)
                s[j & 1].template weight<ROW>(pf[j], ROW ? qf[j] : 0.f, ROW || x - skew + 32 * E * k + j != w.out);
        }
    }
    // the row's first and last word, where they are not whole: with the lane
    // that they would have gone to
    const int32_t first = skew ? E - skew : 0;       // elements before the first whole word
    const int32_t last = max((vocab + skew) / E * E - skew, first);   // the first behind the last whole one
    if (x0 == 0 && lane == 0)
        for (int32_t v = 0; v < min(first, vocab); ++v)
            w.template add_to<ROW>(s[0], v);
    if (last < vocab && x0 <= last + skew && last + skew < x1 && lane == (last + skew) / E % 32)
        for (int32_t v = last; v < vocab; ++v)
            w.template add_to<ROW>(s[0], v);
    s[0].add(s[1]);
    return s[0];
}

// The sum over v0 <= v < v1 by one thread.
template <bool ROW, typename T>
__device__ __forceinline__ PairSum run_sum(const Weights<T> &w, int64_t v0, int64_t v1)
{
    PairSum s;
#pragma unroll 8
    for (int64_t v = v0; v < v1; ++v)
        w.template add_to<ROW>(s, v);
    return s;
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_MAX_THREADS) gdn_verify_drafts_kernel(const VerifyParams a)
{
    __shared__ PairSum part[2][VERIFY_MAX_SEGS];      // segment sums of the cluster, for either attempt
    __shared__ PairSum scan[VERIFY_MAX_WARPS];
    __shared__ PairSum goal_at[2];                   // u W, and the sum before the chosen segment
    __shared__ int chosen, first_over, last_positive;
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index(), threads = blockDim.x, warps = threads >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int32_t i = static_cast<int32_t>(blockIdx.x / size);

    cluster_arrive();
    pdl_wait();

    // what does not depend on the sequence's rows is loaded beside them
    const int32_t *const tokens = a.tokens + i * a.x_seq;
    const float *const uniforms = a.uniforms + i * a.u_seq;
    int32_t x_first = lane < a.D ? tokens[lane * a.x_pos] : 0;
    float u_first = lane < a.D ? uniforms[lane * a.u_pos] : 0.f;
    const float u = fmaxf(uniforms[a.D * a.u_pos], 0.f);              // NaN: 0
    int32_t start, len;
    bool runs = rows_of(a.cu_seqlens, a.T_fixed, a.T_tot, i, &start, &len);
    if (!runs || len - 1 > a.D) {
        runs = false;
        if (rank == 0 && tid == 0)
            report(a.status, GDN_DEV_BAD_SEQLENS);
    }
    runs = runs && len > 0 && !(a.indices && a.indices[i] < 0);
    int32_t *const out = a.out + i * a.o_seq;
    if (!runs) {
        if (rank == 0) {
            for (int j = tid; j <= a.D; j += threads)
                out[j * a.o_pos] = -1;
            if (tid == 0)
                a.num[i * a.n_seq] = 0;
        }
        cluster_wait();
        return;
    }
    const T *const target = static_cast<const T *>(a.target) + start * a.t_row;
    const T *const draft = a.draft ? static_cast<const T *>(a.draft) + i * a.d_seq : nullptr;

    // ---- A: the accepted drafts before the first rejection (every warp finds
    // it for itself)
    const int32_t d = len - 1;
    int32_t A = d;
    Less less = Less::none;
    int32_t refused = -1;
    for (int32_t j0 = 0; j0 < d && A == d; j0 += 32) {
        const int32_t j = j0 + lane;
        bool accepted = true, inside = true;
        int32_t x = 0;
        if (j < d) {
            x = j0 ? tokens[j * a.x_pos] : x_first;
            const float uj = j0 ? uniforms[j * a.u_pos] : u_first;
            inside = x >= 0 && x < a.vocab;
            accepted = false;
            if (inside) {
                const float pv = Elem<T>::get(target[j * a.t_row + x]);
                accepted = accepts(uj, draft ? Elem<T>::get(draft[j * a.d_pos + x]) : 1.f, pv);
            }
        }
        __syncwarp();
        const unsigned no = __ballot_sync(~0u, !accepted);
        if (no) {
            const int at = __ffs(no) - 1;
            A = j0 + at;
            refused = __shfl_sync(~0u, x, at);
            const bool was_inside = __shfl_sync(~0u, inside, at);
            if (was_inside)
                less = draft ? Less::row : Less::token;
            else if (refused != -1 && rank == 0 && tid == 0)
                report(a.status, GDN_DEV_BAD_TOKEN);
        }
    }
    if (rank == 0) {
        for (int j = tid; j <= a.D; j += threads)
            if (j != A)
                out[j * a.o_pos] = j < A ? tokens[j * a.x_pos] : -1;
        if (tid == 0)
            a.num[i * a.n_seq] = A + 1;
    }

    // ---- the sum of each segment
    Weights<T> w = {target + A * a.t_row, less == Less::row ? draft + A * a.d_pos : nullptr,
                    less == Less::token ? refused : -1};
    const int mine = static_cast<int>(rank) * warps + warp, segs = warps * static_cast<int>(size);
    const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(w.p) & 15u) / sizeof(T));
    const int32_t x1 = static_cast<int32_t>(min((static_cast<int64_t>(mine) + 1) * a.seg, static_cast<int64_t>(a.vocab) + skew));
    const int32_t x0 = static_cast<int32_t>(min(static_cast<int64_t>(mine) * a.seg, static_cast<int64_t>(x1)));
    for (int attempt = 0; attempt < 2; ++attempt) {
        PairSum sum = w.q ? lane_sum<true>(w, x0, x1, skew, a.vocab) : lane_sum<false>(w, x0, x1, skew, a.vocab);
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum.add(PairSum{__shfl_xor_sync(~0u, sum.s, o), __shfl_xor_sync(~0u, sum.c, o)});
        if (attempt == 0)
            cluster_wait();                           // every CTA of the cluster has begun
        if (lane < static_cast<int>(size))
            st_peer(peer_addr(&part[attempt][mine], lane), sum.s, sum.c);
        cluster_arrive();
        cluster_wait();

        // ---- where the running sum passes u W: each lane of the first warp
        // takes a run of `per` segments
        if (warp == 0) {
            const int per = (segs + 31) / 32, k0 = lane * per, k1 = min(k0 + per, segs);
            PairSum own;
            for (int k = k0; k < k1; ++k)
                own.add(part[attempt][k]);
            const PairSum upto = warp_upto(own), goal = shfl(upto, 31).times(u);
            // the first segment of positive weight past the goal, else the last
            // of positive weight
            int past = segs, last = -1;
            PairSum base = shfl_up(upto, 1);
            if (lane == 0)
                base = PairSum{};
            for (int k = k0; k < k1 && past == segs; ++k) {
                const PairSum x = part[attempt][k];
                if (x.positive()) {
                    last = k;
                    if (base.passes(x, goal))
                        past = k;
                    else
                        base.add(x);
                }
            }
            __syncwarp();
            const unsigned over = __ballot_sync(~0u, past < segs), some = __ballot_sync(~0u, last >= 0);
            const int from = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : 0);
            const int segment = __shfl_sync(~0u, over ? past : last, from);
            base = shfl(base, from);
            if (lane == 0) {
                chosen = segment;                     // -1: no weight at all
                goal_at[0] = over ? goal : PairSum{INFINITY, 0.f};
                goal_at[1] = base;
                first_over = INT32_MAX;
                last_positive = -1;
            }
        }
        __syncthreads();
        const int segment = chosen;
        if (segment < 0) {
            if (w.q || w.out >= 0) {                  // p <= q everywhere: draw from p itself
                w.q = nullptr;
                w.out = -1;
                continue;
            }
            if (rank == 0 && tid == 0) {
                out[A * a.o_pos] = -1;
                report(a.status, GDN_DEV_BAD_PROBS);
            }
            return;
        }
        pdl_trigger();
        if (segment / warps != static_cast<int>(rank))
            return;

        // ---- that segment again: each thread sums a contiguous run, and the
        // one whose run holds the token goes through it element by element
        const PairSum goal = goal_at[0];
        const int64_t g0 = max(static_cast<int64_t>(segment) * a.seg - skew, static_cast<int64_t>(0));
        const int64_t g1 = min(static_cast<int64_t>(segment + 1) * a.seg - skew, static_cast<int64_t>(a.vocab));
        const int32_t each = (a.seg + threads - 1) / threads;
        const int64_t r0 = min(g0 + static_cast<int64_t>(tid) * each, g1), r1 = min(r0 + each, g1);
        const PairSum own = w.q ? run_sum<true>(w, r0, r1) : run_sum<false>(w, r0, r1);
        const PairSum run = warp_upto(own);
        if (lane == 31)
            scan[warp] = run;
        __syncthreads();
        PairSum at = goal_at[1];                      // the weight before this thread's run
        for (int k = 0; k < warp; ++k)
            at.add(scan[k]);
        const PairSum prior = shfl_up(run, 1);
        if (lane > 0)
            at.add(prior);
        if (own.positive()) {
            if (at.passes(own, goal))
                atomicMin(&first_over, tid);
            atomicMax(&last_positive, tid);
        }
        __syncthreads();
        if (tid == (first_over != INT32_MAX ? first_over : last_positive)) {
            int32_t token = -1;
            for (int64_t v = r0; v < r1; ++v) {
                const PairSum x = w.at(v);
                if (x.positive()) {
                    token = static_cast<int32_t>(v);
                    if (at.passes(x, goal))
                        break;
                    at.add(x);
                }
            }
            out[A * a.o_pos] = token;
        }
        return;
    }
}

}  // namespace spec
}  // namespace gdn
