// gdn_verify_drafts.cuh -- drafted tokens judged and the next token drawn
// (gdn_verify_drafts in include/gdn_spec.h).
//
// Only the row that the token is drawn from is read whole: the judging takes
// two gathered values a draft, u q against p in fp64, where the product of two
// fp32 values is exact.  One cluster per sequence; its warps sum w = max(p - q,
// 0) over contiguous segments of the row.  The segment sums cross the cluster
// through distributed shared memory; every CTA then knows W and which segment
// holds the first v with w_0 + ... + w_v > u W, and the CTA that owns it goes
// through that one segment again (from L2).  The order of all sums is fixed by
// the sizes alone.
//
// The token must not depend on that order, so a running sum keeps what its
// additions round off: a pair (s, c) of fp32 values per lane, s the sum and c
// the exact errors of its additions (and of p - q) added up, about 2^-48
// relative each; lanes and segments are joined in fp64.  fp64 throughout costs
// more: converting and adding an element is 2 (4 with q) fp64 operations at
// about 8 a clock and SM here, 7 (14) fp32 ones at 128.
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
    int32_t seg;                     // elements per warp
};

constexpr int VERIFY_MAX_THREADS = 1024;
constexpr int VERIFY_MAX_WARPS = VERIFY_MAX_THREADS / 32;
constexpr int VERIFY_MAX_CLUSTER = 8;
constexpr int VERIFY_MAX_SEGS = VERIFY_MAX_WARPS * VERIFY_MAX_CLUSTER;

// What the drafted distribution takes off p.
enum class Less { none, row, token };

// A positive finite number (or +0).
__device__ __forceinline__ bool counts(float x) { return __float_as_uint(x) < 0x7f800000u; }

// A running sum that keeps its rounding errors.
struct PairSum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = s + x, b = t - s;
        c += (s - (t - b)) + (x - b);                // s + x = t + this, exactly
        s = t;
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
    __device__ __forceinline__ double value() const { return static_cast<double>(s) + static_cast<double>(c); }
};

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
    // The same weight in fp64.
    __device__ __forceinline__ double at(int64_t v) const
    {
        PairSum s;
        if (q)
            add_to<true>(s, v);
        else
            add_to<false>(s, v);
        return s.value();
    }
};

// This lane's share of the sum over v0 <= v < v1: every 32nd.
template <bool ROW, typename T>
__device__ __forceinline__ double lane_sum(const Weights<T> &w, int64_t v0, int64_t v1)
{
    constexpr int U = 16;                            // loads in flight a thread, of either row
    PairSum s[2];
    int64_t v = v0 + (threadIdx.x & 31);
    for (; v + 32 * (U - 1) < v1; v += 32 * U) {
        T p[U], q[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            p[k] = w.p[v + 32 * k];
            if (ROW)
                q[k] = w.q[v + 32 * k];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            s[k & 1].template weight<ROW>(Elem<T>::get(p[k]), ROW ? Elem<T>::get(q[k]) : 0.f, ROW || v + 32 * k != w.out);
    }
#pragma unroll 4
    for (; v < v1; v += 32)
        w.template add_to<ROW>(s[0], v);
    return s[0].value() + s[1].value();
}

// The sum over v0 <= v < v1 by one thread.
template <bool ROW, typename T>
__device__ __forceinline__ double run_sum(const Weights<T> &w, int64_t v0, int64_t v1)
{
    PairSum s;
#pragma unroll 8
    for (int64_t v = v0; v < v1; ++v)
        w.template add_to<ROW>(s, v);
    return s.value();
}

__device__ __forceinline__ double warp_upto(double x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double b = __shfl_up_sync(~0u, x, o);
        if (lane >= o)
            x += b;
    }
    return x;
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_MAX_THREADS) gdn_verify_drafts_kernel(const VerifyParams a)
{
    __shared__ double part[2][VERIFY_MAX_SEGS];      // segment sums of the cluster, for either attempt
    __shared__ double scan[VERIFY_MAX_WARPS];
    __shared__ double goal_at[2];                    // u W, and the sum before the chosen segment
    __shared__ int chosen, first_over, last_positive;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
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
                const double pv = Elem<T>::get(target[j * a.t_row + x]);
                const double qv = draft ? static_cast<double>(Elem<T>::get(draft[j * a.d_pos + x])) : 1.0;
                accepted = static_cast<double>(uj) * qv < pv;
            }
        }
        const unsigned no = __ballot_sync(~0u, !accepted);
        if (no) {
            const int at = __ffs(no) - 1;
            A = j0 + at;
            refused = __shfl_sync(~0u, x, at);
            if (__shfl_sync(~0u, inside, at))
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
    const int64_t v0 = min(static_cast<int64_t>(mine) * a.seg, static_cast<int64_t>(a.vocab));
    const int64_t v1 = min(v0 + a.seg, static_cast<int64_t>(a.vocab));
    for (int attempt = 0; attempt < 2; ++attempt) {
        double sum = w.q ? lane_sum<true>(w, v0, v1) : lane_sum<false>(w, v0, v1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(~0u, sum, o);
        if (attempt == 0)
            cluster_wait();                           // every CTA of the cluster has begun
        if (lane < static_cast<int>(size))
            st_peer(peer_addr(&part[attempt][mine], lane), sum);
        cluster_arrive();
        cluster_wait();

        // ---- where the running sum passes u W: each lane of the first warp
        // takes a run of `per` segments
        if (warp == 0) {
            const int per = (segs + 31) / 32, k0 = lane * per, k1 = min(k0 + per, segs);
            double own = 0;
            for (int k = k0; k < k1; ++k)
                own += part[attempt][k];
            const double upto = warp_upto(own), total = __shfl_sync(~0u, upto, 31);
            const double goal = static_cast<double>(u) * total, before = __shfl_up_sync(~0u, upto, 1);
            // the first segment of positive weight past the goal, else the last
            // of positive weight
            int past = segs, last = -1;
            double base = lane ? before : 0.0;
            for (int k = k0; k < k1 && past == segs; ++k) {
                const double x = part[attempt][k];
                if (x > 0) {
                    last = k;
                    if (base + x > goal)
                        past = k;
                    else
                        base += x;
                }
            }
            const unsigned over = __ballot_sync(~0u, past < segs), some = __ballot_sync(~0u, last >= 0);
            const int from = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : 0);
            const int segment = __shfl_sync(~0u, over ? past : last, from);
            base = __shfl_sync(~0u, base, from);
            if (lane == 0) {
                chosen = segment;                     // -1: no weight at all
                goal_at[0] = over ? goal : INFINITY;
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
        const double goal = goal_at[0];
        const int64_t g0 = static_cast<int64_t>(segment) * a.seg;
        const int64_t g1 = min(g0 + a.seg, static_cast<int64_t>(a.vocab));
        const int32_t each = (a.seg + threads - 1) / threads;
        const int64_t r0 = min(g0 + static_cast<int64_t>(tid) * each, g1), r1 = min(r0 + each, g1);
        const double own = w.q ? run_sum<true>(w, r0, r1) : run_sum<false>(w, r0, r1);
        const double run = warp_upto(own);
        if (lane == 31)
            scan[warp] = run;
        __syncthreads();
        double at = goal_at[1];
        for (int k = 0; k < warp; ++k)
            at += scan[k];
        const double prior = __shfl_up_sync(~0u, run, 1);
        at += lane ? prior : 0.0;                     // the weight before this thread's run
        if (own > 0) {
            if (at + own > goal)
                atomicMin(&first_over, tid);
            atomicMax(&last_positive, tid);
        }
        __syncthreads();
        if (tid == (first_over != INT32_MAX ? first_over : last_positive)) {
            int32_t token = -1;
            for (int64_t v = r0; v < r1; ++v) {
                const double x = w.at(v);
                if (x > 0) {
                    at += x;
                    token = static_cast<int32_t>(v);
                    if (at > goal)
                        break;
                }
            }
            out[A * a.o_pos] = token;
        }
        return;
    }
}

}  // namespace spec
}  // namespace gdn
