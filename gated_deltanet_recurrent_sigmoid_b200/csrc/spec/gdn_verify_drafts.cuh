// gdn_verify_drafts.cuh -- drafted tokens judged and the next token drawn
// (gdn_verify_drafts in include/gdn_spec.h).
//
// Only the row that the token is drawn from is read whole: the judging takes
// two gathered values a draft.  One cluster per sequence; its warps sum
// w = max(p - q, 0) over contiguous segments of the row.  The segment sums
// cross the cluster through distributed shared memory; every CTA then knows W
// and which segment holds the first v with w_0 + ... + w_v > u W, and the CTA
// that owns it goes through that one segment again (from L2).  The order of all
// sums is fixed by the arguments (sizes, alignment, values), not by timing.
//
// The token must not depend on that order, so every sum is fp64: rows whose
// weights are multiples of 2^-52 of their total are summed exactly.  An
// addition is a conversion (two with q) and an fp64 operation, both at a
// fraction of the fp32 rate and still faster than pairs of fp32, 7 operations
// an element, which keep 36 to 47 bits.
// Bound by HBM while the rows stream: one row of p, one of q at a rejection.
// 128 sequences x 131072 fp32, a third of them rejected: 23.0 us (3.9 TB/s; the
// 67 MB of p alone stream in 11 us), of which about 2 pass before the rows are
// known, 4 in the exchange and the second reading, and the rest waits for the
// sequences that need q too.  One sequence of 32768: 5.2 us of latency.
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

constexpr int VERIFY_MAX_THREADS = 256;
constexpr int VERIFY_MAX_WARPS = VERIFY_MAX_THREADS / 32;
constexpr int VERIFY_MAX_CLUSTER = 8;
constexpr int VERIFY_MAX_SEGS = VERIFY_MAX_WARPS * VERIFY_MAX_CLUSTER;

// What the drafted distribution takes off p.
enum class Less { none, row, token };

// A positive finite number (or +0).
__device__ __forceinline__ bool counts(float x) { return __float_as_uint(x) < 0x7f800000u; }

// A token's weight in 64 bits: p, or p - q (exact unless their exponents lie
// further apart than 64 bits hold).
template <bool ROW>
__device__ __forceinline__ double weight(float p, float q, bool in)
{
    if (ROW) {
        in = in && fabsf(p) < INFINITY && fabsf(q) < INFINITY;
        p = in ? p : 0.f;
        q = in ? fminf(q, p) : 0.f;
        return static_cast<double>(p) - static_cast<double>(q);
    }
    return static_cast<double>(in && counts(p) ? p : 0.f);
}

// A finite x >= 0 as a double, times UNIT.  fp32 by the conversion
// instruction.  Values that were bf16 by moving the bits of exponent and
// fraction to their places, which scales by 2^-896 (exactly, subnormals too)
// and takes two shifts of full rate where the instruction has a quarter of it.
// 128 x 131072: fp32 23.0 us, by shifts 25.0; bf16 15.6, by instruction 16.7.
template <typename T> struct Wide;
template <> struct Wide<float> {
    static constexpr double UNIT = 1.;
    __device__ static double of(float x) { return static_cast<double>(x); }
};
template <> struct Wide<__nv_bfloat16> {
    static constexpr double UNIT = 0x1p-896;
    __device__ static double of(float x)
    {
        const uint32_t b = __float_as_uint(x);
        return __hiloint2double(static_cast<int>(b >> 3), static_cast<int>(b << 29));
    }
};

// Two sums side by side, for p (and q) known to be finite and not negative.
template <bool ROW, typename T>
struct WordSum {
    double a = 0., b = 0.;
    // A q above p counts as p.
    static __device__ __forceinline__ double of(float p, float q)
    {
        return ROW ? Wide<T>::of(p) - Wide<T>::of(fminf(q, p)) : Wide<T>::of(p);
    }
    __device__ __forceinline__ void add(float p0, float p1, float q0, float q1)
    {
        a += of(p0, q0);
        b += of(p1, q1);
    }
    __device__ __forceinline__ double sum() const { return (a + b) * (1. / Wide<T>::UNIT); }
};

// Sums over the lanes up to this one.
__device__ __forceinline__ double warp_upto(double x)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double b = __shfl_up_sync(~0u, x, o);
        x += lane >= o ? b : 0.;
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
    __device__ __forceinline__ double at(int64_t v) const
    {
        return weight<ROW>(Elem<T>::get(p[v]), ROW ? Elem<T>::get(q[v]) : 0.f, ROW || v != out);
    }
    __device__ __forceinline__ double any_at(int64_t v) const { return q ? at<true>(v) : at<false>(v); }
};

// U words of the row, at v, v + step, ...
template <bool ROW, int U, typename T>
struct Words {
    static constexpr int E = Elem<T>::PER16;
    uint4 p[U], q[ROW ? U : 1];
    __device__ __forceinline__ void load(const Weights<T> &w, int32_t v, int32_t step)
    {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            p[k] = __ldg(reinterpret_cast<const uint4 *>(w.p + v + k * step));
            if (ROW)
                q[k] = __ldg(reinterpret_cast<const uint4 *>(w.q + v + k * step));
        }
    }
    // Those that lie before v1; zeros, which weigh nothing, for the others.
    __device__ __forceinline__ void load_before(const Weights<T> &w, int32_t v, int32_t step, int32_t v1)
    {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool in = v + k * step + E <= v1;
            p[k] = in ? __ldg(reinterpret_cast<const uint4 *>(w.p + v + k * step)) : make_uint4(0, 0, 0, 0);
            if (ROW)
                q[k] = in ? __ldg(reinterpret_cast<const uint4 *>(w.q + v + k * step)) : make_uint4(0, 0, 0, 0);
        }
    }
    // Word k added without a look at its values; the largest bit patterns say
    // afterwards whether they were finite and not negative.
    __device__ __forceinline__ void add_valid(WordSum<ROW, T> &s, uint32_t &most, int k) const
    {
        float pf[E], qf[E];
        unpack16(p[k], pf, static_cast<const T *>(nullptr));
        most = most_bits(p[k], most, static_cast<const T *>(nullptr));
        if (ROW) {
            unpack16(q[ROW ? k : 0], qf, static_cast<const T *>(nullptr));
            most = most_bits(q[ROW ? k : 0], most, static_cast<const T *>(nullptr));
        }
#pragma unroll
        for (int j = 0; j < E; j += 2)
            s.add(pf[j], pf[j + 1], ROW ? qf[j] : 0.f, ROW ? qf[j + 1] : 0.f);
    }
    // Word k, whose first element is v.
    __device__ __forceinline__ void add_to(double (&s)[2], const Weights<T> &w, int32_t v, int k) const
    {
        float pf[E], qf[E];
        unpack16(p[k], pf, static_cast<const T *>(nullptr));
        if (ROW)
            unpack16(q[ROW ? k : 0], qf, static_cast<const T *>(nullptr));
#pragma unroll
        for (int j = 0; j < E; ++j)
            s[j & 1] += weight<ROW>(pf[j], ROW ? qf[j] : 0.f, ROW || v + j != w.out);
    }
};

// Whether the rows lie alike in their 16-byte words.
template <bool ROW, typename T>
__device__ __forceinline__ bool alike(const Weights<T> &w)
{
    return !ROW || ((reinterpret_cast<uintptr_t>(w.p) ^ reinterpret_cast<uintptr_t>(w.q)) & 15u) == 0;
}

// This lane's share of the sum over [v0, v1): every 32nd of the words that lie
// inside whole, the elements around them one by one.  (The row begins `skew`
// elements behind a 16-byte boundary.)  Where the rows lie differently in
// their words, or hold values that weigh nothing whatever the other row says
// (NaN, infinities, negative ones), every 32nd element with a look at each.
template <bool ROW, typename T>
__device__ __forceinline__ double lane_sum(const Weights<T> &w, int32_t v0, int32_t v1, int32_t skew)
{
    constexpr int E = Elem<T>::PER16, U = 4;             // elements a word, words in flight a lane
    const int lane = threadIdx.x & 31;
    if (alike<ROW>(w)) {
        WordSum<ROW, T> words;
        uint32_t most = 0;
        const int32_t lead = (E - (v0 + skew) % E) % E, first = v0 + lead;   // elements before the first whole word
        const int32_t last = v1 - (v1 + skew) % E;       // the first element behind the last whole word
        int32_t v = first;
        Words<ROW, U, T> x;
        for (; v + 32 * E * U <= last; v += 32 * E * U) {
            x.load(w, v + lane * E, 32 * E);
#pragma unroll
            for (int k = 0; k < U; ++k)
                x.add_valid(words, most, k);
        }
        if (v < last) {
            x.load_before(w, v + lane * E, 32 * E, last);
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v + 32 * E * k < last)
                    x.add_valid(words, most, k);
        }
        double s = words.sum();
        if (lane < lead && v0 + lane < v1)
            s += w.template at<ROW>(v0 + lane);
        if (last >= first && last + lane < v1)
            s += w.template at<ROW>(last + lane);
        __syncwarp();
        if (!__any_sync(~0u, beyond_finite(most, static_cast<const T *>(nullptr))))
            return s;
    }
    // (eight loads a lane kept ahead of their sums: 128 x 131071 28.0 us against 29.0)
    double s = 0.;
    auto batch = [&](int32_t v, bool whole) {
        T p[8], q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool in = whole || v + 32 * k < v1;
            p[k] = in ? w.p[v + 32 * k] : T();           // (zeros weigh nothing)
            q[k] = ROW && in ? w.q[v + 32 * k] : T();
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += weight<ROW>(Elem<T>::get(p[k]), Elem<T>::get(q[k]), ROW || v + 32 * k != w.out);
    };
    int32_t v = v0 + lane;
    for (; v + 32 * 7 < v1; v += 32 * 8)
        batch(v, true);
    if (v < v1)
        batch(v, false);
    return s;
}

// The sum over [v0, v1) by one thread, in the row's words as above.
template <bool ROW, typename T>
__device__ __forceinline__ double run_sum(const Weights<T> &w, int32_t v0, int32_t v1, int32_t skew)
{
    constexpr int E = Elem<T>::PER16, U = ROW ? 4 : 8;
    double s[2] = {0., 0.};
    int32_t v = v0;
    if (alike<ROW>(w)) {
        const int32_t lead = min((E - (v0 + skew) % E) % E, max(v1 - v0, 0));
        for (int32_t j = 0; j < lead; ++j)
            s[0] += w.template at<ROW>(v0 + j);
        for (v += lead; v + E <= v1; v += E * U) {
            Words<ROW, U, T> x;
            x.load_before(w, v, E, v1);
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (v + E * k + E <= v1)
                    x.add_to(s, w, v + E * k, k);
        }
        v = max(v1 - (v1 + skew) % E, v0 + lead);
    }
#pragma unroll 4
    for (; v < v1; ++v)
        s[0] += w.template at<ROW>(v);
    return s[0] + s[1];
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_MAX_THREADS, 4) gdn_verify_drafts_kernel(const VerifyParams a)
{
    __shared__ double part[2][VERIFY_MAX_SEGS];       // segment sums of the cluster, for either attempt
    __shared__ double scan[VERIFY_MAX_WARPS];
    __shared__ double goal_at[2];                    // u W, and the sum before the chosen segment
    __shared__ unsigned long long got[2];            // the cluster's segment sums are in
    __shared__ int chosen, first_over, last_positive, failed;
    __shared__ float uniform;                        // u, not below 0
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_index(), threads = blockDim.x, warps = threads >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int32_t i = static_cast<int32_t>(blockIdx.x / size);

    if (tid == 0) {
        failed = 0;
        for (int k = 0; k < 2; ++k) {
            sync::mbar_init(&got[k], 1);
            expect_peers(&got[k], static_cast<uint32_t>(warps) * size * sizeof(double));
        }
        sync::fence_barrier_init();
    }
    cluster_arrive(warp == 0);                        // waited for before the first exchange
    pdl_wait();

    // what does not depend on the sequence's rows is loaded beside them
    const int32_t *const tokens = a.tokens + i * a.x_seq;
    const float *const uniforms = a.uniforms + i * a.u_seq;
    int32_t x_first = lane < a.D ? tokens[lane * a.x_pos] : 0;
    float u_first = lane < a.D ? uniforms[lane * a.u_pos] : 0.f;
    if (tid == 0)
        uniform = fmaxf(uniforms[a.D * a.u_pos], 0.f);                // NaN: 0
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
    if (rank == 0)
        for (int j = tid; j <= a.D; j += threads)
            if (j != A)
                out[j * a.o_pos] = j < A ? tokens[j * a.x_pos] : -1;
    // num_tokens is written together with the token, by the CTA that has it, so
    // a count never stands beside a token that was not drawn.  (The sequence's
    // number is derived again and u waits in shared memory: kept in registers
    // over the sums they made others spill, 128 x 131072 fp32 23.1 -> 23.8 us.)
    auto finish = [&](int32_t token) {
        const int32_t seq = static_cast<int32_t>(blockIdx.x / cluster_size());
        a.out[seq * a.o_seq + A * a.o_pos] = token;
        a.num[seq * a.n_seq] = A + 1;
    };

    // ---- the sum of each segment
    Weights<T> w = {target + A * a.t_row, less == Less::row ? draft + A * a.d_pos : nullptr,
                    less == Less::token ? refused : -1};
    const int mine = static_cast<int>(rank) * warps + warp, segs = warps * static_cast<int>(size);
    const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(w.p) & 15u) / sizeof(T));
    // segments are counted from the 16-byte boundary at or before the row
    auto begin_of = [&](int segment) {
        return static_cast<int32_t>(min(max(static_cast<int64_t>(segment) * a.seg - skew, static_cast<int64_t>(0)),
                                        static_cast<int64_t>(a.vocab)));
    };
    const int32_t v0 = begin_of(mine), v1 = begin_of(mine + 1);
    for (int attempt = 0; attempt < 2; ++attempt) {
        double sum = 0.;
        if (w.q) {
            sum = lane_sum<true>(w, v0, v1, skew);
        } else {                                      // around the token that weighs nothing
            const bool cut = w.out >= v0 && w.out < v1;
            for (int32_t from = v0, to = cut ? w.out : v1;; from = to + 1, to = v1) {
                sum += lane_sum<false>(w, from, to, skew);
                if (to == v1)
                    break;
            }
        }
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(~0u, sum, o);
        if (attempt == 0)
            cluster_wait();                           // every CTA's mbarriers are there
        if (lane < static_cast<int>(size))
            st_peer(peer_addr(&part[attempt][mine], lane), sum, peer_addr(&got[attempt], lane));

        // ---- where the running sum passes u W: each lane of the first warp
        // takes a run of `per` segments
        if (warp == 0) {
            const bool in = __all_sync(~0u, mbar_wait_peers(&got[attempt], 0));
            const int per = (segs + 31) / 32, k0 = lane * per, k1 = min(k0 + per, segs);
            double own = 0.;
            for (int k = k0; k < k1; ++k)
                own += part[attempt][k];
            // (a u of 1 asks for the last token whatever the sums below round to)
            const double upto = warp_upto(own), whole = __shfl_sync(~0u, upto, 31);
            const float u = uniform;
            const double goal = u < 1.f ? whole * u : INFINITY;
            // the first segment of positive weight past the goal, else the last
            // of positive weight
            int past = segs, last = -1;
            double base = __shfl_up_sync(~0u, upto, 1);
            if (lane == 0)
                base = 0.;
            for (int k = k0; k < k1 && past == segs; ++k) {
                const double x = part[attempt][k];
                if (x > 0.) {
                    last = k;
                    if (base + x > goal)
                        past = k;
                    else
                        base += x;
                }
            }
            __syncwarp();
            const unsigned over = __ballot_sync(~0u, past < segs), some = __ballot_sync(~0u, last >= 0);
            const int from = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : 0);
            const int segment = __shfl_sync(~0u, over ? past : last, from);
            base = __shfl_sync(~0u, base, from);
            if (lane == 0) {
                chosen = segment;                     // -1: no weight at all
                failed = !in;
                goal_at[0] = over ? goal : INFINITY;
                goal_at[1] = base;
                first_over = INT32_MAX;
                last_positive = -1;
            }
        }
        if (__syncthreads_or(failed)) {
            if (tid == 0) {                           // (the CTA that finds the token may not have given up)
                a.num[static_cast<int32_t>(blockIdx.x / cluster_size()) * a.n_seq] = 0;
                report(a.status, GDN_DEV_TIMEOUT);
            }
            cluster_leave();
            return;
        }
        const int segment = __shfl_sync(~0u, chosen, 0);
        if (segment < 0) {
            if (w.q || w.out >= 0) {                  // p <= q everywhere: draw from p itself
                w.q = nullptr;
                w.out = -1;
                continue;
            }
            if (rank == 0 && tid == 0) {
                finish(-1);
                report(a.status, GDN_DEV_BAD_PROBS);
            }
            return;
        }
        if (segment / warps != static_cast<int>(rank))
            return;

        // ---- that segment again: each thread sums a contiguous run of it
        const double goal = goal_at[0];
        const int32_t g0 = begin_of(segment), g1 = begin_of(segment + 1);
        const int32_t each = ((a.seg + threads - 1) / threads + 7) / 8 * 8;      // whole words
        const int64_t run0 = static_cast<int64_t>(segment) * a.seg + static_cast<int64_t>(tid) * each - skew;
        const int32_t r0 = static_cast<int32_t>(min(max(run0, static_cast<int64_t>(g0)), static_cast<int64_t>(g1)));
        const int32_t r1 = static_cast<int32_t>(min(max(run0 + each, static_cast<int64_t>(g0)), static_cast<int64_t>(g1)));
        const double own = w.q ? run_sum<true>(w, r0, r1, skew) : run_sum<false>(w, r0, r1, skew);
        const double run = warp_upto(own);
        if (lane == 31)
            scan[warp] = run;
        __syncthreads();
        double at = goal_at[1];                       // the weight before this thread's run
        for (int k = 0; k < warp; ++k)
            at += scan[k];
        const double prior = __shfl_up_sync(~0u, run, 1);
        if (lane > 0)
            at += prior;
        if (own > 0.) {
            if (at + own > goal)
                atomicMin(&first_over, tid);
            atomicMax(&last_positive, tid);
        }
        __syncthreads();
        // its warp goes through that thread's run, 32 elements at a time
        const int holder = __shfl_sync(~0u, first_over != INT32_MAX ? first_over : last_positive, 0);
        if (holder / 32 != warp)
            return;
        const int32_t h0 = __shfl_sync(~0u, r0, holder & 31), h1 = __shfl_sync(~0u, r1, holder & 31);
        double upto = __shfl_sync(~0u, at, holder & 31);
        int32_t token = -1;
        for (int32_t v = h0; v < h1; v += 32) {
            const double x = v + lane < h1 ? w.any_at(v + lane) : 0.;
            const double sums = warp_upto(x), before = __shfl_up_sync(~0u, sums, 1);
            const double from = upto + (lane ? before : 0.);
            const unsigned some = __ballot_sync(~0u, x > 0.), over = __ballot_sync(~0u, x > 0. && from + x > goal);
            if (over) {
                token = v + __ffs(over) - 1;
                break;
            }
            if (some)
                token = v + 31 - __clz(some);
            upto += __shfl_sync(~0u, sums, 31);
        }
        if (lane == 0)
            finish(token);
        return;
    }
}

}  // namespace spec
}  // namespace gdn
