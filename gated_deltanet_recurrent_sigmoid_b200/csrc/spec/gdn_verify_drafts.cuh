// gdn_verify_drafts.cuh -- drafted tokens judged and the next token drawn
// (gdn_verify_drafts in include/gdn_spec.h).
//
// Only the row that the token is drawn from is read whole: the judging takes
// two gathered values a draft.  One cluster per sequence; its warps take
// contiguous segments of the row and sum w = max(p - q, 0) in fp64 (products
// u q and differences p - q of fp32 values lose nothing there that could turn
// a comparison).  The segment sums cross the cluster through distributed
// shared memory; every CTA then knows W and which segment holds the first
// v with w_0 + ... + w_v > u W, and the CTA that owns it goes through that
// one segment again (from L2).  The order of all sums is fixed by the sizes
// alone.  Bound by HBM: one row of p, one of q at a rejection.
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

constexpr int VERIFY_THREADS = 256;
constexpr int VERIFY_WARPS = VERIFY_THREADS / 32;
constexpr int VERIFY_MAX_CLUSTER = 8;
constexpr int VERIFY_MAX_SEGS = VERIFY_WARPS * VERIFY_MAX_CLUSTER;
static_assert(VERIFY_MAX_SEGS == 64, "two segment sums a lane");

// What the drafted distribution takes off p.
enum class Less { none, row, token };

// The weight of one token.  p > q and the finiteness tests are exact in fp32.
__device__ __forceinline__ double weight(float p, float q)
{
    return p > q && fabsf(p) < INFINITY && fabsf(q) < INFINITY ? static_cast<double>(p) - static_cast<double>(q) : 0.0;
}

template <typename T>
__device__ __forceinline__ double weight_at(const T *p, const T *q, Less less, int32_t token, int32_t v)
{
    const float pv = Elem<T>::get(p[v]);
    const float qv = less == Less::row ? Elem<T>::get(q[v]) : 0.f;
    return less == Less::token && v == token ? 0.0 : weight(pv, qv);
}

template <typename T>
__global__ void __launch_bounds__(VERIFY_THREADS) gdn_verify_drafts_kernel(const VerifyParams a)
{
    __shared__ double part[2][VERIFY_MAX_SEGS];      // segment sums of the cluster, for either attempt
    __shared__ double scan[VERIFY_WARPS];
    __shared__ int first_over, last_positive;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int32_t i = static_cast<int32_t>(blockIdx.x / size);

    cluster_arrive();
    pdl_wait();

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
            for (int j = tid; j <= a.D; j += VERIFY_THREADS)
                out[j * a.o_pos] = -1;
            if (tid == 0)
                a.num[i * a.n_seq] = 0;
        }
        cluster_wait();
        return;
    }
    const T *const target = static_cast<const T *>(a.target) + start * a.t_row;
    const T *const draft = a.draft ? static_cast<const T *>(a.draft) + i * a.d_seq : nullptr;
    const int32_t *const tokens = a.tokens + i * a.x_seq;
    const float *const uniforms = a.uniforms + i * a.u_seq;

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
            x = tokens[j * a.x_pos];
            inside = x >= 0 && x < a.vocab;
            accepted = false;
            if (inside) {
                const double pv = Elem<T>::get(target[j * a.t_row + x]);
                const double qv = draft ? static_cast<double>(Elem<T>::get(draft[j * a.d_pos + x])) : 1.0;
                accepted = static_cast<double>(uniforms[j * a.u_pos]) * qv < pv;
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
        for (int j = tid; j <= a.D; j += VERIFY_THREADS)
            if (j != A)
                out[j * a.o_pos] = j < A ? tokens[j * a.x_pos] : -1;
        if (tid == 0)
            a.num[i * a.n_seq] = A + 1;
    }

    // ---- the sum of each segment
    const T *const prow = target + A * a.t_row;
    const T *const qrow = less == Less::row ? draft + A * a.d_pos : nullptr;
    const float u = fmaxf(uniforms[a.D * a.u_pos], 0.f);              // NaN: 0
    const int segs = VERIFY_WARPS * static_cast<int>(size);
    bool waited = false;
    for (int attempt = 0; attempt < 2; ++attempt) {
        const int64_t v0 = static_cast<int64_t>(rank * VERIFY_WARPS + warp) * a.seg;
        const int32_t v1 = static_cast<int32_t>(min(v0 + a.seg, static_cast<int64_t>(a.vocab)));
        double sum = 0;
#pragma unroll 8
        for (int64_t v = v0 + lane; v < v1; v += 32)
            sum += weight_at(prow, qrow, less, refused, static_cast<int32_t>(v));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(~0u, sum, o);
        if (!waited)
            cluster_wait();                           // every CTA of the cluster has begun
        waited = true;
        if (lane < static_cast<int>(size))
            st_peer(peer_addr(&part[attempt][rank * VERIFY_WARPS + warp], lane), sum);
        cluster_arrive();
        cluster_wait();

        // ---- where the running sum passes u W (every warp for itself)
        double s0 = 2 * lane < segs ? part[attempt][2 * lane] : 0.0;
        double s1 = 2 * lane + 1 < segs ? part[attempt][2 * lane + 1] : 0.0;
        double upto = s0 + s1;                        // inclusive over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double b = __shfl_up_sync(~0u, upto, o);
            if (lane >= o)
                upto += b;
        }
        const double total = __shfl_sync(~0u, upto, 31);
        if (!(total > 0.0)) {
            if (less != Less::none) {                 // p <= q everywhere: draw from p itself
                less = Less::none;
                continue;
            }
            if (rank == 0 && tid == 0) {
                out[A * a.o_pos] = -1;
                report(a.status, GDN_DEV_BAD_PROBS);
            }
            return;
        }
        const double goal = static_cast<double>(u) * total;
        double before = __shfl_up_sync(~0u, upto, 1);
        before = lane ? before : 0.0;
        // the first segment past the goal, else the last of positive weight
        const int mine = before + s0 > goal && s0 > 0 ? 2 * lane : (upto > goal && s1 > 0 ? 2 * lane + 1 : segs);
        const unsigned over = __ballot_sync(~0u, mine < segs);
        int segment;
        double base;
        if (over) {
            const int l = __ffs(over) - 1;
            segment = __shfl_sync(~0u, mine, l);
            base = __shfl_sync(~0u, segment & 1 ? before + s0 : before, l);
        } else {
            const unsigned some = __ballot_sync(~0u, s0 > 0 || s1 > 0);
            const int l = 31 - __clz(some);
            segment = __shfl_sync(~0u, s1 > 0 ? 2 * lane + 1 : 2 * lane, l);
            base = 0;
        }
        pdl_trigger();
        if (segment / VERIFY_WARPS != static_cast<int>(rank))
            return;

        // ---- that segment again, a contiguous run of it per thread
        if (tid == 0) {
            first_over = INT32_MAX;
            last_positive = -1;
        }
        const int64_t g0 = static_cast<int64_t>(segment) * a.seg;
        const int32_t g1 = static_cast<int32_t>(min(g0 + a.seg, static_cast<int64_t>(a.vocab)));
        const int32_t each = (a.seg + VERIFY_THREADS - 1) / VERIFY_THREADS;
        const int64_t r0 = g0 + static_cast<int64_t>(tid) * each;
        const int32_t r1 = static_cast<int32_t>(min(r0 + each, static_cast<int64_t>(g1)));
        double own = 0;
        for (int64_t v = r0; v < r1; ++v)
            own += weight_at(prow, qrow, less, refused, static_cast<int32_t>(v));
        double run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double b = __shfl_up_sync(~0u, run, o);
            if (lane >= o)
                run += b;
        }
        if (lane == 31)
            scan[warp] = run;
        __syncthreads();
        double at = over ? base : 0.0;
        for (int k = 0; k < warp; ++k)
            at += scan[k];
        at += run - own;                              // the weight before this thread's run
        int32_t last = -1;
        for (int64_t v = r0; v < r1; ++v) {
            const double w = weight_at(prow, qrow, less, refused, static_cast<int32_t>(v));
            if (w > 0) {
                at += w;
                last = static_cast<int32_t>(v);
                if (over && at > goal) {
                    atomicMin(&first_over, last);
                    break;
                }
            }
        }
        if (last >= 0)
            atomicMax(&last_positive, last);
        __syncthreads();
        if (tid == 0)
            out[A * a.o_pos] = first_over != INT32_MAX ? first_over : last_positive;
        return;
    }
}

}  // namespace spec
}  // namespace gdn
