// gdn_token_probs.cuh -- probabilities of logit rows (gdn_token_probs in
// include/gdn_spec.h).
//
// p_v = exp((l_v - m) / t) / sum_w exp((l_w - m) / t), m the row's maximum.
// One cluster per row; each CTA holds a contiguous slice of the row in shared
// memory (one bulk copy per piece, so HBM is read once), and the row's
// maximum and sum come from one pass that keeps both running:
//     (m, s) + x  ->  (m', s 2^((m - m') c) + 2^((x - m') c)),  c = log2(e) / t.
// The CTAs' pairs cross the cluster through distributed shared memory, one
// barrier, and the second pass reads the slice again from shared memory.
// Bound by HBM: each logit read once, each probability written once.
#pragma once

#include "gdn_spec_common.cuh"

namespace gdn {
namespace spec {

struct ProbsParams {
    const void *logits;
    void *probs;
    const float *temperature;
    const int32_t *row_seq;
    uint32_t *status;
    int64_t l_row, p_row, t_stride;
    int32_t vocab;
    int32_t slice;      // elements per CTA, a multiple of 8
    int32_t num_temps;
};

constexpr int PROBS_THREADS = 256;
constexpr int PROBS_PIECE = 8192;                          // bytes per bulk copy and mbarrier
constexpr int PROBS_MAX_SLICE_BYTES = GDN_SPEC_MAX_VOCAB / 8 * 4;
constexpr int PROBS_MAX_PIECES = PROBS_MAX_SLICE_BYTES / PROBS_PIECE + 2;
constexpr int PROBS_MAX_CLUSTER = 8;

struct ProbsShared {
    float2 cta[PROBS_MAX_CLUSTER];                         // (m, s) or (m, index) of each CTA of the cluster
    float2 warp[PROBS_THREADS / 32];
    unsigned long long full[PROBS_MAX_PIECES];
    int failed;
    alignas(16) unsigned char raw[1];                      // the slice, at its global address modulo 16
};

// Bytes of dynamic shared memory for a slice of `bytes`.
inline size_t probs_smem(int64_t bytes) { return offsetof(ProbsShared, raw) + static_cast<size_t>(bytes) + 32; }

// (m, s) joined with (m2, s2); empty sides have m = -inf, s = 0.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2, float c)
{
    const float top = fmaxf(m, m2);
    const float f = m == top ? 1.f : ex2((m - top) * c), f2 = m2 == top ? 1.f : ex2((m2 - top) * c);
    s = s * f + s2 * f2;
    m = top;
}

// The larger value, the lower index of equals; an empty side has v = -inf and
// index INT32_MAX.
__device__ __forceinline__ void first_max(float &v, int32_t &i, float v2, int32_t i2)
{
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(PROBS_THREADS) gdn_token_probs_kernel(const ProbsParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    ProbsShared &sh = *reinterpret_cast<ProbsShared *>(smem);
    constexpr int PI = Elem<TIn>::PER16, PO = Elem<TOut>::PER16;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int64_t row = blockIdx.x / size;

    cluster_arrive();                                      // peers' shared memory is up (waited for below)
    pdl_wait();

    // ---- which row, whose temperature.  A row left out is left out by its
    // whole cluster.
    int64_t ti = row;
    bool skip = false;
    if (p.row_seq) {
        const int32_t q = p.row_seq[row];
        ti = q;
        skip = q < 0 || q >= p.num_temps;
        if (skip && q != -1 && rank == 0 && tid == 0)
            report(p.status, GDN_DEV_BAD_SEQ);
    }
    if (skip) {
        cluster_wait();
        return;
    }

    // ---- the slice into shared memory: the 16-byte words inside it by bulk
    // copies, the ragged edges by plain loads
    const int32_t e0 = min(p.vocab, static_cast<int32_t>(rank) * p.slice);
    const int32_t n = min(p.vocab - e0, p.slice);
    const TIn *src = static_cast<const TIn *>(p.logits) + row * p.l_row + e0;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
    const uint32_t bytes = static_cast<uint32_t>(n) * sizeof(TIn);
    const uint32_t b0 = off ? 16u : 0u, b1 = (off + bytes) & ~15u;   // words inside, offsets in raw
    const uint32_t bulk = b1 > b0 ? b1 - b0 : 0u;
    const int pieces = static_cast<int>((bulk + PROBS_PIECE - 1) / PROBS_PIECE);
    if (tid == 0) {
        sh.failed = 0;
        for (int i = 0; i < pieces; ++i)
            sync::mbar_init(&sh.full[i], 1);
        sync::fence_barrier_init();
        const unsigned char *g = reinterpret_cast<const unsigned char *>(src) - off;
        for (int i = 0; i < pieces; ++i) {
            const uint32_t at = b0 + static_cast<uint32_t>(i) * PROBS_PIECE;
            const uint32_t len = min(static_cast<uint32_t>(PROBS_PIECE), b1 - at);
            sync::mbar_arrive_expect_state_tx(&sh.full[i], len);
            sync::bulk_load(sh.raw + at, g + at, len, &sh.full[i]);
        }
    }
    TIn *const el = reinterpret_cast<TIn *>(sh.raw + off);           // el[0 .. n)
    {
        const int32_t head = bulk ? static_cast<int32_t>((b0 - off) / sizeof(TIn)) : n;   // elements before the words
        const int32_t tail = bulk ? static_cast<int32_t>((b1 - off) / sizeof(TIn)) : n;   // first one behind them
        if (tid < head)
            el[tid] = src[tid];
        if (tail + tid < n)
            el[tail + tid] = src[tail + tid];
    }
    const float t = p.temperature ? p.temperature[ti * p.t_stride] : 1.f;
    const bool bad = !(t >= 0.f) || isinf(t), greedy = t == 0.f;
    // log2(e) / t, at most about 1e38 so that 0 * c is 0
    const float c = greedy || bad ? 0.f : fminf(static_cast<float>(1.4426950408889634 / static_cast<double>(t)), 1e38f);
    if (bad && rank == 0 && tid == 0)
        report(p.status, GDN_DEV_BAD_TEMPERATURE);
    __syncthreads();

    // ---- pass 1: the running (maximum, sum), or (maximum, its first index)
    float m = -INFINITY, s = 0.f;
    int32_t at_max = INT32_MAX;
    const int words = static_cast<int>((off + bytes + 15u) >> 4);
    bool ok = true;
    int have = 0;                                          // pieces known to be in
    for (int w = tid; w < words && ok; w += PROBS_THREADS) {
        const uint32_t b = static_cast<uint32_t>(w) * 16u;
        if (b >= b0 && b < b1) {
            const int piece = static_cast<int>((b - b0) / PROBS_PIECE);
            while (ok && have <= piece)
                ok = sync::mbar_wait(&sh.full[have++], 0, &sh.failed);
            if (!ok)
                break;
        }
        float x[PI];
        unpack16(*reinterpret_cast<const uint4 *>(sh.raw + b), x, static_cast<const TIn *>(nullptr));
        const int32_t first = static_cast<int32_t>(b / sizeof(TIn)) - static_cast<int32_t>(off / sizeof(TIn));
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < PI; ++j) {
            if (first + j < 0 || first + j >= n || !(x[j] == x[j]))
                x[j] = -INFINITY;                          // outside the slice, or NaN
            top = fmaxf(top, x[j]);
        }
        if (top == -INFINITY)
            continue;
        if (greedy) {
#pragma unroll
            for (int j = PI - 1; j >= 0; --j)
                if (x[j] == top && (top > m || (top == m && first + j < at_max)))
                    at_max = first + j, m = top;
        } else {
            const float to = fmaxf(m, top);
            float sum = m == to ? s : s * ex2((m - to) * c);
#pragma unroll
            for (int j = 0; j < PI; ++j)
                sum += x[j] == to ? 1.f : ex2((x[j] - to) * c);
            m = to;
            s = sum;
        }
    }
    if (!ok) {
        sh.failed = 1;
        report(p.status, GDN_DEV_TIMEOUT);
    }
    if (greedy && at_max != INT32_MAX)
        at_max += e0;

    // ---- over the warp, the CTA and the cluster.  For a greedy row the second
    // member carries the index's bits.
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(~0u, m, o), s2 = __shfl_xor_sync(~0u, s, o);
        const int32_t i2 = __shfl_xor_sync(~0u, at_max, o);
        if (greedy)
            first_max(m, at_max, m2, i2);
        else
            join(m, s, m2, s2, c);
    }
    if (lane == 0)
        sh.warp[warp] = make_float2(m, greedy ? __int_as_float(at_max) : s);
    __syncthreads();
    cluster_wait();
    if (tid < static_cast<int>(size)) {
        float2 a = sh.warp[0];
        int32_t ai = __float_as_int(a.y);
        for (int i = 1; i < PROBS_THREADS / 32; ++i) {
            const float2 b = sh.warp[i];
            if (greedy)
                first_max(a.x, ai, b.x, __float_as_int(b.y));
            else
                join(a.x, a.y, b.x, b.y, c);
        }
        st_peer(peer_addr(&sh.cta[rank], tid), a.x, greedy ? __int_as_float(ai) : a.y);
    }
    cluster_arrive();
    cluster_wait();
    float2 all = sh.cta[0];
    int32_t pick = __float_as_int(all.y);
    for (uint32_t i = 1; i < size; ++i) {
        const float2 b = sh.cta[i];
        if (greedy)
            first_max(all.x, pick, b.x, __float_as_int(b.y));
        else
            join(all.x, all.y, b.x, b.y, c);
    }
    pdl_trigger();
    const float top = all.x;
    const float inv = top == -INFINITY || bad ? 0.f : 1.f / all.y;   // masked rows: zeros

    // ---- pass 2: the probabilities, 16 bytes at a time where they are aligned
    if (!sh.failed) {
        TOut *dst = static_cast<TOut *>(p.probs) + row * p.p_row + e0;
        const int32_t o_off = static_cast<int32_t>((reinterpret_cast<uintptr_t>(dst) & 15u) / sizeof(TOut));
        const int groups = (o_off + n + PO - 1) / PO;
        auto value = [&](int32_t j) -> float {
            if (greedy)
                return top > -INFINITY && e0 + j == pick ? 1.f : 0.f;
            const float x = Elem<TIn>::get(el[j]);
            const float e = x == top ? 1.f : ex2((x - top) * c);
            return x == x && inv > 0.f ? e * inv : 0.f;
        };
        for (int g = tid; g < groups; g += PROBS_THREADS) {
            const int32_t j0 = g * PO - o_off;
            if (j0 >= 0 && j0 + PO <= n) {
                alignas(16) TOut v[PO];
#pragma unroll
                for (int j = 0; j < PO; ++j)
                    v[j] = Elem<TOut>::put(value(j0 + j));
                *reinterpret_cast<uint4 *>(dst + j0) = *reinterpret_cast<const uint4 *>(v);
            } else {
                for (int32_t j = max(j0, 0); j < min(j0 + PO, n); ++j)
                    dst[j] = Elem<TOut>::put(value(j));
            }
        }
    } else {
        // copies still in flight must land before the CTA's memory goes
        for (int i = tid; i < pieces; i += PROBS_THREADS) {
            int never = 0;
            sync::mbar_wait(&sh.full[i], 0, &never);
        }
        __syncthreads();
    }
}

}  // namespace spec
}  // namespace gdn
