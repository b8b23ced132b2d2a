// gdn_token_probs.cuh -- probabilities of logit rows (gdn_token_probs in
// include/gdn_spec.h).
//
// p_v = exp((l_v - m) / t) / sum_w exp((l_w - m) / t), m the row's maximum.
// A cluster takes a row at a time, rows in turn; each CTA holds a contiguous
// slice of it in shared memory (bulk copies, so HBM is read once) and passes
// over it three times: maximum (as the pieces come in), sum of 2^((l - m) c)
// with c = log2(e) / t, and the probabilities, whose powers are taken again
// rather than kept.  Each of the first two ends in one exchange over
// distributed shared memory.  What a row needs besides its logits is loaded a
// row ahead.
// Bound by HBM: each logit read once, each probability written once.  512 x
// 131072 bf16 -> fp32 in 69 us, 5.8 TB/s, 0.90 of the measured copy rate; fp32
// -> fp32 in 92 us (0.90); fp32 -> bf16 in 85 us (0.73) and bf16 -> bf16 in 59
// us (0.71: the two powers a logit and the issue slots begin to count).  A
// single row of 32768 takes 3.6 us, all of it latency.  CTAs of 512 threads,
// fewer of them resident, took 84 us; one pass with a running maximum and sum
// 116.
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
    int32_t rows;
};

constexpr int PROBS_MAX_THREADS = 256;
// Bytes per bulk copy and mbarrier.  (8 KB pieces, whose maxima overlap the
// copies of the later ones: up to 2 % slower, 512 x 131072 fp32 93.6 us against
// 92.0, one row of 131072 4.5 against 4.4.)
constexpr int PROBS_PIECE = 32768;
constexpr int PROBS_MAX_CLUSTER = 16;
constexpr int PROBS_MAX_SLICE_BYTES = GDN_SPEC_MAX_VOCAB / PROBS_MAX_CLUSTER * 4;
constexpr int PROBS_MAX_PIECES = PROBS_MAX_SLICE_BYTES / PROBS_PIECE + 2;

struct ProbsShared {
    float cta[2][PROBS_MAX_CLUSTER];                       // one value of each CTA of the cluster; exchanges alternate
    float warp[PROBS_MAX_THREADS / 32];
    float result;
    unsigned long long full[PROBS_MAX_PIECES];             // the slice's pieces
    unsigned long long got[2];                             // the peers' values
    int failed;
    alignas(16) unsigned char raw[1];                      // the slice, at its global address modulo 16
};

// Bytes of dynamic shared memory for a slice of `bytes`.
inline size_t probs_smem(int64_t bytes) { return offsetof(ProbsShared, raw) + static_cast<size_t>(bytes) + 32; }

struct Max {
    static constexpr float EMPTY = -INFINITY;
    __device__ static float of(float a, float b) { return fmaxf(a, b); }
};
struct Sum {
    static constexpr float EMPTY = 0.f;
    __device__ static float of(float a, float b) { return a + b; }
};

// Over all threads of the cluster, the same bits in each of them (the order is
// fixed).  Exchanges are numbered: a peer sends its value for number k + 2 only
// when it has this CTA's for k + 1, which is sent behind the reading of k, so
// two buffers do.  A CTA that has given up a wait (sh.failed) sends nothing
// more, so the cluster's waits run out too and no CTA goes on with values that
// lack its slice; the result is then the same in the CTA, and not used.
template <typename Op>
__device__ __forceinline__ float over_cluster(float x, ProbsShared &sh, uint32_t &number, uint32_t rank, uint32_t size)
{
    const int lane = threadIdx.x & 31, warp = warp_index();
    const uint32_t slot = number & 1u, parity = number >> 1 & 1u;
    ++number;
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = Op::of(x, __shfl_xor_sync(~0u, x, o));
    if (lane == 0)
        sh.warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const bool sends = lane < static_cast<int>(size) && !sh.failed;
        x = lane < static_cast<int>(blockDim.x >> 5) ? sh.warp[lane] : Op::EMPTY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            x = Op::of(x, __shfl_xor_sync(~0u, x, o));
        if (sends)
            st_peer(peer_addr(&sh.cta[slot][rank], lane), x, peer_addr(&sh.got[slot], lane));
        const bool in = __all_sync(~0u, mbar_wait_peers(&sh.got[slot], parity));
        x = lane < static_cast<int>(size) ? sh.cta[slot][lane] : Op::EMPTY;
#pragma unroll
        for (int o = PROBS_MAX_CLUSTER / 2; o > 0; o >>= 1)
            x = Op::of(x, __shfl_xor_sync(~0u, x, o));
        if (lane == 0) {
            sh.result = x;
            if (in)
                expect_peers(&sh.got[slot], size * sizeof(float));
            else
                sh.failed = 1;
        }
    }
    __syncthreads();
    return sh.result;
}

// 2^((x - m) c) up to a factor that is the same for the whole row.  fast:
// one fused multiply-add, x c - by, by = m c, whose rounding is that factor.
// careful: any maximum and temperature, NaN as 0; the difference times `by`,
// which is 1, or 2^64 beside a c that is smaller by as much.
struct Power {
    float c, top, by;
    __device__ float fast(float x) const { return ex2(fmaf(x, c, -by)); }
    __device__ float careful(float x) const { return x == top ? 1.f : (x == x ? ex2((x - top) * by * c) : 0.f); }
};

// This CTA's slice of one row, in shared memory from el[0] on: the 16-byte
// words inside it by bulk copies, the ragged edges (fewer than 16 bytes on
// either side) by plain loads, one element a thread.
template <typename T>
struct Slice {
    const T *src;
    T *el;
    int32_t n, head, tail;                                 // elements; those before the words, the first behind them
    uint32_t b0, b1;                                       // the words, as offsets in raw
    __device__ __forceinline__ Slice(const ProbsParams &p, ProbsShared &sh, int64_t row, int32_t e0)
    {
        src = static_cast<const T *>(p.logits) + row * p.l_row + e0;
        n = min(p.vocab - e0, p.slice);
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
        b0 = off ? 16u : 0u;
        b1 = max(b0, (off + static_cast<uint32_t>(n) * static_cast<uint32_t>(sizeof(T))) & ~15u);
        el = reinterpret_cast<T *>(sh.raw + off);
        head = b1 > b0 ? static_cast<int32_t>((b0 - off) / sizeof(T)) : n;
        tail = b1 > b0 ? static_cast<int32_t>((b1 - off) / sizeof(T)) : n;
    }
    // By one thread, once nothing reads or writes the buffer any more.  Every
    // piece's barrier completes a phase per row, bytes or not.
    __device__ __forceinline__ void fetch(ProbsShared &sh, int pieces) const
    {
        const unsigned char *g = reinterpret_cast<const unsigned char *>(src) -
                                 (reinterpret_cast<const unsigned char *>(el) - sh.raw);
        for (int i = 0; i < pieces; ++i) {
            const uint32_t at = b0 + static_cast<uint32_t>(i) * PROBS_PIECE;
            const uint32_t len = at < b1 ? min(static_cast<uint32_t>(PROBS_PIECE), b1 - at) : 0u;
            if (len) {
                expect_copy(&sh.full[i], len);
                sync::bulk_load(sh.raw + at, g + at, len, &sh.full[i]);
            } else {
                sync::mbar_arrive(&sh.full[i]);
            }
        }
    }
};

// One row's probabilities from its slice in shared memory.
template <typename TIn, typename TOut, typename Value>
__device__ __forceinline__ void write_row(const TIn *el, TOut *dst, int32_t n, Value value)
{
    constexpr int PO = Elem<TOut>::PER16;
    const int tid = threadIdx.x, threads = blockDim.x;
    const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(dst) & 15u) / sizeof(TOut));
    const int32_t first = min(n, skew ? PO - skew : 0);              // elements before the first 16-byte group
    const int groups = (n - first) / PO;
    const int32_t rest = first + groups * PO;                        // elements behind the last
    const int32_t lone = tid < first ? tid : rest + tid - first;
    if (lone < n)
        dst[lone] = Elem<TOut>::put(value(lone, Elem<TIn>::get(el[lone])));
    const TIn *const from = el + first;
    uint4 *const to = reinterpret_cast<uint4 *>(dst + first);
    auto store = [&](int g, const float (&x)[PO]) {
        alignas(16) TOut v[PO];
#pragma unroll
        for (int j = 0; j < PO; ++j)
            v[j] = Elem<TOut>::put(value(first + g * PO + j, x[j]));
        to[g] = *reinterpret_cast<const uint4 *>(v);
    };
    constexpr int GROUP_BYTES = PO * sizeof(TIn);                    // 8, 16 or 32
    if (sync::smem_addr(from) % (GROUP_BYTES < 16 ? GROUP_BYTES : 16) == 0) {
#pragma unroll 4
        for (int g = tid; g < groups; g += threads) {
            float x[PO];
            load_group(from + g * PO, x);
            store(g, x);
        }
    } else {
        for (int g = tid; g < groups; g += threads) {
            float x[PO];
#pragma unroll
            for (int j = 0; j < PO; ++j)
                x[j] = Elem<TIn>::get(from[g * PO + j]);
            store(g, x);
        }
    }
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(PROBS_MAX_THREADS, 6) gdn_token_probs_kernel(const ProbsParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    ProbsShared &sh = *reinterpret_cast<ProbsShared *>(smem);
    constexpr int PI = Elem<TIn>::PER16;
    const int tid = threadIdx.x, threads = static_cast<int>(blockDim.x);
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int32_t clusters = static_cast<int32_t>(gridDim.x / size);
    const int32_t e0 = min(p.vocab, static_cast<int32_t>(rank) * p.slice);
    const int pieces = static_cast<int>((static_cast<uint32_t>(p.slice) * sizeof(TIn) + PROBS_PIECE - 1) / PROBS_PIECE);

    if (tid == 0) {
        sh.failed = 0;
        for (int i = 0; i < pieces; ++i)
            sync::mbar_init(&sh.full[i], 1);
        for (int i = 0; i < 2; ++i) {
            sync::mbar_init(&sh.got[i], 1);
            expect_peers(&sh.got[i], size * sizeof(float));
        }
        sync::fence_barrier_init();
    }
    cluster_arrive(warp_index() == 0);
    pdl_wait();

    // A row's sequence, and whether the row is left out (by its whole cluster).
    auto seq_of = [&](int32_t row) { return p.row_seq && row < p.rows ? p.row_seq[row] : row; };
    auto left_out = [&](int32_t row, int32_t seq) { return row >= p.rows || (p.row_seq && (seq < 0 || seq >= p.num_temps)); };

    int32_t row = static_cast<int32_t>(blockIdx.x / size), seq = seq_of(row);
    cluster_wait();                                        // peers' mbarriers are there
    if (tid == 0 && !left_out(row, seq))
        Slice<TIn>(p, sh, row, e0).fetch(sh, pieces);
    uint32_t exchange = 0, loads = 0;
    bool failed = false;
    while (row < p.rows && !failed) {
        const int32_t next = row + clusters;                // (rows + clusters stay within 32 bits)
        const int32_t next_seq = seq_of(next);
        if (left_out(row, seq)) {
            if (seq != -1 && rank == 0 && tid == 0)
                report(p.status, GDN_DEV_BAD_SEQ);
        } else {
            const Slice<TIn> sl(p, sh, row, e0);
            const int32_t edge = tid < sl.head ? tid : sl.tail + tid - sl.head;   // this thread's ragged element, if < n
            const bool has_edge = edge < sl.n;
            const TIn edge_raw = has_edge ? sl.src[edge] : TIn();
            const float t = p.temperature ? p.temperature[seq * p.t_stride] : 1.f;

            // ---- the maximum (NaN is no operand of it), as the pieces come in
            const uint4 *const words = reinterpret_cast<const uint4 *>(sh.raw + sl.b0);
            const int num_words = static_cast<int>((sl.b1 - sl.b0) / 16u);
            float top = -INFINITY;
            bool ok = true;
            for (int k = 0; k < pieces && ok; ++k) {
                ok = sync::mbar_wait(&sh.full[k], loads & 1u, &sh.failed);
                if (!ok)
                    break;
                const int w1 = min(num_words, (k + 1) * (PROBS_PIECE / 16));
                for (int w = k * (PROBS_PIECE / 16) + tid; w < w1; w += threads)
                    top = fmaxf(top, max16(words[w], static_cast<const TIn *>(nullptr)));
            }
            if (!ok)
                sh.failed = 1;
            ++loads;
            const float edge_x = has_edge ? Elem<TIn>::get(edge_raw) : -INFINITY;
            if (has_edge)
                sl.el[edge] = edge_raw;
            top = over_cluster<Max>(fmaxf(top, edge_x), sh, exchange, rank, size);

            // ---- the sum of the powers, or the first index of the maximum.  The
            // fast form needs m c within 2^20, where its rounding is far below 1.
            const bool bad = !(t >= 0.f) || isinf(t), greedy = t == 0.f;
            if (bad && rank == 0 && tid == 0)
                report(p.status, GDN_DEV_BAD_TEMPERATURE);
            // log2(e) / t, infinite for t < 4.3e-39: m c is not within 2^20 then
            const float c = greedy || bad ? 0.f : 1.44269504f / t;
            Power power = {c, top, top * c};
            bool fast = !greedy && !bad && fabsf(power.by) < 1048576.f;
            const bool zeros = bad || top == -INFINITY;
            float inv = 0.f;
            int32_t pick = -1;
            if (greedy) {
                int32_t first = INT32_MAX;
                if (!zeros)
                    for (int32_t j = tid; j < sl.n; j += threads)
                        if (Elem<TIn>::get(sl.el[j]) == top) {
                            first = j;
                            break;
                        }
                // indices below 2^24 are exact in fp32
                const float g = over_cluster<Max>(first == INT32_MAX ? -INFINITY : -static_cast<float>(e0 + first), sh,
                                                  exchange, rank, size);
                pick = zeros ? -1 : static_cast<int32_t>(-g) - e0;
            } else if (!zeros) {
                if (fast) {
                    float s0 = has_edge ? power.fast(edge_x) : 0.f, s1 = 0.f;
                    for (int w = tid; w < num_words; w += threads) {
                        float x[PI];
                        unpack16(words[w], x, static_cast<const TIn *>(nullptr));
#pragma unroll
                        for (int j = 0; j < PI; j += 2) {
                            s0 += power.fast(x[j]);
                            s1 += power.fast(x[j + 1]);
                        }
                    }
                    const float s = over_cluster<Sum>(s0 + s1, sh, exchange, rank, size);
                    fast = s == s;                         // a NaN logit: again, without it
                    inv = 1.f / s;
                }
                if (!fast) {
                    const bool tiny = isinf(c);
                    power.by = tiny ? 0x1p64f : 1.f;
                    power.c = tiny ? 1.44269504f / (t * 0x1p64f) : c;
                    float s = 0.f;
                    for (int32_t j = tid; j < sl.n; j += threads)
                        s += power.careful(Elem<TIn>::get(sl.el[j]));
                    inv = 1.f / over_cluster<Sum>(s, sh, exchange, rank, size);
                }
            }
            failed = sh.failed;                            // (the same in the CTA behind an exchange)
            if (!failed) {
                TOut *const dst = static_cast<TOut *>(p.probs) + row * p.p_row + e0;
                if (zeros || greedy)
                    write_row(sl.el, dst, sl.n, [&](int32_t j, float) { return j == pick ? 1.f : 0.f; });
                else if (fast)
                    write_row(sl.el, dst, sl.n, [&](int32_t, float x) { return power.fast(x) * inv; });
                else
                    write_row(sl.el, dst, sl.n, [&](int32_t, float x) { return power.careful(x) * inv; });
                if (has_edge)
                    sync::fence_proxy_async();             // its store before the next row's bulk copies
                __syncthreads();                           // the slice is read
            }
        }
        if (tid == 0 && !failed && !left_out(next, next_seq))
            Slice<TIn>(p, sh, next, e0).fetch(sh, pieces);
        row = next;
        seq = next_seq;
    }
    if (failed) {
        // copies still in flight must land before the CTA's memory goes
        if (tid == 0)
            report(p.status, GDN_DEV_TIMEOUT);
        for (int i = tid; i < pieces; i += threads) {
            int never = 0;
            sync::mbar_wait(&sh.full[i], (loads - 1u) & 1u, &never);
        }
        cluster_leave();
    }
}

}  // namespace spec
}  // namespace gdn
