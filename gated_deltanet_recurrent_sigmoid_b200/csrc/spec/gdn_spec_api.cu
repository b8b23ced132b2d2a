// gdn_spec_api.cu -- host side of the C ABI declared in include/gdn_spec.h:
// argument validation, parameter marshalling and the kernel launches.  Every
// check runs before anything is enqueued and none of them touches device
// memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "gdn_commit_states.cuh"
#include "gdn_host_checks.cuh"
#include "gdn_spec.h"
#include "gdn_step_maps.cuh"
#include "gdn_token_probs.cuh"
#include "gdn_verify_drafts.cuh"

namespace {

using namespace gdn::host;

constexpr int64_t kState = 128;            // K = V

int check_call(uint32_t flags, const gdn_extra *x)
{
    if (flags & ~(GDN_LAUNCH_PDL | GDN_SPEC_CHECK_ONLY))
        return GDN_ERR_ARG;
    if (!x)
        return GDN_OK;
    if (x->intermediate_states || x->tile_v || x->tile_rows || x->schedule || x->reserved || x->workspace ||
        x->workspace_bytes)
        return GDN_ERR_ARG;
    return aligned(x->device_status, 4) ? GDN_OK : GDN_ERR_ALIGN;
}

Span span_of_status(const gdn_extra *x)
{
    Span s;
    if (x && x->device_status) {
        s.lo = reinterpret_cast<uintptr_t>(x->device_status);
        s.hi = s.lo + sizeof(uint32_t);
    }
    return s;
}

// No written tensor may overlap another tensor or the status word.
int check_alias(std::initializer_list<const gdn_tensor *> written, std::initializer_list<const gdn_tensor *> read,
                const gdn_extra *x)
{
    const Span status = span_of_status(x);
    for (const gdn_tensor *const *w = written.begin(); w != written.end(); ++w) {
        const Span s = span_of(*w);
        if (overlap(s, status))
            return GDN_ERR_ALIAS;
        for (const gdn_tensor *r : read)
            if (overlap(s, span_of(r)))
                return GDN_ERR_ALIAS;
        for (const gdn_tensor *const *v = w + 1; v != written.end(); ++v)
            if (overlap(s, span_of(*v)))
                return GDN_ERR_ALIAS;
    }
    for (const gdn_tensor *r : read)
        if (overlap(status, span_of(r)))
            return GDN_ERR_ALIAS;
    return GDN_OK;
}

// A contiguous int32 vector of n entries (n < 0: of any length).
int check_vector(const gdn_tensor *t, int64_t n, int32_t dtype = GDN_DTYPE_I32)
{
    GDN_TRY(check_desc(t, dtype));
    if (t->ndim != 1 || (n >= 0 && t->shape[0] != n) || t->shape[0] > INT32_MAX)
        return GDN_ERR_SHAPE;
    if (t->shape[0] > 1 && t->stride[0] != 1)
        return GDN_ERR_SHAPE;
    return aligned(t->data, elem_size(dtype)) ? GDN_OK : GDN_ERR_ALIGN;
}

// Rows of a written matrix must not run into each other.
bool rows_apart(const gdn_tensor *t) { return t->shape[0] <= 1 || t->stride[0] >= t->shape[1]; }

// Whether runs of `unit` elements that begin at i * s0 + j * s1 (i < n0, j < n1)
// lie apart: either index's entries inside one step of the other's.
bool items_apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t unit)
{
    if ((n0 > 1 && s0 < unit) || (n1 > 1 && s1 < unit))
        return false;
    return n0 <= 1 || n1 <= 1 || s0 >= (n1 - 1) * s1 + unit || s1 >= (n0 - 1) * s0 + unit;
}

cudaStream_t stream_of(const gdn_extra *x) { return x ? static_cast<cudaStream_t>(x->stream) : nullptr; }
uint32_t *status_of(const gdn_extra *x) { return x ? x->device_status : nullptr; }

// A launch of thread-block clusters with programmatic stream serialization.
struct ClusterLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int64_t ctas, int cluster, int threads, size_t smem, cudaStream_t stream)
    {
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    ClusterLaunch(const ClusterLaunch &) = delete;
};

template <typename Kernel, typename Params>
cudaError_t launch_cluster(Kernel kernel, int64_t ctas, int cluster, int threads, size_t smem, cudaStream_t stream,
                           const Params &p)
{
    const ClusterLaunch launch(ctas, cluster, threads, smem, stream);
    return cudaLaunchKernelEx(&launch.cfg, kernel, p);
}

int status_from(cudaError_t err) { return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

template <typename TIn, typename TOut>
cudaError_t launch_probs(const gdn::spec::ProbsParams &p, int64_t rows, int cluster, int threads, size_t smem,
                         cudaStream_t stream)
{
    static PerDevice once;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = once_per_device(once, dev, [&]() {
            const auto kernel = gdn::spec::gdn_token_probs_kernel<TIn, TOut>;
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(gdn::spec::probs_smem(gdn::spec::PROBS_MAX_SLICE_BYTES)));
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            return e;
        });
    // The clusters that fit the GPU at once, for the last launch shape asked
    // for on each device: shape in the upper half, clusters in the lower.
    static std::atomic<uint64_t> resident[PerDevice::kMaxDevices];
    // (18 bits of shared memory, 5 of the cluster, 6 of the warps)
    const uint64_t shape = static_cast<uint64_t>(smem) << 11 | static_cast<uint64_t>(cluster) << 6 | threads / 32;
    uint64_t known = err == cudaSuccess ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (err == cudaSuccess && known >> 32 != shape) {
        int clusters = 0;
        ClusterLaunch probe(cluster, cluster, threads, smem, nullptr);
        err = cudaOccupancyMaxActiveClusters(&clusters, gdn::spec::gdn_token_probs_kernel<TIn, TOut>, &probe.cfg);
        known = shape << 32 | static_cast<uint64_t>(clusters > 0 ? clusters : 1);
        if (err == cudaSuccess)
            resident[dev].store(known, std::memory_order_relaxed);
    }
    if (err != cudaSuccess)
        return err;
    // as few clusters as do the rows in the same number of turns
    const int64_t most = static_cast<int64_t>(known & 0xffffffffu), turns = (rows + most - 1) / most;
    const int64_t clusters = (rows + turns - 1) / turns;
    return launch_cluster(gdn::spec::gdn_token_probs_kernel<TIn, TOut>, clusters * cluster, cluster, threads, smem,
                          stream, p);
}

// CTAs per row of token probabilities: slices of at most 16 KB as far as 8 CTAs
// give them, and more CTAs while the grid leaves SMs idle and a slice keeps 512
// elements.  Measured for 512 rows bf16 -> fp32: 4096 logits in 1 CTA 5.8 us, in
// 4 8.5; 32768 in 1 28.8, in 4 22.0, in 8 25.2; 50021 fp32 in 4 43.5, in 8 41.0.
// 16 CTAs where 8 would leave a slice over 55 KB, of which an SM holds fewer than
// four, or SMs idle.  512 rows in 8 and in 16, fp32: 66000 logits 45.8 us and
// 65.0, 110000 74.8 and 81.9, 114688 87.1 and 84.0, 131072 94.4 and 91.5; bf16
// -> fp32: 140000 77.9 and 89.7, 225000 120.2 and 125.5, 229376 128.4 and 126.9;
// one row of 131072 bf16 5.3 and 4.4.  (40 rows of bf16, 131072 to 220000, are 5
// to 8 % faster in 16, of fp32 up to 8 % slower.)
int probs_cluster(int64_t rows, int64_t row_bytes, int64_t vocab, int sms)
{
    int c = 1;
    while (c < 8 && (row_bytes > c * 16384ll || (rows * c < sms && vocab > c * 1024ll)))
        c *= 2;
    if (c == 8 && (row_bytes > 8 * 56320ll || (rows * 16 <= sms && vocab > 16 * 1024ll)))
        c = 16;
    return c;
}

// CTAs per sequence of a verification: as many (up to 8) as stay resident at
// once, eight of 128 threads an SM, while a CTA keeps 512 elements.
int verify_cluster(int64_t sequences, int64_t vocab, int sms)
{
    int c = 1;
    while (c < 8 && sequences * c * 2 <= 8ll * sms && vocab > c * 1024ll)
        c *= 2;
    return c;
}

}  // namespace

extern "C" {

GDN_API int gdn_spec_version(void) { return GDN_SPEC_ABI_VERSION; }

GDN_API int gdn_token_probs(const gdn_tensor *logits, const gdn_tensor *temperature, const gdn_tensor *row_seq,
                            const gdn_tensor *probs, uint32_t flags, const gdn_extra *extra)
{
    GDN_TRY(check_call(flags, extra));
    GDN_TRY(check_desc(logits, GDN_DTYPE_BF16, GDN_DTYPE_F32));
    GDN_TRY(check_desc(probs, GDN_DTYPE_BF16, GDN_DTYPE_F32));
    if (logits->ndim != 2 || probs->ndim != 2 || logits->shape[0] != probs->shape[0] ||
        logits->shape[1] != probs->shape[1])
        return GDN_ERR_SHAPE;
    const int64_t R = logits->shape[0], vocab = logits->shape[1];
    if (R > INT32_MAX || vocab < 1)
        return GDN_ERR_SHAPE;
    if (vocab > 1 && (logits->stride[1] != 1 || probs->stride[1] != 1))
        return GDN_ERR_SHAPE;
    if (!rows_apart(probs))
        return GDN_ERR_SHAPE;
    if (row_seq && !temperature)
        return GDN_ERR_NULL_ARG;
    if (temperature) {
        GDN_TRY(check_desc(temperature, GDN_DTYPE_F32));
        if (temperature->ndim != 1 || temperature->shape[0] > INT32_MAX || (!row_seq && temperature->shape[0] != R))
            return GDN_ERR_SHAPE;
        if (!aligned(temperature->data, 4))
            return GDN_ERR_ALIGN;
    }
    if (row_seq)
        GDN_TRY(check_vector(row_seq, R));
    if (!aligned(logits->data, elem_size(logits->dtype)) || !aligned(probs->data, elem_size(probs->dtype)))
        return GDN_ERR_ALIGN;
    GDN_TRY(check_alias({probs}, {logits, temperature, row_seq}, extra));
    if (vocab > GDN_SPEC_MAX_VOCAB)
        return GDN_ERR_UNSUPPORTED;
    if (R * gdn::spec::PROBS_MAX_CLUSTER > INT32_MAX)
        return GDN_ERR_SHAPE;
    if ((flags & GDN_SPEC_CHECK_ONLY) || R == 0)
        return GDN_OK;

    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess)
        return GDN_ERR_CUDA;
    gdn::spec::ProbsParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = logits->data;
    p.probs = probs->data;
    p.temperature = temperature ? static_cast<const float *>(temperature->data) : nullptr;
    p.row_seq = row_seq ? static_cast<const int32_t *>(row_seq->data) : nullptr;
    p.status = status_of(extra);
    p.l_row = logits->stride[0];
    p.p_row = probs->stride[0];
    p.t_stride = temperature ? temperature->stride[0] : 0;
    p.vocab = static_cast<int32_t>(vocab);
    p.rows = static_cast<int32_t>(R);
    p.num_temps = temperature ? static_cast<int32_t>(temperature->shape[0]) : 0;
    const int cluster = probs_cluster(R, vocab * elem_size(logits->dtype), vocab, sms);
    p.slice = static_cast<int32_t>(((vocab + cluster - 1) / cluster + 7) / 8 * 8);
    // (128 threads a CTA: 512 x 32768 bf16 in 22.0 us against 23.7; 256: 512 x
    // 131072 in 69.7 against 72.7, 180 x 50021 fp32 in 19.0 against 21.2)
    const int64_t slice_bytes = p.slice * elem_size(logits->dtype);
    const int threads = slice_bytes > 16384 || (R * cluster <= sms && slice_bytes > 4096) ? gdn::spec::PROBS_MAX_THREADS : 128;
    const size_t smem = gdn::spec::probs_smem(slice_bytes);
    const cudaStream_t stream = stream_of(extra);
    const bool in16 = logits->dtype == GDN_DTYPE_BF16, out16 = probs->dtype == GDN_DTYPE_BF16;
    using bf16 = __nv_bfloat16;
    return status_from(in16 ? (out16 ? launch_probs<bf16, bf16>(p, R, cluster, threads, smem, stream)
                                     : launch_probs<bf16, float>(p, R, cluster, threads, smem, stream))
                            : (out16 ? launch_probs<float, bf16>(p, R, cluster, threads, smem, stream)
                                     : launch_probs<float, float>(p, R, cluster, threads, smem, stream)));
}

GDN_API int gdn_verify_drafts(const gdn_tensor *target_probs, const gdn_tensor *draft_tokens,
                              const gdn_tensor *draft_probs, const gdn_tensor *uniforms,
                              const gdn_tensor *cu_seqlens, const gdn_tensor *state_indices,
                              const gdn_tensor *out_tokens, const gdn_tensor *num_tokens, uint32_t flags,
                              const gdn_extra *extra)
{
    GDN_TRY(check_call(flags, extra));
    GDN_TRY(check_desc(target_probs, GDN_DTYPE_BF16, GDN_DTYPE_F32));
    GDN_TRY(check_desc(draft_tokens, GDN_DTYPE_I32));
    if (draft_probs)
        GDN_TRY(check_desc(draft_probs, target_probs->dtype));
    GDN_TRY(check_desc(uniforms, GDN_DTYPE_F32));
    GDN_TRY(check_desc(out_tokens, GDN_DTYPE_I32));
    GDN_TRY(check_desc(num_tokens, GDN_DTYPE_I32));
    if (draft_tokens->ndim != 2 || uniforms->ndim != 2 || out_tokens->ndim != 2 || num_tokens->ndim != 1)
        return GDN_ERR_SHAPE;
    const int64_t N = draft_tokens->shape[0], D = draft_tokens->shape[1];
    if (N > INT32_MAX / 8 || D > INT32_MAX / 2)
        return GDN_ERR_SHAPE;
    if (uniforms->shape[0] != N || uniforms->shape[1] != D + 1 || out_tokens->shape[0] != N ||
        out_tokens->shape[1] != D + 1 || num_tokens->shape[0] != N)
        return GDN_ERR_SHAPE;
    const bool varlen = cu_seqlens != nullptr;
    if (varlen)
        GDN_TRY(check_vector(cu_seqlens, N + 1));
    if (state_indices)
        GDN_TRY(check_vector(state_indices, N));
    TokenLayout L;
    GDN_TRY(token_layout(target_probs, 1, varlen, N, &L));
    const int64_t vocab = target_probs->shape[target_probs->ndim - 1];
    if (vocab < 1 || vocab > INT32_MAX - 4096 || L.T_tot > INT32_MAX || L.T > D + 1)
        return GDN_ERR_SHAPE;
    if (draft_probs && (draft_probs->ndim != 3 || draft_probs->shape[0] != N || draft_probs->shape[1] != D ||
                        draft_probs->shape[2] != vocab))
        return GDN_ERR_SHAPE;
    if (vocab > 1 && (target_probs->stride[target_probs->ndim - 1] != 1 || (draft_probs && draft_probs->stride[2] != 1)))
        return GDN_ERR_SHAPE;
    // written entries must not share an address
    if (!items_apart(N, out_tokens->stride[0], D + 1, out_tokens->stride[1], 1) || (N > 1 && num_tokens->stride[0] < 1))
        return GDN_ERR_SHAPE;
    for (const gdn_tensor *t : {target_probs, draft_tokens, draft_probs, uniforms, out_tokens, num_tokens})
        if (t && !aligned(t->data, elem_size(t->dtype)))
            return GDN_ERR_ALIGN;
    GDN_TRY(check_alias({out_tokens, num_tokens},
                        {target_probs, draft_tokens, draft_probs, uniforms, cu_seqlens, state_indices}, extra));
    if ((flags & GDN_SPEC_CHECK_ONLY) || N == 0)
        return GDN_OK;

    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess)
        return GDN_ERR_CUDA;
    gdn::spec::VerifyParams p;
    std::memset(&p, 0, sizeof p);
    p.target = target_probs->data;
    p.draft = draft_probs && D > 0 ? draft_probs->data : nullptr;
    p.tokens = static_cast<const int32_t *>(draft_tokens->data);
    p.uniforms = static_cast<const float *>(uniforms->data);
    p.cu_seqlens = varlen ? static_cast<const int32_t *>(cu_seqlens->data) : nullptr;
    p.indices = state_indices ? static_cast<const int32_t *>(state_indices->data) : nullptr;
    p.out = static_cast<int32_t *>(out_tokens->data);
    p.num = static_cast<int32_t *>(num_tokens->data);
    p.status = status_of(extra);
    p.t_row = L.tok;
    p.x_seq = draft_tokens->stride[0];
    p.x_pos = draft_tokens->stride[1];
    p.d_seq = draft_probs ? draft_probs->stride[0] : 0;
    p.d_pos = draft_probs ? draft_probs->stride[1] : 0;
    p.u_seq = uniforms->stride[0];
    p.u_pos = uniforms->stride[1];
    p.o_seq = out_tokens->stride[0];
    p.o_pos = out_tokens->stride[1];
    p.n_seq = num_tokens->stride[0];
    p.N = static_cast<int32_t>(N);
    p.D = static_cast<int32_t>(D);
    p.T_fixed = varlen ? 0 : static_cast<int32_t>(L.T);
    p.T_tot = static_cast<int32_t>(L.T_tot);
    p.vocab = static_cast<int32_t>(vocab);
    const int cluster = verify_cluster(N, vocab, sms);
    // 256 threads where the CTAs have an SM each and their lanes a batch of loads
    const int threads = N * cluster <= sms && vocab > cluster * 8192ll ? 256 : 128;
    const int64_t segs = static_cast<int64_t>(cluster) * (threads / 32);
    const int64_t warp_words = 32 * 16 / elem_size(target_probs->dtype);
    const int64_t skewed = aligned(target_probs->data, 16) && stride_ok(L.T_tot, L.tok, warp_words / 32) ? 0 : 7;
    p.seg = static_cast<int32_t>(((vocab + skewed + segs - 1) / segs + warp_words - 1) / warp_words * warp_words);
    const cudaStream_t stream = stream_of(extra);
    return status_from(target_probs->dtype == GDN_DTYPE_BF16
                           ? launch_cluster(gdn::spec::gdn_verify_drafts_kernel<__nv_bfloat16>, N * cluster, cluster,
                                            threads, 0, stream, p)
                           : launch_cluster(gdn::spec::gdn_verify_drafts_kernel<float>, N * cluster, cluster,
                                            threads, 0, stream, p));
}

GDN_API int gdn_commit_states(const gdn_tensor *intermediate_states, const gdn_tensor *num_tokens,
                              const gdn_tensor *state_pool, const gdn_tensor *state_indices,
                              const gdn_tensor *cu_seqlens, uint32_t flags, const gdn_extra *extra)
{
    GDN_TRY(check_call(flags, extra));
    GDN_TRY(check_desc(intermediate_states, GDN_DTYPE_F32));
    GDN_TRY(check_desc(state_pool, GDN_DTYPE_F32));
    GDN_TRY(check_vector(state_indices, -1));
    const int64_t N = state_indices->shape[0];
    GDN_TRY(check_vector(num_tokens, N));
    if (cu_seqlens)
        GDN_TRY(check_vector(cu_seqlens, N + 1));
    const gdn_tensor *in = intermediate_states, *pool = state_pool;
    if (in->ndim != 4 || pool->ndim != 4 || in->shape[1] != pool->shape[1])
        return GDN_ERR_SHAPE;
    const int64_t T_tot = in->shape[0], HV = in->shape[1], slots = pool->shape[0];
    if (HV < 1 || HV > INT32_MAX || T_tot > INT32_MAX || slots > INT32_MAX)
        return GDN_ERR_SHAPE;
    if (!cu_seqlens && N > 0 && T_tot % N != 0)
        return GDN_ERR_SHAPE;
    for (const gdn_tensor *t : {in, pool}) {
        if (t->shape[2] != kState || t->shape[3] != kState)
            return GDN_ERR_UNSUPPORTED;
        if (t->stride[3] != 1 || t->stride[2] != kState)
            return GDN_ERR_SHAPE;
        if (!aligned(t->data, 16) || !stride_ok(t->shape[0], t->stride[0], 4) || !stride_ok(HV, t->stride[1], 4))
            return GDN_ERR_ALIGN;
    }
    // states of the pool must not share addresses
    if (!items_apart(slots, pool->stride[0], HV, pool->stride[1], kState * kState))
        return GDN_ERR_SHAPE;
    GDN_TRY(check_alias({pool}, {in, num_tokens, state_indices, cu_seqlens}, extra));
    if (N * HV > INT32_MAX / gdn::spec::COMMIT_PIECES)
        return GDN_ERR_SHAPE;
    if ((flags & GDN_SPEC_CHECK_ONLY) || N == 0 || T_tot == 0)
        return GDN_OK;

    gdn::spec::CommitParams p;
    std::memset(&p, 0, sizeof p);
    p.inter = static_cast<const float *>(in->data);
    p.pool = static_cast<float *>(pool->data);
    p.num = static_cast<const int32_t *>(num_tokens->data);
    p.indices = static_cast<const int32_t *>(state_indices->data);
    p.cu_seqlens = cu_seqlens ? static_cast<const int32_t *>(cu_seqlens->data) : nullptr;
    p.status = status_of(extra);
    p.i_tok = in->stride[0];
    p.i_head = in->stride[1];
    p.s_slot = pool->stride[0];
    p.s_head = pool->stride[1];
    p.N = static_cast<int32_t>(N);
    p.HV = static_cast<int32_t>(HV);
    p.T_fixed = cu_seqlens ? 0 : static_cast<int32_t>(T_tot / N);
    p.T_tot = static_cast<int32_t>(T_tot);
    p.num_slots = static_cast<int32_t>(slots);
    return status_from(launch_ex(gdn::spec::gdn_commit_states_kernel,
                                 dim3(static_cast<unsigned>(N * HV * gdn::spec::COMMIT_PIECES)),
                                 dim3(gdn::spec::COMMIT_THREADS), 0, stream_of(extra),
                                 true, p));
}

GDN_API int gdn_step_maps(const gdn_step_maps_call *c)
{
    if (!c)
        return GDN_ERR_NULL_ARG;
    GDN_TRY(check_call(c->flags, c->extra));
    GDN_TRY(check_vector(c->lengths, -1));
    const int64_t N = c->lengths->shape[0];
    if (N > INT32_MAX - 4 * gdn::spec::MAPS_THREADS)       // requests are counted in 32 bits, so many at a time
        return GDN_ERR_SHAPE;
    GDN_TRY(check_vector(c->context, N));
    GDN_TRY(check_vector(c->slots, N));
    GDN_TRY(check_vector(c->cu_seqlens, N + 1));
    GDN_TRY(check_vector(c->state_indices, N));
    GDN_TRY(check_vector(c->row_seq, -1));
    const int64_t C = c->row_seq->shape[0];
    GDN_TRY(check_vector(c->positions, C));
    const gdn_tensor *cache[] = {c->block_tables, c->blocks_held, c->free_blocks, c->free_head,
                                 c->blocks_held_out, c->free_head_out, c->slot_map};
    int given = 0;
    for (const gdn_tensor *t : cache)
        given += t != nullptr;
    if (given != 0 && given != 7)
        return GDN_ERR_NULL_ARG;
    if (given ? c->block_size < 1 : c->block_size != 0)
        return GDN_ERR_ARG;
    if (given) {
        GDN_TRY(check_desc(c->block_tables, GDN_DTYPE_I32));
        const gdn_tensor *b = c->block_tables;
        if (b->ndim != 2 || b->shape[0] != N || b->shape[1] > INT32_MAX || (b->shape[1] > 1 && b->stride[1] != 1) ||
            !rows_apart(b))
            return GDN_ERR_SHAPE;
        if (!aligned(b->data, 4))
            return GDN_ERR_ALIGN;
        GDN_TRY(check_vector(c->blocks_held, N));
        GDN_TRY(check_vector(c->free_blocks, -1));
        GDN_TRY(check_vector(c->free_head, 1));
        GDN_TRY(check_vector(c->blocks_held_out, N));
        GDN_TRY(check_vector(c->free_head_out, 1));
        GDN_TRY(check_vector(c->slot_map, C, GDN_DTYPE_I64));
    }
    GDN_TRY(check_alias({c->cu_seqlens, c->state_indices, c->row_seq, c->positions, c->block_tables,
                         c->blocks_held_out, c->free_head_out, c->slot_map},
                        {c->lengths, c->context, c->slots, c->blocks_held, c->free_blocks, c->free_head}, c->extra));
    if (c->flags & GDN_SPEC_CHECK_ONLY)
        return GDN_OK;

    gdn::spec::MapsParams p;
    std::memset(&p, 0, sizeof p);
    auto ints = [](const gdn_tensor *t) { return t ? static_cast<int32_t *>(t->data) : nullptr; };
    p.lengths = ints(c->lengths);
    p.context = ints(c->context);
    p.slots = ints(c->slots);
    p.cu_seqlens = ints(c->cu_seqlens);
    p.state_indices = ints(c->state_indices);
    p.row_seq = ints(c->row_seq);
    p.positions = ints(c->positions);
    p.tables = ints(c->block_tables);
    p.blocked = given != 0;
    p.held = ints(c->blocks_held);
    p.free_blocks = ints(c->free_blocks);
    p.free_head = ints(c->free_head);
    p.held_out = ints(c->blocks_held_out);
    p.free_head_out = ints(c->free_head_out);
    p.slot_map = c->slot_map ? static_cast<int64_t *>(c->slot_map->data) : nullptr;
    p.status = status_of(c->extra);
    p.b_row = c->block_tables ? c->block_tables->stride[0] : 0;
    p.N = static_cast<int32_t>(N);
    p.C = static_cast<int32_t>(C);
    p.B = c->block_tables ? static_cast<int32_t>(c->block_tables->shape[1]) : 0;
    p.F = c->free_blocks ? static_cast<int32_t>(c->free_blocks->shape[0]) : 0;
    p.block_size = gdn::spec::Divisor::of(static_cast<uint32_t>(given ? c->block_size : 1));
    // one request or row a thread where there are few
    const bool many_requests = N > gdn::spec::MAPS_THREADS, many_rows = many_requests || C > 65536;
    const auto kernel = many_requests ? gdn::spec::gdn_step_maps_kernel<4, 4>
                        : many_rows   ? gdn::spec::gdn_step_maps_kernel<1, 4>
                                      : gdn::spec::gdn_step_maps_kernel<1, 1>;
    const int64_t tile = gdn::spec::MAPS_THREADS * (many_rows ? 4 : 1), tiles = (C + tile - 1) / tile;
    return status_from(launch_ex(kernel, dim3(static_cast<unsigned>(tiles > 0 ? tiles : 1)),
                                 dim3(gdn::spec::MAPS_THREADS), 0, stream_of(c->extra), true, p));
}

}  // extern "C"
