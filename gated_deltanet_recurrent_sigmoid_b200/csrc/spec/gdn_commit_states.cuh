// gdn_commit_states.cuh -- the state after each sequence's last kept token into
// its slot of the pool (gdn_commit_states in include/gdn_spec.h).
//
// A copy of K V fp32 values per (sequence, head): bound by HBM, each byte read
// once and written once.  128 sequences x 8 heads in 22.6 us (5.9 TB/s, 0.92 of
// the measured copy rate), 486 x 8 in 80 us (0.99).  CTAs of 8 KB; 4, 16 and 32
// KB are within 2 % (a few states want the smaller ones: 4 x 4 in 1.6 us against
// 2.1 with 32 KB).
#pragma once

#include "gdn_spec_common.cuh"

namespace gdn {
namespace spec {

struct CommitParams {
    const float *inter;
    float *pool;
    const int32_t *num, *indices, *cu_seqlens;
    uint32_t *status;
    int64_t i_tok, i_head, s_slot, s_head;
    int32_t N, HV, T_fixed, T_tot, num_slots;
};

constexpr int COMMIT_THREADS = 256;
constexpr int COMMIT_VECS = 2;                                     // 16-byte words a thread
constexpr int COMMIT_PIECES = 128 * 128 / 4 / (COMMIT_THREADS * COMMIT_VECS);

__global__ void __launch_bounds__(COMMIT_THREADS) gdn_commit_states_kernel(const CommitParams a)
{
    pdl_wait();
    const int32_t unit = blockIdx.x / COMMIT_PIECES, piece = blockIdx.x % COMMIT_PIECES;
    const int32_t i = unit / a.HV, hv = unit % a.HV;
    const int32_t slot = a.indices[i], n = a.num[i];
    int32_t start, len;
    const bool rows = rows_of(a.cu_seqlens, a.T_fixed, a.T_tot, i, &start, &len);
    if (slot == -1)
        return;
    const uint32_t bad = (slot < -1 || slot >= a.num_slots ? GDN_DEV_BAD_SLOT : 0u) |
                         (!rows ? GDN_DEV_BAD_SEQLENS : 0u) | (rows && (n < 0 || n > len) ? GDN_DEV_BAD_COUNT : 0u);
    if (bad) {
        if (hv == 0 && piece == 0 && threadIdx.x == 0)
            report(a.status, bad);
        return;
    }
    if (n == 0)
        return;
    const float4 *src = reinterpret_cast<const float4 *>(a.inter + (static_cast<int64_t>(start) + n - 1) * a.i_tok +
                                                         hv * a.i_head);
    float4 *dst = reinterpret_cast<float4 *>(a.pool + slot * a.s_slot + hv * a.s_head);
    const int at = piece * COMMIT_THREADS * COMMIT_VECS + threadIdx.x;
    float4 v[COMMIT_VECS];
#pragma unroll
    for (int k = 0; k < COMMIT_VECS; ++k)
        v[k] = __ldcs(src + at + k * COMMIT_THREADS);
#pragma unroll
    for (int k = 0; k < COMMIT_VECS; ++k)
        __stcs(dst + at + k * COMMIT_THREADS, v[k]);
}

}  // namespace spec
}  // namespace gdn
