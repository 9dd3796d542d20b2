// What the kernels of mla_prefill share: one call's parameters and the
// reading of the sequences' bounds.
#pragma once

#include <cstdint>

#include "mla_device.cuh"

namespace mla {

constexpr int kPrefillQk = 192;      // q and k head dim: 128 of the head's own, 64 shared
constexpr int kPrefillV = 128;       // v head dim
constexpr int kPrefillKv = 256;      // one head's [k_nope | v] of a token

struct PrefillParams {
    const uint16_t* q;        // bf16 [total_q, N, 192]
    const uint16_t* kv;       // bf16 [total_k, N, 256]
    const uint16_t* k_pe;     // bf16 [total_k, 64]
    const int32_t* cu_q;
    const int32_t* cu_k;
    int batch, heads, total_q, total_k;
    int causal;
    int splits;
    int split_rest;           // only the items of the last wave are split
    int group;                // heads that run together
    float scale_log2;
    uint16_t* out;            // bf16 [total_q, N, 128]
    float* lse;               // fp32 [total_q, N] or null
    float* o_part;            // splits > 1: fp32 rows of 128, [total_q, N, S] of them or
                              // (split_rest) [rest_parts, 256]
    float* lse_part;          //             the rows' LSEs, fp32
    int64_t* rest_rows;       // split_rest: their result rows (query * N + head), or -1
    int32_t* rest;            // split_rest: those items, and the parts of each (in the status
                              // header)
    int rest_parts;
    int32_t* status;
    unsigned long long* ticket;   // items drawn after the first of each CTA (in the status
                                  // header; 0 between calls)
    uint32_t* done;               // CTAs that have finished
};

// Rows and keys of sequence b; one whose bounds make no sense has none.
__device__ __forceinline__ void sequence(const PrefillParams& p, int b, int* q0, int* lq, int* k0,
                                         int* lk) {
    const int qa = p.cu_q[b], qe = p.cu_q[b + 1], ka = p.cu_k[b], ke = p.cu_k[b + 1];
    *q0 = qa;
    *k0 = ka;
    *lq = *lk = 0;
    if (qa < 0 || qe < qa || qe > p.total_q) {
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, qe);
        return;
    }
    *lq = qe - qa;
    if (ka < 0 || ke < ka || ke > p.total_k) {
        record_error(p.status, MLA_ERR_BAD_SEQ_LEN, ke);
        return;
    }
    *lk = ke - ka;
}

// The single-row kernel (mla_prefill_row.cu): items of one query row, one head
// and one split.
constexpr int kMaxRowSplits = 8;     // the CTAs of a cluster
int launch_prefill_row(const PrefillParams& p, int num_sms, void* stream);

}  // namespace mla
