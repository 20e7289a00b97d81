// What the two attention kernels over the paged cache share.
#pragma once

#include "kvq_paged.cuh"

namespace kvq {

constexpr float kPShift = 12.0f;  // P is held as e^(x - max) 2^12 ...
constexpr float kPRoom = 15.0f;   // ... and may grow to 2^15 before the maximum is moved
constexpr float kLn2 = 0.69314718055994531f;

struct AttnArgs {
    kvq_paged_cfg c;
    const uint8_t* pool;
    int32_t* status;
    const uint16_t* q;
    int64_t qs;
    const int32_t *cu, *len, *table;
    uint16_t* out;
    float *lse, *part;
    float2* pml;
    int4* rec;        // few-row kernel: what k_paged_join has to join, or NULL
    bool by_request;  // a record per (request, kv head), else per block
    int32_t total_q, max_q, max_len, window;
    int32_t S;         // splits (chunk kernel, of the units behind the whole ones); blocks of a cluster
    int32_t whole;     // chunk kernel: units that one block does alone
    int32_t B, nrb;    // chunk kernel: requests, row blocks of a (request, kv head)
    int64_t part_rows; // chunk kernel: rows of a split's parts: those of the split units, or all of q's
    bool by_unit;      // (the former, else the latter)
    float scale_log2, out_scale;
};

// The rows and tokens of a (request, row block), the same in the main kernel and the merge.
struct Rows {
    int c0, n, nq, R, len, kv;
};
__device__ __forceinline__ Rows rows_of(const AttnArgs& a, int b) {
    Rows r;
    r.c0 = a.cu ? min(max(a.cu[b], 0), a.total_q) : b;
    r.n = a.cu ? min(max(a.cu[b + 1] - a.cu[b], 0), a.total_q - r.c0) : 1;
    r.nq = min(r.n, a.max_q);
    r.R = r.nq * (a.c.Hq / a.c.Hkv);
    r.len = max(a.len[b], 0);
    r.kv = min(min(r.len, a.max_len), a.c.max_pages * a.c.page_tokens);
    return r;
}

// The first token that a query at position p sees (p - window may pass 32 bits, p being negative).
__device__ __forceinline__ int first_seen(const AttnArgs& a, int p) {
    return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

// Chunk kernel and merge: unit u is row block rb of (b, h), the row blocks that see most first.
struct Unit {
    int rb, b, h;
};
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int u) {
    const int seg = u % (a.B * a.c.Hkv);
    return {a.nrb - 1 - u / (a.B * a.c.Hkv), seg / a.c.Hkv, seg % a.c.Hkv};
}

// Chunk kernel and merge: where split s keeps its part of row r (of the unit) = grow (of q), unit
// being the `cut`-th of those that are split.
constexpr int kUnitRows = 256;
__device__ __forceinline__ int64_t part_at(const AttnArgs& a, int s, int cut, int r, int64_t grow) {
    return s * a.part_rows + (a.by_unit ? (int64_t)cut * kUnitRows + r : grow);
}

template <bool BF>
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack16<BF>(a, b), pack16<BF>(c, d));
}

}  // namespace kvq

namespace kvq_host {
// Prompt chunks (kvq_paged_chunk.cu): query rows of a block, and the launch.
constexpr int kChunkRows = kvq::kUnitRows;
int run_chunk(const kvq::AttnArgs& a, cudaStream_t stream);
}  // namespace kvq_host
