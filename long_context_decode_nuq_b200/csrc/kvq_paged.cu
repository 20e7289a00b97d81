// Paged 4-bit cache: page plan, release, append and read-back.
#include "kvq_paged.cuh"

using namespace kvq;
using namespace kvq_host;

namespace kvq_host {

int check_paged_cfg(const kvq_paged_cfg* c) {
    if (!c) return KVQ_ERR_NULL;
    if (c->D != 64 && c->D != 128) return KVQ_ERR_UNSUPPORTED;
    if (c->dtype != KVQ_F16 && c->dtype != KVQ_BF16) return KVQ_ERR_UNSUPPORTED;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 &&
        c->page_tokens != 128)
        return KVQ_ERR_UNSUPPORTED;
    if (c->Hkv < 1 || c->Hkv > 1024) return KVQ_ERR_SHAPE;
    if (c->Hq < c->Hkv || c->Hq % c->Hkv != 0 || c->Hq / c->Hkv > 64) return KVQ_ERR_SHAPE;
    if (c->num_pages < 1 || c->max_pages < 1) return KVQ_ERR_SHAPE;
    if ((int64_t)c->num_pages * c->page_tokens > INT32_MAX) return KVQ_ERR_SHAPE;
    if ((int64_t)c->max_pages * c->page_tokens > INT32_MAX) return KVQ_ERR_SHAPE;
    if (c->k_exp < -64 || c->k_exp > 64 || c->v_exp < -64 || c->v_exp > 64) return KVQ_ERR_RANGE;
    return KVQ_OK;
}

int check_paged_cache(const kvq_paged_cache* c) {
    if (!c || !c->pool || !c->status) return KVQ_ERR_NULL;
    if (!aligned16(c->pool)) return KVQ_ERR_ALIGN;
    return KVQ_OK;
}

}  // namespace kvq_host

namespace {

// ---------------------------------------------------------------------------------
// Page plan.  One cluster walks the requests in chunks of a block: prefix sums of new tokens and
// of lacking pages (every block of the cluster computes all of them, which costs less than
// passing them on), then the chunk's tokens and new pages are spread over all threads, each
// finding its request by bisection of the sums in shared memory.  A new page's number is taken
// from the free list, never from the table entry just written, so no thread waits for another.
// Latency bound; one launch.
struct PlanArgs {
    const int32_t *len, *n_new, *free_pages, *n_free;
    int32_t *table, *cu, *len_out, *n_free_out, *slots, *pos, *status;
    int32_t B, P, num_pages, max_pages, capacity;
};

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Inclusive prefix sums of a and b over the block; the totals in *ta, *tb.
__device__ inline void scan2(long long& a, long long& b, long long (&sm)[2][32], long long* ta,
                             long long* tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o);
        const long long y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) sm[0][warp] = a, sm[1][warp] = b;
    __syncthreads();
    if (warp == 0) {
        long long x = lane < nw ? sm[0][lane] : 0, y = lane < nw ? sm[1][lane] : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o);
            const long long v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) x += u, y += v;
        }
        if (lane < nw) sm[0][lane] = x, sm[1][lane] = y;
    }
    __syncthreads();
    if (warp) a += sm[0][warp - 1], b += sm[1][warp - 1];
    *ta = sm[0][nw - 1];
    *tb = sm[1][nw - 1];
}

// The last j in [0, n) with v[j] <= x (v ascending, v[0] = 0).
__device__ __forceinline__ int find_last(const uint32_t* v, int n, uint32_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const PlanArgs a) {
    __shared__ uint32_t s_tok[kPlanThreads], s_page[kPlanThreads];
    __shared__ int32_t s_len[kPlanThreads];
    __shared__ uint8_t s_ok[kPlanThreads];
    __shared__ long long s_scan[2][32];
    __shared__ int s_used;
    const int tid = threadIdx.x, nt = blockDim.x;
    const int rank = blockIdx.x, nc = gridDim.x;  // the grid is one cluster
    const int n_free = min(max(*a.n_free, 0), a.num_pages);
    long long tok0 = 0, page0 = 0;
    int bad = 0;
    if (tid == 0) s_used = 0;
    for (int base = 0; base < a.B; base += nt) {
        const int b = base + tid, m = min(nt, a.B - base);
        const int len = b < a.B ? max(a.len[b], 0) : 0;
        const int n = b < a.B ? max(a.n_new[b], 0) : 0;
        const long long want = ((long long)len + n + a.P - 1) / a.P;
        const long long have = ((long long)len + a.P - 1) / a.P;
        const bool over = want > a.max_pages;
        const long long need = over ? 0 : want - have;
        long long t = n, p = need, tt, tp;
        scan2(t, p, s_scan, &tt, &tp);
        const long long tend = tok0 + t, pend = page0 + p;
        const bool fits = need == 0 || pend <= n_free;
        const bool ok = !over && tend <= a.capacity && fits;
        s_tok[tid] = (uint32_t)min(t - n, (long long)a.capacity);
        s_page[tid] = (uint32_t)min(p - need, (long long)a.num_pages);
        s_len[tid] = len;
        s_ok[tid] = ok;
        if (b < a.B && ok && need > 0) atomicMax(&s_used, (int)pend);
        if (b < a.B && !ok)
            bad |= (over || tend > a.capacity) ? KVQ_STATUS_LEN_OVERFLOW : KVQ_STATUS_NO_PAGES;
        // every block has read this chunk's lengths before len_out, maybe the same buffer, changes
        if (nc > 1) cluster_sync(); else __syncthreads();
        if (rank == 0 && b < a.B) {
            a.cu[b] = (int32_t)min(tend - n, (long long)INT32_MAX);
            a.len_out[b] = ok ? len + n : len;
        }
        const long long tlast = min(tok0 + tt, (long long)a.capacity);
        for (long long i = tok0 + rank * nt + tid; i < tlast; i += (long long)nc * nt) {
            const uint32_t rel = (uint32_t)(i - tok0);
            const int j = find_last(s_tok, m, rel);
            const long long pos = (long long)s_len[j] + (rel - s_tok[j]);
            int slot = -1;
            if (s_ok[j]) {
                const int pi = (int)(pos / a.P), hv = (int)(((long long)s_len[j] + a.P - 1) / a.P);
                const int page =
                    pi < hv ? a.table[(size_t)(base + j) * a.max_pages + pi]
                            : a.free_pages[n_free - 1 - (int)(page0 + s_page[j] + (pi - hv))];
                if (page >= 0 && page < a.num_pages) slot = page * a.P + (int)(pos % a.P);
                else bad |= KVQ_STATUS_BAD_PAGE;
            }
            a.slots[i] = slot;
            a.pos[i] = (int32_t)min(pos, (long long)INT32_MAX);
        }
        const long long plast = min(tp, (long long)n_free - page0);
        for (long long r = rank * nt + tid; r < plast; r += (long long)nc * nt) {
            const int j = find_last(s_page, m, (uint32_t)r);
            if (!s_ok[j]) continue;
            const int hv = (int)(((long long)s_len[j] + a.P - 1) / a.P);
            a.table[(size_t)(base + j) * a.max_pages + hv + (int)(r - s_page[j])] =
                a.free_pages[n_free - 1 - (int)(page0 + r)];
        }
        tok0 += tt;
        page0 += tp;
        __syncthreads();
    }
    for (long long i = tok0 + rank * nt + tid; i < a.capacity; i += (long long)nc * nt)
        a.slots[i] = -1, a.pos[i] = 0;
    // every block read n_free before the first barrier above
    if (rank == 0 && tid == 0) {
        a.cu[a.B] = (int32_t)min(tok0, (long long)INT32_MAX);
        *a.n_free_out = n_free - s_used;
    }
    if (bad && (rank == 0 || (bad & KVQ_STATUS_BAD_PAGE))) atomicOr(a.status, bad);
}

// Release: the same walk over requests, one block; pages pushed in request order.
__global__ void __launch_bounds__(kPlanThreads)
    k_page_release(int B, int P, int num_pages, int max_pages, int32_t* len, const int32_t* done,
                   int32_t* table, int32_t* free_pages, int32_t* n_free_p, int32_t* status) {
    __shared__ uint32_t s_page[kPlanThreads];
    __shared__ long long s_scan[2][32];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int n_free = min(max(*n_free_p, 0), num_pages);
    long long page0 = 0;
    for (int base = 0; base < B; base += nt) {
        const int b = base + tid, m = min(nt, B - base);
        long long cnt = 0, zero = 0, tc, tz;
        if (b < B && done[b] != 0) {
            cnt = min(((long long)max(len[b], 0) + P - 1) / P, (long long)max_pages);
            len[b] = 0;
        }
        long long c = cnt;
        scan2(c, zero, s_scan, &tc, &tz);
        s_page[tid] = (uint32_t)min(c - cnt, (long long)UINT32_MAX);
        __syncthreads();
        for (long long r = tid; r < tc; r += nt) {
            const int j = find_last(s_page, m, (uint32_t)r);
            int32_t* e = table + (size_t)(base + j) * max_pages + (int)(r - s_page[j]);
            const long long at = n_free + page0 + r;
            if (at < num_pages) free_pages[at] = *e;
            *e = -1;
        }
        page0 += tc;
        __syncthreads();
    }
    if (tid == 0) {
        if (n_free + page0 > num_pages) atomicOr(status, KVQ_STATUS_BAD_PAGE);
        *n_free_p = (int32_t)min(n_free + page0, (long long)num_pages);
    }
}

// ---------------------------------------------------------------------------------
// Append.  A thread quantizes 8 channels (one 16-byte load, one 4-byte store); two neighbours
// share a scale.  The maximum is taken on the 16-bit values (exact).  y / s is y * rn(1/s) with
// one residual step, q + (y - q s) r, which lands on the same side of every decision point
// t in {0.25, 0.75, ..., 5} as y / s does, and on t itself when y = t s (checked over every 11-bit
// y and 4-bit s; without the step 60 of them miss).  HBM bound: 2 + 9/16 bytes a value.
constexpr int kAppThreads = 256;

__device__ __forceinline__ bool slot_ok(int slot, int limit, int32_t* status) {
    if (slot < 0 || slot >= limit) {
        if (slot != -1) set_status(status, KVQ_STATUS_BAD_PAGE);
        return false;
    }
    return true;
}

template <int D, bool BF>
__global__ void __launch_bounds__(kAppThreads)
    k_paged_append(const kvq_paged_cfg cfg, uint8_t* pool, int32_t* status,
                   const uint16_t* __restrict__ k, int64_t ks, const uint16_t* __restrict__ v,
                   int64_t vs, const int32_t* __restrict__ slots, int n) {
    constexpr int TH = D / 8;  // threads of one token's head
    const bool val = blockIdx.y;
    const int per = cfg.Hkv * TH;
    const int64_t total = (int64_t)n * per;
    const uint16_t* src = val ? v : k;
    const int64_t stride = val ? vs : ks;
    const int e = val ? cfg.v_exp : cfg.k_exp;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
    // total and the step are even, so a scale's two threads leave the loop together; the mask of
    // the shuffle names the pair
    const uint32_t pair = 3u << (threadIdx.x & 30);
    for (int64_t it = (int64_t)blockIdx.x * kAppThreads + threadIdx.x; it < total;
         it += (int64_t)gridDim.x * kAppThreads) {
        const int i = (int)(it / per), r = (int)(it % per);
        const uint4 w4 = __ldcs(reinterpret_cast<const uint4*>(src + i * stride + r * 8));
        const int slot = slots[i];
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        // largest |x| of 16 channels; |x| of a 16-bit float orders as its bits, NaNs above
        // infinity
        uint32_t mx = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) mx = __vmaxu2(mx, w[q] & 0x7fff7fffu);
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(pair, mx, 1));
        float x[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[2 * q] = lo16<BF>(w[q]), x[2 * q + 1] = hi16<BF>(w[q]);
        float am = lo16<BF>(mx);
        if (mx >= (BF ? 0x7f80u : 0x7c00u)) {  // infinities or NaNs among the 16
            am = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (x[q] != x[q]) x[q] = 0.0f;
                am = fmaxf(am, fabsf(x[q]));
                x[q] = fminf(fmaxf(x[q], -1e30f), 1e30f);
            }
            am = fmaxf(am, __shfl_xor_sync(pair, am, 1));
        }
        const float a6 = __fdiv_rn(am * down, 6.0f);
        uint16_t sb;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(a6));
        const float s = __half2float(__ushort_as_half((uint16_t)e4m3x2(sb))) * up;
        const float rs = s > 0.0f ? __frcp_rn(s) : 0.0f;
        uint32_t code = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float y0 = x[2 * q + z] * rs;
                y[z] = fmaf(fmaf(-y0, s, x[2 * q + z]), rs, y0);
            }
            uint16_t c2;
            asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\t"
                "cvt.u16.u8 %0, c;\n\t}"
                : "=h"(c2)
                : "f"(y[1]), "f"(y[0]));
            code |= (uint32_t)c2 << (8 * q);
        }
        if (!slot_ok(slot, cfg.num_pages * cfg.page_tokens, status)) continue;
        const int page = slot / cfg.page_tokens, t = slot % cfg.page_tokens;
        const int h = r / TH, c = r % TH;
        uint8_t* g = pool + group_at(cfg, page, h, t / kGroup) + (val ? Paged<D>::kHalf : 0);
        *reinterpret_cast<uint32_t*>(g + (t % kGroup) * Paged<D>::kRow + c * 4) = code;
        if ((c & 1) == 0)
            g[kGroup * Paged<D>::kRow + (t % kGroup) * Paged<D>::kScales + c / 2] = (uint8_t)sb;
    }
}

// Read-back: the same split of work, the other way; HBM bound.
template <int D, bool BF>
__global__ void __launch_bounds__(kAppThreads)
    k_paged_dequant(const kvq_paged_cfg cfg, const uint8_t* __restrict__ pool, int32_t* status,
                    const int32_t* __restrict__ slots, int n, uint16_t* __restrict__ khat,
                    uint16_t* __restrict__ vhat) {
    constexpr int TH = D / 8;
    const bool val = blockIdx.y;
    const int per = cfg.Hkv * TH;
    const int64_t total = (int64_t)n * per;
    uint16_t* dst = val ? vhat : khat;
    const int e = val ? cfg.v_exp : cfg.k_exp;
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    const float top = BF ? 3.38953138925153547590e38f : 65504.0f;
    for (int64_t it = (int64_t)blockIdx.x * kAppThreads + threadIdx.x; it < total;
         it += (int64_t)gridDim.x * kAppThreads) {
        const int i = (int)(it / per), r = (int)(it % per);
        const int slot = slots[i];
        uint4 o = make_uint4(0, 0, 0, 0);
        if (slot_ok(slot, cfg.num_pages * cfg.page_tokens, status)) {
            const int page = slot / cfg.page_tokens, t = slot % cfg.page_tokens;
            const int h = r / TH, c = r % TH;
            const uint8_t* g = pool + group_at(cfg, page, h, t / kGroup) + (val ? Paged<D>::kHalf : 0);
            const uint32_t w = *reinterpret_cast<const uint32_t*>(g + (t % kGroup) * Paged<D>::kRow + c * 4);
            const uint32_t sb = g[kGroup * Paged<D>::kRow + (t % kGroup) * Paged<D>::kScales + c / 2];
            const uint32_t s2 = e4m3x2(sb | sb << 8);
            uint32_t h2[4], q[4];
            e2m1x8(w, h2);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint32_t p = hmul2(h2[z], s2);
                const float lo = fminf(fmaxf(lo16<false>(p) * up, -top), top);
                const float hi = fminf(fmaxf(hi16<false>(p) * up, -top), top);
                q[z] = pack16<BF>(lo, hi);
            }
            o = make_uint4(q[0], q[1], q[2], q[3]);
        }
        __stcs(reinterpret_cast<uint4*>(dst + it * 8), o);
    }
}

int app_blocks(int64_t items) {
    const int64_t b = (items + kAppThreads - 1) / kAppThreads;
    return (int)(b < 1 ? 1 : b > 148 * 64 ? 148 * 64 : b);
}

}  // namespace

extern "C" {

int kvq_paged_validate_cfg(const kvq_paged_cfg* cfg) { return check_paged_cfg(cfg); }

int kvq_paged_layout(const kvq_paged_cfg* cfg, size_t* bytes) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!bytes) return KVQ_ERR_NULL;
    *bytes = (size_t)cfg->num_pages * cfg->Hkv * (cfg->page_tokens / kGroup) *
             paged_group_bytes(cfg->D);
    return KVQ_OK;
}

int kvq_paged_reset(const kvq_paged_cache* c, void* stream) {
    int e = check_paged_cache(c);
    if (e) return e;
    return record_cuda(cudaMemsetAsync(c->status, 0, 4, (cudaStream_t)stream));
}

int kvq_paged_get_status(const kvq_paged_cache* c, int32_t* out, void* stream) {
    if (!c || !c->status || !out) return KVQ_ERR_NULL;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t ce = cudaMemcpyAsync(out, c->status, 4, cudaMemcpyDeviceToHost, st);
    if (ce) return record_cuda(ce);
    return record_cuda(cudaStreamSynchronize(st));
}

int kvq_page_plan(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, int32_t B,
                  const int32_t* len, const int32_t* n_new, int32_t* block_table,
                  const int32_t* free_pages, const int32_t* n_free, int32_t capacity,
                  int32_t* cu_new, int32_t* len_out, int32_t* n_free_out, int32_t* slots,
                  int32_t* positions, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!cache || !cache->status || !len || !n_new || !block_table || !free_pages || !n_free ||
        !cu_new || !len_out || !n_free_out)
        return KVQ_ERR_NULL;
    if (capacity > 0 && (!slots || !positions)) return KVQ_ERR_NULL;
    if (B < 1 || B > (1 << 20) || capacity < 0) return KVQ_ERR_SHAPE;
    PlanArgs a{len,    n_new, free_pages, n_free, block_table,      cu_new,         len_out,        n_free_out, slots,
               positions, cache->status, B, cfg->page_tokens, cfg->num_pages, cfg->max_pages, capacity};
    // one thread a request or token, in one block up to 8192 tokens: a cluster's start and its
    // barriers cost about a microsecond
    const int most = B > capacity ? B : capacity;
    const int threads = most >= kPlanThreads ? kPlanThreads : (most + 31) / 32 * 32;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(capacity > 8192 ? 8 : 1);
    lc.blockDim = dim3(threads);
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = lc.gridDim.x;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return record_cuda(cudaLaunchKernelEx(&lc, k_page_plan, (const PlanArgs)a));
}

int kvq_page_release(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, int32_t B,
                     int32_t* len, const int32_t* done, int32_t* block_table, int32_t* free_pages,
                     int32_t* n_free, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!cache || !cache->status || !len || !done || !block_table || !free_pages || !n_free)
        return KVQ_ERR_NULL;
    if (B < 1 || B > (1 << 20)) return KVQ_ERR_SHAPE;
    k_page_release<<<1, kPlanThreads, 0, (cudaStream_t)stream>>>(
        B, cfg->page_tokens, cfg->num_pages, cfg->max_pages, len, done, block_table, free_pages,
        n_free, cache->status);
    return record_cuda(cudaGetLastError());
}

int kvq_paged_append(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slots,
                     int32_t n, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if ((e = check_paged_cache(cache))) return e;
    if (n < 0) return KVQ_ERR_SHAPE;
    if (n == 0) return KVQ_OK;
    if (!k || !v || !slots) return KVQ_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (k_stride | v_stride) & 7) return KVQ_ERR_ALIGN;
    const int64_t row = (int64_t)cfg->Hkv * cfg->D;
    if (k_stride < row || v_stride < row) return KVQ_ERR_SHAPE;
    const bool bf = cfg->dtype == KVQ_BF16;
    auto* kern = cfg->D == 64 ? (bf ? k_paged_append<64, true> : k_paged_append<64, false>)
                              : (bf ? k_paged_append<128, true> : k_paged_append<128, false>);
    kern<<<dim3(app_blocks(n * (row / 8)), 2), kAppThreads, 0, (cudaStream_t)stream>>>(
        *cfg, cache->pool, cache->status, (const uint16_t*)k, k_stride, (const uint16_t*)v,
        v_stride, slots, n);
    return record_cuda(cudaGetLastError());
}

int kvq_paged_dequantize(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache,
                         const int32_t* slots, int32_t n, void* khat, void* vhat, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if ((e = check_paged_cache(cache))) return e;
    if (n < 0) return KVQ_ERR_SHAPE;
    if (n == 0) return KVQ_OK;
    if (!slots || !khat || !vhat) return KVQ_ERR_NULL;
    if (!aligned16(khat) || !aligned16(vhat)) return KVQ_ERR_ALIGN;
    const bool bf = cfg->dtype == KVQ_BF16;
    auto* kern = cfg->D == 64 ? (bf ? k_paged_dequant<64, true> : k_paged_dequant<64, false>)
                              : (bf ? k_paged_dequant<128, true> : k_paged_dequant<128, false>);
    kern<<<dim3(app_blocks((int64_t)n * cfg->Hkv * cfg->D / 8), 2), kAppThreads, 0,
           (cudaStream_t)stream>>>(*cfg, cache->pool, cache->status, slots, n, (uint16_t*)khat,
                                   (uint16_t*)vhat);
    return record_cuda(cudaGetLastError());
}

}  // extern "C"
