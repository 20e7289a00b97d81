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
    // a tile may begin before a request's last token and end a few hundred past it, in 32 bits
    if ((int64_t)c->max_pages * c->page_tokens > INT32_MAX - 4096) return KVQ_ERR_SHAPE;
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
// Latency bound, one launch: 4096 requests with 102,000 tokens take 17.1 us a call, of which loads
// 1.5, sums 2, the cluster's barrier 1, tokens 7 and pages 1; eight requests 8 us, nearly all host.
struct PlanArgs {
    const int32_t *len, *n_new, *free_pages, *n_free;
    int32_t *table, *cu, *len_out, *n_free_out, *slots, *pos, *status;
    int32_t B, P, num_pages, max_pages, capacity, entries;  // entries: of free_pages, at most num_pages
};

constexpr int kPlanThreads = 1024;

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

// ITEMS requests a thread, consecutive ones.  A cluster of eight blocks at most: 8192 threads.
template <int ITEMS>
__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const PlanArgs a) {
    extern __shared__ uint32_t s_plan[];  // per request of the chunk: first token, first page, length
    __shared__ long long s_scan[2][32];
    __shared__ int s_used;
    const int tid = threadIdx.x, nt = blockDim.x, chunk = nt * ITEMS;
    uint32_t *s_tok = s_plan, *s_page = s_plan + chunk, *s_len = s_plan + 2 * chunk;  // length: top bit, accepted
    const int rank = blockIdx.x, nc = gridDim.x;  // the grid is one cluster
    const int lp = 31 - __clz(a.P), pm = a.P - 1;
    let_next();
    after_previous();
    const int n_free = min(max(*a.n_free, 0), a.entries);
    long long tok0 = 0, page0 = 0;
    int bad = 0;
    if (tid == 0) s_used = 0;
    for (int base = 0; base < a.B; base += chunk) {
        const int b0 = base + tid * ITEMS, m = min(chunk, a.B - base);
        int len[ITEMS], n[ITEMS];
        long long need[ITEMS], t = 0, p = 0, tt, tp;
        bool over[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            len[i] = b0 + i < a.B ? max(a.len[b0 + i], 0) : 0;
            n[i] = b0 + i < a.B ? max(a.n_new[b0 + i], 0) : 0;
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const long long want = ((long long)len[i] + n[i] + pm) >> lp, have = ((long long)len[i] + pm) >> lp;
            over[i] = want > a.max_pages;
            need[i] = over[i] ? 0 : want - have;
            t += n[i];
            p += need[i];
        }
        const long long tm = t, pmine = p;
        scan2(t, p, s_scan, &tt, &tp);
        long long tend = tok0 + t - tm, pend = page0 + p - pmine;
        bool ok[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            s_tok[tid * ITEMS + i] = (uint32_t)min(tend - tok0, (long long)a.capacity);
            s_page[tid * ITEMS + i] = (uint32_t)min(pend - page0, (long long)a.num_pages);
            tend += n[i];
            pend += need[i];
            ok[i] = !over[i] && tend <= a.capacity && (need[i] == 0 || pend <= n_free);
            s_len[tid * ITEMS + i] = (uint32_t)len[i] | (ok[i] ? 0x80000000u : 0u);
            if (b0 + i >= a.B) continue;
            if (ok[i] && need[i] > 0) atomicMax(&s_used, (int)pend);
            if (!ok[i]) bad |= (over[i] || tend > a.capacity) ? KVQ_STATUS_LEN_OVERFLOW : KVQ_STATUS_NO_PAGES;
        }
        // every block has read this chunk's lengths before len_out, maybe the same buffer, changes
        if (nc > 1) cluster_sync(); else __syncthreads();
        if (rank == 0) {
            long long c = tok0 + t - tm;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (b0 + i < a.B) {
                    a.cu[b0 + i] = (int32_t)min(c, (long long)INT32_MAX);
                    a.len_out[b0 + i] = ok[i] ? len[i] + n[i] : len[i];
                    c += n[i];
                }
        }
        const int ntok = (int)min(tt, max((long long)a.capacity - tok0, 0LL));
        // a warp takes a run of tokens, 32 at a time: one bisection at its start, then the 32 next
        // boundaries in the lanes' registers, which a token's lane bisects by shuffles
        const int lane = tid & 31, warps = nc * nt / 32, run = ((ntok + 31) / 32 + warps - 1) / warps * 32;
        const int i0 = (rank * nt + tid) / 32 * run, i1 = min(ntok, i0 + run);
        int j0 = i0 < i1 ? find_last(s_tok, m, (uint32_t)i0) : 0;
        for (int i = i0; i < i1; i += 32) {
            const uint32_t rel = i + lane, next = j0 + 1 + lane < m ? s_tok[j0 + 1 + lane] : UINT32_MAX;
            int j = 0;
#pragma unroll
            for (int step = 16; step; step >>= 1)
                if (__shfl_sync(0xffffffffu, next, j + step - 1) <= rel) j += step;
            if (__shfl_sync(0xffffffffu, next, j) <= rel) ++j;
            j += j0;
            if (j == j0 + 32) j = find_last(s_tok, m, rel);  // as many requests without tokens
            j0 = __shfl_sync(0xffffffffu, j, 31);
            if ((int)rel >= i1) break;
            const uint32_t lj = s_len[j], ln = lj & 0x7fffffffu, pos = ln + (rel - s_tok[j]);
            int slot = -1;
            if (lj >> 31) {  // accepted, so the position fits
                const int pi = (int)(pos >> lp), hv = (int)((ln + pm) >> lp);
                const int page = pi < hv ? a.table[(size_t)(base + j) * a.max_pages + pi]
                                         : a.free_pages[n_free - 1 - ((int)page0 + (int)s_page[j] + (pi - hv))];
                if (page >= 0 && page < a.num_pages) slot = (page << lp) + (int)(pos & pm);
                else bad |= KVQ_STATUS_BAD_PAGE;
            }
            a.slots[tok0 + rel] = slot;
            a.pos[tok0 + rel] = (int32_t)min(pos, (uint32_t)INT32_MAX);
        }
        const long long plast = min(tp, (long long)n_free - page0);
        for (long long r = rank * nt + tid; r < plast; r += (long long)nc * nt) {
            const int j = find_last(s_page, m, (uint32_t)r);
            const uint32_t lj = s_len[j];
            if (!(lj >> 31)) continue;
            const int hv = (int)(((long long)(lj & 0x7fffffffu) + pm) >> lp);
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

template <int ITEMS>
int launch_plan(const PlanArgs& a, int blocks, int threads, cudaStream_t st) {
    const size_t smem = (size_t)threads * ITEMS * 12;
    static SmemOptIn opt;
    if (int e = ITEMS > 1 ? opt.set((const void*)k_page_plan<ITEMS>, kPlanThreads * ITEMS * 12) : KVQ_OK) return e;
    return launch_overlapped(k_page_plan<ITEMS>, dim3(blocks), threads, smem, blocks, st, a);
}

// Release: the same walk over requests, one block; pages pushed in request order, 1024 entries at a
// time with their places counted by ballots, as an entry may be no page.  Latency bound: a handful of
// requests end in a step.  One of 130 pages takes 2.9 us in a graph of calls, 64 of
// 512 at once 28.
__global__ void __launch_bounds__(kPlanThreads)
    k_page_release(int B, int P, int num_pages, int max_pages, int32_t* len, const int32_t* done,
                   int32_t* table, int32_t* free_pages, int32_t* n_free_p, int32_t* status) {
    __shared__ uint32_t s_page[kPlanThreads];
    __shared__ long long s_scan[2][32];
    __shared__ int s_count[2][kPlanThreads / 32];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    let_next();
    after_previous();
    const int n_free = min(max(*n_free_p, 0), num_pages);
    long long pushed = 0;
    bool bad = false;
    int turn = 0;
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
        int32_t* e = nullptr;
        int page = -1;
        auto fetch = [&](long long r) {  // entry r of the chunk's
            e = nullptr, page = -1;
            if (r < tc) {
                const int j = find_last(s_page, m, (uint32_t)r);
                e = table + (size_t)(base + j) * max_pages + (int)(r - s_page[j]);
                page = *e;
            }
        };
        fetch(tid);
        for (long long r0 = 0; r0 < tc; r0 += nt, turn ^= 1) {
            int32_t* const at_e = e;
            const int p = page;
            if (r0 + nt < tc) fetch(r0 + nt + tid);  // to come while these are counted
            if (at_e) *at_e = -1;
            const bool ok = p >= 0 && p < num_pages;
            bad |= !ok && p != -1;
            const uint32_t oks = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) s_count[turn][warp] = __popc(oks);
            __syncthreads();
            const int count = s_count[turn][lane];  // 32 warps
            const long long at = n_free + pushed + __reduce_add_sync(0xffffffffu, lane < warp ? count : 0) +
                                 __popc(oks & ((1u << lane) - 1u));
            if (ok && at < num_pages) free_pages[at] = p;
            pushed += __reduce_add_sync(0xffffffffu, count);
        }
        __syncthreads();
    }
    if (tid == 0) {
        bad |= n_free + pushed > num_pages;
        *n_free_p = (int32_t)min(n_free + pushed, (long long)num_pages);
    }
    if (bad) atomicOr(status, KVQ_STATUS_BAD_PAGE);
}

// ---------------------------------------------------------------------------------
// Append and read-back.  A thread has CH channels of a head -- 16, a scale's, to append; 8, a 16-byte
// store, to read back -- and walks over tokens with them, kAhead at a time so that their loads are
// in flight together; a token's place in the pool costs a shift and a multiply, the rest of the
// address is found once.  HBM bound, 2 + 9/16 bytes a value: 32768 tokens of 32 heads of 128 appended
// in 118 us and read back in 115, 5.8 TB/s (88 % of the measured copy rate); with 8 channels to a
// thread the two calls took 311 us instead of 247.
constexpr int kAppThreads = 256;
constexpr int kAhead = 4;

// Where a thread works: chunk r (CH channels) of the rows of tokens i0, i0 + step, ... < i1.
struct Walk {
    int r, i0, i1, step;
    size_t at;  // bytes from a token's (page, row 0 of group 0) to its code word
};
template <int D, int CH>
__device__ __forceinline__ Walk walk_of(const kvq_paged_cfg& c, int n, int tokens, bool val) {
    constexpr int TH = D / CH;
    const int per = c.Hkv * TH, wide = min(per, kAppThreads);
    const int lanes = kAppThreads / wide;  // tokens side by side in a block
    Walk w;
    const int tok = threadIdx.x / wide;
    w.r = blockIdx.x * wide + threadIdx.x % wide;
    w.step = lanes;
    w.i0 = blockIdx.y * tokens + tok;
    w.i1 = tok < lanes && w.r < per ? min(n, (int)(blockIdx.y + 1) * tokens) : 0;
    const int h = w.r / TH;
    w.at = (size_t)h * (c.page_tokens / kGroup) * Paged<D>::kBytes + (val ? Paged<D>::kHalf : 0) + (w.r % TH) * (CH / 2);
    return w;
}
// Bytes from the pool's start (kv head 0) to the row of a slot.
template <int D>
__device__ __forceinline__ size_t row_at(const kvq_paged_cfg& c, int slot, int lp) {
    const int page = slot >> lp, t = slot & (c.page_tokens - 1);
    return (size_t)page * ((size_t)c.Hkv * (c.page_tokens / kGroup) * Paged<D>::kBytes) + (t / kGroup) * Paged<D>::kBytes +
           (t % kGroup) * Paged<D>::kRow;
}
// From the codes of chunk r to their scale.
template <int D, int CH>
__device__ __forceinline__ int scale_off(int slot, int r) {
    const int t = slot % kGroup, c = r % (D / CH);
    return (kGroup - t) * Paged<D>::kRow + t * Paged<D>::kScales + c * CH / kGroup - c * (CH / 2);
}

__device__ __forceinline__ bool slot_ok(int slot, int limit, int32_t* status) {
    if (slot < 0 || slot >= limit) {
        if (slot != -1) set_status(status, KVQ_STATUS_BAD_PAGE);
        return false;
    }
    return true;
}

// Codes of 16 values and their scale byte.  The maximum is taken on the 16-bit values (exact).
// amax / 6 is amax * rn(1/6), and y / s is q = y r with r near 1/s and one residual step,
// q + (y - q s) r: both land on the same side of every decision point as the quotients do, and on
// the point itself when the quotient is one (checked over every 11-bit significand and every
// scale; without the residual step 60 quotients miss).  Where y r may pass binary32 the residual
// would be inf - inf, so values from `past` on, which lie beyond 6 times the largest scale, are
// brought down to 7 times it first.
template <bool BF>
__device__ __forceinline__ uint2 quantize16(const uint4 (&w4)[2], float down, float up, uint32_t past, uint32_t* scale) {
    const uint32_t w[8] = {w4[0].x, w4[0].y, w4[0].z, w4[0].w, w4[1].x, w4[1].y, w4[1].z, w4[1].w};
    // |x| of a 16-bit float orders as its bits, NaNs above infinity
    uint32_t mx = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) mx = __vmaxu2(mx, w[q] & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    float x[16];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[2 * q] = lo16<BF>(w[q]), x[2 * q + 1] = hi16<BF>(w[q]);
    float am = lo16<BF>(mx);
    if (mx >= past) {  // values far past the largest scale, infinities or NaNs among them
        am = 0.0f;
        const float top = 7.0f * 448.0f * up;  // stored as 6 * 448 * up, like all beyond; x r stays finite
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            if (x[q] != x[q]) x[q] = 0.0f;
            am = fmaxf(am, fabsf(x[q]));
            x[q] = fminf(fmaxf(x[q], -top), top);
        }
    }
    uint16_t sb;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.0f), "f"(am * down * 0.16666667f));
    const float s = __half2float(__ushort_as_half((uint16_t)e4m3x2(sb))) * up;
    float rs;
    asm("rcp.approx.f32 %0, %1;" : "=f"(rs) : "f"(s));
    if (s == 0.0f) rs = 0.0f;
    const unsigned long long r2 = pk(rs, rs), ns2 = pk(-s, -s);
    uint32_t code[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f2 y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned long long v = pk(x[8 * h + 2 * q], x[8 * h + 2 * q + 1]), y0 = mul2(v, r2);
            y[q] = upk(fma2(fma2(y0, ns2, v), r2, y0));
        }
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(code[h])
            : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
    }
    *scale = sb;
    return make_uint2(code[0], code[1]);
}

template <int D, bool BF>
__global__ void __launch_bounds__(kAppThreads)
    k_paged_append(const kvq_paged_cfg cfg, uint8_t* pool, int32_t* status,
                   const uint16_t* __restrict__ k, int64_t ks, const uint16_t* __restrict__ v,
                   int64_t vs, const int32_t* __restrict__ slots, int n, int tokens) {
    const bool val = blockIdx.z;
    let_next();
    after_previous();
    const Walk w = walk_of<D, 16>(cfg, n, tokens, val);
    const uint16_t* src = (val ? v : k) + w.r * 16;
    const int64_t stride = val ? vs : ks;
    const int e = val ? cfg.v_exp : cfg.k_exp, lp = 31 - __clz(cfg.page_tokens), limit = cfg.num_pages << lp;
    const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
    // the type's bits of 2^(e + 12), or of infinity; 0 where that is no normal number
    const uint32_t past = BF ? min(max(127 + e + 12, 0), 255) << 7 : min(max(15 + e + 12, 0), 31) << 10;
    for (int i = w.i0; i < w.i1; i += kAhead * w.step) {
        uint4 x[kAhead][2];
        int slot[kAhead];
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
            const int j = i + z * w.step;
            slot[z] = -1;
            if (j < w.i1) {
                const uint4* p = reinterpret_cast<const uint4*>(src + j * stride);
                slot[z] = slots[j], x[z][0] = p[0], x[z][1] = p[1];
            }
        }
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
            if (!slot_ok(slot[z], limit, status)) continue;
            uint32_t sb;
            const uint2 code = quantize16<BF>(x[z], down, up, past, &sb);
            uint8_t* g = pool + row_at<D>(cfg, slot[z], lp) + w.at;
            *reinterpret_cast<uint2*>(g) = code;
            g[scale_off<D, 16>(slot[z], w.r)] = (uint8_t)sb;
        }
    }
}

template <int D, bool BF>
__global__ void __launch_bounds__(kAppThreads)
    k_paged_dequant(const kvq_paged_cfg cfg, const uint8_t* __restrict__ pool, int32_t* status,
                    const int32_t* __restrict__ slots, int n, uint16_t* __restrict__ khat,
                    uint16_t* __restrict__ vhat, int tokens) {
    const bool val = blockIdx.z;
    let_next();
    after_previous();
    const Walk w = walk_of<D, 8>(cfg, n, tokens, val);
    uint16_t* dst = (val ? vhat : khat) + w.r * 8;
    const int64_t stride = (int64_t)cfg.Hkv * D;
    const int e = val ? cfg.v_exp : cfg.k_exp, lp = 31 - __clz(cfg.page_tokens), limit = cfg.num_pages << lp;
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    const float top = BF ? 3.38953138925153547590e38f : 65504.0f;
    const bool plain = !BF && e == 0;  // the fp16 product is the value
    for (int i = w.i0; i < w.i1; i += kAhead * w.step) {
        uint32_t code[kAhead], sb[kAhead];
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
            const int j = i + z * w.step;
            code[z] = sb[z] = 0;
            if (j < w.i1) {
                const int slot = slots[j];
                if (slot_ok(slot, limit, status)) {
                    const uint8_t* g = pool + row_at<D>(cfg, slot, lp) + w.at;
                    code[z] = *reinterpret_cast<const uint32_t*>(g);
                    sb[z] = g[scale_off<D, 8>(slot, w.r)];
                }
            }
        }
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
            const int j = i + z * w.step;
            if (j >= w.i1) break;
            const uint32_t s2 = e4m3x2(sb[z] | sb[z] << 8);
            uint32_t h2[4];
            e2m1x8(code[z], h2);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                h2[q] = hmul2(h2[q], s2);
                if (!plain) {
                    const float lo = fminf(fmaxf(lo16<false>(h2[q]) * up, -top), top);
                    const float hi = fminf(fmaxf(hi16<false>(h2[q]) * up, -top), top);
                    h2[q] = pack16<BF>(lo, hi);
                }
            }
            __stcs(reinterpret_cast<uint4*>(dst + j * stride), make_uint4(h2[0], h2[1], h2[2], h2[3]));
        }
    }
}

// Blocks of both: across the chunks of a row, over runs of tokens (returned), keys and values.
dim3 app_grid(const kvq_paged_cfg* c, int channels, int n, int* tokens) {
    const int per = c->Hkv * c->D / channels, wide = per < kAppThreads ? per : kAppThreads;
    const int lanes = kAppThreads / wide, across = (per + wide - 1) / wide;
    // a token a thread while that leaves SMs idle, then up to four times kAhead; y stays in range
    int64_t t = lanes;
    while (t < 4 * kAhead * lanes && (int64_t)across * 2 * ((n + t - 1) / t) > 148 * 8) t *= 2;
    while ((n + t - 1) / t > 65535) t *= 2;
    *tokens = (int)t;
    return dim3(across, (unsigned)((n + t - 1) / t), 2);
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

int kvq_page_plan_list(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, int32_t B,
                       const int32_t* len, const int32_t* n_new, int32_t* block_table,
                       const int32_t* free_pages, int32_t free_entries, const int32_t* n_free,
                       int32_t capacity, int32_t* cu_new, int32_t* len_out, int32_t* n_free_out,
                       int32_t* slots, int32_t* positions, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!cache || !cache->status || !len || !n_new || !block_table || !free_pages || !n_free ||
        !cu_new || !len_out || !n_free_out)
        return KVQ_ERR_NULL;
    if (capacity > 0 && (!slots || !positions)) return KVQ_ERR_NULL;
    if (B < 1 || B > (1 << 20) || capacity < 0 || capacity > (1 << 30) || free_entries < 0) return KVQ_ERR_SHAPE;
    const int32_t entries = free_entries < cfg->num_pages ? free_entries : cfg->num_pages;
    PlanArgs a{len,    n_new, free_pages, n_free, block_table,      cu_new,         len_out,        n_free_out, slots,
               positions, cache->status, B, cfg->page_tokens, cfg->num_pages, cfg->max_pages, capacity, entries};
    // a thread a request or token; one block up to 4096 tokens, since a cluster's start and its
    // barriers cost about a microsecond; four requests a thread where there are more than threads
    const int most = B > capacity ? B : capacity;
    const int threads = most >= kPlanThreads ? kPlanThreads : (most + 31) / 32 * 32;
    const int blocks = capacity > 4096 ? 8 : 1;
    cudaStream_t st = (cudaStream_t)stream;
    return B > threads ? launch_plan<4>(a, blocks, threads, st) : launch_plan<1>(a, blocks, threads, st);
}

int kvq_page_plan(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, int32_t B,
                  const int32_t* len, const int32_t* n_new, int32_t* block_table,
                  const int32_t* free_pages, const int32_t* n_free, int32_t capacity,
                  int32_t* cu_new, int32_t* len_out, int32_t* n_free_out, int32_t* slots,
                  int32_t* positions, void* stream) {
    return kvq_page_plan_list(cfg, cache, B, len, n_new, block_table, free_pages, INT32_MAX, n_free, capacity, cu_new,
                              len_out, n_free_out, slots, positions, stream);
}

int kvq_page_release(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, int32_t B,
                     int32_t* len, const int32_t* done, int32_t* block_table, int32_t* free_pages,
                     int32_t* n_free, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!cache || !cache->status || !len || !done || !block_table || !free_pages || !n_free)
        return KVQ_ERR_NULL;
    if (B < 1 || B > (1 << 20)) return KVQ_ERR_SHAPE;
    return launch_overlapped(k_page_release, dim3(1), kPlanThreads, 0, 1, (cudaStream_t)stream, B, cfg->page_tokens,
                             cfg->num_pages, cfg->max_pages, len, done, block_table, free_pages, n_free, cache->status);
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
    int tokens;
    const dim3 grid = app_grid(cfg, 16, n, &tokens);
    return launch_overlapped(kern, grid, kAppThreads, 0, 1, (cudaStream_t)stream, *cfg, cache->pool, cache->status,
                             (const uint16_t*)k, k_stride, (const uint16_t*)v, v_stride, slots, n, tokens);
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
    int tokens;
    const dim3 grid = app_grid(cfg, 8, n, &tokens);
    return launch_overlapped(kern, grid, kAppThreads, 0, 1, (cudaStream_t)stream, *cfg, (const uint8_t*)cache->pool,
                             cache->status, slots, n, (uint16_t*)khat, (uint16_t*)vhat, tokens);
}

}  // extern "C"
