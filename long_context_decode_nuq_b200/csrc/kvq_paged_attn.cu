// Attention over the paged 4-bit cache: one token, a few or a chunk of them per request.
#include "kvq_paged_attn.cuh"

using namespace kvq;
using namespace kvq_host;

namespace {

// ---------------------------------------------------------------------------------
// Few query rows per kv head (decode, drafts to verify): at most RB = 8 * NT of them, row r being
// query r / G, head r % G of the kv head's G.
//
// The work is one line of units, 64 tokens of one (request, kv head) each, in request-major order;
// block w of N takes units [w T / N, (w+1) T / N) of it, so every block has the same share whatever
// the lengths are.  A (request, kv head) inside one block is finished there; one that a block
// boundary cuts leaves (m, l, O) of each piece in the workspace, a block having at most two such
// pieces, and k_paged_join adds them up in order, told by the block of the first piece where they
// are.
//
// Where the work is short (CL), a cluster of C blocks takes one (request, kv head) instead, an equal
// part of its units each, and adds the parts through distributed shared memory: no search for the
// block's place, no workspace and no second kernel (one request of 1000 tokens, 8 kv heads: 9 us a
// call, 11 in a line with the join).
//
// In a block one warp brings the codes: a stage is 32 tokens for each of the W others, a lane one
// group of 16 tokens, which is one contiguous run of the pool.  The W warps take 32 tokens each,
// keep running maxima and sums of the rows and join at the end of a piece.
//
// Both products run on the tensor cores with the tokens as the long side, so one m16n8k16
// instruction serves 16 tokens for 8 rows and a single query head wastes only idle columns:
//   S^T [16 tokens x 8 rows] = K [16 x D] q^T,   O^T [D x 8 rows] += V^T [D x 16] P^T.
// Codes convert two at a time to fp16 and are multiplied by their scale there: the product has 6
// significant bits and a size of 2^-10 .. 2688, so K and V enter exactly.  A bf16 query enters as
// fp16 too: each row is divided by a power of two that puts its largest value at 2^10, which
// leaves every value within 2^-35 of the row's largest exact.  Only P is rounded, to fp16 (half a
// step is 2^-11); it is kept at up to 2^15 of the largest so that tokens 2^-26 below the maximum
// still have all their bits.  Maximum, sums and O are binary32.
//
// The rows of a K tile are permuted (tau) so that both the 16-byte reads of K rows and the 8-byte
// reads of V rows spread over the banks; S^T then leaves its lanes with (token, 2 rows), which
// movmatrix turns into the B operand of the second product.
//
// Bound by latencies that 16 warps an SM do not cover, none of its pipes being full: 4 requests of
// up to 128 K tokens (3.1 M token-heads of 144 bytes, 32/8 heads) take 100 us a call with the join,
// 4.4 TB/s (67 % of the measured copy rate), at 18 warp instructions a token-head, most of them
// conversions, scalings and matrix instructions.  Issue slots are 60 % used, the tensor pipe 26 %;
// warps wait for fixed latencies, the conversion pipe and memory in about equal parts.  8 x 8 K
// with 32 kv heads: 55 us, about 10 of them start, end and join.
constexpr int kUnit = 64;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int NT>
constexpr int kWarps = NT == 1 ? 7 : 5;        // that compute; one more loads
template <int NT>
constexpr int kStages = 3;
template <int NT>
constexpr int kFewThreads = kWarps<NT> * 32 + 32;
template <int D, int NT>
struct FewSmem {
    static constexpr int W = kWarps<NT>, ST = kStages<NT>, RB = 8 * NT;
    static constexpr int stage = W * 2 * Paged<D>::kBytes;
    static constexpr int q = ST * stage;                      // uint2 [NT][D/16][32], then float [RB]
    static constexpr int joint = q + NT * (D / 16) * 256 + RB * 4;  // float [W][4][D + 4]
    static constexpr int ml = joint + W * 4 * (D + 4) * 4;    // float2 [W][4]
    static constexpr int bar = ml + W * 4 * 8;                // full[ST], empty[ST]
    static constexpr int misc = bar + 16 * ST;                // got[ST], dead, start
    static constexpr int scan = misc + 64;                    // int64 [32]
    static constexpr int total = scan + 32 * 8;
};

// What a request contributes: its rows, the tokens they see and its units (per kv head).
struct Seg {
    Rows rw;
    int first;            // position of query 0 (negative: it sees nothing)
    int lo, hi;           // tokens some row sees
    int all_lo, all_hi;   // tokens every row sees
    int tbase, u;
};
__device__ __forceinline__ Seg seg_of(const AttnArgs& a, int b) {
    Seg s;
    s.rw = rows_of(a, b);
    s.first = s.rw.len - s.rw.n;
    s.hi = min(s.rw.kv, s.first + s.rw.nq);
    s.lo = first_seen(a, s.first);
    s.all_hi = min(s.rw.kv, s.first + 1);
    s.all_lo = first_seen(a, s.first + s.rw.nq - 1);
    s.tbase = s.lo & ~(kGroup - 1);
    // one that sees nothing still has a unit, which writes its zeros
    s.u = s.rw.R == 0 ? 0 : s.hi > s.lo ? (s.hi - s.tbase + kUnit - 1) / kUnit : 1;
    return s;
}

// floor(T x / N), in 32 bits where they hold it (a 64-bit division costs a tenth of a microsecond).
__device__ __forceinline__ int64_t share(int64_t T, int x, int N) {
    if (T < (1 << 20) && x <= 4096) return (uint32_t)T * (uint32_t)x / (uint32_t)N;
    return T * x / N;
}

// Wait for a phase, giving up where another warp has.
__device__ __forceinline__ bool wait_or(uint64_t* bar, uint32_t parity, volatile int* dead) {
    for (uint32_t it = 0; it < (1u << 22); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u && *dead) return false;
    }
    *dead = 1;
    return false;
}

template <int D, int NT, bool BF, bool CL>
__global__ void __launch_bounds__(kFewThreads<NT>, 2) k_paged_attn(const AttnArgs a, int B) {
    using L = FewSmem<D, NT>;
    constexpr int W = L::W, ST = L::ST, RB = L::RB;
    constexpr int GB = Paged<D>::kBytes, HALF = Paged<D>::kHalf, ROW = Paged<D>::kRow, SC = Paged<D>::kScales;
    constexpr int KS = D / 16;  // k-steps of S^T, and 16-channel tiles of O^T
    constexpr int KW = D / 32;  // code words of a lane's part of a K row
    constexpr int VW = D / 64;  // code words of a lane's part of a V row
    constexpr int STEP = W * 32;  // tokens of a stage
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar);
    uint64_t* empty = full + ST;
    volatile uint32_t* s_got = reinterpret_cast<uint32_t*>(smem + L::misc);
    volatile int* dead = reinterpret_cast<int*>(smem + L::misc + 16);
    int64_t* s_start = reinterpret_cast<int64_t*>(smem + L::misc + 24);  // units before b0, b0, T
    int64_t* s_scan = reinterpret_cast<int64_t*>(smem + L::scan);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int G = a.c.Hq / a.c.Hkv, Hkv = a.c.Hkv;
    const int lp = 31 - __clz(a.c.page_tokens);

    if (threadIdx.x == 0) {
        *dead = 0;
        for (int i = 0; i < ST; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], W);
        fence_mbar_init();
    }
    let_next();
    after_previous();
    // where this block's units begin: prefix sums of the requests' units
    int64_t base = 0, T = 0;  // units before request b; all units
    int b = 0, N = 1;
    int64_t g0 = 0, g1 = 0;
    if constexpr (CL) {
        const int C = a.S, seg = blockIdx.x / C, rank = blockIdx.x % C;
        b = seg / Hkv;
        const Seg s = seg_of(a, b);
        if (seg % Hkv == 0 && rank == 0 && threadIdx.x == 0 && (s.rw.n > s.rw.nq || s.rw.len > s.rw.kv))
            set_status(a.status, KVQ_STATUS_LEN_OVERFLOW);
        if (s.u == 0) return;  // no rows: the whole cluster leaves
        // positions within the request, as if it were the first: kv heads one after the other
        const int64_t at = (int64_t)(seg % Hkv) * s.u;
        g0 = at + (int64_t)s.u * rank / C, g1 = at + (int64_t)s.u * (rank + 1) / C;
        __syncthreads();
    } else {
    auto report = [&](const Seg& s, int r) {  // by block 0, for every request
        if (s.rw.n > s.rw.nq || s.rw.len > s.rw.kv) set_status(a.status, KVQ_STATUS_LEN_OVERFLOW);
        if (s.u == 0 && a.rec && a.by_request)
            for (int h = 0; h < Hkv; ++h) a.rec[r * Hkv + h] = make_int4(-1, 0, 0, 0);
    };
    if (B <= 32) {  // a lane a request, every warp for itself
        int u = 0;
        if (lane < B) {
            const Seg s = seg_of(a, lane);
            u = s.u;
            if (blockIdx.x == 0 && warp == 0) report(s, lane);
        }
        int64_t incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        T = __shfl_sync(0xffffffffu, incl, 31) * Hkv;
        const int64_t at = share(T, blockIdx.x, (int)min((int64_t)gridDim.x, max(T, (int64_t)1)));
        const uint32_t past = __ballot_sync(0xffffffffu, incl * Hkv > at);
        b = past ? __ffs(past) - 1 : 0;
        base = __shfl_sync(0xffffffffu, incl - u, b) * Hkv;
        __syncthreads();
    } else {  // a thread a run of requests
        const int per = (B + kFewThreads<NT> - 1) / kFewThreads<NT>;
        const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
        int64_t mine = 0;
        for (int r = b0; r < b1; ++r) {
            const Seg s = seg_of(a, r);
            mine += s.u;
            if (blockIdx.x == 0) report(s, r);
        }
        int64_t incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int64_t total = 0;
        for (int i = 0; i <= W; ++i) {
            if (i < warp) incl += s_scan[i];
            total += s_scan[i];
        }
        T = total * Hkv;
        const int64_t at = share(T, blockIdx.x, (int)min((int64_t)gridDim.x, max(T, (int64_t)1)));
        int64_t ub = incl - mine;  // units (per kv head) before request b0
        if (ub * Hkv <= at && at < incl * Hkv) {
            int r = b0;
            for (;; ++r) {
                const int u = seg_of(a, r).u;
                if ((ub + u) * Hkv > at) break;
                ub += u;
            }
            s_start[0] = ub * Hkv, s_start[1] = r;
        }
        __syncthreads();
        if (at < T) base = s_start[0], b = (int)s_start[1];
    }
    N = (int)min((int64_t)gridDim.x, T);  // blocks that have units
    if ((int)blockIdx.x >= N) {
        if (a.rec && !a.by_request && threadIdx.x == 0) a.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    g0 = share(T, blockIdx.x, N), g1 = share(T, blockIdx.x + 1, N);
    }
    Seg sg = seg_of(a, b);

    // the pieces of [g0, g1): request b, kv head h, units [u0, u0 + un)
    int h = 0, u0 = 0, un = 0;
    auto piece = [&](int64_t at) {
        while (at >= base + (int64_t)sg.u * Hkv) {
            base += (int64_t)sg.u * Hkv;
            sg = seg_of(a, ++b);
        }
        const int64_t off = at - base;
        h = off <= INT32_MAX ? (int)((uint32_t)off / (uint32_t)sg.u) : (int)(off / sg.u);
        u0 = (int)(off - (int64_t)h * sg.u);
        un = (int)min((int64_t)(sg.u - u0), g1 - at);
    };

    if (warp == W) {  // the loader
        const size_t page_bytes = group_at(a.c, 1, 0, 0), head_bytes = (size_t)(a.c.page_tokens / kGroup) * GB;
        int k = 0;
        for (int64_t at = g0; at < g1 && !*dead; at += un) {
            piece(at);
            const int32_t* tab = a.table + (size_t)b * a.c.max_pages;
            const uint8_t* pool = a.pool + h * head_bytes;
            const int t0 = sg.tbase + u0 * kUnit, t1 = min(sg.hi, t0 + un * kUnit);
            auto wanted = [&](int tok) { return lane < 2 * W && tok < t1 && tok + kGroup > sg.lo; };
            int tg = t0 + lane * kGroup;
            int page = wanted(tg) ? tab[tg >> lp] : -1;
            for (int ts = t0; ts < t1; ts += STEP, tg += STEP, ++k) {
                const int st = k % ST;
                const bool want = wanted(tg), ok = want && page >= 0 && page < a.c.num_pages;
                const int nxt = wanted(tg + STEP) ? tab[(tg + STEP) >> lp] : -1;
                if (want && !ok) set_status(a.status, KVQ_STATUS_BAD_PAGE);
                if (!__all_sync(0xffffffffu, wait_or(&empty[st], (k / ST + 1) & 1, dead))) break;
                const uint32_t v = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) {
                    s_got[st] = v;
                    mbar_arrive_expect_tx(&full[st], __popc(v) * GB);
                }
                __syncwarp();
                if (ok)
                    bulk_load(smem + st * L::stage + lane * GB,
                              pool + page * page_bytes + ((tg & (a.c.page_tokens - 1)) / kGroup) * GB, GB, &full[st]);
                page = nxt;
            }
        }
        if (*dead)  // a copy did not come: let the others land before the memory is left
            for (int i = max(0, k - ST); i < k; ++i) mbar_wait(&full[i % ST], (i / ST) & 1);
        return;
    }

    const int tau = (g & 1) ? 4 + ((g >> 1) ^ 1) : (g >> 1);
    const int tv[4] = {t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1)};
    uint2* s_q = reinterpret_cast<uint2*>(smem + L::q);
    float* s_sl2 = reinterpret_cast<float*>(s_q + NT * KS * 32);
    float* so = reinterpret_cast<float*>(smem + L::joint);
    float2* sml = reinterpret_cast<float2*>(smem + L::ml);
    int k = 0;
    for (int64_t at = g0; at < g1; at += un) {
        piece(at);
        const Rows& rw = sg.rw;
        // queries, as the columns of B: lane (g, t) has channels [t*D/4, (t+1)*D/4) of row g.  They
        // wait in shared memory, where a step's 8 bytes a lane cost less than the registers would.
        for (int nt = warp; nt < NT; nt += W) {
            const int r = nt * 8 + g;
            uint32_t w[KS * 2] = {};
            if (r < rw.R) {
                const uint16_t* src = a.q + (int64_t)(rw.c0 + r / G) * a.qs + (h * G + r % G) * D + t * (D / 4);
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    const uint4 x = reinterpret_cast<const uint4*>(src)[i];
                    w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
                }
            }
            // a negative scale goes into the query, so that the largest score is the largest product
            const uint32_t neg = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
            for (int i = 0; i < KS * 2; ++i) w[i] ^= neg;
            int e = 0;
            if (BF) {
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < KS * 2; ++i) mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
                mx = max(mx & 0xffffu, mx >> 16);
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int eb = (int)(mx >> 7);
                if (eb < 255) e = max(eb - 127 - 10, -120);
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < KS * 2; ++i) w[i] = pack_h2(lo16<true>(w[i]) * f, hi16<true>(w[i]) * f);
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) s_q[(nt * KS + j) * 32 + lane] = make_uint2(w[2 * j], w[2 * j + 1]);
            if (t == 0) s_sl2[nt * 8 + g] = fmaxf(fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
        float sl2[NT][2];
        int pos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                sl2[nt][z] = s_sl2[nt * 8 + 2 * t + z];
                pos[nt][z] = sg.first + (nt * 8 + 2 * t + z) / G;
            }

        float o[NT][KS][4] = {}, m[NT][2], l[NT][2] = {};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY;
        const int ts0 = sg.tbase + u0 * kUnit, ts1 = min(sg.hi, ts0 + un * kUnit);
        for (int ts = ts0; ts < ts1; ts += STEP, ++k) {
            const int stage = k % ST, t0 = ts + warp * 32;
            if (!__all_sync(0xffffffffu, wait_or(&full[stage], (k / ST) & 1, dead))) break;
            const uint32_t got = s_got[stage] >> (2 * warp) & 3u;
            if (t0 >= ts1) {
                if (lane == 0) mbar_arrive(&empty[stage]);
                continue;
            }
            const uint8_t* buf = smem + stage * L::stage + warp * 2 * GB;
            const bool mask = got != 3u || t0 + 32 > sg.all_hi || t0 < sg.all_lo;

            float sc[2][NT][4];
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                uint32_t kc[2][KW], ks[2][2];
                const uint8_t* kb = buf + gr * GB;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint8_t* row = kb + (tau + 8 * z) * ROW + t * (D / 8);
                    const uint8_t* srow = kb + kGroup * ROW + (tau + 8 * z) * SC;
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(row);
                        kc[z][0] = x.x, kc[z][1] = x.y, kc[z][2] = x.z, kc[z][3] = x.w;
                        const uint32_t two = e4m3x2(*reinterpret_cast<const uint16_t*>(srow + 2 * t));
                        ks[z][0] = __byte_perm(two, 0, 0x1010);
                        ks[z][1] = __byte_perm(two, 0, 0x3232);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(row);
                        kc[z][0] = x.x, kc[z][1] = x.y;
                        const uint32_t one = srow[t];
                        ks[z][0] = ks[z][1] = e4m3x2(one | one << 8);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int z = 0; z < 4; ++z) sc[gr][nt][z] = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint32_t x0[4], x1[4];
                    e2m1x8(kc[0][w], x0);
                    e2m1x8(kc[1][w], x1);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint2 qf[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) qf[nt] = s_q[(nt * KS + 2 * w + u) * 32 + lane];
                        const uint32_t s0 = ks[0][w * 2 / KW], s1 = ks[1][w * 2 / KW];
                        const uint32_t A[4] = {hmul2(x0[2 * u], s0), hmul2(x1[2 * u], s1), hmul2(x0[2 * u + 1], s0), hmul2(x1[2 * u + 1], s1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(sc[gr][nt], A, qf[nt].x, qf[nt].y);
                    }
                }
            }
            if (mask) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int tok = t0 + gr * kGroup + tau + (z & 2) * 4;
                            const int p = pos[nt][z & 1];
                            const bool see = (got >> gr & 1u) && tok < ts1 && tok <= p && tok >= first_seen(a, p);
                            if (!see) sc[gr][nt][z] = -INFINITY;
                        }
            }
            // V is asked for here, to come while the softmax is computed (3 % at 4 x 128K)
            uint32_t vc[2][4][VW], sv[2][4];
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    sv[gr][z] = buf[gr * GB + HALF + kGroup * ROW + g * (D / 8) / kGroup + tv[z] * SC];
                    const uint8_t* row = buf + gr * GB + HALF + tv[z] * ROW + g * (D / 16);
                    if constexpr (D == 128) {
                        const uint2 x = *reinterpret_cast<const uint2*>(row);
                        vc[gr][z][0] = x.x, vc[gr][z][1] = x.y;
                    } else {
                        vc[gr][z][0] = *reinterpret_cast<const uint32_t*>(row);
                    }
                }
            // the maximum moves only when some lane's scores ask for it, so the common case needs
            // no exchange between lanes
            float tm[NT][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    tm[nt][z] = fmaxf(fmaxf(sc[0][nt][z], sc[0][nt][z + 2]), fmaxf(sc[1][nt][z], sc[1][nt][z + 2])) * sl2[nt][z];
                    grow |= tm[nt][z] - m[nt][z] > kPRoom;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float x = tm[nt][z];
#pragma unroll
                        for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
                        const float mn = fmaxf(m[nt][z], x - kPShift);
                        const float al = m[nt][z] == mn ? 1.0f : ex2(m[nt][z] - mn);
                        m[nt][z] = mn;
                        l[nt][z] *= al;
#pragma unroll
                        for (int j = 0; j < KS; ++j) o[nt][j][z] *= al, o[nt][j][z + 2] *= al;
                    }
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.0f : -m[nt][0];
                const float m1 = m[nt][1] == -INFINITY ? 0.0f : -m[nt][1];
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    const float p0 = ex2(fmaf(sc[gr][nt][0], sl2[nt][0], m0)), p1 = ex2(fmaf(sc[gr][nt][1], sl2[nt][1], m1));
                    const float p2 = ex2(fmaf(sc[gr][nt][2], sl2[nt][0], m0)), p3 = ex2(fmaf(sc[gr][nt][3], sl2[nt][1], m1));
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    pf[gr][nt][0] = transpose8x8(pack_h2(p0, p1));
                    pf[gr][nt][1] = transpose8x8(pack_h2(p2, p3));
                }
            }
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                uint32_t sb[4] = {sv[gr][0], sv[gr][1], sv[gr][2], sv[gr][3]};
                if (mask) {
                    // bytes nobody wrote may hold a NaN scale, and 0 * NaN is not 0
                    const int tg = t0 + gr * kGroup;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (!(got >> gr & 1u) || tg + tv[z] >= rw.kv) sb[z] = 0;
                }
                const uint32_t s01 = e4m3x2(sb[0] | sb[1] << 8), s23 = e4m3x2(sb[2] | sb[3] << 8);
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    // bytes of (token a, token b) codes of one channel: even channels, then odd ones
                    uint32_t e01[4], o01[4], e23[4], o23[4];
                    e2m1x8((vc[gr][0][w] & 0x0f0f0f0fu) | (vc[gr][1][w] << 4 & 0xf0f0f0f0u), e01);
                    e2m1x8((vc[gr][0][w] >> 4 & 0x0f0f0f0fu) | (vc[gr][1][w] & 0xf0f0f0f0u), o01);
                    e2m1x8((vc[gr][2][w] & 0x0f0f0f0fu) | (vc[gr][3][w] << 4 & 0xf0f0f0f0u), e23);
                    e2m1x8((vc[gr][2][w] >> 4 & 0x0f0f0f0fu) | (vc[gr][3][w] & 0xf0f0f0f0u), o23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t A[4] = {hmul2(e01[i], s01), hmul2(o01[i], s01),
                                               hmul2(e23[i], s23), hmul2(o23[i], s23)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[nt][4 * w + i], A, pf[gr][nt][0], pf[gr][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
        }

        const bool whole = !CL && un == sg.u;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (at != g0);
        // the first piece says where all are: its slot, the block of the last one, and whose rows
        if (!CL && a.rec && threadIdx.x == 0) {
            int4 rec = make_int4(-1, 0, 0, 0);
            if (u0 == 0 && !whole) {
                const int64_t end = at + sg.u;
                rec = make_int4((int)((end * N - 1) / T), (int)slot, rw.c0, h << 8 | rw.R);
            }
            if (a.by_request) {
                if (u0 == 0) a.rec[b * Hkv + h] = rec;
            } else if (rec.x >= 0 || at + un >= g1) {  // only a block's last piece can be one
                a.rec[blockIdx.x] = rec;
            }
        }
        // join the warps: (m, l) and O of 4 rows at a time through shared memory
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][z] += __shfl_xor_sync(0xffffffffu, l[nt][z], x);
#pragma unroll
        for (int part = 0; part < 2 * NT; ++part) {
            const int nt = part / 2;
            if (part * 4 >= rw.R) break;
            if (t >> 1 == (part & 1)) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int row = warp * 4 + 2 * (t & 1) + z;
                    float* dst = so + row * (D + 4) + g * (D / 8);
#pragma unroll
                    for (int j = 0; j < KS; j += 2)  // tiles j: channels 2j, 2j + 1 of the lane's D/8
                        *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][z], o[nt][j][z + 2], o[nt][j + 1][z], o[nt][j + 1][z + 2]);
                    if (g == 0) sml[row] = make_float2(m[nt][z], l[nt][z]);
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
            for (int it = threadIdx.x; it < 4 * (D / 4); it += W * 32) {
                const int r4 = it / (D / 4), row = part * 4 + r4, c4 = it % (D / 4) * 4;
                if (row >= rw.R) break;
                float M = -INFINITY, LL = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, sml[w * 4 + r4].x);
                float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 ml = sml[w * 4 + r4];
                    if (ml.y == 0.0f) continue;  // saw nothing; a row of NaN scores has m = -inf, l = NaN
                    const float f = ex2(ml.x - M);
                    const float4 x = *reinterpret_cast<const float4*>(so + (w * 4 + r4) * (D + 4) + c4);
                    LL += f * ml.y;
                    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
                }
                if (whole) {
                    const int64_t grow = (int64_t)(rw.c0 + row / G) * a.c.Hq + h * G + row % G;
                    const float inv = LL == 0.0f ? 0.0f : a.out_scale / LL;
                    store4<BF>(a.out + grow * D + c4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                    if (c4 == 0 && a.lse) a.lse[grow] = LL == 0.0f ? -INFINITY : (M + log2f(LL)) * kLn2;
                } else if (CL) {  // the ring is no longer read
                    *reinterpret_cast<float4*>(smem + (row * D + c4) * 4) = acc;
                    if (c4 == 0) *reinterpret_cast<float2*>(smem + RB * D * 4 + row * 8) = make_float2(M, LL);
                } else {
                    *reinterpret_cast<float4*>(a.part + (slot * RB + row) * D + c4) = acc;
                    if (c4 == 0) a.pml[slot * RB + row] = make_float2(M, LL);
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
        }
    }
    if constexpr (CL) {
        const int C = a.S, rank = blockIdx.x % C, hh = blockIdx.x / C % Hkv;
        const Rows& rw = sg.rw;
        if (g0 >= g1)  // no units: an empty part
            for (int row = threadIdx.x; row < RB; row += W * 32)
                *reinterpret_cast<float2*>(smem + RB * D * 4 + row * 8) = make_float2(-INFINITY, 0.0f);
        __syncwarp();
        cluster_sync();
        // part p of a row from block p, in that order; the rows' quarters over the blocks' threads
        const uint32_t here = smem_u32(smem);
        for (int it = rank * (W * 32) + threadIdx.x; it < rw.R * (D / 4); it += C * W * 32) {
            const int row = it / (D / 4), c4 = it % (D / 4) * 4;
            float M = -INFINITY, LL = 0.0f;
            float4 acc = make_float4(0, 0, 0, 0);
            for (int p = 0; p < C; ++p) {
                float2 ml;
                float4 x;
                uint32_t from;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(here), "r"(p));
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "r"(from + RB * D * 4 + row * 8));
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                             : "r"(from + (row * D + c4) * 4));
                if (ml.y == 0.0f) continue;
                const float mn = fmaxf(M, ml.x), f = LL == 0.0f ? 0.0f : ex2(M - mn), e = ex2(ml.x - mn);
                LL = LL * f + e * ml.y;
                acc.x = acc.x * f + e * x.x, acc.y = acc.y * f + e * x.y;
                acc.z = acc.z * f + e * x.z, acc.w = acc.w * f + e * x.w;
                M = mn;
            }
            const int64_t grow = (int64_t)(rw.c0 + row / G) * a.c.Hq + hh * G + row % G;
            const float inv = LL == 0.0f ? 0.0f : a.out_scale / LL;
            store4<BF>(a.out + grow * D + c4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (c4 == 0 && a.lse) a.lse[grow] = LL == 0.0f ? -INFINITY : (M + log2f(LL)) * kLn2;
        }
        __syncwarp();
        cluster_sync();  // no block leaves while another reads its part
    }
    if (threadIdx.x == 0 && *dead) set_status(a.status, KVQ_STATUS_WAIT_TIMEOUT);
}

// Joins what block boundaries cut: block (x, row) takes record x, and adds its pieces in order of
// their blocks, eight apart per warp and then over the warps.  Latency bound: about 3 us, its start
// under the main kernel's end.
constexpr int kJoinWarps = 8;
template <int D, bool BF>
__global__ void __launch_bounds__(kJoinWarps * 32) k_paged_join(const AttnArgs a, int RB) {
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float2 s_ml[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    let_next();
    after_previous();
    const int4 rec = a.rec[blockIdx.x];
    const int w1 = rec.x, w0 = rec.y >> 1, h = rec.w >> 8, R = rec.w & 255;
    if (w1 < 0 || row >= R) return;
    constexpr int V = D / 32;
    float acc[V] = {}, M = -INFINITY, L = 0.0f;
#pragma unroll 4
    for (int w = w0 + warp; w <= w1; w += kJoinWarps) {
        const int64_t at = (w == w0 ? (int64_t)rec.y : 2 * (int64_t)w) * RB + row;
        const float2 ml = a.pml[at];
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = a.part[at * D + lane * V + i];
        const float mn = fmaxf(M, ml.x);
        // l = 0: saw nothing, m = -inf; a row of NaN scores has m = -inf, l = NaN
        const float f = L == 0.0f ? 0.0f : ex2(M - mn), e = ml.y == 0.0f ? 0.0f : ex2(ml.x - mn);
        L = L * f + e * ml.y;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = acc[i] * f + e * x[i];
        M = mn;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = acc[i];
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
    float o0 = 0.0f, o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        if (s_ml[w].y == 0.0f) continue;
        const float f = ex2(s_ml[w].x - M);
        L += f * s_ml[w].y;
        o0 += f * s_o[w][2 * threadIdx.x], o1 += f * s_o[w][2 * threadIdx.x + 1];
    }
    const int G = a.c.Hq / a.c.Hkv;
    const int64_t grow = (int64_t)(rec.z + row / G) * a.c.Hq + h * G + row % G;
    const float inv = L == 0.0f ? 0.0f : a.out_scale / L;
    reinterpret_cast<uint32_t*>(a.out + grow * D)[threadIdx.x] = pack16<BF>(o0 * inv, o1 * inv);
    if (threadIdx.x == 0 && a.lse) a.lse[grow] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// Joins the chunk kernel's splits of a row, in split order: a warp per row of the units that were
// split.  Bound by L2: its input has just been written.
constexpr int kMergeWarps = 4;
template <int D, bool BF>
__global__ void __launch_bounds__(kMergeWarps * 32) k_paged_merge(const AttnArgs a) {
    constexpr int PB = kChunkRows / kMergeWarps;  // blocks of a unit
    const int cut = (int)blockIdx.x / PB, r0 = (int)blockIdx.x % PB * kMergeWarps + (threadIdx.x >> 5);
    const Unit unit = unit_of(a, a.whole + cut);
    const int h = unit.h, b = unit.b, lane = threadIdx.x & 31;
    const int G = a.c.Hq / a.c.Hkv;
    let_next();
    after_previous();
    const Rows rw = rows_of(a, b);
    const int r = unit.rb * kChunkRows + r0;
    if (r >= rw.R) return;
    const int64_t grow = (int64_t)(rw.c0 + r / G) * a.c.Hq + h * G + r % G;
    const int64_t at = part_at(a, 0, cut, r0, grow);
    float M = -INFINITY;
    for (int s = lane; s < a.S; s += 32) M = fmaxf(M, a.pml[s * a.part_rows + at].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float L = 0.0f, acc[D / 32] = {};
    for (int s = 0; s < a.S; ++s) {
        const float2 ml = a.pml[s * a.part_rows + at];
        if (ml.y == 0.0f) continue;  // an empty split; one of NaN scores has m = -inf, l = NaN
        const float f = ex2(ml.x - M);
        const float* x = a.part + (s * a.part_rows + at) * D + lane * (D / 32);
        L += f * ml.y;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] += f * x[i];
    }
    const float inv = L == 0.0f ? 0.0f : a.out_scale / L;
    uint16_t* out = a.out + grow * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2)
        *reinterpret_cast<uint32_t*>(out + i) = pack16<BF>(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0 && a.lse) a.lse[grow] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------------------------
// Host: which kernel, blocks or splits, workspace.
struct Plan {
    int nt;   // 8-row tiles of k_paged_attn; 0: the chunk kernel
    int nrb;  // chunk kernel: row blocks
    int64_t units, whole;  // chunk kernel: row blocks of all (request, kv head)s; those not split
    int S;    // chunk kernel: splits of the other units;  k_paged_attn: blocks, or blocks of a cluster
    int64_t part_rows;  // chunk kernel: rows of a split's parts,
    bool by_unit;       // the split units' (true) or all of q's, whichever are fewer
    bool cluster;
    bool join;
};

constexpr int kSms = 148;
// More rows of a kv head than this go to the chunk kernel.
constexpr int kFewRows = 16;

// Most tokens of a split of the chunk kernel.  The tensor cores cut their binary32 sums off instead
// of rounding them, so O drifts toward 0 with every 16 tokens added: by 8e-4 of itself over 2^20
// tokens of like sign (measured), by 1e-4, a fifth of fp16's half step, over 2^17.
constexpr int kSplitTokens = 1 << 17;

// Blocks of split units by the library's choice, at most: it is what bounds the workspace, and
// the model below asks for more only beyond 2^17 tokens (up to 5000 units).
constexpr int64_t kCutBlocks = 6 * kSms;

// Most tokens of one request that a warp of k_paged_attn adds up in a row, for the same reason: its
// O drifts by 1.1e-7 for each 16 tokens, half of that on average over a growing sum, so by 1e-4 over
// 2^15 (and by 3e-2 over 2^26 / 7, before there was a limit).
constexpr int kWarpTokens = 1 << 15;

int64_t least_splits(int64_t span) { return (span + kSplitTokens - 1) / kSplitTokens; }

// How the chunk kernel's units (256 rows of a kv head each) are spread: the first `whole` get a
// block each, the others S, whose parts k_paged_merge adds.  The least time of a model in which a
// block costs 10 us and 2 us per 128 tokens (measured: 2.0), blocks run one per SM in waves, and a
// split writes and reads its part at 5 TB/s; whole units come in full waves, and there are none
// where a split must not have all tokens.  Against 32768 tokens, 8 kv heads, in short runs: 64
// queries 514 us in one part, 59 in 18; 1184 queries (152 units) 728 all whole, 560 with the last 4
// split.
void chunk_splits(const kvq_paged_cfg* c, int64_t units, int64_t span, int64_t* whole, int* splits) {
    const int64_t tiles = (span + 127) / 128, must = least_splits(span);
    const int64_t waves = must > 1 ? 0 : units / kSms, most = must > kSms ? must : kSms;
    *whole = must > 1 ? 0 : units, *splits = (int)must;
    double least = must > 1 ? 1e30 : (double)((units + kSms - 1) / kSms) * (10.0 + 2.0 * (double)tiles);
    for (int64_t w = waves; w >= 0; w = w == 0 ? -1 : w == waves ? w - 1 : 0)  // all full waves whole, one less, none
        for (int64_t S = must > 1 ? must : 2; S <= most && S <= tiles; ++S) {
            const int64_t rest = units - w * kSms;
            if (rest == 0 || (S > must && rest * S > kCutBlocks)) break;
            const double t = (double)w * (10.0 + 2.0 * (double)tiles) + 4.0 + (double)rest * S * kChunkRows * c->D * 8 / 5e6 +
                             (double)((rest * S + kSms - 1) / kSms) * (10.0 + 2.0 * (double)((tiles + S - 1) / S));
            if (t < 0.98 * least) least = t, *whole = w * kSms, *splits = (int)S;
        }
}

Plan plan_of(const kvq_paged_cfg* c, int B, int total_q, int max_q, int max_len, int splits, int window) {
    const int64_t R = (int64_t)max_q * (c->Hq / c->Hkv);
    // no row block sees more tokens than this
    int64_t span = max_len;
    if (window > 0 && span > (int64_t)window + max_q + 128) span = (int64_t)window + max_q + 128;
    Plan p{};
    p.nt = R <= 8 ? 1 : R <= kFewRows ? 2 : 0;
    p.nrb = p.nt ? 1 : (int)((R + kChunkRows - 1) / kChunkRows);
    const int64_t units = p.units = (int64_t)B * c->Hkv * p.nrb;
    if (p.nt == 0) {
        if (splits) {
            const int64_t least = least_splits(span);
            p.whole = 0, p.S = (int)(splits < least ? least : splits);
            if (p.S == 1) p.whole = units;
        } else {
            chunk_splits(c, units, span, &p.whole, &p.S);
        }
        p.join = p.S > 1;
        const int64_t by_unit = (units - p.whole) * kChunkRows, by_row = (int64_t)total_q * c->Hq;
        p.by_unit = by_unit < by_row;
        p.part_rows = p.by_unit ? by_unit : by_row;
        return p;
    }
    p.cluster = false;
    const int64_t per = (span + kUnit - 1) / kUnit + 1;  // units of one, at most
    if (!splits) {
        // clusters where they fill no more than a wave and no block gets over 512 tokens
        int C = 8;
        while (C > 1 && (units * C > 2 * kSms || C / 2 >= per)) C /= 2;
        if (units * C <= 2 * kSms && per <= 8 * C) {
            p.cluster = true, p.S = C, p.join = false;
            return p;
        }
    }
    // two blocks are resident on an SM: one wave of equal shares, or fewer where there are not
    // that many units of 64 tokens
    const int64_t most = units * per;
    int64_t N = splits ? units * splits : 2 * kSms;
    if (N > most) N = most;
    const int64_t share = (int64_t)(p.nt == 1 ? kWarps<1> : kWarps<2>) * kWarpTokens;
    if (per * kUnit > share && N < (most * kUnit + share - 1) / share) N = (most * kUnit + share - 1) / share;
    p.S = (int)(N > (1 << 20) ? 1 << 20 : N);
    p.join = span > kUnit && !(splits == 1 && B == 1 && p.S == units);
    return p;
}

// Records of k_paged_attn for k_paged_join: one per (request, kv head), or per block if those are
// fewer.
int64_t records(const kvq_paged_cfg* cfg, const Plan& p, int32_t B) {
    const int64_t segs = (int64_t)B * cfg->Hkv;
    return segs < p.S ? segs : p.S;
}

// What a call needs.
size_t ws_bytes(const kvq_paged_cfg* cfg, const Plan& p, int32_t B) {
    if (!p.join) return 0;
    if (p.nt == 0) return (size_t)p.S * p.part_rows * (cfg->D + 2) * 4;
    return (size_t)(2 * p.S) * 8 * p.nt * (cfg->D + 2) * 4 + (size_t)records(cfg, p, B) * 16;
}

// What the query answers: what the call needs or, for chunks by the library's choice, a bound that
// grows with every size, so that it also serves whatever is smaller (a few rows' calls among it;
// those grow with the sizes by themselves).  A split unit's blocks number kCutBlocks at most, or
// the least that the tokens ask for.
size_t ws_query(const kvq_paged_cfg* cfg, int B, int total_q, int max_q, int max_len, int splits) {
    const Plan p = plan_of(cfg, B, total_q, max_q, max_len, splits, 0);
    if (p.nt || splits) return ws_bytes(cfg, p, B);
    const int64_t by_unit = p.units * kChunkRows, by_row = (int64_t)total_q * cfg->Hq;
    const int64_t tiles = ((int64_t)max_len + 127) / 128, most = tiles < kSms ? tiles : kSms;
    const int64_t all = by_unit < by_row ? by_unit : by_row;
    int64_t rows = kCutBlocks * kChunkRows;
    if (most < 2) rows = 0;
    else if (all < rows && all * most < rows) rows = all * most;
    const int64_t least = least_splits(max_len);
    if (least > 1 && all * least > rows) rows = all * least;
    size_t bytes = (size_t)rows * (cfg->D + 2) * 4;
    const int G = cfg->Hq / cfg->Hkv;
    if (G <= kFewRows) {
        const size_t few = ws_bytes(cfg, plan_of(cfg, B, total_q, kFewRows / G, max_len, 0, 0), B);
        if (few > bytes) bytes = few;
    }
    return bytes;
}

// Few rows: the main kernel, and the join where a (request, kv head) may have been cut.
template <int D, int NT, bool BF>
int run_few(const AttnArgs& a, const Plan& p, int B, int rows, cudaStream_t st) {
    using L = FewSmem<D, NT>;
    if (p.cluster) {
        auto* kern = k_paged_attn<D, NT, BF, true>;
        static SmemOptIn opt;
        if (int e = opt.set((const void*)kern, L::total)) return e;
        return launch_overlapped(kern, dim3((unsigned)(p.S * B * a.c.Hkv)), kFewThreads<NT>, L::total, p.S, st, a, B);
    }
    auto* kern = k_paged_attn<D, NT, BF, false>;
    static SmemOptIn opt;
    if (int e = opt.set((const void*)kern, L::total)) return e;
    const int e = launch_overlapped(kern, dim3(p.S), kFewThreads<NT>, L::total, 1, st, a, B);
    if (e || !p.join || p.S == 1) return e;
    return launch_overlapped(k_paged_join<D, BF>, dim3((unsigned)records(&a.c, p, B), rows), kJoinWarps * 32, 0, 1, st, a, L::RB);
}

int check_sizes(const kvq_paged_cfg* cfg, int32_t B, int32_t total_q, int32_t max_q,
                int32_t max_len, int32_t splits) {
    if (B < 1 || B > 65535 || total_q < 0 || max_q < 1 || max_q > (1 << 24) || max_len < 1)
        return KVQ_ERR_SHAPE;
    if (splits < 0 || splits > 256) return KVQ_ERR_RANGE;
    return KVQ_OK;
}

}  // namespace

extern "C" {

int kvq_paged_attention_workspace(const kvq_paged_cfg* cfg, int32_t B, int32_t total_q,
                                  int32_t max_q, int32_t max_len, int32_t splits, size_t* bytes) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!bytes) return KVQ_ERR_NULL;
    if ((e = check_sizes(cfg, B, total_q, max_q, max_len, splits))) return e;
    *bytes = ws_query(cfg, B, total_q, max_q, max_len, splits);
    return KVQ_OK;
}

int kvq_paged_attention(const kvq_paged_cfg* cfg, const kvq_paged_cache* cache, const void* q,
                        int64_t q_stride, const int32_t* cu_q, int32_t B, int32_t total_q,
                        const int32_t* len, const int32_t* block_table, int32_t max_q,
                        int32_t max_len, float sm_scale, int32_t window, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, int32_t splits, void* stream) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if ((e = check_paged_cache(cache))) return e;
    if ((e = check_sizes(cfg, B, total_q, max_q, max_len, splits))) return e;
    const float scale_log2 = (float)ldexp((double)sm_scale * 1.4426950408889634, cfg->k_exp);
    if (window < 0 || !isfinite(scale_log2)) return KVQ_ERR_RANGE;
    if (!cu_q && (total_q != B || max_q != 1)) return KVQ_ERR_SHAPE;
    if (total_q == 0) return KVQ_OK;
    if (!q || !len || !block_table || !out) return KVQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || (q_stride & 7)) return KVQ_ERR_ALIGN;
    if (q_stride < (int64_t)cfg->Hq * cfg->D) return KVQ_ERR_SHAPE;
    const Plan p = plan_of(cfg, B, total_q, max_q, max_len, splits, window);
    // blocks of the chunk kernel and of its merge
    const int64_t per_unit = !p.join ? 1 : p.S > kChunkRows / kMergeWarps ? p.S : kChunkRows / kMergeWarps;
    if (p.nt == 0 && p.units * per_unit > INT32_MAX) return KVQ_ERR_RANGE;
    const size_t need = ws_bytes(cfg, p, B);
    if (need > 0) {
        if (!workspace) return KVQ_ERR_NULL;
        if (!aligned16(workspace)) return KVQ_ERR_ALIGN;
        if (workspace_bytes < need) return KVQ_ERR_WORKSPACE;
    }
    AttnArgs a{};
    a.c = *cfg;
    a.pool = cache->pool;
    a.status = cache->status;
    a.q = (const uint16_t*)q;
    a.qs = q_stride;
    a.cu = cu_q, a.len = len, a.table = block_table;
    a.out = (uint16_t*)out;
    a.lse = lse;
    a.part = (float*)workspace;
    const size_t prow = p.nt ? (size_t)2 * p.S * 8 * p.nt : (size_t)p.S * p.part_rows;
    if (p.join) {
        a.pml = (float2*)(a.part + prow * cfg->D);
        if (p.nt) {
            a.rec = (int4*)(a.pml + prow);
            a.by_request = (int64_t)B * cfg->Hkv <= p.S;
        }
    }
    a.total_q = total_q, a.max_q = max_q, a.max_len = max_len, a.window = window, a.S = p.S;
    a.scale_log2 = scale_log2;
    a.out_scale = ldexpf(1.0f, cfg->v_exp);
    const bool bf = cfg->dtype == KVQ_BF16;
    cudaStream_t st = (cudaStream_t)stream;
    if (p.nt == 0) {
        a.whole = (int)p.whole, a.B = B, a.nrb = p.nrb;
        a.part_rows = p.part_rows, a.by_unit = p.by_unit;
        if ((e = run_chunk(a, st))) return e;
        if (p.join) {
            auto* mk = cfg->D == 64 ? (bf ? k_paged_merge<64, true> : k_paged_merge<64, false>)
                                    : (bf ? k_paged_merge<128, true> : k_paged_merge<128, false>);
            return launch_overlapped(mk, dim3((unsigned)((p.units - p.whole) * (kChunkRows / kMergeWarps))), kMergeWarps * 32, 0, 1, st, a);
        }
        return KVQ_OK;
    }
    const int rows = max_q * (cfg->Hq / cfg->Hkv);
    if (cfg->D == 64)
        return p.nt == 1 ? (bf ? run_few<64, 1, true>(a, p, B, rows, st) : run_few<64, 1, false>(a, p, B, rows, st))
                         : (bf ? run_few<64, 2, true>(a, p, B, rows, st) : run_few<64, 2, false>(a, p, B, rows, st));
    return p.nt == 1 ? (bf ? run_few<128, 1, true>(a, p, B, rows, st) : run_few<128, 1, false>(a, p, B, rows, st))
                     : (bf ? run_few<128, 2, true>(a, p, B, rows, st) : run_few<128, 2, false>(a, p, B, rows, st));
}

}  // extern "C"
