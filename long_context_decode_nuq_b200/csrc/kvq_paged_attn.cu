// Attention over the paged 4-bit cache: one token, a few or a chunk of them per request.
#include "kvq_paged_attn.cuh"

using namespace kvq;
using namespace kvq_host;

namespace {

// ---------------------------------------------------------------------------------
// A block takes RB = 8 * NT query rows of one (request, kv head) -- row r is query r / G, head
// r % G of the kv head's G -- and one split of the tokens they see.  Each warp walks tiles of 32
// tokens of its own (a ring of bulk copies, a group of 16 tokens is one contiguous run of the
// pool), keeps the running maximum and sum of its rows, and the block joins its warps at the end.
//
// Both products run on the tensor cores with the tokens as the long side, so one m16n8k16
// instruction serves 16 tokens for 8 rows and a single query head wastes only idle columns:
//   S^T [16 tokens x 8 rows] = K [16 x D] q^T,   O^T [D x 8 rows] += V^T [D x 16] P^T.
// Codes convert two at a time to fp16 and are multiplied by their scale there: the product has 6
// significant bits and a size of 2^-10 .. 2688, so K and V enter exactly.  A bf16 query enters as
// fp16 too: each row is divided by a power of two that puts its largest value at 2^10, which
// leaves every value within 2^-35 of the row's largest exact.  Only P is rounded, to fp16 (half a
// step is 2^-11); it is kept at up to 2^15 of the largest so that tokens 2^-26 below the maximum still have all
// their bits.  Maximum, sums and O are binary32.
//
// The rows of a K tile are permuted (tau) so that both the 16-byte reads of K rows and the 8-byte
// reads of V rows spread over the banks; S^T then leaves its lanes with (token, 2 rows), which
// movmatrix turns into the B operand of the second product.
constexpr int kTile = 32;

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
struct Shape {
    static constexpr int W = NT == 1 ? 8 : 4;   // warps
    static constexpr int ST = NT == 1 ? 3 : 4;  // ring stages per warp
};
template <int D, int NT>
constexpr int attn_smem() {
    constexpr int ring = Shape<NT>::W * Shape<NT>::ST * 2 * Paged<D>::kBytes;
    constexpr int join = Shape<NT>::W * 8 * NT * (D + 4 + 2) * 4;
    return (ring > join ? ring : join) + 8 * Shape<NT>::W * Shape<NT>::ST;
}

template <int D, int NT, bool BF>
__global__ void __launch_bounds__(Shape<NT>::W * 32, NT == 1 ? 2 : 1)
    k_paged_attn(const AttnArgs a) {
    constexpr int W = Shape<NT>::W, ST = Shape<NT>::ST, RB = 8 * NT;
    constexpr int GB = Paged<D>::kBytes, HALF = Paged<D>::kHalf, ROW = Paged<D>::kRow, SC = Paged<D>::kScales;
    constexpr int KS = D / 16;  // k-steps of S^T, and 16-channel tiles of O^T
    constexpr int KW = D / 32;  // code words of a lane's part of a K row
    constexpr int VW = D / 64;  // code words of a lane's part of a V row
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int s = blockIdx.x % a.S, rb = blockIdx.x / a.S, h = blockIdx.y, b = blockIdx.z;
    const int G = a.c.Hq / a.c.Hkv, P = a.c.page_tokens;
    const Rows rw = rows_of(a, b);
    const int r0 = rb * RB;
    if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0 && (rw.n > rw.nq || rw.len > rw.kv))
        set_status(a.status, KVQ_STATUS_LEN_OVERFLOW);
    if (r0 >= rw.R) return;
    const int i0 = r0 / G, i1 = (min(r0 + RB, rw.R) - 1) / G;
    const int first = rw.len - rw.n;  // position of query 0 (negative: it sees nothing)
    const int hi = min(rw.kv, first + i1 + 1);
    const int lo = a.window > 0 ? max(0, first + i0 + 1 - a.window) : 0;
    const int all_hi = min(rw.kv, first + i0 + 1);  // tokens every row sees: [all_lo, all_hi)
    const int all_lo = a.window > 0 ? max(0, first + i1 + 1 - a.window) : 0;
    const int tbase = lo & ~(kTile - 1);
    const int tiles = hi > lo ? (hi - tbase + kTile - 1) / kTile : 0;
    const int te = (int)((int64_t)tiles * (s + 1) / a.S);
    const int tb = (int)((int64_t)tiles * s / a.S) + warp;

    uint8_t* ring = smem + warp * ST * 2 * GB;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + attn_smem<D, NT>() - 8 * W * ST) + warp * ST;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    __syncwarp();

    // loader: lanes 0 and 1 each bring one group of a tile; a page number read one tile ahead
    const int32_t* tab = a.table + (size_t)b * a.c.max_pages;
    auto page_of = [&](int tile) {
        const int tg = tbase + tile * kTile + lane * kGroup;
        return lane < 2 && tile < te && tg < hi && tg + kGroup > lo ? tab[tg / P] : -1;
    };
    uint32_t have = 0;  // two bits a stage: groups that were brought
    auto issue = [&](int stage, int tile, int page) {
        const int tg = tbase + tile * kTile + lane * kGroup;
        const bool want = lane < 2 && tile < te && tg < hi && tg + kGroup > lo;
        const bool ok = want && page >= 0 && page < a.c.num_pages;
        if (want && !ok) set_status(a.status, KVQ_STATUS_BAD_PAGE);
        const uint32_t v = __ballot_sync(0xffffffffu, ok);
        have = (have & ~(3u << (2 * stage))) | v << (2 * stage);
        if (lane == 0) mbar_arrive_expect_tx(&bar[stage], __popc(v) * GB);
        __syncwarp();
        if (ok)
            bulk_load(ring + (stage * 2 + lane) * GB, a.pool + group_at(a.c, page, h, tg % P / kGroup), GB, &bar[stage]);
    };
    int issued = 0;
    for (; issued < ST && tb + issued * W < te; ++issued) issue(issued, tb + issued * W, page_of(tb + issued * W));
    int next_page = page_of(tb + issued * W);

    // queries: lane (g, t) holds channels [t*D/4, (t+1)*D/4) of row g, as the columns of B
    uint32_t qf[NT][KS][2];
    float sl2[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 8 + g;
        uint32_t w[KS * 2] = {};
        if (r < rw.R) {
            const uint16_t* src = a.q + (int64_t)(rw.c0 + r / G) * a.qs + (h * G + r % G) * D + t * (D / 4);
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
                const uint4 x = reinterpret_cast<const uint4*>(src)[i];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        }
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
        for (int j = 0; j < KS; ++j) qf[nt][j][0] = w[2 * j], qf[nt][j][1] = w[2 * j + 1];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int er = __shfl_sync(0xffffffffu, e, (2 * t + z) * 4);
            sl2[nt][z] = a.scale_log2 * __uint_as_float((uint32_t)(127 + er) << 23);
            pos[nt][z] = first + (r0 + nt * 8 + 2 * t + z) / G;
        }
    }

    float o[NT][KS][4] = {}, m[NT][2], l[NT][2] = {};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY;
    const int tau = (g & 1) ? 4 + ((g >> 1) ^ 1) : (g >> 1);
    const int tv[4] = {t, 4 + (t ^ 1), 8 + t, 12 + (t ^ 1)};
    bool dead = false;

    int k = 0;
    for (int tile = tb; tile < te; tile += W, ++k) {
        const int stage = k % ST;
        dead = !__all_sync(0xffffffffu, mbar_wait(&bar[stage], (k / ST) & 1));
        if (dead) break;
        const uint8_t* buf = ring + stage * 2 * GB;
        const int t0 = tbase + tile * kTile;
        const uint32_t got = have >> (2 * stage) & 3u;
        const bool mask = got != 3u || t0 + kTile > all_hi || t0 < all_lo;

        float sc[2][NT][4];
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
            const uint8_t* kb = buf + gr * GB;
            uint32_t kc[2][KW];
            uint32_t ks[2][(D + 127) / 128 * 2];  // scale pairs (s, s) of the lane's channels
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
                    const uint32_t s0 = ks[0][w * 2 / KW], s1 = ks[1][w * 2 / KW];
                    const uint32_t A[4] = {hmul2(x0[2 * u], s0), hmul2(x1[2 * u], s1),
                                           hmul2(x0[2 * u + 1], s0), hmul2(x1[2 * u + 1], s1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(sc[gr][nt], A, qf[nt][2 * w + u][0], qf[nt][2 * w + u][1]);
                }
            }
        }
        // scores in the log2 domain; masked ones are -inf
        float tm[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            tm[nt][0] = tm[nt][1] = -INFINITY;
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    float x = sc[gr][nt][z] * sl2[nt][z & 1];
                    if (mask) {
                        const int tok = t0 + gr * kGroup + tau + (z & 2) * 4;
                        const int p = pos[nt][z & 1];
                        const bool see = (got >> gr & 1u) && tok < rw.kv && tok <= p &&
                                         (a.window <= 0 || tok > p - a.window);
                        if (!see) x = -INFINITY;
                    }
                    sc[gr][nt][z] = x;
                    tm[nt][z & 1] = fmaxf(tm[nt][z & 1], x);
                }
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                tm[nt][z] = fmaxf(tm[nt][z], __shfl_xor_sync(0xffffffffu, tm[nt][z], 4));
                tm[nt][z] = fmaxf(tm[nt][z], __shfl_xor_sync(0xffffffffu, tm[nt][z], 8));
                tm[nt][z] = fmaxf(tm[nt][z], __shfl_xor_sync(0xffffffffu, tm[nt][z], 16));
                grow |= tm[nt][z] - m[nt][z] > kPRoom;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float mn = fmaxf(m[nt][z], tm[nt][z] - kPShift);
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
            const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
            const float m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                const float p0 = ex2(sc[gr][nt][0] - m0), p1 = ex2(sc[gr][nt][1] - m1);
                const float p2 = ex2(sc[gr][nt][2] - m0), p3 = ex2(sc[gr][nt][3] - m1);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pf[gr][nt][0] = transpose8x8(pack_h2(p0, p1));
                pf[gr][nt][1] = transpose8x8(pack_h2(p2, p3));
            }
        }
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
            const uint8_t* vb = buf + gr * GB + HALF;
            const uint8_t* vs = vb + kGroup * ROW + g * (D / 8) / kGroup;
            uint32_t sb[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) sb[z] = vs[tv[z] * SC];
            if (mask) {
                // bytes nobody wrote may hold a NaN scale, and 0 * NaN is not 0
                const int tg = t0 + gr * kGroup;
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (!(got >> gr & 1u) || tg + tv[z] >= rw.kv) sb[z] = 0;
            }
            const uint32_t s01 = e4m3x2(sb[0] | sb[1] << 8), s23 = e4m3x2(sb[2] | sb[3] << 8);
            uint32_t vc[4][VW];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint8_t* row = vb + tv[z] * ROW + g * (D / 16);
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(row);
                    vc[z][0] = x.x, vc[z][1] = x.y;
                } else {
                    vc[z][0] = *reinterpret_cast<const uint32_t*>(row);
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // bytes of (token a, token b) codes of one channel: even channels, then odd ones
                uint32_t e01[4], o01[4], e23[4], o23[4];
                e2m1x8((vc[0][w] & 0x0f0f0f0fu) | (vc[1][w] << 4 & 0xf0f0f0f0u), e01);
                e2m1x8((vc[0][w] >> 4 & 0x0f0f0f0fu) | (vc[1][w] & 0xf0f0f0f0u), o01);
                e2m1x8((vc[2][w] & 0x0f0f0f0fu) | (vc[3][w] << 4 & 0xf0f0f0f0u), e23);
                e2m1x8((vc[2][w] >> 4 & 0x0f0f0f0fu) | (vc[3][w] & 0xf0f0f0f0u), o23);
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
        if (tile + ST * W < te) {
            issue(stage, tile + ST * W, next_page);
            next_page = page_of(tile + (ST + 1) * W);
            ++issued;
        }
    }
    if (dead) {  // a copy did not come: say so, and let the others land before the memory is left
        set_status(a.status, KVQ_STATUS_WAIT_TIMEOUT);
        drain_chunks(bar, k, issued, ST);
    }

    // join the warps: rows' (m, l) and O through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[nt][z] += __shfl_xor_sync(0xffffffffu, l[nt][z], x);
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);  // [W][RB][D + 4]
    float2* sml = reinterpret_cast<float2*>(so + W * RB * (D + 4));  // [W][RB]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int row = nt * 8 + 2 * t + z;
            float* dst = so + (warp * RB + row) * (D + 4) + g * (D / 8);
#pragma unroll
            for (int j = 0; j < KS; j += 2)  // tiles j: channels 2j, 2j + 1 of the lane's D/8
                *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][z], o[nt][j][z + 2], o[nt][j + 1][z], o[nt][j + 1][z + 2]);
            if (g == 0) sml[warp * RB + row] = make_float2(m[nt][z], l[nt][z]);
        }
    __syncthreads();
    const int64_t nrow = (int64_t)a.total_q * a.c.Hq;
    for (int it = threadIdx.x; it < RB * (D / 4); it += W * 32) {
        const int row = it / (D / 4), c4 = it % (D / 4) * 4, r = r0 + row;
        if (r >= rw.R) break;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sml[w * RB + row].x);
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 ml = sml[w * RB + row];
            const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
            const float4 x = *reinterpret_cast<const float4*>(so + (w * RB + row) * (D + 4) + c4);
            L += f * ml.y;
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
        const int64_t grow = (int64_t)(rw.c0 + r / G) * a.c.Hq + h * G + r % G;
        if (a.S == 1) {
            const float inv = L == 0.0f ? 0.0f : a.out_scale / L;
            store4<BF>(a.out + grow * D + c4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (c4 == 0 && a.lse) a.lse[grow] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
        } else {
            *reinterpret_cast<float4*>(a.part + (s * nrow + grow) * D + c4) = acc;
            if (c4 == 0) a.pml[s * nrow + grow] = make_float2(M, L);
        }
    }
}

// Joins the splits of a row, in split order: a warp per row.
constexpr int kMergeWarps = 4;
template <int D, bool BF>
__global__ void __launch_bounds__(kMergeWarps * 32) k_paged_merge(const AttnArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int G = a.c.Hq / a.c.Hkv;
    const Rows rw = rows_of(a, b);
    const int64_t nrow = (int64_t)a.total_q * a.c.Hq;
    const int r = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (r >= rw.R) return;
    const int64_t grow = (int64_t)(rw.c0 + r / G) * a.c.Hq + h * G + r % G;
    float M = -INFINITY;
    for (int s = lane; s < a.S; s += 32) M = fmaxf(M, a.pml[s * nrow + grow].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float L = 0.0f, acc[D / 32] = {};
    for (int s = 0; s < a.S; ++s) {
        const float2 ml = a.pml[s * nrow + grow];
        if (ml.y == 0.0f) continue;  // an empty split; one of NaN scores has m = -inf, l = NaN
        const float f = ex2(ml.x - M);
        const float* x = a.part + (s * nrow + grow) * D + lane * (D / 32);
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
// Host: which kernel, rows per block, splits.
struct Plan {
    int nt;  // 8-row tiles of a block of k_paged_attn; 0: the chunk kernel
    int nrb, S;
};

constexpr int kSms = 148;
// More rows of a kv head than this go to the chunk kernel.
constexpr int kFewRows = 32;

// Splits of the chunk kernel: the least time of a model in which a block costs 6 us and 1.2 us per
// 128 tokens, blocks run one per SM in waves, and a split writes and reads its part at 5 TB/s.
int chunk_splits(const kvq_paged_cfg* c, int64_t units, int64_t tiles) {
    int best = 1;
    double least = 1e30;
    for (int S = 1; S <= 32 && S <= tiles; ++S) {
        const int64_t waves = (units * S + kSms - 1) / kSms;
        double t = (double)waves * (6.0 + 1.2 * (double)((tiles + S - 1) / S));
        if (S > 1) t += 4.0 + (double)units * S * kChunkRows * c->D * 8 / 5e6;
        if (t < 0.98 * least) least = t, best = S;
    }
    return best;
}

int splits_of(const kvq_paged_cfg* c, const Plan& p, int B, int64_t span) {
    const int64_t units = (int64_t)B * c->Hkv * p.nrb;
    if (p.nt == 0) return chunk_splits(c, units, (span + 127) / 128);
    // the tokens a row block can see bound the useful splits at a tile a warp
    const int warps = p.nt == 1 ? 8 : 4;
    const int64_t tiles = (span + kTile - 1) / kTile;
    int64_t S = (kSms * 4 + units - 1) / units;
    const int64_t most = (tiles + warps - 1) / warps;
    if (S > most) S = most;
    return (int)(S > 256 ? 256 : S < 1 ? 1 : S);
}

Plan plan_of(const kvq_paged_cfg* c, int B, int max_q, int max_len, int splits, int window) {
    const int64_t R = (int64_t)max_q * (c->Hq / c->Hkv);
    Plan p;
    p.nt = R <= 8 ? 1 : R <= 16 ? 2 : R <= kFewRows ? 4 : 0;
    const int rows = p.nt ? 8 * p.nt : kChunkRows;
    p.nrb = (int)((R + rows - 1) / rows);
    p.S = splits ? splits : splits_of(c, p, B, max_len);
    if (!splits && window > 0 && max_len > (int64_t)window + max_q + 128) {
        // a window only lowers the splits: the workspace is sized without it
        const int S = splits_of(c, p, B, (int64_t)window + max_q + 128);
        if (S < p.S) p.S = S;
    }
    return p;
}

using AttnKernel = void (*)(AttnArgs);

template <int D, bool BF>
AttnKernel attn_kernel(int nt, int* smem, int* warps) {
    *warps = nt == 1 ? 8 : 4;
    *smem = nt == 1 ? attn_smem<D, 1>() : nt == 2 ? attn_smem<D, 2>() : attn_smem<D, 4>();
    return nt == 1 ? k_paged_attn<D, 1, BF> : nt == 2 ? k_paged_attn<D, 2, BF> : k_paged_attn<D, 4, BF>;
}

int check_sizes(const kvq_paged_cfg* cfg, int32_t B, int32_t total_q, int32_t max_q,
                int32_t max_len, int32_t splits) {
    if (B < 1 || B > 65535 || total_q < 0 || max_q < 1 || max_q > (1 << 24) || max_len < 1)
        return KVQ_ERR_SHAPE;
    if (splits < 0 || splits > 256) return KVQ_ERR_RANGE;
    return KVQ_OK;
}

// The workspace is sized without the window, which only lowers the splits the library chooses.
size_t ws_bytes(const kvq_paged_cfg* cfg, const Plan& p, int32_t total_q) {
    if (p.S == 1) return 0;
    return (size_t)p.S * total_q * cfg->Hq * (cfg->D + 2) * 4;
}

}  // namespace

extern "C" {

int kvq_paged_attention_workspace(const kvq_paged_cfg* cfg, int32_t B, int32_t total_q,
                                  int32_t max_q, int32_t max_len, int32_t splits, size_t* bytes) {
    int e = check_paged_cfg(cfg);
    if (e) return e;
    if (!bytes) return KVQ_ERR_NULL;
    if ((e = check_sizes(cfg, B, total_q, max_q, max_len, splits))) return e;
    *bytes = ws_bytes(cfg, plan_of(cfg, B, max_q, max_len, splits, 0), total_q);
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
    if (window < 0 || !isfinite(sm_scale)) return KVQ_ERR_RANGE;
    if (!cu_q && (total_q != B || max_q != 1)) return KVQ_ERR_SHAPE;
    if (total_q == 0) return KVQ_OK;
    if (!q || !len || !block_table || !out) return KVQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || (q_stride & 7)) return KVQ_ERR_ALIGN;
    if (q_stride < (int64_t)cfg->Hq * cfg->D) return KVQ_ERR_SHAPE;
    const Plan p = plan_of(cfg, B, max_q, max_len, splits, window);
    if ((int64_t)p.S * p.nrb > INT32_MAX) return KVQ_ERR_RANGE;
    const size_t need = ws_bytes(cfg, p, total_q);
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
    a.pml = (float2*)(a.part + (size_t)p.S * total_q * cfg->Hq * cfg->D);
    a.total_q = total_q, a.max_q = max_q, a.max_len = max_len, a.window = window, a.S = p.S;
    a.scale_log2 = (float)ldexp((double)sm_scale * 1.4426950408889634, cfg->k_exp);
    a.out_scale = ldexpf(1.0f, cfg->v_exp);
    const bool bf = cfg->dtype == KVQ_BF16;
    cudaError_t ce;
    cudaStream_t st = (cudaStream_t)stream;
    if (p.nt == 0) {
        if ((e = run_chunk(a, p.nrb, B, st))) return e;
    } else {
    int smem, warps;
    const AttnKernel kern = cfg->D == 64 ? (bf ? attn_kernel<64, true>(p.nt, &smem, &warps)
                                               : attn_kernel<64, false>(p.nt, &smem, &warps))
                                         : (bf ? attn_kernel<128, true>(p.nt, &smem, &warps)
                                               : attn_kernel<128, false>(p.nt, &smem, &warps));
    ce = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (ce) return record_cuda(ce);
    kern<<<dim3((unsigned)(p.S * p.nrb), cfg->Hkv, B), warps * 32, smem, st>>>(a);
    if ((ce = cudaGetLastError())) return record_cuda(ce);
    }
    if (p.S > 1) {
        auto* mk = cfg->D == 64 ? (bf ? k_paged_merge<64, true> : k_paged_merge<64, false>)
                                : (bf ? k_paged_merge<128, true> : k_paged_merge<128, false>);
        const int64_t R = (int64_t)max_q * (cfg->Hq / cfg->Hkv);
        mk<<<dim3((unsigned)((R + kMergeWarps - 1) / kMergeWarps), cfg->Hkv, B), kMergeWarps * 32, 0, st>>>(a);
        return record_cuda(cudaGetLastError());
    }
    return KVQ_OK;
}

}  // extern "C"
