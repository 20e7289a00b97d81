// Attention of prompt chunks (and of many rows of any kind) over the paged 4-bit cache.
#include "kvq_paged_attn.cuh"

using namespace kvq;
using namespace kvq_host;

namespace {

// ---------------------------------------------------------------------------------
// A block takes 256 query rows of one (request, kv head), as two tiles of 128, and all of the
// tokens they see or, for the units that would not fill a last wave, one split of them, 128 tokens
// at a time.  Tensor memory holds, per tile, the scores S [128 x
// 128] and O [128 x D] in binary32; P overwrites S as fp16 and is the second product's operand
// from there.  Roles, by warp:
//   0-3, 4-7   softmax of a row tile, a thread a row: scores out of tensor memory, maximum, e^x,
//              P back; the maximum moves only when it has grown by 2^3, so O is seldom rescaled
//   8-11       codes to fp16 in shared memory (a 128-byte swizzled tile of K or V, four slots)
//   12         bulk copies of the codes, a lane a group of 16 tokens, three tiles ahead
//   13         one thread issues the products:  S_i = Q_i K^T,  O_i += P_i V
// The two row tiles alternate, so one's softmax runs under the other's products, and each
// dequantized tile serves both: 32768 conversions feed 2 x 128 x 128 x D x 2 multiply-adds.
// The arithmetic is that of the few-row kernel: K and V exact in fp16, the query exact as fp16
// with its row's power of two taken out, P rounded to fp16 at 2^12 .. 2^15 of its row's largest.
// Products of one block run in the order they are issued, which is what lets S_i of the next
// tokens be issued behind the product that still reads P_i from the same columns.
//
// Bound by the round trip between products and softmax: a step takes about 3700 cycles, 2048 of
// them products; without the exponentials it would be 5 % less, without the conversions 11 %.
// 2048 queries against 32768 tokens, 32/8 heads of 128: 1017 us at the power limit, 1.05 PFLOP/s
// (63 % of a measured library product's rate in a short run, 74 % of its sustained one); 933 in runs
// too short to reach that limit.  Sixteen softmax warps of half a row each were slower (1187 against
// 1083 us in runs of their time), as were P in quarters (1061 against 1015) and part of the
// exponentials on the multiply-add pipe (1034 against 1017).
constexpr int kRows = kChunkRows;   // 2 tiles of 128
constexpr int kTok = 128;           // tokens a step
constexpr int kSlots = 4;           // K or V tiles in shared memory
constexpr int kRaw = 3;             // code tiles (of K or V) in flight
constexpr int kThreads = 512;
constexpr uint32_t kPollLimit = 1u << 22;
// registers per thread after the split; their sum over the four warpgroups stays within the
// launch's 4 x 128
constexpr int kRegSoft = 184, kRegDeq = 96, kRegIssue = 48;

template <int D>
struct Smem {
    static constexpr int q = 0;                              // [D/64][256][128 B] swizzled
    static constexpr int slot = kRows * D * 2;               // [kSlots][D/64][128][128 B] swizzled
    static constexpr int slot_bytes = kTok * D * 2;
    static constexpr int raw = slot + kSlots * slot_bytes;   // [kRaw][8 groups]: keys or values
    static constexpr int raw_bytes = kTok / kGroup * Paged<D>::kHalf;
    static constexpr int bar = raw + kRaw * raw_bytes;
    static constexpr int n_bar = 2 * kRaw + 2 * kSlots + 9;
    static constexpr int misc = bar + 8 * n_bar;             // tmem address, dead flag, group masks
    static constexpr int total = misc + 64;
};

__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* dead) {
    for (uint32_t it = 0; it < kPollLimit; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u && *dead) return false;
    }
    *dead = 1;
    return false;
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)(addr >> 4 & 0x3fffu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           1ull << 46 | 2ull << 61;  // 128-byte swizzle
}
// fp16 operands, binary32 accumulator, 128 rows; b_mn: B's columns are contiguous
constexpr uint32_t mma_desc(int n, bool b_mn) {
    return 1u << 4 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 32 or 64 columns of the warp's 32 lanes, from and to tensor memory.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
          "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t (&r)[64], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
          "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, "
          "%33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, "
          "%52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
          "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
          "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
          "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
          "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
          "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
          "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) k_paged_chunk(const AttnArgs a) {
    using L = Smem<D>;
    constexpr int GPT = kTok / kGroup;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::bar);
    uint64_t* raw_empty = raw_full + kRaw;
    uint64_t* kv_full = raw_empty + kRaw;
    uint64_t* kv_empty = kv_full + kSlots;
    uint64_t* s_full = kv_empty + kSlots;  // [2]
    uint64_t* p_full = s_full + 2;         // [2][2]: P's first and second 64 columns
    uint64_t* pv_done = p_full + 4;        // [2]
    uint64_t* q_full = pv_done + 2;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + L::misc);
    volatile int* dead = reinterpret_cast<volatile int*>(smem + L::misc + 4);
    uint8_t* gmask = smem + L::misc + 8;   // [8] groups that were brought, of the last 8 tiles

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cut = (int)blockIdx.x - a.whole, S = cut < 0 ? 1 : a.S, s = cut < 0 ? 0 : cut % S;
    const Unit unit = unit_of(a, cut < 0 ? (int)blockIdx.x : a.whole + cut / S);
    const int rb = unit.rb, h = unit.h, b = unit.b;
    const int G = a.c.Hq / a.c.Hkv, P = a.c.page_tokens;
    let_next();
    after_previous();
    const Rows rw = rows_of(a, b);
    const int r0 = rb * kRows;
    if (threadIdx.x == 0 && h == 0 && rb == 0 && s == 0 && (rw.n > rw.nq || rw.len > rw.kv))
        set_status(a.status, KVQ_STATUS_LEN_OVERFLOW);
    if (r0 >= rw.R) return;
    const int rows = min(kRows, rw.R - r0), nact = rows > 128 ? 2 : 1;
    const int i0 = r0 / G, i1 = (r0 + rows - 1) / G;
    const int first = rw.len - rw.n;
    const int hi = min(rw.kv, first + i1 + 1);
    const int lo = first_seen(a, first + i0);
    const int all_hi = min(rw.kv, first + i0 + 1);
    const int all_lo = first_seen(a, first + i1);
    const int tbase = lo & ~(kGroup - 1);
    const int tiles = hi > lo ? (hi - tbase + kTok - 1) / kTok : 0;
    const int tb = (int)((int64_t)tiles * s / S);
    const int n = (int)((int64_t)tiles * (s + 1) / S) - tb;  // steps of this block
    const int tok0 = tbase + tb * kTok;

    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (threadIdx.x == 0) {
        *dead = 0;
        for (int i = 0; i < kRaw; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 4);
        for (int i = 0; i < kSlots; ++i) mbar_init(&kv_full[i], 4), mbar_init(&kv_empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&pv_done[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
        mbar_init(q_full, 8);
        fence_mbar_init();
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;

    if (warp < 8) {
        regs_up<kRegSoft>();
        // queries: a thread a row, its power of two kept for the scores
        const int row = threadIdx.x;  // of the block
        const int r = r0 + row;
        uint4 in[D / 8] = {};
        if (r < rw.R) {
            const uint16_t* src = a.q + (int64_t)(rw.c0 + r / G) * a.qs + (h * G + r % G) * D;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) in[i] = reinterpret_cast<const uint4*>(src)[i];
        }
        int e = 0;
        if (BF) {
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(in[i].x & 0x7fff7fffu, in[i].y & 0x7fff7fffu), __vmaxu2(in[i].z & 0x7fff7fffu, in[i].w & 0x7fff7fffu)));
            const int eb = (int)(max(mx & 0xffffu, mx >> 16) >> 7);
            if (eb < 255) e = max(eb - 127 - 10, -120);
        }
        // a negative scale goes into the query, so that the largest score is the largest product
        const float f = __uint_as_float((uint32_t)(127 - e) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);
        const float sl2 = fmaxf(fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = pack_h2(lo16<BF>(w[z]) * f, hi16<BF>(w[z]) * f);
            *reinterpret_cast<uint4*>(smem + L::q + (i / 8) * (kRows * 128) + row * 128 + ((i % 8 ^ (row & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        float m = -INFINITY, l = 0.0f;
        const int i = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, in bits 16 and up
        const uint32_t st = tmem + lanes + i * 128, ot = tmem + lanes + 256 + i * D;
        const int pos = first + r / G;
        const int hi_r = min(rw.kv, pos + 1), lo_r = first_seen(a, pos);
        if (i < nact)
            for (int j = 0; j < n; ++j) {
                if (!__all_sync(0xffffffffu, wait_on(&s_full[i], j & 1, dead))) break;
                fence_after();
                // these scores are complete, and with them all that was issued before: K_j's slot
                // and V_(j-1)'s are free
                if (i == nact - 1 && (threadIdx.x & 127) == 0) {
                    mbar_arrive(&kv_empty[2 * j % kSlots]);
                    if (j > 0) mbar_arrive(&kv_empty[(2 * j - 1) % kSlots]);
                }
                uint32_t x[2][64];
                tmem_ld64(x[0], st);
                tmem_ld64(x[1], st + 64);
                const int t0 = tok0 + j * kTok;
                const uint32_t got = gmask[j & 7];
                if (got != 0xffu || t0 + kTok > all_hi || t0 < all_lo) {
#pragma unroll
                    for (int c = 0; c < kTok; ++c) {
                        const int t = t0 + c;
                        if (!(t < hi_r && t >= lo_r && (got >> (c / kGroup) & 1u))) x[c / 64][c % 64] = 0xff800000u;
                    }
                }
                float mx[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(x[0][c]);
#pragma unroll
                for (int c = 8; c < kTok; c += 16)
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                        const float y = __uint_as_float(x[c / 64][c % 64 + z]);
                        mx[z] = c + 8 < kTok ? fmaxf(mx[z], fmaxf(y, __uint_as_float(x[(c + 8) / 64 % 2][(c + 8) % 64 + z]))) : fmaxf(mx[z], y);
                    }
                const float tm = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl2;
                if (__any_sync(0xffffffffu, tm - m > kPRoom)) {
                    const float mn = fmaxf(m, tm - kPShift);
                    const float al = m == mn ? 1.0f : ex2(m - mn);
                    m = mn;
                    l *= al;
                    if (j > 0) {  // O is complete up to the step before, as S of this one is
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(o, ot + c);
#pragma unroll
                            for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * al);
                            tmem_st32(ot + c, o);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : -m;
                const unsigned long long sl2p = pk(sl2, sl2), nmp = pk(nm, nm);
                unsigned long long sum[2] = {0, 0};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const unsigned long long y = fma2(pk(__uint_as_float(x[half][2 * c]), __uint_as_float(x[half][2 * c + 1])), sl2p, nmp);
                        const f2 z = upk(y);
                        const float e0 = ex2(z.x), e1 = ex2(z.y);
                        sum[c & 1] = add2(sum[c & 1], pk(e0, e1));
                        p[c] = pack_h2(e0, e1);
                    }
                    tmem_st32(st + half * 32, p);
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * i + half]);
                }
                const f2 u = upk(sum[0]), v = upk(sum[1]);
                l += (u.x + u.y) + (v.x + v.y);
            }
        // the row's output
        if (i < nact && n > 0) {
            __all_sync(0xffffffffu, wait_on(&pv_done[i], 0, dead));
            fence_after();
        }
        const bool real = i < nact && r < rw.R;
        const int64_t grow = (int64_t)(rw.c0 + r / G) * a.c.Hq + h * G + r % G;
        const int64_t at = S > 1 ? part_at(a, s, cut / S, row, grow) : 0;
        const float inv = l == 0.0f ? 0.0f : a.out_scale / l;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (n > 0 && i < nact) {
                tmem_ld32(o, ot + c);
            } else {
#pragma unroll
                for (int z = 0; z < 32; ++z) o[z] = 0u;
            }
            // a row that saw nothing has P = 0 times finite values: O = 0 exactly
            if (!real) continue;
            if (S == 1) {
#pragma unroll
                for (int z = 0; z < 32; z += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        w[y] = pack16<BF>(__uint_as_float(o[z + 2 * y]) * inv, __uint_as_float(o[z + 2 * y + 1]) * inv);
                    *reinterpret_cast<uint4*>(a.out + grow * D + c + z) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int z = 0; z < 32; z += 4)
                    *reinterpret_cast<uint4*>(a.part + at * D + c + z) = make_uint4(o[z], o[z + 1], o[z + 2], o[z + 3]);
            }
        }
        if (real) {
            if (S > 1) a.pml[at] = make_float2(m, l);
            else if (a.lse) a.lse[grow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        fence_before();
    } else if (warp < 12) {
        regs_down<kRegDeq>();
        const int tid = threadIdx.x - 256;
        constexpr int LPR = D / 32;          // lanes of a token's row, 16 code bytes each
        constexpr int RPP = 128 / LPR;       // rows a pass
        const int q = tid % LPR, rr = tid / LPR;
        for (int seq = 0; seq < 2 * n; ++seq) {  // K_0, V_0, K_1, ...
            const int rs = seq % kRaw, slot = seq % kSlots, j = seq >> 1;
            const bool val = seq & 1;
            if (!__all_sync(0xffffffffu, wait_on(&raw_full[rs], (seq / kRaw) & 1, dead) &&
                                             wait_on(&kv_empty[slot], (seq / kSlots + 1) & 1, dead)))
                break;
            const uint32_t got = gmask[j & 7];
            const int t0 = tok0 + j * kTok;
            uint8_t* dst = smem + L::slot + slot * L::slot_bytes + (q >> 1) * (kTok * 128);
            const uint8_t* src = smem + L::raw + rs * L::raw_bytes;
#pragma unroll
            for (int pass = 0; pass < LPR; ++pass) {
                const int t = pass * RPP + rr;
                const uint8_t* g = src + (t / kGroup) * Paged<D>::kHalf;
                const uint4 c4 = *reinterpret_cast<const uint4*>(g + (t % kGroup) * Paged<D>::kRow + q * 16);
                uint32_t sc = *reinterpret_cast<const uint16_t*>(g + kGroup * Paged<D>::kRow + (t % kGroup) * Paged<D>::kScales + q * 2);
                // bytes nobody wrote may hold NaN scales; as values they must be 0
                if (val && (t0 + t >= rw.kv || !(got >> (t / kGroup) & 1u))) sc = 0;
                const uint32_t two = e4m3x2(sc);
                const uint32_t s2[2] = {__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232)};
                const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
                // the lanes of the second half of the channels go in another order, so that
                // eight lanes write eight different 16-byte columns
                const int flip = D == 128 ? (q >> 1) * 2 : 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t word = flip ? cw[w ^ 2] : cw[w];
                    const uint32_t sw = flip ? s2[(w ^ 2) / 2] : s2[w / 2];
                    uint32_t x[4];
                    e2m1x8(word, x);
                    const int chunk = 4 * (q & 1) + (w ^ flip);
                    *reinterpret_cast<uint4*>(dst + t * 128 + ((chunk ^ (t & 7)) << 4)) =
                        make_uint4(hmul2(x[0], sw), hmul2(x[1], sw), hmul2(x[2], sw), hmul2(x[3], sw));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&kv_full[slot]);
                mbar_arrive(&raw_empty[rs]);
            }
        }
    } else {
        regs_down<kRegIssue>();
        if (warp == 12) {
            const int32_t* tab = a.table + (size_t)b * a.c.max_pages;
            auto wanted = [&](int j) {
                const int tg = tok0 + j * kTok + lane * kGroup;
                return lane < GPT && j < n && tg < hi && tg + kGroup > lo;
            };
            auto page_of = [&](int j) { return wanted(j) ? tab[(tok0 + j * kTok + lane * kGroup) / P] : -1; };
            int page = page_of(0), next = page_of(1), seq = 0;
            for (; seq < 2 * n; ++seq) {
                const int rs = seq % kRaw, j = seq >> 1;
                if (!__all_sync(0xffffffffu, wait_on(&raw_empty[rs], (seq / kRaw + 1) & 1, dead))) break;
                const int tg = tok0 + j * kTok + lane * kGroup;
                const bool want = wanted(j), ok = want && page >= 0 && page < a.c.num_pages;
                if (want && !ok) set_status(a.status, KVQ_STATUS_BAD_PAGE);
                const uint32_t v = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) {
                    gmask[j & 7] = (uint8_t)v;
                    mbar_arrive_expect_tx(&raw_full[rs], __popc(v) * Paged<D>::kHalf);
                }
                __syncwarp();
                if (ok)
                    bulk_load(smem + L::raw + rs * L::raw_bytes + lane * Paged<D>::kHalf,
                              a.pool + group_at(a.c, page, h, tg % P / kGroup) + (seq & 1) * Paged<D>::kHalf,
                              Paged<D>::kHalf, &raw_full[rs]);
                if (seq & 1) page = next, next = page_of(j + 2);
            }
            if (*dead)  // let the copies in flight land before the memory is left
                for (int k = max(0, seq - kRaw); k < seq; ++k) mbar_wait(&raw_full[k % kRaw], (k / kRaw) & 1);
        } else if (warp == 13 && elect_one()) {
            constexpr uint32_t is = mma_desc(kTok, false), io = mma_desc(D, true);
            // an address enters a descriptor in units of 16 bytes, in its low bits
            const uint64_t qd = smem_desc(smem_u32(smem + L::q), 16, 1024);
            const uint64_t kd = smem_desc(smem_u32(smem + L::slot), 16, 1024);
            const uint64_t vd = smem_desc(smem_u32(smem + L::slot), kTok * 128, 1024);
            auto scores = [&](int i, int slot) {
                const uint64_t qi = qd + i * (128 * 128 / 16), ki = kd + slot * (L::slot_bytes / 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(tmem + i * 128, qi + ((k / 4) * (kRows * 128) + (k % 4) * 32) / 16,
                           ki + ((k / 4) * (kTok * 128) + (k % 4) * 32) / 16, is, k > 0);
                mma_commit(&s_full[i]);
            };
            auto values = [&](int i, int slot, int half, bool add) {
                const uint64_t vi = vd + slot * (L::slot_bytes / 16);
#pragma unroll
                for (int k = 4 * half; k < 4 * half + 4; ++k)
                    mma_ts(tmem + 256 + i * D, tmem + i * 128 + k * 8, vi + k * (2048 / 16), io, add || k > 0);
            };
            bool ok = n > 0 && wait_on(q_full, 0, dead) && wait_on(&kv_full[0], 0, dead);
            if (ok) {
                fence_after();
                for (int i = 0; i < nact; ++i) scores(i, 0);
            }
            for (int j = 0; j < n && ok; ++j) {
                const int vs = 2 * j + 1, ks = 2 * j + 2;
                ok = wait_on(&kv_full[vs % kSlots], (vs / kSlots) & 1, dead);
                for (int i = 0; i < nact && ok; ++i) {
                    for (int half = 0; half < 2 && ok; ++half) {
                        ok = wait_on(&p_full[2 * i + half], j & 1, dead);
                        fence_after();
                        if (ok) values(i, vs % kSlots, half, j > 0);
                    }
                    if (j + 1 == n) {
                        mma_commit(&pv_done[i]);
                    } else if (ok) {
                        if (i == 0) {
                            ok = wait_on(&kv_full[ks % kSlots], (ks / kSlots) & 1, dead);
                            fence_after();
                            if (!ok) break;
                        }
                        scores(i, ks % kSlots);
                    }
                }
            }
            if (*dead) {  // products in flight end before the memory is given back
                mma_commit(&s_full[0]);
                for (uint32_t it = 0; it < 4096; ++it) mbar_try_wait(&s_full[0], 0);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 13) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        if (lane == 0 && *dead) set_status(a.status, KVQ_STATUS_WAIT_TIMEOUT);
    }
}

template <int D, bool BF>
int launch(const AttnArgs& a, cudaStream_t st) {
    auto* kern = k_paged_chunk<D, BF>;
    constexpr int smem = Smem<D>::total;
    static_assert(smem <= 232448, "shared memory of a block");
    static SmemOptIn opt;
    if (int e = opt.set((const void*)kern, smem)) return e;
    // the register split needs the launch's 128 registers a thread
    static const int regs = [&] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs * 4 < 2 * kRegSoft + kRegDeq + kRegIssue) return KVQ_ERR_UNSUPPORTED;
    const int units = a.B * a.c.Hkv * a.nrb;
    return launch_overlapped(kern, dim3((unsigned)(a.whole + (units - a.whole) * a.S)), kThreads, smem, 1, st, a);
}

}  // namespace

namespace kvq_host {
int run_chunk(const AttnArgs& a, cudaStream_t st) {
    const bool bf = a.c.dtype == KVQ_BF16;
    if (a.c.D == 64) return bf ? launch<64, true>(a, st) : launch<64, false>(a, st);
    return bf ? launch<128, true>(a, st) : launch<128, false>(a, st);
}
}  // namespace kvq_host
