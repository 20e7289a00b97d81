// Rotary positions with one or several axes, forward and inverse.
#include "kvq_paged.cuh"

using namespace kvq;
using namespace kvq_host;

namespace {

// A block takes a few tokens.  First the angles: position * frequency in binary64, reduced to
// [-pi, pi] there (a position of a million leaves no digits to a binary32 product), cos and sin of
// the remainder in binary32, once per (token, pair) into shared memory.  Then a thread keeps the 8
// (cos, sin) of its 8 pairs in registers and turns them for one head after the other, two (four
// for binary32) 16-byte loads and stores each.  HBM bound, each value read and written once: 32768
// tokens of 40 heads of 128 in bf16 take 115 us, 5.8 TB/s (89 % of the measured copy rate).
constexpr int kRopeThreads = 256;

struct RopeArgs {
    kvq_rope_cfg c;
    const void *q, *k;
    void *qo, *ko;
    int64_t qs, ks, qos, kos;
    const int32_t* pos;
    const double* freqs;
    int32_t n, tokens;  // tokens: per block
    float sign;
};

template <typename T>
struct Vec8;  // 8 values from and to memory
template <>
struct Vec8<float> {
    static __device__ __forceinline__ void get(const float* p, float (&x)[8]) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void put(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <bool BF>
struct Vec16 {
    static __device__ __forceinline__ void get(const uint16_t* p, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = lo16<BF>(u[i]), x[2 * i + 1] = hi16<BF>(u[i]);
    }
    static __device__ __forceinline__ void put(uint16_t* p, const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack16<BF>(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <typename E, typename V, bool ADJ>
__device__ __forceinline__ void turn(const E* in, E* out, int c, int half, const float2 (&cs)[8]) {
    // ADJ: channels c .. c + 15 are 8 pairs; else channels c .. c + 7 and c + half ..
    float u[8], v[8], a[8], b[8];
    V::get(in + c, u);
    V::get(in + (ADJ ? c + 8 : c + half), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = ADJ ? (i < 4 ? u[2 * i] : v[2 * i - 8]) : u[i];
        const float y = ADJ ? (i < 4 ? u[2 * i + 1] : v[2 * i - 7]) : v[i];
        const float p = x * cs[i].x - y * cs[i].y, q = y * cs[i].x + x * cs[i].y;
        if (ADJ) {
            if (i < 4) a[2 * i] = p, a[2 * i + 1] = q;
            else b[2 * i - 8] = p, b[2 * i - 7] = q;
        } else {
            a[i] = p, b[i] = q;
        }
    }
    V::put(out + c, a);
    V::put(out + (ADJ ? c + 8 : c + half), b);
}

template <typename E, typename V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeArgs a) {
    extern __shared__ float2 s_cs[];  // [tokens][pairs]
    const int half = a.c.rot_dim / 2, t0 = blockIdx.x * a.tokens;
    const int nt = min(a.tokens, a.n - t0);
    let_next();
    after_previous();
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int p = i % half, t = t0 + i / half;
        const double two_pi = 6.283185307179586476925286766559;
        double ang = (double)a.pos[(size_t)a.c.pair_axis[p] * a.n + t] * a.freqs[p];
        ang -= two_pi * rint(ang * (1.0 / two_pi));
        float s, c;
        sincosf((float)ang, &s, &c);
        s_cs[i] = make_float2(c, s * a.sign);
    }
    __syncthreads();
    // work of a token: D/16 pieces (8 pairs, or 16 copied channels) x heads
    const int pieces = a.c.D / 16, turned = a.c.rot_dim / 16, heads = a.c.Hq + a.c.Hkv;
    const int lanes = kRopeThreads / (nt * pieces);  // threads that share a (token, piece)
    const int slot = threadIdx.x / (nt * pieces), tp = threadIdx.x % (nt * pieces);
    if (slot >= lanes) return;
    const int piece = tp % pieces, lt = tp / pieces;
    const size_t t = t0 + lt;
    const E* q = static_cast<const E*>(a.q) + t * a.qs;
    const E* k = static_cast<const E*>(a.k) + t * a.ks;
    E* qo = static_cast<E*>(a.qo) + t * a.qos;
    E* ko = static_cast<E*>(a.ko) + t * a.kos;
    float2 cs[8] = {};
    if (piece < turned)
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = s_cs[lt * half + piece * 8 + i];
    for (int h = blockIdx.y * lanes + slot; h < heads; h += gridDim.y * lanes) {
        const E* in = h < a.c.Hq ? q + h * a.c.D : k + (h - a.c.Hq) * a.c.D;
        E* out = h < a.c.Hq ? qo + h * a.c.D : ko + (h - a.c.Hq) * a.c.D;
        if (piece < turned) {
            turn<E, V, ADJ>(in, out, piece * (ADJ ? 16 : 8), half, cs);
        } else if (in != out) {
            constexpr int W = sizeof(E);  // 16 values are W 16-byte words
            const uint4* from = reinterpret_cast<const uint4*>(in + piece * 16);
            uint4* to = reinterpret_cast<uint4*>(out + piece * 16);
#pragma unroll
            for (int i = 0; i < W; ++i) to[i] = from[i];
        }
    }
}

}  // namespace

extern "C" int kvq_rope(const kvq_rope_cfg* cfg, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const int32_t* positions, const double* freqs, int32_t n,
                        int32_t inverse, void* q_out, int64_t q_out_stride, void* k_out,
                        int64_t k_out_stride, void* stream) {
    if (!cfg) return KVQ_ERR_NULL;
    if (cfg->dtype != KVQ_F16 && cfg->dtype != KVQ_BF16 && cfg->dtype != KVQ_F32) return KVQ_ERR_UNSUPPORTED;
    if (cfg->D < 16 || cfg->D > 256 || cfg->D % 16 || cfg->rot_dim < 16 || cfg->rot_dim > cfg->D ||
        cfg->rot_dim % 16)
        return KVQ_ERR_UNSUPPORTED;
    if (cfg->Hq < 1 || cfg->Hkv < 0 || cfg->Hq > 65536 || cfg->Hkv > 65536) return KVQ_ERR_SHAPE;
    if (cfg->axes < 1 || cfg->axes > 8 || (cfg->adjacent != 0 && cfg->adjacent != 1) ||
        (inverse != 0 && inverse != 1) || n < 0)
        return KVQ_ERR_SHAPE;
    for (int i = 0; i < cfg->rot_dim / 2; ++i)
        if (cfg->pair_axis[i] >= cfg->axes) return KVQ_ERR_RANGE;
    if (n == 0) return KVQ_OK;
    if (!q || !q_out || !positions || !freqs) return KVQ_ERR_NULL;
    if (cfg->Hkv > 0 && (!k || !k_out)) return KVQ_ERR_NULL;
    const int size = cfg->dtype == KVQ_F32 ? 4 : 2, mask = 16 / size - 1;
    if (!aligned16(q) || !aligned16(q_out) || (q_stride | q_out_stride) & mask) return KVQ_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(freqs) & 7) return KVQ_ERR_ALIGN;
    if (q_stride < (int64_t)cfg->Hq * cfg->D || q_out_stride < (int64_t)cfg->Hq * cfg->D) return KVQ_ERR_SHAPE;
    if (cfg->Hkv > 0) {
        if (!aligned16(k) || !aligned16(k_out) || (k_stride | k_out_stride) & mask) return KVQ_ERR_ALIGN;
        if (k_stride < (int64_t)cfg->Hkv * cfg->D || k_out_stride < (int64_t)cfg->Hkv * cfg->D) return KVQ_ERR_SHAPE;
    }
    // in place only over the very same rows
    if ((q == q_out && q_stride != q_out_stride) || (cfg->Hkv > 0 && k == k_out && k_stride != k_out_stride))
        return KVQ_ERR_SHAPE;
    RopeArgs a{*cfg, q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, positions, freqs, n, 1,
               inverse ? -1.0f : 1.0f};
    // four tokens to a block when that still fills the GPU: 256 angles for 256 threads at D = 128
    const int pieces = cfg->D / 16, heads = cfg->Hq + cfg->Hkv;
    a.tokens = n >= 148 * 16 && pieces * 4 <= kRopeThreads ? 4 : 1;
    const int lanes = kRopeThreads / (a.tokens * pieces);
    // few tokens: the heads over several blocks, one head a thread
    int gy = 1;
    if (n < 148 * 2) gy = (heads + lanes - 1) / lanes;
    const dim3 grid((unsigned)(((int64_t)n + a.tokens - 1) / a.tokens), gy);
    const size_t smem = (size_t)a.tokens * (cfg->rot_dim / 2) * sizeof(float2);
    cudaStream_t st = (cudaStream_t)stream;
    const bool adj = cfg->adjacent;
    auto go = [&](auto* adjk, auto* halfk) {
        return launch_overlapped(adj ? adjk : halfk, grid, kRopeThreads, smem, 1, st, a);
    };
    if (cfg->dtype == KVQ_F32) return go(k_rope<float, Vec8<float>, true>, k_rope<float, Vec8<float>, false>);
    if (cfg->dtype == KVQ_BF16) return go(k_rope<uint16_t, Vec16<true>, true>, k_rope<uint16_t, Vec16<true>, false>);
    return go(k_rope<uint16_t, Vec16<false>, true>, k_rope<uint16_t, Vec16<false>, false>);
}
