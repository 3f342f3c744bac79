// What stands before and behind attention in a serving step: the norm and rotation of
// queries and keys, and the verification of drafted tokens.

#include <cuda_runtime.h>
#include <math.h>

#include "gqa_attn.h"
#include "ptx.cuh"
#include "runtime.cuh"

namespace gqa {
namespace step {

template <typename... A>
cudaError_t launch(void (*kern)(A...), dim3 grid, int threads, int cluster, cudaStream_t stream,
                   A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    // The grid may start while the previous kernel of the stream finishes; it reads no
    // global memory before griddepcontrol.wait.
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ------------------------------------------------------------ norm and rotation
//
//   z_c = x_c / sqrt(mean_c x_c^2 + eps) * w_c                  (each head of q and k)
//   y_1 = z_1 cos a - z_2 sin a,  y_2 = z_2 cos a + z_1 sin a   (each pair of channels)
//
// with a = position * inv_freq. Rounded to bf16 once, at the end. A lane holds two chunks
// of 8 channels of a head, chosen so that they are the two sides of 8 pairs: nothing but
// the sum of squares goes between lanes, and a warp takes 4 heads (d = 128) or 8 (d = 64)
// at a time. cos and sin of the block's tokens are computed once, into shared memory; a
// lane multiplies them with its weights once per token, and then needs two products for
// a channel.
//
// Bound by HBM for many tokens (8203 tokens of 64/8 heads, d = 128, 302 MB: 52.6 us, 5.75
// TB/s, 0.86 of the measured copy rate), by the chain launch, angles, heads for few (8 tokens
// 2.8 us in a graph). Measured for the many / for 5000 tokens of 28/4 heads (19.4): one
// chunk a lane, partners by shuffle, 69 / 28 (180 instructions a warp for two heads); blocks
// of 256 threads 56 / 22; registers capped at 80 to fit a sixth block, with spills, 57 / 20;
// one head's loads in flight 61 / 22; two tokens to a block of four warps 55 / 21.
constexpr int kNormThreads = 128;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxAxes = 4;
constexpr int kNormBatch = 2;  // heads of a lane whose loads are in flight

struct NormParams {
    const uint16_t *q, *k;
    uint16_t *qo, *ko;
    const void *qw, *kw;         // [d] bf16 or fp32, or null
    const int32_t* positions;    // [axes, tokens]
    const float* inv_freq;       // [pairs]
    int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;
    int tokens, H_q, H_kv, pairs, wide_weights;
    int section_end[kMaxAxes];   // first pair behind each axis' section
    int block_tokens;            // 1, 2 or 4 tokens of a block
    float eps;
};

// cos and sin of position * frequency, with the angle in turns as a 64-bit fixed-point
// fraction: whole turns fall out of the product as its overflow, so far positions lose
// nothing (an angle of 10^6 radians rounded to 32 bits would be off by 0.03). The
// fraction of one position's angle is m 2^e / (2 pi) with m, e of the 32-bit frequency,
// from the first 64 bits of 1 / (2 pi): off by 2^-65 for frequencies up to 1, so by
// 2^-34 turns at 2^31 positions. (64-bit floating point has a sixty-fourth of the
// 32-bit rate here.) Frequencies below 2^24.
__device__ __forceinline__ float2 rotation(int position, float freq) {
    constexpr unsigned long long kInv2Pi = 0xa2f9836e4e441529ull;  // 2^66 / (2 pi)
    const unsigned bits = __float_as_uint(freq), exp = (bits >> 23) & 0xffu;
    const unsigned long long m = (bits & 0x7fffffu) | (exp ? 0x800000u : 0u);
    const int shift = 152 - int(exp ? exp : 1u);  // 2 - e
    const unsigned long long hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;
    unsigned long long per = 0;  // turns of one position, 2^64 to a turn
    if (shift >= 64) per = shift < 128 ? hi >> (shift - 64) : 0;
    else if (shift > 0) per = (hi << (64 - shift)) | (lo >> shift);
    if (bits >> 31) per = 0ull - per;
    const unsigned long long turns = per * static_cast<unsigned long long>(int64_t(position));
    float2 r;  // the nearest whole turn taken off: [-1/2, 1/2) turns, in halves
    sincospif(float(int(turns >> 32)) * 0x1p-31f, &r.y, &r.x);
    return r;
}

template <int D, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads, 5) norm_rope_kernel(const NormParams p) {
    constexpr int kHeadLanes = D / 16, kHeads = 32 / kHeadLanes;  // of a warp
    __shared__ __align__(16) float cos_s[kNormWarps][D / 2], sin_s[kNormWarps][D / 2];
    __shared__ __align__(16) float weights[2][D];
    grid_launch_dependents();
    grid_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.block_tokens;
    // the block's warps share its tokens; blockIdx.y shares a token's heads further
    const int per_token = kNormWarps / p.block_tokens;
    const int mine = warp / per_token;  // which of the block's tokens
    const int t = t0 + mine;
    const bool live = t < p.tokens;
    const int worker = blockIdx.y * per_token + warp % per_token;
    const int workers = per_token * gridDim.y;
    const int l = lane % kHeadLanes, sub = lane / kHeadLanes;
    // This lane's chunks of 8 channels. With S = pairs / 8 the chunks 0 .. S - 1 and S ..
    // 2 S - 1 are the two sides of the pairs (not interleaved); those behind are not turned.
    const int S = p.pairs / 8;
    const bool turned = l < S;
    const int chunk_a = turned ? l : S + l;
    const int chunk_b = turned ? l + S : l + kHeadLanes;

    struct Rows {
        const uint16_t* x;
        int64_t step;
        int h;
    };
    auto load = [&](const Rows& r, int heads, uint4& a, uint4& b) {
        if (r.h < heads) {
            a = *reinterpret_cast<const uint4*>(r.x + chunk_a * 8);
            b = *reinterpret_cast<const uint4*>(r.x + chunk_b * 8);
        } else {
            a = b = make_uint4(0, 0, 0, 0);
        }
    };
    auto rows_of = [&](const uint16_t* x, int64_t st, int64_t sh) {
        const int h = worker * kHeads + sub;
        return Rows{x + t * st + h * sh, workers * kHeads * sh, h};
    };
    uint4 va[kNormBatch], vb[kNormBatch];
    auto load_batch = [&](Rows& r, int heads) {
#pragma unroll
        for (int u = 0; u < kNormBatch; ++u) {
            load(r, heads, va[u], vb[u]);
            r.x += r.step;
            r.h += workers * kHeads;
        }
    };
    // the first heads are on their way while the angles are computed
    Rows rq = rows_of(p.q, p.q_st, p.q_sh);
    load_batch(rq, live ? p.H_q : 0);

    for (int i = threadIdx.x; i < p.block_tokens * (D / 2); i += kNormThreads) {
        const int pair = i % (D / 2), tok = i / (D / 2), at = t0 + tok;
        if (pair >= p.pairs || at >= p.tokens) continue;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kMaxAxes - 1; ++a) axis += pair >= p.section_end[a];
        const float2 r = rotation(p.positions[int64_t(axis) * p.tokens + at], p.inv_freq[pair]);
        cos_s[tok][pair] = r.x;
        sin_s[tok][pair] = r.y;
    }
    if constexpr (kNorm) {
        for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) {
            const void* w = i < D ? p.qw : p.kw;
            const int ch = i % D;
            weights[i / D][ch] =
                !w               ? 1.f
                : p.wide_weights ? static_cast<const float*>(w)[ch]
                                 : __uint_as_float(
                                       uint32_t(static_cast<const uint16_t*>(w)[ch]) << 16);
        }
    }
    __syncthreads();
    if (!live) return;

    auto part = [&](int which, Rows rows, int heads, uint16_t* y, int64_t y_st, int64_t y_sh) {
        // Pairs (first, second) of this lane and what they are multiplied with:
        //   y_first = r (fc first - ss second),  y_second = r (sc second + fs first)
        float fc[8], ss[8], sc[8], fs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int ch1 = kInterleaved ? (j < 4 ? chunk_a : chunk_b) * 8 + (j & 3) * 2
                                         : chunk_a * 8 + j;
            const int ch2 = kInterleaved ? ch1 + 1 : chunk_b * 8 + j;
            const float w1 = kNorm ? weights[which][ch1] : 1.f;
            const float w2 = kNorm ? weights[which][ch2] : 1.f;
            const int pair = kInterleaved ? ch1 >> 1 : ch1;
            const float c = turned ? cos_s[mine][pair] : 1.f;
            const float s = turned ? sin_s[mine][pair] : 0.f;
            fc[j] = w1 * c;
            ss[j] = -w2 * s;
            sc[j] = w2 * c;
            fs[j] = w1 * s;
        }
        int h = worker * kHeads + sub;
        uint16_t* out = y + t * y_st + h * y_sh;
        const int64_t out_step = workers * kHeads * y_sh;
#pragma unroll 1
        for (int h0 = worker * kHeads; h0 < heads;) {
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                if (h0 >= heads) break;
                const uint32_t ra[4] = {va[u].x, va[u].y, va[u].z, va[u].w};
                const uint32_t rb[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
                load(rows, heads, va[u], vb[u]);
                rows.x += rows.step;
                rows.h += workers * kHeads;
                float f[8], s[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = __uint_as_float(ra[i] << 16);
                    const float a1 = __uint_as_float(ra[i] & 0xffff0000u);
                    const float b0 = __uint_as_float(rb[i] << 16);
                    const float b1 = __uint_as_float(rb[i] & 0xffff0000u);
                    if constexpr (kInterleaved) {
                        f[i] = a0; s[i] = a1; f[4 + i] = b0; s[4 + i] = b1;
                    } else {
                        f[2 * i] = a0; f[2 * i + 1] = a1; s[2 * i] = b0; s[2 * i + 1] = b1;
                    }
                }
                uint64_t r2 = f2pack(1.f, 1.f);
                if constexpr (kNorm) {
                    uint64_t q0 = 0ull, q1 = 0ull;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t x = f2pack(f[2 * i], f[2 * i + 1]);
                        const uint64_t z = f2pack(s[2 * i], s[2 * i + 1]);
                        q0 = ffma2(x, x, q0);
                        q1 = ffma2(z, z, q1);
                    }
                    float s0, s1;
                    f2unpack(fadd2(q0, q1), s0, s1);
                    float sum = s0 + s1;
#pragma unroll
                    for (int o = kHeadLanes / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float r = rsqrtf(sum * (1.f / D) + p.eps);
                    r2 = f2pack(r, r);
                }
                float yf[8], ys[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 2 * i;
                    const uint64_t x = f2pack(f[j], f[j + 1]), z = f2pack(s[j], s[j + 1]);
                    uint64_t a = fmul2(f2pack(fc[j], fc[j + 1]), x);
                    uint64_t b = fmul2(f2pack(sc[j], sc[j + 1]), z);
                    // (channels that are not turned take nothing of another's infinity)
                    if (turned) {
                        a = ffma2(f2pack(ss[j], ss[j + 1]), z, a);
                        b = ffma2(f2pack(fs[j], fs[j + 1]), x, b);
                    }
                    if constexpr (kNorm) {
                        a = fmul2(a, r2);
                        b = fmul2(b, r2);
                    }
                    f2unpack(a, yf[j], yf[j + 1]);
                    f2unpack(b, ys[j], ys[j + 1]);
                }
                if (h < heads) {
                    uint32_t wa[4], wb[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        wa[i] = kInterleaved ? pack_bf16x2(yf[i], ys[i])
                                             : pack_bf16x2(yf[2 * i], yf[2 * i + 1]);
                        wb[i] = kInterleaved ? pack_bf16x2(yf[4 + i], ys[4 + i])
                                             : pack_bf16x2(ys[2 * i], ys[2 * i + 1]);
                    }
                    *reinterpret_cast<uint4*>(out + chunk_a * 8) =
                        make_uint4(wa[0], wa[1], wa[2], wa[3]);
                    *reinterpret_cast<uint4*>(out + chunk_b * 8) =
                        make_uint4(wb[0], wb[1], wb[2], wb[3]);
                }
                out += out_step;
                h += workers * kHeads;
                h0 += workers * kHeads;
            }
        }
    };
    part(0, rq, p.H_q, p.qo, p.qo_st, p.qo_sh);
    if (worker * kHeads >= p.H_kv) return;
    Rows rk = rows_of(p.k, p.k_st, p.k_sh);
    load_batch(rk, p.H_kv);
    part(1, rk, p.H_kv, p.ko, p.ko_st, p.ko_sh);
}

// ------------------------------------------------------------ drafted tokens
//
// Row b has n drafted tokens x_i and n + 1 rows p_i of target probabilities. x_i stands
// if u_i q_i(x_i) < p_i(x_i) and all before it stand; with k the number that stand, the
// next token is drawn from w = max(p_k - q_k, 0) (k < n) or w = p_n by inverting its sum:
// the lowest v with w_0 + .. + w_v > u (w_0 + .. + w_(V-1)).
//
// Bound by reading one row of p (and one of q). A cluster of CTAs takes a row: every
// warp sums a contiguous piece, the CTAs exchange their sums through distributed shared
// memory, and the CTA in whose piece the token lies reads one warp's piece again.
//
// Rounding. The token has to be the one that the sum in 64 bits gives, but 64-bit
// arithmetic runs at a sixty-fourth of the 32-bit rate: with it in every thread a row took 29 us
// and a batch of 48 rows 58. A lane adds its terms in two 32-bit words, the difference
// p - q and every sum with the exact error of its rounding, lanes and warps are added the
// same way, and one warp adds the warps' and the CTAs' sums in 64 bits.
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 16;

struct VerifyParams {
    const float *p, *q;          // [total + B, V], [total, V] or null
    const int32_t* tokens;       // [total]
    const float *u_accept, *u_sample;
    const int32_t* cu;           // [B + 1] or null
    int32_t *accepted, *next;    // [B]
    unsigned* status;
    int64_t p_st, q_st;
    int B, total, V, piece;      // piece: elements of a warp, a multiple of 128
};

struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float err) {
        const float s = hi + x, t = s - hi;
        lo += ((hi - (s - t)) + (x - t)) + err;
        hi = s;
    }
    __device__ __forceinline__ double value() const { return double(hi) + double(lo); }
};
// The term of one element: max(p - q, 0) as a 32-bit value and the error of its rounding.
__device__ __forceinline__ void add_difference(Sum2& s, float p, float q) {
    const float d = p - q, t = d - p;
    const float err = (p - (d - t)) + (-q - t);
    if (d > 0.f) s.add(d, err);
}
__device__ __forceinline__ void add_plain(Sum2& s, float p) {
    if (p > 0.f) s.add(p, 0.f);
}

// Where a sum over the lanes passes a threshold: x >= 0 is a lane's part, incl its
// inclusive prefix sum and base what comes before. The first lane whose sum is above
// limit, or the last lane with any part (rounding kept the sum below); before: the sum
// up to that lane. For whole warps.
__device__ __forceinline__ int passing_lane(double x, double incl, double base, double limit,
                                            double& before) {
    const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
    const unsigned above = __ballot_sync(0xffffffffu, x > 0.0 && base + incl > limit);
    const int at = above ? __ffs(above) - 1 : 31 - __clz(some | 1u);
    const double prev = __shfl_sync(0xffffffffu, incl, max(at - 1, 0));
    before = at > 0 ? base + prev : base;
    return at;
}
__device__ __forceinline__ double inclusive16(double x, int lane) {
    for (int o = 1; o < 16; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams p) {
    static_assert(kVerifyWarps == 16 && kMaxCluster == 16, "inclusive16");
    __shared__ int first_fall;
    __shared__ float2 warp_sum[kVerifyWarps];
    __shared__ double cta_sum[2][kMaxCluster];  // written by the cluster's CTAs
    // what one warp finds for all: the CTA (-1: nothing to draw from) and the warp where
    // the sum passes the threshold, the sum before that warp
    __shared__ int owner_cta, owner_warp;
    __shared__ double owner_before;
    grid_launch_dependents();
    grid_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cluster = gridDim.x, rank = blockIdx.x, b = blockIdx.y;

    // the row's drafted tokens; prefix sums that are not are clamped and reported
    int first, n;
    bool bad = false;
    if (p.cu) {
        const int a = p.cu[b], e = p.cu[b + 1];
        first = min(max(a, 0), p.total);
        const int last = min(max(e, first), p.total);
        n = last - first;
        bad = first != a || last != e;
    } else {
        n = p.total / p.B;
        first = b * n;
    }
    if (threadIdx.x == 0) first_fall = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kVerifyThreads) {
        const int x = p.tokens[first + i];
        bool stands = false;
        if (x < 0 || x >= p.V) {
            bad = true;
        } else {
            // (the product of two 32-bit values is exact in 64 bits)
            const double q = p.q ? double(p.q[(int64_t(first) + i) * p.q_st + x]) : 1.0;
            stands = double(p.u_accept[first + i]) * q <
                     double(p.p[(int64_t(first) + b + i) * p.p_st + x]);
        }
        if (!stands) atomicMin(&first_fall, i);
    }
    if (bad && rank == 0) atomicOr(p.status, kStatusBadSeqlen);
    __syncthreads();
    const int k = first_fall;
    if (rank == 0 && threadIdx.x == 0) p.accepted[b] = k;
    const float* pr = p.p + (int64_t(first) + b + k) * p.p_st;
    // what is taken off p: a row of q, or all of one token
    const float* qr = k < n && p.q ? p.q + (int64_t(first) + k) * p.q_st : nullptr;
    int gone = k < n && !p.q ? p.tokens[first + k] : -1;
    const bool vec = ((reinterpret_cast<uintptr_t>(pr) | reinterpret_cast<uintptr_t>(qr)) & 15) == 0;

    const int begin = min(int64_t(p.V), (int64_t(rank) * kVerifyWarps + warp) * p.piece);
    const int end = min(p.V, begin + p.piece);
    // In the second round nothing is taken off: only if p is nowhere above q.
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        Sum2 s[2];
        auto add = [&](int at, int v, float pv, float qv) {
            if (qr) add_difference(s[at], pv, qv);
            else if (v != gone) add_plain(s[at], pv);
        };
        int v = begin;
        if (vec) {
            constexpr int kBatch = 4;
#pragma unroll 1
            for (; v + 128 * kBatch <= end; v += 128 * kBatch) {
                float4 x[kBatch], y[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    x[u] = *reinterpret_cast<const float4*>(pr + v + 128 * u + lane * 4);
                    y[u] = qr ? *reinterpret_cast<const float4*>(qr + v + 128 * u + lane * 4)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int e = v + 128 * u + lane * 4;
                    add(0, e, x[u].x, y[u].x);
                    add(1, e + 1, x[u].y, y[u].y);
                    add(0, e + 2, x[u].z, y[u].z);
                    add(1, e + 3, x[u].w, y[u].w);
                }
            }
        }
        constexpr int kBatch = 8;
#pragma unroll 1
        for (; v < end; v += 32 * kBatch) {
            float x[kBatch], y[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int e = v + 32 * u + lane;
                x[u] = e < end ? pr[e] : 0.f;
                y[u] = qr && e < end ? qr[e] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) add(u & 1, v + 32 * u + lane, x[u], y[u]);
        }
        s[0].add(s[1].hi, s[1].lo);
        for (int o = 16; o > 0; o >>= 1) {
            const float hi = __shfl_xor_sync(0xffffffffu, s[0].hi, o);
            const float lo = __shfl_xor_sync(0xffffffffu, s[0].lo, o);
            s[0].add(hi, lo);
        }
        if (lane == 0) warp_sum[warp] = make_float2(s[0].hi, s[0].lo);
        __syncthreads();
        double part = 0.0, incl = 0.0;  // warp 0, one lane per warp of the CTA
        if (warp == 0) {
            if (lane < kVerifyWarps) part = double(warp_sum[lane].x) + double(warp_sum[lane].y);
            incl = inclusive16(part, lane);
            const double mine = __shfl_sync(0xffffffffu, incl, kVerifyWarps - 1);
            if (cluster == 1) {
                if (lane == 0) cta_sum[round][0] = mine;
                __syncwarp();
            } else if (lane < cluster) {
                st_dsmem_f64(map_to_rank(smem_u32(&cta_sum[round][rank]), lane), mine);
            }
        }
        if (cluster > 1) {
            cluster_arrive_release();
            cluster_wait_acquire();
        }
        double limit = 0.0;
        if (warp == 0) {
            const double c = lane < cluster ? cta_sum[round][lane] : 0.0;
            const double c_incl = inclusive16(c, lane);
            const double total = __shfl_sync(0xffffffffu, c_incl, kMaxCluster - 1);
            limit = double(p.u_sample[b]) * total;
            double before;
            const int cta = passing_lane(c, c_incl, 0.0, limit, before);
            double warp_before = 0.0;
            const int w = passing_lane(part, incl, before, limit, warp_before);
            if (lane == 0) {
                owner_cta = total > 0.0 && total < INFINITY ? cta : -1;
                owner_warp = w;
                owner_before = warp_before;
            }
        }
        __syncthreads();
        if (owner_cta >= 0) {
            if (owner_cta != rank) return;
            // that warp's piece again: a sixteenth of it for each warp, a run of
            // consecutive elements for each lane
            const int share = p.piece / kVerifyWarps, each = (share + 31) / 32;
            const int64_t from =
                (int64_t(rank) * kVerifyWarps + owner_warp) * p.piece + warp * share;
            const int64_t stop = min(int64_t(p.V), from + share);
            const int lo = int(min(stop, from + lane * each));
            const int hi = int(min(stop, from + lane * each + each));
            Sum2 run;
            for (int e = lo; e < hi; ++e) {
                if (qr) add_difference(run, pr[e], qr[e]);
                else if (e != gone) add_plain(run, pr[e]);
            }
            Sum2 upto = run;
            for (int o = 1; o < 32; o <<= 1) {
                const float yh = __shfl_up_sync(0xffffffffu, upto.hi, o);
                const float yl = __shfl_up_sync(0xffffffffu, upto.lo, o);
                if (lane >= o) upto.add(yh, yl);
            }
            const double base = owner_before;
            if (lane == 31) warp_sum[warp] = make_float2(upto.hi, upto.lo);
            __syncthreads();
            if (warp == 0) {
                if (lane < kVerifyWarps) part = double(warp_sum[lane].x) + double(warp_sum[lane].y);
                double before;
                const int w =
                    passing_lane(part, inclusive16(part, lane), base, limit, before);
                if (lane == 0) {
                    owner_warp = w;
                    owner_before = before;
                    cta_sum[0][0] = limit;
                }
            }
            __syncthreads();
            if (warp != owner_warp) return;
            limit = cta_sum[0][0];
            double at;
            const int l = passing_lane(run.value(), upto.value(), owner_before, limit, at);
            if (lane == l) {
                int token = lo;
                for (int e = lo; e < hi; ++e) {
                    if (e == gone) continue;
                    const double w = double(pr[e]) - (qr ? double(qr[e]) : 0.0);
                    if (!(w > 0.0)) continue;
                    token = e;
                    at += w;
                    if (at > limit) break;
                }
                p.next[b] = token;
            }
            return;
        }
        if (!qr && gone < 0) break;
        qr = nullptr;
        gone = -1;
    }
    // no probability above 0 anywhere, or an infinite one
    if (rank == 0 && threadIdx.x == 0) {
        p.next[b] = -1;
        atomicOr(p.status, kStatusBadSeqlen);
    }
}

}  // namespace step
}  // namespace gqa

using namespace gqa;

namespace {

// Token and head strides of a [tokens, heads, d] tensor: multiples of 8 that are not
// negative (a dimension of size 1 has none); outputs also have no two rows in one place.
int check_rows(const void* x, int64_t st, int64_t sh, int tokens, int heads, int d, bool output) {
    if (tokens <= 1) st = 8;
    if (heads <= 1) sh = 8;
    const int64_t lim = int64_t(1) << 39;
    if (st <= 0 || sh <= 0 || st >= lim || sh >= lim) return GQA_ERR_INVALID_ARG;
    if ((st | sh) & 7 || !aligned16(x)) return GQA_ERR_MISALIGNED;
    if (output && ((heads > 1 && sh < d) || (tokens > 1 && st < d) ||
                   (tokens > 1 && heads > 1 && st < sh * (heads - 1) + d &&
                    sh < st * (tokens - 1) + d)))
        return GQA_ERR_INVALID_ARG;
    return GQA_OK;
}

template <int D>
cudaError_t launch_norm(const step::NormParams& p, bool norm, bool interleaved, dim3 grid,
                        cudaStream_t stream) {
    using namespace step;
    auto kern = norm ? (interleaved ? norm_rope_kernel<D, true, true>
                                    : norm_rope_kernel<D, true, false>)
                     : (interleaved ? norm_rope_kernel<D, false, true>
                                    : norm_rope_kernel<D, false, false>);
    return launch(kern, grid, kNormThreads, 1, stream, p);
}

}  // namespace

extern "C" int gqa_attn_qk_norm_rope(
    const uint16_t* q, const uint16_t* k, uint16_t* q_out, uint16_t* k_out, const void* q_weight,
    const void* k_weight, int weights_fp32, const int32_t* positions, const float* inv_freq,
    const int32_t* sections, int axes, int tokens, int H_q, int H_kv, int d, int pairs,
    int interleaved, int norm, float eps, int64_t q_stride_t, int64_t q_stride_h,
    int64_t k_stride_t, int64_t k_stride_h, int64_t qo_stride_t, int64_t qo_stride_h,
    int64_t ko_stride_t, int64_t ko_stride_h, cudaStream_t stream) {
    using namespace step;
    if (tokens < 0 || H_q <= 0 || H_kv < 0 || pairs < 1 || axes < 1 || (axes > 1 && !sections) ||
        (norm && !(isfinite(eps) && eps >= 0.f)))
        return GQA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED;
    if (axes > kMaxAxes || pairs % 8 != 0) return GQA_ERR_UNSUPPORTED;
    if (2 * pairs > d) return GQA_ERR_INVALID_ARG;
    if (tokens > 0 && (!q || !q_out || !positions || !inv_freq || (H_kv > 0 && (!k || !k_out))))
        return GQA_ERR_INVALID_ARG;
    NormParams p{};
    int at = 0;
    for (int a = 0; a < kMaxAxes; ++a) {
        if (axes > 1 && a < axes) {
            if (sections[a] < 0 || sections[a] > pairs) return GQA_ERR_INVALID_ARG;
            at += sections[a];
        } else if (axes == 1) {
            at = pairs;
        }
        p.section_end[a] = at;
    }
    if (at != pairs) return GQA_ERR_INVALID_ARG;
    int rc = check_rows(q, q_stride_t, q_stride_h, tokens, H_q, d, false);
    if (rc == GQA_OK) rc = check_rows(q_out, qo_stride_t, qo_stride_h, tokens, H_q, d, true);
    if (rc == GQA_OK && H_kv > 0) rc = check_rows(k, k_stride_t, k_stride_h, tokens, H_kv, d, false);
    if (rc == GQA_OK && H_kv > 0)
        rc = check_rows(k_out, ko_stride_t, ko_stride_h, tokens, H_kv, d, true);
    if (rc != GQA_OK) return rc;
    const uintptr_t wide = weights_fp32 ? 3u : 1u;
    if (((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq)) & 3u) ||
        ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & wide))
        return GQA_ERR_MISALIGNED;
    if (tokens == 0) return GQA_OK;
    const int sms = num_sms();
    if (sms <= 0) return GQA_ERR_CUDA;
    p.q = q; p.k = k; p.qo = q_out; p.ko = k_out;
    p.qw = q_weight; p.kw = k_weight; p.wide_weights = weights_fp32 != 0;
    p.positions = positions; p.inv_freq = inv_freq;
    auto fix = [](int64_t s, int n) { return n > 1 ? s : int64_t(0); };
    p.q_st = fix(q_stride_t, tokens); p.q_sh = fix(q_stride_h, H_q);
    p.k_st = fix(k_stride_t, tokens); p.k_sh = fix(k_stride_h, H_kv);
    p.qo_st = fix(qo_stride_t, tokens); p.qo_sh = fix(qo_stride_h, H_q);
    p.ko_st = fix(ko_stride_t, tokens); p.ko_sh = fix(ko_stride_h, H_kv);
    p.tokens = tokens; p.H_q = H_q; p.H_kv = H_kv; p.pairs = pairs; p.eps = eps;
    const int rounds = (H_q * (d / 16) + 31) / 32;  // of one warp for a token's query heads
    int block_tokens = kNormWarps, split = 1;
    while (block_tokens > 1 && tokens < block_tokens * 4 * sms) block_tokens /= 2;
    while (tokens * split < 2 * sms && split * kNormWarps < rounds) ++split;
    p.block_tokens = block_tokens;
    const dim3 grid(unsigned((tokens + block_tokens - 1) / block_tokens), unsigned(split));
    return (d == 128 ? launch_norm<128>(p, norm != 0, interleaved != 0, grid, stream)
                     : launch_norm<64>(p, norm != 0, interleaved != 0, grid, stream)) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}

extern "C" int gqa_attn_verify_drafts(const float* target_probs, const float* draft_probs,
                                      const int32_t* draft_tokens, const float* u_accept,
                                      const float* u_sample, const int32_t* cu_seqlens,
                                      int32_t* accepted, int32_t* next_tokens, int B, int total,
                                      int V, int64_t target_stride, int64_t draft_stride,
                                      cudaStream_t stream) {
    using namespace step;
    if (B < 0 || B > 65535 || total < 0 || V < 1) return GQA_ERR_INVALID_ARG;
    if (V > (1 << 30)) return GQA_ERR_UNSUPPORTED;
    if (B == 0) return total == 0 ? GQA_OK : GQA_ERR_INVALID_ARG;
    if (!target_probs || !u_sample || !accepted || !next_tokens ||
        (total > 0 && (!draft_tokens || !u_accept)) || (!cu_seqlens && total % B != 0))
        return GQA_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 39;
    if ((int64_t(total) + B > 1 && (target_stride < V || target_stride >= lim)) ||
        (draft_probs && total > 1 && (draft_stride < V || draft_stride >= lim)))
        return GQA_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(target_probs), static_cast<const void*>(draft_probs),
                          static_cast<const void*>(draft_tokens), static_cast<const void*>(u_accept),
                          static_cast<const void*>(u_sample), static_cast<const void*>(cu_seqlens),
                          static_cast<const void*>(accepted), static_cast<const void*>(next_tokens)})
        if (reinterpret_cast<uintptr_t>(x) & 3u) return GQA_ERR_MISALIGNED;
    unsigned* status = status_word();
    const int sms = num_sms(), dev = current_device();
    if (!status || sms <= 0) return GQA_ERR_CUDA;
    static std::atomic<uint64_t> attr_done{0};
    if (device_attrs_pending(attr_done, dev)) {
        if (cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                 1) != cudaSuccess)
            return GQA_ERR_CUDA;
        device_attrs_mark(attr_done, dev);
    }
    int cluster = kMaxCluster;
    while (cluster > 1 && (int64_t(B) * cluster > 2 * sms || V < 2048 * cluster)) cluster /= 2;
    VerifyParams p{};
    p.p = target_probs; p.q = draft_probs;
    p.tokens = draft_tokens; p.u_accept = u_accept; p.u_sample = u_sample; p.cu = cu_seqlens;
    p.accepted = accepted; p.next = next_tokens; p.status = status;
    p.p_st = target_stride; p.q_st = draft_stride;
    p.B = B; p.total = total; p.V = V;
    const int pieces = cluster * kVerifyWarps * 128;
    p.piece = (V + pieces - 1) / pieces * 128;
    return launch(verify_kernel, dim3(unsigned(cluster), unsigned(B)), kVerifyThreads, cluster,
                  stream, p) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}
