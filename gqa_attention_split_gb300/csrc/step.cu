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
// with a = position * inv_freq. Rounded to bf16 once, at the end. A head is 8 channels
// a lane, so a warp takes 2 heads (d = 128) or 4 (d = 64) at a time. cos and sin of the
// block's tokens are computed once, into shared memory; a lane multiplies those of its
// channels with its weights once per token, and then needs two products for a channel.
constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxAxes = 4;
constexpr int kNormBatch = 4;  // heads' loads in flight a lane

struct NormParams {
    const uint16_t *q, *k;
    uint16_t *qo, *ko;
    const void *qw, *kw;         // [d] bf16 or fp32, or null
    const int32_t* positions;    // [axes, tokens]
    const float* inv_freq;       // [pairs]
    int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;
    int tokens, H_q, H_kv, pairs, wide_weights;
    int section_end[kMaxAxes];   // first pair behind each axis' section
    int block_tokens;            // 1, 2, 4 or 8 tokens of a block
    float eps;
};

// cos and sin of position * frequency. The angle has up to 55 bits: it is taken in
// turns, in 64 bits, and only what is left of the last whole turn is rounded to 32
// (a far position's angle rounded to 32 bits first would be off by 2^-24 of itself).
__device__ __forceinline__ float2 rotation(int position, float freq) {
    const double turns = double(position) * double(freq) * 0.15915494309189535;  // 1 / (2 pi)
    const float part = float(turns - rint(turns));  // -0.5 .. 0.5
    float2 r;
    sincospif(2.f * part, &r.y, &r.x);
    return r;
}

template <int D, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const NormParams p) {
    constexpr int kHeadLanes = D / 8, kHeads = 32 / kHeadLanes;  // of a warp
    __shared__ float2 turn[kNormWarps][D / 2];
    grid_launch_dependents();
    grid_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.block_tokens;
    for (int i = threadIdx.x; i < p.block_tokens * (D / 2); i += kNormThreads) {
        const int pair = i % (D / 2), t = t0 + i / (D / 2);
        if (pair >= p.pairs || t >= p.tokens) continue;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kMaxAxes - 1; ++a) axis += pair >= p.section_end[a];
        turn[i / (D / 2)][pair] = rotation(p.positions[int64_t(axis) * p.tokens + t],
                                           p.inv_freq[pair]);
    }
    __syncthreads();
    // the block's warps share its tokens; blockIdx.y shares a token's heads further
    const int per_token = kNormWarps / p.block_tokens;
    const int t = t0 + warp / per_token;
    if (t >= p.tokens) return;
    const int worker = blockIdx.y * per_token + warp % per_token;
    const int workers = per_token * gridDim.y;
    const int c = lane % kHeadLanes;  // channels 8 c .. 8 c + 7
    // the lane that holds the partners of this lane's channels (kInterleaved: itself)
    const int span = p.pairs / 8;
    const bool turned = 8 * c < 2 * p.pairs, second = c >= span;
    const int partner = kInterleaved || !turned ? lane : second ? lane - span : lane + span;

#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        const uint16_t* x = (part ? p.k : p.q) + t * (part ? p.k_st : p.q_st) + c * 8;
        uint16_t* y = (part ? p.ko : p.qo) + t * (part ? p.ko_st : p.qo_st) + c * 8;
        const int64_t xh = part ? p.k_sh : p.q_sh, yh = part ? p.ko_sh : p.qo_sh;
        const int heads = part ? p.H_kv : p.H_q;
        if (worker * kHeads >= heads) continue;
        // y = r (own x + other x_partner)
        float own[8], other[8];
        {
            const void* w = part ? p.kw : p.qw;
            auto weight = [&](int ch) {
                return !kNorm || !w ? 1.f
                       : p.wide_weights
                           ? static_cast<const float*>(w)[ch]
                           : __uint_as_float(uint32_t(static_cast<const uint16_t*>(w)[ch]) << 16);
            };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ch = 8 * c + i;
                own[i] = weight(ch);
                other[i] = 0.f;
                if (!turned) continue;
                const int pair = kInterleaved ? ch >> 1 : second ? ch - p.pairs : ch;
                const bool up = kInterleaved ? i & 1 : second;
                const int mate = kInterleaved ? ch ^ 1 : second ? pair : ch + p.pairs;
                const float2 cs = turn[warp / per_token][pair];
                own[i] *= cs.x;
                other[i] = weight(mate) * (up ? cs.y : -cs.y);
            }
        }
        const int sub = lane / kHeadLanes;
#pragma unroll 1
        for (int h0 = worker; h0 * kHeads < heads; h0 += workers * kNormBatch) {
            uint4 v[kNormBatch];
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                const int h = (h0 + u * workers) * kHeads + sub;
                v[u] = h < heads ? *reinterpret_cast<const uint4*>(x + h * xh)
                                 : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                if ((h0 + u * workers) * kHeads >= heads) break;
                const uint32_t raw[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                float a[8], b[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[2 * i] = __uint_as_float(raw[i] << 16);
                    a[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
                    if constexpr (kInterleaved) {
                        b[2 * i] = a[2 * i + 1];
                        b[2 * i + 1] = a[2 * i];
                    } else {
                        const uint32_t m = __shfl_sync(0xffffffffu, raw[i], partner);
                        b[2 * i] = __uint_as_float(m << 16);
                        b[2 * i + 1] = __uint_as_float(m & 0xffff0000u);
                    }
                }
                float r = 1.f;
                if constexpr (kNorm) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s0 = fmaf(a[2 * i], a[2 * i], s0);
                        s1 = fmaf(a[2 * i + 1], a[2 * i + 1], s1);
                    }
                    float s = s0 + s1;
#pragma unroll
                    for (int o = kHeadLanes / 2; o > 0; o >>= 1)
                        s += __shfl_xor_sync(0xffffffffu, s, o);
                    r = rsqrtf(s * (1.f / D) + p.eps);
                }
                uint32_t out[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float z[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = 2 * i + e;
                        z[e] = own[k] * a[k];
                        // (channels that are not turned take nothing of another's infinity)
                        if (turned) z[e] = fmaf(other[k], b[k], z[e]);
                        if constexpr (kNorm) z[e] *= r;
                    }
                    out[i] = pack_bf16x2(z[0], z[1]);
                }
                const int h = (h0 + u * workers) * kHeads + sub;
                if (h < heads)
                    *reinterpret_cast<uint4*>(y + h * yh) =
                        make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
    }
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
// arithmetic is slow here (the adds of a batch of 48 rows would take about five times as long as its
// bytes): a lane adds its terms in two 32-bit words, the difference p - q and every sum
// with the exact error of its rounding, and only the lanes' results are added in 64 bits.
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

__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
    __shared__ int first_fall, found, last_some;
    __shared__ double warp_sum[2][kVerifyWarps];
    __shared__ double cta_sum[2][kMaxCluster];  // written by the cluster's CTAs
    __shared__ double scan[kVerifyWarps];
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
    if (threadIdx.x == 0) {
        first_fall = n;
        found = 0x7fffffff;
        last_some = -1;
    }
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
        double sum = (double(s[0].hi) + double(s[1].hi)) + (double(s[0].lo) + double(s[1].lo));
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) warp_sum[round][warp] = sum;
        __syncthreads();
        double mine = 0.0;  // every thread adds in the same order
        for (int i = 0; i < kVerifyWarps; ++i) mine += warp_sum[round][i];
        if (cluster > 1) {
            if (threadIdx.x < cluster)
                st_dsmem_f64(map_to_rank(smem_u32(&cta_sum[round][rank]), threadIdx.x), mine);
            cluster_arrive_release();
            cluster_wait_acquire();
        } else {
            if (threadIdx.x == 0) cta_sum[round][0] = mine;
            __syncthreads();
        }
        double total = 0.0;
        for (int i = 0; i < cluster; ++i) total += cta_sum[round][i];
        if (total > 0.0 && total < INFINITY) {
            // the CTA, then the warp's piece in which the sum passes the threshold (the
            // last one with any weight if rounding keeps it below)
            const double limit = double(p.u_sample[b]) * total;
            double before = 0.0;
            int owner = -1, last = 0;
            double owner_before = 0.0, last_before = 0.0;
            for (int i = 0; i < cluster; ++i) {
                const double c = cta_sum[round][i];
                if (c > 0.0) {
                    last = i;
                    last_before = before;
                }
                if (owner < 0 && before + c > limit) {
                    owner = i;
                    owner_before = before;
                }
                before += c;
            }
            if (owner < 0) {
                owner = last;
                owner_before = last_before;
            }
            if (owner != rank) return;
            before = owner_before;
            owner = -1;
            last = 0;
            for (int i = 0; i < kVerifyWarps; ++i) {
                const double c = warp_sum[round][i];
                if (c > 0.0) {
                    last = i;
                    last_before = before;
                }
                if (owner < 0 && before + c > limit) {
                    owner = i;
                    owner_before = before;
                }
                before += c;
            }
            if (owner < 0) {
                owner = last;
                owner_before = last_before;
            }
            // that piece again, a run of consecutive elements for each thread
            const int64_t from = (int64_t(rank) * kVerifyWarps + owner) * p.piece;
            const int each = (p.piece + kVerifyThreads - 1) / kVerifyThreads;
            const int lo = int(min(int64_t(p.V), from + int64_t(threadIdx.x) * each));
            const int hi = int(min(min(int64_t(p.V), from + p.piece), int64_t(lo) + each));
            auto term = [&](int e) {
                if (e == gone) return 0.0;
                const double d = double(pr[e]) - (qr ? double(qr[e]) : 0.0);
                return d > 0.0 ? d : 0.0;
            };
            double run = 0.0;
            for (int e = lo; e < hi; ++e) run += term(e);
            double incl = run;
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) scan[warp] = incl;
            __syncthreads();
            double at = owner_before;
            for (int i = 0; i < warp; ++i) at += scan[i];
            at += incl - run;
            if (run > 0.0) {
                int some = lo;
                for (int e = lo; e < hi; ++e) {
                    const double w = term(e);
                    if (w <= 0.0) continue;
                    some = e;
                    at += w;
                    if (at > limit) {
                        atomicMin(&found, e);
                        break;
                    }
                }
                atomicMax(&last_some, some);
            }
            __syncthreads();
            if (threadIdx.x == 0) p.next[b] = found != 0x7fffffff ? found : last_some;
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
    const int rounds = (H_q * (d / 8) + 31) / 32;  // of one warp for a token's query heads
    int block_tokens = 4, split = 1;
    while (block_tokens > 1 && tokens < block_tokens * 4 * sms) block_tokens /= 2;
    while (tokens * split < 2 * sms && split * 8 < rounds) ++split;
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
