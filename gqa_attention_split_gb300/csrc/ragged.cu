// Attention over ragged batches: packed prompts, and drafted token trees on
// top of the KV cache; and appending packed tokens to the cache.
//
//   O = softmax(scale * Q K^T over the visible keys) V,   lse = ln sum exp(.)
//
// Both calls stream the same two sources of keys per row of the batch: the
// context in the cache (decode_tree only; every slot below context_lens[b] is
// visible), then the row's own packed tokens (prefill_packed: a causal limit
// or all of them; decode_tree: the bits of a mask, or a line). A key that a
// query does not see never reaches its result, whatever K and V hold there.

#include <cuda_runtime.h>
#include <math.h>

#include "gqa_attn.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "runtime.cuh"

namespace gqa {
namespace ragged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTreeTokens = 128;

struct Params {
    const uint16_t *q, *k, *v;    // packed [total, heads, d], strides below
    const uint16_t *kc, *vc;      // cache [B, H_kv, S_max, d] (decode_tree)
    uint16_t* o;                  // [total_q, H_q, d]
    float* lse;                   // [total_q, H_q] or null
    const int32_t *cu_q, *cu_k, *ctx;
    const uint32_t* mask;         // [total_q, mask_words] or null
    unsigned* status;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
    int B, H_q, H_kv, G, total_q, total_k, S_max, max_tokens, mask_words, causal, tree;
    float scale_log2;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// First packed token and token count of row b under prefix sums cu (null:
// every row has total / B tokens). Bad prefix sums are clamped: the row stays
// inside [0, total), and *bad is set.
__device__ __forceinline__ void row_range(const int32_t* cu, int B, int total, int b, int& first,
                                          int& count, bool& bad) {
    if (!cu) {
        count = total / B;
        first = b * count;
        return;
    }
    const int a = cu[b], e = cu[b + 1];
    first = clampi(a, 0, total);
    const int last = clampi(e, first, total);
    count = last - first;
    bad = bad || first != a || last != e;
}

__device__ __forceinline__ int context_of(const Params& p, int b, bool& bad) {
    const int c = p.ctx[b], n = clampi(c, 0, p.S_max);
    bad = bad || n != c;
    return n;
}

// One warp per (packed token, query head).
template <int D>
__global__ void __launch_bounds__(256) rows_kernel(const Params p) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (w >= int64_t(p.total_q) * p.H_q) return;
    const int tok = int(w / p.H_q), h = int(w % p.H_q), hk = h / p.G;
    int b = 0, q0 = 0, T = 0;
    bool bad = false;
    for (; b < p.B; ++b) {
        row_range(p.cu_q, p.B, p.total_q, b, q0, T, bad);
        if (p.tree && T > p.max_tokens) {
            T = p.max_tokens;
            bad = true;
        }
        if (tok >= q0 && tok < q0 + T) break;
    }
    if (bad && lane == 0) atomicOr(p.status, kStatusBadSeqlen);
    if (b == p.B) return;  // behind the last sequence
    const int t = tok - q0;
    int k0 = q0, n_own = T, ctx = 0;
    if (p.cu_k) row_range(p.cu_k, p.B, p.total_k, b, k0, n_own, bad);
    if (p.tree) ctx = context_of(p, b, bad);
    if (bad && lane == 0) atomicOr(p.status, kStatusBadSeqlen);
    const int lim = p.causal ? clampi(n_own - T + t + 1, 0, n_own) : n_own;
    float qv[kPer], acc[kPer], m = -INFINITY, l = 0.f;
    for (int i = 0; i < kPer; ++i) {
        qv[i] = __uint_as_float(uint32_t(p.q[tok * p.q_st + h * p.q_sh + lane * kPer + i]) << 16);
        acc[i] = 0.f;
    }
    for (int j = 0; j < ctx + n_own; ++j) {
        const uint16_t *kr, *vr;
        if (j < ctx) {
            const size_t at = ((size_t(b) * p.H_kv + hk) * p.S_max + j) * D;
            kr = p.kc + at;
            vr = p.vc + at;
        } else {
            const int i = j - ctx;
            const bool seen = p.mask ? (p.mask[size_t(tok) * p.mask_words + (i >> 5)] >> (i & 31)) & 1
                                     : i < lim;
            if (!seen) continue;
            kr = p.k + (k0 + i) * p.k_st + hk * p.k_sh;
            vr = p.v + (k0 + i) * p.v_st + hk * p.v_sh;
        }
        float s = 0.f;
        for (int i = 0; i < kPer; ++i)
            s += qv[i] * __uint_as_float(uint32_t(kr[lane * kPer + i]) << 16);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        if (mn == -INFINITY) continue;
        const float corr = exp2f(m - mn), e = exp2f(s - mn);
        m = mn;
        l = l * corr + e;
        for (int i = 0; i < kPer; ++i)
            acc[i] = acc[i] * corr + e * __uint_as_float(uint32_t(vr[lane * kPer + i]) << 16);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < kPer; ++i)
        p.o[size_t(w) * D + lane * kPer + i] =
            __bfloat16_as_ushort(__float2bfloat16_rn(acc[i] * inv));
    if (lane == 0 && p.lse) p.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

bool bad_strides(int64_t st, int64_t sh, int64_t tokens, int heads) {
    // TMA strides are multiples of 16 bytes below 2^40
    const int64_t lim = int64_t(1) << 39;
    if (heads > 1 && (sh <= 0 || sh >= lim)) return true;
    return tokens > 1 && (st <= 0 || st >= lim);
}
bool odd_strides(int64_t st, int64_t sh) { return (st | sh) & 7; }

int check_common(const void* q, const void* k, const void* v, const void* o, const void* lse,
                 int B, int H_q, int H_kv, int d, float scale) {
    if (B < 0 || B > 65535 || H_q <= 0 || H_kv <= 0) return GQA_ERR_INVALID_ARG;
    // scale > 0: the row maximum is taken over the raw scores
    if (H_q % H_kv != 0 || !isfinite(scale) || !(scale > 0.f)) return GQA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return GQA_ERR_MISALIGNED;
    return GQA_OK;
}

int launch_rows(const Params& p, int d, cudaStream_t stream) {
    const int64_t warps = int64_t(p.total_q) * p.H_q;
    const unsigned grid = unsigned((warps + 7) / 8);
    if (d == 128)
        rows_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        rows_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// ------------------------------------------------------------ cache append

struct AppendParams {
    uint16_t *kc, *vc;
    const uint16_t *k, *v;
    const int32_t *cu, *starts, *index;
    unsigned* status;
    int64_t k_st, k_sh, v_st, v_sh;
    int B, H_kv, d, S_max, total, total_new;
};

// One warp per entry: K and V of one token, every head.
__global__ void __launch_bounds__(128) append_kernel(const AppendParams p) {
    const int lane = threadIdx.x & 31;
    const int e = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (e >= p.total) return;
    bool bad = false;
    int b = 0, first = 0, n = 0;
    for (; b < p.B; ++b) {
        row_range(p.cu, p.B, p.total, b, first, n, bad);
        if (e >= first && e < first + n) break;
    }
    if (bad && lane == 0) atomicOr(p.status, kStatusBadSeqlen);
    if (b == p.B) return;
    const int64_t slot = int64_t(p.starts[b]) + (e - first);
    const int src = p.index ? p.index[e] : e;
    if (slot < 0 || slot >= p.S_max || src < 0 || src >= p.total_new) {
        if (lane == 0) atomicOr(p.status, kStatusBadSeqlen);
        return;
    }
    const int per = p.d / 8;
    for (int i = lane; i < p.H_kv * per; i += 32) {
        const int h = i / per, c = i % per;
        const size_t dst = ((size_t(b) * p.H_kv + h) * p.S_max + slot) * p.d + c * 8;
        *reinterpret_cast<uint4*>(p.kc + dst) =
            *reinterpret_cast<const uint4*>(p.k + src * p.k_st + h * p.k_sh + c * 8);
        *reinterpret_cast<uint4*>(p.vc + dst) =
            *reinterpret_cast<const uint4*>(p.v + src * p.v_st + h * p.v_sh + c * 8);
    }
}

}  // namespace ragged
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_attn_prefill_packed(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                       uint16_t* o, float* lse, const int32_t* cu_q,
                                       const int32_t* cu_k, int B, int H_q, int H_kv, int d,
                                       int total_q, int total_k, int64_t q_stride_t,
                                       int64_t q_stride_h, int64_t k_stride_t,
                                       int64_t k_stride_h, int64_t v_stride_t,
                                       int64_t v_stride_h, int causal, float scale,
                                       cudaStream_t stream) {
    using namespace ragged;
    const int rc = check_common(q, k, v, o, lse, B, H_q, H_kv, d, scale);
    if (rc != GQA_OK) return rc;
    if (!cu_q || total_q < 0 || total_k < 0 || (total_q > 0 && (!q || !o)) ||
        (total_k > 0 && (!k || !v)) || (!cu_k && total_k != total_q))
        return GQA_ERR_INVALID_ARG;
    if (H_q / H_kv > 128) return GQA_ERR_UNSUPPORTED;
    if (bad_strides(q_stride_t, q_stride_h, total_q, H_q) ||
        bad_strides(k_stride_t, k_stride_h, total_k, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total_k, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (odd_strides(q_stride_t, q_stride_h) || odd_strides(k_stride_t, k_stride_h) ||
        odd_strides(v_stride_t, v_stride_h) || (reinterpret_cast<uintptr_t>(cu_q) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_k) & 3u))
        return GQA_ERR_MISALIGNED;
    if (B == 0 || total_q == 0) return GQA_OK;
    Params p{};
    p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
    p.cu_q = cu_q; p.cu_k = cu_k;
    p.status = status_word();
    if (!p.status) return GQA_ERR_CUDA;
    p.q_st = q_stride_t; p.q_sh = q_stride_h; p.k_st = k_stride_t; p.k_sh = k_stride_h;
    p.v_st = v_stride_t; p.v_sh = v_stride_h;
    p.B = B; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv; p.total_q = total_q; p.total_k = total_k;
    p.causal = causal != 0;
    p.scale_log2 = scale * kLog2e;
    return launch_rows(p, d, stream);
}

extern "C" size_t gqa_attn_decode_tree_workspace_size(int H_q, int H_kv, int d, int max_tokens) {
    if (H_q <= 0 || H_kv <= 0 || H_q % H_kv || (d != 64 && d != 128) || max_tokens < 1 ||
        max_tokens > ragged::kMaxTreeTokens || H_q / H_kv > 16)
        return 0;
    return 256;
}

extern "C" int gqa_attn_decode_tree(
    const uint16_t* q, const uint16_t* k_new, const uint16_t* v_new, const uint16_t* k_cache,
    const uint16_t* v_cache, uint16_t* o, float* lse, const int32_t* cu_seqlens,
    const int32_t* context_lens, const int32_t* tree_mask, int mask_words, int B, int H_q,
    int H_kv, int d, int total, int max_tokens, int S_max, int64_t q_stride_t,
    int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
    int64_t v_stride_h, float scale, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
    using namespace ragged;
    const int rc = check_common(q, k_new, v_new, o, lse, B, H_q, H_kv, d, scale);
    if (rc != GQA_OK) return rc;
    const bool empty = B == 0 || total == 0;  // nothing to do: the tensors may be null
    if ((!empty && (!q || !k_new || !v_new || !k_cache || !v_cache || !o || !context_lens ||
                    !workspace)) ||
        total < 0 || S_max < 1 || max_tokens < 1 || (B > 0 && !cu_seqlens && total % B != 0) ||
        (B > 0 && !cu_seqlens && total / B > max_tokens) ||
        (tree_mask && int64_t(mask_words) * 32 < max_tokens))
        return GQA_ERR_INVALID_ARG;
    if (H_q / H_kv > 16 || max_tokens > kMaxTreeTokens ||
        int64_t(B) * H_kv * S_max >= (int64_t(1) << 31))
        return GQA_ERR_UNSUPPORTED;
    if (bad_strides(q_stride_t, q_stride_h, total, H_q) ||
        bad_strides(k_stride_t, k_stride_h, total, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (odd_strides(q_stride_t, q_stride_h) || odd_strides(k_stride_t, k_stride_h) ||
        odd_strides(v_stride_t, v_stride_h) || !aligned16(k_cache) || !aligned16(v_cache) ||
        ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(tree_mask)) & 3u))
        return GQA_ERR_MISALIGNED;
    if (!empty && ((reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max_tokens)))
        return GQA_ERR_WORKSPACE;
    if (empty) return GQA_OK;
    Params p{};
    p.q = q; p.k = k_new; p.v = v_new; p.kc = k_cache; p.vc = v_cache; p.o = o; p.lse = lse;
    p.cu_q = cu_seqlens; p.ctx = context_lens;
    p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.status = status_word();
    if (!p.status) return GQA_ERR_CUDA;
    p.q_st = q_stride_t; p.q_sh = q_stride_h; p.k_st = k_stride_t; p.k_sh = k_stride_h;
    p.v_st = v_stride_t; p.v_sh = v_stride_h;
    p.B = B; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv; p.total_q = total; p.total_k = total;
    p.S_max = S_max; p.max_tokens = max_tokens; p.mask_words = mask_words;
    p.causal = 1; p.tree = 1;
    p.scale_log2 = scale * kLog2e;
    return launch_rows(p, d, stream);
}

extern "C" int gqa_attn_cache_append(uint16_t* k_cache, uint16_t* v_cache, const uint16_t* k_new,
                                     const uint16_t* v_new, const int32_t* cu_seqlens,
                                     const int32_t* starts, const int32_t* index, int B,
                                     int H_kv, int d, int S_max, int total, int total_new,
                                     int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                                     int64_t v_stride_h, cudaStream_t stream) {
    using namespace ragged;
    const bool empty = B == 0 || total == 0;
    if ((!empty && (!k_cache || !v_cache || !starts)) || B < 0 || B > 65535 || H_kv <= 0 ||
        S_max < 1 || total < 0 || total_new < 0 || (total_new > 0 && (!k_new || !v_new)) ||
        (!index && total > total_new) || (B > 0 && !cu_seqlens && total % B != 0))
        return GQA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED;
    if (int64_t(B) * H_kv * S_max >= (int64_t(1) << 31)) return GQA_ERR_UNSUPPORTED;
    if (bad_strides(k_stride_t, k_stride_h, total_new, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total_new, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_new) || !aligned16(v_new) ||
        odd_strides(k_stride_t, k_stride_h) || odd_strides(v_stride_t, v_stride_h) ||
        ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(starts) |
          reinterpret_cast<uintptr_t>(index)) & 3u))
        return GQA_ERR_MISALIGNED;
    if (empty) return GQA_OK;
    unsigned* status = status_word();
    if (!status) return GQA_ERR_CUDA;
    const AppendParams p{k_cache, v_cache, k_new, v_new, cu_seqlens, starts, index, status,
                         k_stride_t, k_stride_h, v_stride_t, v_stride_h, B, H_kv, d, S_max,
                         total, total_new};
    append_kernel<<<unsigned((total + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}
