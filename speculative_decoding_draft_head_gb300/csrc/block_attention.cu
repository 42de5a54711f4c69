// Attention of each request's block rows over a shared prefix and the
// request's own tokens, both in the quantised cache.
//
// One block per (packed row, query head): its warps take every fourth token,
// lanes hold four elements of the head each, and a running maximum and sum
// carry the softmax in one pass over the tokens.
#include "paged_rows.cuh"

namespace dspark {
namespace {

constexpr int kWarps = 4;

template <typename T, int kFormat>
__global__ void __launch_bounds__(kWarps * 32)
attention_rows_kernel(AttentionArgs a) {
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kMaxHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x, head = blockIdx.y;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, ps = c.page_size, h = head / (a.n_q_heads / c.n_kv_heads);
    if (r == 0 && head == 0)
        for (int i = threadIdx.x; i <= a.rows.B; i += blockDim.x) {
            const int64_t x = a.rows.row0[i], y = i > 0 ? a.rows.row0[i - 1] : 0;
            if (x < y || x > a.rows.n_rows) atomicOr(c.flags, kFlagBadLength);
        }
    const int b = find_request(a.rows.row0, a.rows.B, r, lane);
    if (b < 0) return;
    const int64_t first = a.rows.row0[b], n = a.rows.row0[b + 1] - first;
    const int len = a.rows.start[b];
    const bool bad = first < 0 || len < n || (int64_t)len > (int64_t)a.rows.max_pages * ps || (a.row_mask && n > 64);
    const int i = (int)(r - first), ctx = (int)(len - n);
    const uint64_t seen = a.row_mask ? a.row_mask[r] : 0;
    const float c2 = a.scale * kLog2e;

    float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.f;
    if (lane * 4 < D) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const T *>(a.q) + r * a.q_stride +
                                                         (int64_t)head * D + lane * 4);
        const float2 x = pair_to_float<T>(w.x), y = pair_to_float<T>(w.y);
        q[0] = x.x, q[1] = x.y, q[2] = y.x, q[3] = y.y;
    }
    if (bad) {
        if (threadIdx.x == 0) atomicOr(c.flags, kFlagBadLength);
        m = l = NAN;
    }
    const int total = bad ? 0 : a.prefix_len + len;
    for (int j = warp; j < total; j += kWarps) {
        const int t = j - a.prefix_len;
        if (t >= ctx) {
            const int u = t - ctx;
            if (a.row_mask ? !((seen >> u) & 1) : (a.mask == DSPARK_MASK_CAUSAL && u > i)) continue;
        }
        const int pos = t < 0 ? j : t, slot = pos / ps;
        const int page = t < 0 ? a.prefix_pages[slot] : a.rows.block_table[(int64_t)b * a.rows.max_pages + slot];
        if (page < 0 || page >= c.n_pages) {
            if (lane == 0) atomicOr(c.flags, kFlagBadPage);
            m = l = NAN;
            break;
        }
        const int64_t at = ((int64_t)page * c.n_kv_heads + h) * ps + (pos - slot * ps);
        __half2 k2[2] = {}, v2[2] = {};
        if (lane * 4 < D) {
            decode4<kFormat>(*reinterpret_cast<const uint32_t *>(static_cast<const char *>(c.k) + at * D + lane * 4), k2[0], k2[1]);
            decode4<kFormat>(*reinterpret_cast<const uint32_t *>(static_cast<const char *>(c.v) + at * D + lane * 4), v2[0], v2[1]);
        }
        const float2 k0 = __half22float2(k2[0]), k1 = __half22float2(k2[1]);
        float s = q[0] * k0.x + q[1] * k0.y + q[2] * k1.x + q[3] * k1.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= c.k_scale[at] * c2;
        const float m_new = s > m ? s : m;  // a NaN score leaves m and makes p NaN
        const float f = m == -INFINITY ? 0.f : exp2f(m - m_new), p = exp2f(s - m_new), pv = p * c.v_scale[at];
        const float2 v0 = __half22float2(v2[0]), v1 = __half22float2(v2[1]);
        l = l * f + p;
        o[0] = o[0] * f + pv * v0.x, o[1] = o[1] * f + pv * v0.y;
        o[2] = o[2] * f + pv * v1.x, o[3] = o[3] * f + pv * v1.y;
        m = m_new;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < 4; ++e) so[warp][lane * 4 + e] = o[e];
    __syncthreads();
    if (warp != 0) return;
    float mm = -INFINITY, ll = 0.f, acc[4] = {};
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < kWarps; ++w) {
        const float f = sm[w] == -INFINITY && sl[w] == 0.f ? 0.f : exp2f(sm[w] - mm);
        ll += f * sl[w];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += f * so[w][lane * 4 + e];
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    if (lane * 4 < D) {
        uint2 w;
        w.x = float_to_pair<T>(acc[0] * inv, acc[1] * inv);
        w.y = float_to_pair<T>(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + ((int64_t)r * a.n_q_heads + head) * D + lane * 4) = w;
    }
    if (lane == 0 && a.lse)
        a.lse[(int64_t)r * a.n_q_heads + head] = ll == 0.f ? -INFINITY : kLn2 * (mm + log2f(ll));
}

}  // namespace

size_t attention_ws_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_block_attention(const AttentionArgs &a, cudaStream_t s) {
    const dim3 grid(a.rows.n_rows, a.n_q_heads);
    const bool e4m3 = a.cache.format == DSPARK_KV_E4M3;
    if (a.dt == DSPARK_BF16) {
        if (e4m3) attention_rows_kernel<__nv_bfloat16, DSPARK_KV_E4M3><<<grid, kWarps * 32, 0, s>>>(a);
        else attention_rows_kernel<__nv_bfloat16, DSPARK_KV_INT8><<<grid, kWarps * 32, 0, s>>>(a);
    } else {
        if (e4m3) attention_rows_kernel<__half, DSPARK_KV_E4M3><<<grid, kWarps * 32, 0, s>>>(a);
        else attention_rows_kernel<__half, DSPARK_KV_INT8><<<grid, kWarps * 32, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace dspark
