// rope.cu -- rotary positions, and the append of a step's keys and values to
// a paged cache.
//
//   pair (a, b) of a head, i < R/2: a = x[i], b = x[i + R/2] (half layout) or
//   x[2i], x[2i + 1] (interleaved):
//     t = pos f_i,  a' = m (a cos t - b sin t),  b' = m (a sin t + b cos t)
//   elements from R on are copied; k' and v go to the token's cache slot.
//
// Memory bound: every q, k and v element is read once and written once, in
// one launch.  The angle is made once per (token, pair) and shared by all
// heads; the product pos * f and its reduction to +-pi are fp64 (in fp32 an
// angle at position 10^6 would be off by 0.03 rad), the sine and cosine of
// the reduced angle fp32.
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr int RP_THREADS = 256;

// sequence of token t: the last b with q_start[b] <= t, or -1 when no
// sequence holds the row (rows behind the last one are left as they were)
__device__ __forceinline__ int rope_seq(const RopeArgs &a, int t)
{
    int lo = 0, hi = a.batch;   // q_start[lo] <= t < q_start[hi], if any
    if (t < a.q_start[0] || t >= a.q_start[a.batch])
        return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct U8 {
    uint16_t e[8];
};

// 8 consecutive elements, as one 16-byte access or one by one
template <bool VEC>
__device__ __forceinline__ U8 ld8(const uint16_t *p, int n)
{
    U8 u;
    if (VEC) {
        *reinterpret_cast<uint4 *>(&u) = *reinterpret_cast<const uint4 *>(p);
    } else {
        for (int i = 0; i < 8; ++i)
            u.e[i] = i < n ? p[i] : (uint16_t)0;
    }
    return u;
}
template <bool VEC>
__device__ __forceinline__ void st8(uint16_t *p, const U8 &u, int n)
{
    if (VEC) {
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&u);
    } else {
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = u.e[i];
    }
}

// One CTA per token.  VEC: every 8-element unit and its partner are whole and
// 16-byte aligned; otherwise the same walk with single elements.
template <class T, bool VEC>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];   // [rot / 2] m cos, m sin
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = a.rot >> 1;
    int seq = -1, slot = 0;
    if (a.batch > 0) {
        seq = rope_seq(a, t);
        if (seq < 0)
            return;
        slot = max(a.kv_len[seq], 0) - a.q_start[seq + 1] + t;
    }
    const int pos = a.positions ? a.positions[t] : slot;
    for (int i = tid; i < half; i += RP_THREADS) {
        const double ang = (double)pos * a.inv_freq[i];
        const double r = fma(-6.283185307179586, rint(ang * 0.15915494309189535), ang);
        float sn, c;
        sincosf((float)r, &sn, &c);
        cs[i] = make_float2(a.scale * c, a.scale * sn);
    }
    // where this token's keys and values go
    long long base = -1;
    if (a.k) {
        const long long room = (long long)a.max_pages * a.page_size;
        if (slot >= 0 && slot < room) {
            const int pg = slot / a.page_size;
            const int id = a.table[(size_t)seq * a.max_pages + pg];
            if ((unsigned)id < (unsigned)a.num_pages)
                base = id * a.page_stride + (long long)(slot - pg * a.page_size) * a.token_stride;
        }
        if (base < 0 && tid == 0)
            flag_status(a.status, QMOE_DEV_BAD_PAGE);
    }
    __syncthreads();
    // units of a head: the rotated part's pairs of 8 (half layout: first-half
    // unit with its partner; interleaved: one unit), then the copied rest
    const int pu = a.interleaved ? (a.rot + 7) / 8 : (half + 7) / 8;
    const int ru = (a.dim - a.rot + 7) / 8;
    const int hu = pu + ru;
    const int nq = a.q ? a.heads : 0, nk = base >= 0 ? a.kv_heads : 0;
    const int vu = (a.dim + 7) / 8;
    const int total = (nq + nk) * hu + nk * vu;
    for (int i = tid; i < total; i += RP_THREADS) {
        int h = i / hu, u = i - h * hu;
        const uint16_t *src;
        uint16_t *dst;
        if (h < nq) {
            src = a.q + t * a.q_token + h * a.q_head;
            dst = a.q_out + t * a.qo_token + h * a.qo_head;
        } else if (h < nq + nk) {
            h -= nq;
            src = a.k + t * a.k_token + h * a.k_head;
            dst = a.ck + base + h * a.head_stride;
        } else {
            const int iv = i - (nq + nk) * hu;
            h = iv / vu;
            u = (iv - h * vu) * 8;
            src = a.v + t * a.v_token + h * a.v_head + u;
            dst = a.cv + base + h * a.head_stride + u;
            st8<VEC>(dst, ld8<VEC>(src, a.dim - u), a.dim - u);
            continue;
        }
        if (u >= pu) {
            const int e = a.rot + (u - pu) * 8;
            st8<VEC>(dst + e, ld8<VEC>(src + e, a.dim - e), a.dim - e);
        } else if (a.interleaved) {
            const int e = u * 8, n = a.rot - e;
            U8 x = ld8<VEC>(src + e, n);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (VEC || 2 * j < n) {
                    const float2 w = cs[e / 2 + j];
                    const float p = Num16<T>::up(x.e[2 * j]), q = Num16<T>::up(x.e[2 * j + 1]);
                    x.e[2 * j] = Num16<T>::down(p * w.x - q * w.y);
                    x.e[2 * j + 1] = Num16<T>::down(p * w.y + q * w.x);
                }
            st8<VEC>(dst + e, x, n);
        } else {
            const int e = u * 8, n = half - e;
            U8 x = ld8<VEC>(src + e, n), y = ld8<VEC>(src + half + e, n);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (VEC || j < n) {
                    const float2 w = cs[e + j];
                    const float p = Num16<T>::up(x.e[j]), q = Num16<T>::up(y.e[j]);
                    x.e[j] = Num16<T>::down(p * w.x - q * w.y);
                    y.e[j] = Num16<T>::down(p * w.y + q * w.x);
                }
            st8<VEC>(dst + e, x, n);
            st8<VEC>(dst + half + e, y, n);
        }
    }
}

template <class T>
cudaError_t launch_t(const RopeArgs &a, const LaunchCfg &c)
{
    auto al = [](const void *p, long long s0, long long s1) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0);
    };
    const bool vec = a.dim % 8 == 0 && (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0) &&
                     al(a.q, a.q_token, a.q_head) && al(a.q_out, a.qo_token, a.qo_head) &&
                     al(a.k, a.k_token, a.k_head) && al(a.v, a.v_token, a.v_head) &&
                     al(a.ck, a.token_stride, a.head_stride) && al(a.cv, a.page_stride, 0);
    LaunchCfg c2 = c;
    c2.pdl = false;
    const size_t smem = (size_t)(a.rot / 2) * 8;
    auto kern = vec ? rope_kernel<T, true> : rope_kernel<T, false>;
    return launch_ex(kern, dim3(a.tokens), dim3(RP_THREADS), smem, c2, 1, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool bf16, const LaunchCfg &c)
{
    return bf16 ? launch_t<__nv_bfloat16>(a, c) : launch_t<__half>(a, c);
}

}  // namespace qmoe
