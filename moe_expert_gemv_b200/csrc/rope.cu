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
// the reduced angle fp32.  A CTA is a token; what it waits for -- which
// sequence, how long it is, which page -- is three loads in a row, so its
// first two units per thread are on their way before.  Measured, in a graph
// of 20 calls: 5325 tokens of 32 + 8 + 8 heads of 128 (133 MB), 28.9 us, 4.6 TB/s
// (a plain elementwise kernel over as many bytes: 24); 7 tokens 3.1 us; 5325
// tokens' queries alone (87 MB), 19.4.  The rest is the issue of instructions,
// 74% of the cycles.  One replay at a time CTAs of 128 threads took 31.0 in
// place of 32.4 at that size but 6.2 in place of 4.2 for the 7 tokens.
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr int RP_THREADS = 256;

// Sequence of token t, the last b with q_start[b] <= t, or -1 when no
// sequence holds the row (rows behind the last one are left as they were): a
// warp looks at 32 places at a time.
__device__ __forceinline__ int rope_seq(const RopeArgs &a, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = a.batch + 1;   // the last of q_start[lo .. lo + n) that is <= t
    while (true) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool le = lane * step < n && a.q_start[at] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m == 0)
            return -1;
        const int l = 31 - __clz(m);
        lo += l * step;
        n = min(step, n - l * step);
        if (step == 1)
            break;
    }
    return lo < a.batch ? lo : -1;
}

union U8 {
    uint4 q;
    uint32_t w[4];
    uint16_t e[8];
};

// 8 consecutive elements, as one 16-byte access or one by one
template <bool VEC>
__device__ __forceinline__ U8 ld8(const uint16_t *p, int n)
{
    U8 u;
    if (VEC) {
        u.q = *reinterpret_cast<const uint4 *>(p);
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
        *reinterpret_cast<uint4 *>(p) = u.q;
    } else {
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = u.e[i];
    }
}

// What a thread does with unit i of a token: 8 elements and, in the half
// layout, their partners.
struct Unit {
    const uint16_t *src;
    uint16_t *dst;
    int e;      // first pair or element, -1: copy only
    int n;      // elements that are there
};

// One CTA per token.  VEC: every 8-element unit and its partner are whole and
// 16-byte aligned; otherwise the same walk with single elements.
template <class T, bool VEC>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const RopeArgs a)
{
    extern __shared__ __align__(16) float2 cs[];   // [rot / 2, rounded up to even] m cos, m sin
    const int t = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int half = a.rot >> 1;
    // units of a head: the rotated part's pairs of 8 (half layout: first-half
    // unit with its partner; interleaved: one unit), then the copied rest
    const int pu = a.interleaved ? (a.rot + 7) / 8 : (half + 7) / 8;
    const int ru = (a.dim - a.rot + 7) / 8;
    const int hu = pu + ru, vu = (a.dim + 7) / 8;
    const int nq = a.q ? a.heads : 0, nk = a.k ? a.kv_heads : 0;
    const int total = (nq + nk) * hu + nk * vu;
    auto unit = [&](int i) {   // its destination in the cache: from the token's place on
        Unit w;
        int h = a.by_unit(i), u = i - h * hu;
        if (h < nq) {
            w.src = a.q + t * a.q_token + h * a.q_head;
            w.dst = a.q_out + t * a.qo_token + h * a.qo_head;
        } else if (h < nq + nk) {
            h -= nq;
            w.src = a.k + t * a.k_token + h * a.k_head;
            w.dst = a.ck + h * a.head_stride;
        } else {
            const int iv = i - (nq + nk) * hu;
            h = a.by_v(iv);
            u = iv - h * vu;
            w.src = a.v + t * a.v_token + h * a.v_head + u * 8;
            w.dst = a.cv + h * a.head_stride + u * 8;
            w.e = -1;
            w.n = a.dim - u * 8;
            return w;
        }
        if (u >= pu) {
            const int e = a.rot + (u - pu) * 8;
            w.src += e;
            w.dst += e;
            w.e = -1;
            w.n = a.dim - e;
        } else {
            w.src += u * 8;
            w.dst += u * 8;
            w.e = a.interleaved ? u * 4 : u * 8;
            w.n = (a.interleaved ? a.rot : half) - u * 8;
        }
        return w;
    };
    constexpr int AHEAD = 2;
    Unit w[AHEAD];
    U8 x[AHEAD], y[AHEAD];
    auto fetch = [&](int k, int i) {
        w[k] = unit(i);
        x[k] = ld8<VEC>(w[k].src, w[k].n);
        if (w[k].e >= 0 && !a.interleaved)
            y[k] = ld8<VEC>(w[k].src + half, w[k].n);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (tid + k * RP_THREADS < total)
            fetch(k, tid + k * RP_THREADS);

    int seq = -1, slot = 0;
    if (a.batch > 0) {
        seq = rope_seq(a, t);
        if (seq < 0)
            return;
        slot = max(a.kv_len[seq], 0) - a.q_start[seq + 1] + t;
    }
    const int pos = a.positions ? a.positions[t] : slot;
    // where this token's keys and values go
    long long base = -1;
    if (a.k) {
        const long long room = (long long)a.max_pages * a.page_size;
        if (slot >= 0 && slot < room) {
            const int pg = a.by_page(slot);
            const int id = a.table[(size_t)seq * a.max_pages + pg];
            if ((unsigned)id < (unsigned)a.num_pages)
                base = id * a.page_stride + (long long)(slot - pg * a.page_size) * a.token_stride;
        }
        if (base < 0 && tid == 0)
            flag_status(a.status, QMOE_DEV_BAD_PAGE);
    }
    for (int i = tid; i < half; i += RP_THREADS) {
        const double ang = (double)pos * a.inv_freq[i];
        const double r = fma(-6.283185307179586, rint(ang * 0.15915494309189535), ang);
        float sn, c;
        sincosf((float)r, &sn, &c);
        cs[i] = make_float2(a.scale * c, a.scale * sn);
    }
    __syncthreads();
    for (int i0 = tid; i0 < total; i0 += AHEAD * RP_THREADS) {
        if (i0 != tid) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i0 + k * RP_THREADS < total)
                    fetch(k, i0 + k * RP_THREADS);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k * RP_THREADS;
            if (i >= total)
                break;
            uint16_t *dst = w[k].dst;
            if (i >= nq * hu) {   // keys and values: in the cache, if it has the place
                if (base < 0)
                    continue;
                dst += base;
            }
            const int n = w[k].n;
            if (w[k].e < 0) {
                st8<VEC>(dst, x[k], n);
            } else if (a.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (VEC || 2 * j < n) {
                        const float2 c = cs[w[k].e + j];
                        const float2 v = Num16<T>::up2(x[k].w[j]);
                        x[k].w[j] = Num16<T>::down2(v.x * c.x - v.y * c.y, v.x * c.y + v.y * c.x);
                    }
                st8<VEC>(dst, x[k], n);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (VEC || 2 * j < n) {
                        const float4 c = *reinterpret_cast<const float4 *>(cs + w[k].e + 2 * j);   // two pairs'
                        const float2 p = Num16<T>::up2(x[k].w[j]), q = Num16<T>::up2(y[k].w[j]);
                        x[k].w[j] = Num16<T>::down2(p.x * c.x - q.x * c.y, p.y * c.z - q.y * c.w);
                        y[k].w[j] = Num16<T>::down2(p.x * c.y + q.x * c.x, p.y * c.w + q.y * c.z);
                    }
                st8<VEC>(dst, x[k], n);
                st8<VEC>(dst + half, y[k], n);
            }
        }
    }
}

template <class T>
cudaError_t launch_t(const RopeArgs &args, const LaunchCfg &c)
{
    RopeArgs a = args;
    const int pairs = a.interleaved ? (a.rot + 7) / 8 : (a.rot / 2 + 7) / 8;   // the kernel's units of a head
    a.by_unit = FastDiv((uint32_t)(pairs + (a.dim - a.rot + 7) / 8));
    a.by_v = FastDiv((uint32_t)((a.dim + 7) / 8));
    a.by_page = FastDiv((uint32_t)(a.page_size > 0 ? a.page_size : 1));
    auto al = [](const void *p, long long s0, long long s1) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0);
    };
    const bool vec = a.dim % 8 == 0 && (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0) &&
                     al(a.q, a.q_token, a.q_head) && al(a.q_out, a.qo_token, a.qo_head) &&
                     al(a.k, a.k_token, a.k_head) && al(a.v, a.v_token, a.v_head) &&
                     al(a.ck, a.token_stride, a.head_stride) && al(a.cv, a.page_stride, 0);
    const size_t smem = (size_t)(a.rot / 2 + 1) / 2 * 16;
    auto kern = vec ? rope_kernel<T, true> : rope_kernel<T, false>;
    return launch_ex(kern, dim3(a.tokens), dim3(RP_THREADS), smem, c, 1, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool bf16, const LaunchCfg &c)
{
    return bf16 ? launch_t<__nv_bfloat16>(a, c) : launch_t<__half>(a, c);
}

}  // namespace qmoe
