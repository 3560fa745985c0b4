// attn.cuh -- what the attention kernels share: the division of the work over
// the CTAs, the rows' visible keys, and the joining of a unit that several
// CTAs worked on.
//
// A unit is (sequence, block of M query rows, K/V head).  The rows of a unit
// are (token, query head of the K/V head's group) pairs, token-major, so that
// one K/V tile in shared memory serves every query head that reads it.  The
// unit's keys are walked in tiles of KT.  All tiles of all units form one
// line, cut into equal intervals, one per CTA: a batch of ragged
// lengths keeps every SM busy to the end, one long context spreads over the
// whole GPU, and nothing about the lengths is needed on the host (a captured
// graph replays with new ones).  Each unit is EX places longer on the line
// than its tiles: what it costs to begin and end one, in tiles.  A unit that crosses CTA borders is finished
// by its last CTA to arrive, which adds the fp32 partial results in tile
// order; nobody waits, and results do not depend on the order of arrival.  A CTA
// that gives up a wait arrives all the same, so that the counters end at zero.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace qmoe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <class T>
struct Num16;
template <>
struct Num16<__half> {
    static __device__ __forceinline__ float up(uint16_t v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ uint16_t down(float v) { return __half_as_ushort(__float2half_rn(v)); }
    static __device__ __forceinline__ uint32_t down2(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 up2(uint32_t v)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static constexpr uint32_t kExp = 0x7C007C00u;   // exponent bits of a pair
    // log2 of a row's largest weight as its maximum is set: with the 2^8 that the
    // maximum may lag behind, at most 2^15, and 2^-32 of it is the smallest step
    static constexpr float kLift = 7.f;
};
template <>
struct Num16<__nv_bfloat16> {
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t down(float v)
    {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    static __device__ __forceinline__ uint32_t down2(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 up2(uint32_t v)
    {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static constexpr uint32_t kExp = 0x7F807F80u;
    static constexpr float kLift = 0.f;   // its exponents are fp32's
};

// whether one of the two 16-bit numbers of a word is an infinity or a NaN
template <class T>
__device__ __forceinline__ bool nonfinite2(uint32_t w)
{
    const uint32_t e = w & Num16<T>::kExp;
    return (e & 0xFFFFu) == (Num16<T>::kExp & 0xFFFFu) || (e >> 16) == (Num16<T>::kExp >> 16);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2(e) cap tanh(scale x / cap) of a product x, t = scale x / cap.
//   high: tanh(t) = 1 - 2 / (1 + e^2t), one exponential and one reciprocal (the
//     hardware's tanh is good to 2^-11 only, which would show in the weights).
//     Off by up to 2^-22 of the cap: near t = 0 the 1 cancels.
//   low, |t| < 1/2: t P(t^2), P by Chebyshev interpolation of tanh(sqrt w) /
//     sqrt w in 5 points of [0, 1/4] (off by 1.4e-8; 1.1e-7 with its roundings):
//     a cap that is large beside the scores leaves them as they are.
// attn_rows_kernel takes both for every score and chooses (64 sequences of up to
// 4096 tokens: 110.4 us instead of 108.8 with high alone; a branch around them
// cost calls without a cap 131 instead of 93).  attn_tc_kernel, whose
// exponentials count, takes high alone up to a cap of 64 -- 2^-16 of a score at
// most, far below a 16-bit weight's half step -- and above it each score by its
// t, a warp none of whose scores is high the polynomial alone (at_cap; 8 drafts of
// 24 with heads of 256: 38.6 us, 35.9 by high alone).
struct AttnCap {
    float k, to_t, to_e, cap;   // scale log2 e, scale / cap, 2 log2 e scale / cap, cap log2 e
    bool wide;

    // (a tiny cap makes t infinite, but for a score of 0, whose t stays 0)
    __device__ __forceinline__ AttnCap(float scale, float softcap)
        : k(scale * kLog2e), to_t(fminf(scale / softcap, 1e37f)), to_e(to_t * 2.f * kLog2e), cap(softcap * kLog2e),
          wide(softcap > 64.f)
    {
    }
    __device__ __forceinline__ float high(float x) const
    {
        return cap * (1.f - __fdividef(2.f, 1.f + exp2_approx(x * to_e)));
    }
    __device__ __forceinline__ float low(float x) const
    {
        const float t = x * to_t, w = t * t;
        float p = fmaf(w, 0.01713134f, -0.05298424f);
        p = fmaf(p, w, 0.13324751f);
        p = fmaf(p, w, -0.33333068f);
        p = fmaf(p, w, 1.f);
        return x * k * p;
    }
    __device__ __forceinline__ float any(float x) const
    {
        const float h = high(x);
        return fabsf(x * to_t) < 0.5f ? low(x) : h;
    }
    // whether a thread of the warp has a score that is not for low(); most: the
    // thread's largest |x| (NaN stays NaN in both)
    __device__ __forceinline__ bool above(float most) const
    {
        return __any_sync(0xffffffffu, !(most * to_t < 0.5f));
    }
};

// ------------------------------------------------------------------- units --
struct AttnSeq {
    int q0, n, len;   // first query row, new tokens, cached tokens with them
};

// Lengths as the device finds them, kept inside the buffers: a length beyond
// the page table is cut there and flagged.
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int b)
{
    AttnSeq s;
    s.q0 = min(max(a.q_start[b], 0), a.tokens);
    s.n = min(max(a.q_start[b + 1], s.q0), a.tokens) - s.q0;
    const long long room = (long long)a.max_pages * a.page_size;
    const int len = max(a.kv_len[b], 0);
    s.len = (long long)len > room ? (int)room : len;
    return s;
}

// keys of one token: [lo, hi)
__device__ __forceinline__ void attn_keys(const AttnArgs &a, const AttnSeq &s, int token, int &lo, int &hi)
{
    const int p = s.len - s.n + token;
    hi = a.causal ? max(p + 1, 0) : s.len;
    lo = a.window > 0 ? max(p - a.window + 1, 0) : 0;
}

// first tile and number of tiles of row block rt (at least one, so that rows
// that see nothing are written too), and the keys any of its rows sees
template <int M, int KT>
__device__ __forceinline__ void attn_tiles(const AttnArgs &a, const AttnSeq &s, int rt, int &t0, int &nt,
                                           int &lo, int &hi)
{
    const int rows = s.n * a.group;
    int d;
    attn_keys(a, s, a.by_group(rt * M), lo, d);
    attn_keys(a, s, a.by_group(min(rt * M + M, rows) - 1), d, hi);
    if (hi <= lo) {   // nothing visible
        t0 = lo = hi = 0;
        nt = 1;
        return;
    }
    t0 = lo / KT;
    nt = (hi + KT - 1) / KT - t0;
}

template <int M>
__device__ __forceinline__ int attn_blocks(const AttnArgs &a, const AttnSeq &s)
{
    return (int)(((long long)s.n * a.group + M - 1) / M);
}

template <int M, int KT, int EX>
__device__ __forceinline__ long long attn_seq_tiles(const AttnArgs &a, const AttnSeq &s)
{
    long long w = 0;
    const int nb = attn_blocks<M>(a, s);
    for (int rt = 0; rt < nb; ++rt) {
        int t0, nt, lo, hi;
        attn_tiles<M, KT>(a, s, rt, t0, nt, lo, hi);
        w += EX + nt;
    }
    return w * a.kv_heads;
}

// This CTA's interval [x, end) of the line of tiles, and the sequence that
// holds tile x with the line's index of its first tile.
struct AttnSpan {
    long long total, x, end, first;
    int b;
    int ctas;   // CTAs with work: each has at least one tile
};

// total * c / n, in 32 bits where that holds it (a 64-bit division is a
// hundred instructions); at most 3 x 160 CTAs.
__device__ __forceinline__ long long attn_place(long long total, int c, int n)
{
    return total < (1ll << 23) ? (long long)((uint32_t)total * (uint32_t)c / (uint32_t)n) : total * c / n;
}

// Every warp works it out by itself, a lane a sequence: no block barrier, and
// the lengths are read once (from L1 by the later warps).
template <int M, int KT, int EX>
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs &a)
{
    const int lane = threadIdx.x & 31;
    AttnSpan sp;
    long long mine = 0, sum = 0;
    for (int b = lane; b < a.batch; b += 32) {
        if (blockIdx.x == 0 && threadIdx.x < 32 && a.kv_len[b] > (long long)a.max_pages * a.page_size)
            flag_status(a.status, QMOE_DEV_BAD_PAGE);
        mine = attn_seq_tiles<M, KT, EX>(a, attn_seq(a, b));
        sum += mine;
    }
    const bool small = !__any_sync(0xffffffffu, sum >= (1 << 25));
    if (small) {
        sum = __reduce_add_sync(0xffffffffu, (unsigned)sum);
    } else {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    sp.total = sum;
    sp.ctas = (int)min(sum, (long long)gridDim.x);
    const int c = min((int)blockIdx.x, sp.ctas);
    sp.x = sp.ctas ? attn_place(sum, c, sp.ctas) : 0;
    sp.end = c < sp.ctas ? attn_place(sum, c + 1, sp.ctas) : sp.x;
    sp.first = 0;
    sp.b = 0;
    if (sp.x >= sp.end || a.batch == 1)
        return sp;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        if (a.batch > 32)
            mine = b0 + lane < a.batch ? attn_seq_tiles<M, KT, EX>(a, attn_seq(a, b0 + lane)) : 0;
        long long incl;
        if (small) {
            int v = (int)mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o)
                    v += u;
            }
            incl = v;
        } else {
            incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += u;
            }
        }
        const unsigned holds = __ballot_sync(0xffffffffu, sp.first + incl > sp.x);
        if (holds) {
            const int l = __ffs(holds) - 1;
            sp.b = b0 + l;
            sp.first += __shfl_sync(0xffffffffu, incl - mine, l);
            break;
        }
        sp.first += __shfl_sync(0xffffffffu, incl, 31);
    }
    return sp;
}

// the CTA whose interval holds place x of the line
__device__ __forceinline__ int attn_cta(const AttnSpan &sp, long long x)
{
    if (sp.total < (1ll << 23))
        return (int)(((uint32_t)(x + 1) * (uint32_t)sp.ctas - 1) / (uint32_t)sp.total);
    return (int)(((x + 1) * sp.ctas - 1) / sp.total);
}

// A walk over the units of a CTA's interval.
template <int M, int KT, int EX>
struct AttnWalk {
    AttnSpan sp;
    AttnSeq s;
    int rt, nb, h;           // row block (of nb), K/V head
    int t0, nt, lo, hi;      // tiles and keys of the row block
    long long u0;            // the unit's first place on the line; its tiles begin EX places on

    __device__ __forceinline__ void start(const AttnArgs &a, const AttnSpan &span)
    {
        sp = span;
        if (sp.x >= sp.end)
            return;
        s = attn_seq(a, sp.b);
        nb = attn_blocks<M>(a, s);
        u0 = sp.first;
        for (rt = 0;; ++rt) {
            attn_tiles<M, KT>(a, s, rt, t0, nt, lo, hi);
            if (sp.x < u0 + (long long)(EX + nt) * a.kv_heads || rt + 1 >= nb)
                break;
            u0 += (long long)(EX + nt) * a.kv_heads;
        }
        const long long d = sp.x - u0;
        h = d < (1ll << 31) ? (int)((uint32_t)d / (uint32_t)(EX + nt)) : (int)(d / (EX + nt));
        u0 += (long long)h * (EX + nt);
    }
    __device__ __forceinline__ bool done() const { return sp.x >= sp.end || sp.end <= u0 + EX; }
    // the unit's tiles that are this CTA's: [ta, tb) of 0..nt, at least one
    __device__ __forceinline__ int ta() const { return (int)max(sp.x - u0 - EX, 0ll); }
    __device__ __forceinline__ int tb() const { return (int)min(sp.end - u0 - EX, (long long)nt); }
    // first and last CTA with tiles of the unit
    __device__ __forceinline__ int c0() const { return attn_cta(sp, u0 + EX); }
    __device__ __forceinline__ int c1() const { return attn_cta(sp, u0 + EX + nt - 1); }
    __device__ __forceinline__ void next(const AttnArgs &a)
    {
        u0 += EX + nt;
        sp.x = u0;
        if (sp.x >= sp.end)
            return;
        if (++h < a.kv_heads)
            return;
        h = 0;
        ++rt;
        while (rt >= nb) {   // sp.x < sp.end <= total: a later sequence has tiles
            s = attn_seq(a, ++sp.b);
            nb = attn_blocks<M>(a, s);
            rt = 0;
        }
        attn_tiles<M, KT>(a, s, rt, t0, nt, lo, hi);
    }
};

// Where the first element of cached token j of sequence b (K/V head h) lies,
// or -1 for a page id outside the cache (flagged by the caller).
__device__ __forceinline__ long long attn_slot(const AttnArgs &a, int b, int h, int j)
{
    const int pg = a.by_page(j);
    const int id = __ldg(a.table + (size_t)b * a.max_pages + pg);
    if ((unsigned)id >= (unsigned)a.num_pages)
        return -1;
    return id * a.page_stride + (long long)(j - pg * a.page_size) * a.token_stride + h * a.head_stride;
}

// one look at a barrier, without being parked
__device__ __forceinline__ bool mbar_try_wait_now(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait of at most a.wait_ns (flags QMOE_DEV_TIMEOUT; 0: one look) that gives up
// at once after another thread of the CTA did.  Copies and products in flight are
// awaited by mbar_wait, whose limit is not the caller's.
__device__ __forceinline__ bool at_wait(uint64_t *bar, uint32_t parity, const AttnArgs &a, volatile int *abort_word)
{
    if (mbar_try_wait_now(bar, parity))
        return true;
    const unsigned long long t0 = global_timer_ns();
    while (!*abort_word) {
        if (global_timer_ns() - t0 >= a.wait_ns) {
            flag_status(a.status, QMOE_DEV_TIMEOUT);
            *abort_word = 1;
        } else if (mbar_try_wait(bar, parity)) {
            return true;
        }
    }
    return false;
}

// byte offset of 16-byte unit c of row r in a tile of `rows` rows, in 128-byte
// swizzled blocks of 64 columns
__device__ __forceinline__ uint32_t at_sw(int rows, int r, int c)
{
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ----------------------------------------------------------------- TMA --
// Tensor maps of the cache: boxes of 64 columns x a.tma slots of one page and
// head, 128-byte swizzled.
struct AttnMaps {
    CUtensorMap k, v, q;
};

// False where the cache's shape has no such map: pages must divide into
// boxes of a multiple of 8 slots (the swizzle's period) that divide a tile of
// kt keys, and the strides must nest.
bool attn_maps(const AttnArgs &a, bool bf16, int kt, AttnMaps *m, int *rows, int *heads_inner);
// q in boxes of 64 columns x the group's heads x 128 / group tokens; false
// where a group does not divide 128 rows.
bool attn_q_map(const AttnArgs &a, bool bf16, CUtensorMap *m);

__device__ __forceinline__ void tma_load_3d(void *dst, const void *map, int c0, int c1, int c2, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// The page that holds the box of keys [j, j + a.tma) of sequence b, as the
// table says, or a.num_pages (beyond the cache: the copy writes zeros) where
// the unit reads none of them.
__device__ __forceinline__ int attn_page(const AttnArgs &a, int b, int j, int lo, int hi)
{
    if (j >= hi || j + a.tma <= lo)
        return a.num_pages;
    return __ldg(a.table + (size_t)b * a.max_pages + a.by_page(j));
}

// ----------------------------------------------------------------- joining --
// Partial results of CTA c: two slots of M rows x DP fp32 sums, then M maxima
// (log2 units) and M weight sums.  Slot 0 holds the part of a unit that began
// in an earlier CTA, slot 1 of one that goes on in a later one.
template <int M, int DP>
__device__ __forceinline__ float *attn_part(const AttnArgs &a, int cta, int slot)
{
    return a.part + (size_t)(2 * cta + slot) * M * (DP + 2);
}

// Announces this CTA's part of a unit that CTAs c0..c1 share; true for the
// last one, which then reads all parts.  The first NT threads of the CTA, on
// named barrier 1.
template <int NT>
__device__ __forceinline__ bool attn_arrive(const AttnArgs &a, int c0, int c1, int *sm)
{
    named_bar_sync(1, NT);
    if (threadIdx.x == 0) {
        __threadfence();   // everybody's parts: written before the barrier
        const int got = atomicAdd(a.ctr + c0, 1);
        *sm = got == c1 - c0;
        if (got == c1 - c0)
            a.ctr[c0] = 0;
        __threadfence();
    }
    named_bar_sync(1, NT);
    return *sm != 0;
}

// One row's output from the parts c0..c1 of its unit, by one warp: a lane
// reads the maximum and sum of one part each, the parts' weights go round by
// shuffles, and DP / 32 columns a lane are added in the parts' order.  r: row
// of the unit; row: of the sequence, whose first token is row q0.
template <class T, int M, int DP, int B>
__device__ __forceinline__ void attn_join_row(const AttnArgs &a, int c0, int c1, int r, int q0, int row, int h)
{
    const int lane = threadIdx.x & 31, np = c1 - c0 + 1;
    constexpr int V = DP / 32;
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        o[i] = 0.f;
    for (int k0 = 0; k0 < np; k0 += 32) {
        const int k = k0 + lane;
        const float *p = attn_part<M, DP>(a, c0 + (k < np ? k : 0), k == 0 || k >= np);
        const float mk = k < np ? __ldcg(p + M * DP + r) : -INFINITY;
        const float lk = k < np ? __ldcg(p + M * DP + M + r) : 0.f;
        const int n = min(32, np - k0);
        float w = 0.f;
        // B parts' columns are on their way at once, the first B beside the maxima
        for (int x0 = 0; x0 < n; x0 += B) {
            float v[B][V];
#pragma unroll
            for (int x = 0; x < B; ++x) {
                const int kk = k0 + x0 + x;
                const float *q = attn_part<M, DP>(a, c0 + kk, kk == 0) + (size_t)r * DP + lane * V;
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    float2 u = make_float2(0.f, 0.f);
                    if (x0 + x < n)
                        u = __ldcg(reinterpret_cast<const float2 *>(q + i));
                    v[x][i] = u.x;
                    v[x][i + 1] = u.y;
                }
            }
            if (x0 == 0) {
                float top = mk;
#pragma unroll
                for (int s = 16; s; s >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                top = fmaxf(top, m);
                const float base = top == -INFINITY ? 0.f : top;
                const float f = exp2_approx(m - base);
                w = exp2_approx(mk - base);
                float sum = w * lk;
#pragma unroll
                for (int s = 16; s; s >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, s);
                l = l * f + sum;
                m = top;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o[i] *= f;
            }
#pragma unroll
            for (int x = 0; x < B; ++x) {
                const float wx = __shfl_sync(0xffffffffu, w, x0 + x);
                if (x0 + x < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o[i] = fmaf(wx, v[x][i], o[i]);
                }
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = a.by_group(row), hq = h * a.group + row - tok * a.group;
    uint16_t *dst = a.out + (q0 + tok) * a.o_token + hq * a.o_head + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        if (lane * V + i < a.dim)
            *reinterpret_cast<uint32_t *>(dst + i) = Num16<T>::down2(o[i] * inv, o[i + 1] * inv);
    if (a.lse && lane == 0)
        a.lse[(size_t)(q0 + tok) * a.heads + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace qmoe
