// attention.cu -- new tokens over a paged K/V cache, few query rows per K/V
// head: the decode step (one token per sequence).
//
//   s_ij = scale q_i.k_j (capped by a tanh), softmax over the visible j, out_i
//   = sum_j p_ij v_j; grouped-query heads, causal and sliding-window masks.
//
// The bytes of the cache bound it: G query heads share each K/V byte, so a
// decode step does 2 G operations per byte.  One pass over K and V with the
// running maximum and sum of the softmax; scores and weights never leave
// registers.  Up to 16 query rows; 4 warps share a tile's 64 keys (each with
// its own maximum and sum, joined at the end of a unit), products on mma.sync
// m16n8k16 with the rows padded to 16 -- a 128-row tcgen05 tile would hold
// 112 empty rows or more, and a step of it costs a warpgroup's round trip
// through tensor memory.
// A producer warp brings K and V by TMA, a box of up to a page each, into a
// ring of stages that runs on into the next unit; caches without a tensor map
// (see attn_maps) are read by the four warps with 16-byte cp.async from
// wherever the page table says.  Measured: 64 ragged sequences of up to 4096
// tokens, 8 K/V heads of 128 (529 MB), 93 us, 5.7 TB/s; 2 of 100000, 4 K/V
// heads (410 MB), 78 us, 5.2 TB/s (a plain reduction of as many bytes takes
// 86); 2 of 400000, 6.3 TB/s; one of 900, 10 us, which is latency: lengths,
// page table, cache, the joining of up to 15 CTAs' parts, one after the other
// (calls one after the other).
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr int AM_THREADS = 128;
constexpr int AM_KT = 64;
// Beginning and ending a unit, in tiles: 512 units of 2 to 64 tiles take 105 us
// with 0, 98 with 1, 93 with 3, 97 with 9.
constexpr int AM_EX = 3;
constexpr int AM_ROWS = 16;      // more rows than this go to tcgen05 (launch_attn)
constexpr float AM_LAZY = 8.f;   // log2 of the growth of a maximum that sums are not rescaled for

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <class T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                     uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP, bool TMA>
struct AmLayout {
    static constexpr int M = 16;
    static constexpr int tile = AM_KT * DP * 2;
    static constexpr int S = (DP == 256 ? 196608 : 98304) / (2 * tile);   // stages of K and V: 1 CTA on an SM, or 2
    static constexpr int OP = DP + 4;   // row pitch of the joined sums
    static constexpr int st_off = 0;
    static constexpr int q_off = st_off + S * 2 * tile;
    static constexpr int ob_off = q_off + M * DP * 2;
    static constexpr int ml_off = ob_off + M * OP * 4;
    static constexpr int bar_off = ml_off + 4 * M * 8;
    static constexpr int misc_off = bar_off + 2 * S * 8;
    static constexpr int off_off = misc_off + 16;       // cp.async: where the keys lie
    static constexpr int total = off_off + (TMA ? 0 : S * AM_KT * 8) + 1024;   // + alignment slack
};

template <class T, int DP, bool TMA>
__global__ void __launch_bounds__(AM_THREADS + (TMA ? 32 : 0))
    attn_rows_kernel(const AttnArgs a, const __grid_constant__ AttnMaps maps)
{
    using L = AmLayout<DP, TMA>;
    constexpr int M = L::M, S = L::S;
    constexpr int KW = AM_KT / 4;         // keys of a tile per warp
    constexpr int CPR = DP / 8;           // 16-byte units per row
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *ob = reinterpret_cast<float *>(smem + L::ob_off);
    float2 *ml = reinterpret_cast<float2 *>(smem + L::ml_off);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::bar_off), *empty = full + S;
    int *flag = reinterpret_cast<int *>(smem + L::misc_off);   // [0] last arrival, [1] V was cleaned
    volatile int *abort_word = reinterpret_cast<volatile int *>(smem + L::misc_off + 8);
    long long *off = reinterpret_cast<long long *>(smem + L::off_off);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tg = lane & 3;

    if (tid == 0) {
        if (TMA) {
            for (int i = 0; i < S; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], 4);
            }
            mbar_init_fence();
        }
        flag[1] = 0;
        *abort_word = 0;
    }
    if (TMA && tid == AM_THREADS) {   // fetched while the lengths are
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    pdl_wait();
    pdl_trigger();
    AttnWalk<M, AM_KT, AM_EX> w;
    w.start(a, attn_span<M, AM_KT, AM_EX>(a));
    __syncthreads();

    if (TMA && warp == 4) {
        // ================================================= TMA producer
        // (all of DP: blocks of columns past dim arrive as zeros)
        const int nbox = AM_KT / a.tma, nblk = DP / 64;
        const int x = lane >> 4, bx = lane & 15;   // half a warp for K, half for V
        const void *map = x ? &maps.v : &maps.k;
        uint32_t n = 0;
        bool dead = false;
        for (; !w.done() && !dead; w.next(a)) {
            const int tb = w.tb();
            int j = (w.t0 + w.ta()) * AM_KT + bx * a.tma;
            int ahead = bx < nbox ? attn_page(a, w.sp.b, j, w.lo, w.hi) : 0;
            for (int t = w.ta(); t < tb; ++t, ++n, j += AM_KT) {
                int page = ahead;
                const int slot = j - a.by_page(j) * a.page_size;
                if (t + 1 < tb && bx < nbox)   // on its way while this tile's copies go out
                    ahead = attn_page(a, w.sp.b, j + AM_KT, w.lo, w.hi);
                if (n >= S &&
                    !__all_sync(0xffffffffu, at_wait(&empty[n % S], (n / S - 1) & 1, a, abort_word))) {
                    dead = true;
                    break;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[n % S], 2 * AM_KT * 128 * nblk);
                __syncwarp();
                if (bx < nbox) {
                    if ((unsigned)page > (unsigned)a.num_pages ||
                        (page == a.num_pages && j < w.hi && j + a.tma > w.lo)) {
                        flag_status(a.status, QMOE_DEV_BAD_PAGE);
                        page = a.num_pages;
                    }
                    const uint32_t dst = smem_u32(smem) + ((n % S) * 2 + x) * L::tile + bx * a.tma * 128;
                    for (int k = 0; k < nblk; ++k)
                        tma_load_4d(dst + k * AM_KT * 128, map, k * 64, a.heads_inner ? w.h : slot,
                                    a.heads_inner ? slot : w.h, page, &full[n % S]);
                }
                __syncwarp();
            }
        }
        // no copy may still be landing when the CTA exits
        if (lane == 0)
            for (uint32_t i = n > S ? n - S : 0; i < n; ++i)
                mbar_wait(&full[i % S], (i / S) & 1, a.status);
        return;
    }

    // ==================================================== 4 warps of products
    const AttnCap cap(a.scale, a.softcap);
    const float sc2 = a.scale * kLog2e;
    uint32_t n = 0;       // tiles so far
    // A wait gave up in this warp; after its unit, in any of the CTA's.  The tiles
    // are passed over then (the outputs are flagged as invalid), and the CTA
    // arrives as ever, so that the counters of shared units come to zero.
    bool dead = false;
    for (; !w.done(); w.next(a)) {
        const int ta = w.ta(), tb = w.tb();
        const int row0 = w.rt * M;
        const int rows = min(M, w.s.n * a.group - row0);
        // the block's query rows (rows past the end, columns past dim: zero)
        for (int i = tid; i < M * CPR; i += AM_THREADS) {
            const int r = i / CPR, c = i % CPR;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && c * 8 < a.dim) {
                const int tok = a.by_group(row0 + r), hq = w.h * a.group + (row0 + r) - tok * a.group;
                v = *reinterpret_cast<const uint4 *>(a.q + (w.s.q0 + tok) * a.q_token + hq * a.q_head + c * 8);
            }
            *reinterpret_cast<uint4 *>(smem + L::q_off + at_sw(M, r, c)) = v;
        }
        // keys that every row of the block sees
        int lo_max, hi_min;
        {
            int d;
            attn_keys(a, w.s, a.by_group(row0), d, hi_min);
            attn_keys(a, w.s, a.by_group(row0 + rows - 1), lo_max, d);
        }
        auto fill_off = [&](int t, int r) {
            const int j = (w.t0 + t) * AM_KT + r;
            long long o = -1;
            if (t < tb && j >= w.lo && j < w.hi) {
                o = attn_slot(a, w.sp.b, w.h, j);
                if (o < 0)
                    flag_status(a.status, QMOE_DEV_BAD_PAGE);
            }
            return o;
        };
        auto load = [&](int t) {
            if (t < tb) {
                const uint32_t kt = smem_u32(smem) + (t % S) * 2 * L::tile;
                const long long *o = off + (t % S) * AM_KT;
                // a thread stays in its column; the offsets of its rows are read
                // before any copy goes out, so that no copy waits for them
                constexpr int RP = AM_THREADS / CPR, N = AM_KT / RP, B = N < 8 ? N : 8;
                const int c = tid % CPR;
                const bool in = c * 8 < a.dim;
#pragma unroll
                for (int i0 = 0; i0 < N; i0 += B) {
                    long long e[B];
#pragma unroll
                    for (int i = 0; i < B; ++i)
                        e[i] = o[tid / CPR + (i0 + i) * RP];
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const int r = tid / CPR + (i0 + i) * RP;
                        const bool live = in && e[i] >= 0;
                        const long long src = live ? e[i] + c * 8 : 0;
                        cp_async16(kt + at_sw(AM_KT, r, c), a.k + src, live);
                        cp_async16(kt + L::tile + at_sw(AM_KT, r, c), a.v + src, live);
                    }
                }
            }
            cp_async_commit();
        };
        if (!TMA) {
            for (int i = tid; i < S * AM_KT; i += AM_THREADS) {
                const int t = ta + i / AM_KT;
                off[(t % S) * AM_KT + i % AM_KT] = fill_off(t, i % AM_KT);
            }
            named_bar_sync(1, AM_THREADS);
            for (int t = ta; t < ta + S - 1; ++t)
                load(t);
        }
        int lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            lo[i] = hi[i] = 0;
            if (r < rows)
                attn_keys(a, w.s, a.by_group(row0 + r), lo[i], hi[i]);
        }
        named_bar_sync(1, AM_THREADS);
        uint32_t qf[DP <= 128 ? DP / 16 : 1][4];
        const uint32_t qaddr = smem_u32(smem + L::q_off);
        if (DP <= 128) {
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
                ldsm4(qf[DP <= 128 ? kk : 0], qaddr + at_sw(M, lane & 15, kk * 2 + (lane >> 4)));
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int t = ta; t < tb; ++t, ++n) {
            long long noff = -1;
            const int st = TMA ? n % S : t % S;
            if (TMA) {
                dead = dead || !__all_sync(0xffffffffu, at_wait(&full[st], (n / S) & 1, a, abort_word));
            } else {
                cp_async_wait<S - 2>();
                named_bar_sync(1, AM_THREADS);
                load(t + S - 1);
                if (tid < AM_KT)
                    noff = fill_off(t + S, tid);
            }
            unsigned char *kt = smem + st * 2 * L::tile;
            const int j0 = (w.t0 + t) * AM_KT;
            // Keys that only some rows see, and keys outside the unit whose stale
            // slots a TMA box brought along: a weight of zero times an infinite
            // or NaN value would still reach the rows through the product.
            // Values outside the unit become zeros; infinite and NaN ones at the
            // limits are taken out and added to the rows that see them at the
            // end of the unit.
            if (j0 < lo_max || j0 + AM_KT > hi_min) {
                for (int i = tid; i < AM_KT * CPR; i += AM_THREADS) {
                    const int r = i / CPR, j = j0 + r;
                    if (j >= lo_max && j < hi_min)
                        continue;
                    uint4 *q = reinterpret_cast<uint4 *>(kt + L::tile + at_sw(AM_KT, r, i % CPR));
                    if (j < w.lo || j >= w.hi) {
                        *q = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 x = *q;
                    if (nonfinite2<T>(x.x) || nonfinite2<T>(x.y) || nonfinite2<T>(x.z) || nonfinite2<T>(x.w)) {
                        uint32_t *p = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = Num16<T>::up2(p[e]);
                            p[e] = Num16<T>::down2(isfinite(f.x) ? f.x : 0.f, isfinite(f.y) ? f.y : 0.f);
                        }
                        *q = x;
                        flag[1] = 1;
                    }
                }
                // ordered before the copy that fills this stage again
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                named_bar_sync(1, AM_THREADS);   // (a warp that gave up comes here too)
            }
            if (dead)
                continue;
            const uint32_t kb = smem_u32(kt), vb = kb + L::tile;
            float s[KW / 8][4];
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t q1[4], b[4];
                if (DP > 128)
                    ldsm4(q1, qaddr + at_sw(M, lane & 15, kk * 2 + (lane >> 4)));
                ldsm4(b, kb + at_sw(AM_KT, warp * KW + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
                mma16<T>(s[0], DP <= 128 ? qf[DP <= 128 ? kk : 0] : q1, b[0], b[1]);
                mma16<T>(s[1], DP <= 128 ? qf[DP <= 128 ? kk : 0] : q1, b[2], b[3]);
            }
            const int jw = j0 + warp * KW + 2 * tg;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = jw + 8 * i + (e & 1), r = e >> 1;
                    float x = a.softcap > 0.f ? cap.any(s[i][e]) : s[i][e] * sc2;
                    x = j >= lo[r] && j < hi[r] ? x : -INFINITY;
                    s[i][e] = x;
                    mx[r] = fmaxf(mx[r], x);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2)) - Num16<T>::kLift;
            }
            // the sums are rescaled only when a maximum has grown by more than 2^8:
            // until then the weights are at most 2^(8 + kLift), of the same base
            const bool grow = mx[0] > m[0] + AM_LAZY || mx[1] > m[1] + AM_LAZY ||
                              (m[0] == -INFINITY && mx[0] > m[0]) || (m[1] == -INFINITY && mx[1] > m[1]);
            if (__any_sync(0xffffffffu, grow)) {
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float mn = fmaxf(m[r], mx[r]);
                    f[r] = m[r] == -INFINITY ? 0.f : exp2_approx(m[r] - mn);
                    m[r] = mn;
                    l[r] *= f[r];
                }
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    o[i][0] *= f[0];
                    o[i][1] *= f[0];
                    o[i][2] *= f[1];
                    o[i][3] *= f[1];
                }
            }
            const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < KW / 8; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i][e] = exp2_approx(s[i][e] - base[e >> 1]);
                    l[e >> 1] += s[i][e];
                }
                // the weights enter the product in the cache's type (at most half
                // a step each); their sum stays fp32 and unrounded
                p[2 * i] = Num16<T>::down2(s[i][0], s[i][1]);
                p[2 * i + 1] = Num16<T>::down2(s[i][2], s[i][3]);
            }
#pragma unroll
            for (int d2 = 0; d2 < DP / 16; ++d2) {
                uint32_t b[4];
                ldsm4t(b, vb + at_sw(AM_KT, warp * KW + (lane & 15), d2 * 2 + (lane >> 4)));
                mma16<T>(o[2 * d2], p, b[0], b[1]);
                mma16<T>(o[2 * d2 + 1], p, b[2], b[3]);
            }
            if (TMA) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&empty[st]);
            } else if (tid < AM_KT) {
                off[st * AM_KT + tid] = noff;   // tile t + S
            }
        }
        // ---- join the warps: in turn into one block of sums
        if (!TMA)
            cp_async_wait<0>();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (tg == 0)
                ml[warp * M + g + 8 * r] = make_float2(m[r], l[r]);
        }
        dead = bar_any(1, AM_THREADS, dead);
        for (int k = 0; k < 4; ++k) {
            if (warp == k) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = g + 8 * r;
                    if (row >= rows)
                        continue;
                    float mt = ml[row].x;
#pragma unroll
                    for (int x = 1; x < 4; ++x)
                        mt = fmaxf(mt, ml[x * M + row].x);
                    const float f = exp2_approx(m[r] - (mt == -INFINITY ? 0.f : mt));
                    float2 *dst = reinterpret_cast<float2 *>(ob + row * L::OP + 2 * tg);
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        float2 v = k == 0 ? make_float2(0.f, 0.f) : dst[4 * i];
                        v.x = fmaf(f, o[i][2 * r], v.x);
                        v.y = fmaf(f, o[i][2 * r + 1], v.y);
                        dst[4 * i] = v;
                    }
                }
            }
            named_bar_sync(1, AM_THREADS);
        }
        const bool whole = ta == 0 && tb == w.nt;
        float *part = attn_part<M, DP>(a, blockIdx.x, ta == 0);
        const int d4 = a.dim / 4;
        const bool cleaned = flag[1] != 0;
        for (int i = tid; i < rows * d4; i += AM_THREADS) {
            const int r = i / d4, d = (i - r * d4) * 4;
            float mt = ml[r].x, lt = 0.f;
#pragma unroll
            for (int k = 1; k < 4; ++k)
                mt = fmaxf(mt, ml[k * M + r].x);
            const float b0 = mt == -INFINITY ? 0.f : mt;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                lt = fmaf(exp2_approx(ml[k * M + r].x - b0), ml[k * M + r].y, lt);
            float4 v = *reinterpret_cast<const float4 *>(ob + r * L::OP + d);
            const int tok = a.by_group(row0 + r), hq = w.h * a.group + (row0 + r) - tok * a.group;
            if (cleaned) {   // the values taken out above, for the rows that see them
                int klo, khi;
                attn_keys(a, w.s, tok, klo, khi);
                klo = max(klo, (w.t0 + ta) * AM_KT);
                khi = min(khi, (w.t0 + tb) * AM_KT);
                for (int j = klo; j < khi; ++j) {
                    if (j >= lo_max && j < hi_min) {
                        j = hi_min - 1;
                        continue;
                    }
                    const long long e = attn_slot(a, w.sp.b, w.h, j);
                    if (e < 0)
                        continue;
                    const float x[4] = {Num16<T>::up(a.v[e + d]), Num16<T>::up(a.v[e + d + 1]),
                                        Num16<T>::up(a.v[e + d + 2]), Num16<T>::up(a.v[e + d + 3])};
                    v.x += isfinite(x[0]) ? 0.f : x[0];
                    v.y += isfinite(x[1]) ? 0.f : x[1];
                    v.z += isfinite(x[2]) ? 0.f : x[2];
                    v.w += isfinite(x[3]) ? 0.f : x[3];
                }
            }
            if (whole) {
                const float inv = lt == 0.f ? 0.f : 1.f / lt;
                uint2 w2;
                w2.x = Num16<T>::down2(v.x * inv, v.y * inv);
                w2.y = Num16<T>::down2(v.z * inv, v.w * inv);
                *reinterpret_cast<uint2 *>(a.out + (w.s.q0 + tok) * a.o_token + hq * a.o_head + d) = w2;
                if (a.lse && d == 0)
                    a.lse[(size_t)(w.s.q0 + tok) * a.heads + hq] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(part + (size_t)r * DP + d) = v;
                if (d == 0) {
                    part[M * DP + r] = mt;
                    part[M * DP + M + r] = lt;
                }
            }
        }
        if (!whole) {
            const int c0 = w.c0(), c1 = w.c1();
            if (attn_arrive<AM_THREADS>(a, c0, c1, flag))
                for (int r = warp; r < rows; r += AM_THREADS / 32)
                    attn_join_row<T, M, DP, DP == 256 ? 8 : 16>(a, c0, c1, r, w.s.q0, row0 + r, w.h);
        }
        named_bar_sync(1, AM_THREADS);   // the blocks and flags are free for the next unit
        if (cleaned && tid == 0)
            flag[1] = 0;
    }
}

template <class T, int DP, bool TMA>
cudaError_t launch_rows(const AttnArgs &a, const AttnMaps &maps, const LaunchCfg &c)
{
    using L = AmLayout<DP, TMA>;
    auto kern = attn_rows_kernel<T, DP, TMA>;
    cudaError_t e = set_smem(kern, L::total);
    if (e != cudaSuccess)
        return e;
    // (and up to 168 registers a thread: 224 once took 131 us where 165 take 93; a
    // bound of two blocks in the declaration spills 24 bytes and takes 94)
    constexpr int per_sm = DP == 256 ? 1 : 2;
    static_assert(per_sm * (L::total + 1024) <= 228 * 1024 && per_sm <= 3, "shared memory");
    return launch_ex(kern, dim3(c.num_sms * per_sm), dim3(AM_THREADS + (TMA ? 32 : 0)), L::total, c, 1, a, maps);
}

template <class T>
cudaError_t launch_dim(const AttnArgs &args, bool bf16, const LaunchCfg &c)
{
    AttnArgs a = args;
    AttnMaps maps = {};
    if (attn_maps(a, bf16, AM_KT, &maps, &a.tma, &a.heads_inner))
        return a.dim <= 64    ? launch_rows<T, 64, true>(a, maps, c)
               : a.dim <= 128 ? launch_rows<T, 128, true>(a, maps, c)
                              : launch_rows<T, 256, true>(a, maps, c);
    a.tma = 0;
    return a.dim <= 64    ? launch_rows<T, 64, false>(a, maps, c)
           : a.dim <= 128 ? launch_rows<T, 128, false>(a, maps, c)
                          : launch_rows<T, 256, false>(a, maps, c);
}

}  // namespace

typedef CUresult (*AttnEncode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static AttnEncode attn_encode()
{
    static const AttnEncode fn = []() -> AttnEncode {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<AttnEncode>(p);
        (void)cudaGetLastError();
        return nullptr;
    }();
    return fn;
}

bool attn_q_map(const AttnArgs &a, bool bf16, CUtensorMap *m)
{
    const AttnEncode fn = attn_encode();
    if (!fn || a.group > 128 || 128 % a.group || a.dim < 64)
        return false;
    const cuuint64_t head = a.heads > 1 ? 2 * a.q_head : 2 * a.dim;
    const cuuint64_t tok = a.tokens > 1 ? 2 * a.q_token : head * a.heads;
    if (head < 2 * (cuuint64_t)a.dim || head % 16 || tok < head || tok % head || tok >= (cuuint64_t)1 << 40)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.heads, (cuuint64_t)a.tokens};
    const cuuint64_t strides[2] = {head, tok};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(128 / a.group)};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<uint16_t *>(a.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_maps(const AttnArgs &a, bool bf16, int kt, AttnMaps *m, int *rows, int *heads_inner)
{
    const AttnEncode fn = attn_encode();
    int r = kt;
    while (r > a.page_size || a.page_size % r)
        r /= 2;   // kt is a power of two
    if (!fn || r < 8 || a.dim < 64)
        return false;
    // strides in bytes; that of a dimension of one element says nothing
    cuuint64_t tok = a.page_size > 1 ? 2 * a.token_stride : 2 * a.dim;
    cuuint64_t head = a.kv_heads > 1 ? 2 * a.head_stride : 2 * a.dim;
    const bool hi = a.kv_heads > 1 ? head < tok : true;   // heads inside slots
    if (a.kv_heads == 1)
        head = 2 * (cuuint64_t)a.dim;
    const cuuint64_t s0 = hi ? head : tok, s1 = hi ? tok : head;
    const cuuint64_t last = s1 * (hi ? a.page_size : a.kv_heads);
    const cuuint64_t s2 = a.num_pages > 1 ? 2 * (cuuint64_t)a.page_stride : last;
    const cuuint64_t most = (cuuint64_t)1 << 40;
    if (s0 < 2 * (cuuint64_t)a.dim || s0 % 16 || s1 % s0 || s1 < s0 || s2 % s1 || s2 < s1 || s2 >= most)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.dim, (cuuint64_t)(hi ? a.kv_heads : a.page_size),
                                (cuuint64_t)(hi ? a.page_size : a.kv_heads), (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {s0, s1, s2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(hi ? 1 : r), (cuuint32_t)(hi ? r : 1), 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    *rows = r;
    *heads_inner = hi;
    for (int i = 0; i < 2; ++i)
        if (fn(i ? &m->v : &m->k, type, 4, const_cast<uint16_t *>(i ? a.v : a.k), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    return true;
}

size_t attn_workspace_bytes(int dim, long long max_rows)
{
    const int dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    const size_t row = (size_t)2 * (dp + 2) * 4;   // two slots
    if (max_rows > AM_ROWS)
        return kAttnCounterBytes + kAttnMaxSms * (256 * row + 32);   // and what the units are
    return kAttnCounterBytes + (size_t)kAttnMaxSms * 3 * 16 * row;
}

cudaError_t launch_attn(const AttnArgs &a, bool bf16, long long max_rows, const LaunchCfg &c)
{
    if (c.num_sms > kAttnMaxSms)
        return cudaErrorInvalidValue;
    // Measured, this kernel and the tcgen05 one: 4 rows, 64 sequences of up to
    // 4096 tokens, 98 and 125 us, one of 900, 12 and 17; 8 rows of heads of 64,
    // 63 and 100; 16 rows 64 and 67; 32 rows (two blocks of 16 read everything
    // twice) 59 and 45; 48 rows 75 and 37.
    if (max_rows > AM_ROWS)
        // two row tiles per unit once there are units for every SM: 4 chunks of
        // 2048 tokens take 344 us with two, 423 with one; a chunk of 512, 62 both
        // ways; of 128, 37 with two, 31 with one
        return launch_attn_tc(a, bf16, (long long)a.tokens * a.group / 256 * a.kv_heads >= c.num_sms ? 2 : 1, c);
    return bf16 ? launch_dim<__nv_bfloat16>(a, true, c) : launch_dim<__half>(a, false, c);
}

}  // namespace qmoe
