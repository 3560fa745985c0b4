// attention.cu -- new tokens over a paged K/V cache, few query rows per K/V
// head: the decode step (one token per sequence) and the verification of a
// handful of draft tokens.
//
//   s_ij = scale q_i.k_j (capped by a tanh), softmax over the visible j, out_i
//   = sum_j p_ij v_j; grouped-query heads, causal and sliding-window masks.
//
// The bytes of the cache bound it: G query heads share each K/V byte, so a
// decode step does 2 G operations per byte.  One pass over K and V with the
// running maximum and sum of the softmax; scores and weights never leave
// registers.  4 warps: WR x 16 query rows, and WK warps share a tile's keys
// (each with its own maximum and sum; joined at the end of a unit), products
// on mma.sync m16n8k16 with the rows padded to 16 -- the tensor cores idle
// most of the time here, and a 128-row tcgen05 tile would hold 120 empty rows.
// Tiles of 64 keys arrive by 16-byte cp.async from wherever the page table
// says (any page size: each key's address is looked up one tile ahead) into a
// ring of 3 stages, 16-byte units XORed with the row for conflict-free
// ldmatrix.
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr int AM_THREADS = 128;
constexpr int AM_KT = 64;
constexpr int AM_EX = 0;

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

// byte offset of 16-byte unit c of row r in a tile of DP-wide rows
template <int DP>
__device__ __forceinline__ uint32_t sw(int r, int c)
{
    return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

template <int DP, int WR>
struct AmLayout {
    static constexpr int M = 16 * WR, WK = 4 / WR;
    static constexpr int S = DP == 256 && WR == 4 ? 2 : 3;   // stages that fit beside the query rows
    static constexpr int tile = AM_KT * DP * 2;
    static constexpr int OP = DP + 4;   // row pitch of the joined sums
    static constexpr int st_off = M * DP * 2;
    static constexpr int off_off = st_off + S * 2 * tile;
    static constexpr int ml_off = off_off + S * AM_KT * 8;
    static constexpr int misc_off = ml_off + 2 * WK * M * 4;
    static constexpr int total = misc_off + 16;
    static_assert(WK * M * OP * 4 <= S * 2 * tile, "joined sums fit the ring");
};

template <class T, int DP, int WR>
__global__ void __launch_bounds__(AM_THREADS) attn_rows_kernel(const AttnArgs a)
{
    using L = AmLayout<DP, WR>;
    constexpr int M = L::M, WK = L::WK, S = L::S;
    constexpr int KW = AM_KT / WK;        // keys of a tile per warp
    constexpr int CPR = DP / 8;           // 16-byte units per row
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char *stage = smem + L::st_off;
    long long *off = reinterpret_cast<long long *>(smem + L::off_off);
    float *ml = reinterpret_cast<float *>(smem + L::ml_off);
    int *flag = reinterpret_cast<int *>(smem + L::misc_off);            // [0] last arrival, [1] V not finite
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp / WK, wk = warp % WK;
    const int g = lane >> 2, tg = lane & 3;

    AttnWalk<M, AM_KT, AM_EX> w;
    w.start(a, attn_span<M, AM_KT, AM_EX>(a));
    const float sc2 = a.softcap > 0.f ? a.scale * 2.f * kLog2e / a.softcap : a.scale * kLog2e;
    const float cap = a.softcap * kLog2e;

    for (; !w.done(); w.next(a)) {
        const int ta = w.ta(), tb = w.tb();
        const int row0 = w.rt * M;
        const int rows = min(M, w.s.n * a.group - row0);
        // keys that some rows of the block see and others do not
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
                unsigned char *kt = stage + (t % S) * 2 * L::tile;
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
                        cp_async16(smem_u32(kt) + sw<DP>(r, c), a.k + src, live);
                        cp_async16(smem_u32(kt) + L::tile + sw<DP>(r, c), a.v + src, live);
                    }
                }
            }
            cp_async_commit();
        };
        for (int i = tid; i < S * AM_KT; i += AM_THREADS) {
            const int t = ta + i / AM_KT;
            off[(t % S) * AM_KT + i % AM_KT] = fill_off(t, i % AM_KT);
        }
        if (tid == 0)
            flag[1] = 0;
        __syncthreads();
        for (int t = ta; t < ta + S - 1; ++t)
            load(t);
        // the block's query rows (rows past the end, columns past dim: zero)
        for (int i = tid; i < M * CPR; i += AM_THREADS) {
            const int r = i / CPR, c = i % CPR;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && c * 8 < a.dim) {
                const int tok = a.by_group(row0 + r), hq = w.h * a.group + (row0 + r) - tok * a.group;
                v = *reinterpret_cast<const uint4 *>(a.q + (w.s.q0 + tok) * a.q_token + hq * a.q_head + c * 8);
            }
            *reinterpret_cast<uint4 *>(smem + sw<DP>(r, c)) = v;
        }
        int lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = wr * 16 + g + 8 * i;
            lo[i] = hi[i] = 0;
            if (r < rows)
                attn_keys(a, w.s, a.by_group(row0 + r), lo[i], hi[i]);
        }
        __syncthreads();
        uint32_t qf[DP <= 128 ? DP / 16 : 1][4];
        const uint32_t qaddr = smem_u32(smem);
        if (DP <= 128) {
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
                ldsm4(qf[DP <= 128 ? kk : 0], qaddr + sw<DP>(wr * 16 + (lane & 15), kk * 2 + (lane >> 4)));
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int t = ta; t < tb; ++t) {
            cp_async_wait<S - 2>();
            __syncthreads();
            load(t + S - 1);
            long long noff = -1;
            if (tid < AM_KT)
                noff = fill_off(t + S, tid);
            unsigned char *kt = stage + (t % S) * 2 * L::tile;
            const int j0 = (w.t0 + t) * AM_KT;
            // Keys that only some rows see: a weight of zero times an infinite
            // or NaN value would reach the other rows through the product, so
            // such values are taken out here and added to their own rows at
            // the end of the unit.
            if ((j0 < lo_max && j0 + AM_KT > w.lo) || (j0 + AM_KT > hi_min && j0 < w.hi)) {
                for (int i = tid; i < AM_KT * CPR; i += AM_THREADS) {
                    const int r = i / CPR, j = j0 + r;
                    if (j >= lo_max && j < hi_min)
                        continue;
                    uint32_t *p = reinterpret_cast<uint32_t *>(kt + L::tile + sw<DP>(r, i % CPR));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nonfinite2<T>(p[e])) {
                            const float2 f = Num16<T>::up2(p[e]);
                            p[e] = Num16<T>::down2(isfinite(f.x) ? f.x : 0.f, isfinite(f.y) ? f.y : 0.f);
                            flag[1] = 1;
                        }
                }
                __syncthreads();
            }
            const uint32_t kb = smem_u32(kt), vb = kb + L::tile;
            float s[KW / 8][4];
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t q1[4];
                if (DP > 128)
                    ldsm4(q1, qaddr + sw<DP>(wr * 16 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
                for (int n2 = 0; n2 < KW / 16; ++n2) {
                    uint32_t b[4];
                    ldsm4(b, kb + sw<DP>(wk * KW + n2 * 16 + (lane & 7) + ((lane >> 4) << 3),
                                         kk * 2 + ((lane >> 3) & 1)));
                    mma16<T>(s[2 * n2], DP <= 128 ? qf[DP <= 128 ? kk : 0] : q1, b[0], b[1]);
                    mma16<T>(s[2 * n2 + 1], DP <= 128 ? qf[DP <= 128 ? kk : 0] : q1, b[2], b[3]);
                }
            }
            const int jw = j0 + wk * KW + 2 * tg;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = jw + 8 * n + (e & 1), i = e >> 1;
                    float x = a.softcap > 0.f ? capped(s[n][e], sc2, cap) : s[n][e] * sc2;
                    x = j >= lo[i] && j < hi[i] ? x : -INFINITY;
                    s[n][e] = x;
                    mx[i] = fmaxf(mx[i], x);
                }
            float base[2], corr[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                mx[i] = fmaxf(mx[i], m[i]);
                base[i] = mx[i] == -INFINITY ? 0.f : mx[i];
                corr[i] = exp2_approx(m[i] - base[i]);
                m[i] = mx[i];
                l[i] *= corr[i];
            }
            uint32_t p[KW / 16][4];
#pragma unroll
            for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = exp2_approx(s[n][e] - base[e >> 1]);
                    l[e >> 1] += s[n][e];
                }
                // the weights enter the product in the cache's type (at most half
                // a step of 1 each); their sum stays fp32 and unrounded
                p[n / 2][(n & 1) * 2] = Num16<T>::down2(s[n][0], s[n][1]);
                p[n / 2][(n & 1) * 2 + 1] = Num16<T>::down2(s[n][2], s[n][3]);
            }
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                o[i][0] *= corr[0];
                o[i][1] *= corr[0];
                o[i][2] *= corr[1];
                o[i][3] *= corr[1];
            }
#pragma unroll
            for (int k2 = 0; k2 < KW / 16; ++k2)
#pragma unroll
                for (int d2 = 0; d2 < DP / 16; ++d2) {
                    uint32_t b[4];
                    ldsm4t(b, vb + sw<DP>(wk * KW + k2 * 16 + (lane & 15), d2 * 2 + (lane >> 4)));
                    mma16<T>(o[2 * d2], p[k2], b[0], b[1]);
                    mma16<T>(o[2 * d2 + 1], p[k2], b[2], b[3]);
                }
            if (tid < AM_KT)
                off[(t % S) * AM_KT + tid] = noff;   // tile t + S
        }
        // ---- join the WK warps of each row
        cp_async_wait<0>();
        __syncthreads();
        float *ob = reinterpret_cast<float *>(stage);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            const int r = wr * 16 + g + 8 * i;
            if (tg == 0) {
                ml[(wk * M + r) * 2] = m[i];
                ml[(wk * M + r) * 2 + 1] = l[i];
            }
            float *dst = ob + (size_t)(wk * M + r) * L::OP + 2 * tg;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
        __syncthreads();
        const bool whole = ta == 0 && tb == w.nt;
        const int c0 = w.c0(), c1 = w.c1();
        float *part = attn_part<M, DP>(a, blockIdx.x, ta == 0);
        const int d4 = a.dim / 4;
        for (int i = tid; i < rows * d4; i += AM_THREADS) {
            const int r = i / d4, d = (i - r * d4) * 4;
            float mt = -INFINITY, lt = 0.f;
#pragma unroll
            for (int k = 0; k < WK; ++k)
                mt = fmaxf(mt, ml[(k * M + r) * 2]);
            const float b0 = mt == -INFINITY ? 0.f : mt;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < WK; ++k) {
                const float f = exp2_approx(ml[(k * M + r) * 2] - b0);
                const float4 x = *reinterpret_cast<const float4 *>(ob + (size_t)(k * M + r) * L::OP + d);
                lt = fmaf(f, ml[(k * M + r) * 2 + 1], lt);
                v.x = fmaf(f, x.x, v.x);
                v.y = fmaf(f, x.y, v.y);
                v.z = fmaf(f, x.z, v.z);
                v.w = fmaf(f, x.w, v.w);
            }
            const int tok = a.by_group(row0 + r), hq = w.h * a.group + (row0 + r) - tok * a.group;
            if (flag[1]) {   // the values taken out above, for the rows that see them
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
        if (!whole && attn_arrive<AM_THREADS>(a, c0, c1, flag))
            for (int r = warp; r < rows; r += AM_THREADS / 32)
                attn_join_row<T, M, DP>(a, c0, c1, r, w.s.q0, row0 + r, w.h);
        __syncthreads();   // the ring and the flags are free for the next unit
    }
}

template <class T, int DP, int WR>
cudaError_t launch_rows(const AttnArgs &a, const LaunchCfg &c)
{
    using L = AmLayout<DP, WR>;
    auto kern = attn_rows_kernel<T, DP, WR>;
    cudaError_t e = set_smem(kern, L::total);
    if (e != cudaSuccess)
        return e;
    constexpr int per_sm = 227 * 1024 / (L::total + 1024) > 3 ? 3 : 227 * 1024 / (L::total + 1024);
    const int ctas = c.num_sms * per_sm;
    LaunchCfg c2 = c;
    c2.pdl = false;
    return launch_ex(kern, dim3(ctas), dim3(AM_THREADS), L::total, c2, 1, a);
}

template <class T, int DP>
cudaError_t launch_dim(const AttnArgs &a, long long max_rows, const LaunchCfg &c)
{
    if (max_rows <= 16)
        return launch_rows<T, DP, 1>(a, c);
    if (max_rows <= 32)
        return launch_rows<T, DP, 2>(a, c);
    return launch_rows<T, DP, 4>(a, c);
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
    const int m = max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : 64;
    const size_t row = (size_t)2 * (dp + 2) * 4;   // two slots
    if (max_rows > 64)
        return kAttnCounterBytes + kAttnMaxSms * (256 * row + 32);   // and what the units are
    return kAttnCounterBytes + (size_t)kAttnMaxSms * 3 * m * row;
}

cudaError_t launch_attn(const AttnArgs &a, bool bf16, long long max_rows, const LaunchCfg &c)
{
    if (c.num_sms > kAttnMaxSms)
        return cudaErrorInvalidValue;
    if (max_rows > 64)
        // two row tiles per unit once there are units for every SM
        return launch_attn_tc(a, bf16, (long long)a.tokens * a.group / 256 * a.kv_heads >= c.num_sms ? 2 : 1, c);
    if (a.dim <= 64)
        return bf16 ? launch_dim<__nv_bfloat16, 64>(a, max_rows, c) : launch_dim<__half, 64>(a, max_rows, c);
    if (a.dim <= 128)
        return bf16 ? launch_dim<__nv_bfloat16, 128>(a, max_rows, c) : launch_dim<__half, 128>(a, max_rows, c);
    return bf16 ? launch_dim<__nv_bfloat16, 256>(a, max_rows, c) : launch_dim<__half, 256>(a, max_rows, c);
}

}  // namespace qmoe
