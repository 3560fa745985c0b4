// attention_tc.cu -- new tokens over a paged K/V cache, many query rows per
// K/V head (prompt chunks, verified drafts), on the 5th-generation tensor
// cores.  The formula and the division of the work are attn.cuh's.
//
// 4 D operations per visible (query, key) pair bound it: the two products on
// tcgen05.mma, and beside them one exponential per pair -- at D = 128 the
// exponentials of a 128 x 128 tile (16 a cycle and SM) cost as much time as
// its two products, so the kernel keeps both busy at once:
//   S = Q K^T   both operands in shared memory, S in tensor memory (fp32)
//   softmax     one thread per row: its S row from tensor memory, running
//               maximum and sum in registers, the weights back to tensor
//               memory over S in the cache's 16-bit type
//   O += P V    P from tensor memory, V as it lies in the cache (MN-major),
//               O in tensor memory
// NROW = 2 (head_dim <= 128): a unit is 256 query rows, two row tiles with a
// softmax warpgroup each; while one tile's weights are made, the other's
// products run.  NROW = 1 (128 rows; head_dim 256, or few rows): the scores
// of the next key tile are made while the softmax works on this one.
// O is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time: until then the weights are at most 2^8 more (exact powers of
// the same base, no rounding is lost), so most tiles touch O in the product only.
//
// Roles: the softmax warpgroups; a warp that issues the products; a TMA warp
// each for K, V and Q; and a warpgroup that cleans values at the limits and
// writes the units' outputs, so that the softmax goes on to the next unit
// meanwhile.  K and V arrive in the 128-byte-swizzled blocks of 64 columns that both operand
// descriptors read, by TMA in boxes of up to a page where the cache has a
// tensor map, else (page sizes that no multiple of 8 divides, heads below 64)
// by 16-byte cp.async: 27 cycles per warp instruction, which held a 128-key
// tile of K and V to 5200 cycles where the products need 2048.
// Measured (of 1.65 PFLOP/s, counting visible pairs only): 4 ragged chunks of
// 2048 tokens over 8192, 32 heads of 128, bf16, 380 us, 810 TFLOP/s in calls one
// after the other (power), 336, 915 TFLOP/s in one replay of a graph at a time,
// as the other times here were taken -- a row
// tile's chain (scores, softmax, weights, products) is as long as two row
// tiles' products take, the tensor pipe is busy 47% of the time, the exponentials'
// 47%.  A half row a softmax thread, four softmax warpgroups, made it 357 (80
// registers a thread are too few); a chunk of 128 tokens over 4096, 31 us, of
// which 9 are the tiles (each CTA reads 60 bytes a ns from L2; key tiles by
// turns to two softmax warpgroups made it 33), the rest lengths, page table,
// first tiles, the parts and their joining; 8 of 24 tokens, window, cap, heads
// of 256: 37 us, 60 MB.
// Every wait is bounded; on a timeout the roles stop, the copies and products
// in flight finish and the tensor memory is freed.
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr float TC_LAZY = 8.f;   // log2 of the growth of a maximum that O is not rescaled for

// Beginning and ending a unit, in tiles: 4 chunks of 2048 tokens take 397 us
// with 1, 354 with 2, 336 with 3, 349 with 6; 8 of 24 tokens 38.2, 37.0, 37.4, 38.9.
constexpr int TC_EX = 3;

template <int DP, int NROW>
struct TcCfg {
    static constexpr int KT = DP == 256 ? 64 : 128;      // keys per tile
    static constexpr int M = 128 * NROW;
    static constexpr int KS = 2, VS = 2;                 // stages; S buffers: also 2, row tiles or tiles in turn
    static constexpr int tile = KT * DP * 2;
    static constexpr int SOFT = 128 * NROW;              // softmax threads
    static constexpr int LOAD = 128;                     // loader threads
    // beside them a warpgroup of the MMA warp, the K and the V warp of TMA
    static constexpr int THREADS = SOFT + 128 + LOAD;
    // registers a thread: the softmax holds a row's scores
    static constexpr int R_SOFT = NROW == 2 ? 168 : 232, R_REST = NROW == 2 ? 88 : 128;
    // tensor memory columns
    static constexpr int s_col = 0;                      // + 128 per buffer
    static constexpr int o_col = 256;                    // + DP per row tile
    static constexpr int q_off = 0;
    static constexpr int k_off = q_off + M * DP * 2;
    static constexpr int v_off = k_off + KS * tile;
    static constexpr int off_off = v_off + VS * tile;    // [2][KT] int64
    static constexpr int bar_off = off_off + 2 * KT * 8;
    static constexpr int misc_off = bar_off + 32 * 8;
    static constexpr int walk_off = misc_off + 64;       // a warp's place in its interval
    static constexpr int ml_off = walk_off + THREADS / 32 * 128;   // the rows' maxima and sums
    static constexpr int stg_off = ml_off + M * 8;       // 2 KB per loader warp, which also write the output
    static constexpr int total = stg_off + LOAD / 32 * 2048 + 1024;   // + alignment slack
    static_assert(KT <= LOAD, "a loader thread per key");
    static_assert(o_col + NROW * DP <= 512, "tensor memory");
    static_assert(total <= 227 * 1024, "shared memory");
};

enum {
    TB_QF = 0, TB_QE, TB_KF, TB_KE = TB_KF + 2, TB_VF = TB_KE + 2, TB_VE = TB_VF + 2, TB_SF = TB_VE + 2,
    TB_PF = TB_SF + 2, TB_OF = TB_PF + 2, TB_OE = TB_OF + 2, TB_VX = TB_OE + 2, TB_P2 = TB_VX + 2, TB_LF = TB_P2 + 2, TB_PV = TB_LF + 2, TB_DRAIN, TB_COUNT
};
static_assert(TB_COUNT <= 32, "barriers");
constexpr int TC_BAR_LOAD = 1;   // named barrier

// 128-byte-swizzled operand blocks of 64 columns (128-byte rows, 8-row groups
// 1024 bytes apart); lead: bytes between blocks of 64 columns, read for the
// MN-major operand only
__device__ __forceinline__ uint64_t at_desc(uint32_t saddr, uint32_t lead)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// fp32 D, M = 128, N = n; A and B both fp16 or both bf16; b_mn: B is MN-major
template <class T>
__device__ __forceinline__ uint32_t at_idesc(int n, bool b_mn)
{
    const uint32_t f = sizeof(T) == 2 && Num16<T>::kExp == 0x7F807F80u ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void at_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// true for one thread of a converged warp, the same one each time
__device__ __forceinline__ bool at_elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void at_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void at_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void at_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// two fp32 operations in one instruction
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 32 lanes x 32 consecutive columns of tensor memory, without the wait
__device__ __forceinline__ void at_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void at_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void at_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// The loads into r have landed.  The registers are operands, so that nothing
// that uses them can be moved before the wait.
__device__ __forceinline__ void at_wait_ld(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void at_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// nothing that uses these registers can be moved before this point
__device__ __forceinline__ void at_pin(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// 16 columns times f
__device__ __forceinline__ void at_scale16(uint32_t taddr, float f)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    at_st16(taddr, r);
}

// bounded wait until a stage has been armed for tile `n`
__device__ __forceinline__ bool at_armed(volatile int *arm, int n, const AttnArgs &a, volatile int *abort_word)
{
    if (*arm == n)
        return true;
    const unsigned long long t0 = global_timer_ns();
    while (*arm != n) {
        __nanosleep(20);
        if (*abort_word)
            return false;
        if (global_timer_ns() - t0 >= a.wait_ns) {
            flag_status(a.status, QMOE_DEV_TIMEOUT);
            *abort_word = 1;
            return false;
        }
    }
    return true;
}

// A unit that begins in a CTA and goes on in later ones, up to c1 (0: none).
// The parts are up to 128 KB each and as many as the GPU has SMs, too much for
// one CTA to add up (64 us for 9 parts when the last to arrive did it): a second
// kernel joins them with the whole GPU, launched while this one runs (it ends 6
// us after the last part is written, 128 tokens over 4096).
struct TcShared {
    int c1, q0, row0, rows, h;
};
template <int M, int DP>
__device__ __forceinline__ TcShared *tc_shared(const AttnArgs &a)
{
    return reinterpret_cast<TcShared *>(a.part + (size_t)kAttnMaxSms * 2 * M * (DP + 2));
}

// Where in a part four sums lie, columns 4u.. of row r: a thread that holds a
// row and a warp that holds 32 of them both go through memory in order.
template <int M>
__device__ __forceinline__ int tc_at(int u, int r)
{
    return (u * M + r) * 4;
}

// Keys that every row of a block sees: [lo_max, hi_min).
__device__ __forceinline__ void at_limits(const AttnArgs &a, const AttnSeq &s, int row0, int rows, int &lo_max,
                                          int &hi_min)
{
    int d;
    attn_keys(a, s, a.by_group(row0), d, hi_min);
    attn_keys(a, s, a.by_group(row0 + rows - 1), lo_max, d);
}

// Adds the infinite and NaN values that clean_v took out of the tiles at the
// limits to the rows of O that see them: a warp's 32 rows in tensor memory.
template <class T, class Walk, int KT>
__device__ __noinline__ void at_restore(const AttnArgs &a, const Walk &w, int row0, int rows, int r, uint32_t taddr)
{
    int lo = 0, hi = 0, lo_max, hi_min;
    if (r < rows)
        attn_keys(a, w.s, a.by_group(row0 + r), lo, hi);
    at_limits(a, w.s, row0, rows, lo_max, hi_min);
    lo = max(lo, (w.t0 + w.ta()) * KT);
    hi = min(hi, (w.t0 + w.tb()) * KT);
    for (int c = 0; c < a.dim; c += 32) {
        uint32_t u[32];
        at_ld32(taddr + c, u);
        at_wait_ld(u);
        for (int j = lo; j < hi; ++j) {
            if (j >= lo_max && j < hi_min) {
                j = hi_min - 1;
                continue;
            }
            const long long e = attn_slot(a, w.sp.b, w.h, j);
            if (e < 0)
                continue;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < a.dim) {
                    const float x = Num16<T>::up(a.v[e + c + i]);
                    if (!isfinite(x))
                        u[i] = __float_as_uint(__uint_as_float(u[i]) + x);
                }
        }
        __syncwarp();
        at_st32(taddr + c, u);
    }
    at_wait_st();
}

// A warp's rows of scores in tensor memory, capped by a wide cap.  A call, so
// that its forms take no registers from the softmax of other calls' scores.
template <int KT>
__device__ __noinline__ void at_cap(const AttnArgs &a, uint32_t taddr)
{
    const AttnCap cap(a.scale, a.softcap);
#pragma unroll 1
    for (int c = 0; c < KT; c += 32) {
        uint32_t s[32];
        at_ld32(taddr + c, s);
        at_wait_ld(s);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            most = fmaxf(most, fabsf(__uint_as_float(s[i])));
        if (cap.above(most)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i] = __float_as_uint(cap.any(__uint_as_float(s[i])));
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i] = __float_as_uint(cap.low(__uint_as_float(s[i])));
        }
        at_st32(taddr + c, s);
    }
    at_wait_st();
}

template <class T, int DP, int NROW>
__global__ void __launch_bounds__(TcCfg<DP, NROW>::THREADS, 1) attn_tc_kernel(const AttnArgs a, const __grid_constant__ AttnMaps maps)
{
    using C = TcCfg<DP, NROW>;
    constexpr int KT = C::KT, M = C::M;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::bar_off);
    uint32_t *tmem_word = reinterpret_cast<uint32_t *>(smem + C::misc_off);
    volatile int *abort_word = reinterpret_cast<volatile int *>(smem + C::misc_off + 4);
    volatile int *poison = reinterpret_cast<volatile int *>(smem + C::misc_off + 16);   // V of this unit was cleaned
    float2 *ml = reinterpret_cast<float2 *>(smem + C::ml_off);
    volatile int *armed_v = reinterpret_cast<volatile int *>(smem + C::misc_off + 32);  // [2], tile in the V stage
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W_MMA = C::SOFT / 32;

    if (tid == 0) {
        const int full = a.tma ? 1 : C::LOAD;
        mbar_init(&bar[TB_QF], a.tma_q ? 1 : C::LOAD);
        mbar_init(&bar[TB_QE], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[TB_KF + i], full);
            mbar_init(&bar[TB_KE + i], 1);
            mbar_init(&bar[TB_VF + i], full);
            mbar_init(&bar[TB_VX + i], C::LOAD);
            mbar_init(&bar[TB_VE + i], 1);
            mbar_init(&bar[TB_SF + i], 1);
            mbar_init(&bar[TB_PF + i], 128);
            mbar_init(&bar[TB_P2 + i], 128);
            mbar_init(&bar[TB_LF + i], 128);
            mbar_init(&bar[TB_OF + i], 1);
            mbar_init(&bar[TB_OE + i], 128);
        }
        mbar_init(&bar[TB_PV], 1);
        mbar_init(&bar[TB_DRAIN], 1);
        *abort_word = 0;
        armed_v[0] = armed_v[1] = -1;
        mbar_init_fence();
    }
    if (warp == W_MMA) {   // all of the SM's tensor memory (this warp frees it)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_word)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == W_MMA + 1 && lane == 0 && a.tma) {   // fetched while the lengths are
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        if (a.tma_q)
            prefetch_tensormap(&maps.q);
    }
    pdl_wait();
    pdl_trigger();   // the joining kernel may be launched; it waits for this one's end
    if (tid == 0)
        tc_shared<M, DP>(a)[blockIdx.x].c1 = 0;
    const AttnSpan span = attn_span<M, KT, TC_EX>(a);
    at_fence_before();
    __syncthreads();
    at_fence_after();
    const uint32_t tmem = *tmem_word;
    // Each warp's place in the CTA's interval lies in shared memory: in registers
    // it would push a row's scores out of them.
    using Walk = AttnWalk<M, KT, TC_EX>;
    static_assert(sizeof(Walk) <= 128, "walk");
    Walk &w = *reinterpret_cast<Walk *>(smem + C::walk_off + warp * 128);
    if (lane == 0)
        w.start(a, span);
    __syncwarp();
    auto advance = [&]() {
        __syncwarp();
        if (lane == 0)
            w.next(a);
        __syncwarp();
    };

    if (warp >= W_MMA) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_REST));
        if (warp == W_MMA) {
            // ================================================= MMA issuer
            // The whole warp walks and waits; one elected thread issues.
            const uint32_t idesc_s = at_idesc<T>(KT, false);
            const int n_o = (a.dim + 15) & ~15, ksteps = (a.dim + 15) / 16;
            const uint32_t idesc_o = at_idesc<T>(n_o, true);
            const uint64_t qd = at_desc(smem_u32(smem + C::q_off), 16), kd = at_desc(smem_u32(smem + C::k_off), 16),
                           vd = at_desc(smem_u32(smem + C::v_off), KT * 128);
            uint32_t kc = 0, vc = 0, un = 0;          // tiles and units so far
            // parities of the barrier pairs, a bit each (arrays would lie in local
            // memory); given: bit r once row tile r's O has been handed over
            uint32_t pc = 0, oc = 0, xc = 0, given = 0;
            bool ok = true, issued = false;
            auto wait = [&](int b, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, at_wait(&bar[b], parity & 1, a, abort_word));
                return ok;
            };
            auto commit = [&](int b) {
                if (at_elect())
                    at_commit(&bar[b]);
                __syncwarp();
            };
            // Products are issued from straight code, the descriptors' start
            // addresses (in units of 16 bytes) stepped by constants: built anew
            // for each step, they took the thread longer than the 64 cycles that
            // the step takes.
            auto scores = [&](int buf, int rt, uint32_t ks) {
                const uint64_t q = qd + rt * (128 * 128 / 16), k = kd + ks * (C::tile / 16);
                const uint32_t d = tmem + C::s_col + buf * 128;
                if (ksteps == DP / 16) {
                    if (at_elect()) {
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
                            at_mma_ss(d, q + ((i >> 2) * M * 128 + (i & 3) * 32) / 16,
                                      k + ((i >> 2) * KT * 128 + (i & 3) * 32) / 16, idesc_s, i > 0);
                    }
                } else {
                    if (at_elect()) {
#pragma unroll 1
                        for (int i = 0; i < ksteps; ++i)
                            at_mma_ss(d, q + ((i >> 2) * M * 128 + (i & 3) * 32) / 16,
                                      k + ((i >> 2) * KT * 128 + (i & 3) * 32) / 16, idesc_s, i > 0);
                    }
                }
                __syncwarp();
                commit(TB_SF + buf);
                issued = true;
            };
            // one half of a tile's keys: the first can start while the softmax
            // still works on the second
            auto values = [&](int buf, int rt, uint32_t vs, int half, bool acc) {
                const uint64_t v = vd + vs * (C::tile / 16) + half * (KT / 32) * 128;
                const uint32_t d = tmem + C::o_col + rt * DP, p = tmem + C::s_col + buf * 128 + half * (KT / 32) * 8;
                if (at_elect()) {
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i)
                        at_mma_ts(d, p + i * 8, v + i * 128, idesc_o, i > 0 || acc);
                }
                __syncwarp();
            };
            for (; !w.done() && ok; advance(), ++un) {
                const int nt = w.tb() - w.ta();
                const int rows = min(M, w.s.n * a.group - w.rt * M);
                const int nr = NROW == 2 && rows > 128 ? 2 : 1;   // row tiles with rows
                int lo_max, hi_min;
                at_limits(a, w.s, w.rt * M, rows, lo_max, hi_min);
                if (!wait(TB_QF, un) || !wait(TB_KF + kc % 2, kc / 2))
                    break;
                at_fence_after();
                for (int r = 0; r < nr; ++r)
                    scores(NROW == 2 ? r : 0, r, kc % 2);
                commit(TB_KE + kc % 2);
                ++kc;
                if (nt == 1)
                    commit(TB_QE);
                for (int j = 0; j < nt && ok; ++j, ++vc) {
                    const bool more = j + 1 < nt;
                    if (NROW == 1 && more) {
                        if (!wait(TB_KF + kc % 2, kc / 2))
                            break;
                        at_fence_after();
                        scores((j + 1) & 1, 0, kc % 2);
                        commit(TB_KE + kc % 2);
                        ++kc;
                        if (j + 2 == nt)
                            commit(TB_QE);
                    }
                    const int j0 = (w.t0 + w.ta() + j) * KT;
                    if (a.tma && (j0 < lo_max || j0 + KT > hi_min)) {
                        if (!wait(TB_VX + vc % 2, xc >> (vc % 2)))
                            break;
                        xc ^= 1u << (vc % 2);
                    } else if (!wait(TB_VF + vc % 2, vc / 2)) {
                        break;
                    }
                    if (NROW == 2 && more && !wait(TB_KF + kc % 2, kc / 2))
                        break;
                    for (int r = 0; r < nr; ++r) {
                        const int buf = NROW == 2 ? r : j & 1;
                        if (!wait(TB_PF + buf, pc >> buf))
                            break;
                        if (j == 0 && ((given >> r) & 1) && !wait(TB_OE + r, (oc >> r) ^ 1))
                            break;   // the last unit's O has been read
                        at_fence_after();
                        values(buf, r, vc % 2, 0, j > 0);
                        if (!wait(TB_P2 + buf, pc >> buf))
                            break;
                        pc ^= 1u << buf;
                        at_fence_after();
                        values(buf, r, vc % 2, 1, true);
                        if (NROW == 1)
                            commit(TB_PV);
                        if (NROW == 2 && more)
                            scores(buf, r, kc % 2);
                        if (!more) {
                            commit(TB_OF + r);
                            oc ^= 1u << r;
                            given |= 1u << r;
                        }
                    }
                    if (!ok)
                        break;
                    commit(TB_VE + vc % 2);
                    if (NROW == 2 && more) {
                        commit(TB_KE + kc % 2);
                        ++kc;
                        if (j + 2 == nt)
                            commit(TB_QE);
                    }
                }
            }
            if (issued) {   // nothing is in flight when the tensor memory is freed
                commit(TB_DRAIN);
                mbar_wait(&bar[TB_DRAIN], 0, a.status);
            }
            __syncwarp();
        } else {
            // ==================================================== loaders
            constexpr int CPR = DP / 8;
            const int cpr = ((a.dim + 15) & ~15) / 8;   // 16-byte units that the products read
            const uint32_t qs = smem_u32(smem + C::q_off);
            bool dead = false;
            // a block's query rows, by threads t of NT: each stays in its column
            auto load_q = [&](int t, int nt, int row0, int rows) {
                const int c = t % CPR;
                const int tok0 = a.by_group(row0), rem = row0 - tok0 * a.group;
                const bool in = c * 8 < a.dim;
                if (c >= cpr)
                    return;
                const int rows_q = NROW == 2 && rows <= 128 ? 128 : M;
#pragma unroll 4
                for (int r = t / CPR; r < rows_q; r += nt / CPR) {
                    const int dt = a.by_group(rem + r);
                    const int hq = w.h * a.group + rem + r - dt * a.group;
                    const bool live = in && r < rows;
                    const long long e = (w.s.q0 + tok0 + dt) * a.q_token + hq * a.q_head + c * 8;
                    cp_async16(qs + at_sw(M, r, c), a.q + (live ? e : 0), live);
                }
            };
            // Keys that only some rows see, and keys outside the unit whose
            // stale slots a TMA box brought along: a weight of zero times an
            // infinite or NaN value would still reach the rows through the
            // product.  Values outside the unit become zeros; infinite and NaN
            // ones at the limits are taken out and added to the rows that see
            // them at the end of the unit.
            auto clean_v = [&](int stage, int j0, int lo_max, int hi_min, int t, int nt) {
                unsigned char *v = smem + C::v_off + stage * C::tile;
                const int r1 = min(max(lo_max - j0, 0), KT), r2 = max(min(hi_min - j0, KT), r1);
                const int c = t % CPR;
                const int step = nt / CPR, lo = w.lo, hi = w.hi;
                // The rows at the limits one after the other; without TMA each thread
                // stays with those its own cp.async brings: it has waited for no others.
                const int n = a.tma ? KT - (r2 - r1) : KT;
                if (c < cpr)
                    for (int i0 = t / CPR; i0 < n; i0 += 4 * step) {
                        uint4 x[4];   // four rows' loads are under way at once
                        int r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = i0 + k * step;
                            r[k] = i >= n ? -1 : i < r1 ? i : a.tma ? i + (r2 - r1) : i >= r2 ? i : -1;
                            if (r[k] >= 0)
                                x[k] = *reinterpret_cast<const uint4 *>(v + at_sw(KT, r[k], c));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (r[k] < 0)
                                continue;
                            uint4 *q = reinterpret_cast<uint4 *>(v + at_sw(KT, r[k], c));
                            if (j0 + r[k] < lo || j0 + r[k] >= hi) {
                                *q = make_uint4(0, 0, 0, 0);
                            } else if (nonfinite2<T>(x[k].x) || nonfinite2<T>(x[k].y) || nonfinite2<T>(x[k].z) ||
                                       nonfinite2<T>(x[k].w)) {
                                uint32_t *p = reinterpret_cast<uint32_t *>(&x[k]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = Num16<T>::up2(p[e]);
                                    p[e] = Num16<T>::down2(isfinite(f.x) ? f.x : 0.f, isfinite(f.y) ? f.y : 0.f);
                                }
                                *q = x[k];
                                *poison = 1;
                            }
                        }
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            };
            // The output of a unit, by the loader warps (so that the softmax goes on
            // to the next unit): O from tensor memory, 16 rows x 128 bytes at a
            // time through shared memory, so that 8 lanes write a row's 128 bytes
            // together.  oc: parities, a bit for each row tile.
            uint32_t oc = 0;
            auto output = [&]() {
                const int ta = w.ta(), tb = w.tb(), row0 = w.rt * M;
                const int rows = min(M, w.s.n * a.group - row0);
                const bool whole = ta == 0 && tb == w.nt;
                const int quad = warp & 3;
                unsigned char *stg = smem + C::stg_off + quad * 2048;
                float *part = attn_part<M, DP>(a, blockIdx.x, ta == 0);
                if (warp == W_MMA + 4 && lane == 0 && ta == 0 && tb < w.nt) {   // begins here, goes on in later CTAs
                    TcShared *d = tc_shared<M, DP>(a) + blockIdx.x;
                    d->q0 = w.s.q0;
                    d->row0 = row0;
                    d->rows = rows;
                    d->h = w.h;
                    d->c1 = w.c1();
                }
                for (int rt = 0; rt < NROW && rt * 128 < rows; ++rt) {
                    if (!__all_sync(0xffffffffu, at_wait(&bar[TB_LF + rt], (oc >> rt) & 1, a, abort_word) &&
                                                     at_wait(&bar[TB_OF + rt], (oc >> rt) & 1, a, abort_word))) {
                        dead = true;
                        return;
                    }
                    oc ^= 1u << rt;
                    at_fence_after();
                    const int r0 = rt * 128 + quad * 32, rr = r0 + lane;
                    const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + C::o_col + rt * DP;
                    const float2 mlr = ml[rr];
                    if (*poison != 0)
                        at_restore<T, Walk, KT>(a, w, row0, rows, rr, to);
                    const int tok = a.by_group(row0 + rr), hq = w.h * a.group + (row0 + rr) - tok * a.group;
                    if (!whole) {
#pragma unroll 1
                        for (int c0 = 0; c0 < a.dim; c0 += 32) {
                            uint32_t v[32];
                            at_ld32(to + c0, v);
                            at_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (rr < rows && c0 + i * 4 < a.dim)
                                    *reinterpret_cast<uint4 *>(part + tc_at<M>(c0 / 4 + i, rr)) =
                                        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    } else {
                        // where this lane's row goes; the others are told by shuffle
                        const long long mine = (w.s.q0 + tok) * a.o_token + hq * a.o_head;
                        const float inv = mlr.y == 0.f ? 0.f : 1.f / mlr.y;
                        const int unit = lane & 7;
#pragma unroll 1
                        for (int c0 = 0; c0 < a.dim; c0 += 64) {
                            uint32_t v[32];
                            at_ld32(to + c0, v);
                            at_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                v[i] = Num16<T>::down2(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
                            if (c0 + 32 < a.dim) {
                                uint32_t u[32];
                                at_ld32(to + c0 + 32, u);
                                at_wait_ld(u);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    v[16 + i] = Num16<T>::down2(__uint_as_float(u[2 * i]) * inv,
                                                                __uint_as_float(u[2 * i + 1]) * inv);
                            }
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if ((lane >> 4) == half) {
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        *reinterpret_cast<uint4 *>(stg + (lane & 15) * 128 + ((i ^ (lane & 7)) << 4)) =
                                            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                                }
                                __syncwarp();
                                uint4 x[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int r = i * 4 + (lane >> 3);
                                    x[i] = *reinterpret_cast<const uint4 *>(stg + r * 128 + ((unit ^ (r & 7)) << 4));
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int r = half * 16 + i * 4 + (lane >> 3);
                                    const long long at = __shfl_sync(0xffffffffu, mine, r);
                                    if (r0 + r < rows && c0 + unit * 8 < a.dim)
                                        *reinterpret_cast<uint4 *>(a.out + at + c0 + unit * 8) = x[i];
                                }
                                __syncwarp();
                            }
                        }
                    }
                    at_fence_before();
                    mbar_arrive(&bar[TB_OE + rt]);
                    if (rr < rows) {
                        if (!whole) {
                            part[M * DP + rr] = mlr.x;
                            part[M * DP + M + rr] = mlr.y;
                        } else if (a.lse) {
                            a.lse[(size_t)(w.s.q0 + tok) * a.heads + hq] =
                                mlr.y == 0.f ? -INFINITY : (mlr.x + log2f(mlr.y)) * kLn2;
                        }
                    }
                }
            };
            if (warp < W_MMA + 4) {
                // ---- TMA: one warp for K, one for V (so that K never waits for
                // a slot of V), each lane a box of the tile's keys; one for Q
                const int x = warp - W_MMA - 1;
                const int nbox = KT / max(a.tma, 1), nblk = (a.dim + 63) / 64;
                const uint32_t bytes = KT * 128 * nblk;
                const void *map = x ? &maps.v : &maps.k;
                uint32_t n = 0;   // tiles so far
                for (; a.tma && x < 2 && !w.done() && !dead; advance()) {
                    const int ta = w.ta(), tb = w.tb();
                    int j = (w.t0 + ta) * KT + lane * a.tma;
                    int ahead = lane < nbox ? attn_page(a, w.sp.b, j, w.lo, w.hi) : 0;
                    for (int t = ta; t < tb; ++t, ++n, j += KT) {
                        int page = ahead;
                        const int slot = j - a.by_page(j) * a.page_size;
                        if (t + 1 < tb && lane < nbox)   // on its way while this tile's copies go out
                            ahead = attn_page(a, w.sp.b, j + KT, w.lo, w.hi);
                        if (n >= 2 && !__all_sync(0xffffffffu, at_wait(&bar[(x ? TB_VE : TB_KE) + n % 2], (n / 2 - 1) & 1,
                                                                       a, abort_word))) {
                            dead = true;
                            break;
                        }
                        uint64_t *full = &bar[(x ? TB_VF : TB_KF) + n % 2];
                        if (lane == 0) {
                            mbar_arrive_expect_tx(full, bytes);
                            if (x)
                                armed_v[n % 2] = (int)n;
                        }
                        __syncwarp();
                        if (lane < nbox) {
                            if ((unsigned)page > (unsigned)a.num_pages ||
                                (page == a.num_pages && j < w.hi && j + a.tma > w.lo)) {
                                flag_status(a.status, QMOE_DEV_BAD_PAGE);
                                page = a.num_pages;
                            }
                            const uint32_t dst = smem_u32(smem + (x ? C::v_off : C::k_off) + (n % 2) * C::tile) +
                                                 lane * a.tma * 128;
                            for (int k = 0; k < nblk; ++k)
                                tma_load_4d(dst + k * KT * 128, map, k * 64, a.heads_inner ? w.h : slot,
                                            a.heads_inner ? slot : w.h, page, full);
                        }
                        __syncwarp();
                    }
                }
                if (x == 2 && a.tma_q) {
                    // ---- the query rows: 128 rows are 128 / group tokens x the group's heads
                    uint32_t un = 0;
                    for (; !w.done() && !dead; advance(), ++un) {
                        const int row0 = w.rt * M, rows = min(M, w.s.n * a.group - row0);
                        const int nr = NROW == 2 && rows > 128 ? 2 : 1;
                        if (un > 0 && !__all_sync(0xffffffffu,
                                                  at_wait(&bar[TB_QE], (un - 1) & 1, a, abort_word))) {
                            dead = true;
                            break;
                        }
                        if (lane == 0)
                            mbar_arrive_expect_tx(&bar[TB_QF], nr * nblk * 128 * 128);
                        __syncwarp();
                        const int k = lane % nblk, r = lane / nblk;
                        if (r < nr)
                            tma_load_3d(smem + C::q_off + k * M * 128 + r * 128 * 128, &maps.q, k * 64, w.h * a.group,
                                        w.s.q0 + a.by_group(row0 + r * 128), &bar[TB_QF]);
                        __syncwarp();
                    }
                    if (lane == 0 && un > 0)
                        mbar_wait(&bar[TB_QF], (un - 1) & 1, a.status);
                }
                // no copy may still be landing when the CTA exits
                if (lane == 0 && x < 2)
                    for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i)
                        mbar_wait(&bar[(x ? TB_VF : TB_KF) + i % 2], (i / 2) & 1, a.status);
                __syncwarp();
            } else if (a.tma) {
                // ---- beside it: the query rows, and V at the limits
                const int t = tid - C::SOFT - 128;
                uint32_t un = 0, n = 0;
                for (; !w.done(); advance(), ++un) {
                    const int ta = w.ta(), tb = w.tb();
                    const int row0 = w.rt * M, rows = min(M, w.s.n * a.group - row0);
                    // (with Q on TMA these warps must not wait for it: its next use may
                    // be over before they come here)
                    if (un > 0 && !a.tma_q && !at_wait(&bar[TB_QE], (un - 1) & 1, a, abort_word))
                        dead = true;
                    if (bar_any(TC_BAR_LOAD, C::LOAD, dead))
                        break;
                    if (t == 0)
                        *poison = 0;
                    if (!a.tma_q) {
                        load_q(t, C::LOAD, row0, rows);
                        cp_async_commit();
                        cp_async_wait<0>();
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        mbar_arrive(&bar[TB_QF]);
                    }
                    named_bar_sync(TC_BAR_LOAD, C::LOAD);   // the cleared poison flag is seen
                    int lo_max, hi_min;
                    at_limits(a, w.s, row0, rows, lo_max, hi_min);
                    for (int i = ta; i < tb && !dead; ++i) {
                        const int j0 = (w.t0 + i) * KT;
                        if (j0 >= lo_max && j0 + KT <= hi_min)
                            continue;
                        const uint32_t s = n + (i - ta);
                        // armed first: a parity tells two uses of a stage apart only
                        // once the earlier one is over
                        if (!at_armed(&armed_v[s % 2], (int)s, a, abort_word) ||
                            !at_wait(&bar[TB_VF + s % 2], (s / 2) & 1, a, abort_word)) {
                            dead = true;
                            break;
                        }
                        clean_v(s % 2, j0, lo_max, hi_min, t, C::LOAD);
                        mbar_arrive(&bar[TB_VX + s % 2]);
                    }
                    n += tb - ta;
                    // (a warp that gives up leaves here or at the next barrier)
                    if (!__any_sync(0xffffffffu, dead))
                        output();
                }
            } else {
                // ---- cp.async
                const int lt = tid - C::SOFT - 128;
                long long *off = reinterpret_cast<long long *>(smem + C::off_off);
                uint32_t kc = 0, un = 0;
                // copies in flight, oldest first: the barrier to arrive at and, for
                // a V tile with keys that only some rows see, where it lies
                int pend_bar[3] = {0, 0, 0}, pend_j0[3] = {-1, -1, -1}, np = 0;
                int lo_max = 0, hi_min = 0;
                auto finish = [&](int i) {
                    if (pend_j0[i] >= 0)
                        clean_v(pend_bar[i] - TB_VF, pend_j0[i], lo_max, hi_min, lt, C::LOAD);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive(&bar[pend_bar[i]]);
                };
                auto flush = [&]() {
                    cp_async_wait<0>();
                    for (int i = 0; i < np; ++i)
                        finish(i);
                    np = 0;
                };
                auto push = [&](int b, int j0) {
                    cp_async_commit();
                    pend_bar[np] = b;
                    pend_j0[np] = j0;
                    if (++np == 3) {
                        cp_async_wait<2>();
                        finish(0);
                        pend_bar[0] = pend_bar[1];
                        pend_bar[1] = pend_bar[2];
                        pend_j0[0] = pend_j0[1];
                        pend_j0[1] = pend_j0[2];
                        np = 2;
                    }
                };
                // the slot of the n-th use of a barrier pair is free again; what is
                // in flight is handed over before blocking
                auto acquire = [&](int b, uint32_t n, uint32_t stages) {
                    if (n < stages || dead)
                        return;
                    const uint32_t parity = (n / stages - 1) & 1;
                    if (mbar_try_wait_now(&bar[b], parity))
                        return;
                    flush();
                    if (!at_wait(&bar[b], parity, a, abort_word))
                        dead = true;
                };
                auto slot = [&](int t, int tb, int r) {
                    const int j = (w.t0 + t) * KT + r;
                    long long o = -1;
                    if (r < KT && t < tb && j >= w.lo && j < w.hi) {
                        o = attn_slot(a, w.sp.b, w.h, j);
                        if (o < 0)
                            flag_status(a.status, QMOE_DEV_BAD_PAGE);
                    }
                    return o;
                };
                for (; !w.done(); advance(), ++un) {
                    const int ta = w.ta(), tb = w.tb();
                    const int row0 = w.rt * M, rows = min(M, w.s.n * a.group - row0);
                    long long o0 = slot(ta, tb, lt);
                    acquire(TB_QE, un, 1);
                    at_limits(a, w.s, row0, rows, lo_max, hi_min);
                    if (bar_any(TC_BAR_LOAD, C::LOAD, dead || *abort_word != 0))
                        break;
                    if (lt == 0)
                        *poison = 0;
                    load_q(lt, C::LOAD, row0, rows);
                    push(TB_QF, -1);
                    for (int t = ta; t < tb; ++t, ++kc) {
                        long long *o = off + (t & 1) * KT;
                        if (lt < KT)
                            o[lt] = o0;
                        // (the barrier also keeps the loaders together after a timeout)
                        if (bar_any(TC_BAR_LOAD, C::LOAD, dead))
                            break;
                        o0 = slot(t + 1, tb, lt);
                        for (int x = 0; x < 2; ++x) {   // K, then V
                            const int fb = (x ? TB_VF : TB_KF) + (int)(kc % 2);
                            acquire((x ? TB_VE : TB_KE) + (int)(kc % 2), kc, 2);
                            if (dead)
                                break;
                            const uint32_t dst = smem_u32(smem + (x ? C::v_off : C::k_off) + (kc % 2) * C::tile);
                            const uint16_t *base = x ? a.v : a.k;
                            // a thread stays in its column; 8 rows' offsets are read
                            // before their copies go out, so that no copy waits for
                            // shared memory
                            constexpr int RP = C::LOAD / CPR;   // rows per pass
                            const int c = lt % CPR;
                            if (c < cpr) {
                                const bool in = c * 8 < a.dim;
                                for (int r0 = lt / CPR; r0 < KT; r0 += 8 * RP) {
                                    long long s[8];
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        s[i] = r0 + i * RP < KT ? o[r0 + i * RP] : 0;
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        if (r0 + i * RP < KT) {
                                            const bool live = in && s[i] >= 0;
                                            cp_async16(dst + at_sw(KT, r0 + i * RP, c),
                                                       base + (live ? s[i] + c * 8 : 0), live);
                                        }
                                }
                            }
                            const int j0 = (w.t0 + t) * KT;
                            const bool some = (j0 < lo_max && j0 + KT > w.lo) || (j0 + KT > hi_min && j0 < w.hi);
                            push(fb, x && some ? j0 : -1);
                        }
                    }
                    flush();   // this unit's V is looked over with its own rows' limits
                    if (bar_any(TC_BAR_LOAD, C::LOAD, dead))
                        break;
                    output();
                }
            }
        }
    } else {
        // ====================================================== softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::R_SOFT));
        const int rt = warp >> 2, quad = warp & 3;
        const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
        const int rr = rt * 128 + quad * 32 + lane;   // row of the unit
        uint32_t sc = 0, oc = 0, pv = 0;   // sc: parities, a bit each
        bool dead = false;
        const float sc2 = a.softcap > 0.f ? 1.f : a.scale * kLog2e;
        const bool wide = AttnCap(a.scale, a.softcap).wide;
        for (; !w.done(); advance()) {
            const int nt = w.tb() - w.ta();
            const int rows = min(M, w.s.n * a.group - w.rt * M);
            float m = -INFINITY, l = 0.f;
            if (rt * 128 < rows) {
                // the row's keys, from the first of this CTA's tiles (rows past the
                // end: all, so that they ask for no mask)
                int l0 = 0, h0 = 0x7FFFFFFF;
                if (rr < rows) {
                    attn_keys(a, w.s, a.by_group(w.rt * M + rr), l0, h0);
                    l0 -= (w.t0 + w.ta()) * KT;
                    h0 -= (w.t0 + w.ta()) * KT;
                }
                for (int t = 0; t < nt; ++t, l0 -= KT, h0 -= KT) {
                    const int buf = NROW == 2 ? rt : t & 1;
                    if (!__all_sync(0xffffffffu, at_wait(&bar[TB_SF + buf], (sc >> buf) & 1, a, abort_word))) {
                        dead = true;
                        break;
                    }
                    sc ^= 1u << buf;
                    at_fence_after();
                    const uint32_t ts = tq + C::s_col + buf * 128;
                    const bool cut = __any_sync(0xffffffffu, l0 > 0 || h0 < KT);
                    if (wide)
                        at_cap<KT>(a, ts);
                    uint32_t s[KT];
#pragma unroll
                    for (int c = 0; c < KT; c += 32)
                        at_ld32(ts + c, s + c);
                    at_wait_ld(s);
#pragma unroll
                    for (int c = 32; c < KT; c += 32)
                        at_pin(s + c);
                    if (a.softcap > 0.f && !wide) {
                        const AttnCap cap(a.scale, a.softcap);
#pragma unroll
                        for (int c = 0; c < KT; ++c)
                            s[c] = __float_as_uint(cap.high(__uint_as_float(s[c])));
                    }
                    if (cut) {
#pragma unroll
                        for (int c = 0; c < KT; c += 32) {
                            // of 32 keys the row sees those from lo on and below hi
                            const int lo = min(max(l0 - c, 0), 32), hi = min(max(h0 - c, 0), 32);
                            const uint32_t see = (uint32_t)((1ull << hi) - 1) & ~(uint32_t)((1ull << lo) - 1);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((see >> i) & 1))
                                    s[c + i] = 0xFF800000u;   // -inf
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < KT; c += 2)
                        mx[(c >> 1) & 3] =
                            fmaxf(fmaxf(mx[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                    const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), sc2, -Num16<T>::kLift);
                    if (__any_sync(0xffffffffu, top > m + TC_LAZY || (m == -INFINITY && top > m))) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.f : exp2_approx(m - mn);
                        m = mn;
                        l *= f;
                        if (t > 0) {
                            // O holds the products up to the last tile's
                            if (NROW == 1 &&
                                !__all_sync(0xffffffffu, at_wait(&bar[TB_PV], (pv - 1) & 1, a, abort_word))) {
                                dead = true;
                                break;
                            }
                            at_fence_after();
#pragma unroll 1
                            for (int c = 0; c < a.dim; c += 16)
                                at_scale16(tq + C::o_col + rt * DP + c, f);
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    const float2 k2 = make_float2(sc2, sc2), b2 = make_float2(-base, -base);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < KT; c += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = ffma2(make_float2(__uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1])),
                                             k2, b2);
                            x.x = exp2_approx(x.x);
                            x.y = exp2_approx(x.y);
                            sum[i & 1] = fadd2(sum[i & 1], x);
                            // the weights enter the product in the cache's type (at
                            // most half a step each); their sum stays unrounded
                            p[i] = Num16<T>::down2(x.x, x.y);
                        }
                        at_st16(ts + c / 2, p);
                        if (c + 32 == KT / 2 || c + 32 == KT) {
                            at_wait_st();
                            at_fence_before();
                            mbar_arrive(&bar[(c + 32 == KT ? TB_P2 : TB_PF) + buf]);
                        }
                    }
                    const float2 s2 = fadd2(sum[0], sum[1]);
                    l += s2.x + s2.y;
                    ++pv;
                }
                // the row's maximum and sum for the output, once the last unit's have
                // been read (before its O was given back)
                if (!dead && oc > 0 &&
                    !__all_sync(0xffffffffu, at_wait(&bar[TB_OE + rt], (oc - 1) & 1, a, abort_word)))
                    dead = true;
                if (!dead) {
                    ++oc;
                    ml[rr] = make_float2(m, l);
                    mbar_arrive(&bar[TB_LF + rt]);
                }
            }
            if (dead)
                break;
        }
    }
    __syncthreads();
    if (warp == W_MMA) {
        at_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// Joins the parts of the units that several CTAs shared.  CTA (x, y) takes 32
// rows and 64 columns of the unit that begins in CTA x: a lane a row, a warp 8
// columns, so that reads are whole lines; 8 parts' loads are under way at once.
constexpr int TJ_THREADS = 256, TJ_PARTS = 8;

template <class T, int DP, int M>
__global__ void __launch_bounds__(TJ_THREADS) attn_join_kernel(const AttnArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = (int)blockIdx.y % (M / 32) * 32, r = r0 + lane;
    const int u = ((int)blockIdx.y / (M / 32) * 8 + warp) * 2;   // columns 4u.. of 8
    pdl_wait();
    pdl_trigger();
    const TcShared d = tc_shared<M, DP>(a)[blockIdx.x];
    if (d.c1 == 0 || r0 >= d.rows || u * 4 >= a.dim)
        return;
    const int np = d.c1 - (int)blockIdx.x + 1;
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int k0 = 0; k0 < np; k0 += TJ_PARTS) {
        float mk[TJ_PARTS], lk[TJ_PARTS];
        float4 v[TJ_PARTS][2];
#pragma unroll
        for (int x = 0; x < TJ_PARTS; ++x) {
            const int k = k0 + x;
            const float *p = attn_part<M, DP>(a, blockIdx.x + k, k == 0);
            mk[x] = -INFINITY;
            lk[x] = 0.f;
            v[x][0] = v[x][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < np) {
                mk[x] = __ldcg(p + M * DP + r);
                lk[x] = __ldcg(p + M * DP + M + r);
                v[x][0] = __ldcg(reinterpret_cast<const float4 *>(p + tc_at<M>(u, r)));
                v[x][1] = __ldcg(reinterpret_cast<const float4 *>(p + tc_at<M>(u + 1, r)));
            }
        }
        float top = m;
#pragma unroll
        for (int x = 0; x < TJ_PARTS; ++x)
            top = fmaxf(top, mk[x]);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = exp2_approx(m - base);
        m = top;
        l *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] *= f;
#pragma unroll
        for (int x = 0; x < TJ_PARTS; ++x) {   // in the parts' order
            const float w = exp2_approx(mk[x] - base);
            l += w * lk[x];
            const float *vx = reinterpret_cast<const float *>(v[x]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] += w * vx[i];
        }
    }
    if (r >= d.rows)
        return;
    const int tok = a.by_group(d.row0 + r), hq = d.h * a.group + d.row0 + r - tok * a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = Num16<T>::down2(o[2 * i] * inv, o[2 * i + 1] * inv);
    *reinterpret_cast<uint4 *>(a.out + (d.q0 + tok) * a.o_token + hq * a.o_head + u * 4) =
        make_uint4(out[0], out[1], out[2], out[3]);
    if (u == 0 && a.lse)
        a.lse[(size_t)(d.q0 + tok) * a.heads + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class T, int DP, int NROW>
cudaError_t launch_tc(const AttnArgs &args, const LaunchCfg &c)
{
    using C = TcCfg<DP, NROW>;
    auto kern = attn_tc_kernel<T, DP, NROW>;
    AttnArgs a = args;
    AttnMaps maps = {};
    if (!attn_maps(a, Num16<T>::kExp == 0x7F807F80u, C::KT, &maps, &a.tma, &a.heads_inner))
        a.tma = 0;
    a.tma_q = a.tma != 0 && attn_q_map(a, Num16<T>::kExp == 0x7F807F80u, &maps.q);
    // the register split asks for no more than the block is launched with
    static const int regs = [&]() {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess ? f.numRegs : 0;
    }();
    if (regs * C::THREADS < C::SOFT * C::R_SOFT + 256 * C::R_REST)
        return cudaErrorInvalidConfiguration;
    cudaError_t e = set_smem(kern, C::total);
    if (e != cudaSuccess)
        return e;
    e = launch_ex(kern, dim3(c.num_sms), dim3(C::THREADS), C::total, c, 1, a, maps);
    if (e != cudaSuccess)
        return e;
    return launch_ex(attn_join_kernel<T, DP, C::M>, dim3(c.num_sms, C::M / 32 * (DP / 64)), dim3(TJ_THREADS), 0, c, 1, a);
}

template <class T>
cudaError_t launch_t(const AttnArgs &a, int row_tiles, const LaunchCfg &c)
{
    if (a.dim <= 64)
        return row_tiles == 2 ? launch_tc<T, 64, 2>(a, c) : launch_tc<T, 64, 1>(a, c);
    if (a.dim <= 128)
        return row_tiles == 2 ? launch_tc<T, 128, 2>(a, c) : launch_tc<T, 128, 1>(a, c);
    return launch_tc<T, 256, 1>(a, c);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, bool bf16, int row_tiles, const LaunchCfg &c)
{
    return bf16 ? launch_t<__nv_bfloat16>(a, row_tiles, c) : launch_t<__half>(a, row_tiles, c);
}

}  // namespace qmoe
