// logits.cu -- penalties for repeated tokens, biases and a grammar mask on the
// rows of a vocabulary projection.
//
//   x = logits[r][v];  seen: v in the row's history;  n: how often it stands
//   behind the prompt
//   seen:  x = x > 0 ? x / rep : x * rep
//   x -= frequency * n + presence * [n > 0]
//   x += sum of the row's bias entries with id v, in their order
//   mask bit v clear: x = -inf
//
// Memory bound: the row is read once and written once (in place if asked),
// everything else is small.  A CTA takes a slice of a row: its logits are on
// their way to registers, 16 bytes a load, while the slice's part of the
// history is counted into one 32-bit word per token in shared memory (the
// count n, a "seen" bit and the number of the token's first bias entry).  The
// slice is written, masked, and then its tokens that have a word once more:
// whoever takes the word out (an exchange with zero) writes the token -- few
// threads with a token each, where a look at every word by the thread that
// holds the logit sends whole warps through the rules for one lane (109 us
// instead of 93 for this kernel alone on the case below).  A token that no rule
// touches leaves as the bits it came.  Counting is integer, so the order of the
// atomics does not show.
// A short history is looked through by every slice.  Where that is much work
// (launch_tile) it is first sorted by ranges of slices, in a kernel of a CTA
// per row that the slices' kernel overlaps (its logits do not wait for it).
// Measured, 256 x 262144 bf16 with histories of up to 12000 tokens, a mask: 86
// us (44 without a history, which is 6.4 TB/s), of which the sort is the first
// 15; then a slice's chain of loads (its range, its tokens, their logits) takes
// 5 us, and 5 CTAs fit on an SM.  There the looking through unsorted histories
// took 112 us, a full sort by slice 106 us; tokens counted in hash tables and
// written by a second kernel 87 us, but 7.6 us instead of 4.2 for one short
// row; a cluster's CTAs counting into one another's words 238 us (texts repeat
// a few tokens, whose words all lie in one CTA); slices taken through shared
// memory by bulk copies 128 us.  48 x 151937 fp32 with everything on: 21 us.
#include <algorithm>

#include "attn.cuh"

namespace qmoe {
namespace {

constexpr uint32_t LG_SEEN = 1u << 31;
constexpr int LG_BIAS_SHIFT = 20;             // 11 bits: 1 + index of the first entry with this id
constexpr uint32_t LG_COUNT = (1u << LG_BIAS_SHIFT) - 1;
constexpr int LG_THREADS = 256;
constexpr int LG_RANGES = 8;                  // ranges of slices that a history is sorted by
constexpr int LG_SORT = 512;                  // threads of the sort: two CTAs on an SM

template <class T>
struct Elem;
template <>
struct Elem<float> {
    using raw = float;
    static constexpr uint32_t none = 0xFF800000u;   // -inf, in every element of a word
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct Elem<__half> : Num16<__half> {
    using raw = uint16_t;
    static constexpr uint32_t none = 0xFC00FC00u;
};
template <>
struct Elem<__nv_bfloat16> : Num16<__nv_bfloat16> {
    using raw = uint16_t;
    static constexpr uint32_t none = 0xFF80FF80u;
};

// places that a row begins behind a 16-byte boundary
template <class R>
__device__ __forceinline__ int row_shift(const LogitsArgs &a, int row)
{
    return (int)((reinterpret_cast<uintptr_t>(static_cast<const R *>(a.in) + row * a.in_stride) % 16) / sizeof(R));
}

// -------------------------------------------------------------------- sort --
// CTA per row: a.sorted[row][..] the row's valid tokens by range of `per`
// slices (the sign bit: behind the prompt), a.begin[row][r] where range r's
// begin.  So each slice looks through its own range's tokens; 8 ranges leave
// at most an eighth more of them than a sort by slice, which costs more than
// that.  Counting sort, LG_CHUNK tokens at a time: a thread's counts of the 8
// ranges are 16-bit fields of two words, scanned over the CTA, after which it
// knows its tokens' places; they go there in shared memory and from there to
// the row in order.
constexpr int LG_KEEP = 24, LG_CHUNK = LG_KEEP * LG_SORT;   // tokens a thread, and at a time
static_assert(LG_RANGES == 8 && LG_CHUNK < 65536, "fields");

template <class T>
__global__ void __launch_bounds__(LG_SORT, 2) logits_sort_kernel(const LogitsArgs a, const FastDiv by_range)
{
    using R = typename Elem<T>::raw;
    extern __shared__ __align__(16) int placed[];   // [LG_CHUNK]
    __shared__ unsigned long long warps[LG_SORT / 32][2], all[2];
    __shared__ int place[LG_RANGES];   // where the ranges' next tokens go
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();   // after the wait: the next kernel reads the logits at once
    const int n = min(max(a.history_len[row], 0), a.max_history);
    const int p = a.prompt_len ? a.prompt_len[row] : 0;
    const int32_t *h = a.history + row * a.history_stride;
    int *out = a.sorted + (size_t)row * a.max_history;
    const int shift = row_shift<R>(a, row);
    int id[LG_KEEP];
    unsigned long long c[2];
    auto field = [](const unsigned long long *f, int r) { return (int)((r < 4 ? f[0] : f[1]) >> (16 * (r & 3)) & 0xFFFF); };
    auto range = [&](int id) { return (int)by_range((uint32_t)(id + shift)); };
    auto count = [&](int i0) {   // tokens i0.. of the row: ids (-1: none) and this thread's counts
        c[0] = c[1] = 0;
#pragma unroll
        for (int k = 0; k < LG_KEEP; ++k)
            id[k] = i0 + k * LG_SORT + tid < n ? __ldg(h + i0 + k * LG_SORT + tid) : -1;
#pragma unroll
        for (int k = 0; k < LG_KEEP; ++k) {
            if ((unsigned)id[k] >= (unsigned)a.vocab) {
                if (id[k] != -1)
                    flag_status(a.status, QMOE_DEV_BAD_TOKEN);
                id[k] = -1;
                continue;
            }
            const int r = range(id[k]);
            c[0] += r < 4 ? 1ull << (16 * r) : 0;
            c[1] += r < 4 ? 0 : 1ull << (16 * (r - 4));
        }
    };
    // counts of the threads before this one; `all`: of the chunk
    auto scan = [&]() {
        unsigned long long s[2] = {c[0], c[1]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const unsigned long long u = __shfl_up_sync(0xffffffffu, s[x], o);
                s[x] += lane >= o ? u : 0;
            }
        if (lane == 31) {
            warps[warp][0] = s[0];
            warps[warp][1] = s[1];
        }
        __syncthreads();
        if (warp < 2) {   // a word each
            const unsigned long long mine = lane < LG_SORT / 32 ? warps[lane][warp] : 0;
            unsigned long long t = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long u = __shfl_up_sync(0xffffffffu, t, o);
                t += lane >= o ? u : 0;
            }
            if (lane < LG_SORT / 32)
                warps[lane][warp] = t - mine;
            if (lane == 31)
                all[warp] = t;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x)
            c[x] = s[x] - c[x] + warps[warp][x];
    };
    if (tid < LG_RANGES)
        place[tid] = 0;
    if (n > LG_CHUNK) {   // the ranges' sizes first
        for (int i0 = 0; i0 < n; i0 += LG_CHUNK) {
            count(i0);
            scan();
            if (tid < LG_RANGES)
                place[tid] += field(all, tid);
        }
        __syncthreads();
    }
    for (int i0 = 0; i0 == 0 || i0 < n; i0 += LG_CHUNK) {
        count(i0);
        scan();
        if (i0 == 0) {
            if (tid == 0) {
                int sum = 0;
                for (int r = 0; r < LG_RANGES; ++r) {
                    const int size = n > LG_CHUNK ? place[r] : field(all, r);
                    a.begin[(size_t)row * (LG_RANGES + 1) + r] = place[r] = sum;
                    sum += size;
                }
                a.begin[(size_t)row * (LG_RANGES + 1) + LG_RANGES] = sum;
            }
        }
        int first[LG_RANGES + 1];   // of the ranges, in the chunk
        first[0] = 0;
#pragma unroll
        for (int r = 0; r < LG_RANGES; ++r)
            first[r + 1] = first[r] + field(all, r);
        // this thread's next places in the chunk: the fields' sums fit 16 bits
#pragma unroll
        for (int r = 0; r < LG_RANGES; ++r)
            c[r >> 2] += (unsigned long long)first[r] << (16 * (r & 3));
#pragma unroll
        for (int k = 0; k < LG_KEEP; ++k)
            if (id[k] >= 0) {
                const int r = range(id[k]);
                placed[field(c, r)] = i0 + k * LG_SORT + tid >= p ? id[k] | (int)0x80000000 : id[k];
                c[0] += r < 4 ? 1ull << (16 * r) : 0;
                c[1] += r < 4 ? 0 : 1ull << (16 * (r - 4));
            }
        __syncthreads();
        for (int i = tid; i < first[LG_RANGES]; i += LG_SORT) {
            int at = i;
            if (n > LG_CHUNK) {
                int r = 0;
#pragma unroll
                for (int x = 1; x < LG_RANGES; ++x)
                    r += i >= first[x];
                int f = 0;
#pragma unroll
                for (int x = 1; x < LG_RANGES; ++x)
                    f = r == x ? first[x] : f;
                at = place[r] + i - f;
            }
            out[at] = placed[i];
        }
        if (n > LG_CHUNK) {
            __syncthreads();
            if (tid < LG_RANGES)
                place[tid] += field(all, tid);
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ slices --
// bit 7 of lo in every bit of the lower half, bit 15 of hi in every one of the upper
__device__ __forceinline__ uint32_t halves(uint32_t lo, uint32_t hi)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, 0xDD88;" : "=r"(d) : "r"(lo), "r"(hi));
    return d;
}

// CTA (row, t): TILE places of the row; slices later than rows in the grid's
// order, because a text's tokens crowd in the first slices and those should
// not come last.  WORDS: there is a history or a bias;
// SORTED: the history has been sorted.
template <class T, int TILE, bool WORDS, bool SORTED, bool MASK>
__global__ void __launch_bounds__(LG_THREADS, 5) logits_kernel(const LogitsArgs a, int per)
{
    using R = typename Elem<T>::raw;
    constexpr int NT = LG_THREADS;
    constexpr int E = 16 / (int)sizeof(R);   // elements of a 16-byte unit
    constexpr int NV = TILE / (E * NT);
    extern __shared__ __align__(16) uint32_t lsm[];
    uint32_t *word = lsm;                                        // [TILE]
    int *bid = reinterpret_cast<int *>(lsm + TILE);              // [max_bias]
    float *bval = reinterpret_cast<float *>(bid + a.max_bias);   // [max_bias]
    float *bsum = bval + a.max_bias;                             // [max_bias]
    const int row = blockIdx.x, slice = blockIdx.y, tid = threadIdx.x;
    const R *in = static_cast<const R *>(a.in) + row * a.in_stride;
    R *out = static_cast<R *>(a.out) + row * a.out_stride;
    const uint32_t *mask = MASK ? a.mask + row * a.mask_stride : nullptr;
    const int shift = row_shift<R>(a, row), v0 = slice * TILE - shift;
    if (v0 >= a.vocab)
        return;
    const bool vec_out = reinterpret_cast<uintptr_t>(out - shift) % 16 == 0;
    if (!SORTED) {   // with a sort before, that has waited
        pdl_wait();
        pdl_trigger();
    }
    union Vec {
        uint4 q;
        uint32_t w[4];
        R e[E];
    };
    Vec x[NV];
    uint32_t bits[NV];   // the mask word of each unit's first token
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = v0 + (k * NT + tid) * E;
        if (v >= 0 && v + E <= a.vocab) {
            x[k].q = *reinterpret_cast<const uint4 *>(in + v);
            if (MASK)
                bits[k] = __ldg(mask + (v >> 5));
        } else if (v + E > 0 && v < a.vocab) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (v + i >= 0 && v + i < a.vocab)
                    x[k].e[i] = in[v + i];
        }
    }
    // the tokens to look through, [begin, end) of ids; a thread's first four
    // stay in registers between the two times
    constexpr int KEEP = 4;
    const int32_t *ids = nullptr;
    int begin = 0, end = 0, p = 0, kept[KEEP];
    if (WORDS) {
#pragma unroll
        for (int k = 0; k < TILE / (4 * NT); ++k)
            reinterpret_cast<uint4 *>(word)[k * NT + tid] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < a.max_bias; i += NT) {
            bid[i] = a.bias_ids[(size_t)row * a.max_bias + i];
            bval[i] = a.bias[(size_t)row * a.max_bias + i];
        }
        __syncthreads();
        if (SORTED) {
            pdl_wait();   // the history has been sorted
            const int *b = a.begin + (size_t)row * (LG_RANGES + 1) + slice / per;
            begin = __ldcg(b);
            end = __ldcg(b + 1);
            ids = a.sorted + (size_t)row * a.max_history;
        } else if (a.history) {
            end = min(max(a.history_len[row], 0), a.max_history);
            p = a.prompt_len ? a.prompt_len[row] : 0;
            ids = a.history + row * a.history_stride;
        }
        auto count = [&](int i, int id) {
            const bool made = SORTED ? id < 0 : i >= p;
            const int token = SORTED ? id & 0x7FFFFFFF : id;
            const unsigned u = (unsigned)(token - v0);
            if (!SORTED && (unsigned)id >= (unsigned)a.vocab) {
                if (id != -1 && slice == 0)
                    flag_status(a.status, QMOE_DEV_BAD_TOKEN);
            } else if (u < (unsigned)TILE) {
                if (made)
                    atomicAdd(word + u, 1u);   // a count says "seen" too
                else
                    atomicOr(word + u, LG_SEEN);
            }
        };
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            kept[k] = begin + k * NT + tid < end ? __ldcg(ids + begin + k * NT + tid) : -1;
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int i = begin + k * NT + tid;
            if (i < end)
                count(i, kept[k]);
        }
        for (int i0 = begin + KEEP * NT + tid; i0 < end; i0 += 8 * NT) {
            int id[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                id[k] = i0 + k * NT < end ? __ldcg(ids + i0 + k * NT) : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + k * NT < end)
                    count(i0 + k * NT, id[k]);
        }
        for (int i = tid; i < a.max_bias; i += NT) {
            const int id = bid[i];
            const unsigned u = (unsigned)(id - v0);
            if ((unsigned)id >= (unsigned)a.vocab) {
                if (id != -1 && slice == 0)
                    flag_status(a.status, QMOE_DEV_BAD_TOKEN);
            } else if (u < (unsigned)TILE) {
                // an id's entries add up, in their order, at its first one
                float sum = 0.f;
                bool first = true;
#pragma unroll 8
                for (int k = 0; k < a.max_bias; ++k) {
                    const bool same = bid[k] == id;
                    first = first && !(same && k < i);
                    if (same)
                        sum += bval[k];
                }
                if (first) {
                    bsum[i] = sum;
                    atomicOr(word + u, (uint32_t)(i + 1) << LG_BIAS_SHIFT);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = v0 + (k * NT + tid) * E;
        if (v >= 0 && v + E <= a.vocab) {
            if (MASK) {
                uint32_t m = bits[k] >> (v & 31);
                if ((v & 31) > 32 - E)   // the unit goes on in the next word
                    m |= __ldg(mask + (v >> 5) + 1) << (32 - (v & 31));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // an element's bit becomes a mask of its width
                    const uint32_t keep = E == 4 ? 0u - ((m >> j) & 1u) : halves(m << (7 - 2 * j), m << (14 - 2 * j));
                    x[k].w[j] = (x[k].w[j] & keep) | (Elem<T>::none & ~keep);
                }
            }
            if (vec_out) {
                __stcs(reinterpret_cast<uint4 *>(out + v), x[k].q);
            } else {   // the output begins elsewhere within 16 bytes than the input
#pragma unroll
                for (int i = 0; i < E; ++i)
                    out[v + i] = x[k].e[i];
            }
        } else if (v + E > 0 && v < a.vocab) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (v + i >= 0 && v + i < a.vocab)
                    out[v + i] = MASK && !((mask[(v + i) >> 5] >> ((v + i) & 31)) & 1u) ? Elem<T>::down(-INFINITY) : x[k].e[i];
        }
    }
    if (!WORDS)
        return;
    const float rep = a.repetition ? a.repetition[row] : 1.f;
    const float pres = a.presence ? a.presence[row] : 0.f;
    const float freq = a.frequency ? a.frequency[row] : 0.f;
    __syncthreads();   // the counts are complete, the slice is written
    // Whoever takes a token's word out writes the token, four at a time so that
    // their logits come together (what the mask let through has its old value,
    // in place too).
    auto settle = [&](const int *id) {
        uint32_t w[KEEP], m[KEEP];
        R y[KEEP];
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const unsigned u = (unsigned)(id[k] - v0);
            w[k] = 0;
            if ((unsigned)id[k] < (unsigned)a.vocab && u < (unsigned)TILE &&
                *const_cast<volatile uint32_t *>(word + u) != 0)
                w[k] = atomicExch(word + u, 0u);
        }
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (w[k]) {
                y[k] = in[id[k]];
                m[k] = MASK ? __ldg(mask + (id[k] >> 5)) >> (id[k] & 31) : 1u;
            }
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (w[k] && (m[k] & 1u)) {
                float v = Elem<T>::up(y[k]);
                const uint32_t c = w[k] & LG_COUNT, b = (w[k] & ~LG_SEEN) >> LG_BIAS_SHIFT;
                if (c || (w[k] & LG_SEEN))
                    v = v > 0.f ? v / rep : v * rep;
                if (c)
                    v = v - freq * (float)c - pres;
                if (b)
                    v += bsum[b - 1];
                out[id[k]] = Elem<T>::down(v);
            }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        kept[k] = begin + k * NT + tid < end ? (SORTED ? kept[k] & 0x7FFFFFFF : kept[k]) : -1;
    settle(kept);
    for (int i0 = begin + KEEP * NT + tid; i0 < end; i0 += KEEP * NT) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int id = i0 + k * NT < end ? __ldcg(ids + i0 + k * NT) : -1;
            kept[k] = SORTED && i0 + k * NT < end ? id & 0x7FFFFFFF : id;
        }
        settle(kept);
    }
    for (int i0 = tid; i0 < a.max_bias; i0 += KEEP * NT) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            kept[k] = i0 + k * NT < a.max_bias ? bid[i0 + k * NT] : -1;
        settle(kept);
    }
}

template <class T, int TILE>
cudaError_t launch_tile(const LogitsArgs &a, const LaunchCfg &c)
{
    using R = typename Elem<T>::raw;
    const int slices = (int)((a.vocab + 16 / (long long)sizeof(R) - 1 + TILE - 1) / TILE);
    const dim3 grid(a.rows, slices);
    if (a.max_history == 0 && a.max_bias == 0)
        return a.mask ? launch_ex(logits_kernel<T, TILE, false, false, true>, grid, dim3(LG_THREADS), 0, c, 1, a, 1)
                      : launch_ex(logits_kernel<T, TILE, false, false, false>, grid, dim3(LG_THREADS), 0, c, 1, a, 1);
    const size_t smem = TILE * 4 + (size_t)a.max_bias * 12;
    const int per = (slices + LG_RANGES - 1) / LG_RANGES;
    static_assert(TILE * 4 + kMaxLogitBias * 12 <= 48 * 1024, "shared memory without asking for more");
    auto go = [&](auto kern) { return launch_ex(kern, grid, dim3(LG_THREADS), smem, c, 1, a, per); };
    // Looking through a history takes each slice its length.  Measured (fp16),
    // looking through unsorted and sorted histories: 256 rows of
    // 262144 with 1024 tokens 51 and 55 us, 2048 66 and 61, 4096 92 and 68, 8192
    // 149 and 82; 48 of 151937 with 8192 27 and 25 (fp32, twice the slices, 4096:
    // 23 and 21 with biases and a mask); one of 32000 with 4096 10 and 15, 8192
    // 17 and 23.
    if (a.max_history <= kLogitsUnsorted || (long long)a.rows * slices * a.max_history < 7000000)
        return a.mask ? go(logits_kernel<T, TILE, true, false, true>) : go(logits_kernel<T, TILE, true, false, false>);
    constexpr size_t chunk = LG_CHUNK * 4;
    cudaError_t e = set_smem(logits_sort_kernel<T>, chunk);
    if (e == cudaSuccess)
        e = launch_ex(logits_sort_kernel<T>, dim3(a.rows), dim3(LG_SORT), chunk, c, 1, a, FastDiv((uint32_t)(TILE * per)));
    if (e != cudaSuccess)
        return e;
    return a.mask ? go(logits_kernel<T, TILE, true, true, true>) : go(logits_kernel<T, TILE, true, true, false>);
}

template <class T>
cudaError_t launch_t(const LogitsArgs &a, const LaunchCfg &c)
{
    // slices of 16 KB, unless that would leave SMs without one
    constexpr int TILE = 16384 / (int)sizeof(typename Elem<T>::raw);
    if ((long long)a.rows * ((a.vocab + TILE - 1) / TILE) >= 2 * c.num_sms)
        return launch_tile<T, TILE>(a, c);
    return launch_tile<T, 2048>(a, c);
}

}  // namespace

size_t logits_workspace_bytes(int rows, int max_history)
{
    if (max_history <= kLogitsUnsorted)
        return 0;
    return align_up((size_t)rows * (LG_RANGES + 1) * 4, 16) + (size_t)rows * max_history * 4;
}

cudaError_t launch_logits(const LogitsArgs &args, int dtype, void *ws, const LaunchCfg &c)
{
    LogitsArgs a = args;
    a.begin = static_cast<int *>(ws);
    a.sorted = reinterpret_cast<int *>(static_cast<char *>(ws) + align_up((size_t)a.rows * (LG_RANGES + 1) * 4, 16));
    return dtype == QMOE_F32 ? launch_t<float>(a, c)
           : dtype == QMOE_BF16 ? launch_t<__nv_bfloat16>(a, c) : launch_t<__half>(a, c);
}

}  // namespace qmoe
