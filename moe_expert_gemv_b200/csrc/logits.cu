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
// everything else is small.  Each CTA owns a slice of the vocabulary and
// keeps one 32-bit word per token of it in shared memory: the count n, a
// "seen" bit and the number of the token's first bias entry; counting is
// integer, so the order of the atomics does not show.
#include "attn.cuh"

namespace qmoe {
namespace {

constexpr int LG_THREADS = 512;
constexpr int LG_TILE = 8192;                 // vocabulary entries per CTA
constexpr uint32_t LG_SEEN = 1u << 31;
constexpr int LG_BIAS_SHIFT = 20;             // 11 bits: 1 + index of the first entry with this id
constexpr uint32_t LG_COUNT = (1u << LG_BIAS_SHIFT) - 1;

template <class T>
struct Elem;
template <>
struct Elem<float> {
    using raw = float;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct Elem<__half> : Num16<__half> {
    using raw = uint16_t;
};
template <>
struct Elem<__nv_bfloat16> : Num16<__nv_bfloat16> {
    using raw = uint16_t;
};

struct RowRule {
    float rep, pres, freq;
};

__device__ __forceinline__ float apply(float x, uint32_t w, const RowRule &r, const float *bsum)
{
    if (w & LG_SEEN)
        x = x > 0.f ? x / r.rep : x * r.rep;
    const uint32_t n = w & LG_COUNT;
    if (n)
        x = x - r.freq * (float)n - r.pres;
    const uint32_t b = (w & ~LG_SEEN) >> LG_BIAS_SHIFT;
    if (b)
        x += bsum[b - 1];
    return x;
}

template <class T>
__global__ void __launch_bounds__(LG_THREADS) logits_kernel(const LogitsArgs a)
{
    extern __shared__ uint32_t lsm[];
    uint32_t *word = lsm;                                        // [LG_TILE]
    int *bid = reinterpret_cast<int *>(lsm + LG_TILE);           // [max_bias]
    float *bval = reinterpret_cast<float *>(bid + a.max_bias);   // [max_bias]
    float *bsum = bval + a.max_bias;                             // [max_bias]
    using R = typename Elem<T>::raw;
    const int row = blockIdx.y, tid = threadIdx.x;
    const int v0 = blockIdx.x * LG_TILE, nv = min(LG_TILE, a.vocab - v0);
    for (int i = tid; i < nv; i += LG_THREADS)
        word[i] = 0;
    for (int i = tid; i < a.max_bias; i += LG_THREADS) {
        bid[i] = a.bias_ids[(size_t)row * a.max_bias + i];
        bval[i] = a.bias[(size_t)row * a.max_bias + i];
    }
    __syncthreads();
    if (a.history) {
        const int n = min(max(a.history_len[row], 0), a.max_history);
        const int p = a.prompt_len ? a.prompt_len[row] : 0;
        const int32_t *h = a.history + row * a.history_stride;
        for (int i = tid; i < n; i += LG_THREADS) {
            const int id = h[i];
            const unsigned u = (unsigned)(id - v0);
            if (u < (unsigned)nv) {
                atomicOr(&word[u], LG_SEEN);
                if (i >= p)
                    atomicAdd(&word[u], 1u);
            } else if (blockIdx.x == 0 && (unsigned)id >= (unsigned)a.vocab && id != -1) {
                flag_status(a.status, QMOE_DEV_BAD_TOKEN);
            }
        }
    }
    for (int i = tid; i < a.max_bias; i += LG_THREADS) {
        const int id = bid[i];
        const unsigned u = (unsigned)(id - v0);
        if (u < (unsigned)nv) {
            float sum = 0.f;
            bool first = true;
            for (int k = 0; k < a.max_bias; ++k)
                if (bid[k] == id) {
                    if (k < i) {
                        first = false;
                        break;
                    }
                    sum += bval[k];
                }
            if (first) {
                bsum[i] = sum;
                atomicOr(&word[u], (uint32_t)(i + 1) << LG_BIAS_SHIFT);
            }
        } else if (blockIdx.x == 0 && (unsigned)id >= (unsigned)a.vocab && id != -1) {
            flag_status(a.status, QMOE_DEV_BAD_TOKEN);
        }
    }
    __syncthreads();
    RowRule r;
    r.rep = a.repetition ? a.repetition[row] : 1.f;
    r.pres = a.presence ? a.presence[row] : 0.f;
    r.freq = a.frequency ? a.frequency[row] : 0.f;
    const R *in = static_cast<const R *>(a.in) + row * a.in_stride + v0;
    R *out = static_cast<R *>(a.out) + row * a.out_stride + v0;
    const uint32_t *mask = a.mask ? a.mask + row * a.mask_stride : nullptr;
    for (int i = tid; i < nv; i += LG_THREADS) {
        float x = apply(Elem<T>::up(in[i]), word[i], r, bsum);
        if (mask && !((mask[(v0 + i) >> 5] >> ((v0 + i) & 31)) & 1u))
            x = -INFINITY;
        out[i] = Elem<T>::down(x);
    }
}

template <class T>
cudaError_t launch_t(const LogitsArgs &a, const LaunchCfg &c)
{
    const size_t smem = LG_TILE * 4 + (size_t)a.max_bias * 12;
    cudaError_t e = set_smem(logits_kernel<T>, LG_TILE * 4 + kMaxLogitBias * 12);
    if (e != cudaSuccess)
        return e;
    LaunchCfg c2 = c;
    c2.pdl = false;
    return launch_ex(logits_kernel<T>, dim3((a.vocab + LG_TILE - 1) / LG_TILE, a.rows), dim3(LG_THREADS), smem,
                     c2, 1, a);
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs &a, int dtype, const LaunchCfg &c)
{
    return dtype == QMOE_F32 ? launch_t<float>(a, c)
           : dtype == QMOE_BF16 ? launch_t<__nv_bfloat16>(a, c) : launch_t<__half>(a, c);
}

}  // namespace qmoe
