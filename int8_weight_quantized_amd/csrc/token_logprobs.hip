// token_logprobs.hip -- log probabilities of given tokens, with the entropy
// and the most likely alternatives of each row of logits.

struct LogprobArgs {
    const void* logits;
    const int64_t* tokens;
    float* logprob;
    float* entropy;
    int64_t* top_ids;
    float* top_logprobs;
    int64_t ld, rows, vocab, top;
    int dtype;
};

// Whole numbers in the order of the values: NaN above all, the two zeros alike.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ __launch_bounds__(256) void token_logprobs_kernel(LogprobArgs a)
{
    __shared__ float rf[256];
    __shared__ double rs[256], rw[256];
    __shared__ unsigned long long rk[256];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    auto at = [&](int64_t i) {
        i += row * a.ld;
        if (a.dtype == CK_OUT_FP32) return static_cast<const float*>(a.logits)[i];
        const uint32_t w = static_cast<const uint16_t*>(a.logits)[i];
        return a.dtype == CK_OUT_FP16 ? widen2<CK_DT_FP16>(w).x : widen2<CK_DT_BF16>(w).x;
    };
    float m = -INFINITY;
    for (int64_t i = tid; i < a.vocab; i += 256) m = fmaxf(m, at(i));
    rf[tid] = m;
    __syncthreads();
    for (int i = 0; i < 256; ++i) m = fmaxf(m, rf[i]);
    double s = 0.0, w = 0.0;
    for (int64_t i = tid; i < a.vocab; i += 256) {
        const float t = at(i) - m, e = expf(t);
        s += e;
        w += e * fmaxf(t, -1e4f);                            // a masked token: 0, not 0 times infinity
    }
    rs[tid] = s;
    rw[tid] = w;
    __syncthreads();
    s = w = 0.0;
    for (int i = 0; i < 256; ++i) s += rs[i], w += rw[i];
    const double logs = log(s);
    if (tid == 0) {
        if (a.logprob) {
            const int64_t t = a.tokens[row];
            a.logprob[row] = t >= 0 && t < a.vocab ? (float)((double)at(t) - (double)m - logs) : NAN;
        }
        if (a.entropy) a.entropy[row] = (float)(logs - w / s);
    }
    unsigned long long last = ~0ull;
    for (int64_t k = 0; k < a.top; ++k) {
        unsigned long long best = 0;
        for (int64_t i = tid; i < a.vocab; i += 256) {
            const unsigned long long key = (unsigned long long)order_key(at(i)) << 32 | (0xffffffffu - (uint32_t)i);
            if (key < last && key > best) best = key;
        }
        __syncthreads();
        rk[tid] = best;
        __syncthreads();
        for (int i = 0; i < 256; ++i) best = max(best, rk[i]);
        last = best;
        if (tid == 0) {
            const int64_t id = 0xffffffffu - (uint32_t)best;
            a.top_ids[row * a.top + k] = id;
            a.top_logprobs[row * a.top + k] = (float)((double)at(id) - (double)m - logs);
        }
    }
}

namespace {

constexpr int64_t kLogprobTop = 64;

}  // namespace

extern "C" int64_t ck_token_logprobs_workspace(int64_t rows, int64_t vocab, int64_t top)
{
    return rows < 0 || vocab < 1 || vocab > 0x7fffffff || top < 0 || top > kLogprobTop || top > vocab ? -1 : 0;
}

extern "C" ck_status ck_token_logprobs(const ck_logprob_args* args, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_logprob_args& p = *args;
    if (p.dtype != CK_OUT_BF16 && p.dtype != CK_OUT_FP16 && p.dtype != CK_OUT_FP32) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.rows < 0 || p.vocab < 1 || p.top < 0) return fail(CK_ERR_INVALID_ARG, "negative size, or no vocabulary");
    if (p.top > p.vocab) return fail(CK_ERR_INVALID_ARG, "top larger than the vocabulary");
    if (p.top > kLogprobTop) return fail(CK_ERR_UNSUPPORTED, "top past %d", (int)kLogprobTop);
    if (p.vocab > 0x7fffffff || p.rows > 0x7fffffff) return fail(CK_ERR_UNSUPPORTED, "rows or vocab past 2^31");
    if (p.rows == 0) return ok();
    if (!p.logits) return fail(CK_ERR_INVALID_ARG, "NULL logits");
    if (!p.tokens != !p.logprob) return fail(CK_ERR_INVALID_ARG, "tokens and logprob go together");
    if (p.top > 0 && (!p.top_ids || !p.top_logprobs)) return fail(CK_ERR_INVALID_ARG, "NULL top_ids or top_logprobs");
    if (p.rows > 1 && p.ld < p.vocab) return fail(CK_ERR_INVALID_ARG, "ld smaller than vocab");
    if (!aligned(p.logits, p.dtype == CK_OUT_FP32 ? 4 : 2) || !aligned(p.tokens, 8) || !aligned(p.top_ids, 8) ||
        !aligned(p.logprob, 4) || !aligned(p.entropy, 4) || !aligned(p.top_logprobs, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned logits, tokens or outputs");
    ck_status s = check_device();
    if (s != CK_OK) return s;
    LogprobArgs a{p.logits, p.tokens, p.logprob, p.entropy, p.top_ids, p.top_logprobs, p.ld, p.rows, p.vocab, p.top, p.dtype};
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&token_logprobs_kernel), (unsigned)p.rows, 256, kargs, stream, "token_logprobs");
    return s == CK_OK ? ok() : s;
}
