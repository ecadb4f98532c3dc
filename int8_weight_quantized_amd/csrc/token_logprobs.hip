// token_logprobs.hip -- log probabilities of given tokens, with the entropy
// and the most likely alternatives of each row of logits.
//
// Mathematics.  For any reference m, with d_j = x_j - m,
//   S = sum_j e^d_j,  W = sum_j e^d_j d_j,  L = m + log S,
//   logprob = x[token] - m - log S,  entropy = log S - W / S.
// m is the running maximum of a lane, raised once for a batch of its logits;
// S and W move to the new one by e^(m - m'), W' = (W + S (m - m')) e^(m - m').
// So the largest logit's own term is 1 exactly, and the sums of lanes, waves
// and chunks are joined in 64 bits: a log probability near zero keeps its
// digits, but for the few terms of the largest's own lane, which are added to 1 in
// fp32 (2^-24 at most for each).  A masked logit has e^d = 0 and d = -inf: d is cut at -10^4 in W.
//
// The alternatives, k of them, cost the pass over the logits nothing: of the
// maxima of 256 lanes (or groups of four) the k-th is a bound that k logits reach, and those that do
// are in lanes whose maximum does, few more than k of them.  The logits of these
// lanes are read again and what reaches the bound is ranked, as 64-bit keys
// (value, then lowest index), each by how many others are larger.  Where too
// many reach it (rows of equal logits, masks that leave fewer than k) the waves
// go through all logits again with a sorted list each.
//
// A block of four waves takes a row, or a chunk of it where there are few rows;
// a second launch joins the chunks.  Where that launch would cost more than the
// chunks save, 16 waves take the row.

struct LogprobArgs {
    const void* logits;
    const int64_t* tokens;
    float* logprob;
    float* entropy;
    int64_t* top_ids;
    float* top_logprobs;
    double2* sums;                       // [rows][splits] (S, W)
    float* refs;                         // [rows][splits] m
    unsigned long long* keys;            // [rows][splits][top]
    int64_t ld, rows;
    int vocab, top, splits;
};

typedef unsigned long long u64;

constexpr int kLogprobBatch = 4;         // 16-byte loads of a lane at a time
constexpr int kLogprobKeys = 1024;       // keys that are ranked by counting

// e^d.  log2(e) as one fp32 number is 1.3e-8 of it too small, which would make every
// term of a row too large by |d| times that, and sums do not average out what all
// terms share (a log probability of -0.2 beside terms of d = -11 was 3e-8 off on
// average, an entropy 2e-7 to 3e-7): the part below it comes along (2048 x 131072
// bf16 logits 113 us with and without it, 1 x 32000 9.75 and 9.6).
__device__ __forceinline__ float exp_of(float d)
{
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269502f, d * 1.925963e-8f));
}

// Whole numbers in the order of the values: NaN above all, the two zeros
// alike; 0 is below every value's.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float order_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);   // NaN: itself
}

__device__ __forceinline__ u64 top_key(float x, uint32_t index) { return (u64)order_key(x) << 32 | ~index; }

__device__ __forceinline__ u64 lane_value(u64 v, int lane)
{
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// A wave's largest keys, descending from lane 0; 0 where there is none.
struct TopList {
    u64 key, last;                       // this lane's; that of lane top - 1

    // Takes every lane's key (0: none) that belongs into the list.
    __device__ __forceinline__ void offer(u64 mine, int top)
    {
        const int lane = threadIdx.x & 63;
        u64 left = __ballot(mine > last);
        while (left) {
            const int from = __builtin_ctzll(left);
            left &= left - 1;
            const u64 k = lane_value(mine, from);
            if (k <= last) continue;
            const int at = __popcll(__ballot(key > k));
            const u64 up = (u64)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(key >> 32), 0x138, 0xf, 0xf, false) << 32 |
                           (uint32_t)__builtin_amdgcn_update_dpp(0, (int)key, 0x138, 0xf, 0xf, false);   // the lane before
            key = lane < at ? key : lane == at ? k : up;
            last = lane_value(key, top - 1);
        }
    }
};

// Sums relative to m, of several lanes together.
struct LogSums {
    double s, w;
    float m;
};

constexpr float kLogLow = -3.402823466e38f;                  // m before any logit: -inf - m is -inf

__device__ __forceinline__ LogSums wave_sums(float m, float s, float w)
{
    float high = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) high = fmaxf(high, __shfl_xor(high, off));
    const float d = fmaxf(m - high, -1e4f), f = exp_of(d);    // 1 exactly where m == high
    double ds = (double)(s * f), dw = (double)((w + s * d) * f);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        ds += __shfl_xor(ds, off);
        dw += __shfl_xor(dw, off);
    }
    return {ds, dw, high};
}

// The wave's 64 sums together, in an order that is always the same.
__device__ __forceinline__ LogSums join_sums(LogSums t)
{
    float high = t.m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) high = fmaxf(high, __shfl_xor(high, off));
    const double d = fmaxf(t.m - high, -1e4f), f = exp_of((float)d);    // 1 exactly where m is the highest
    t.w = (t.w + t.s * d) * f;
    t.s *= f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        t.s += __shfl_xor(t.s, off);
        t.w += __shfl_xor(t.w, off);
    }
    t.m = high;
    return t;
}

template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int64_t i)
{
    if constexpr (DT == CK_OUT_FP32) return static_cast<const float*>(row)[i];
    else return widen2<DT == CK_OUT_FP16 ? CK_DT_FP16 : CK_DT_BF16>(static_cast<const uint16_t*>(row)[i]).x;
}

template <int DT, int E>
__device__ __forceinline__ void widen_logits(const v4i& v, float (&x)[E])
{
    if constexpr (DT == CK_OUT_FP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __int_as_float(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen2<DT == CK_OUT_FP16 ? CK_DT_FP16 : CK_DT_BF16>((uint32_t)v[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// What a row's sums give: the last steps in 64 bits, one rounding.
__device__ __forceinline__ float log_probability(float x, const LogSums& t, double logs)
{
    return (float)((double)x - (double)t.m - logs);
}

// The given token's logit, NaN for a token outside the vocabulary; loaded
// before the row's sums are there.
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobArgs& a, int64_t row)
{
    if (!a.logprob) return 0.0f;
    const int64_t tok = a.tokens[row];
    return tok >= 0 && tok < a.vocab ? logit_at<DT>(a.logits, row * a.ld + tok) : NAN;
}

__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, float x, const LogSums& t, double logs)
{
    if (a.logprob) a.logprob[row] = log_probability(x, t, logs);
    if (a.entropy) a.entropy[row] = (float)(logs - t.w / t.s);
}

__device__ __forceinline__ void write_top(const LogprobArgs& a, int64_t at, u64 key, const LogSums& t, double logs)
{
    a.top_ids[at] = (int64_t)(~(uint32_t)key);
    a.top_logprobs[at] = log_probability(order_value((uint32_t)(key >> 32)), t, logs);
}

// Keys in LDS, in no order, and how many; a 0 follows an odd number.
struct Candidates {
    __attribute__((aligned(16))) u64 keys[kLogprobKeys + 2];
    int count;
    __device__ __forceinline__ void add(u64 key)
    {
        const int at = atomicAdd(&count, 1);
        if (at < kLogprobKeys) keys[at] = key;
    }
    // take(place, key) for the largest `top` of them, by the block's threads.
    template <int T, class Take>
    __device__ __forceinline__ void rank(int top, Take take)
    {
        if (threadIdx.x == 0) keys[count] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += T) {
            const u64 k = keys[i];
            int place = 0;
            for (int j = 0; j < count; j += 2) {
                const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&keys[j]);
                place += (o.x > k) + (o.y > k);
            }
            if (place < top) take(place, k);
        }
    }
};

template <int DT, bool TOP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void token_logprobs_kernel(LogprobArgs a)
{
    constexpr int E = DT == CK_OUT_FP32 ? 4 : 8, B = kLogprobBatch;   // logits of a load, loads of a batch
    constexpr int T = 64 * WAVES;
    __shared__ LogSums sums[WAVES];
    __shared__ Candidates cand;
    __shared__ uint32_t highs[TOP ? 256 : 4];
    __shared__ uint16_t owners[TOP ? T : 4];
    __shared__ int owning;
    __shared__ float bound;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row = blockIdx.x / a.splits;
    const int split = (int)(blockIdx.x - row * a.splits);
    const char* const base = static_cast<const char*>(a.logits) + row * a.ld * (16 / E);
    // The row in whole 16-byte pieces, and the few logits before and after
    // them, one a lane of the first and the last chunk's first waves.
    const int head = min(a.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / (16 / E));
    const int pieces = (a.vocab - head) / E, done = head + pieces * E;
    const v4i* const vec = reinterpret_cast<const v4i*>(base + head * (16 / E));
    const int p0 = (int)((int64_t)pieces * split / a.splits), p1 = (int)((int64_t)pieces * (split + 1) / a.splits);
    int few = -1;                                            // this lane's single logit
    if (split == 0 && tid < head) few = tid;
    if (split == a.splits - 1 && tid >= 64 && tid - 64 < a.vocab - done) few = done + tid - 64;

    float m = kLogLow, s = 0.0f, w = 0.0f, top = -INFINITY;  // top: the largest, -inf too
    bool any = false;
    // One batch: pieces p + T j + tid, n of them left.
    auto take = [&](const v4i (&v)[B], int n) {
        float x[B][E], high = -INFINITY;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            widen_logits<DT, E>(v[j], x[j]);
            if (T * j + tid >= n) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[j][e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) high = fmaxf(high, x[j][e]);
        }
        const float old = m;
        top = fmaxf(top, high);
        m = fmaxf(m, high);
        float s0 = 0.0f, s1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float d0 = x[j][e] - m, d1 = x[j][e + 1] - m;
                const float e0 = exp_of(d0), e1 = exp_of(d1);
                s0 += e0;
                s1 += e1;
                w0 = __builtin_fmaf(e0, fmaxf(d0, -1e4f), w0);
                w1 = __builtin_fmaf(e1, fmaxf(d1, -1e4f), w1);
            }
        const float d = fmaxf(old - m, -1e4f), f = exp_of(d);
        w = __builtin_fmaf(__builtin_fmaf(s, d, w), f, w0 + w1);
        s = __builtin_fmaf(s, f, s0 + s1);
    };
    v4i v[B], next[B];
    auto load = [&](v4i (&to)[B], int p) {
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (p + T * j + tid < p1) to[j] = vec[p + T * j + tid];
    };
    load(v, p0);
    float given = 0.0f;
    if (tid == 0 && a.splits == 1) given = token_logit<DT>(a, row);
    any = p0 + tid < p1;
    for (int p = p0; p < p1; p += T * B) {
        load(next, p + T * B);
        take(v, p1 - p);
#pragma unroll
        for (int j = 0; j < B; ++j) v[j] = next[j];
    }
    if (few >= 0) {
        const float x = logit_at<DT>(base, few), old = m;
        any = true;
        top = fmaxf(top, x);
        m = fmaxf(m, x);
        const float d = fmaxf(old - m, -1e4f), f = exp_of(d);
        const float dx = x - m, e = exp_of(dx);
        w = __builtin_fmaf(__builtin_fmaf(s, d, w), f, e * fmaxf(dx, -1e4f));
        s = __builtin_fmaf(s, f, e);
    }
    const LogSums mine = wave_sums(m, s, w);
    if (lane == 0) sums[wave] = mine;
    if constexpr (TOP) {
        // The bound: what the k-th of the lanes' maxima begins with, found bit by
        // bit by the first wave, as many bits as it takes until k reach it and no
        // more, or as the type has (of fp32 20).  (Lanes without a logit, 0, are among them only in a small chunk,
        // which has few logits: no bound then.)
        uint32_t high = any ? order_key(top) : 0;
        if constexpr (WAVES == 16) {                         // of four lanes together
            high = max(high, (uint32_t)__builtin_amdgcn_mov_dpp((int)high, 0xb1, 0xf, 0xf, false));
            high = max(high, (uint32_t)__builtin_amdgcn_mov_dpp((int)high, 0x4e, 0xf, 0xf, false));
            if (lane % 4 == 0) highs[tid / 4] = high;
        } else {
            highs[tid] = high;
        }
        if (tid == 0) {
            cand.count = 0;
            owning = 0;
        }
        __syncthreads();
        if (wave == 0) {
            const uint32_t h0 = highs[lane], h1 = highs[lane + 64], h2 = highs[lane + 128], h3 = highs[lane + 192];
            uint32_t reach = 0;
            for (uint32_t bit = 0x80000000u; bit >= (DT == CK_OUT_BF16 ? 0x10000u : 0x1000u); bit >>= 1) {
                const uint32_t t = reach | bit;
                const int n = __popcll(__ballot(h0 >= t)) + __popcll(__ballot(h1 >= t)) + __popcll(__ballot(h2 >= t)) + __popcll(__ballot(h3 >= t));
                if (n < a.top) continue;
                reach = t;
                if (n == a.top) break;
            }
            if (lane == 0) bound = reach >= 0x00800000u ? order_value(reach) : -INFINITY;
        }
        __syncthreads();
        const float least = bound;
        if (any && top >= least) owners[atomicAdd(&owning, 1)] = (uint16_t)tid;
        __syncthreads();
        // The logits of the lanes that reach it.
        const int rounds = (p1 - p0 + T - 1) / T, total = owning * rounds;
        for (int q = tid; q < total; q += T) {
            const int i = q / owning, p = p0 + T * i + owners[q - i * owning];
            if (p >= p1) continue;
            float x[E];
            widen_logits<DT, E>(vec[p], x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] >= least) cand.add(top_key(x[e], (uint32_t)(head + p * E + e)));
        }
        if (few >= 0) {
            const float x = logit_at<DT>(base, few);
            if (x >= least) cand.add(top_key(x, (uint32_t)few));
        }
        // Too many, or a NaN (which maxima pass over; +inf makes a sum one too).
        bool nan = false;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) nan |= sums[i].s != sums[i].s;
        __syncthreads();
        if (cand.count > kLogprobKeys || nan) {
            TopList list{0, 0};
            if (__any(few >= 0)) list.offer(few >= 0 ? top_key(logit_at<DT>(base, few), (uint32_t)few) : 0, a.top);
            for (int p = p0 + 64 * wave; p < p1; p += T) {
                float x[E];
                if (p + lane < p1) widen_logits<DT, E>(vec[p + lane], x);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    list.offer(p + lane < p1 ? top_key(x[e], (uint32_t)(head + (p + lane) * E + e)) : 0, a.top);
            }
            __syncthreads();
            if (tid == 0) cand.count = 0;
            __syncthreads();
            if (lane < a.top && list.key) cand.add(list.key);
            __syncthreads();
        }
    } else {
        __syncthreads();
    }
    const LogSums t = join_sums(lane < WAVES ? sums[lane] : LogSums{0.0, 0.0, kLogLow});
    if (WAVES == 4 && a.splits > 1) {
        const int64_t at = row * a.splits + split;
        if (tid == 0) {
            a.sums[at] = make_double2(t.s, t.w);
            a.refs[at] = t.m;
        }
        if constexpr (TOP) {
            if (tid >= cand.count && tid < a.top) a.keys[at * a.top + tid] = 0;
            cand.template rank<T>(a.top, [&](int place, u64 key) { a.keys[at * a.top + place] = key; });
        }
        return;
    }
    const double logs = log(t.s);
    if (tid == 0) write_row(a, row, given, t, logs);
    if constexpr (TOP) {
        cand.template rank<T>(a.top, [&](int place, u64 key) { write_top(a, row * a.top + place, key, t, logs); });
    }
}

// Joins a row's chunks, at most 64: their sums in a fixed order, and their
// lists, of which only what reaches every chunk's last can be among the row's.
template <int DT>
__global__ __launch_bounds__(256) void token_logprobs_join_kernel(LogprobArgs a)
{
    __shared__ Candidates cand;
    __shared__ u64 least;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    LogSums t{0.0, 0.0, kLogLow};
    float given = 0.0f;
    if (tid == 0) given = token_logit<DT>(a, row);
    if (lane < a.splits) {
        const double2 v = a.sums[row * a.splits + lane];
        t = {v.x, v.y, a.refs[row * a.splits + lane]};
    }
    const u64* const keys = a.keys + row * a.splits * a.top;
    if (a.top > 0) {
        if (tid == 0) {
            cand.count = 0;
            least = 1;
        }
        __syncthreads();
        if (tid < a.splits) atomicMax(&least, keys[tid * a.top + a.top - 1]);
        __syncthreads();
        for (int i = tid; i < a.splits * a.top; i += 256)
            if (keys[i] >= least) cand.add(keys[i]);
    }
    t = join_sums(t);
    const double logs = log(t.s);
    if (tid == 0) write_row(a, row, given, t, logs);
    if (a.top == 0) return;
    __syncthreads();
    cand.rank<256>(a.top, [&](int place, u64 key) { write_top(a, row * a.top + place, key, t, logs); });
}

namespace {

constexpr int64_t kLogprobTop = 64;
constexpr int64_t kLogprobWide = 32768;  // logits of a row for one block of 16 waves

struct LogprobPlan {
    int64_t waves, splits, bytes;
    bool fits;                                               // into a launch
};

// Rows of 4097 to 32768 logits, at most one a CU: 16 waves each, one launch (us
// with five alternatives, in bf16, against chunks: 1x32000 9.6 and 10.4, 48x32000
// 10.3 and 11.8, 200x8192 10.5 and 11.6; 1x50000 12.3 and 10.9).  Else chunks of
// a row: as many as give every CU two blocks, of 4096 logits at least, and so
// few that their lists can be ranked by counting.
LogprobPlan logprob_plan(int64_t rows, int64_t vocab, int64_t top)
{
    LogprobPlan p{4, 1, 0, false};
    if (rows <= kNumCUs && vocab > 4096 && vocab <= kLogprobWide) p.waves = 16;
    else if (rows > 0) p.splits = std::min(std::min<int64_t>(2 * kNumCUs / rows, cdiv(vocab, 4096)), kLogprobKeys / std::max<int64_t>(top, 16));
    p.splits = std::max<int64_t>(p.splits, 1);
    if (p.splits > 1) p.bytes = rows * p.splits * (16 + 8 * top + 4);
    p.fits = grid_ok(rows, p.splits * p.waves * 64);
    return p;
}

template <int DT>
const void* logprob_fn(bool top, bool wide)
{
    return wide ? top ? reinterpret_cast<const void*>(&token_logprobs_kernel<DT, true, 16>)
                      : reinterpret_cast<const void*>(&token_logprobs_kernel<DT, false, 16>)
           : top ? reinterpret_cast<const void*>(&token_logprobs_kernel<DT, true, 4>)
                 : reinterpret_cast<const void*>(&token_logprobs_kernel<DT, false, 4>);
}

}  // namespace

extern "C" int64_t ck_token_logprobs_workspace(int64_t rows, int64_t vocab, int64_t top)
{
    if (rows < 0 || vocab < 1 || vocab > 0x7fffffff || top < 0 || top > kLogprobTop || top > vocab) return -1;
    const LogprobPlan plan = logprob_plan(rows, vocab, top);
    return plan.fits ? plan.bytes : -1;
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
    const LogprobPlan plan = logprob_plan(p.rows, p.vocab, p.top);
    if (!plan.fits) return fail(CK_ERR_UNSUPPORTED, "too many rows");
    if (plan.bytes > 0 && (!p.workspace || p.workspace_bytes < plan.bytes))
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)plan.bytes);
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    ck_status s = check_device();
    if (s != CK_OK) return s;
    LogprobArgs a{p.logits, p.tokens, p.logprob, p.entropy, p.top_ids, p.top_logprobs, (double2*)p.workspace, nullptr, nullptr,
                  p.ld, p.rows, (int)p.vocab, (int)p.top, (int)plan.splits};
    a.keys = (unsigned long long*)(a.sums + p.rows * plan.splits);
    a.refs = (float*)(a.keys + p.rows * plan.splits * p.top);
    const bool top = p.top > 0, wide = plan.waves == 16;
    const void* const fn = p.dtype == CK_OUT_FP32   ? logprob_fn<CK_OUT_FP32>(top, wide)
                           : p.dtype == CK_OUT_FP16 ? logprob_fn<CK_OUT_FP16>(top, wide)
                                                    : logprob_fn<CK_OUT_BF16>(top, wide);
    const void* const join = p.dtype == CK_OUT_FP32   ? reinterpret_cast<const void*>(&token_logprobs_join_kernel<CK_OUT_FP32>)
                             : p.dtype == CK_OUT_FP16 ? reinterpret_cast<const void*>(&token_logprobs_join_kernel<CK_OUT_FP16>)
                                                      : reinterpret_cast<const void*>(&token_logprobs_join_kernel<CK_OUT_BF16>);
    void* kargs[] = {&a};
    if ((s = launch(fn, (unsigned)(p.rows * plan.splits), (unsigned)plan.waves * 64, kargs, stream, "token_logprobs")) != CK_OK) return s;
    if (plan.splits > 1 && (s = launch(join, (unsigned)p.rows, 256, kargs, stream, "token_logprobs_join")) != CK_OK) return s;
    return ok();
}
