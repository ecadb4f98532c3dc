// paged_attention.hip -- attention of one new token per sequence over a
// paged key/value cache, split over the cache's length and joined.

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    const int32_t* table;
    const int32_t* lens;
    float* part;                         // [batch, hq, splits, 2 + d]: max, sum, weighted values
    const uint8_t* ck;
    const uint8_t* cv;
    const float* cks;
    const float* cvs;
    int64_t q_bs, q_hs, o_bs, o_hs, table_stride, c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int64_t pages, capacity;             // capacity: tokens a table row can name
    int64_t window, sinks;
    float scale;
    int hq, group, d, page_shift, splits, chunk;
};

// The visible tokens of a sequence, counted from 0: the first `head` are
// tokens 0 .. head - 1, the others follow from token `gap` + index on.
struct Visible {
    int64_t count, head, gap;
    __device__ __forceinline__ int64_t token(int64_t i) const { return i < head ? i : i + gap; }
};

__device__ __forceinline__ Visible visible(const AttnArgs& a, int64_t len)
{
    const int64_t n = min(max(len, (int64_t)0), a.capacity);
    if (a.window <= 0 || n <= a.window) return {n, n, 0};
    const int64_t lo = n - a.window, head = min(a.sinks, lo);
    return {head + a.window, head, lo - head};
}

// One block per sequence, query head and chunk of 256 visible tokens: a
// thread scores one token, the block takes the maximum and the sum, and then
// a thread sums one element of the values.
template <int DT, bool I8>
__global__ __launch_bounds__(256) void attention_simple_kernel(AttnArgs a)
{
    __shared__ float qs[256], ps[256], red[4];
    __shared__ int64_t rows[256];
    const int split = blockIdx.x % a.splits;
    const int64_t bh = blockIdx.x / a.splits;
    const int h = (int)(bh % a.hq);
    const int64_t b = bh / a.hq;
    const int kvh = h / a.group, tid = threadIdx.x;
    const Visible vis = visible(a, a.lens[b]);
    float* part = a.part + (bh * a.splits + split) * (2 + a.d);
    const int64_t first = (int64_t)split * 256;
    const int n = (int)min<int64_t>(256, vis.count - first);
    if (n <= 0) {
        if (tid == 0) { part[0] = -INFINITY; part[1] = 0.0f; }
        return;
    }
    if (tid < a.d) qs[tid] = widen2<DT>(a.q[b * a.q_bs + h * a.q_hs + tid]).x * a.scale;
    __syncthreads();
    float score = -INFINITY;
    if (tid < n) {
        const int64_t tok = vis.token(first + tid);
        const int64_t page = a.table[b * a.table_stride + (tok >> a.page_shift)];
        const int64_t at = tok & ((1 << a.page_shift) - 1);
        const bool bad = page < 0 || page >= a.pages;
        rows[tid] = bad ? -1 : page * a.c_ps + kvh * a.c_hs + at * a.c_ts;
        score = NAN;
        if (!bad) {
            float sum = 0.0f;
            for (int i = 0; i < a.d; ++i) {
                const float kv = I8 ? (float)(int8_t)a.ck[rows[tid] + i]
                                    : widen2<DT>(reinterpret_cast<const uint16_t*>(a.ck)[rows[tid] + i]).x;
                sum = __builtin_fmaf(qs[i], kv, sum);
            }
            score = I8 ? sum * a.cks[page * a.s_ps + kvh * a.s_hs + at * a.s_ts] : sum;
        }
    }
    float m = score;
    for (int off = 32; off > 0; off >>= 1) {
        const float o = __shfl_xor(m, off);
        m = m != m || o != o ? NAN : fmaxf(m, o);
    }
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = red[0];
    for (int i = 1; i < 4; ++i) m = m != m || red[i] != red[i] ? NAN : fmaxf(m, red[i]);
    float p = tid < n ? expf(score - m) : 0.0f;
    float sum = p;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    if (I8 && tid < n && rows[tid] >= 0) {
        const int64_t tok = vis.token(first + tid);
        const int64_t page = a.table[b * a.table_stride + (tok >> a.page_shift)];
        p *= a.cvs[page * a.s_ps + kvh * a.s_hs + (tok & ((1 << a.page_shift) - 1)) * a.s_ts];
    }
    ps[tid] = p;
    __syncthreads();
    if (tid == 0) {
        part[0] = m;
        part[1] = red[0] + red[1] + red[2] + red[3];
    }
    if (tid < a.d) {
        float o = 0.0f;
        for (int j = 0; j < n; ++j) {
            if (rows[j] < 0) continue;
            const float vv = I8 ? (float)(int8_t)a.cv[rows[j] + tid]
                                : widen2<DT>(reinterpret_cast<const uint16_t*>(a.cv)[rows[j] + tid]).x;
            o = __builtin_fmaf(ps[j], vv, o);
        }
        part[2 + tid] = o;
    }
}

// Joins the splits of one sequence and head, in their order.
template <int DT>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a)
{
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.hq);
    const int64_t b = bh / a.hq;
    const float* part = a.part + bh * a.splits * (2 + a.d);
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) {
        const float o = part[s * (2 + a.d)];
        m = m != m || o != o ? NAN : fmaxf(m, o);
    }
    if ((int)threadIdx.x >= a.d) return;
    float sum = 0.0f, o = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        const float* p = part + s * (2 + a.d);
        if (p[0] == -INFINITY) continue;           // nothing visible there
        const float f = expf(p[0] - m);
        sum = __builtin_fmaf(f, p[1], sum);
        o = __builtin_fmaf(f, p[2 + threadIdx.x], o);
    }
    const float r = m == -INFINITY ? 0.0f : o / sum;
    a.out[b * a.o_bs + h * a.o_hs + threadIdx.x] = (uint16_t)(narrow2<DT>(r, 0.0f) & 0xffffu);
}

namespace {

bool attention_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// The most tokens that can be visible to any sequence.
int64_t most_visible(int64_t table_width, int64_t page_size, int64_t window, int64_t sinks)
{
    const int64_t cap = table_width * page_size;
    if (window <= 0 || window >= cap) return cap;
    return window + std::min(sinks, cap - window);
}

}  // namespace

extern "C" int64_t ck_paged_attention_workspace(int64_t batch, int64_t hq, int64_t hk, int64_t head_dim,
                                                int64_t table_width, int64_t page_size, int64_t window,
                                                int64_t sinks)
{
    if (batch < 0 || hq < 1 || hk < 1 || hq % hk != 0 || !attention_dim_ok(head_dim) || table_width < 0 ||
        !is_pow2(page_size) || page_size > 32768 || window < 0 || sinks < 0 || batch > (1 << 20) || hq > 65536 ||
        table_width > (int64_t(1) << 31) - 1)
        return -1;
    const int64_t splits = std::max<int64_t>(1, cdiv(most_visible(table_width, page_size, window, sinks), 256));
    return batch * hq * splits * (2 + head_dim) * 4;
}

extern "C" ck_status ck_paged_attention(const ck_attention_args* args, const ck_kv_cache* cache,
                                        hipStream_t stream)
{
    if (!args || !cache) return fail(CK_ERR_INVALID_ARG, "NULL args or cache");
    const ck_attention_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.batch < 0 || p.hq < 0 || p.table_width < 0 || p.window < 0 || p.sinks < 0)
        return fail(CK_ERR_INVALID_ARG, "negative size");
    if (!attention_dim_ok(cache->head_dim)) return fail(CK_ERR_UNSUPPORTED, "head_dim must be 64, 96, 128, 192 or 256");
    ck_status s = check_cache(cache, p.dtype, cache->head_dim, 16);
    if (s != CK_OK) return s;
    if (p.hq % cache->heads != 0) return fail(CK_ERR_INVALID_ARG, "query heads are not a multiple of the cache's");
    if (p.batch == 0 || p.hq == 0) return ok();
    if (p.batch > (1 << 20) || p.hq > 65536 || p.table_width > (int64_t(1) << 31) - 1)
        return fail(CK_ERR_UNSUPPORTED, "too large a batch, table or number of heads");
    if (!p.q || !p.out || !p.lens || (!p.table && p.table_width > 0))
        return fail(CK_ERR_INVALID_ARG, "NULL q, out, table or lens");
    if (!rows16(p.q, p.q_batch_stride, p.q_head_stride) || !rows16(p.out, p.out_batch_stride, p.out_head_stride))
        return fail(CK_ERR_UNSUPPORTED, "q and out rows must start 16 bytes apart");
    if (!aligned(p.table, 4) || !aligned(p.lens, 4)) return fail(CK_ERR_UNSUPPORTED, "misaligned table or lens");
    if (p.table_stride < p.table_width && p.batch > 1) return fail(CK_ERR_INVALID_ARG, "table_stride smaller than table_width");
    if (!(p.scale == p.scale)) return fail(CK_ERR_INVALID_ARG, "scale is NaN");
    const int64_t need = ck_paged_attention_workspace(p.batch, p.hq, cache->heads, cache->head_dim, p.table_width,
                                                      cache->page_size, p.window, p.sinks);
    if (need > 0 && (!p.workspace || p.workspace_bytes < need))
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)need);
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    AttnArgs a{};
    a.splits = (int)std::max<int64_t>(1, cdiv(most_visible(p.table_width, cache->page_size, p.window, p.sinks), 256));
    const int64_t blocks = p.batch * p.hq * a.splits;
    if (blocks > 0x7fffffffLL) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if ((s = check_device()) != CK_OK) return s;
    a.q = (const uint16_t*)p.q; a.out = (uint16_t*)p.out; a.table = p.table; a.lens = p.lens;
    a.part = (float*)p.workspace;
    a.ck = (const uint8_t*)cache->k; a.cv = (const uint8_t*)cache->v; a.cks = cache->k_scale; a.cvs = cache->v_scale;
    a.q_bs = p.q_batch_stride; a.q_hs = p.q_head_stride; a.o_bs = p.out_batch_stride; a.o_hs = p.out_head_stride;
    a.table_stride = p.table_stride;
    a.c_ps = cache->page_stride; a.c_hs = cache->head_stride; a.c_ts = cache->token_stride;
    a.s_ps = cache->scale_page_stride; a.s_hs = cache->scale_head_stride; a.s_ts = cache->scale_token_stride;
    a.pages = cache->pages; a.capacity = p.table_width * cache->page_size;
    a.window = p.window; a.sinks = p.sinks; a.scale = p.scale;
    a.hq = (int)p.hq; a.group = (int)(p.hq / cache->heads); a.d = (int)cache->head_dim;
    a.page_shift = ilog2(cache->page_size);
    const bool i8 = cache->dtype == CK_DT_INT8, f16 = p.dtype == CK_DT_FP16;
    const void* fn = f16 ? (i8 ? reinterpret_cast<const void*>(&attention_simple_kernel<CK_DT_FP16, true>)
                               : reinterpret_cast<const void*>(&attention_simple_kernel<CK_DT_FP16, false>))
                         : (i8 ? reinterpret_cast<const void*>(&attention_simple_kernel<CK_DT_BF16, true>)
                               : reinterpret_cast<const void*>(&attention_simple_kernel<CK_DT_BF16, false>));
    void* kargs[] = {&a};
    if ((s = launch(fn, (unsigned)blocks, 256, kargs, stream, "paged_attention")) != CK_OK) return s;
    const void* join = f16 ? reinterpret_cast<const void*>(&attention_join_kernel<CK_DT_FP16>)
                           : reinterpret_cast<const void*>(&attention_join_kernel<CK_DT_BF16>);
    s = launch(join, (unsigned)(p.batch * p.hq), 256, kargs, stream, "paged_attention_join");
    return s == CK_OK ? ok() : s;
}
