// shared_prefix.hip -- attention of one new token per sequence over a paged
// cache, where the sequences of a group begin with the same tokens.

struct PrefixArgs {
    const uint16_t* q;
    uint16_t* out;
    const int32_t* ptable;
    const int32_t* plens;
    const int32_t* starts;
    const int32_t* table;
    const int32_t* lens;
    const uint8_t* ck;
    const uint8_t* cv;
    const float* cks;
    const float* cvs;
    int64_t q_bs, q_hs, o_bs, o_hs, pt_stride, table_stride, c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int64_t pages, pcap, cap;                                // pcap, cap: tokens that a row of ptable, table can name
    float scale;
    int batch, hq, hk, prefixes, page_shift, d, i8, f16;
};

// One block per sequence and query head, 256 threads over the tokens: scores,
// then the weights' sum, then the values.
__global__ __launch_bounds__(256) void shared_prefix_kernel(PrefixArgs a)
{
    __shared__ float red[256], qs[256], acc[256];
    __shared__ int bad;
    const int tid = threadIdx.x, h = blockIdx.x % a.hq;
    const int64_t b = blockIdx.x / a.hq;
    const int kvh = h / (a.hq / a.hk);
    int p = -1, wrong = 0;
    for (int i = 0; i <= a.prefixes && a.prefixes > 0; ++i) {
        const int s = a.starts[i];
        wrong |= s < 0 || s > a.batch || (i > 0 && s < a.starts[i - 1]);
        p += s <= b;
    }
    if (p >= a.prefixes) p = -1;
    const int64_t np = p < 0 ? 0 : min(max((int64_t)a.plens[p], (int64_t)0), a.pcap);
    const int64_t n = np + min(max((int64_t)a.lens[b], (int64_t)0), a.cap);
    auto at16 = [&](const uint8_t* base, int64_t i) {
        const uint32_t w = reinterpret_cast<const uint16_t*>(base)[i];
        return a.f16 ? widen2<CK_DT_FP16>(w).x : widen2<CK_DT_BF16>(w).x;
    };
    auto place = [&](int64_t j, int64_t& row, int64_t& srow) {
        const int64_t t = j < np ? j : j - np;
        const int32_t* const tab = j < np ? a.ptable + p * a.pt_stride : a.table + b * a.table_stride;
        const int64_t page = tab[t >> a.page_shift], in = t & ((1 << a.page_shift) - 1);
        row = page * a.c_ps + kvh * a.c_hs + in * a.c_ts;
        srow = page * a.s_ps + kvh * a.s_hs + in * a.s_ts;
        return page >= 0 && page < a.pages;
    };
    if (tid == 0) bad = wrong;
    for (int e = tid; e < a.d; e += 256) qs[e] = at16(reinterpret_cast<const uint8_t*>(a.q), b * a.q_bs + h * a.q_hs + e);
    acc[tid] = 0.0f;
    __syncthreads();
    float m = -3.402823466e38f, l = 0.0f;
    for (int64_t j0 = 0; j0 < n && !bad; j0 += 256) {
        float s = -INFINITY;
        int64_t row = 0, srow = 0;
        if (j0 + tid < n) {
            if (place(j0 + tid, row, srow)) {
                s = 0.0f;
                for (int e = 0; e < a.d; ++e) s += qs[e] * (a.i8 ? (float)(int8_t)a.ck[row + e] : at16(a.ck, row + e));
                s *= a.scale * 1.44269504f * (a.i8 ? a.cks[srow] : 1.0f);
            } else {
                bad = 1;
            }
        }
        red[tid] = s;
        __syncthreads();
        float top = m;
        for (int i = 0; i < 256; ++i) top = fmaxf(top, red[i]);
        __syncthreads();
        red[tid] = exp2f(s - top);
        __syncthreads();
        const float f = exp2f(m - top);
        l *= f;
        m = top;
        float o = acc[tid] * f;
        for (int i = 0; i < 256 && j0 + i < n; ++i) {
            l += red[i];
            if (tid < a.d && place(j0 + i, row, srow))
                o += red[i] * (a.i8 ? (float)(int8_t)a.cv[row + tid] * a.cvs[srow] : at16(a.cv, row + tid));
        }
        acc[tid] = o;
        __syncthreads();
    }
    if (tid < a.d) {
        const float v = bad ? NAN : n == 0 ? 0.0f : acc[tid] / l;
        a.out[b * a.o_bs + h * a.o_hs + tid] = (uint16_t)((a.f16 ? narrow2<CK_DT_FP16>(v, 0.0f) : narrow2<CK_DT_BF16>(v, 0.0f)) & 0xffffu);
    }
}

extern "C" int64_t ck_shared_prefix_attention_workspace(int64_t batch, int64_t hq, int64_t hk, int64_t head_dim,
                                                        int64_t prefixes, int64_t prefix_width, int64_t table_width,
                                                        int64_t page_size)
{
    if (batch < 0 || hq < 0 || hk < 1 || hq % hk != 0 || !attention_dim_ok(head_dim) || prefixes < 0 || prefix_width < 0 ||
        table_width < 0 || !is_pow2(page_size) || page_size > 32768 || prefixes > (1 << 20) ||
        batch * hq > 0x7fffffff || !attention_sizes_ok(batch, hq, hk, table_width, page_size) || !attention_sizes_ok(batch, hq, hk, prefix_width, page_size))
        return -1;
    return 0;
}

extern "C" ck_status ck_shared_prefix_attention(const ck_prefix_args* args, const ck_kv_cache* cache, hipStream_t stream)
{
    if (!args || !cache) return fail(CK_ERR_INVALID_ARG, "NULL args or cache");
    const ck_prefix_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.batch < 0 || p.hq < 0 || p.table_width < 0 || p.prefixes < 0 || p.prefix_width < 0)
        return fail(CK_ERR_INVALID_ARG, "negative size");
    if (!attention_dim_ok(cache->head_dim)) return fail(CK_ERR_UNSUPPORTED, "head_dim must be 64, 96, 128, 192 or 256");
    ck_status s = check_cache(cache, p.dtype, cache->head_dim, 16);
    if (s != CK_OK) return s;
    if (p.hq % cache->heads != 0) return fail(CK_ERR_INVALID_ARG, "query heads are not a multiple of the cache's");
    if (p.batch == 0 || p.hq == 0) return ok();
    if (!attention_sizes_ok(p.batch, p.hq, cache->heads, p.table_width, cache->page_size) ||
        !attention_sizes_ok(p.batch, p.hq, cache->heads, p.prefix_width, cache->page_size) || p.prefixes > (1 << 20))
        return fail(CK_ERR_UNSUPPORTED, "too large a batch, table or number of heads or prefixes");
    if (!p.q || !p.out || !p.lens || (!p.table && p.table_width > 0))
        return fail(CK_ERR_INVALID_ARG, "NULL q, out, table or lens");
    if (p.prefixes > 0 && (!p.starts || !p.prefix_lens || (!p.prefix_table && p.prefix_width > 0)))
        return fail(CK_ERR_INVALID_ARG, "NULL starts, prefix_lens or prefix_table");
    if (!rows16(p.q, p.batch, p.q_batch_stride, p.hq, p.q_head_stride) ||
        !rows16(p.out, p.batch, p.out_batch_stride, p.hq, p.out_head_stride))
        return fail(CK_ERR_UNSUPPORTED, "q and out rows must start 16 bytes apart");
    if (!aligned(p.table, 4) || !aligned(p.lens, 4) || !aligned(p.prefix_table, 4) || !aligned(p.prefix_lens, 4) || !aligned(p.starts, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned table, lens or starts");
    if ((p.table_stride < p.table_width && p.batch > 1) || (p.prefix_table_stride < p.prefix_width && p.prefixes > 1))
        return fail(CK_ERR_INVALID_ARG, "table_stride smaller than table_width");
    if (!(p.scale == p.scale)) return fail(CK_ERR_INVALID_ARG, "scale is NaN");
    const bool i8 = cache->dtype == CK_DT_INT8, f16 = p.dtype == CK_DT_FP16;
    const int64_t d = cache->head_dim, row_bytes = d * (i8 ? 1 : 2);
    if (cache_reach(cache, cache->page_stride, cache->head_stride, cache->token_stride, d) * (row_bytes / d) > 0x1p36)
        return fail(CK_ERR_UNSUPPORTED, "the cache spans more than 64 GiB");
    if (!rows_apart(d, {p.batch, p.out_batch_stride}, {p.hq, p.out_head_stride}))
        return fail(CK_ERR_INVALID_ARG, "rows of out overlap");
    if (p.batch * p.hq > 0x7fffffff) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if ((s = check_device()) != CK_OK) return s;
    PrefixArgs a{};
    a.q = (const uint16_t*)p.q; a.out = (uint16_t*)p.out; a.ptable = p.prefix_table; a.plens = p.prefix_lens; a.starts = p.starts;
    a.table = p.table; a.lens = p.lens;
    a.ck = (const uint8_t*)cache->k; a.cv = (const uint8_t*)cache->v; a.cks = cache->k_scale; a.cvs = cache->v_scale;
    a.q_bs = p.q_batch_stride; a.q_hs = p.q_head_stride; a.o_bs = p.out_batch_stride; a.o_hs = p.out_head_stride;
    a.pt_stride = p.prefix_table_stride; a.table_stride = p.table_stride;
    a.c_ps = cache->page_stride; a.c_hs = cache->head_stride; a.c_ts = cache->token_stride;
    a.s_ps = cache->scale_page_stride; a.s_hs = cache->scale_head_stride; a.s_ts = cache->scale_token_stride;
    a.pages = cache->pages; a.pcap = p.prefix_width * cache->page_size; a.cap = p.table_width * cache->page_size;
    a.scale = p.scale; a.batch = (int)p.batch; a.hq = (int)p.hq; a.hk = (int)cache->heads; a.prefixes = (int)p.prefixes;
    a.page_shift = ilog2(cache->page_size); a.d = (int)d; a.i8 = i8; a.f16 = f16;
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&shared_prefix_kernel), (unsigned)(p.batch * p.hq), 256, kargs, stream, "shared_prefix");
    return s == CK_OK ? ok() : s;
}
