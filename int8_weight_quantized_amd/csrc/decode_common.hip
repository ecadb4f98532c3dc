// decode_common.hip -- what the decode-step operators share: 16-bit element
// types and the checks of a paged cache.

// Two 16-bit values of a word to fp32 (exact), `lo` in bits 0..15.
template <int DT>
__device__ __forceinline__ float2 widen2(uint32_t w)
{
    if constexpr (DT == CK_DT_FP16) {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        return make_float2((float)h[0], (float)h[1]);
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

// Two fp32 values to a word of 16-bit ones, each rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    return pack2<DT == CK_DT_FP16 ? EPI_F16 : EPI_BF16>(lo, hi);
}

// The quiet NaN of a 16-bit type, twice.
template <int DT>
constexpr uint32_t kNan2 = DT == CK_DT_FP16 ? 0x7e007e00u : 0x7fc07fc0u;

namespace {

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

int ilog2(int64_t v)
{
    int l = 0;
    while ((int64_t(1) << (l + 1)) <= v) ++l;
    return l;
}

// Whether a launch takes so many blocks: fewer than 2^32 threads in all.
bool grid_ok(int64_t blocks, int64_t threads) { return blocks <= 0xffffffffLL / threads; }

// 16-bit rows of a [tokens, heads, head_dim] tensor that start 16 bytes apart
// (the stride of a dimension with one element is not looked at).
bool rows16(const void* p, int64_t tokens, int64_t ts, int64_t heads, int64_t hs)
{
    return aligned(p, 16) && (tokens <= 1 || ts % 8 == 0) && (heads <= 1 || hs % 8 == 0);
}

struct Dim {
    int64_t count, stride;
};

// Whether the rows (`row` elements) of a tensor of these dimensions lie apart,
// in any order of the dimensions.
bool rows_apart(int64_t row, Dim a, Dim b, Dim c = {1, 0})
{
    if (a.stride > b.stride) std::swap(a, b);
    if (b.stride > c.stride) std::swap(b, c);
    if (a.stride > b.stride) std::swap(a, b);
    double span = (double)row;                               // of the dimensions so far
    for (const Dim& d : {a, b, c}) {
        if (d.count <= 1) continue;
        if ((double)d.stride < span) return false;
        span += (double)(d.count - 1) * (double)d.stride;
    }
    return true;
}

// How far a [pages, heads, page_size] tensor reaches, in elements past its
// start (as a double: the products may pass 64 bits); negative if a stride
// that counts is.  The stride of a dimension with one element does not.
double cache_reach(const ck_kv_cache* c, int64_t ps, int64_t hs, int64_t ts, int64_t row)
{
    const int64_t n[3] = {c->pages, c->heads, c->page_size}, stride[3] = {ps, hs, ts};
    double reach = (double)row;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (stride[i] < 0) return -1.0;
        reach += (double)(n[i] - 1) * (double)stride[i];
    }
    return reach;
}

// A paged cache for activations of type dtype; `align` bytes between rows.
ck_status check_cache(const ck_kv_cache* c, int dtype, int64_t head_dim, int align)
{
    if (c->dtype != CK_DT_INT8 && c->dtype != dtype)
        return fail(CK_ERR_INVALID_ARG, "the cache is neither int8 nor of the activations' type");
    if (c->pages < 0 || c->heads < 1) return fail(CK_ERR_INVALID_ARG, "bad cache sizes");
    if (!is_pow2(c->page_size) || c->page_size > 32768)
        return fail(CK_ERR_INVALID_ARG, "page_size must be a power of two up to 32768");
    if (c->pages > (int64_t(1) << 31) - 1) return fail(CK_ERR_UNSUPPORTED, "too many pages");
    if (c->head_dim != head_dim) return fail(CK_ERR_INVALID_ARG, "cache and heads disagree on head_dim");
    if (c->pages > 0 && (!c->k || !c->v)) return fail(CK_ERR_INVALID_ARG, "NULL cache");
    const double reach = cache_reach(c, c->page_stride, c->head_stride, c->token_stride, head_dim);
    const double scale_reach = c->dtype == CK_DT_INT8
        ? cache_reach(c, c->scale_page_stride, c->scale_head_stride, c->scale_token_stride, 1) : 0.0;
    if (reach < 0.0 || scale_reach < 0.0) return fail(CK_ERR_INVALID_ARG, "negative cache stride");
    if (reach > 0x1p60 || scale_reach > 0x1p60) return fail(CK_ERR_UNSUPPORTED, "cache strides too large");
    if (c->page_size > 1 && c->token_stride < head_dim)
        return fail(CK_ERR_INVALID_ARG, "token_stride smaller than head_dim");
    const int esz = c->dtype == CK_DT_INT8 ? 1 : 2;
    if (!aligned(c->k, align) || !aligned(c->v, align) || (c->pages > 1 && c->page_stride * esz % align != 0) ||
        (c->heads > 1 && c->head_stride * esz % align != 0) || (c->page_size > 1 && c->token_stride * esz % align != 0))
        return fail(CK_ERR_UNSUPPORTED, "cache rows must start %d bytes apart", align);
    if (c->dtype == CK_DT_INT8) {
        if (c->pages > 0 && (!c->k_scale || !c->v_scale))
            return fail(CK_ERR_INVALID_ARG, "an int8 cache needs k_scale and v_scale");
        if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
            return fail(CK_ERR_UNSUPPORTED, "misaligned cache scales");
    }
    return CK_OK;
}

}  // namespace
