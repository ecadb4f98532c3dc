// lora_add.hip -- y + s (x A^T) B^T with a low-rank adapter for every row.

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int32_t* ids;
    const void* y;
    void* out;
    int64_t ldx, ldy, ldo, a_stride, b_stride, m, n, k, rank, adapters;
    int dtype, out_dtype;
};

__global__ __launch_bounds__(256) void lora_kernel(LoraArgs a)
{
    __shared__ float v[256], red[256];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int id = a.ids[row];
    const bool has = id >= 0 && id < a.adapters;
    auto at = [&](const uint16_t* p, int64_t i) {
        return a.dtype == CK_DT_FP16 ? widen2<CK_DT_FP16>(p[i]).x : widen2<CK_DT_BF16>(p[i]).x;
    };
    for (int r = 0; r < a.rank && has; ++r) {
        float s = 0.0f;
        for (int64_t i = tid; i < a.k; i += 256) s += at(a.x, row * a.ldx + i) * at(a.a, id * a.a_stride + r * a.k + i);
        red[tid] = s;
        __syncthreads();
        for (int off = 128; off > 0; off >>= 1) {
            if (tid < off) red[tid] += red[tid + off];
            __syncthreads();
        }
        if (tid == 0) v[r] = red[0];
        __syncthreads();
    }
    for (int64_t c = tid; c < a.n; c += 256) {
        float s = 0.0f;
        for (int r = 0; r < a.rank && has; ++r) s += v[r] * at(a.b, id * a.b_stride + c * a.rank + r);
        if (has && a.scale) s *= a.scale[id];
        const int64_t yi = row * a.ldy + c, oi = row * a.ldo + c;
        if (a.out_dtype == CK_OUT_FP32) {
            const float y = static_cast<const float*>(a.y)[yi];
            static_cast<float*>(a.out)[oi] = has ? y + s : y;
        } else {
            const uint32_t w = static_cast<const uint16_t*>(a.y)[yi];
            const float y = a.out_dtype == CK_OUT_FP16 ? widen2<CK_DT_FP16>(w).x : widen2<CK_DT_BF16>(w).x;
            const uint32_t o = a.out_dtype == CK_OUT_FP16 ? narrow2<CK_DT_FP16>(y + s, 0.0f) : narrow2<CK_DT_BF16>(y + s, 0.0f);
            static_cast<uint16_t*>(a.out)[oi] = (uint16_t)(has ? o & 0xffffu : w);
        }
    }
}

namespace {

bool lora_sizes_ok(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return m >= 0 && n >= 0 && k >= 0 && m <= (1 << 24) && n <= (1 << 24) && k <= (1 << 24) && k % 8 == 0 && rank >= 8 &&
           rank <= 256 && rank % 8 == 0;
}

}  // namespace

extern "C" int64_t ck_lora_add_workspace(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return lora_sizes_ok(m, n, k, rank) ? 0 : -1;
}

extern "C" ck_status ck_lora_add(const ck_lora_args* args, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_lora_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.out_dtype != CK_OUT_BF16 && p.out_dtype != CK_OUT_FP16 && p.out_dtype != CK_OUT_FP32)
        return fail(CK_ERR_INVALID_ARG, "bad out_dtype");
    if (p.m < 0 || p.n < 0 || p.k < 0 || p.rank < 0 || p.adapters < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    if (p.rank < 8 || p.rank > 256 || p.rank % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "rank must be a multiple of 8 from 8 to 256");
    if (p.k % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "k must be a multiple of 8");
    if (!lora_sizes_ok(p.m, p.n, p.k, p.rank) || p.adapters > (1 << 24)) return fail(CK_ERR_UNSUPPORTED, "m, n, k or adapters past 2^24");
    if (p.m == 0 || p.n == 0) return ok();
    if (!p.y || !p.out || !p.ids) return fail(CK_ERR_INVALID_ARG, "NULL y, out or ids");
    if (p.m > 1 && (p.ldy < p.n || p.ldo < p.n)) return fail(CK_ERR_INVALID_ARG, "ldy or ldo smaller than n");
    if (p.adapters > 0) {
        if (!p.b || (p.k > 0 && (!p.x || !p.a))) return fail(CK_ERR_INVALID_ARG, "NULL x, a or b");
        if (p.k > 0 && p.m > 1 && p.ldx < p.k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if (p.adapters > 1 && (p.a_stride < p.rank * p.k || p.b_stride < p.rank * p.n))
            return fail(CK_ERR_INVALID_ARG, "a_stride or b_stride smaller than an adapter");
        if ((p.k > 0 && p.m > 1 && p.ldx % 8 != 0) || (p.adapters > 1 && (p.a_stride % 8 != 0 || p.b_stride % 8 != 0)) ||
            !aligned(p.x, 16) || !aligned(p.a, 16) || !aligned(p.b, 16))
            return fail(CK_ERR_UNSUPPORTED, "rows of x and adapters must start 16 bytes apart");
    }
    const int esz = p.out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(p.y, esz) || !aligned(p.out, esz) || !aligned(p.ids, 4) || !aligned(p.scale, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned y, out, ids or scale");
    ck_status s = check_device();
    if (s != CK_OK) return s;
    LoraArgs a{(const uint16_t*)p.x, (const uint16_t*)p.a, (const uint16_t*)p.b, p.scale, p.ids, p.y, p.out, p.ldx, p.ldy, p.ldo,
               p.a_stride, p.b_stride, p.m, p.n, p.k, p.rank, p.adapters, p.dtype, p.out_dtype};
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&lora_kernel), (unsigned)p.m, 256, kargs, stream, "lora_add");
    return s == CK_OK ? ok() : s;
}
