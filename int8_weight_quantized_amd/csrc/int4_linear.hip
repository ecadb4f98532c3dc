// int4_linear.hip -- x W^T with 4-bit weights and a scale (and zero point)
// per group of weights along K, for 16-bit x, and the layout of the weights.

struct Int4PackArgs {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    uint32_t* w;
    uint16_t* ws;
    uint8_t* wz;
    int64_t ldc, lds, ldz, n, k, chunks, groups;
};

// One thread per packed word: columns k0 .. k0 + 7 of a row, the even ones in
// the lower half, so that column pairs (2 i, 2 i + 1) sit 16 bits apart.
__global__ __launch_bounds__(256) void int4_pack_kernel(Int4PackArgs a)
{
    const int64_t word = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t tiles = (a.n + 15) / 16;
    if (word < tiles * a.chunks * 256) {
        const int i = word & 3, lane = (int)(word >> 2) & 63;
        const int64_t block = word >> 8, tile = block / a.chunks, chunk = block - tile * a.chunks;
        const int64_t row = tile * 16 + (lane & 15), k0 = chunk * 128 + 32 * i + 8 * (lane >> 4);
        uint32_t v = 0;
        if (row < a.n && k0 < a.k) {         // k % 8 == 0: all eight columns or none
            const uint8_t* p = a.codes + row * a.ldc + k0 / 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t byte = p[j];
                v |= (byte & 15u) << (4 * j) | (byte >> 4) << (16 + 4 * j);
            }
        }
        a.w[word] = v;
    }
    if (word < tiles * a.groups * 16) {
        const int64_t tile = word / (a.groups * 16), g = word / 16 % a.groups, row = tile * 16 + (word & 15);
        a.ws[word] = row < a.n ? a.scales[row * a.lds + g] : 0;
        if (a.wz) a.wz[word] = row < a.n ? a.zeros[row * a.ldz + g] : 0;
    }
}

struct Int4Args {
    const uint16_t* x;
    const uint8_t* w;
    const uint16_t* ws;
    const uint8_t* wz;
    const void* bias;
    void* out;
    int64_t ldx, ldo, m, n, k, chunks, groups;
    int group_shift;
};

// One wave per output column and four rows of x; a lane takes every 64th
// word of eight columns.
template <int DT, int EPI>
__global__ __launch_bounds__(256) void int4_simple_kernel(Int4Args a)
{
    const int lane = threadIdx.x & 63;
    const int64_t col = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t m0 = (int64_t)blockIdx.y * 4;
    if (col >= a.n) return;
    const int64_t tile = col / 16;
    const int r = (int)(col & 15);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a.w) + tile * a.chunks * 256;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t u = lane; u < a.k / 8; u += 64) {
        const int64_t k0 = u * 8, g = k0 >> a.group_shift;
        const uint32_t v = w[(k0 / 128) * 256 + ((k0 / 8 % 4) * 16 + r) * 4 + k0 / 32 % 4];
        const float s = widen2<DT>(a.ws[(tile * a.groups + g) * 16 + r]).x;
        const float z = a.wz ? (float)a.wz[(tile * a.groups + g) * 16 + r] : 8.0f;
        float c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = (float)((v >> (4 * (e / 2) + 16 * (e & 1))) & 15u) - z;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[8], p = 0.0f;
            widen8<DT>(*reinterpret_cast<const v4i*>(a.x + min(m0 + i, a.m - 1) * a.ldx + k0), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) p = __builtin_fmaf(c[e], x[e], p);
            sum[i] = __builtin_fmaf(p, s, sum[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = group_sum<64>(sum[i]);
        if (lane != 0 || m0 + i >= a.m) continue;
        if (a.bias) v = v + bias_at<EPI>(a.bias, col);
        if constexpr (EPI == EPI_F32) reinterpret_cast<float*>(a.out)[(m0 + i) * a.ldo + col] = v;
        else reinterpret_cast<uint16_t*>(a.out)[(m0 + i) * a.ldo + col] = (uint16_t)(pack2<EPI>(v, 0.0f) & 0xffffu);
    }
}

namespace {

ck_status check_int4_sizes(int64_t n, int64_t k, int64_t group)
{
    if (n < 0 || k < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    if (group != 32 && group != 64 && group != 128) return fail(CK_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
    if (k % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "k must be a multiple of 8");
    if (n > (int64_t(1) << 31) - 1 || k > (int64_t(1) << 31) - 1) return fail(CK_ERR_UNSUPPORTED, "n or k too large");
    return CK_OK;
}

}  // namespace

extern "C" ck_status ck_int4_pack(const uint8_t* codes, int64_t ldc, const uint16_t* scales, int64_t lds,
                                  const uint8_t* zeros, int64_t ldz, uint8_t* w, uint16_t* w_scale,
                                  uint8_t* w_zero, int64_t n, int64_t k, int64_t group, hipStream_t stream)
{
    ck_status s = check_int4_sizes(n, k, group);
    if (s != CK_OK) return s;
    if (n == 0 || k == 0) return ok();
    if (!codes || !scales || !w || !w_scale) return fail(CK_ERR_INVALID_ARG, "NULL codes, scales, w or w_scale");
    if (!zeros != !w_zero) return fail(CK_ERR_INVALID_ARG, "zeros and w_zero go together");
    const int64_t groups = cdiv(k, group);
    if (ldc < k / 2 || lds < groups || (zeros && ldz < groups))
        return fail(CK_ERR_INVALID_ARG, "ldc, lds or ldz smaller than a row");
    if (!aligned(scales, 2) || !aligned(w, 16) || !aligned(w_scale, 16) || !aligned(w_zero, 16))
        return fail(CK_ERR_UNSUPPORTED, "misaligned scales, w, w_scale or w_zero");
    Int4PackArgs a{codes, scales, zeros, (uint32_t*)w, w_scale, w_zero, ldc, lds, ldz, n, k, cdiv(k, 128), groups};
    const int64_t blocks = cdiv(n, 16) * a.chunks;           // 256 words a block; 16 scales a group fit
    if (blocks > 0x7fffffffLL) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if ((s = check_device()) != CK_OK) return s;
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&int4_pack_kernel), (unsigned)blocks, 256, kargs, stream, "int4_pack");
    return s == CK_OK ? ok() : s;
}

extern "C" ck_status ck_int4_linear(const void* x, int64_t ldx, ck_dtype dtype, const uint8_t* w,
                                    const uint16_t* w_scale, const uint8_t* w_zero, const void* bias, void* out,
                                    int64_t ldo, ck_out_dtype out_dtype, int64_t m, int64_t n, int64_t k,
                                    int64_t group, hipStream_t stream)
{
    if (dtype != CK_DT_BF16 && dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (out_dtype != CK_OUT_BF16 && out_dtype != CK_OUT_FP16 && out_dtype != CK_OUT_FP32)
        return fail(CK_ERR_INVALID_ARG, "bad out_dtype");
    if (m < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    ck_status s = check_int4_sizes(n, k, group);
    if (s != CK_OK) return s;
    if (m == 0 || n == 0) return ok();
    if (!out) return fail(CK_ERR_INVALID_ARG, "NULL out");
    if (ldo < n) return fail(CK_ERR_INVALID_ARG, "ldo smaller than n");
    if (k > 0) {
        if (!x || !w || !w_scale) return fail(CK_ERR_INVALID_ARG, "NULL x, w or w_scale");
        if (ldx < k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if (ldx % 8 != 0 || !aligned(x, 16))
            return fail(CK_ERR_UNSUPPORTED, "x rows must start 16 bytes apart (ldx %% 8 == 0)");
    }
    const int esz = out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(w, 16) || !aligned(w_scale, 16) || !aligned(w_zero, 16) || !aligned(out, esz) ||
        (bias && !aligned(bias, esz)))
        return fail(CK_ERR_UNSUPPORTED, "misaligned w, w_scale, w_zero, bias or out");
    const int64_t bx = cdiv(n, 4), by = cdiv(m, 4);
    if (by > 65535) return fail(CK_ERR_UNSUPPORTED, "too many rows");
    if ((s = check_device()) != CK_OK) return s;
    Int4Args a{(const uint16_t*)x, w, w_scale, w_zero, bias, out, ldx, ldo, m, n, k, cdiv(k, 128), cdiv(k, group),
               ilog2(group)};
#define CK_INT4_SIMPLE(D)                                                                             \
    (out_dtype == CK_OUT_FP32   ? reinterpret_cast<const void*>(&int4_simple_kernel<D, EPI_F32>)      \
     : out_dtype == CK_OUT_FP16 ? reinterpret_cast<const void*>(&int4_simple_kernel<D, EPI_F16>)      \
                                : reinterpret_cast<const void*>(&int4_simple_kernel<D, EPI_BF16>))
    const void* fn = dtype == CK_DT_FP16 ? CK_INT4_SIMPLE(CK_DT_FP16) : CK_INT4_SIMPLE(CK_DT_BF16);
#undef CK_INT4_SIMPLE
    void* kargs[] = {&a};
    hipError_t e = hipLaunchKernel(fn, dim3((unsigned)bx, (unsigned)by), dim3(256), kargs, 0, stream);
    if (e != hipSuccess) return fail(CK_ERR_HIP, "int4_linear launch: %s", hipGetErrorString(e));
    return ok();
}
